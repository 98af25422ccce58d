"""Copies of a bank read their own tensors; what holds addresses of its own cannot be copied by accident."""
import copy
import os
import pickle

import pytest
import torch

import int8_mixed_precision_gb300 as dit


@pytest.fixture(scope="module", autouse=True)
def built():
    from int8_mixed_precision_gb300 import _lib, build
    if not os.path.exists(_lib.library_path()):
        try:
            build.build_library()
        except RuntimeError as e:          # no nvcc on this machine
            pytest.skip(str(e))


def test_a_copied_bank_reads_its_own_tensors():
    bank = dit.AdapterBank(torch.ones(2, 16, 64, dtype=torch.bfloat16), torch.ones(2, 72, 16, dtype=torch.bfloat16), torch.ones(2))
    for other in (copy.deepcopy(bank), pickle.loads(pickle.dumps(bank))):
        at = [t.data_ptr() for t in (other.a, other.b, other.scale)]
        assert [f() for f in other._pointers] == at == list(other._at)
        assert not set(at) & set(bank._at)
        assert (other.rank, other.k, other.n, other.n_adapters) == (16, 64, 72, 2)
    same = copy.copy(bank)
    assert same._at == bank._at and same.a is bank.a


def test_a_plan_is_not_copied():
    plan = dit.AdapterPlan([3, 200], [0, 1], 2, device="cpu")
    for how in (copy.copy, copy.deepcopy, pickle.dumps):
        with pytest.raises(dit.DitError, match="plan"):
            how(plan)
