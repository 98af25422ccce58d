"""Serving plans: which short runs get a 128-row tile of their own."""
import os

import pytest

import int8_mixed_precision_gb300 as dit


@pytest.fixture(scope="module", autouse=True)
def built():
    from int8_mixed_precision_gb300 import _lib, build
    if not os.path.exists(_lib.library_path()):
        try:
            build.build_library()
        except RuntimeError as e:          # no nvcc on this machine
            pytest.skip(str(e))


def plan(large, shorts):
    return dit.AdapterPlan([128 * large] + [1] * shorts, [0] + [1 + i % 2 for i in range(shorts)], 3, device="cpu")


def test_few_short_runs_beside_large_ones_get_tiles_of_their_own():
    for large, shorts in ((16, 4), (64, 16), (276, 24)):
        p = plan(large, shorts)
        assert (p.n_tiles, p.n_small) == (large + shorts, 0)


def test_many_short_runs_share_small_tiles():
    """A tile of its own costs a short run 128 rows of x and y; beyond some two dozen of them that is more than the
    launch that they save, however many large tiles there are."""
    for large, shorts in ((16, 5), (276, 25), (276, 69), (2000, 400)):
        p = plan(large, shorts)
        assert p.n_tiles == large and p.n_small == -(-(-(-shorts // 2)) // 16) + -(-(shorts // 2) // 16)
