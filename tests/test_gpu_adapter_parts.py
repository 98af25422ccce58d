"""fp32 outputs and gradients are computed from three parts of h and e: what test_adapter_parts_cpu.py shows two parts to
miss, on every kernel that makes them and every cut of its work."""
import pytest
import torch

import adapter_parts as P

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import int8_mixed_precision_gb300 as dit  # noqa: E402

CUTS = [None, "1,0,1", "2,0,1", "2,9,2", "1,9,2"]


@pytest.mark.parametrize("cut", CUTS)
@pytest.mark.parametrize("training", [False, True])
@pytest.mark.parametrize("rank", [8, 24, 64, 128])
def test_three_parts(rank, training, cut, monkeypatch):
    if not training and cut:
        pytest.skip("short requests are not cut")
    c = P.case(T=12, rank=rank, k=136, n=264, seed=rank)
    want = P.results(c)
    d = {n: v.cuda() for n, v in c.items() if torch.is_tensor(v)}
    plan, bank = dit.AdapterPlan(c["lengths"], c["adapters"], 12, training=training), dit.AdapterBank(d["a"], d["b"], d["scale"])
    assert (plan.n_tiles == 0) != training
    scratch, ws = dit.adapter_scratch(plan, bank), dit.workspace()
    saved = dit.adapter_saved(plan, bank) if training else None
    if cut:
        monkeypatch.setenv("DIT6_TEST_CUT", cut)
    dit.lora_forward(plan, bank, d["x"], d["y"], scratch, ws, saved=saved)
    got = {"y": d["y"]}
    if training:
        got.update(dx=d["dx"], da=torch.empty_like(d["a"], dtype=torch.float32), db=torch.empty_like(d["b"], dtype=torch.float32))
        dit.lora_backward(plan, bank, d["x"], d["dy"], saved, got["da"], got["db"], scratch, ws, dx=got["dx"])
    for name, v in got.items():
        assert P.worst(v, want[name])[0] <= P.BOUND, (name, P.worst(v, want[name])[0])
    assert dit.device_status(ws) == 0
