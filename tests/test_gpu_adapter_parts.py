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


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), 3.0e38])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("training", [False, True])
def test_infinities_in_the_factors_reach_what_the_formulas_say(training, dtype, value):
    """An infinity or NaN in B (one row of it) makes that column of y infinite or NaN for the rows of the adapter, one in
    A (one element) every column of theirs; every other element has the bits of a clean call.  With parts of h, an
    infinity may come out as NaN.  A finite factor of any size changes nothing of this."""
    g = torch.Generator().manual_seed(3)
    G, r, k, n, lengths, adapters = 2, 24, 136, 264, [5, 140, 9], [0, 1, 0]
    x, a, b = torch.randn(154, k, generator=g), torch.randn(G, r, k, generator=g) * 0.1, torch.randn(G, n, r, generator=g) * 0.1
    out = []
    for where in (None, "b", "a"):
        a1, b1 = a.clone(), b.clone()
        if where == "b":
            b1[0, 77, 3] = value
        if where == "a":
            a1[0, 3, 50] = value
        bank = dit.AdapterBank(a1.bfloat16().cuda(), b1.bfloat16().cuda(), torch.ones(G, device="cuda"))
        plan, ws = dit.AdapterPlan(lengths, adapters, G, training=training), dit.workspace()
        y = torch.ones(154, n, dtype=dtype, device="cuda")
        dit.lora_forward(plan, bank, x.bfloat16().cuda(), y, dit.adapter_scratch(plan, bank), ws)
        out.append(y.cpu())
        assert dit.device_status(ws) == 0
    clean, in_b, in_a = out
    mine = torch.ones(154, dtype=torch.bool)
    mine[5:145] = False
    assert torch.equal(in_b[~mine], clean[~mine]) and torch.equal(in_a[~mine], clean[~mine])
    others = torch.arange(n) != 77
    assert torch.equal(in_b[mine][:, others], clean[mine][:, others])
    if value != 3.0e38:
        assert not torch.isfinite(in_b[mine][:, 77]).any() and not torch.isfinite(in_a[mine]).any()
        assert torch.isfinite(clean).all()
