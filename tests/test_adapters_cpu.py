"""What the adapters and the optimiser do on the host: the plan's table, the chunk table, buffer sizes, and every
refusal that comes before a launch."""
import ctypes
import os
import random

import pytest
import torch

import int8_mixed_precision_gb300 as dit
from adapter_reference import spans


@pytest.fixture(scope="module", autouse=True)
def L():
    from int8_mixed_precision_gb300 import _lib, build
    if not os.path.exists(_lib.library_path()):
        try:
            build.build_library()
        except RuntimeError as e:          # no nvcc on this machine
            pytest.skip(str(e))
    return _lib.lib()


def rows_of(plan, G):
    """{row: adapter} of the plan's tiles, and the sizes of both kinds."""
    t = plan.table.tolist()
    seen, big, small = {}, [], []
    for i in range(plan.n_tiles):
        row0, rows, g, _ = t[4 * i:4 * i + 4]
        big.append((g, rows))
        for r in range(row0, row0 + rows):
            assert r not in seen
            seen[r] = g
    first = t[4 * plan.n_tiles:4 * plan.n_tiles + G + 1]
    at = (4 * plan.n_tiles + G + 1 + 3) // 4 * 4
    for i in range(plan.n_small):
        e = t[at + 20 * i:at + 20 * i + 20]
        small.append((e[0], e[1]))
        for r in e[4:4 + e[1]]:
            assert r not in seen
            seen[r] = e[0]
    return seen, big, small, first


@pytest.mark.parametrize("training", [False, True])
@pytest.mark.parametrize("seed", range(20))
def test_the_tiles_of_a_plan_cover_its_rows(seed, training):
    rng = random.Random(seed)
    G = rng.choice([1, 3, 20])
    lengths = [rng.choice([0, 1, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300, 1000]) for _ in range(rng.choice([0, 1, 7, 60]))]
    adapters = [rng.randrange(-1, G) for _ in lengths]
    plan = dit.AdapterPlan(lengths, adapters, G, training=training, device="cpu")
    seen, big, small, first = rows_of(plan, G)
    assert seen == {r: g for rows, g in spans(lengths, adapters) for r in range(rows.start, rows.stop)}
    assert plan.rows == sum(lengths)
    # the big tiles lie in the adapters' order, and `first` says where each adapter's begin
    assert [g for g, _ in big] == sorted(g for g, _ in big)
    assert first == [sum(1 for g, _ in big if g < a) for a in range(G + 1)]
    assert plan.info.most_tiles == max([sum(1 for g, _ in big if g == a) for a in range(G)])
    assert all(1 <= n <= 128 for _, n in big) and all(1 <= n <= 16 for _, n in small)
    if training:
        assert not small
    # no adapter has two small tiles that are not full
    for a in range(G):
        assert sum(1 for g, n in small if g == a and n < 16) <= 1


def test_single_tokens_of_one_adapter_share_tiles():
    plan = dit.AdapterPlan([1] * 64, [i % 3 for i in range(64)], 3, device="cpu")
    assert plan.n_tiles == 0 and plan.n_small == 6          # 22, 21 and 21 rows


def test_adjacent_requests_of_one_adapter_are_one_run():
    assert dit.AdapterPlan([20, 0, 20], [0, 1, 0], 2, device="cpu").n_tiles == 1
    assert dit.AdapterPlan([20, 1, 20], [0, -1, 0], 2, device="cpu").n_tiles == 0


def test_plan_refusals(L):
    for lengths, adapters, G in (([1], [1], 1), ([1], [-2], 1), ([-1], [0], 1), ([1, 2], [0], 1), ([2 ** 31], [0], 1),
                                 ([2 ** 31 - 256] * 2, [0, 0], 1), ([1], [0], 0), ([1], [2 ** 40], 1)):
        with pytest.raises(dit.DitError):
            dit.AdapterPlan(lengths, adapters, G, device="cpu")
    with pytest.raises(dit.DitError, match="UNSUPPORTED"):
        dit.AdapterPlan([1], [0], 2 ** 21, device="cpu")
    # a table too small for the plan, and no plan at all
    from int8_mixed_precision_gb300.adapters import _Plan
    info = _Plan()
    ln, ad = (ctypes.c_int64 * 1)(300), (ctypes.c_int32 * 1)(0)
    table = (ctypes.c_int32 * 4)()
    assert L.dit_adapter_plan(ln, ad, 1, 1, 0, ctypes.byref(info), table, 4) == 1
    assert L.dit_adapter_plan(ln, ad, 1, 1, 0, None, None, 0) == 1
    assert L.dit_adapter_plan(None, ad, 1, 1, 0, ctypes.byref(info), None, 0) == 1


def parts(T=40, G=2, r=16, K=64, N=72, training=True, y=torch.bfloat16):
    bf = torch.bfloat16
    bank = dit.AdapterBank(torch.zeros(G, r, K, dtype=bf), torch.zeros(G, N, r, dtype=bf), torch.ones(G))
    plan = dit.AdapterPlan([T], [0], G, training=training, device="cpu")
    return plan, bank, torch.zeros(T, K, dtype=bf), torch.zeros(T, N, dtype=y)


def test_bank_refusals():
    bf = torch.bfloat16
    ok = dict(a=torch.zeros(2, 16, 64, dtype=bf), b=torch.zeros(2, 72, 16, dtype=bf), scale=torch.ones(2))
    for change in (dict(a=torch.zeros(2, 12, 64, dtype=bf), b=torch.zeros(2, 72, 12, dtype=bf)),       # rank not a multiple of 8
                   dict(a=torch.zeros(2, 136, 64, dtype=bf), b=torch.zeros(2, 72, 136, dtype=bf)),     # rank above 128
                   dict(a=torch.zeros(2, 16, 60, dtype=bf)), dict(b=torch.zeros(2, 70, 16, dtype=bf)),
                   dict(a=torch.zeros(2, 16, 64)), dict(scale=torch.ones(3)), dict(scale=torch.ones(2, dtype=bf)),
                   dict(a=torch.zeros(3, 16, 64, dtype=bf)), dict(b=torch.zeros(2, 72, 8, dtype=bf)),
                   dict(a=torch.zeros(2, 64, 16, dtype=bf).transpose(1, 2))):
        with pytest.raises(dit.DitError):
            dit.AdapterBank(**{**ok, **change})


def test_call_refusals():
    plan, bank, x, y = parts()
    ws = torch.zeros(dit.workspace_bytes(), dtype=torch.uint8)
    scratch, saved = dit.adapter_scratch(plan, bank), dit.adapter_saved(plan, bank)
    with pytest.raises(dit.DitError, match="CUDA"):
        dit.lora_forward(plan, bank, x, y, scratch, ws)
    for bad in (x[:39], x[:, :56], x.float(), x.reshape(-1)):
        with pytest.raises(dit.DitError, match="x:"):
            dit.lora_forward(plan, bank, bad, y, scratch, ws)
    other = dit.AdapterPlan([40], [0], 3, device="cpu")
    with pytest.raises(dit.DitError, match="3 adapters"):
        dit.lora_forward(other, bank, x, y, scratch, ws)
    serving = dit.AdapterPlan([40], [0], 2, device="cpu")
    with pytest.raises(dit.DitError, match="training"):
        dit.lora_backward(serving, bank, x, y, saved, torch.zeros(2, 16, 64), torch.zeros(2, 72, 16), scratch, ws)


def test_c_refusals_before_any_launch(L):
    plan, bank, x, y = parts()
    ws, p, odd = ctypes.c_void_p(0x2000), ctypes.c_void_p(0x4000), ctypes.c_void_p(0x4008)
    wsb, big = dit.workspace_bytes(), 1 << 40

    def fwd(info=plan._info_p, table=p, x=p, a=p, b=p, s=p, r=16, k=64, n=72, y=p, dt=1, saved=ctypes.c_void_p(0x6000), vb=big,
            scratch=ctypes.c_void_p(0x8000), sb=big, w=ws, wb=wsb):
        return L.dit_lora_forward(info, table, x, a, b, s, r, k, n, y, dt, saved, vb, scratch, sb, w, wb, None)
    for kw in (dict(info=None), dict(table=None), dict(x=None), dict(a=None), dict(b=None), dict(s=None), dict(y=None), dict(k=0), dict(n=-8),
               dict(r=0), dict(dt=2), dict(sb=16), dict(vb=16), dict(wb=100), dict(w=None), dict(saved=ctypes.c_void_p(0x8000))):
        assert fwd(**kw) == 1, kw
    for kw in (dict(r=12), dict(r=136), dict(k=60), dict(n=70)):
        assert fwd(**kw) == 3, kw
    for kw in (dict(x=odd), dict(a=odd), dict(b=odd), dict(y=odd), dict(table=odd), dict(s=ctypes.c_void_p(0x4002)), dict(saved=odd), dict(scratch=odd)):
        assert fwd(**kw) == 2, kw

    def bwd(info=plan._info_p, dy=p, saved=ctypes.c_void_p(0x6000), vb=big, dx=p, dt=1, da=p, db=p):
        return L.dit_lora_backward(info, p, p, dy, p, p, p, 16, 64, 72, saved, vb, dx, dt, da, db, ctypes.c_void_p(0x8000), big, ws, wsb, None)
    for kw in (dict(dy=None), dict(saved=None), dict(vb=16), dict(da=None), dict(db=None), dict(dt=2), dict(saved=ctypes.c_void_p(0x8000)),
               dict(info=dit.AdapterPlan([40], [0], 2, device="cpu")._info_p)):
        assert bwd(**kw) == 1, kw
    for kw in (dict(dy=odd), dict(dx=odd), dict(da=odd), dict(db=odd), dict(saved=odd)):
        assert bwd(**kw) == 2, kw
    # a plan that no call of dit_adapter_plan made
    broken = type(plan.info).from_buffer_copy(plan.info)
    broken.n_tiles = -1
    assert fwd(info=ctypes.addressof(broken)) == 1


def test_chunks(L):
    sizes = [0, 1, 4096, 4097, 10000]
    s = (ctypes.c_int64 * 5)(*sizes)
    n = L.dit_adamw_chunks(s, 5, None, 0)
    assert n == 0 + 1 + 1 + 2 + 3
    t = (ctypes.c_int32 * (2 * n))()
    assert L.dit_adamw_chunks(s, 5, t, n) == n
    assert list(zip(t[::2], t[1::2])) == [(1, 0), (2, 0), (3, 0), (3, 1), (4, 0), (4, 1), (4, 2)]
    assert L.dit_adamw_chunks(s, 5, t, n - 1) == -1
    assert L.dit_adamw_chunks((ctypes.c_int64 * 1)(-1), 1, None, 0) == -1


def test_adamw_refusals(L):
    t = torch.zeros
    p, g = [t(300)], [t(300)]
    with pytest.raises(dit.DitError, match="CUDA"):
        dit.AdamW(p, g, **dit.adamw_moments(p))
    with pytest.raises(dit.DitError, match="8 or 32"):
        dit.adamw_moments(p, 16)
    m8 = dit.adamw_moments(p, 8)
    assert m8["m"][0].dtype == torch.float8_e4m3fn and m8["m_scale"][0].numel() == 2
    for bad in (dict(grads=[]), dict(grads=[t(299)]), dict(grads=[t(300, dtype=torch.float16)]), dict(m=[t(300, dtype=torch.bfloat16)]),
                dict(m_scale=[t(2)]), dict(copies=[t(300)]), dict(m_values=[t(300, dtype=torch.bfloat16)]), dict(params=[])):
        with pytest.raises(dit.DitError):
            dit.AdamW(**{**dict(params=p, grads=g, m=[t(300)], v=[t(300)]), **bad})
    with pytest.raises(dit.DitError, match="m_scale"):
        dit.AdamW(p, g, m8["m"], m8["v"])
    # the C entry
    from int8_mixed_precision_gb300.optim import _Args
    ws, q, wsb = ctypes.c_void_p(0x2000), ctypes.c_void_p(0x4000), dit.workspace_bytes()

    def step(args=(1e-3, 0.9, 0.999, 1e-8, 0.01, 1), d=q, c=q, n=1, nc=1, pd=0, gd=0, bits=32, gs=None, wb=wsb):
        a = ctypes.byref(_Args(*args)) if args else None
        return L.dit_adamw_step(d, n, c, nc, pd, gd, bits, a, gs, ws, wb, None)
    for kw in (dict(args=None), dict(args=(1e-3, 0.9, 0.999, 1e-8, 0.01, 0)), dict(args=(1e-3, 1.0, 0.999, 1e-8, 0.01, 1)),
               dict(args=(float("nan"), 0.9, 0.999, 1e-8, 0.01, 1)), dict(args=(1e-3, 0.9, -0.1, 1e-8, 0.01, 1)),
               dict(args=(1e-3, 0.9, 0.999, -1.0, 0.01, 1)), dict(d=None), dict(c=None), dict(n=-1), dict(n=0), dict(pd=2), dict(gd=3),
               dict(bits=16), dict(wb=8)):
        assert step(**kw) == 1, kw
    for kw in (dict(d=ctypes.c_void_p(0x4008)), dict(c=ctypes.c_void_p(0x4004)), dict(gs=ctypes.c_void_p(0x4002))):
        assert step(**kw) == 2, kw
    assert step(nc=0) == 0                                   # nothing to do
    assert L.dit_adamw_moments(q, 1, q, 0, ws, wsb, None) == 0 and L.dit_adamw_moments(None, 1, q, 1, ws, wsb, None) == 1
