"""Norms of query and key heads with the position rotation, and their gradients, against the formulas in 64 bits."""
import pytest
import torch

import attention_reference as R

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def dit():
    import int8_mixed_precision_gb300 as d
    return d


def case(tokens, heads, kv_heads, dim, dims, kind, interleaved, seed=0, scale=None, far=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x = (new(tokens, heads + 2 * kv_heads, dim) * 1.5 + 0.2).to(BF16)
    positions = torch.randint(-5, 200, (tokens, max(len(dims), 1)), device="cuda", generator=g, dtype=torch.int32) + far
    params = None if kind is None else 1.0 + 0.3 * new(4 if kind == "layer" else 2, dim)
    return x, positions, params, [1.0] * len(dims) if scale is None else scale, new


def parts(params, kind, side):
    if kind is None:
        return 1.0, 0.0
    p = params.double()
    return (p[2 * side], p[2 * side + 1]) if kind == "layer" else (p[side], 0.0)


CASES = [
    (1, 30, 30, 64, (16, 24, 24), "layer", True),
    (37, 30, 30, 64, (16, 24, 24), "layer", True),
    (300, 3, 1, 128, (32, 48, 48), "rms", False),
    (5, 1, 1, 8, (8,), "rms", True),
    (129, 7, 7, 40, (8, 16, 16), "layer", False),
    (64, 2, 5, 72, (24, 24, 24), "rms", True),
    (33, 4, 2, 96, (32, 32), "layer", False),
    (10, 65, 3, 256, (64, 64, 64, 64), "rms", False),
    (77, 6, 6, 64, (16, 22, 22), None, True),       # a rotation of some dimensions, no norm
    (77, 6, 6, 64, (16, 8, 8), "layer", False),
    (50, 4, 4, 64, (), "layer", True),              # a norm alone
    (1000, 1, 1, 16, (2,), "rms", True),
]


def run_case(dit, tokens, heads, kv_heads, dim, dims, kind, interleaved, backward, in_place=False, **more):
    x, positions, params, scale, new = case(tokens, heads, kv_heads, dim, dims, kind, interleaved, **more)
    rot = dit.Rotary(dims, dim, scale=scale, interleaved=interleaved) if dims else None
    norm = dit.QKNorm(params, kind, 1e-6) if kind else None
    pos = positions if dims else None
    q, k = x[:, :heads], x[:, heads:heads + kv_heads]
    q0, k0 = q.double(), k.double()
    out = x if in_place else torch.full((tokens, heads + kv_heads, dim), 7.0, dtype=BF16, device="cuda")
    values = x[:, heads + kv_heads:].clone()
    dit.qk_norm_rope(q, k, out[:, :heads], out[:, heads:heads + kv_heads], norm, rot, pos)
    assert torch.equal(x[:, heads + kv_heads:], values)
    angle = R.angles(positions, dims, 10000.0, scale) if dims else torch.zeros(tokens, 0, dtype=torch.float64, device="cuda")
    pairs = angle.shape[1]
    if backward:
        dy = new(tokens, heads + kv_heads, dim).to(BF16)
        dx = dy.clone() if in_place else torch.full_like(dy, 9.0)
        src = dx if in_place else dy
        dparams = torch.full_like(params, 5.0) if kind else None
        ws, scratch = dit.workspace(), dit.qk_norm_scratch(dim)
        xs = (q0.to(BF16), k0.to(BF16))
        dit.qk_norm_rope_backward(*xs, src[:, :heads], src[:, heads:], dx[:, :heads], dx[:, heads:], norm, rot, pos, dparams, scratch, ws)
        assert dit.device_status(ws) == 0
    for side, (v, at) in enumerate(((q0, slice(0, heads)), (k0, slice(heads, heads + kv_heads)))):
        w, b = parts(params, kind, side)
        hat, r, n = R.normalise(v, kind, w, b, 1e-6)
        want = R.turn(n, angle, interleaved)
        # half a step of the result; sines, cosines and the norm in fp32, on the pair's magnitudes and on the largest of x
        big = v.abs().amax(-1, keepdim=True) * r * (w.abs() if kind else 1.0)
        bound = R.HALF * want.abs() + R.FINE * (R.pair_sum(n, pairs, interleaved) + R.pair_sum(big + 0 * n, pairs, interleaved)) + 1e-30
        got = out[:, at].double()
        assert ((got - want).abs() <= bound).all(), (side, float(((got - want).abs() / bound).max()))
        if not backward:
            continue
        d = R.turn(dy[:, at].double(), -angle, interleaved)
        gw = d * w
        m1 = gw.mean(-1, keepdim=True) if kind == "layer" else 0.0
        m2 = (gw * hat).mean(-1, keepdim=True) if kind else 0.0
        want = (gw - m1 - hat * m2) * r
        mag = R.pair_sum(dy[:, at].double(), pairs, interleaved) * (w.abs() if kind else 1.0)
        top = mag.amax(-1, keepdim=True)
        bound = R.HALF * want.abs() + R.FINE * r * (mag + top + hat.abs() * top * hat.abs().amax(-1, keepdim=True)) + 1e-30
        got = dx[:, at].double()
        assert ((got - want).abs() <= bound).all(), (side, float(((got - want).abs() / bound).max()))
        if kind:
            row = 2 * side if kind == "layer" else side
            for i, t in enumerate(([d * hat, d] if kind == "layer" else [d * hat])):
                # fp32 sums: their error goes with the sum of magnitudes, far below 2^-14 of it
                lim = R.FINE * (t.abs() + R.pair_sum(dy[:, at].double(), pairs, interleaved) * hat.abs().clamp(min=1.0)).sum((0, 1)) + 1e-30
                assert ((dparams[row + i].double() - t.sum((0, 1))).abs() <= lim).all()


@pytest.mark.parametrize("c", CASES)
def test_forward_and_backward(dit, c):
    run_case(dit, *c, backward=True)


@pytest.mark.parametrize("c", [CASES[1], CASES[2], CASES[4], CASES[8]])
def test_in_place(dit, c):
    run_case(dit, *c, backward=True, in_place=True)


@pytest.mark.parametrize("far", [100003, 2 ** 31 - 300, -2 ** 31 + 10])
def test_far_positions(dit, far):
    """The angle is exact at every position: in fp32 the product alone would be off by far more than the bound."""
    run_case(dit, 40, 2, 2, 64, (16, 24, 24), "rms", True, backward=True, far=far, scale=[1.0, 0.375, 0.5])


@pytest.mark.parametrize("interleaved", [True, False])
def test_axes_that_the_positions_do_not_have_turn_nothing(dit, interleaved):
    """A table of three axes in a call with one: the pairs of the first turn, the others' positions are not looked for."""
    import ctypes
    from int8_mixed_precision_gb300.block_attention import _Rotary, _lay, _view
    t, h, dim, dims = 77, 3, 64, (16, 24, 24)
    x, positions, _, scale, new = case(t, h, 1, dim, dims, None, interleaved)
    q, at = x[:, :h], positions[:, :1].contiguous()
    rot = dit.Rotary(dims, dim, interleaved=interleaved)
    info = _Rotary(rot.table.data_ptr(), sum(dims) // 2, 1, int(interleaved), 0)
    angle = R.angles(positions, dims, 10000.0, scale)
    angle[:, dims[0] // 2:] = 0
    dy, ws = new(t, h, dim).to(BF16), dit.workspace()
    out, dx = torch.empty_like(dy), torch.empty_like(dy)
    view = lambda v, name: _view(v, t, h, dim, name, 0)  # noqa: E731
    rest = (t, dim, 0, None, 0.0, ctypes.byref(info), at.data_ptr())
    stream = torch.cuda.current_stream().cuda_stream
    views = _lay(view(q, "q"), None, view(out, "q_out"), None)
    assert dit.lib().dit_qk_norm_rope(*views, *rest, stream) == 0
    views = _lay(view(q, "q"), None, view(dy, "dq_out"), None, view(dx, "dq"), None)
    assert dit.lib().dit_qk_norm_rope_backward(*views, *rest, None, None, 0, ws.data_ptr(), ws.nbytes, stream) == 0
    for got, v, sign in ((out, q, 1), (dx, dy, -1)):
        want = R.turn(v.double(), sign * angle, interleaved)
        bound = R.HALF * want.abs() + R.FINE * R.pair_sum(v.double(), sum(dims) // 2, interleaved) + 1e-30
        assert ((got.double() - want).abs() <= bound).all()


def test_no_tokens(dit):
    x = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    params = torch.ones(2, 64, device="cuda")
    norm, ws, scratch = dit.QKNorm(params, "rms"), dit.workspace(), dit.qk_norm_scratch(64)
    dit.qk_norm_rope(x, x, x, x, norm)
    dparams = torch.full_like(params, 3.0)
    dit.qk_norm_rope_backward(x, x, x, x, x.clone(), x.clone(), norm, None, None, dparams, scratch, ws)
    assert (dparams == 0).all()


def test_queries_alone_and_other_streams(dit):
    x, positions, params, scale, _ = case(333, 5, 5, 64, (16, 24, 24), "rms", True)
    rot, norm = dit.Rotary((16, 24, 24), 64), dit.QKNorm(params, "rms")
    q, k = x[:, :5], x[:, 5:10]
    both = torch.empty(333, 10, 64, dtype=BF16, device="cuda")
    dit.qk_norm_rope(q, k, both[:, :5], both[:, 5:], norm, rot, positions)
    alone = torch.empty(333, 5, 64, dtype=BF16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dit.qk_norm_rope(q, None, alone, None, norm, rot, positions, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(alone, both[:, :5])


def test_same_bits_and_graph(dit):
    """Two calls give the same bits, and so does a captured one on new inputs; the parameters are read at each replay."""
    x, positions, params, scale, new = case(2011, 6, 2, 128, (32, 48, 48), "rms", False)
    rot, norm = dit.Rotary((32, 48, 48), 128, interleaved=False), dit.QKNorm(params, "rms")
    dy = new(2011, 8, 128).to(BF16)
    out, dx, dparams = torch.empty_like(dy), torch.empty_like(dy), torch.empty_like(params)
    ws, scratch = dit.workspace(), dit.qk_norm_scratch(128)

    def both():
        dit.qk_norm_rope(x[:, :6], x[:, 6:8], out[:, :6], out[:, 6:], norm, rot, positions)
        dit.qk_norm_rope_backward(x[:, :6], x[:, 6:8], dy[:, :6], dy[:, 6:], dx[:, :6], dx[:, 6:], norm, rot, positions, dparams, scratch, ws)
    both()
    first = [t.clone() for t in (out, dx, dparams)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for t in (out, dx, dparams):
        t.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, (out, dx, dparams)))
    params.mul_(1.5)
    graph.replay()
    got = [t.clone() for t in (out, dx, dparams)]
    both()
    assert all(torch.equal(a, b) for a, b in zip(got, (out, dx, dparams)))
    assert not torch.equal(got[0], first[0])
