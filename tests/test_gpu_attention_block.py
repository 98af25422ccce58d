"""The norms, the rotation and the attention run together: between a block's projections, and in training with adapters."""
import os
import sys

import pytest
import torch

import attention_reference as R
from conftest import ROOT

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def dit():
    import int8_mixed_precision_gb300 as d
    return d


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import attention
    return attention


def chain(qkv, params, positions, lengths, heads, kv_heads, dim):
    """Norms, rotation and attention of the projection's output, in 64 bits with autograd."""
    angle = R.angles(positions, (16, 24, 24), 10000.0, [1.0] * 3)
    parts = []
    for i, (at, n) in enumerate(((0, heads), (heads, kv_heads))):
        x = qkv[:, at:at + n]
        r = (x.square().mean(-1, keepdim=True) + 1e-6) ** -0.5
        parts.append(R.turn(x * r * params[i], angle, True))
    q, k, v = parts[0], parts[1].repeat_interleave(heads // kv_heads, 1), qkv[:, heads + kv_heads:].repeat_interleave(heads // kv_heads, 1)
    out, at = [], 0
    for n in lengths:
        s = torch.einsum("nhd,mhd->hnm", q[at:at + n], k[at:at + n]) * dim ** -0.5
        out.append(torch.einsum("hnm,mhd->nhd", torch.softmax(s, -1), v[at:at + n]))
        at += n
    return torch.cat(out)


def test_between_quantised_projections(dit):
    heads, kv_heads, dim, lengths = 6, 2, 64, [70, 200, 33]
    t, hidden = sum(lengths), heads * dim
    g = torch.Generator(device="cuda").manual_seed(3)
    ws = dit.workspace()
    wide = (heads + 2 * kv_heads) * dim
    qkv_lin = dit.RoutedLinear(dit.QuantizedWeight(torch.randn(wide, hidden, device="cuda", generator=g) * hidden ** -0.5, 64, ws), t, ws)
    out_lin = dit.RoutedLinear(dit.QuantizedWeight(torch.randn(hidden, hidden, device="cuda", generator=g) * hidden ** -0.5, 64, ws), t, ws)
    params = 1 + 0.2 * torch.randn(2, dim, device="cuda", generator=g)
    positions = torch.randint(0, 30, (t, 3), device="cuda", generator=g, dtype=torch.int32)
    x = torch.randn(t, hidden, device="cuda", generator=g).to(BF16)
    part = dit.RoutedAttention(qkv_lin, out_lin, heads, kv_heads, dit.QKNorm(params, "rms"), dit.Rotary((16, 24, 24), dim))
    plan = dit.AttentionPlan(lengths, heads, dim, kv_heads=kv_heads)
    qkv, attended = torch.empty(t, heads + 2 * kv_heads, dim, dtype=BF16, device="cuda"), torch.empty(t, heads, dim, dtype=BF16, device="cuda")
    y = torch.empty(t, hidden, dtype=BF16, device="cuda")
    scratch = dit.attention_scratch(plan)
    for routes in ((dit.ROUTE_INT8, dit.ROUTE_NVFP4), (dit.ROUTE_NVFP4, dit.ROUTE_INT8)):
        part(x, routes, y, plan, qkv, attended, scratch, positions)
        plain = torch.empty_like(qkv)
        qkv_lin(x, routes[0], plain.view(t, -1))
        want = chain(plain.double(), params.double(), positions, lengths, heads, kv_heads, dim)
        # bf16 between the steps: q and k (2^-8 of each, on scores of some units), p and the output
        assert (attended.double() - want).abs().max() <= 8 * R.HALF * want.abs().max()
        assert torch.equal(qkv[:, heads + kv_heads:], plain[:, heads + kv_heads:])
        again = torch.empty_like(y)
        out_lin(attended.view(t, -1), routes[1], again)
        assert torch.equal(again, y)
    assert dit.device_status(ws) == 0


def test_refusals_before_anything_is_written(dit):
    heads, dim, t = 2, 64, 50
    ws = dit.workspace()
    lin = dit.RoutedLinear(dit.QuantizedWeight(torch.randn(3 * 128, 128, device="cuda"), 64, ws), t, ws)
    out = dit.RoutedLinear(dit.QuantizedWeight(torch.randn(128, 128, device="cuda"), 64, ws), t, ws)
    with pytest.raises(dit.DitError):
        dit.RoutedAttention(lin, out, 3)
    with pytest.raises(dit.DitError):
        dit.RoutedAttention(out, out, 2)
    part = dit.RoutedAttention(lin, out, heads, rotary=dit.Rotary((16, 24, 24), dim))
    plan = dit.AttentionPlan([t], heads, dim)
    ok = dict(x=torch.randn(t, 128, device="cuda").to(BF16), routes=(1, 1), y=torch.full((t, 128), 3.0, dtype=BF16, device="cuda"), plan=plan,
              qkv=torch.full((t, 6, dim), 4.0, dtype=BF16, device="cuda"), attended=torch.full((t, 2, dim), 5.0, dtype=BF16, device="cuda"),
              scratch=dit.attention_scratch(plan), positions=torch.zeros(t, 3, dtype=torch.int32, device="cuda"))
    for change in (dict(positions=None), dict(positions=ok["positions"].long()), dict(positions=ok["positions"][:-1]), dict(plan=dit.AttentionPlan([t - 1], heads, dim)),
                   dict(plan=dit.AttentionPlan([t], 4, 32)), dict(qkv=ok["qkv"][:, :5]), dict(attended=ok["qkv"][:, :2]), dict(attended=ok["attended"].float())):
        with pytest.raises(dit.DitError):
            part(**{**ok, **change})
    torch.cuda.synchronize()
    assert (ok["y"] == 3).all() and (ok["qkv"] == 4).all() and (ok["attended"] == 5).all()
    part(**ok)


def test_refusals_of_the_calls(dit):
    h, d, t = 2, 64, 20
    x = torch.zeros(t, 3 * h, d, dtype=BF16, device="cuda")
    q, k, v = x[:, :h], x[:, h:2 * h], x[:, 2 * h:]
    plan, ws = dit.AttentionPlan([t], h, d, training=True), dit.workspace()
    scratch, saved, out = dit.attention_scratch(plan), dit.attention_saved(plan), torch.empty(t, h, d, dtype=BF16, device="cuda")
    ok = dict(plan=plan, q=q, k=k, v=v, out=out, scratch=scratch, ws=ws, saved=saved)
    dit.attention(**ok)
    for change in (dict(q=q.float()), dict(q=q[:-1]), dict(q=q[:, :1]), dict(k=k[..., :32]), dict(out=q), dict(out=x[:, 1:1 + h]), dict(scale=0.0),
                   dict(scale=float("nan")), dict(saved=saved[:-4]), dict(scratch=scratch[:4]), dict(ws=ws[:64]), dict(v=v.transpose(0, 1)), dict(k=k[:1].expand(t, h, d)),
                   dict(q=torch.empty(t, h, d + 4, dtype=BF16, device="cuda")[..., :d]), dict(v=v.cpu())):
        with pytest.raises(dit.DitError):
            dit.attention(**{**ok, **change})
    g = torch.empty_like(x)
    back = dict(plan=plan, q=q, k=k, v=v, out=out, dout=torch.zeros_like(out), saved=saved, dq=g[:, :h], dk=g[:, h:2 * h], dv=g[:, 2 * h:], scratch=scratch, ws=ws)
    dit.attention_backward(**back)
    for change in (dict(dq=q), dict(dk=g[:, :h]), dict(dv=back["dout"]), dict(plan=dit.AttentionPlan([t], h, d)), dict(saved=saved[:4]), dict(dout=out.float())):
        with pytest.raises(dit.DitError):
            dit.attention_backward(**{**back, **change})
    norm, rot, pos = dit.QKNorm(torch.ones(2, d, device="cuda"), "rms"), dit.Rotary((16, 24, 24), d), torch.zeros(t, 3, dtype=torch.int32, device="cuda")
    ok = dict(q=q, k=k, q_out=g[:, :h], k_out=g[:, h:2 * h], norm=norm, rotary=rot, positions=pos)
    dit.qk_norm_rope(**ok)
    for change in (dict(q_out=k), dict(q_out=x[:, 1:1 + h]), dict(k_out=g[:, 1:1 + h]), dict(k=None), dict(k_out=None), dict(positions=None), dict(positions=pos[:, :2]),
                   dict(positions=pos.T.contiguous().T), dict(norm=dit.QKNorm(torch.ones(2, 32, device="cuda"), "rms")), dict(rotary=dit.Rotary((32,), 32)),
                   dict(rotary=None), dict(q=q[:-1]), dict(q_out=g[:-1, :h]), dict(norm=dit.QKNorm(torch.ones(2, d), "rms"))):
        with pytest.raises(dit.DitError):
            dit.qk_norm_rope(**{**ok, **change})
    assert dit.device_status(ws) == 0


def test_training_chain_gradients(dit, example):
    """Gradients of adapters, norms' weights and input through the whole chain, against autograd in 64 bits."""
    heads, dim, rank, lengths = 2, 64, 8, [40, 1, 90]
    t, hidden = sum(lengths), heads * dim
    g = torch.Generator(device="cuda").manual_seed(5)
    new = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    ws = dit.workspace()
    w = new(3 * hidden, hidden) * hidden ** -0.5
    lin = dit.RoutedLinear(dit.QuantizedWeight(w, 64, ws), t, ws)
    bank = dit.AdapterBank((new(1, rank, hidden) * hidden ** -0.5).to(BF16), (new(1, 3 * hidden, rank) * 0.1).to(BF16), torch.full((1,), 0.7, device="cuda"))
    params = 1 + 0.2 * new(2, dim)
    positions = torch.randint(0, 20, (t, 3), device="cuda", generator=g, dtype=torch.int32)
    block = example.Trainable(dit.AdaptedLinear(lin, bank), dit.QKNorm(params, "rms"), dit.Rotary((16, 24, 24), dim), heads, dim,
                              dit.AdapterPlan([t], [0], 1, training=True), dit.AttentionPlan(lengths, heads, dim, training=True), positions)
    x, dout = new(t, hidden).to(BF16), new(t, heads, dim).to(BF16)
    out = block.forward(x).clone()
    block.backward(x, dout)

    frozen = torch.empty(t, 3 * hidden, dtype=BF16, device="cuda")
    lin(x, dit.ROUTE_INT8, frozen)
    leaves = [v.double().requires_grad_() for v in (bank.a[0], bank.b[0], params)]
    qkv = frozen.double() + 0.7 * (x.double() @ leaves[0].T) @ leaves[1].T
    want = chain(qkv.view(t, 3 * heads, dim), leaves[2], positions, lengths, heads, heads, dim)
    (want * dout.double()).sum().backward()
    # the values between the steps are held in bf16: some 2^-8 of the largest entries, and as much again on the way back
    assert (out.double() - want).abs().max() <= 8 * R.HALF * want.abs().max()
    for got, leaf in ((block.da[0], leaves[0]), (block.db[0], leaves[1]), (block.dparams, leaves[2])):
        assert torch.isfinite(got).all()
        off = (got.double() - leaf.grad).norm() / leaf.grad.norm()
        assert off <= 6 * R.HALF, float(off)
    assert dit.device_status(ws) == 0


def test_step_captured_beside_a_live_eager_one(dit, example):
    """The whole step captured into a graph while the tensors of an eager one live: same bits, and replays follow the inputs."""
    heads, dim, lengths = 2, 64, [130, 77]
    t, hidden = sum(lengths), heads * dim
    ws = dit.workspace()
    g = torch.Generator(device="cuda").manual_seed(6)
    new = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    lin = dit.RoutedLinear(dit.QuantizedWeight(new(3 * hidden, hidden) * hidden ** -0.5, 64, ws), t, ws)
    bank = dit.AdapterBank((new(1, 8, hidden) * 0.1).to(BF16), (new(1, 3 * hidden, 8) * 0.1).to(BF16), torch.ones(1, device="cuda"))
    block = example.Trainable(dit.AdaptedLinear(lin, bank), dit.QKNorm(torch.ones(2, dim, device="cuda"), "rms"), dit.Rotary((16, 24, 24), dim), heads, dim,
                              dit.AdapterPlan([t], [0], 1, training=True), dit.AttentionPlan(lengths, heads, dim, training=True),
                              torch.randint(0, 20, (t, 3), device="cuda", generator=g, dtype=torch.int32))
    x, dout = new(t, hidden).to(BF16), new(t, heads, dim).to(BF16)
    outputs = lambda: [v.clone() for v in (block.out, block.da, block.db, block.dparams, block.dx)]  # noqa: E731

    def step():
        block.forward(x)
        block.backward(x, dout)
    step()
    first = outputs()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step()
    for v in (block.out, block.da, block.db, block.dparams, block.dx):
        v.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, outputs()))
    x.copy_(new(t, hidden))
    graph.replay()
    got = outputs()
    step()
    assert all(torch.equal(a, b) for a, b in zip(got, outputs()))
    assert dit.device_status(ws) == 0


def test_example_runs(example):
    got = example.main(steps=3)
    assert got["rows"] == 122 + 41 + 80 and torch.isfinite(got["y"]).all()
    assert all(v == v for v in got["loss"])


def test_heads_in_front_of_tokens(dit):
    """Queries, keys and values of each head behind one another, [heads, 3, tokens, dim], and their gradients in such a buffer:
    the bits of the calls on tensors of their own."""
    h, t, d = 3, 300, 64
    g = torch.Generator(device="cuda").manual_seed(11)
    new = lambda *s: torch.randn(*s, device="cuda", generator=g).to(BF16)  # noqa: E731
    x, dout = new(h, 3, t, d), new(t, h, d)
    parts = lambda b: [b[:, i].transpose(0, 1) for i in range(3)]  # noqa: E731
    norm, rot = dit.QKNorm(torch.rand(2, d, device="cuda", generator=g) + 0.5, "rms"), dit.Rotary((16, 24, 24), d)
    positions = torch.randint(0, 40, (t, 3), device="cuda", generator=g, dtype=torch.int32)
    plan, ws = dit.AttentionPlan([200, 100], h, d, training=True), dit.workspace()
    scratch, saved = dit.attention_scratch(plan), dit.attention_saved(plan)
    got = []
    for together in (True, False):
        if together:
            q, k, v = parts(x.clone())
            dq, dk, dv = parts(torch.empty_like(x))
        else:
            q, k, v = (p.contiguous() for p in parts(x))
            dq, dk, dv = (torch.empty_like(q) for _ in range(3))
        raw = q.clone(), k.clone()
        dit.qk_norm_rope(q, k, q, k, norm, rot, positions)
        out, dparams = torch.empty(t, h, d, dtype=BF16, device="cuda"), torch.empty_like(norm.params)
        dit.attention(plan, q, k, v, out, scratch, ws, saved=saved)
        dit.attention_backward(plan, q, k, v, out, dout, saved, dq, dk, dv, scratch, ws)
        dit.qk_norm_rope_backward(*raw, dq, dk, dq, dk, norm, rot, positions, dparams, dit.qk_norm_scratch(d), ws)
        got.append([a.clone() for a in (q, k, out, dq, dk, dv, dparams)])
    assert all(torch.isfinite(a).all() and torch.equal(a, b) for a, b in zip(*got))
    assert dit.device_status(ws) == 0


def test_what_the_projections_refuse_is_refused_first(dit):
    heads, dim, t = 2, 64, 50
    ws = dit.workspace()
    weight = lambda n, **kw: dit.QuantizedWeight(torch.randn(n, 128, device="cuda"), 64, ws, **kw)  # noqa: E731
    lin, out = dit.RoutedLinear(weight(3 * 128), t, ws), dit.RoutedLinear(weight(128), t, ws)
    part, small = dit.RoutedAttention(lin, out, heads), dit.RoutedAttention(lin, dit.RoutedLinear(weight(128), t - 1, ws), heads)
    plan = dit.AttentionPlan([t], heads, dim)
    buffers = dict(y=torch.full((t, 128), 3.0, dtype=BF16, device="cuda"), qkv=torch.full((t, 6, dim), 4.0, dtype=BF16, device="cuda"),
                   attended=torch.full((t, 2, dim), 5.0, dtype=BF16, device="cuda"))
    ok = dict(x=torch.randn(t, 128, device="cuda").to(BF16), routes=(1, 0), plan=plan, scratch=dit.attention_scratch(plan), **buffers)
    y, bias = ok["y"], torch.zeros(128, device="cuda")
    room = torch.full((t * 128 + 8,), 3.0, dtype=BF16, device="cuda")
    for change in (dict(routes=(1,)), dict(routes=(1, dit.ROUTE_BF16)), dict(routes=(dit.ROUTE_BF16, 1)), dict(y=y[:-1]), dict(y=y.T), dict(y=y.cpu()),
                   dict(y=y.to(torch.float16)), dict(y=room[8:].view(t, 128)), dict(bias=(None,)), dict(bias=(None, bias.double())), dict(bias=(None, bias[:-1])),
                   dict(bias=(bias, None)), dict(bias=(None, bias.cpu()))):
        with pytest.raises(dit.DitError):
            part(**{**ok, **change})
    with pytest.raises(dit.DitError):
        small(**ok)
    torch.cuda.synchronize()
    assert (ok["y"] == 3).all() and (ok["qkv"] == 4).all() and (ok["attended"] == 5).all() and (room == 3).all()
    part(**ok)
    want = y.clone()
    part(**{**ok, "y": ok["attended"].view(t, 128)})  # a quantised route has read the attention before it writes
    assert torch.equal(want, ok["attended"].view(t, 128))
    kept = dit.RoutedAttention(lin, dit.RoutedLinear(weight(128, keep_bf16=True), t, ws), heads)
    kept(**{**ok, "routes": (1, dit.ROUTE_BF16)})
    with pytest.raises(dit.DitError):
        kept(**{**ok, "routes": (1, dit.ROUTE_BF16), "y": ok["attended"].view(t, 128)})
    assert dit.device_status(ws) == 0


def test_projections_refuse_rows_of_another_width(dit):
    """Codes of narrower rows would be read as rows of the weight's width."""
    t, ws = 50, dit.workspace()
    weight = lambda n: dit.QuantizedWeight(torch.randn(n, 128, device="cuda"), 64, ws, keep_bf16=True)  # noqa: E731
    lin, out = dit.RoutedLinear(weight(3 * 128), t, ws), dit.RoutedLinear(weight(128), t, ws)
    plan = dit.AttentionPlan([t], 2, 64)
    y, qkv, attended = (torch.full(s, 3.0, dtype=BF16, device="cuda") for s in ((t, 128), (t, 6, 64), (t, 2, 64)))
    for route in (0, 1, 2):
        for x in (torch.randn(t, 64, device="cuda"), torch.randn(t, 192, device="cuda"), torch.randn(t, 1, 128, device="cuda")):
            with pytest.raises(dit.DitError):
                out(x.to(BF16), route, y)
            with pytest.raises(dit.DitError):
                dit.RoutedAttention(lin, out, 2)(x.to(BF16), (route, 1), y, plan, qkv, attended, dit.attention_scratch(plan))
    torch.cuda.synchronize()
    assert (y == 3).all() and (qkv == 3).all() and (attended == 3).all()
