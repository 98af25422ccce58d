"""Low-rank adapters on the GPU against their definition in 64 bits, at the lengths, ranks and widths
where tiles end; what one request holds never reaches another; repeatability; streams; graphs."""
import pytest
import torch

from adapter_reference import check, inputs, reference, spans

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import int8_mixed_precision_gb300 as dit  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class Setup:
    def __init__(self, c, training, n_adapters=None):
        self.c = c
        self.d = {k: v.cuda() for k, v in c.items() if torch.is_tensor(v)}
        G = self.d["a"].shape[0]
        self.plan = dit.AdapterPlan(c["lengths"], c["adapters"], G, training=training)
        self.bank = dit.AdapterBank(self.d["a"], self.d["b"], self.d["scale"])
        self.scratch = dit.adapter_scratch(self.plan, self.bank).fill_(0xff)   # contents are free
        self.ws = dit.workspace()
        self.saved = dit.adapter_saved(self.plan, self.bank).fill_(0xff) if training else None
        self.da = torch.full_like(self.d["a"], 7.0, dtype=F32)
        self.db = torch.full_like(self.d["b"], 7.0, dtype=F32)

    def forward(self, **kw):
        dit.lora_forward(self.plan, self.bank, self.d["x"], self.d["y"], self.scratch, self.ws, saved=self.saved, **kw)
        return self.d["y"]

    def backward(self, dx=True, **kw):
        dit.lora_backward(self.plan, self.bank, self.d["x"], self.d["dy"], self.saved, self.da, self.db, self.scratch,
                          self.ws, dx=self.d["dx"] if dx else None, **kw)
        return self.d["dx"]

    def ok(self):
        torch.cuda.synchronize()
        assert dit.device_status(self.ws) == 0


# (lengths, adapters, bank, rank, k, n): one row; tile edges of 128 and 16 rows; ranks that are no multiple of 16;
# widths that end inside a block of 64, 128 and 256 columns; empty requests; requests without an adapter; runs of
# one adapter from several requests, next to each other and apart; adapters without rows
SHAPES = [
    ([1], [0], 1, 8, 8, 8),
    ([1], [1], 3, 16, 1920, 5760),
    ([2, 1, 1, 0, 3], [0, 1, -1, 1, 0], 2, 16, 128, 256),
    ([1] * 40, [i % 5 - 1 for i in range(40)], 4, 32, 264, 520),
    ([127], [0], 1, 24, 72, 136),
    ([128], [0], 1, 64, 512, 256),
    ([129, 0, 31, 33], [1, 0, 0, 1], 2, 40, 200, 328),
    ([300, 5, 64, 17], [0, 1, -1, 0], 3, 128, 320, 264),
    ([70, 60], [0, 0], 1, 72, 136, 72),
    ([1000, 1, 517], [1, 0, 1], 2, 8, 1032, 24),
    ([260, 515, 16, 32, 33], [0, 1, 0, 1, 0], 2, 104, 648, 776),
    ([3000], [0], 1, 16, 64, 1920),
]


@pytest.mark.parametrize("y_dtype", [BF16, F32])
@pytest.mark.parametrize("training", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{sum(s[0])}-r{s[3]}-{s[4]}-{s[5]}")
def test_forward(shape, training, y_dtype):
    c = inputs(*shape, y_dtype)
    want, off = reference(c)
    s = Setup(c, training)
    check(s.forward(), want["y"], off["y"], "y")
    s.ok()


@pytest.mark.parametrize("y_dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{sum(s[0])}-r{s[3]}-{s[4]}-{s[5]}")
def test_backward(shape, y_dtype):
    c = inputs(*shape, y_dtype, seed=1)
    want, off = reference(c)
    s = Setup(c, True)
    s.forward()
    check(s.backward(), want["dx"], off["dx"], "dx")
    check(s.da, want["da"], off["da"], "da")
    check(s.db, want["db"], off["db"], "db")
    s.ok()


def test_backward_without_the_input_gradient():
    c = inputs([200, 70], [1, 0], 2, 16, 256, 128, BF16, seed=2)
    want, off = reference(c)
    s = Setup(c, True)
    s.forward()
    before = s.d["dx"].clone()
    s.backward(dx=False)
    assert torch.equal(before, s.d["dx"])
    check(s.da, want["da"], off["da"], "da")
    check(s.db, want["db"], off["db"], "db")


def test_gradients_against_differences():
    """The gradients of L = sum(y * dy) against central differences of the forward pass in fp32.  L is
    linear in each of x, A and B, so a difference is exact but for the fp32 rounding of y: with
    rounding 2^-24 |y| at each of `count` outputs, |error| <= 2 count 2^-24 max|y dy| / step."""
    c = inputs([40, 90, 30], [0, 1, 0], 2, 16, 64, 72, F32, seed=3)
    s = Setup(c, True)
    y0 = s.d["y"].clone()
    dx0 = s.d["dx"].clone()
    s.forward()
    s.backward()
    grads = {"a": s.da.double(), "b": s.db.double(), "x": (s.d["dx"] - dx0).double()}

    def loss():
        s.d["y"].copy_(y0)
        dit.lora_forward(s.plan, s.bank, s.d["x"], s.d["y"], s.scratch, s.ws)
        return float((s.d["y"].double() * s.d["dy"].double()).sum()), float((s.d["y"].abs() * s.d["dy"].abs()).max())

    gen = torch.Generator().manual_seed(0)
    for name in ("a", "b", "x"):
        for _ in range(6):
            i = tuple(int(torch.randint(0, v, (1,), generator=gen)) for v in grads[name].shape)
            t = s.d[name]
            old = t[i].clone()
            t[i] = old + 1.0
            hi, top = loss()
            up = float(t[i])
            t[i] = old - 1.0
            lo, _ = loss()
            step = up - float(t[i])
            t[i] = old
            slope = (hi - lo) / step
            # the fp32 roundings of h (held with 16 bits), y and the sums
            bound = 2 * y0.numel() ** 0.5 * 8 * (2.0 ** -23 * top) + 2.0 ** -15 * abs(slope) + 2.0 ** -15 * top * 16
            assert abs(slope - float(grads[name][i])) <= bound, (name, i, slope, float(grads[name][i]), bound)


@pytest.mark.parametrize("training", [False, True])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), 3.0e38])
def test_a_request_never_reaches_another(value, training):
    """Rows of one request filled with infinities, NaN or the largest values (x, dy and the factors of its
    adapter): every other request's outputs and gradients are bit for bit those of a clean batch."""
    lengths, adapters = [50, 3, 140, 1, 70], [0, 1, 2, 1, 0]
    clean = inputs(lengths, adapters, 3, 24, 200, 136, F32, seed=4)
    dirty = {k: v.clone() if torch.is_tensor(v) else v for k, v in clean.items()}
    rows = slice(53, 193)
    for name in ("x", "dy"):
        dirty[name][rows] = value
    dirty["a"][2], dirty["b"][2] = value, value
    out = []
    for c in (clean, dirty):
        s = Setup(c, training)
        s.forward()
        if training:
            s.backward()
        s.ok()
        out.append((s.d["y"].clone(), s.d["dx"].clone(), s.da, s.db))
    keep = torch.ones(sum(lengths), dtype=torch.bool)
    keep[rows] = False
    assert torch.equal(out[0][0].cpu()[keep], out[1][0].cpu()[keep])
    if training:
        assert torch.equal(out[0][1].cpu()[keep], out[1][1].cpu()[keep])
        assert torch.equal(out[0][2][:2], out[1][2][:2]) and torch.equal(out[0][3][:2], out[1][3][:2])


def test_rows_without_an_adapter_are_not_touched():
    lengths, adapters = [20, 200, 7], [-1, 0, -1]
    c = inputs(lengths, adapters, 2, 16, 128, 256, BF16, seed=5)
    c["y"][:20], c["y"][220:], c["dx"][:20] = float("nan"), float("inf"), float("nan")
    s = Setup(c, True)
    s.forward()
    s.backward()
    for name in ("y", "dx"):
        got, was = s.d[name].cpu(), c[name]
        for rows in (slice(0, 20), slice(220, 227)):
            assert torch.equal(got[rows].view(torch.int16), was[rows].view(torch.int16))
    assert not s.da[1].any() and not s.db[1].any()


@pytest.mark.parametrize("training", [False, True])
def test_nothing_to_do(training):
    """No rows at all, and no row with an adapter: gradients are zeros and nothing else changes."""
    for lengths, adapters in (([], []), ([0, 0], [0, 1]), ([5], [-1])):
        c = inputs(lengths, adapters, 2, 16, 64, 64, BF16)
        s = Setup(c, training)
        s.forward()
        if training:
            s.backward()
            assert not s.da.any() and not s.db.any()
        s.ok()
        assert torch.equal(s.d["y"].cpu(), c["y"])


@pytest.mark.parametrize("shape", [([9000, 3000, 40, 77], [0, 1, -1, 1], 2, 64, 1920), ([300, 5, 64, 1], [0, 1, -1, 0], 2, 128, 264)],
                         ids=["large", "small"])
@pytest.mark.parametrize("training", [False, True])
def test_y_may_be_x_and_dx_may_be_dy(shape, training):
    lengths, adapters, G, r, k = shape
    c = inputs(lengths, adapters, G, r, k, k, BF16, seed=12)
    s = Setup(c, training)
    s.d["y"].copy_(s.d["x"])
    s.d["dx"].copy_(s.d["dy"])
    y = s.forward().clone()
    if training:
        dx = s.backward().clone()
        for _ in range(5):
            t = Setup(c, True)
            dit.lora_forward(t.plan, t.bank, t.d["x"], t.d["y"], t.scratch, t.ws, saved=t.saved)
            dit.lora_backward(t.plan, t.bank, t.d["x"], t.d["dy"], t.saved, t.da, t.db, t.scratch, t.ws, dx=t.d["dy"])
            assert torch.equal(t.d["dy"], dx) and torch.equal(t.da, s.da) and torch.equal(t.db, s.db)
            t.ok()
    dit.lora_forward(s.plan, s.bank, s.d["x"], s.d["x"], s.scratch, s.ws)
    assert torch.equal(s.d["x"], y)
    s.ok()


def test_the_same_call_gives_the_same_bits():
    lengths, adapters = [700, 33, 1500, 260], [0, 1, 0, 2]
    c = inputs(lengths, adapters, 3, 48, 1032, 520, BF16, seed=6)
    outs = []
    for _ in range(3):
        s = Setup(c, True)
        s.forward()
        s.backward()
        outs.append([t.clone() for t in (s.d["y"], s.d["dx"], s.da, s.db)])
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(o, outs[0]))


def test_one_scratch_serves_layers_of_other_sizes():
    """Calls of different layers, plans and directions in a row through one scratch and workspace."""
    big = inputs([400, 130], [0, 1], 2, 64, 520, 1032, F32, seed=7)
    one = inputs([3, 1, 2], [1, 0, 1], 2, 16, 64, 136, F32, seed=8)
    a, b, t = Setup(big, True), Setup(one, False), Setup(one, True)
    b.scratch = t.scratch = a.scratch
    b.ws = t.ws = a.ws
    wants = [reference(c) for c in (big, one, one)]
    for _ in range(2):
        for s, (want, off) in zip((a, b, t), wants):
            s.d["y"].copy_(s.c["y"])
            s.d["dx"].copy_(s.c["dx"])
            check(s.forward(), want["y"], off["y"], "y")
            if s.saved is not None:
                check(s.backward(), want["dx"], off["dx"], "dx")
                check(s.da, want["da"], off["da"], "da")
                check(s.db, want["db"], off["db"], "db")
    a.ok()


def test_another_stream():
    c = inputs([300, 20], [0, 1], 2, 16, 256, 512, BF16, seed=9)
    want, off = reference(c)
    s = Setup(c, True)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    s.forward(stream=st)
    s.backward(stream=st)
    st.synchronize()
    check(s.d["y"], want["y"], off["y"], "y")
    check(s.da, want["da"], off["da"], "da")


def test_graph_replay():
    c = inputs([200, 1, 16], [0, 1, 1], 2, 32, 256, 384, F32, seed=10)
    s = Setup(c, True)
    s.forward()
    s.backward()
    first = [t.clone() for t in (s.d["y"], s.d["dx"], s.da, s.db)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            s.forward()
            s.backward()
    torch.cuda.synchronize()
    for _ in range(2):
        s.d["y"].copy_(c["y"])
        s.d["dx"].copy_(c["dx"])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(first, (s.d["y"], s.d["dx"], s.da, s.db)))


def test_a_wrong_table_is_skipped_and_reported():
    """Entries that point outside the batch or the bank: nothing out of range is read or written, and
    the status word says so."""
    for training, where, value in ((True, 0, 10 ** 6), (True, 1, 500), (True, 2, 9), (False, 16, 99), (False, 16 + 5, 10 ** 6)):
        c = inputs([100, 5, 200], [0, 1, 0], 2, 16, 64, 64, BF16, seed=11)
        s = Setup(c, training)
        if not training:
            assert s.plan.n_tiles == 3 and s.plan.n_small == 1
        s.plan.table[where] = value
        s.forward()
        if training:
            s.backward()
        torch.cuda.synchronize()
        assert dit.device_status(s.ws) == 1 << 1
        dit.clear_device_status(s.ws)


def test_beside_a_routed_projection():
    """AdaptedLinear: the projection's own output plus the adapters, and dx through both."""
    T, K, N, G, r = 300, 256, 512, 2, 16
    c = inputs([180, 120], [1, 0], G, r, K, N, BF16, seed=12)
    g = torch.Generator().manual_seed(1)
    w = (torch.randn(N, K, generator=g) * 0.02).cuda()
    ws = dit.workspace()
    wq = dit.QuantizedWeight(w, 64, ws, keep_bf16=True)
    lin = dit.RoutedLinear(wq, T, ws)
    s = Setup(c, True)
    layer = dit.AdaptedLinear(lin, s.bank, w_t=w.t().contiguous().to(BF16))
    for route in (dit.ROUTE_NVFP4, dit.ROUTE_INT8, dit.ROUTE_BF16):
        base = torch.empty(T, N, dtype=F32, device="cuda")
        lin(s.d["x"], route, base)
        y = torch.empty(T, N, dtype=F32, device="cuda")
        layer(s.d["x"], route, y, s.plan, s.scratch, saved=s.saved)
        want, off = reference({**c, "y": base.cpu()})
        check(y, want["y"], off["y"], "y")
    dx = torch.empty(T, K, dtype=F32, device="cuda")
    layer.backward(s.d["x"], s.d["dy"], s.plan, s.saved, s.da, s.db, dx, s.scratch)
    through = torch.empty(T, K, dtype=F32, device="cuda")
    dit.gemm_bf16(s.d["dy"], layer.w_t, through, ws)
    want, off = reference({**c, "dx": through.cpu()})
    check(dx, want["dx"], off["dx"], "dx")
    check(s.da, want["da"], off["da"], "da")
    with pytest.raises(dit.DitError, match="activation"):
        layer(s.d["x"], dit.ROUTE_INT8, y, s.plan, s.scratch, act=dit.ACT_GELU_ERF)
    assert dit.device_status(ws) == 0


def test_spans_of_the_plan_cover_the_batch():
    """Every row with an adapter is in exactly one tile of either kind, with its adapter."""
    lengths, adapters = [300, 5, 64, 17, 1, 1, 33, 32], [0, 1, -1, 0, 1, 1, 2, 1]
    for training in (False, True):
        plan = dit.AdapterPlan(lengths, adapters, 3, training=training)
        t = plan.table.cpu().tolist()
        seen = {}
        for i in range(plan.n_tiles):
            row0, rows, g, _ = t[4 * i:4 * i + 4]
            for r in range(row0, row0 + rows):
                assert r not in seen
                seen[r] = g
        at = (4 * plan.n_tiles + 4 + 3) // 4 * 4
        for i in range(plan.n_small):
            e = t[at + 20 * i:at + 20 * i + 20]
            for r in e[4:4 + e[1]]:
                assert r not in seen
                seen[r] = e[0]
        want = {r: g for rows, g in spans(lengths, adapters) for r in range(rows.start, rows.stop)}
        assert seen == want


def test_refusals_of_device_buffers():
    c = inputs([40], [0], 2, 16, 64, 72, BF16)
    s = Setup(c, True)
    d, call = s.d, lambda **kw: dit.lora_forward(**{**dict(plan=s.plan, bank=s.bank, x=s.d["x"], y=s.d["y"], scratch=s.scratch, ws=s.ws), **kw})
    for bad in (d["y"][:39], d["y"][:, :64], d["y"].to(torch.float16), torch.zeros(72, 40, dtype=BF16, device="cuda").t()):
        with pytest.raises(dit.DitError, match="y|contiguous"):
            call(y=bad)
    for kw in (dict(y=d["y"].cpu()), dict(scratch=s.scratch[:64]), dict(ws=s.ws[:64]), dict(saved=s.saved[:64]), dict(saved=s.scratch),
               dict(x=d["x"][1:]), dict(plan=dit.AdapterPlan([40], [0], 2, device="cpu"))):
        with pytest.raises(dit.DitError):
            call(**kw)
    back = lambda **kw: dit.lora_backward(**{**dict(plan=s.plan, bank=s.bank, x=d["x"], dy=d["dy"], saved=s.saved, da=s.da, db=s.db,   # noqa: E731
                                                    scratch=s.scratch, ws=s.ws, dx=d["dx"]), **kw})
    for kw, what in ((dict(da=s.db), "da"), (dict(db=s.db.bfloat16()), "db"), (dict(dx=d["dy"]), "dx"), (dict(dy=d["dy"].float()), "dy"),
                     (dict(saved=s.saved[:64]), "INVALID"), (dict(da=s.da.cpu()), "CUDA")):
        with pytest.raises(dit.DitError, match=what):
            back(**kw)
    # a row further on is 16 bytes off the 32 that the library wants
    off = torch.zeros(41 * 64 + 8, dtype=BF16, device="cuda")[8:8 + 40 * 64].view(40, 64)
    with pytest.raises(dit.DitError, match="ALIGNMENT"):
        call(x=off)
    s.ok()


@pytest.mark.parametrize("what", ["forward", "backward"])
def test_waits_that_run_out_are_reported_and_leave_the_workspace_usable(what, monkeypatch):
    """Producers that load nothing (the library's test hook): every wait gives up after a second, the status word
    says so, and the next calls on the same workspace are right."""
    c = inputs([260, 40, 129], [0, 1, 0], 2, 24, 200, 328, F32, seed=13)
    want, off = reference(c)
    s = Setup(c, True)
    s.forward()
    s.d["y"].copy_(c["y"])
    monkeypatch.setenv("DIT6_TEST_STALL_PRODUCER", "1")
    s.forward() if what == "forward" else s.backward()
    torch.cuda.synchronize()
    assert dit.device_status(s.ws) == 1 << 5
    monkeypatch.delenv("DIT6_TEST_STALL_PRODUCER")
    dit.clear_device_status(s.ws)
    s.d["y"].copy_(c["y"])
    s.d["dx"].copy_(c["dx"])
    check(s.forward(), want["y"], off["y"], "y")
    check(s.backward(), want["dx"], off["dx"], "dx")
    check(s.da, want["da"], off["da"], "da")
    check(s.db, want["db"], off["db"], "db")
    s.ok()


def test_offsets_past_32_bits():
    """x, y, dx and dy of more than 2^31 elements: the rows at both ends against their definition, and the rows in
    between untouched (they have no adapter)."""
    T, K, N, r = 280000, 7680, 7680, 8
    lengths, adapters = [150, T - 300, 150], [0, -1, 1]
    assert T * K > 2 ** 31
    ends = inputs([150, 150], [0, 1], 2, r, K, N, BF16, seed=14)
    want, off = reference(ends)
    put = lambda t: torch.cat([t[:150].cuda(), torch.ones(T - 300, t.shape[1], dtype=t.dtype, device="cuda"), t[150:].cuda()])  # noqa: E731
    x, y, dy, dx = (put(ends[n]) for n in ("x", "y", "dy", "dx"))
    bank = dit.AdapterBank(*(ends[n].cuda() for n in ("a", "b", "scale")))
    plan, ws = dit.AdapterPlan(lengths, adapters, 2, training=True), dit.workspace()
    scratch, saved = dit.adapter_scratch(plan, bank), dit.adapter_saved(plan, bank)
    da, db = torch.empty_like(bank.a, dtype=F32), torch.empty_like(bank.b, dtype=F32)
    dit.lora_forward(plan, bank, x, y, scratch, ws, saved=saved)
    dit.lora_backward(plan, bank, x, dy, saved, da, db, scratch, ws, dx=dx)
    for got, name in ((y, "y"), (dx, "dx")):
        check(torch.cat([got[:150], got[-150:]]), want[name], off[name], name)
        assert bool((got[150:-150:997] == 1).all()) and bool((got[150:160] == 1).all()) and bool((got[-160:-150] == 1).all())
    check(da, want["da"], off["da"], "da")
    check(db, want["db"], off["db"], "db")
    assert dit.device_status(ws) == 0


def test_the_example_trains_and_serves():
    """The example's training loss falls to a tenth, and it serves each request with its own adapter: outputs are
    within 15 % of the wanted projection (INT8 alone is within 2 %), which the unadapted one misses by far more."""
    import os
    import sys
    from conftest import ROOT
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import adapters as example
        got = example.main(steps=300)
    finally:
        sys.path.pop(0)
        sys.modules.pop("adapters", None)
    assert got["loss"][1] < 0.1 * got["loss"][0], got
    assert got["errors"][-1] < 0.02 and max(got["errors"][0], got["errors"][1]) < 0.15, got
