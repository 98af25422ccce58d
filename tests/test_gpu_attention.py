"""Attention over packed documents and its gradients, against the formulas in 64 bits."""
import pytest
import torch

import attention_reference as R

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def dit():
    import int8_mixed_precision_gb300 as d
    return d


class Batch:
    """A batch in one buffer [rows, heads + 2 kv_heads, dim], or with keys in a cache; rows of no document hold NaN."""

    def __init__(self, dit, lengths, heads, kv_heads, dim, frame=0, prefix=0, kv_lengths=None, room=None, train=True, seed=0, sharp=1.0, tail=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.dit, self.lengths, self.h, self.hk, self.d, self.frame = dit, lengths, heads, kv_heads, dim, frame
        self.keys = lengths if kv_lengths is None else kv_lengths
        self.prefix = [prefix] * len(lengths) if isinstance(prefix, int) else prefix
        n = sum(lengths)
        self.q = torch.full((n + tail, heads, dim), float("nan"), dtype=BF16, device="cuda")
        self.q[:n] = (new(n, heads, dim) * sharp).to(BF16)
        self.begins = [sum(self.keys[:i]) for i in range(len(self.keys))] if room is None else [i * room + 1 for i in range(len(self.keys))]
        rows = max([b + m for b, m in zip(self.begins, self.keys)] + [0]) + tail
        kv = torch.full((rows, 2 * kv_heads, dim), float("nan"), dtype=BF16, device="cuda")
        for b, m in zip(self.begins, self.keys):
            kv[b:b + m] = new(m, 2 * kv_heads, dim).to(BF16)
        self.k, self.v = kv[:, :kv_heads], kv[:, kv_heads:]
        self.out = torch.full((n + tail, heads, dim), 7.0, dtype=BF16, device="cuda")
        self.plan = dit.AttentionPlan(lengths, heads, dim, kv_heads=kv_heads, kv_lengths=self.keys, kv_begins=None if room is None else self.begins,
                                      frame=frame, prefix=self.prefix, training=train)
        self.ws, self.scratch = dit.workspace(), dit.attention_scratch(self.plan)
        self.scratch.fill_(255)
        self.saved = dit.attention_saved(self.plan) if train else None
        if train:
            self.saved.fill_(255)
            self.dout = torch.full_like(self.q, float("nan"))
            self.dout[:n] = new(n, heads, dim).to(BF16)
            self.dq = torch.full_like(self.q, 5.0)
            grad = torch.full_like(kv, 5.0)
            self.dk, self.dv = grad[:, :kv_heads], grad[:, kv_heads:]

    def forward(self, **more):
        self.dit.attention(self.plan, self.q, self.k, self.v, self.out, self.scratch, self.ws, saved=self.saved, **more)

    def backward(self, **more):
        self.dit.attention_backward(self.plan, self.q, self.k, self.v, self.out, self.dout, self.saved, self.dq, self.dk, self.dv, self.scratch,
                                    self.ws, **more)

    def check(self, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        train, group, q0 = self.saved is not None, self.h // self.hk, 0
        covered = torch.zeros(self.k.shape[0], dtype=torch.bool)
        for n, m, b, pre in zip(self.lengths, self.keys, self.begins, self.prefix):
            seen = R.visible(n, m, self.frame, pre, "cuda")
            covered[b:b + m] = True
            rows, keys = slice(q0, q0 + n), slice(b, b + m)
            for j in range(self.hk):
                k, v = self.k[keys, j].double(), self.v[keys, j].double()
                sums = [[0.0, 0.0], [0.0, 0.0]]
                for head in range(j * group, (j + 1) * group):
                    q = self.q[rows, head].double()
                    o, p, bound = R.attention(q, k, v, seen, scale)
                    self.close("out", self.out[rows, head], o, bound)
                    if not train:
                        continue
                    dq, dk, dv = R.attention_grads(q, k, v, p, o, self.dout[rows, head].double(), scale)
                    self.close("dq", self.dq[rows, head], *dq)
                    for s, t in zip(sums, (dk, dv)):
                        s[0], s[1] = s[0] + t[0], s[1] + t[1]
                if train and m:
                    zero = torch.zeros(m, self.d, dtype=torch.float64, device="cuda")
                    self.close("dk", self.dk[keys, j], sums[0][0] + zero, sums[0][1] + zero)
                    self.close("dv", self.dv[keys, j], sums[1][0] + zero, sums[1][1] + zero)
            q0 += n
        assert (self.out[q0:] == 7.0).all()  # rows of no document are as they were
        if train:
            assert (self.dq[q0:] == 5.0).all() and (self.dk[~covered] == 5.0).all() and (self.dv[~covered] == 5.0).all()
        assert self.dit.device_status(self.ws) == 0

    def close(self, what, got, want, bound):
        if not want.numel():
            return
        off = (got.double() - want).abs()
        assert torch.isfinite(got).all(), what
        assert (off <= bound).all(), (what, float((off / bound).max()), float(off.max()))


CASES = [
    # lengths, heads, kv_heads, dim, frame, prefix
    ([128], 1, 1, 64, 0, 0),
    ([1], 1, 1, 64, 0, 0),
    ([300], 2, 2, 64, 0, 0),
    ([257, 1, 0, 130, 64], 3, 3, 64, 0, 0),
    ([700], 1, 1, 64, 1, 0),
    ([700, 45], 2, 2, 64, 60, 33),
    ([64, 65, 63], 4, 2, 128, 0, 0),
    ([513], 3, 1, 128, 1, 17),
    ([200, 31], 6, 2, 40, 7, 100),
    ([90], 2, 2, 8, 0, 0),
    ([333], 5, 1, 72, 50, 0),
    ([130, 257], 1, 1, 96, 0, 0),
    ([1, 1, 1, 2], 8, 1, 128, 1, 0),
    ([20], 4, 4, 64, 1000000000, 2000000000),
    ([5, 0, 0, 3], 2, 2, 64, 0, 0),
]


@pytest.mark.parametrize("c", CASES)
def test_forward_and_backward(dit, c):
    lengths, heads, kv_heads, dim, frame, prefix = c
    b = Batch(dit, lengths, heads, kv_heads, dim, frame, prefix)
    b.forward()
    b.backward()
    b.check()


@pytest.mark.parametrize("dim", [64, 128])
def test_longer_than_every_ring(dit, dim):
    b = Batch(dit, [1700, 900], 4, 2, dim, 0, 0)
    b.forward()
    b.backward()
    b.check()


@pytest.mark.parametrize("frame,prefix", [(0, 0), (1, 0), (70, 45)])
@pytest.mark.parametrize("heads,kv_heads,dim", [(60, 60, 64), (120, 60, 40)])
def test_two_blocks_of_rows_to_a_cta(dit, heads, kv_heads, dim, frame, prefix):
    """Short documents beside a long one, in items that stay whole: last blocks that are lone or not full."""
    b = Batch(dit, [300, 1, 129, 256, 77, 2200], heads, kv_heads, dim, frame, prefix, train=False)
    assert b.plan.info.row_blocks == 2 and b.plan.info.items[1] == 0
    b.forward()
    b.check()


@pytest.mark.parametrize("heads,kv_heads,dim", [(3, 3, 64), (6, 2, 64), (14, 1, 40), (32, 1, 8), (6, 2, 128), (20, 20, 72)])
def test_one_block_of_rows_to_a_cta(dit, heads, kv_heads, dim):
    """Short documents: no key, one, tiles of all but one and of one more, as many as the ring has and some more."""
    queries = [5, 1, 127, 128, 129, 300, 0, 2, 260]
    keys = [0, 1, 127, 256, 129, 1290, 7, 2048, 260]
    for frame, prefix in ((0, 0), (1, 0), (50, 33)):
        b = Batch(dit, queries * 8, heads, kv_heads, dim, frame, prefix, kv_lengths=keys * 8, train=frame == 50)
        assert b.plan.info.row_blocks == 1
        b.forward()
        if frame == 50:
            b.backward()
        b.check()


@pytest.mark.parametrize("c", [
    # queries, keys, heads, kv_heads, dim, frame, prefix, room
    ([1, 1, 1, 1], [700, 1, 65, 3000], 16, 4, 128, 1, 0, 3100),
    ([1], [5000], 1, 1, 64, 1, 0, 5003),
    ([135], [900], 3, 3, 64, 135, 90, 1000),
    ([3, 0, 7], [1300, 5, 129], 6, 1, 64, 4, 2, 1400),
    ([5, 2], [3, 0], 2, 2, 64, 1, 0, 10),          # fewer keys than queries: the first queries see none
    ([6], [2], 2, 1, 128, 2, 1, 4),
    ([40], [0], 2, 2, 64, 0, 0, 4),                # no keys at all
    ([200], [77], 3, 3, 64, 0, 0, 80),             # a few keys for many queries
    ([1, 1], [2000, 2000], 128, 1, 64, 1, 0, 2000),
])
def test_keys_in_a_cache(dit, c):
    queries, keys, heads, kv_heads, dim, frame, prefix, room = c
    for train in (False, True):
        b = Batch(dit, queries, heads, kv_heads, dim, frame, prefix, kv_lengths=keys, room=room, train=train)
        b.forward()
        if train:
            b.backward()
        b.check()


@pytest.mark.parametrize("dim", [40, 64, 128])
@pytest.mark.parametrize("queries,heads,kv_heads", [(1, 1, 1), (100, 2, 2), (9, 14, 1), (128, 1, 1), (129, 1, 1), (300, 1, 1)])
def test_pieces_of_one_block_of_rows(dit, queries, heads, kv_heads, dim):
    """Tiles that the halves of a CTA take in turn, of odd and even numbers, with a last one that is not whole; and items of two blocks."""
    for keys in (257, 2000, 5000 + queries):
        b = Batch(dit, [queries, 3], heads, kv_heads, dim, frame=7, prefix=5, kv_lengths=[keys, 700], room=keys + 20, train=False)
        b.forward()
        b.check()


def test_many_splits(dit):
    """Long keys of one head are cut among the SMs and joined."""
    b = Batch(dit, [3], 1, 1, 64, kv_lengths=[40000], train=False)
    assert b.plan.info.slots > 0
    b.forward()
    b.check()


@pytest.mark.parametrize("sharp", [0.0, 20.0, 200.0])
def test_flat_and_sharp_scores(dit, sharp):
    """All weights equal, and maxima that grow from tile to tile by far more than the exponent's range."""
    b = Batch(dit, [520], 2, 2, 64, sharp=sharp)
    b.forward(scale=0.5)
    b.backward(scale=0.5)
    q0 = b.q[:520].double()
    # scores of this size: fp32 leaves them off by 2^-22 of the sum of magnitudes, which the weights feel in full
    worst = (q0.abs().transpose(0, 1) @ b.k[:520].double().abs().permute(1, 2, 0)).amax() * 0.5 * 2.0 ** -22
    fine, R.FINE = R.FINE, R.FINE + float(worst)
    try:
        b.check(scale=0.5)
    finally:
        R.FINE = fine


def test_other_documents_do_not_reach_a_result(dit):
    """NaN and infinity in one document leave every bit of the others as it was."""
    lengths = [70, 200, 33]
    b = Batch(dit, lengths, 2, 1, 64)
    b.forward()
    b.backward()
    first = [t.clone() for t in (b.out, b.dq, b.dk, b.dv)]
    for t, bad in ((b.q, float("nan")), (b.k, float("inf")), (b.v, float("nan")), (b.dout, float("-inf"))):
        t[70:270] = bad
    b.forward()
    b.backward()
    for a, t in zip(first, (b.out, b.dq, b.dk, b.dv)):
        assert torch.equal(a[:70], t[:70]) and torch.equal(a[270:303], t[270:303])
    assert torch.isnan(b.out[70:270]).all() and torch.isnan(b.dv[70:270]).all()


def test_nan_stays_in_its_rows(dit):
    """Under a causal mask NaN in a query reaches that query's output alone."""
    b = Batch(dit, [200], 1, 1, 64, frame=1, train=False)
    b.forward()
    first = b.out.clone()
    b.q[77] = float("nan")
    b.forward()
    assert torch.isnan(b.out[77]).all()
    b.out[77] = first[77]
    assert torch.equal(b.out, first)


def test_same_bits_and_graph(dit):
    """Eager calls and a replay give the same bits, and a replay reads new inputs."""
    b = Batch(dit, [400, 77, 1300], 6, 2, 64, frame=50, prefix=11)
    b.forward()
    b.backward()
    names = ("out", "dq", "dk", "dv")
    first = [getattr(b, n).clone() for n in names]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward()
        b.backward()
    for n in names:
        getattr(b, n)[:1777] = 0
    graph.replay()
    assert all(torch.equal(a, getattr(b, n)) for a, n in zip(first, names))
    b.v[:1777] *= 2
    graph.replay()
    b.check()


def test_streams_share_nothing_but_inputs(dit):
    """Two batches of one plan on two streams at a time, each with its own scratch and workspace."""
    a = Batch(dit, [900, 300], 4, 4, 64, seed=1)
    b = Batch(dit, [900, 300], 4, 4, 64, seed=2)
    b.plan = a.plan
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a.forward()
        b.forward(stream=side)
        a.backward()
        b.backward(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    a.check()
    b.check()


@pytest.mark.parametrize("lengths,keys", [([0, 0], [5, 300]), ([0], [0]), ([4, 0], [0, 9])])
def test_documents_without_queries_or_keys(dit, lengths, keys):
    b = Batch(dit, lengths, 2, 1, 64, kv_lengths=keys, room=400)
    b.forward()
    b.backward()
    b.check()


@pytest.mark.parametrize("n,m", [(200, 200), (1, 9000)])  # whole items, and keys cut into pieces
def test_scores_of_minus_infinity_and_nan(dit, n, m):
    """A query whose scores are all -infinity gets NaN, as the formula's; one with some of them does not; NaN in a key reaches the
    queries that see it."""
    b = Batch(dit, [n], 1, 1, 64, kv_lengths=[m], room=m, train=False)
    assert (b.plan.info.slots > 0) == (n == 1)
    b.q[:n] = 1.0
    key = b.k[1:1 + m]
    key[7] = float("-inf")
    b.forward()
    assert torch.isfinite(b.out[:n]).all()
    key.fill_(float("-inf"))
    b.forward()
    assert torch.isnan(b.out[:n]).all()
    key.fill_(0.5)
    key[m // 3] = float("nan")
    b.forward()
    assert torch.isnan(b.out[:n]).all()


def test_wrong_table_entries_are_skipped(dit):
    """Entries that do not fit the plan write nothing and raise the status word."""
    for field, value in ((0, 10 ** 6), (1, 10 ** 6), (2, 10 ** 6), (3, 10 ** 6), (4, -1), (5, 10 ** 6), (6, -128), (7, -1), (8, 10 ** 6)):
        b = Batch(dit, [100, 60], 2, 2, 64)
        b.forward()
        good = b.out.clone()
        table = b.plan.table.view(-1)[: 16 * sum(b.plan.info.items)].view(-1, 16)
        table[:, field] = value
        b.out[:] = 7.0
        b.forward()
        assert (b.out == 7.0).all(), field
        b.backward()
        assert (b.dq == 5.0).all() and (b.dk == 5.0).all(), field
        assert dit.device_status(b.ws) == 1 << 1
        assert not torch.equal(good, b.out)


@pytest.mark.parametrize("row", [100, 10 ** 6, 2 ** 31 - 1])
def test_rows_behind_the_document_are_skipped(dit, row):
    """An entry whose own rows begin behind its document writes nothing, statistics included, and raises the status word."""
    b = Batch(dit, [100, 60], 2, 2, 64)
    b.forward()
    table = b.plan.table.view(-1)[: 16 * sum(b.plan.info.items)].view(-1, 16)
    table[:, 6] = row
    b.saved.fill_(255)
    b.scratch.fill_(255)
    b.out[:] = 7.0
    b.forward()
    b.backward()
    assert (b.out == 7.0).all() and (b.dq == 5.0).all() and (b.dk == 5.0).all() and (b.dv == 5.0).all()
    assert (b.saved == 255).all() and (b.scratch == 255).all()
    assert dit.device_status(b.ws) == 1 << 1


def test_entries_that_no_plan_makes_are_skipped(dit):
    """Queries' gradients that do not begin at a whole tile (their statistics would reach behind the last one), and tiles from the
    last to the first."""
    for row, begin, end in ((1, 0, 2), (127, 0, 2), (0, 1, 0)):
        b = Batch(dit, [128], 2, 2, 64)
        b.forward()
        first, n = sum(b.plan.info.items[:2]), b.plan.info.items[2]
        item = b.plan.table.view(-1)[16 * first: 16 * (first + n)].view(-1, 16)
        item[:, 6], item[:, 7], item[:, 8] = row, begin, end
        b.scratch.fill_(255)
        b.backward()
        assert (b.dq == 5.0).all() and (b.scratch == 255).all()
        assert dit.device_status(b.ws) == 1 << 1


@pytest.mark.parametrize("pieces", [0, -1])
def test_joins_of_no_piece_are_skipped(dit, pieces):
    b = Batch(dit, [3], 1, 1, 64, kv_lengths=[40000], train=False)
    assert b.plan.info.items[1] == 1
    item = b.plan.table.view(-1)[16 * b.plan.info.items[0]:].view(-1, 16)
    item[:, 8] = pieces
    b.forward()
    assert (b.out == 7.0).all()
    assert dit.device_status(b.ws) == 1 << 1


def test_pieces_that_nothing_joins_are_skipped(dit):
    """A plan without joins has no place for partial results: an entry that names one writes nothing and raises the status word."""
    b = Batch(dit, [100, 60], 2, 2, 64, train=False)
    assert b.plan.info.items[1] == 0
    table = b.plan.table.view(-1)[: 16 * b.plan.info.items[0]].view(-1, 16)
    table[:, 10] = 1  # without a partial result this asks for nothing
    b.forward()
    b.check()
    table[:, 9] = 0
    b.out[:] = 7.0
    b.forward()
    assert (b.out == 7.0).all()
    assert dit.device_status(b.ws) == 1 << 1


def test_offsets_past_32_bits(dit):
    """Keys and values far apart: offsets in elements pass 2^31."""
    n, stride = 34000, 65536
    cache = torch.empty(n * stride, dtype=BF16, device="cuda")
    k, v = (cache.as_strided((n, 1, 64), (stride, 64, 1), at) for at in (0, 64))
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(5, 1, 64, device="cuda", generator=g).to(BF16)
    k.copy_(torch.randn(n, 1, 64, device="cuda", generator=g))
    v.copy_(torch.randn(n, 1, 64, device="cuda", generator=g))
    plan = dit.AttentionPlan([2, 3], 1, 64, kv_lengths=[10, 300], kv_begins=[3, n - 300], training=True)
    ws, scratch, saved, out = dit.workspace(), dit.attention_scratch(plan), dit.attention_saved(plan), torch.empty_like(q)
    dit.attention(plan, q, k, v, out, scratch, ws, saved=saved)
    grad = torch.empty_like(cache)
    dk, dv = (grad.as_strided((n, 1, 64), (stride, 64, 1), at) for at in (0, 64))
    dq, dout = torch.empty_like(q), torch.randn(5, 1, 64, device="cuda", generator=g).to(BF16)
    dit.attention_backward(plan, q, k, v, out, dout, saved, dq, dk, dv, scratch, ws)
    for rows, keys in ((slice(0, 2), slice(3, 13)), (slice(2, 5), slice(n - 300, n))):
        o, p, bound = R.attention(q[rows, 0].double(), k[keys, 0].double(), v[keys, 0].double(), torch.ones(rows.stop - rows.start, keys.stop - keys.start, dtype=torch.bool, device="cuda"), 0.125)
        assert ((out[rows, 0].double() - o).abs() <= bound).all()
        grads = R.attention_grads(q[rows, 0].double(), k[keys, 0].double(), v[keys, 0].double(), p, o, dout[rows, 0].double(), 0.125)
        for got, (want, lim) in zip((dq[rows, 0], dk[keys, 0], dv[keys, 0]), grads):
            assert ((got.double() - want).abs() <= lim).all()
    assert dit.device_status(ws) == 0


def test_calls_back_to_back(dit):
    """Calls that follow one another without a pause, each on what a kernel just before has written, give the bits of an idle device:
    the kernel of dk and dv starts ahead of its predecessor's end."""
    b = Batch(dit, [900, 31, 500], 8, 4, 64, frame=70, prefix=9)
    n, start = 1431, [t.clone() for t in (b.q, b.k, b.dout)]

    def run(wait):
        for t, v in zip((b.q, b.k, b.dout), start):
            t.copy_(v)
        got = []
        for i in range(6):
            for t in (b.q, b.k, b.dout):
                t[:n].mul_(-0.75)
            if wait:
                torch.cuda.synchronize()
            b.forward()
            if wait:
                torch.cuda.synchronize()
            b.backward()
            if wait:
                torch.cuda.synchronize()
            got += [t[:n].clone() for t in (b.out, b.dq, b.dk, b.dv)]
        return got
    apart = run(True)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(apart, run(False)))


@pytest.mark.parametrize("dim", [64, 128])
def test_whoever_follows_finds_dq_complete(dit, dim):
    """Few queries over many keys: the kernel of dk and dv has little to do and runs beside a long one of dq.  What comes behind both
    on the stream, here the norms' gradients, reads all of dq."""
    b = Batch(dit, [128], 2, 2, dim, kv_lengths=[20000], tail=0)
    norm = dit.QKNorm(torch.rand(2, dim, device="cuda") + 0.5, "rms")
    got, want = torch.empty_like(b.q), torch.empty_like(b.q)
    b.forward()
    for _ in range(3):
        b.dq.fill_(5.0)
        b.backward()
        dit.qk_norm_rope_backward(b.q, None, b.dq, None, got, None, norm, None, None, None, None, b.ws)
        torch.cuda.synchronize()
        dit.qk_norm_rope_backward(b.q, None, b.dq, None, want, None, norm, None, None, None, None, b.ws)
        assert torch.equal(got, want)
    b.check()


@pytest.mark.parametrize("dim", [64, 128])
def test_whoever_follows_finds_dk_and_dv_complete(dit, dim):
    """Many queries over few keys: the kernel of dq has little to do beside a long one of dk and dv."""
    b = Batch(dit, [20000], 2, 2, dim, kv_lengths=[128], tail=0)
    norm = dit.QKNorm(torch.rand(2, dim, device="cuda") + 0.5, "rms")
    got, want = torch.empty_like(b.k), torch.empty_like(b.k)
    b.forward()
    for dx in (b.dk, b.dv):
        for _ in range(3):
            dx.fill_(5.0)
            b.backward()
            dit.qk_norm_rope_backward(b.k, None, dx, None, got, None, norm, None, None, None, None, b.ws)
            torch.cuda.synchronize()
            dit.qk_norm_rope_backward(b.k, None, dx, None, want, None, norm, None, None, None, None, b.ws)
            assert torch.equal(got, want)
    b.check()


def test_gradients_match_differences(dit):
    """The gradients against differences of the 64-bit formula, so that both could not share a mistake."""
    b = Batch(dit, [9, 20], 2, 1, 64, frame=3, prefix=4)
    b.forward()
    b.backward()
    n = 29
    leaves = [t[:n].double().clone().requires_grad_() for t in (b.q, b.k, b.v)]

    def loss(q, k, v):
        total, q0 = 0.0, 0
        for m in (9, 20):
            seen = R.visible(m, m, 3, 4, "cuda")
            for head in range(2):
                s = (q[q0:q0 + m, head] @ k[q0:q0 + m, 0].T) / 8.0
                p = torch.softmax(s.masked_fill(~seen, float("-inf")), 1)
                total = total + (p @ v[q0:q0 + m, 0] * b.dout[q0:q0 + m, head].double()).sum()
            q0 += m
        return total
    loss(*leaves).backward()
    for leaf, got in zip(leaves, (b.dq, b.dk, b.dv)):
        # bf16 operands and results: some 2^-8 of the largest entries
        assert (leaf.grad - got[:n].double()).abs().max() <= 4 * R.HALF * leaf.grad.abs().max()
        at, step = (5, 0, 7), 1e-5
        moved = []
        for sign in (1, -1):
            args = [t.detach().clone() for t in leaves]
            args[[i for i, t in enumerate(leaves) if t is leaf][0]][at] += sign * step
            moved.append(loss(*args))
        assert abs(float((moved[0] - moved[1]) / (2 * step) - leaf.grad[at])) < 1e-6


@pytest.mark.parametrize("keys,heads,dim", [(300, 2, 64), (5000, 2, 64), (300, 8, 128), (5000, 2, 128), (2200, 60, 64)])
def test_bounded_wait_in_every_form_of_the_forward_pass(dit, monkeypatch, keys, heads, dim):
    """One and two blocks of rows to a CTA, pieces, halves that take tiles in turn."""
    b = Batch(dit, [300, 64], heads, heads, dim, kv_lengths=[keys, 64], train=False)
    monkeypatch.setenv("DIT6_TEST_STALL_PRODUCER", "1")
    b.forward()
    assert dit.device_status(b.ws) & (1 << 5)
    dit.clear_device_status(b.ws)
    monkeypatch.delenv("DIT6_TEST_STALL_PRODUCER")
    b.out[:364] = 0
    b.forward()
    b.check()


def test_bounded_wait_reports_timeout_and_recovers(dit, monkeypatch):
    b = Batch(dit, [300, 64], 2, 2, 64)
    monkeypatch.setenv("DIT6_TEST_STALL_PRODUCER", "1")
    b.forward()
    assert dit.device_status(b.ws) & (1 << 5)
    dit.clear_device_status(b.ws)
    b.backward()
    assert dit.device_status(b.ws) & (1 << 5)
    dit.clear_device_status(b.ws)
    monkeypatch.delenv("DIT6_TEST_STALL_PRODUCER")
    b.out[:364], b.dq[:364], b.dk[:364], b.dv[:364] = 0, 0, 0, 0
    b.forward()
    b.backward()
    b.check()
