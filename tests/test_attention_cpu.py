"""Host side of the norms and the attention, without a GPU: the rotation's table, the plan's cuts and what is refused."""
import copy
import ctypes
import decimal
import math
import os
import random

import pytest
import torch

import attention_reference as R

INVALID, ALIGNMENT, UNSUPPORTED = 1, 2, 3


@pytest.fixture(scope="module")
def dit():
    import int8_mixed_precision_gb300 as d
    from int8_mixed_precision_gb300 import _lib, build
    if not os.path.exists(_lib.library_path()):
        try:
            build.build_library()
        except RuntimeError as e:
            pytest.skip(str(e))
    return d


# ----------------------------------------------------------------------------------------
# the rotation's table
# ----------------------------------------------------------------------------------------

def test_rotary_table_holds_turns(dit):
    rot = dit.Rotary((16, 24, 24), 64, theta=10000.0, scale=(1.0, 0.375, 7.5), device="cpu")
    words = rot.table.view(-1, 2)
    assert words.shape[0] == 32
    p = 0
    for a, (d, s) in enumerate(zip((16, 24, 24), (1.0, 0.375, 7.5))):
        for i in range(d // 2):
            turns = s * 10000.0 ** (-2 * i / d) / (2 * math.pi) % 1.0
            held = (int(words[p, 0]) & (2 ** 64 - 1)) / 2 ** 64
            assert abs(held - turns) < 2.0 ** -49
            assert int(words[p, 1]) & 0xffffffff == a
            p += 1


@pytest.mark.parametrize("theta", [10000.0, 500000.0, 1e8, 1.0, 0.3, 1e300])
@pytest.mark.parametrize("scales", [(1.0, 0.375, 7.5), (100.0, 1 / 3, -2.5), (1e6, 1e-9, 2.0 ** 30)])
def test_rotary_table_against_long_arithmetic(dit, theta, scales):
    """A position has 32 bits and an angle is promised to 2^-21 of a radian, so a turn's fraction is to be right to 2^-55 at
    least; 64 bits hold it to 2^-64.  Against 80 decimal digits."""
    decimal.getcontext().prec = 80
    tau = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534")
    dims = (16, 24, 216)
    words = dit.Rotary(dims, 256, theta=theta, scale=scales, device="cpu").table.view(-1, 2).tolist()
    p = 0
    for d, s in zip(dims, scales):
        for i in range(d // 2):
            frequency = decimal.Decimal(s) * decimal.Decimal(theta) ** (decimal.Decimal(-2 * i) / d)
            off = (frequency / tau - decimal.Decimal(words[p][0] & (2 ** 64 - 1)) / 2 ** 64) % 1
            off = min(abs(off), 1 - abs(off))
            assert abs(frequency) > 2 ** 30 or off <= decimal.Decimal(2) ** -63, (d, i, float(off * 2 ** 64))
            p += 1


@pytest.mark.parametrize("theta", [5e-324, 1e-310, 1e-300, 1.7e308])
def test_rotary_table_of_extreme_bases(dit, theta):
    """Bases without low parts of their own, and powers of them past the range of doubles under a small scale."""
    decimal.getcontext().prec = 80
    words = dit.Rotary((64,), 64, theta=theta, scale=1e-12, device="cpu").table.view(-1, 2).tolist()
    for i in range(3):
        turns = decimal.Decimal(1e-12) * decimal.Decimal(theta) ** (decimal.Decimal(-2 * i) / 64) / decimal.Decimal(2 * math.pi)
        off = (turns - decimal.Decimal(words[i][0] & (2 ** 64 - 1)) / 2 ** 64) % 1
        assert min(abs(off), 1 - abs(off)) <= 2.0 ** -40 * float(turns) + 2.0 ** -63


def test_rotary_refuses_frequencies_without_bounds(dit):
    for theta, scale in ((1e-300, 1e200), (1e-300, -1e200)):
        with pytest.raises(dit.DitError):
            dit.Rotary((64,), 64, theta=theta, scale=scale, device="cpu")
    assert dit.Rotary((64,), 64, theta=1e-300, device="cpu").table.numel() == 64


@pytest.mark.parametrize("kw", [dict(dims=(16, 23, 25)), dict(dims=(32, 48)), dict(dims=(8,) * 5), dict(dims=()), dict(dims=(64,), scale=(1.0, 1.0)),
                                dict(dims=(-2, 4)), dict(dims=(12,), interleaved=False), dict(dims=(64,), theta=0.0), dict(dims=(64,), theta=math.inf),
                                dict(dims=(64,), scale=math.nan)])
def test_rotary_refusals(dit, kw):
    with pytest.raises(dit.DitError):
        dit.Rotary(head_dim=64, device="cpu", **kw)


def test_norm_refusals(dit):
    for params, kind, eps in ((torch.ones(2, 64), "layer", 1e-6), (torch.ones(4, 64), "rms", 1e-6), (torch.ones(2, 64), "other", 1e-6),
                              (torch.ones(2, 64).double(), "rms", 1e-6), (torch.ones(64, 2).T, "rms", 1e-6), (torch.ones(2, 64), "rms", -1.0),
                              (torch.ones(2, 64), "rms", math.nan)):
        with pytest.raises(dit.DitError):
            dit.QKNorm(params, kind, eps)


# ----------------------------------------------------------------------------------------
# the plan
# ----------------------------------------------------------------------------------------

def lists(plan):
    """The four lists of items, each (document's q0, queries, k0, keys, prefix, first padded tile; row, begin, end, slot, turns), and the buckets."""
    i, t = plan.info, plan.table.tolist()
    at, out = 0, []
    for n in i.items:
        out.append([t[at + 16 * k:at + 16 * k + 11] for k in range(n)])
        at += 16 * n
    assert at == i.table_ints
    buckets = [[list(i.bucket[k][2 * b:2 * b + 2]) for b in range(n)] for k, n in enumerate(i.buckets)]
    return out, buckets


def check_plan(dit, queries, keys, heads, kv_heads, dim, frame, prefix):
    plan = dit.AttentionPlan(queries, heads, dim, kv_heads=kv_heads, kv_lengths=keys, frame=frame, prefix=prefix, training=True, device="cpu")
    found, buckets = lists(plan)
    # each document's statistics begin at a multiple of 128
    places, q0, k0, at = {}, 0, 0, 0
    for i, (n, m, pre) in enumerate(zip(queries, keys, [prefix] * len(keys))):
        places[(q0, n, k0 if m else 0, m, pre, at)] = i
        q0, k0, at = q0 + n, k0 + m, at + -(-n // 128)
    assert plan.info.padded_rows == at * 128
    fwd, joins, gq, gk = ([(places[tuple(item[:6])], *item[6:]) for item in items] for items in found)
    cols, rt, back = 128, 128 // (heads // kv_heads), 64
    wide = plan.info.row_blocks * rt
    assert plan.info.row_blocks in ((1,) if dim > 64 else (2,) if joins else (1, 2))
    assert plan.q_rows == sum(queries)
    for items, found in zip((fwd, joins, gq, gk), buckets):  # the buckets are the list, in order
        at = 0
        for first, count in found:
            assert first == at and count > 0
            at += count
        assert at == len(items)
    seen = [R.visible(n, m, frame, prefix) for n, m in zip(queries, keys)]
    # forward: every query once, or in pieces that a join adds up; each pair that is seen lies in exactly one piece
    met = [torch.zeros(n, m, dtype=torch.int32) for n, m in zip(queries, keys)]
    rows = [torch.zeros(n, dtype=torch.int32) for n in queries]
    slots = {}
    for doc, row0, begin, end, slot, turns in fwd:
        part = slice(row0, min(queries[doc], row0 + wide))
        met[doc][part, begin * cols:end * cols] += 1
        assert end * cols < keys[doc] + cols
        if slot < 0:
            rows[doc][part] += 1
        else:
            n = part.stop - part.start
            # the halves of a CTA that take a lone block's tiles in turn leave a partial result each
            assert turns == (dim <= 64 and queries[doc] - row0 <= rt)
            slots[slot] = (doc, row0, n, begin, end, 2 if turns else 1)
            assert slot + n * (2 if turns else 1) <= plan.info.slots
    used = torch.zeros(plan.info.slots, dtype=torch.int32)
    for doc, row0, first, pieces, n, _ in joins:
        rows[doc][row0:row0 + n] += 1
        at, k = 0, 0
        while k < pieces:
            d, r, c, begin, end, halves = slots[first + k * n]
            assert (d, r, c, begin) == (doc, row0, n, at) and end > begin
            at = end
            used[first + k * n:first + (k + halves) * n] += 1
            k += halves
        assert k == pieces
    assert (used == 1).all()
    for n, m, r, s in zip(queries, keys, rows, seen):
        assert (r == 1).all()
    assert all((m <= 1).all() and (m[s] == 1).all() for m, s in zip(met, seen))
    # gradients: every query and key once, with all that it meets
    for items, of_keys in ((gq, False), (gk, True)):
        whole = [torch.zeros(m if of_keys else n, dtype=torch.int32) for n, m in zip(queries, keys)]
        for doc, row0, begin, end, *_ in items:
            s = seen[doc].T if of_keys else seen[doc]
            part = slice(row0, row0 + 128)
            whole[doc][part] += 1
            left = s[part].clone()
            left[:, begin * back:end * back] = False
            assert not left.any()
            assert end * back < s.shape[1] + back
        assert all((w == 1).all() for w in whole)
    return plan


@pytest.mark.parametrize("c", [
    ([300, 0, 17], [300, 0, 17], 4, 4, 64, 0, 0),
    ([300, 1, 517], [300, 1, 517], 6, 2, 128, 1, 0),
    ([1, 1, 1], [4000, 1, 333], 8, 1, 128, 1, 0),
    ([1350], [8326], 30, 30, 64, 1350, 226),
    ([5, 2, 9], [3, 0, 1], 2, 2, 64, 1, 0),
    ([40, 3], [0, 5], 2, 2, 64, 0, 0),
    ([200], [900], 12, 4, 96, 37, 50),
    ([7], [2000], 128, 1, 64, 0, 0),
    ([], [], 1, 1, 64, 0, 0),
])
def test_plan_covers_every_pair_once(dit, c):
    check_plan(dit, *c)


def test_items_that_fill_whole_rounds_stay_whole(dit):
    """5 of 6 items of 30 heads are 150 CTAs, a round of the SMs; the sixth alone, one block of rows, is cut and joined."""
    plan = check_plan(dit, [1350], [8326], 30, 30, 64, 0, 0)
    fwd, joins = lists(plan)[0][:2]
    whole = [item for item in fwd if item[9] < 0]
    assert [item[6] for item in joins] == [1280] and len(whole) == 5
    assert all(item[7] == 0 and item[8] == 66 for item in whole)
    assert all(item[10] == 1 for item in fwd if item[9] >= 0)


@pytest.mark.parametrize("keys,dim,blocks", [(2048, 64, 1), (2049, 64, 2), (5000, 72, 1), (1, 8, 1)])
def test_items_of_one_block_of_rows(dit, keys, dim, blocks):
    plan = check_plan(dit, [129] * 40, [keys] * 40, 30, 30, dim, 0, 0)
    assert plan.info.row_blocks == blocks and plan.info.items[0] == 40 * (2 if blocks == 1 else 1) and plan.info.items[1] == 0


def test_tables_of_any_size(dit):
    """No entry, and more of them than a first buffer holds."""
    assert dit.AttentionPlan([0, 0], 2, 64, device="cpu").table.numel() == 0
    plan = check_plan(dit, [3] * 700, [3] * 700, 2, 2, 64, 1, 0)
    assert plan.table.numel() == plan.info.table_ints == 16 * 3 * 700


def test_plans_of_random_batches(dit):
    rng = random.Random(0)
    for _ in range(25):
        n = rng.randint(1, 6)
        queries = [rng.choice([0, 1, rng.randint(2, 900)]) for _ in range(n)]
        keys = [rng.choice([q, q + rng.randint(0, 700), rng.randint(0, 300)]) for q in queries]
        kv = rng.randint(1, 4)
        frame = rng.choice([0, 1, rng.randint(2, 100)])
        check_plan(dit, queries, keys, kv * rng.choice([1, 2, 3]), kv, 8 * rng.randint(1, 16), frame, rng.choice([0, rng.randint(1, 90)]) if frame else 0)


def test_numbers_of_other_libraries(dit):
    """One prefix or scale for all is a number, whoever made it."""
    import numpy as np
    plans = [dit.AttentionPlan([10, 20], 2, 64, frame=2, prefix=p, device="cpu").table for p in (3, np.int64(3), torch.tensor(3), [3, 3], np.array([3, 3]))]
    assert all(torch.equal(plans[0], t) for t in plans)
    tables = [dit.Rotary((32, 32), 64, scale=s, device="cpu").table for s in (2.0, np.float32(2.0), torch.tensor(2.0), [2, 2], np.array([2.0, 2.0]))]
    assert all(torch.equal(tables[0], t) for t in tables)


def test_few_rows_are_split_over_the_keys(dit):
    plan = dit.AttentionPlan([1], 4, 128, kv_heads=1, kv_lengths=[20000], frame=1, device="cpu")
    assert plan.info.items[0] > 50 and plan.info.items[1] == 1
    whole = dit.AttentionPlan([17776], 30, 64, device="cpu")  # enough work for every SM
    assert whole.info.slots == 0 and whole._scratch_bytes == 0


def test_plan_refusals(dit):
    ok = dict(lengths=[5, 6], heads=4, dim=64, device="cpu")
    dit.AttentionPlan(**ok)
    for change in (dict(lengths=[-1, 3]), dict(kv_heads=3), dict(dim=68), dict(dim=136), dict(dim=0), dict(heads=0), dict(heads=8192), dict(frame=-1),
                   dict(prefix=3), dict(prefix=[1, 2]), dict(frame=2, prefix=[1]), dict(frame=2, prefix=-1), dict(kv_lengths=[5]), dict(kv_begins=[0]),
                   dict(kv_begins=[0, -1]), dict(lengths=[2 ** 31 - 1, 5]), dict(lengths=[2 ** 31, 5]), dict(kv_lengths=[2 ** 31 - 300, 600]),
                   dict(heads=129 * 2, kv_heads=2), dict(frame=2 ** 31), dict(training=True, kv_lengths=[5, 6], kv_begins=[0, 4])):
        with pytest.raises(dit.DitError):
            dit.AttentionPlan(**{**ok, **change})
    dit.AttentionPlan(**{**ok, "kv_lengths": [5, 6], "kv_begins": [0, 4]})  # shared keys serve
    with pytest.raises(dit.DitError):
        copy.copy(dit.AttentionPlan(**ok))
    with pytest.raises(dit.DitError):
        copy.deepcopy(dit.Rotary((8,), 64, device="cpu"))


# ----------------------------------------------------------------------------------------
# refusals of the calls (nothing is launched)
# ----------------------------------------------------------------------------------------

class Heads(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def heads(ptr, n, dim, stride=None, head=None):
    return Heads(ptr, n * dim if stride is None else stride, dim if head is None else head, n, 0)


def test_attention_refusals(dit):
    L, A = dit.lib(), 1 << 20
    plan = dit.AttentionPlan([300], 4, 64, kv_heads=2, training=True, device="cpu")

    def call(backward=False, p=plan.info, table=A, ws=A, ws_bytes=1 << 16, scale=0.125, saved=A, saved_bytes=1 << 30, scratch=A, scratch_bytes=1 << 30, **views):
        v = {n: heads(A, 4, 64) for n in ("q", "out", "dout", "dq")}
        v.update({n: heads(A, 2, 64) for n in ("k", "v", "dk", "dv")})
        v.update(views)
        names = ("q", "k", "v", "out") + (("dout", "dq", "dk", "dv") if backward else ())
        f = L.dit_attention_backward if backward else L.dit_attention
        return f(ctypes.byref(p) if p is not None else None, table, *(ctypes.byref(v[n]) if v[n] is not None else None for n in names), scale, saved, saved_bytes,
                 scratch, scratch_bytes, ws, ws_bytes, None)
    for back in (False, True):
        assert call(back, p=None) == INVALID
        assert call(back, table=None) == INVALID
        assert call(back, table=A + 4) == ALIGNMENT
        assert call(back, ws=None) == INVALID
        assert call(back, ws=A + 16) == ALIGNMENT
        assert call(back, ws_bytes=100) == INVALID
        for scale in (0.0, -1.0, math.inf, math.nan):
            assert call(back, scale=scale) == INVALID
        assert call(back, saved_bytes=plan._saved_bytes - 1) == INVALID
        assert call(back, scratch_bytes=plan._scratch_bytes - 1) == INVALID
        assert call(back, scratch=None) == INVALID
        for name in ("q", "k", "v", "out") + (("dout", "dq", "dk", "dv") if back else ()):
            n = 2 if name in ("k", "v", "dk", "dv") else 4
            assert call(back, **{name: None}) == INVALID
            assert call(back, **{name: heads(None, n, 64)}) == INVALID
            assert call(back, **{name: heads(A, n + 1, 64)}) == INVALID
            assert call(back, **{name: heads(A + 8, n, 64)}) == ALIGNMENT
            assert call(back, **{name: heads(A, n, 64, stride=n * 64 + 4)}) == ALIGNMENT
            assert call(back, **{name: heads(A, n, 64, head=68)}) == ALIGNMENT
            assert call(back, **{name: heads(A, n, 64, stride=0)}) == INVALID
            assert call(back, **{name: heads(A, n, 64, head=0)}) == INVALID
            assert call(back, **{name: heads(A, n, 64, stride=1 << 31)}) == UNSUPPORTED
    serving = dit.AttentionPlan([300], 4, 64, kv_heads=2, device="cpu")
    assert call(True, p=serving.info) == INVALID
    assert call(False, p=serving.info) == INVALID  # saved goes with training plans
    from int8_mixed_precision_gb300.block_attention import _Plan
    for field, value in (("heads", 3), ("dim", 72 + 4), ("dim", 256), ("table_ints", 1), ("slots", -1), ("slots", 500), ("q_rows", -1), ("padded_rows", 1), ("saved_bytes", 0)):
        bad = _Plan.from_buffer_copy(plan.info)
        setattr(bad, field, value)
        assert call(p=bad) == INVALID, field


@pytest.mark.parametrize("keys,dim,good", [([3000], 64, (2,)), ([300] * 400, 64, (1, 2)), ([300] * 400, 128, (1,))])
def test_plans_have_the_blocks_of_rows_that_kernels_have(dit, keys, dim, good):
    """Pieces of up to 64 dimensions are of two blocks, whole items of one or two, and more dimensions have one."""
    L, A, n = dit.lib(), 1 << 20, len(keys)
    plan = dit.AttentionPlan([3] * n, 4, dim, kv_lengths=keys, device="cpu")
    assert (plan.info.items[1] > 0) == (n == 1) and plan.info.row_blocks in good
    view = ctypes.byref(heads(A, 4, dim))
    for blocks in (-1, 0, 1, 2, 3):
        p = type(plan.info).from_buffer_copy(plan.info)
        p.row_blocks = blocks
        # what passes this check fails at the table's alignment
        status = L.dit_attention(ctypes.byref(p), A + 4, view, view, view, view, 0.1, None, 0, A, 1 << 40, A, 1 << 16, None)
        assert status == (ALIGNMENT if blocks in good else INVALID), blocks


def test_norm_call_refusals(dit):
    L, A = dit.lib(), 1 << 20
    from int8_mixed_precision_gb300.block_attention import _Rotary

    def call(backward=False, tokens=10, dim=64, norm=1, params=A, eps=1e-6, rot=_Rotary(A, 32, 3, 1, 0), positions=A, dparams=A, scratch=A, scratch_bytes=1 << 30,
             ws=A, ws_bytes=1 << 16, **views):
        v = {n: heads(A, 4, 64) for n in ("q", "q_out", "dq_out", "dq")}
        v.update({n: heads(A, 2, 64) for n in ("k", "k_out", "dk_out", "dk")})
        v.update(views)
        names = ("q", "k", "dq_out", "dk_out", "dq", "dk") if backward else ("q", "k", "q_out", "k_out")
        args = (*(ctypes.byref(v[n]) if v[n] is not None else None for n in names), tokens, dim, norm, params, eps, ctypes.byref(rot) if rot is not None else None, positions)
        return L.dit_qk_norm_rope_backward(*args, dparams, scratch, scratch_bytes, ws, ws_bytes, None) if backward else L.dit_qk_norm_rope(*args, None)
    for back in (False, True):
        for change in (dict(tokens=-1), dict(dim=0), dict(norm=3), dict(norm=-1), dict(params=None), dict(eps=-1.0), dict(eps=math.nan), dict(q=None),
                       dict(rot=_Rotary(A, 33, 3, 1, 0)), dict(rot=_Rotary(A, 32, 5, 1, 0)), dict(rot=_Rotary(A, 32, 0, 1, 0)), dict(rot=_Rotary(None, 32, 3, 1, 0)),
                       dict(positions=None), dict(q=heads(None, 4, 64)), dict(k=None)):
            assert call(back, **change) == INVALID, change
        for change in (dict(dim=60), dict(dim=264), dict(rot=_Rotary(A, 30, 3, 0, 0))):
            assert call(back, **change) == UNSUPPORTED, change
        for change in (dict(params=A + 2), dict(positions=A + 2), dict(rot=_Rotary(A + 8, 32, 3, 1, 0)), dict(q=heads(A + 8, 4, 64)), dict(k=heads(A, 2, 64, stride=132))):
            assert call(back, **change) == ALIGNMENT, change
    for change in (dict(ws=None), dict(ws_bytes=3), dict(scratch=None), dict(scratch_bytes=100), dict(norm=0)):
        assert call(True, **change) == INVALID, change
    assert call(True, ws=A + 16) == ALIGNMENT
    assert call(False, tokens=0) == 0  # nothing to do


def test_outputs_whose_heads_overlap_are_refused(dit):
    """Threads would write over one another.  What passes the check of the views fails at the alignment of a buffer behind it."""
    L, A, rng = dit.lib(), 1 << 20, random.Random(4)

    def norm(back, v, n, dim, tokens):
        x = ctypes.byref(heads(A, n, dim))
        args = (tokens, dim, 0, None, 0.0, None, None)
        if back:
            return L.dit_qk_norm_rope_backward(x, None, x, None, ctypes.byref(v), None, *args, None, None, 0, A + 16, 1 << 16, None)
        return L.dit_qk_norm_rope(x, None, ctypes.byref(v), None, *args, None)

    def attend(v, n, dim, tokens, name=None):
        plan = dit.AttentionPlan([tokens], n, dim, training=True, device="cpu")
        views = {k: ctypes.byref(heads(A, n, dim)) for k in ("q", "k", "v", "out") + (() if name == "out" else ("dout", "dq", "dk", "dv"))}
        views[name] = ctypes.byref(v)
        f = L.dit_attention if name == "out" else L.dit_attention_backward
        return f(ctypes.byref(plan.info), A + 4, *views.values(), 0.1, A, 1 << 30, A, 1 << 30, A, 1 << 16, None)
    seen = set()
    for _ in range(400):
        n, tokens, dim = rng.randint(1, 5), rng.randint(1, 6), 8 * rng.randint(1, 3)
        token, head = (8 * rng.randint(-20, 20) for _ in range(2))
        at = sorted((t * token if tokens > 1 else 0) + (h * head if n > 1 else 0) for t in range(tokens) for h in range(n))
        apart = all(b - a >= dim for a, b in zip(at, at[1:]))
        seen.add(apart)
        v = heads(A, n, dim, token, head)
        assert norm(True, v, n, dim, tokens) == (ALIGNMENT if apart else INVALID)
        if not apart:
            assert norm(False, v, n, dim, tokens) == INVALID
        if token > 0 and head > 0:  # the others are refused in any case
            for name in ("out", "dq", "dk", "dv"):
                assert attend(v, n, dim, tokens, name) == (ALIGNMENT if apart else INVALID)
    assert seen == {True, False}
    big = 1 << 62  # products of strides past 64 bits
    assert norm(True, heads(A, 4, 64, big, -big), 4, 64, 3) == INVALID and norm(True, heads(A, 1, 64, 0, 0), 1, 64, 1) == ALIGNMENT


def test_buffers_that_share_memory_are_refused(dit):
    """What a call keeps, its scratch and its workspace: the scratch of the backward pass would be written over what it reads."""
    L, A = dit.lib(), 1 << 20
    plan = dit.AttentionPlan([300, 7], 4, 64, training=True, device="cpu")
    view, n = ctypes.byref(heads(A, 4, 64)), plan._saved_bytes
    assert n == 4 * 4 * 512 and plan._scratch_bytes >= n

    def attend(saved, scratch, ws):
        rest = (0.1, saved, 1 << 30, scratch, 1 << 30, ws, 1 << 16, None)
        back = L.dit_attention_backward(ctypes.byref(plan.info), A, *[view] * 8, *rest)
        return {back, L.dit_attention(ctypes.byref(plan.info), A, *[view] * 4, *rest)}
    far = 1 << 24
    for saved, scratch, ws in ((far, far, 2 * far), (far, far + n - 32, 2 * far), (far + plan._scratch_bytes - 32, far, 2 * far), (far, 2 * far, far + n - 32),
                               (far + 65536 - 32, 2 * far, far), (far, 2 * far, 2 * far)):
        assert attend(saved, scratch, ws) == {INVALID}, (saved, scratch, ws)

    def norm(params=far, dparams=2 * far, scratch=3 * far, ws=4 * far, positions=5 * far):
        from int8_mixed_precision_gb300.block_attention import _Rotary
        rot = _Rotary(A, 32, 3, 1, 0)
        return L.dit_qk_norm_rope_backward(*[view] * 6, 10, 64, 2, params, 1e-6, ctypes.byref(rot), positions, dparams, scratch, 1 << 30, ws, 1 << 16, None)
    for change in (dict(dparams=3 * far), dict(dparams=3 * far - 4 * 4 * 64 + 4), dict(params=3 * far), dict(ws=3 * far), dict(ws=2 * far), dict(positions=3 * far),
                   dict(positions=3 * far - 116)):
        assert norm(**change) == INVALID, change


def test_views_that_share_memory_are_found(dit):
    from int8_mixed_precision_gb300.block_attention import _meet

    def view(t):
        at, (n, h, d), (row, head, _) = t.data_ptr(), t.shape, t.stride()
        return at, row, head, h, at + 2 * ((n - 1) * row + (h - 1) * head + d) if n else at

    def meet(a, b):
        got = _meet(view(a), view(b), a.shape[2])
        assert got == _meet(view(b), view(a), a.shape[2])
        return got
    x = torch.empty(10, 7, 8, dtype=torch.bfloat16)
    assert not meet(x[:, :3], x[:, 3:]) and meet(x[:, :4], x[:, 3:]) and meet(x, x)
    assert not meet(x[:5], x[5:]) and meet(x[:6], x[5:])
    y = torch.empty(10, 4, 3, 8, dtype=torch.bfloat16)  # query, key and value of a head side by side
    assert not meet(y[:, :, 0], y[:, :, 1]) and not meet(y[:, :, 2], y[:, :, 0]) and meet(y[:, :, 1], y[:, :, 1])
    assert not meet(y[:, 1:, 0], y[:, :, 1]) and meet(y[:, :1, 1], y[:, :, 1])
    z = torch.empty(10, 7, 8, dtype=torch.bfloat16)
    assert not meet(x, z) and not meet(x[:0], x)


def test_views_that_share_no_memory_are_not_refused(dit):
    """Against the addresses themselves: buffers whose heads lie in front of their tokens, and views of any strides in one buffer."""
    from int8_mixed_precision_gb300.block_attention import _meet

    def view(at, rows, heads, dim, row, head):  # as the calls describe a tensor
        row, head = row if rows > 1 else heads * dim, head if heads > 1 else dim
        return at, row, head, heads, at + 2 * ((rows - 1) * row + (heads - 1) * head + dim)

    def places(at, rows, heads, dim, row, head):
        return {at // 2 + t * row + h * head + i for t in range(rows) for h in range(heads) for i in range(dim)}
    # [heads, 3, tokens, dim]: query, key and value of each head behind one another
    t, h, d = 50, 6, 64
    three = [view(2 * i * t * d, t, h, d, d, 3 * t * d) for i in range(3)]
    assert not any(_meet(three[i], three[j], d) for i in range(3) for j in range(3) if i != j) and all(_meet(v, v, d) for v in three)
    assert _meet(three[0], view(2 * (t - 1) * d, t, h, d, d, 3 * t * d), d)
    rng, found = random.Random(7), {}
    for _ in range(20000):
        dim, row, head = 8 * rng.randint(1, 2), 8 * rng.randint(1, 24), 8 * rng.randint(1, 24)
        same = rng.random() < 0.7
        a = (0, rng.randint(1, 5), rng.randint(1, 5), dim, row, head)
        b = (16 * rng.randint(0, 40), rng.randint(1, 5), rng.randint(1, 5), dim, *((row, head) if same else (8 * rng.randint(1, 24), 8 * rng.randint(1, 24))))
        truth, got = bool(places(*a) & places(*b)), _meet(view(*a), view(*b), dim)
        assert got == _meet(view(*b), view(*a), dim)
        assert got or not truth, (a, b)
        if same and row >= dim:
            assert got == truth, (a, b)
        found[same, truth] = found.get((same, truth), 0) + 1
    assert len(found) == 4


def test_host_tensors_are_refused(dit):
    x = torch.zeros(4, 6, 64, dtype=torch.bfloat16)
    with pytest.raises(dit.DitError):
        dit.qk_norm_rope(x[:, :2], x[:, 2:4], x[:, :2], x[:, 2:4])
    plan = dit.AttentionPlan([4], 2, 64, device="cpu")
    with pytest.raises(dit.DitError):
        dit.attention(plan, x[:, :2], x[:, 2:4], x[:, 4:], torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.empty(0), torch.empty(0))
