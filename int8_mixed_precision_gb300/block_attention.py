"""Attention of a block: norms of queries and keys with the position rotation, and softmax attention.

``qk_norm_rope`` and ``attention`` with their backward passes are the calls of the C ABI one for one;
``Rotary``, ``QKNorm`` and ``AttentionPlan`` hold what a program keeps for all blocks and steps, and
``RoutedAttention`` puts the calls between a block's QKV and output projections.  Argument marshalling and
host-side checks only: the formulas, layouts and roundings are those of ``include/dit6.h``.
"""
from __future__ import annotations

import ctypes
import math
import struct
import threading

import torch

from . import ROUTE_BF16, ROUTE_INT8, DitError, _bias_ok, _check, _dt, _p, _same_device
from ._lib import lib
from .adapters import raw_stream

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
NORMS = {None: 0, "rms": 1, "layer": 2}
MAX_AXES = 4


class _Rotary(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("pairs", ctypes.c_int32), ("axes", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _Plan(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int64) for name in ("q_rows", "k_rows", "padded_rows", "table_ints", "saved_bytes", "scratch_bytes")] + \
        [(name, ctypes.c_int32) for name in ("documents", "heads", "kv_heads", "dim", "frame", "training", "slots")] + \
        [("items", ctypes.c_int32 * 4), ("buckets", ctypes.c_int32 * 4), ("bucket", ctypes.c_int32 * 32 * 4), ("row_blocks", ctypes.c_int32)]


# ----------------------------------------------------------------------------------------
# checks of a call, one pass over each tensor's properties: a short call's kernel takes a few microseconds
# ----------------------------------------------------------------------------------------

class _Views(threading.local):
    """Where a thread's call lays out its dit_heads_t structures: (pointer, token stride, head stride, heads, 0) each."""
    MOST = 8

    def __init__(self):
        self.room = ctypes.create_string_buffer(32 * self.MOST)
        base = ctypes.addressof(self.room)
        self.at = tuple(base + 32 * i for i in range(self.MOST))


_views = _Views()
_pack = tuple(struct.Struct("=" + "Qqqii" * n).pack_into for n in range(_Views.MOST + 1))


def _lay(*views):
    """The addresses of the views' structures, valid until the thread's next call; None stays None."""
    there = [v for v in views if v is not None]
    flat = []
    for v in there:
        flat += v[:4]
        flat.append(0)
    _pack[len(there)](_views.room, 0, *flat)
    if len(there) == len(views):
        return _views.at[:len(views)]
    at = iter(_views.at)
    return tuple(None if v is None else next(at) for v in views)


def _view(t, rows, heads, dim, what, index, exact=False):
    """`t` as [tokens, heads, dim] with at least `rows` tokens (exactly, if `exact`): pointer, strides, heads, and the end of
    the memory that `rows` tokens span."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim or shape[0] < rows or (exact and shape[0] != rows):
        raise DitError(f"{what}: {tuple(shape)}, the call needs [{rows}, {heads}, {dim}]")
    if t.dtype is not _BF16:
        raise DitError(f"{what}: unsupported dtype {t.dtype}")
    if t.get_device() != index or index < 0:
        raise DitError(f"buffers must be CUDA tensors on one device ({what} is on {t.device})")
    row, head, one = t.stride()
    if one != 1:
        raise DitError(f"{what}: a head's dimensions must be contiguous")
    at = t.data_ptr()
    if rows <= 1:
        row = heads * dim
    if heads <= 1:
        head = dim
    if at & 15 or row & 7 or head & 7:
        raise DitError(f"{what}: 16-byte aligned heads are needed ({lib().dit_status_str(2).decode()})")
    if row <= 0 or head <= 0:
        raise DitError(f"{what}: an expanded tensor")
    return at, row, head, heads, at + 2 * ((rows - 1) * row + (heads - 1) * head + dim) if rows else at


def _flat(t, nbytes, what, index, dtype=None, align=4):
    if t.get_device() != index:
        raise DitError(f"buffers must be CUDA tensors on one device ({what} is on {t.device})")
    if not t.is_contiguous():
        raise DitError(f"buffers must be contiguous ({what})")
    if dtype is not None and t.dtype is not dtype:
        raise DitError(f"{what}: unsupported dtype {t.dtype}")
    if t.nbytes < nbytes:
        raise DitError(f"{what}: {t.nbytes} bytes, the call needs {nbytes}")
    at = t.data_ptr()
    if nbytes and at % align:
        raise DitError(f"{what}: {lib().dit_status_str(2).decode()}")
    return at


def _meet(a, b, dim: int) -> bool:
    """Whether two views share memory: exact for views of one pair of strides, as those of one buffer have; of other interleavings those
    count as apart whose tokens or heads lie in runs that do not touch, or whose strides have a divisor that keeps them apart."""
    if a[4] <= b[0] or b[4] <= a[0] or a[4] == a[0] or b[4] == b[0]:
        return False
    pitch = a[1]
    if pitch == b[1]:  # the heads of a token lie in one run, repeated for each token
        d = (b[0] - a[0]) // 2 % pitch
        if d >= (a[3] - 1) * a[2] + dim and d + (b[3] - 1) * b[2] + dim <= pitch:
            return False
    return _interleave(a, b, dim)


def _interleave(a, b, dim):
    (row_a, head_a, heads_a), (row_b, head_b, heads_b), apart = a[1:4], b[1:4], (b[0] - a[0]) // 2
    rows_a, rows_b = (1 + ((v[4] - v[0]) // 2 - dim - (v[3] - 1) * v[2]) // v[1] for v in (a, b))
    # a stride that no access uses is as good as the other's
    if rows_a == 1 or rows_b == 1:
        row_a = row_b = max(row_a, row_b) if rows_a == rows_b else row_b if rows_a == 1 else row_a
    if heads_a == 1 or heads_b == 1:
        head_a = head_b = max(head_a, head_b) if heads_a == heads_b else head_b if heads_a == 1 else head_a
    g = math.gcd(row_a, row_b, head_a, head_b)
    if dim <= apart % g <= g - dim:
        return False
    # the tokens of a head lie in one run, repeated for each head
    if head_a == head_b and (rows_a - 1) * row_a + dim <= apart % head_a <= head_a - (rows_b - 1) * row_b - dim:
        return False
    if row_a != row_b or head_a != head_b or row_a < dim:
        return True
    for i in range(1 - heads_a, heads_b):  # b's heads against a's that are i heads before, of the tokens that come nearest
        j = -(apart + i * head_a) // row_a
        if any(1 - rows_a <= k < rows_b and abs(apart + i * head_a + k * row_a) < dim for k in (j, j + 1)):
            return True
    return False


def _apart(outputs, inputs, dim, own=()):
    """Refuses outputs that share memory with one another or with an input, but for the pairs `own` that may be one view."""
    for i, (name, out) in enumerate(outputs):
        begin, end = out[0], out[4]
        for other, t in (*inputs, *outputs[:i]):
            if begin < t[4] and t[0] < end and not (out == t and (name, other) in own) and _meet(out, t, dim):
                raise DitError(f"{name} overlaps {other}")


def _each(value, n, kind):
    """n numbers from one, of whatever library, or from as many as there are."""
    try:
        return [kind(v) for v in value]
    except TypeError:
        return [kind(value)] * n


# ----------------------------------------------------------------------------------------
# norms and rotation
# ----------------------------------------------------------------------------------------

class Rotary:
    """A rotation by positions with one to four axes (time, height, width).

    dims: dimensions that belong to each axis (even numbers; their sum is at most head_dim, what is left is not
    turned), in order.  Index i of axis a's pairs turns by position[a] scale[a] theta^(-2 i / dims[a]).
    interleaved: pairs are neighbours (2p, 2p + 1), else (p, p + sum(dims) / 2).  The table is copied on the
    current stream: other streams wait for that one before they use it."""

    def __init__(self, dims, head_dim: int, theta: float = 10000.0, scale=1.0, interleaved: bool = True, device="cuda"):
        self.dims, self.head_dim, self.interleaved = tuple(int(d) for d in dims), int(head_dim), bool(interleaved)
        axes = len(self.dims)
        scale = _each(scale, axes, float)
        if not 1 <= axes <= MAX_AXES or len(scale) != axes:
            raise DitError(f"Rotary: one to {MAX_AXES} axes, and a scale for each")
        if any(d < 0 or d % 2 for d in self.dims) or sum(self.dims) > self.head_dim:
            raise DitError(f"Rotary: even numbers of dimensions, {self.head_dim} at most")
        if not self.interleaved and sum(self.dims) % 8:
            raise DitError("Rotary: pairs half a rotation apart want a multiple of 8 dimensions")
        pairs = sum(self.dims) // 2
        host = torch.zeros(max(pairs, 1), 2, dtype=torch.int64)
        _check(lib().dit_rotary_table((ctypes.c_int32 * axes)(*self.dims), axes, float(theta), (ctypes.c_double * axes)(*scale),
                                      host.data_ptr(), host.nbytes), "dit_rotary_table")
        self._table = host.to(device)
        self.axes = axes
        self._index = self._table.get_device()
        self._info = _Rotary(self._table.data_ptr(), pairs, axes, int(self.interleaved), 0)
        self._p = ctypes.c_void_p(ctypes.addressof(self._info))

    table = property(lambda self: self._table)

    def __reduce_ex__(self, protocol):
        raise DitError("a Rotary holds addresses: make another one instead of a copy")


class QKNorm:
    """The norms' parameters: fp32 [4, dim] (query weight and bias, key weight and bias) for kind "layer", [2, dim] (query and
    key weight) for "rms".  The tensor is the caller's, read as it is at each call."""

    def __init__(self, params, kind: str = "rms", eps: float = 1e-6):
        if kind not in ("rms", "layer"):
            raise DitError(f"QKNorm: kind {kind!r}")
        rows = 4 if kind == "layer" else 2
        if params.dim() != 2 or params.shape[0] != rows or params.dtype != _F32 or not params.is_contiguous():
            raise DitError(f"QKNorm: contiguous float32 [{rows}, dim] for {kind!r}")
        if not (math.isfinite(eps) and eps >= 0):
            raise DitError("QKNorm: eps is finite and not negative")
        self.params, self.kind, self.eps, self.dim = params, kind, float(eps), params.shape[1]
        self._code = NORMS[kind]


def qk_norm_scratch(dim: int, device="cuda"):
    """Scratch for the gradients of the norms' parameters; calls ordered on one stream may share it."""
    return torch.empty(int(lib().dit_qk_norm_scratch_bytes(dim)), dtype=torch.uint8, device=device)


def _norm_args(q, k, norm, rotary, positions):
    """The views of q and k, and the call's other arguments."""
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise DitError("q and k: [tokens, heads, dim]")
    rows, heads, dim = q.shape
    index = q.get_device()
    if dim < 8 or dim % 8 or dim > 256 or heads < 1 or (k is not None and k.shape[1] < 1):
        raise DitError(f"a head of {dim} dimensions: multiples of 8 up to 256 are supported")
    qv = _view(q, rows, heads, dim, "q", index)
    kv = None if k is None else _view(k, rows, k.shape[1], dim, "k", index, True)
    if norm is None:
        kind, params, eps = 0, None, 0.0
    else:
        kind, eps = norm._code, norm.eps
        if norm.dim != dim:
            raise DitError(f"a norm of {norm.dim} dimensions, heads of {dim}")
        params = _flat(norm.params, 8 * dim * kind, "params", index, _F32)
    rot, at = None, None
    if rotary is not None:
        if rotary.head_dim != dim:
            raise DitError(f"a rotation of heads of {rotary.head_dim} dimensions, heads of {dim}")
        if rotary._index != index:
            raise DitError(f"the rotation is on {rotary.table.device}, q on {q.device}")
        if positions is None or positions.shape != (rows, rotary.axes):
            raise DitError(f"positions: int32 [{rows}, {rotary.axes}] is needed")
        at, rot = _flat(positions, 4 * rows * rotary.axes, "positions", index, _I32), rotary._p
    elif positions is not None:
        raise DitError("positions without a rotation")
    return qv, kv, index, (rows, dim, kind, params, eps, rot, at)


def _beside(t, of, name, dim, rows, index):
    """The view of a tensor that goes with q or k."""
    if (t is None) != (of is None):
        raise DitError(f"{name}: goes with k")
    return None if t is None else _view(t, rows, of[3], dim, name, index, True)


def _norm_rope_call(q, k, q_out, k_out, norm, rotary, positions, stream):
    qv, kv, index, rest = _norm_args(q, k, norm, rotary, positions)
    rows, dim = rest[0], rest[1]
    qo, ko = _beside(q_out, qv, "q_out", dim, rows, index), _beside(k_out, kv, "k_out", dim, rows, index)
    if kv is None:
        _apart((("q_out", qo),), (("q", qv),), dim, (("q_out", "q"),))
    else:
        _apart((("q_out", qo), ("k_out", ko)), (("q", qv), ("k", kv)), dim, (("q_out", "q"), ("k_out", "k")))
    raw = raw_stream(stream, index)

    def call():
        st = lib().dit_qk_norm_rope(*_lay(qv, kv, qo, ko), *rest, raw)
        if st:
            _check(st, "dit_qk_norm_rope")
    return call


def qk_norm_rope(q, k, q_out, k_out, norm: QKNorm | None = None, rotary: Rotary | None = None, positions=None, stream=None):
    """The norm of every head of q [tokens, heads, dim] and k [tokens, kv_heads, dim] (bf16 views, e.g. of the QKV
    projection's output), then the rotation at `positions` (int32 [tokens, axes]), into q_out and k_out, which may
    be the views q and k themselves.  norm or rotary None: without that part.  k None: queries alone."""
    _norm_rope_call(q, k, q_out, k_out, norm, rotary, positions, stream)()


def qk_norm_rope_backward(q, k, dq_out, dk_out, dq, dk, norm, rotary, positions, dparams, scratch, ws, stream=None):
    """dq, dk (bf16; may be dq_out and dk_out themselves) from the outputs' gradients dq_out, dk_out and the forward pass'
    inputs q, k; dparams (fp32, the shape of norm.params, overwritten; None: not wanted, and scratch may be
    None) over all tokens and heads."""
    qv, kv, index, rest = _norm_args(q, k, norm, rotary, positions)
    rows, dim = rest[0], rest[1]
    views = [_beside(t, of, name, dim, rows, index) for t, of, name in ((dq_out, qv, "dq_out"), (dk_out, kv, "dk_out"), (dq, qv, "dq"), (dk, kv, "dk"))]
    names = [n for n in (("q", qv), ("k", kv), ("dq_out", views[0]), ("dk_out", views[1])) if n[1] is not None]
    _apart([n for n in (("dq", views[2]), ("dk", views[3])) if n[1] is not None], names, dim, (("dq", "dq_out"), ("dk", "dk_out")))
    dp, sp, sn = None, None, 0
    if dparams is not None:
        if norm is None:
            raise DitError("dparams without a norm")
        if dparams.shape != norm.params.shape:
            raise DitError(f"dparams: float32 {tuple(norm.params.shape)} is needed")
        if k is None:
            raise DitError("dparams want q and k")
        dp = _flat(dparams, 8 * dim * rest[2], "dparams", index, _F32)
        sn = scratch.nbytes if scratch is not None else 0
        sp = _flat(scratch, int(lib().dit_qk_norm_scratch_bytes(dim)), "scratch", index, align=16) if scratch is not None else None
    wp = _flat(ws, 0, "ws", index)
    raw = raw_stream(stream, index)
    st = lib().dit_qk_norm_rope_backward(*_lay(qv, kv, *views), *rest, dp, sp, sn, wp, ws.nbytes, raw)
    if st:
        _check(st, "dit_qk_norm_rope_backward")


# ----------------------------------------------------------------------------------------
# attention
# ----------------------------------------------------------------------------------------

class AttentionPlan:
    """The documents of a batch, and what each token of them sees.

    lengths: query tokens of every document, in batch order (0 is allowed).  kv_lengths: its key tokens (None: the same); the
    queries are the last of them.  kv_begins: the row of k and v where each document's keys begin (None: one document
    behind the other; a cache of `room` rows for each has i * room).  frame 0: a token sees its whole
    document.  frame F > 0: tokens see the document's first `prefix` tokens (a number, or one for each document) and, behind
    those, the frames of F tokens up to their own (1: causal).

    A plan is made once for a batch and serves every block and every step with these lengths; training=True makes one
    that the backward pass takes too.  Over caches that grow each step wants a plan of its own: 0.1 ms on the host for a few
    requests or for whole videos, 1 to 2 ms for 64 requests of 8 key heads, 3 to 25 ms for 256 to 1000 single tokens, whose pieces
    are searched for.  The copy of its table waits for the stream, and a captured call keeps the plan it was captured with.  The table is laid out on the host and copied to `device` on the current stream: other streams wait
    for that one before they use the plan."""

    def __init__(self, lengths, heads: int, dim: int, kv_heads: int | None = None, kv_lengths=None, kv_begins=None, frame: int = 0,
                 prefix=0, training: bool = False, device="cuda"):
        lengths = [int(v) for v in lengths]
        n = len(lengths)
        kv_lengths = lengths if kv_lengths is None else [int(v) for v in kv_lengths]
        prefix = _each(prefix, n, int)
        begins = None if kv_begins is None else [int(v) for v in kv_begins]
        for name, v in (("kv_lengths", kv_lengths), ("prefix", prefix), ("kv_begins", begins)):
            if v is not None and len(v) != n:
                raise DitError(f"AttentionPlan: {len(v)} {name} and {n} lengths")
        if any(not 0 <= v < 2 ** 31 for v in (*lengths, *kv_lengths, *prefix, *(begins or ()), int(frame))):
            raise DitError("AttentionPlan: a length, prefix, begin or frame out of range")
        kv_heads = heads if kv_heads is None else int(kv_heads)
        if any(not 0 < v < 2 ** 31 for v in (int(heads), int(kv_heads), int(dim))):
            raise DitError("AttentionPlan: heads, kv_heads and dim are positive")
        arr = [None if v is None else torch.tensor(v, dtype=torch.int64) for v in (lengths, kv_lengths, begins, prefix)]
        self.info = _Plan()
        args = (*(None if a is None else a.data_ptr() for a in arr), n, int(frame), int(heads), kv_heads, int(dim), int(bool(training)),
                ctypes.byref(self.info))
        host = torch.empty(1 << 14, dtype=_I32)  # most tables fit: a plan is made once, not a first time for its size
        st = lib().dit_attention_plan(*args, host.data_ptr(), host.numel())
        if st and self.info.table_ints > host.numel():
            host = torch.empty(self.info.table_ints, dtype=_I32)
            st = lib().dit_attention_plan(*args, host.data_ptr(), host.numel())
        _check(st, "dit_attention_plan")
        self._table = host[:self.info.table_ints].clone().to(device)
        self.q_rows, self.k_rows, self.training = self.info.q_rows, self.info.k_rows, bool(training)
        self.heads, self.kv_heads, self.dim = int(heads), kv_heads, int(dim)
        self._info_p, self._table_p = ctypes.c_void_p(ctypes.addressof(self.info)), ctypes.c_void_p(self._table.data_ptr())
        self._index = self._table.get_device()
        self._scratch_bytes, self._saved_bytes = self.info.scratch_bytes, self.info.saved_bytes
        self._shape = (self._index, self.dim, self.q_rows, self.k_rows, self.heads, kv_heads)
        self._default_scale = self.dim ** -0.5

    table = property(lambda self: self._table)

    def __reduce_ex__(self, protocol):
        raise DitError("an AttentionPlan holds addresses: make another plan instead of a copy")


def attention_scratch(plan: AttentionPlan):
    """Scratch for the calls with this plan; calls ordered on one stream may share it."""
    return torch.empty(plan._scratch_bytes, dtype=torch.uint8, device=plan.table.device)


def attention_saved(plan: AttentionPlan):
    """What the forward pass of one block keeps for its backward pass."""
    return torch.empty(plan._saved_bytes, dtype=torch.uint8, device=plan.table.device)


def _scale_of(plan, scale):
    if scale is None:
        return plan._default_scale
    scale = float(scale)
    if not (scale > 0 and math.isfinite(scale)):
        raise DitError("attention: scale is finite and positive")
    return scale


def _attention_call(plan, q, k, v, out, scratch, ws, scale, saved, stream):
    i, dim, rows, keys, heads, kv_heads = plan._shape
    hq, hk, hv = _view(q, rows, heads, dim, "q", i), _view(k, keys, kv_heads, dim, "k", i), _view(v, keys, kv_heads, dim, "v", i)
    ho = _view(out, rows, heads, dim, "out", i)
    _apart((("out", ho),), (("q", hq), ("k", hk), ("v", hv)), dim)
    scale = _scale_of(plan, scale)
    if saved is None:
        vp, vn = None, 0
    elif plan.training:
        vp, vn = _flat(saved, plan._saved_bytes, "saved", i, align=16), saved.nbytes
    else:
        raise DitError("saved needs AttentionPlan(..., training=True)")
    sp, wp = _flat(scratch, plan._scratch_bytes, "scratch", i, align=16), _flat(ws, 65536, "ws", i, align=32)
    raw = raw_stream(stream, i)

    def call():
        st = lib().dit_attention(plan._info_p, plan._table_p, *_lay(hq, hk, hv, ho), scale, vp, vn, sp, scratch.nbytes, wp, ws.nbytes, raw)
        if st:
            _check(st, "dit_attention")
    return call


def attention(plan: AttentionPlan, q, k, v, out, scratch, ws, scale: float | None = None, saved=None, stream=None):
    """out = softmax(scale q k^T) v over what each token sees (scale None: dim^-1/2).  q, out [tokens, heads, dim] and k, v
    [key rows, kv_heads, dim] are bf16 views; rows of no document are neither read into a result nor written.
    saved (attention_saved) keeps what attention_backward needs."""
    _attention_call(plan, q, k, v, out, scratch, ws, scale, saved, stream)()


def attention_backward(plan: AttentionPlan, q, k, v, out, dout, saved, dq, dk, dv, scratch, ws, scale: float | None = None, stream=None):
    """dq, dk, dv (bf16 views, overwritten) from the output's gradient dout; out and saved as the forward pass left them with the
    same plan, q, k, v and scale."""
    if not plan.training:
        raise DitError("attention_backward needs AttentionPlan(..., training=True)")
    i, dim, qn, kn, h, hk = plan._shape
    ins = (("q", _view(q, qn, h, dim, "q", i)), ("k", _view(k, kn, hk, dim, "k", i)), ("v", _view(v, kn, hk, dim, "v", i)),
           ("out", _view(out, qn, h, dim, "out", i)), ("dout", _view(dout, qn, h, dim, "dout", i)))
    outs = (("dq", _view(dq, qn, h, dim, "dq", i)), ("dk", _view(dk, kn, hk, dim, "dk", i)), ("dv", _view(dv, kn, hk, dim, "dv", i)))
    _apart(outs, ins, dim)
    scale = _scale_of(plan, scale)
    vp = _flat(saved, plan._saved_bytes, "saved", i, align=16)
    sp, wp = _flat(scratch, plan._scratch_bytes, "scratch", i, align=16), _flat(ws, 65536, "ws", i, align=32)
    raw = raw_stream(stream, i)
    st = lib().dit_attention_backward(plan._info_p, plan._table_p, *_lay(*(t[1] for t in (*ins, *outs))), scale, vp, saved.nbytes, sp,
                                      scratch.nbytes, wp, ws.nbytes, raw)
    if st:
        _check(st, "dit_attention_backward")


def _projectable(linear, x, route, y, bias, what):
    """What a routed projection of x into y refuses, for a caller that launches something before it.  Along the BF16 route x is
    read while y is written."""
    w, rows = linear.w, x.shape[0]
    if route == ROUTE_BF16:
        if w.bf16 is None:
            raise DitError(f"{what}: the BF16 route needs QuantizedWeight(..., keep_bf16=True)")
        if x.data_ptr() < y.data_ptr() + y.nbytes and y.data_ptr() < x.data_ptr() + x.nbytes:
            raise DitError(f"{what}: the output overlaps what the BF16 route reads")
    else:
        room = (linear.a8["q"] if route == ROUTE_INT8 else linear.a4["codes"]).shape[0]
        if rows > room:
            raise DitError(f"{what}: {rows} tokens, the projection was made for {room}")
    _bias_ok(bias, w.n)
    if y.numel() < rows * w.n:
        raise DitError(f"{what}: an output of {y.numel()} elements, the projection writes {rows * w.n}")
    if _dt(y) > 1:
        raise DitError(f"{what}: unsupported dtype {y.dtype}")
    _same_device(x, y, bias, linear.ws)
    _p(y), _p(bias)
    if y.data_ptr() % 32 or (bias is not None and bias.data_ptr() % 16):
        raise DitError(f"{what}: {lib().dit_status_str(2).decode()}")


class RoutedAttention:
    """The attention part of a block between two routed quantised projections: QKV, norms and rotation in place,
    attention, output projection.  The QKV projection's outputs are all query heads, all key heads, all value heads."""

    def __init__(self, qkv, out, heads: int, kv_heads: int | None = None, norm: QKNorm | None = None, rotary: Rotary | None = None):
        self.qkv, self.out, self.heads, self.kv_heads = qkv, out, int(heads), int(heads if kv_heads is None else kv_heads)
        if self.heads < 1 or self.kv_heads < 1 or out.w.k % self.heads:
            raise DitError(f"RoutedAttention: {heads} heads for an output projection of {out.w.k}")
        self.dim = out.w.k // self.heads
        if qkv.w.n != (self.heads + 2 * self.kv_heads) * self.dim:
            raise DitError(f"RoutedAttention: a QKV projection to {qkv.w.n}, the heads need {(self.heads + 2 * self.kv_heads) * self.dim}")
        self.norm, self.rotary = norm, rotary

    def __call__(self, x, routes, y, plan: AttentionPlan, qkv, attended, scratch, positions=None, bias=(None, None), stream=None):
        """y = attention of x's tokens along routes[0] (QKV) and routes[1] (output).  qkv [tokens, heads + 2 kv_heads, dim] and
        attended [tokens, heads, dim] are bf16 buffers of the caller; the plan is one of these heads whose keys are the batch's
        own tokens.  A call that is refused has written nothing."""
        t, h, hk, d = x.shape[0], self.heads, self.kv_heads, self.dim
        if (plan.heads, plan.kv_heads, plan.dim) != (h, hk, d) or plan.q_rows > t or plan.k_rows > t:
            raise DitError("RoutedAttention: a plan of other heads, or of more tokens")
        for name, b, width in (("qkv", qkv, h + 2 * hk), ("attended", attended, h)):
            if tuple(b.shape) != (t, width, d) or b.dtype != _BF16 or not b.is_contiguous():
                raise DitError(f"RoutedAttention: {name} is a contiguous bf16 [{t}, {width}, {d}]")
        if plan.q_rows < t:
            raise DitError(f"RoutedAttention: a plan of {plan.q_rows} tokens, {t} are given")
        if len(routes) != 2 or len(bias) != 2:
            raise DitError("RoutedAttention: a route and a bias for each of the two projections")
        _projectable(self.qkv, x, routes[0], qkv, bias[0], "RoutedAttention, QKV")
        _projectable(self.out, attended, routes[1], y, bias[1], "RoutedAttention, output")
        q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        steps = [_attention_call(plan, q, k, v, attended, scratch, self.out.ws, None, None, stream)]
        if self.norm is not None or self.rotary is not None:
            steps.insert(0, _norm_rope_call(q, k, q, k, self.norm, self.rotary, positions, stream))
        self.qkv(x, routes[0], qkv.view(t, -1), bias=bias[0], stream=stream)
        for step in steps:
            step()
        self.out(attended.view(t, -1), routes[1], y, bias=bias[1], stream=stream)
        return y
