"""Low-rank adapters of many requests beside one shared (frozen, quantised) projection.

``AdapterPlan`` describes a batch (which rows use which adapter), ``AdapterBank`` holds the factors
of one layer, ``lora_forward`` and ``lora_backward`` are the calls of the C ABI one for one, and
``AdaptedLinear`` puts them beside a ``RoutedLinear``.  Argument marshalling and host-side checks
only: the arithmetic runs in the kernels behind ``include/dit6.h``.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import ACT_NONE, DitError, _check, gemm_bf16
from ._lib import lib

MAX_RANK = 128
_F32, _BF16 = torch.float32, torch.bfloat16
_CODE = {_F32: 0, _BF16: 1}
_C = torch._C


def raw_stream(stream, index: int) -> int:
    """The handle of `stream`, or of device `index`'s current stream (by torch's bare functions: a Stream object
    costs more than the checks and the launch of a short call together).  The library launches on
    the current device, so both have to be on it."""
    current = _C._cuda_getDevice()
    if stream is None and current == index:
        return _C._cuda_getCurrentRawStream(index)
    if stream is not None and getattr(stream, "device_index", index) != index:
        raise DitError(f"the buffers are on cuda:{index}, the stream is on cuda:{stream.device_index}")
    if current != index:
        raise DitError(f"the buffers are on cuda:{index}, the current device is cuda:{current}")
    return stream.cuda_stream


class _Plan(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("table_ints", ctypes.c_int64), ("n_adapters", ctypes.c_int32),
                ("training", ctypes.c_int32), ("n_tiles", ctypes.c_int32), ("n_small", ctypes.c_int32),
                ("most_tiles", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class AdapterPlan:
    """The rows of a batch and the adapter of each request.

    lengths: rows of every request, in batch order (0 is allowed).  adapters: the adapter of
    every request, -1 for none.  Rows past the last request are no part of the plan.  A plan is made
    once per batch and serves every layer and step; training=True makes one that the backward
    pass takes too.  The table is laid out on the host and copied to `device` on the current
    stream: other streams wait for that one before they use the plan."""

    def __init__(self, lengths, adapters, n_adapters: int, training: bool = False, device="cuda"):
        lengths, adapters = [int(v) for v in lengths], [int(v) for v in adapters]
        if len(lengths) != len(adapters):
            raise DitError(f"AdapterPlan: {len(lengths)} lengths and {len(adapters)} adapters")
        if any(not -2 ** 31 <= g < 2 ** 31 for g in adapters):
            raise DitError("AdapterPlan: adapter out of range")
        if any(not 0 <= v < 2 ** 31 for v in lengths):
            raise DitError("AdapterPlan: length out of range")
        ln = torch.tensor(lengths, dtype=torch.int64)
        ad = torch.tensor(adapters, dtype=torch.int32)
        self.info = _Plan()
        args = (ln.data_ptr(), ad.data_ptr(), len(lengths), int(n_adapters), int(bool(training)), ctypes.byref(self.info))
        _check(lib().dit_adapter_plan(*args, None, 0), "dit_adapter_plan")
        host = torch.empty(self.info.table_ints, dtype=torch.int32)
        _check(lib().dit_adapter_plan(*args, host.data_ptr(), host.numel()), "dit_adapter_plan")
        self._table = host.to(device)
        self.rows, self.n_adapters, self.training = self.info.rows, int(n_adapters), bool(training)
        self.n_tiles, self.n_small = self.info.n_tiles, self.info.n_small
        # converted once: a call of few microseconds passes twenty arguments
        self._info_p, self._table_p = ctypes.c_void_p(ctypes.addressof(self.info)), ctypes.c_void_p(self._table.data_ptr())
        self._index = self._table.get_device()

    table = property(lambda self: self._table)

    def __reduce_ex__(self, protocol):
        raise DitError("an AdapterPlan holds addresses: make another plan instead of a copy")


class AdapterBank:
    """The factors of one layer: a [n_adapters, rank, k] and b [n_adapters, n, rank] in bf16, scale
    [n_adapters] in fp32.  An adapter of a lower rank than the bank's is padded with zeros.  The
    tensors are the caller's, held and read as they are at each call; other tensors are another bank."""

    def __init__(self, a, b, scale):
        if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
            raise DitError("AdapterBank: a [n_adapters, rank, k] and b [n_adapters, n, rank]")
        if a.dtype != _BF16 or b.dtype != _BF16 or scale.dtype != _F32:
            raise DitError("AdapterBank: a and b in bf16, scale in float32")
        if scale.numel() != a.shape[0]:
            raise DitError(f"AdapterBank: {scale.numel()} scales for {a.shape[0]} adapters")
        if any(not t.is_contiguous() for t in (a, b, scale)):
            raise DitError("buffers must be contiguous")
        if a.device != b.device or a.device != scale.device:
            raise DitError("AdapterBank: buffers on different devices")
        self.n_adapters, self.rank, self.k = a.shape
        self.n = b.shape[1]
        if self.n_adapters < 1 or not 8 <= self.rank <= MAX_RANK or self.rank % 8 or self.k % 8 or self.n % 8 or \
                self.k < 8 or self.n < 8:
            raise DitError(f"AdapterBank: rank 8 to {MAX_RANK} in steps of 8, k and n multiples of 8")
        self._a, self._b, self._scale, self.device = a, b, scale, a.device
        self._index = a.get_device()
        self._shapes = (a.shape, b.shape)
        self._pointers = (a.data_ptr, b.data_ptr, scale.data_ptr)
        self._at = tuple(at() for at in self._pointers)
        self._sizes = (ctypes.c_int(self.rank), ctypes.c_int64(self.k), ctypes.c_int64(self.n))

    a, b, scale = (property(lambda self, name=name: getattr(self, name)) for name in ("_a", "_b", "_scale"))

    def __reduce__(self):
        return AdapterBank, (self._a, self._b, self._scale)


def adapter_scratch(plan: AdapterPlan, bank: AdapterBank):
    """Scratch for the calls with this plan and bank; calls ordered on one stream may share it, and
    one made for a larger layer serves a smaller one."""
    n = int(lib().dit_adapter_scratch_bytes(plan._info_p, bank.rank, bank.k, bank.n))
    return torch.empty(n, dtype=torch.uint8, device=bank.device)


def adapter_saved(plan: AdapterPlan, bank: AdapterBank):
    """What the forward pass of one layer keeps for its backward pass."""
    n = int(lib().dit_adapter_saved_bytes(plan._info_p, bank.rank))
    return torch.empty(n, dtype=torch.uint8, device=bank.device)


# The checks of a call.  They take one pass over each tensor's properties: a serving call's kernel takes
# a few microseconds, and so must its checks.

def _refuse(t, what, index):
    if not t.is_cuda:
        raise DitError(f"buffers must be CUDA tensors ({what} is on {t.device})")
    if t.get_device() != index:
        raise DitError(f"{what} is on {t.device}, the bank on cuda:{index}")
    raise DitError(f"buffers must be contiguous ({what})")


def _not_bf16(t, what):
    raise DitError(f"{what}: unsupported dtype {t.dtype}")


def _type_code(t, what):
    code = _CODE.get(t.dtype)
    if code is None:
        raise DitError(f"{what}: unsupported dtype {t.dtype}")
    return code


def _rows_of(t, rows, width, what, index):
    shape = t.shape
    if len(shape) != 2 or shape[1] != width or shape[0] < rows:
        raise DitError(f"{what}: {tuple(shape)}, the call needs [{rows}, {width}]")
    if t.get_device() != index or not t.is_contiguous():
        _refuse(t, what, index)
    return t.data_ptr()


def _bytes_of(t, what, index):
    if t.get_device() != index or not t.is_contiguous():
        _refuse(t, what, index)
    return t.data_ptr()


def _moved():
    raise DitError("the storage of the bank's tensors was exchanged: make a new AdapterBank")


def _disagree(plan, bank):
    if plan.n_adapters != bank.n_adapters:
        raise DitError(f"the plan is for {plan.n_adapters} adapters, the bank has {bank.n_adapters}")
    raise DitError(f"the plan is on {plan.table.device}, the bank on {bank.device}")


def lora_forward(plan: AdapterPlan, bank: AdapterBank, x, y, scratch, ws, saved=None, stream=None, _first=None):
    """y[t] += scale[g] (x[t] A[g]^T) B[g]^T for every row t with an adapter g (y bf16 or fp32, holding
    the shared projection's output; other rows are not touched).  saved (adapter_saved) keeps what
    lora_backward needs."""
    # _first: what a caller launches ahead of the adapters, once they have refused nothing
    i, rows = bank._index, plan.rows
    if plan._index != i or plan.n_adapters != bank.n_adapters:
        _disagree(plan, bank)
    a, b, scale = bank._pointers
    at = a(), b(), scale()
    if at != bank._at:
        _moved()
    if x.dtype is not _BF16:
        _not_bf16(x, "x")
    xp, y_code = _rows_of(x, rows, bank.k, "x", i), _type_code(y, "y")
    yp = _rows_of(y, rows, bank.n, "y", i)
    if i < 0:
        _refuse(x, "x", i)
    if saved is None:
        vp, vn = None, 0
    elif plan.training:
        vp, vn = _bytes_of(saved, "saved", i), saved.nbytes
    else:
        raise DitError("saved needs AdapterPlan(..., training=True)")
    sp, wp, raw = _bytes_of(scratch, "scratch", i), _bytes_of(ws, "ws", i), raw_stream(stream, i)
    if _first is not None:
        _first()
    st = lib().dit_lora_forward(plan._info_p, plan._table_p, xp, *at, *bank._sizes, yp, y_code, vp, vn, sp, scratch.nbytes,
                                wp, ws.nbytes, raw)
    if st:
        _check(st, "dit_lora_forward")


def lora_backward(plan: AdapterPlan, bank: AdapterBank, x, dy, saved, da, db, scratch, ws, dx=None, stream=None, _first=None):
    """dx[t] += scale[g] (dy[t] B[g]) A[g] (bf16 or fp32, holding the shared projection's part; None: not
    wanted), and da, db (fp32, the shapes of the bank's a and b, overwritten) the gradients of every
    adapter over all rows that use it.  dx may be dy itself (a residual's gradient).  saved: filled by
    lora_forward with the same plan, x, a and scale."""
    i, rows = bank._index, plan.rows
    if plan._index != i or plan.n_adapters != bank.n_adapters:
        _disagree(plan, bank)
    if not plan.training:
        raise DitError("lora_backward needs AdapterPlan(..., training=True)")
    a, b, scale = bank._pointers
    at = a(), b(), scale()
    if at != bank._at:
        _moved()
    if x.dtype is not _BF16:
        _not_bf16(x, "x")
    if dy.dtype is not _BF16:
        _not_bf16(dy, "dy")
    xp, dyp = _rows_of(x, rows, bank.k, "x", i), _rows_of(dy, rows, bank.n, "dy", i)
    if i < 0:
        _refuse(x, "x", i)
    if dx is None:
        dxp, dx_code = None, 1
    else:
        dx_code, dxp = _type_code(dx, "dx"), _rows_of(dx, rows, bank.k, "dx", i)
    a_shape, b_shape = bank._shapes
    if da.dtype is not _F32 or da.shape != a_shape:
        raise DitError(f"da: float32 {tuple(a_shape)} is needed")
    if db.dtype is not _F32 or db.shape != b_shape:
        raise DitError(f"db: float32 {tuple(b_shape)} is needed")
    vp, dap, dbp = _bytes_of(saved, "saved", i), _bytes_of(da, "da", i), _bytes_of(db, "db", i)
    sp, wp, raw = _bytes_of(scratch, "scratch", i), _bytes_of(ws, "ws", i), raw_stream(stream, i)
    if _first is not None:
        _first()
    st = lib().dit_lora_backward(plan._info_p, plan._table_p, xp, dyp, *at, *bank._sizes, vp, saved.nbytes, dxp, dx_code, dap, dbp,
                                 sp, scratch.nbytes, wp, ws.nbytes, raw)
    if st:
        _check(st, "dit_lora_backward")


def _launchable(plan, bank, scratch, ws, saved, *tensors):
    """What the library itself refuses, for callers that launch something before its call."""
    sizes = [(scratch, "scratch", lib().dit_adapter_scratch_bytes(plan._info_p, bank.rank, bank.k, bank.n)),
             (ws, "ws", lib().dit_workspace_bytes())]
    if saved is not None:
        sizes.append((saved, "saved", lib().dit_adapter_saved_bytes(plan._info_p, bank.rank)))
        if plan.n_tiles and saved.data_ptr() == scratch.data_ptr():
            raise DitError("AdaptedLinear: saved is scratch")
    for t, name, need in sizes:
        if t.nbytes < need:
            raise DitError(f"AdaptedLinear: {name} of {t.nbytes} bytes, {need} are needed")
    if any(t.data_ptr() % 32 for t in (bank.a, bank.b, *(s[0] for s in sizes), *tensors)):
        raise DitError(f"AdaptedLinear: {lib().dit_status_str(2).decode()}")


def _apart(out, out_name, *inputs):
    """Refuses an output over an input that is read after the output is first written."""
    o0 = out.data_ptr()
    for t, name in inputs:
        i0 = t.data_ptr()
        if o0 < i0 + t.nbytes and i0 < o0 + out.nbytes:
            raise DitError(f"AdaptedLinear: {out_name} overlaps {name}, which the adapters read after {out_name} is written")


class AdaptedLinear:
    """A routed quantised projection with low-rank adapters beside it.

    The frozen weight stays in its quantised forms; the adapters add to its output.  For training,
    `w_t` (the untransformed weight transposed, bf16 [k, n]) carries the gradient through the
    frozen projection; without it `backward` gives the adapters' part of dx alone."""

    def __init__(self, linear, bank: AdapterBank, w_t=None):
        if linear.w.k != bank.k or linear.w.n != bank.n:
            raise DitError(f"AdaptedLinear: a projection {linear.w.k} -> {linear.w.n} and adapters {bank.k} -> {bank.n}")
        if w_t is not None and (tuple(w_t.shape) != (bank.k, bank.n) or w_t.dtype != _BF16):
            raise DitError(f"AdaptedLinear: w_t is bf16 [{bank.k}, {bank.n}]")
        self.linear, self.bank, self.w_t = linear, bank, w_t

    def __call__(self, x, route, y, plan, scratch, saved=None, bias=None, act=ACT_NONE, stream=None):
        """y = x W^T (+ bias) along `route`, plus the adapters.  The adapters add to the projection
        itself, so an activation cannot be fused into it.  y shares no memory with x."""
        if act != ACT_NONE:
            raise DitError("AdaptedLinear: the activation follows the adapters and cannot be fused into the projection")

        def project():
            _launchable(plan, self.bank, scratch, self.linear.ws, saved, x, y)
            _apart(y, "y", (x, "x"))
            self.linear(x, route, y, bias=bias, stream=stream)
        lora_forward(plan, self.bank, x, y, scratch, self.linear.ws, saved=saved, stream=stream, _first=project)
        return y

    def backward(self, x, dy, plan, saved, da, db, dx, scratch, stream=None):
        """dx = dy W + the adapters' part; da, db the adapters' gradients.  dx shares no memory with dy or x."""
        def project():
            _launchable(plan, self.bank, scratch, self.linear.ws, saved, x, dy, dx, da, db)
            _apart(dx, "dx", (dy, "dy"), (x, "x"))
            if self.w_t is not None:
                gemm_bf16(dy, self.w_t, dx, self.linear.ws, stream=stream)
                return
            with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
                dx.zero_()
        lora_backward(plan, self.bank, x, dy, saved, da, db, scratch, self.linear.ws, dx=dx, stream=stream, _first=project)
        return dx
