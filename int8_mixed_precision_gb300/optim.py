"""AdamW over many tensors in one launch, with the moments in 32 or in 8 bits.

``AdamW`` keeps the tables of its tensors on the device; every buffer is the caller's.  The formulas,
the 8-bit form and its roundings are those of ``dit_adamw_step`` in ``include/dit6.h``.
"""
from __future__ import annotations

import ctypes

import torch

from . import DitError, _check, workspace
from ._lib import lib
from .adapters import raw_stream

BLOCK = 256        # consecutive elements of a tensor that share a scale of an 8-bit moment
_F32, _BF16, _E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
_CODE = {_F32: 0, _BF16: 1}


class _Tensor(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("p", "g", "m", "v", "m_scale", "v_scale", "copy", "m_values", "v_values")] + \
        [("n", ctypes.c_int64)]


class _Args(ctypes.Structure):
    _fields_ = [(name, ctypes.c_double) for name in ("lr", "beta1", "beta2", "eps", "weight_decay")] + [("step", ctypes.c_int64)]


def adamw_moments(params, bits: int = 32) -> dict:
    """Zero moments for `params`: keyword arguments of AdamW (m, v and, for 8 bits, their scales)."""
    if bits == 32:
        return {name: [torch.zeros(p.numel(), dtype=_F32, device=p.device) for p in params] for name in ("m", "v")}
    if bits != 8:
        raise DitError(f"AdamW: moments in 8 or 32 bits, not {bits}")
    out = {name: [torch.zeros(p.numel(), dtype=torch.uint8, device=p.device).view(_E4M3) for p in params] for name in ("m", "v")}
    out.update({name: [torch.zeros(-(-p.numel() // BLOCK), dtype=_F32, device=p.device) for p in params]
                for name in ("m_scale", "v_scale")})
    return out


class AdamW:
    """params, grads, m, v: lists of tensors of equal sizes, held by the caller and updated in place.

    params fp32 or bf16; grads fp32 or bf16; m, v fp32, or float8_e4m3fn codes with m_scale and
    v_scale (fp32, one for each 256 elements; v then holds the codes of the second moment's
    root).  copies: bf16 tensors that receive the parameters rounded to bf16 (for fp32
    masters).  m_values, v_values: bf16 tensors for export_moments.  step: steps made so far.

    The tables hold the tensors' addresses: a tensor that is given another storage (``.data = ...``) is no longer
    the one that is stepped.  They are copied on the current stream; other streams wait for that one before their
    first step.  The step count lives on the host: a step captured in a CUDA graph keeps its own."""

    def __init__(self, params, grads, m, v, m_scale=None, v_scale=None, copies=None, m_values=None, v_values=None,
                 lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                 weight_decay: float = 0.01, step: int = 0):
        lists = {"p": params, "g": grads, "m": m, "v": v, "m_scale": m_scale, "v_scale": v_scale, "copy": copies,
                 "m_values": m_values, "v_values": v_values}
        lists = {name: list(ts) for name, ts in lists.items() if ts is not None}
        count = len(lists["p"])
        if not count:
            raise DitError("AdamW: no tensors")
        self.bits = 8 if lists["m"] and lists["m"][0].dtype == _E4M3 else 32
        if (self.bits == 8) != ("m_scale" in lists and "v_scale" in lists) or ("m_scale" in lists) != ("v_scale" in lists):
            raise DitError("AdamW: m_scale and v_scale go with 8-bit moments")
        if self.bits == 32 and ("m_values" in lists or "v_values" in lists):
            raise DitError("AdamW: m_values and v_values go with 8-bit moments")
        state = _E4M3 if self.bits == 8 else _F32
        types = {"p": _CODE, "g": _CODE, "m": (state,), "v": (state,), "m_scale": (_F32,), "v_scale": (_F32,)}
        device = lists["p"][0].device
        for name, ts in lists.items():
            if len(ts) != count:
                raise DitError(f"AdamW: {len(ts)} tensors in {name}, {count} parameters")
            for t, p in zip(ts, lists["p"]):
                need = -(-p.numel() // BLOCK) if name.endswith("_scale") else p.numel()
                if t.numel() != need:
                    raise DitError(f"AdamW: {name} of {t.numel()} elements, {need} are needed")
                if t.dtype not in types.get(name, (_BF16,)) or t.dtype != ts[0].dtype:
                    raise DitError(f"AdamW: {name}: unsupported dtype {t.dtype}")
                if not t.is_cuda:
                    raise DitError(f"buffers must be CUDA tensors (got one on {t.device})")
                if t.device != device:
                    raise DitError("AdamW: buffers on different devices")
                if not t.is_contiguous():
                    raise DitError("buffers must be contiguous")
                if t.numel() and t.data_ptr() % (4 if name.endswith("_scale") else 32):
                    raise DitError(f"AdamW: {name}: {lib().dit_status_str(2).decode()}")
        self._lists, self.device, self.step_count = lists, device, int(step)
        # the memory behind the tables' addresses, should a tensor be given another storage
        self._storages = [t.untyped_storage() for ts in lists.values() for t in ts]
        self._args = _Args(lr, beta1, beta2, eps, weight_decay, 0)
        descs = (_Tensor * count)()
        for i in range(count):
            for name, ts in lists.items():
                setattr(descs[i], name, ts[i].data_ptr() or None)
            descs[i].n = lists["p"][i].numel()
        sizes = torch.tensor([p.numel() for p in lists["p"]], dtype=torch.int64)
        n = lib().dit_adamw_chunks(sizes.data_ptr(), count, None, 0)
        if n < 0:
            raise DitError("AdamW: too many elements")
        chunks = torch.empty(max(n, 1), 2, dtype=torch.int32)
        lib().dit_adamw_chunks(sizes.data_ptr(), count, chunks.data_ptr(), n)
        self._descs = torch.frombuffer(bytearray(descs), dtype=torch.uint8).to(device)
        self._chunks = chunks.to(device)
        self._count, self._n_chunks = count, n
        self.ws = workspace(device)
        self._head = (ctypes.c_void_p(self._descs.data_ptr()), ctypes.c_int64(count), ctypes.c_void_p(self._chunks.data_ptr()),
                      ctypes.c_int64(n))
        self._types = tuple(ctypes.c_int(v) for v in (_CODE[lists["p"][0].dtype], _CODE[lists["g"][0].dtype], self.bits))
        self._tail = (ctypes.c_void_p(self.ws.data_ptr()), ctypes.c_size_t(self.ws.numel()))
        self._args_p = ctypes.c_void_p(ctypes.addressof(self._args))
        self._index = self._descs.get_device()

    @property
    def lr(self) -> float:
        return self._args.lr

    @lr.setter
    def lr(self, value: float) -> None:
        self._args.lr = value

    def step(self, grad_scale=None, stream=None) -> None:
        """One step on the gradients that the buffers hold; grad_scale (device float32 [1]) multiplies them
        (a clipping factor, or one over a loss scale)."""
        gp = None
        if grad_scale is not None:
            if grad_scale.dtype != _F32 or grad_scale.numel() != 1 or grad_scale.get_device() != self._index:
                raise DitError("AdamW: grad_scale is a float32 [1] on the parameters' device")
            gp = grad_scale.data_ptr()
        self._args.step = self.step_count + 1
        st = lib().dit_adamw_step(*self._head, *self._types, self._args_p, gp, *self._tail, raw_stream(stream, self._index))
        if st:
            _check(st, "dit_adamw_step")
        self.step_count += 1

    def export_moments(self, stream=None) -> None:
        """The values of 8-bit moments, in bf16, into m_values and v_values (the second moment itself)."""
        if "m_values" not in self._lists and "v_values" not in self._lists:
            raise DitError("AdamW: export_moments needs 8-bit moments with m_values or v_values")
        _check(lib().dit_adamw_moments(*self._head, *self._tail, raw_stream(stream, self._index)), "dit_adamw_moments")

    def state_dict(self) -> dict:
        """Host copies of the moments as they are held, and the step count."""
        names = [n for n in ("m", "v", "m_scale", "v_scale") if n in self._lists]
        return {"step": self.step_count, "bits": self.bits, **{n: [t.detach().cpu() for t in self._lists[n]] for n in names}}

    def load_state_dict(self, sd: dict) -> None:
        """The state of the same set of tensors; one that does not fit is refused before anything is copied."""
        names = [n for n in ("m", "v", "m_scale", "v_scale") if n in self._lists]
        if sd["bits"] != self.bits or int(sd["step"]) < 0 or any(n not in sd or len(sd[n]) != self._count for n in names):
            raise DitError("AdamW: the state of another set of tensors")
        for n in names:
            for t, s in zip(self._lists[n], sd[n]):
                if t.numel() != s.numel() or t.dtype != s.dtype:
                    raise DitError("AdamW: the state of another set of tensors")
        for n in names:
            for t, s in zip(self._lists[n], sd[n]):
                t.view(-1).copy_(s.reshape(-1))
        self.step_count = int(sd["step"])
