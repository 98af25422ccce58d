"""AdaptedLinear and the calls beside it on the host: what runs on which stream, and what is refused before anything
is launched.  The tensors are stand-ins that claim to be on a CUDA device; the launches are recorded."""
import contextlib
import os
import types

import pytest
import torch

import int8_mixed_precision_gb300 as dit
from int8_mixed_precision_gb300 import adapters

BF16, F32 = torch.bfloat16, torch.float32
BYTES = {BF16: 2, F32: 4, torch.uint8: 1, torch.int32: 4}


@pytest.fixture(scope="module", autouse=True)
def built():
    from int8_mixed_precision_gb300 import _lib, build
    if not os.path.exists(_lib.library_path()):
        try:
            build.build_library()
        except RuntimeError as e:          # no nvcc on this machine
            pytest.skip(str(e))


class Buffer:
    """A contiguous tensor of CUDA device `index` at an address, as the binding sees one."""
    is_cuda = True

    def __init__(self, address, shape, dtype=BF16, index=0, log=None):
        self.address, self.shape, self.dtype, self.index, self.log = address, torch.Size(shape), dtype, index, log
        self.device = torch.device("cuda", index)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    @property
    def nbytes(self):
        return self.numel() * BYTES[self.dtype]

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index

    def data_ptr(self):
        return self.address

    def zero_(self):
        self.log.append(("zero", torch.cuda.current_stream()))


class Library:
    """The real sizes and names; launches are recorded with the stream they went to."""

    def __init__(self, real, log):
        self.real, self.log = real, log

    def __getattr__(self, name):
        if name not in ("dit_lora_forward", "dit_lora_backward"):
            return getattr(self.real, name)
        return lambda *args: self.log.append((name, args[-1])) or 0


class Scene:
    T, G, R, K, N = 40, 2, 16, 64, 64

    def __init__(self, monkeypatch, training=True, index=0):
        self.log = log = []
        real = adapters.lib()
        monkeypatch.setattr(adapters, "lib", lambda: Library(real, log))
        self.current = 0x10
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: self.current)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: self.current, raising=False)

        @contextlib.contextmanager
        def stream(s):
            was, self.current = self.current, s.cuda_stream
            yield
            self.current = was
        monkeypatch.setattr(torch.cuda, "stream", stream)
        T, G, R, K, N = self.T, self.G, self.R, self.K, self.N
        at = iter(range(1 << 20, 1 << 30, 1 << 20))
        new = lambda *shape, dtype=BF16: Buffer(next(at), shape, dtype, index, log)  # noqa: E731
        self.bank = dit.AdapterBank(new(G, R, K), new(G, N, R), new(G, dtype=F32))
        self.plan = dit.AdapterPlan([T], [0], G, training=training, device="cpu")
        self.plan._index = index
        self.x, self.y, self.dy, self.dx = new(T, K), new(T, N, dtype=F32), new(T, N), new(T, K, dtype=F32)
        self.da, self.db = new(G, R, K, dtype=F32), new(G, N, R, dtype=F32)
        size = lambda f: int(f)  # noqa: E731
        scratch = real.dit_adapter_scratch_bytes(self.plan._info_p, R, K, N)
        saved = real.dit_adapter_saved_bytes(self.plan._info_p, R)
        self.scratch, self.saved = new(size(scratch), dtype=torch.uint8), new(size(saved), dtype=torch.uint8)
        self.ws = new(dit.workspace_bytes(), dtype=torch.uint8)
        self.new = new

        def linear(x, route, y, bias=None, stream=None):
            log.append(("projection", stream))
        linear.w, linear.ws = types.SimpleNamespace(k=K, n=N), self.ws
        self.layer = dit.AdaptedLinear(linear, self.bank)

    def forward(self, **kw):
        return self.layer(**{**dict(x=self.x, route=dit.ROUTE_INT8, y=self.y, plan=self.plan, scratch=self.scratch), **kw})

    def backward(self, **kw):
        return self.layer.backward(**{**dict(x=self.x, dy=self.dy, plan=self.plan, saved=self.saved, da=self.da, db=self.db,
                                             dx=self.dx, scratch=self.scratch), **kw})


def test_the_input_gradient_is_cleared_on_the_stream_of_the_call(monkeypatch):
    s = Scene(monkeypatch)
    s.backward(stream=types.SimpleNamespace(cuda_stream=0x77))
    assert s.log == [("zero", 0x77), ("dit_lora_backward", 0x77)]
    del s.log[:]
    s.backward()
    assert s.log == [("zero", 0x10), ("dit_lora_backward", 0x10)]


def test_outputs_over_inputs_are_refused_before_anything_is_written(monkeypatch):
    """The projection (or the zeros) would be written over x or dy before the adapters read them, so what the calls
    themselves allow (y over x, dx over dy) is no option beside a projection."""
    s = Scene(monkeypatch)
    behind = lambda t, n: Buffer(t.address + n, t.shape, t.dtype, 0, s.log)  # noqa: E731
    over = lambda t: Buffer(t.address, t.shape, BF16, 0, s.log)  # noqa: E731
    for y in (over(s.x), behind(s.x, 64), behind(s.x, s.x.nbytes - 32), behind(s.x, -32)):
        with pytest.raises(dit.DitError, match="y overlaps x"):
            s.forward(y=y)
    for kw, what in ((dict(dx=over(s.dy)), "dy"), (dict(dx=over(s.x)), "x"), (dict(dx=behind(s.dy, 32)), "dy")):
        with pytest.raises(dit.DitError, match=f"dx overlaps {what}"):
            s.backward(**kw)
    assert not s.log
    s.forward(y=behind(over(s.x), s.x.nbytes))           # next to it is fine
    assert [e[0] for e in s.log] == ["projection", "dit_lora_forward"]


def test_what_the_adapters_refuse_is_refused_before_the_projection_writes(monkeypatch):
    """Types, shapes, sizes, alignment and plans that the adapters' calls refuse, in either of their layers: y and dx
    are still what they were."""
    s = Scene(monkeypatch)
    serving = dit.AdapterPlan([s.T], [0], s.G, device="cpu")
    serving._index = 0
    other = dit.AdapterPlan([s.T], [0], 3, device="cpu")
    longer = dit.AdapterPlan([s.T + 1], [0], s.G, training=True, device="cpu")
    longer._index = 0
    odd = lambda t: Buffer(t.address + 16, t.shape, t.dtype, 0, s.log)  # noqa: E731
    small = lambda t: s.new(t.nbytes - 256, dtype=torch.uint8)  # noqa: E731
    shared = (dict(plan=other), dict(plan=longer), dict(scratch=small(s.scratch)), dict(scratch=odd(s.scratch)),
              dict(x=s.new(s.T, s.K, dtype=F32)), dict(x=s.new(s.T - 1, s.K)), dict(x=odd(s.x)), dict(saved=small(s.saved)),
              dict(saved=odd(s.saved)), dict(saved=s.scratch))
    for kw in (*shared, dict(y=s.new(s.T, s.N + 8)), dict(y=odd(s.y)), dict(plan=serving, saved=s.saved)):
        with pytest.raises(dit.DitError):
            s.forward(**{"saved": s.saved, **kw})
        assert not s.log, kw
    for kw in (*shared, dict(plan=serving), dict(dx=s.new(s.T, s.K + 8)), dict(dx=odd(s.dx)), dict(dy=s.new(s.T, s.N, dtype=F32)),
               dict(dy=odd(s.dy)), dict(da=s.db), dict(da=odd(s.da)), dict(db=odd(s.db)), dict(db=s.new(s.G, s.N, s.R))):
        with pytest.raises(dit.DitError):
            s.backward(**kw)
        assert not s.log, kw
    s.layer.linear.ws = s.new(64, dtype=torch.uint8)
    for call in (s.forward, s.backward):
        with pytest.raises(dit.DitError):
            call()
    assert not s.log


@pytest.mark.parametrize("index", [0, 1])
def test_a_call_for_another_device_than_the_current_one_is_refused(monkeypatch, index):
    """The library launches on the current device: with buffers of another one it would hand it foreign pointers."""
    from int8_mixed_precision_gb300 import optim
    s = Scene(monkeypatch, index=index)
    stream = types.SimpleNamespace(cuda_stream=0x77, device_index=1 - index)
    opt = object.__new__(optim.AdamW)
    opt._index, opt._lists, opt._head, opt._tail = index, {"m_values": []}, (), ()
    calls = (lambda **kw: dit.lora_forward(s.plan, s.bank, s.x, s.y, s.scratch, s.ws, **kw),
             lambda **kw: dit.lora_backward(s.plan, s.bank, s.x, s.dy, s.saved, s.da, s.db, s.scratch, s.ws, **kw),
             s.forward, s.backward, lambda **kw: adapters.raw_stream(kw.get("stream"), index))
    if index:
        calls += (lambda **kw: opt.export_moments(**kw),)
    for call in calls:
        with pytest.raises(dit.DitError, match="stream is on cuda"):
            call(stream=stream)
        if index == 0:
            call()
            assert s.log or call is calls[-1]
        else:
            for kw in ({}, dict(stream=types.SimpleNamespace(cuda_stream=0x77, device_index=1))):
                with pytest.raises(dit.DitError, match="current device is cuda:0"):
                    call(**kw)
            assert not s.log
        del s.log[:]


def test_a_bank_keeps_to_the_tensors_it_was_made_of(monkeypatch):
    """The bank's calls take the addresses that it checked.  Its tensors cannot be replaced, and one whose storage was
    exchanged underneath (``.data = ...``) is refused instead of read where it no longer is."""
    s = Scene(monkeypatch)
    for name in ("a", "b", "scale"):
        with pytest.raises(AttributeError):
            setattr(s.bank, name, getattr(s.bank, name))
    with pytest.raises(AttributeError):
        s.plan.table = s.plan.table
    call = lambda: dit.lora_forward(s.plan, s.bank, s.x, s.y, s.scratch, s.ws)  # noqa: E731
    back = lambda: dit.lora_backward(s.plan, s.bank, s.x, s.dy, s.saved, s.da, s.db, s.scratch, s.ws)  # noqa: E731
    for t in (s.bank.a, s.bank.b, s.bank.scale):
        call(), back()
        del s.log[:]
        was, t.address = t.address, 1 << 29
        for c in (call, back, s.forward, s.backward):
            with pytest.raises(dit.DitError, match="storage"):
                c()
        assert not s.log
        t.address = was
