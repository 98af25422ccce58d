"""Every way in which the adapters' work is cut over CTAs, forced on small shapes (the library's test hook), against the
definition in 64 bits: whole output tiles, equal shares whose partial results are added up by a kernel of their own
or by dx's, clusters of two to eight CTAs, and every width of the gradients' tiles."""
import functools

import pytest
import torch

from adapter_reference import check, inputs, reference

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import int8_mixed_precision_gb300 as dit  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
WHOLE, SHARES, CLUSTERS = 1, 2, 3

# (lengths, adapters, bank, rank, k, n): enough columns for eight CTAs to share a contraction; tiles that end inside
# 128 rows and 64 columns; an adapter without rows, requests without an adapter, uneven numbers of tiles
SHAPES = {
    "rank8": ([300, 5, 64, 17], [0, 1, -1, 0], 3, 8, 520, 584),
    "rank40": ([129, 0, 31, 900], [0, 0, 0, 0], 1, 40, 1032, 520),
    "rank64": ([700, 40, 1], [0, -1, 0], 1, 64, 776, 648),
    "rank128": ([260, 70, 300], [0, 0, 1], 2, 128, 520, 520),
}
CUTS = [(WHOLE, 0), (WHOLE, 3), (SHARES, 0), (SHARES, 1), (SHARES, 2), (SHARES, 7), (SHARES, 11)] + [(CLUSTERS, c) for c in range(2, 9)]


@functools.lru_cache(maxsize=None)
def case(name, dtype):
    c = inputs(*SHAPES[name], dtype, seed=31)
    return (c, *reference(c))


class Setup:
    def __init__(self, c, training=True):
        self.d = {k: v.cuda() for k, v in c.items() if torch.is_tensor(v)}
        self.plan = dit.AdapterPlan(c["lengths"], c["adapters"], self.d["a"].shape[0], training=training)
        self.bank = dit.AdapterBank(self.d["a"], self.d["b"], self.d["scale"])
        self.scratch = dit.adapter_scratch(self.plan, self.bank).fill_(0xff)
        self.ws = dit.workspace()
        self.saved = dit.adapter_saved(self.plan, self.bank).fill_(0xff) if training else None
        self.da, self.db = torch.full_like(self.d["a"], 7.0, dtype=F32), torch.full_like(self.d["b"], 7.0, dtype=F32)

    def forward(self):
        dit.lora_forward(self.plan, self.bank, self.d["x"], self.d["y"], self.scratch, self.ws, saved=self.saved)

    def backward(self, dx=True):
        dit.lora_backward(self.plan, self.bank, self.d["x"], self.d["dy"], self.saved, self.da, self.db, self.scratch, self.ws,
                          dx=self.d["dx"] if dx else None)


def force(monkeypatch, cut, n, width=0):
    monkeypatch.setenv("DIT6_TEST_CUT", f"{cut},{n},{width}")


def outputs(name, width):
    _, _, G, _, k, n = SHAPES[name]
    return sum(-(-v // (128 * width)) for v in (k, n)) * G


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cut", CUTS, ids=lambda c: f"{c[0]}-{c[1]}")
@pytest.mark.parametrize("name", SHAPES)
def test_forward(name, cut, dtype, monkeypatch):
    c, want, off = case(name, dtype)
    force(monkeypatch, *cut)
    for training in (False, True):
        s = Setup(c, training)
        s.forward()
        check(s.d["y"], want["y"], off["y"], "y")
        torch.cuda.synchronize()
        assert dit.device_status(s.ws) == 0


@pytest.mark.parametrize("width", [1, 2, 4])
@pytest.mark.parametrize("cut", CUTS, ids=lambda c: f"{c[0]}-{c[1]}")
@pytest.mark.parametrize("name", SHAPES)
def test_backward(name, cut, width, monkeypatch):
    """With dx, which then adds up what equal shares left, and without, where a kernel of its own does."""
    dtype = BF16 if (cut[1] + width) % 2 else F32
    c, want, off = case(name, dtype)
    s, t = Setup(c), Setup(c)
    for u in (s, t):
        u.forward()
    force(monkeypatch, *cut, width)
    if width == 4 and SHAPES[name][3] > 64:              # 512 columns of rank 128 are more than tensor memory holds
        with pytest.raises(dit.DitError, match="UNSUPPORTED"):
            s.backward()
        return
    if cut[0] == CLUSTERS and outputs(name, width) * cut[1] > 112:
        pytest.skip("more clusters than run at a time")
    s.backward()
    t.backward(dx=False)
    check(s.d["dx"], want["dx"], off["dx"], "dx")
    for u in (s, t):
        check(u.da, want["da"], off["da"], "da")
        check(u.db, want["db"], off["db"], "db")
        assert dit.device_status(u.ws) == 0
    assert torch.equal(s.da, t.da) and torch.equal(s.db, t.db)


@pytest.mark.parametrize("name", SHAPES)
def test_the_hook_refuses_what_does_not_fit(name, monkeypatch):
    s = Setup(case(name, F32)[0])
    for cut in ((CLUSTERS, 9), (CLUSTERS, 1)):
        force(monkeypatch, *cut)
        with pytest.raises(dit.DitError, match="UNSUPPORTED"):
            s.forward()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_large_batch_as_it_is_cut(dtype):
    """Tens of thousands of rows, uneven over the adapters, with the library's own choice."""
    c = inputs([9000, 3000, 40, 77, 8000, 1], [0, 1, -1, 1, 2, 0], 4, 64, 1032, 776, dtype, seed=32)
    want, off = reference(c)
    s = Setup(c)
    s.forward()
    s.backward()
    for got, name in ((s.d["y"], "y"), (s.d["dx"], "dx"), (s.da, "da"), (s.db, "db")):
        check(got, want[name], off[name], name)
    assert dit.device_status(s.ws) == 0
