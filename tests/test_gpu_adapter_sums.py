"""The fp32 sums of short requests' adapters, at sizes where the tensor cores' truncation would add up.

An addition of the tensor cores cuts its result to 24 bits: up to one unit of it, 2^-23 of the value, half of one
on average, always towards zero.  With positive terms these errors add up, and how many additions
a sum goes through at its full size shows in its mean error."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import int8_mixed_precision_gb300 as dit  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
UNIT = 2.0 ** -23


def run(lengths, adapters, x, a, b, scale):
    bank = dit.AdapterBank(a.to(BF16).cuda(), b.to(BF16).cuda(), scale.cuda())
    plan, ws = dit.AdapterPlan(lengths, adapters, a.shape[0]), dit.workspace()
    assert plan.n_tiles == 0 and plan.n_small > 0                # every row is in a small tile
    y = torch.zeros(sum(lengths), b.shape[1], device="cuda")
    dit.lora_forward(plan, bank, x.to(BF16).cuda(), y, dit.adapter_scratch(plan, bank), ws)
    assert dit.device_status(ws) == 0
    return y.double().cpu(), plan


def test_the_parts_of_h_enter_small_ones_first():
    """h has three parts of 8 bits.  Rank 128 is eight instructions for each: in the order of the parts' sizes eight
    additions meet the sum at its full size (those of the largest parts), at most eight units and four on
    average; the others meet 2^-8 of it.  h itself is rounded once (it is one product of each row)."""
    g = torch.Generator().manual_seed(0)
    u = lambda *s: torch.rand(*s, generator=g) / 2 + 0.5  # noqa: E731
    r, k, n = 128, 128, 264
    x, a = u(16, k).to(BF16), torch.diag(u(r)).to(BF16)[None]
    b = u(1, n, r)
    b[:, :, 32:] /= 64                                           # the first instructions make the sum what it is
    b, scale = b.to(BF16), u(1)
    y, _ = run([16], [0], x, a, b, scale)
    h = (x.double() * torch.diagonal(a[0]).double() * scale.double())
    want = h @ b[0].double().T
    off = (y - want) / want
    assert float(off.abs().max()) <= 10 * UNIT, float(off.abs().max() / UNIT)
    assert abs(float(off.mean())) <= 5 * UNIT, float(off.mean() / UNIT)


@pytest.mark.parametrize("rank", [8, 128])
def test_long_contractions_are_drained(rank):
    """One CTA contracts 30720 elements in eight warps, sixteen at a time.  Drained every 256, an addition meets i of the
    sixteen sixteenths of its 256 elements' sum: 4.25 units of it on average at most, and the rounded
    additions behind have no preference.  Undrained a warp makes 240 of them: 60 units."""
    g = torch.Generator().manual_seed(1)
    u = lambda *s: torch.rand(*s, generator=g) / 2 + 0.5  # noqa: E731
    k, n = 30720, rank
    lengths, adapters = [32] * 80, [i % 2 for i in range(80)]
    x, a = u(2560, k).to(BF16), (u(2, rank, k) / 16384).to(BF16)
    b = torch.eye(rank).to(BF16)[None].repeat(2, 1, 1)
    y, plan = run(lengths, adapters, x, a, b, torch.ones(2))
    assert plan.n_small == 160                                   # too many tiles for clusters
    rows = torch.arange(2560) // 32 % 2
    want = torch.stack([x.double() @ a[i].double().T for i in (0, 1)])[rows, torch.arange(2560)]
    off = (y - want) / want
    assert float(off.abs().max()) <= 28 * UNIT, float(off.abs().max() / UNIT)
    assert abs(float(off.mean())) <= 5 * UNIT, float(off.mean() / UNIT)
