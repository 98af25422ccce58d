"""Weight decay at small learning rates.  Zero gradients and moments leave the decay alone: p (1 - lr wd)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import int8_mixed_precision_gb300 as dit  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lr,wd", [(1e-3, 0.01), (1e-5, 0.01), (4e-5, 0.01), (3e-6, 0.1), (1.0, 0.3)])
def test_the_decay_is_what_was_asked_for(bits, lr, wd):
    """p - q, with q = RN(p RN(lr wd)): q is off by 2^-24 of itself twice and the difference is rounded once, so p' is
    within half a unit of p's binade (2^-24 of its power of two) and 2^-23 of q from the exact value.  A factor
    1 - lr wd rounded to fp32 is off by up to 2^-25 of p on top, which is 19 % of the decay at 1e-5 and 0.01."""
    g = torch.Generator().manual_seed(0)
    p = torch.randn(20000, generator=g) * 0.02
    q = p.cuda()
    opt = dit.AdamW([q], [torch.zeros_like(q)], **dit.adamw_moments([q], bits), lr=lr, weight_decay=wd)
    opt.step()
    want = p.double() * (1 - lr * wd)
    half = 2.0 ** -24 * torch.exp2(torch.floor(torch.log2(want.abs())))
    off = (q.cpu().double() - want).abs()
    bound = half * (1 + 2.0 ** -10) + 2.0 ** -23 * lr * wd * p.double().abs()
    assert bool((off <= bound).all()), (int((off > bound).sum()), float((off / half).max()))


@pytest.mark.parametrize("bits", [32, 8])
def test_decay_and_step_together(bits):
    """From zero moments the first step is lr g / (|g| + eps') with eps' = eps sqrt(1 - beta2): against 64 bits, with
    one rounding of p and 2^-20 of the step for the eleven roundings of its terms (2^-24 each at most, twice that
    for the quotient with 8-bit moments)."""
    g = torch.Generator().manual_seed(1)
    p, grad = torch.randn(5000, generator=g), torch.randn(5000, generator=g)
    q = p.cuda()
    lr, wd, eps, b2 = 1e-4, 0.1, 1e-8, 0.999
    opt = dit.AdamW([q], [grad.cuda()], **dit.adamw_moments([q], bits), lr=lr, weight_decay=wd, beta2=b2, eps=eps)
    opt.step()
    step = lr * grad.double() / (grad.double().abs() + eps) + lr * wd * p.double()
    want = p.double() - step
    bound = 2.0 ** -24 * want.abs().clamp(min=2.0 ** -126) + 2.0 ** -20 * (lr + lr * wd * p.double().abs())
    assert bool(((q.cpu().double() - want).abs() <= bound).all())
