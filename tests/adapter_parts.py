"""Inputs on which the number of bf16 parts that h and e are held with shows: every sum of the adapters' products has one
term, so that nothing but the roundings of that term is left.

Each row has an adapter of its own; row j of A has one element that is not 0, column j of B one.  Then
  h[t, j] = s x[t, k_j] A[j, k_j]          one rounding of 24 bits (by the scale; the product has 16)
  y[t, n_j] = h[t, j] B[n_j, j]            32 bits, one more rounding, and cuts of the small parts' sum far below it
  dA[t] = e[t]^T x[t], dB[t] = dy[t]^T h[t] likewise, element by element.
Three parts hold the 24 bits exactly; with the parts' products added small ones first each sum is cut once at its full
size and its partial sums are cut at 2^-8 of it: 2^-24 + 2^-23 + 2^-31 and less of the value, so BOUND = 2^-22 holds.
With the largest part first it is cut twice, 2^-24 + 2^-22: BOUND_ANY_ORDER = 2^-21.  Two parts leave out up to 2^-17."""
import torch

BF16 = torch.bfloat16
BOUND, BOUND_ANY_ORDER = 2.0 ** -22, 2.0 ** -21


def case(T=40, rank=24, k=72, n=136, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a, b = torch.zeros(T, rank, k), torch.zeros(T, n, rank)
    j = torch.arange(rank)
    for t in range(T):
        a[t, j, torch.randperm(k, generator=g)[:rank]] = r(rank)
        b[t, torch.randperm(n, generator=g)[:rank], j] = r(rank)
    return {"lengths": [1] * T, "adapters": list(range(T)), "x": r(T, k).to(BF16), "dy": r(T, n).to(BF16), "a": a.to(BF16),
            "b": b.to(BF16), "scale": torch.rand(T, generator=g) + 0.5, "y": torch.zeros(T, n), "dx": torch.zeros(T, k)}


def split(v, parts):
    """What `parts` bf16 parts hold of v."""
    held = torch.zeros_like(v)
    for _ in range(parts):
        held = held + (v - held).to(BF16).to(v.dtype)
    return held


def results(c, parts=None):
    """y, dx, da, db in 64 bits, from h and e as they are or as `parts` parts hold them."""
    d = {n: v.double() for n, v in c.items() if torch.is_tensor(v)}
    h = d["scale"][:, None] * torch.einsum("tk,tjk->tj", d["x"], d["a"])
    e = d["scale"][:, None] * torch.einsum("tn,tnj->tj", d["dy"], d["b"])
    if parts:
        h, e = (split(v.float().double(), parts) for v in (h, e))
    return {"y": torch.einsum("tj,tnj->tn", h, d["b"]), "dx": torch.einsum("tj,tjk->tk", e, d["a"]),
            "da": torch.einsum("tj,tk->tjk", e, d["x"]), "db": torch.einsum("tn,tj->tnj", d["dy"], h)}


def worst(got, want):
    """The largest relative error, and the share of elements above BOUND_ANY_ORDER."""
    off = (got.double().cpu() - want).abs() / want.abs().clamp(min=1e-300)
    return float(off.max()), float((off > BOUND_ANY_ORDER).double().mean())
