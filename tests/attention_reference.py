"""Plain forms in 64 bits of the norms with rotation and of attention, and bounds on what roundings may add.

Half a step of bf16 is HALF = 2^-8 of a value.  FINE covers everything that is held in fp32 (sums, exponents,
scores): a few hundred units of 2^-24 on the magnitudes that enter, taken as 2^-14."""
import torch

HALF, FINE = 2.0 ** -8, 2.0 ** -14


def angles(positions, dims, theta, scale):
    parts = []
    for a, d in enumerate(dims):
        i = torch.arange(d // 2, dtype=torch.float64, device=positions.device)
        parts.append(positions[:, a, None].double() * scale[a] * theta ** (-2.0 * i / max(d, 1)))
    return torch.cat(parts, 1)


def turn(x, angle, interleaved):
    """x [t, h, d] turned by angle [t, pairs]."""
    n = angle.shape[1]
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    out = x.clone()
    i = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    out[..., i[0]] = x[..., i[0]] * c - x[..., i[1]] * s
    out[..., i[1]] = x[..., i[0]] * s + x[..., i[1]] * c
    return out


def pair_sum(x, n, interleaved):
    """|x| of an element and of its partner."""
    out = x.abs().clone()
    i = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    both = x[..., i[0]].abs() + x[..., i[1]].abs()
    out[..., i[0]], out[..., i[1]] = both, both
    return out


def normalise(x, kind, w, b, eps):
    if kind is None:
        return x, torch.ones_like(x[..., :1]), x
    m = x.mean(-1, keepdim=True) if kind == "layer" else 0.0
    r = ((x - m).square().mean(-1, keepdim=True) + eps) ** -0.5
    hat = (x - m) * r
    return hat, r, hat * w + (b if kind == "layer" else 0.0)


def visible(n, m, frame, prefix, device="cpu"):
    """bool [n, m]: what the last n tokens of m see, one token at a time."""
    out = torch.zeros(n, m, dtype=torch.bool)
    for i in range(n):
        t = i + m - n
        if frame == 0:
            end = m
        elif t < 0:
            end = 0
        elif t < prefix:
            end = prefix
        else:
            end = prefix + ((t - prefix) // frame + 1) * frame
        out[i, :min(end, m)] = True
    return out.to(device)


def attention(q, k, v, seen, scale):
    """One head: q [n, d], k, v [m, d]; the output, the weights, and a bound on the kernel's error."""
    s = (q @ k.T) * scale
    s = s.masked_fill(~seen, float("-inf"))
    some = seen.any(1, keepdim=True)
    p = torch.where(some, torch.softmax(s.masked_fill(~some, 0.0), 1), 0.0)
    p = torch.where(seen, p, 0.0)
    o = p @ v
    # p rounded to bf16 and the output rounded once
    return o, p, (HALF + FINE) * (p @ v.abs()) + (HALF + FINE) * o.abs() + 1e-30


def attention_grads(q, k, v, p, o, do, scale):
    """dq, dk, dv of one head, each with its bound."""
    dv = p.T @ do
    dp, delta = do @ v.T, (do * o).sum(1, keepdim=True)
    ds = p * (dp - delta)
    dq, dk = scale * ds @ k, scale * ds.T @ q
    # delta is taken from the rounded output, ds is rounded to bf16, each result once
    off = (do.abs() * ((HALF + FINE) * (p @ v.abs()) + (HALF + FINE) * o.abs())).sum(1, keepdim=True)
    e = (HALF + FINE) * ds.abs() + p * (off * (1 + HALF) + FINE * ((do.abs() @ v.abs().T) + (do * o).abs().sum(1, keepdim=True)))
    return ((dq, scale * e @ k.abs() + (HALF + FINE) * dq.abs() + 1e-30), (dk, scale * e.T @ q.abs() + (HALF + FINE) * dk.abs() + 1e-30),
            (dv, (HALF + FINE) * (p.T @ do.abs()) + (HALF + FINE) * dv.abs() + 1e-30))
