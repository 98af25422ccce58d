"""Low-rank adapters and AdamW in 64 bits on the CPU, with bounds on what the kernels may be off."""
import torch

EPS = 2.0 ** -22      # of one accumulation step of the kernels' fp32 sums (truncation allowed for)
HELD = 2.0 ** -16     # of h and e, which are held with at least 16 significant bits
BF16 = 2.0 ** -8      # half a unit of a value with 8 significant bits
F32 = 2.0 ** -23


def inputs(lengths, adapters, n_adapters, rank, k, n, y_dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    rows = sum(lengths)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return {"lengths": lengths, "adapters": adapters, "x": r(rows, k).to(torch.bfloat16),
            "a": (r(n_adapters, rank, k) * k ** -0.5).to(torch.bfloat16), "b": (r(n_adapters, n, rank) * 0.1).to(torch.bfloat16),
            "scale": torch.rand(n_adapters, generator=g) + 0.5, "y": r(rows, n).to(y_dtype),
            "dy": r(rows, n).to(torch.bfloat16), "dx": r(rows, k).to(y_dtype)}


def spans(lengths, adapters):
    at = 0
    for rows, g in zip(lengths, adapters):
        if rows and g >= 0:
            yield slice(at, at + rows), g
        at += rows


def reference(c):
    """(values, bounds): y, dx, da, db from the definition, and how far fp32 sums may be from them."""
    d = {k: v.double() for k, v in c.items() if torch.is_tensor(v)}
    k, n, rank = d["a"].shape[2], d["b"].shape[1], d["a"].shape[1]
    out = {"y": d["y"].clone(), "dx": d["dx"].clone(), "da": torch.zeros_like(d["a"]), "db": torch.zeros_like(d["b"])}
    off = {name: torch.zeros_like(v) for name, v in out.items()}
    used = {}
    for rows, g in spans(c["lengths"], c["adapters"]):
        x, dy, a, b, s = d["x"][rows], d["dy"][rows], d["a"][g], d["b"][g], d["scale"][g]
        h, e = s * x @ a.T, s * dy @ b
        # |error of h| and of e: their fp32 sums, then the bits they are held with
        h_off = s * (k / 16 + 4) * EPS * (x.abs() @ a.abs().T) + HELD * h.abs()
        e_off = s * (n / 16 + 4) * EPS * (dy.abs() @ b.abs()) + HELD * e.abs()
        out["y"][rows] += h @ b.T
        off["y"][rows] += h_off @ b.abs().T + (rank / 8 + 4) * EPS * (h.abs() @ b.abs().T)
        out["dx"][rows] += e @ a
        off["dx"][rows] += e_off @ a.abs() + (rank / 8 + 4) * EPS * (e.abs() @ a.abs())
        out["da"][g] += e.T @ x
        out["db"][g] += dy.T @ h
        of = used.setdefault(g, [0, 0.0, 0.0])
        of[0] += h.shape[0]
        of[1] = of[1] + e.abs().T @ x.abs()
        of[2] = of[2] + dy.abs().T @ h.abs()
        off["da"][g] += e_off.T @ x.abs()
        off["db"][g] += dy.abs().T @ h_off
    for g, (rows, ea, hb) in used.items():
        steps = rows / 16 + 2 * len(c["lengths"]) + 8
        off["da"][g] += steps * EPS * ea
        off["db"][g] += steps * EPS * hb
    for name, like in (("y", c["y"]), ("dx", c["dx"])):
        # one rounding of the updated rows; the others stay as they are
        unit = BF16 if like.dtype == torch.bfloat16 else F32
        for rows, _ in spans(c["lengths"], c["adapters"]):
            off[name][rows] += unit * out[name][rows].abs() + 1e-30
    return out, off


def check(got, want, off, what):
    bad = ~((got.double().cpu() - want).abs() <= off)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           float(((got.double().cpu() - want).abs() / off.clamp(min=1e-300)).max()))


def e4m3(x):
    """The nearest E4M3 value, ties to the even code; |x| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)
