"""Cases that measure the adapter operators and the optimiser step.

Three operators are measured.  Each has a plain form, made of elementary torch operations in 32
bits, and the framework's calls.

* ``forward``: low-rank adapters of many requests beside one shared projection.  Row t of the
  batch belongs to one request and uses that request's adapter g (or none):
  ``y[t] += scale[g] * (x[t] A[g]^T) B[g]^T``.
* ``train``: the same forward pass, keeping the rank-sized product, and its backward pass:
  ``dx[t] += scale[g] * (dy[t] B[g]) A[g]``, and for each adapter, over all rows that use it,
  ``dA[g] = scale[g] * (dy B[g])^T x`` and ``dB[g] = dy^T (scale[g] * x A[g]^T)``.
* ``adamw``: one AdamW step over many tensors, with the two moments held in 32 bits, or in 8 bits
  (E4M3 codes with one scale for each 256 consecutive elements of a tensor; the second moment as
  its square root, whose code is never 0 unless the moment is 0).

``own`` chooses the form that ``run`` takes.  The projections' widths are those of the
CogVideoX-2B-shaped block of this repository (hidden 1920, QKV 5760, feed-forward 7680).
"""
import random

import torch

own = False

BLOCK = 256          # elements of a tensor that share one scale of an 8-bit moment
E4M3_MAX = 448.0
E4M3_LEAST = 2.0 ** -9
TINY = 2.0 ** -100   # a block whose largest magnitude is below this is held as zeros
HYPER = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01}
STEPS_BEFORE = 100


# ------------------------------------------------------------------------------------------
# the cases
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # one request generating one token through a QKV projection: pure latency
        {"name": "forward one token", "op": "forward", "requests": 1, "tokens": 1, "spread": "even", "layout": 1, "adapters": 4, "rank": 16, "k": 1920, "n": 5760, "y": "bf16"},
        # a serving batch of single tokens, 16 adapters and requests without one among them
        {"name": "forward 64 single tokens", "op": "forward", "requests": 64, "tokens": 64, "spread": "even", "layout": 2, "adapters": 16, "rank": 32, "k": 1920, "n": 7680, "y": "bf16"},
        # prompts of odd lengths (empty and one-token ones too), a rank that is no power of two, fp32 outputs
        {"name": "forward ragged prompts", "op": "forward", "requests": 11, "tokens": 2011, "spread": "ragged", "layout": 3, "adapters": 6, "rank": 24, "k": 1920, "n": 1920, "y": "f32"},
        # two videos denoised together, one adapter each, beside the up projection of the feed-forward part
        {"name": "forward two videos", "op": "forward", "requests": 2, "tokens": 35552, "spread": "even", "layout": 4, "adapters": 2, "rank": 64, "k": 1920, "n": 7680, "y": "bf16"},
        # training on one text prompt
        {"name": "train one prompt", "op": "train", "requests": 1, "tokens": 226, "spread": "even", "layout": 5, "adapters": 1, "rank": 16, "k": 1920, "n": 1920, "y": "bf16"},
        # training three adapters on clips of odd lengths, several clips to an adapter
        {"name": "train ragged clips", "op": "train", "requests": 9, "tokens": 5003, "spread": "ragged", "layout": 6, "adapters": 3, "rank": 40, "k": 1920, "n": 5760, "y": "bf16"},
        # training one adapter on one video, beside the down projection
        {"name": "train one video", "op": "train", "requests": 1, "tokens": 17776, "spread": "even", "layout": 7, "adapters": 1, "rank": 64, "k": 7680, "n": 1920, "y": "bf16"},
        # the highest rank, beside the output projection, gradients of the input in fp32
        {"name": "train rank 128", "op": "train", "requests": 2, "tokens": 17776, "spread": "ragged", "layout": 8, "adapters": 2, "rank": 128, "k": 1920, "n": 1920, "y": "f32"},
        # the two factors of one adapter
        {"name": "adamw one adapter", "op": "adamw", "tensors": 2, "elements": 61440, "spread": "even", "layout": 9, "param": "f32", "grad": "f32", "bits": 32, "copies": True},
        # every adapter of a 30-block model at rank 64: 240 factors, fp32 masters with bf16 copies, 8-bit moments
        {"name": "adamw all adapters", "op": "adamw", "tensors": 240, "elements": 58982400, "spread": "even", "layout": 10, "param": "f32", "grad": "f32", "bits": 8, "copies": True},
        # many small tensors of odd sizes, everything 16 bits wide but the moments
        {"name": "adamw odd sizes", "op": "adamw", "tensors": 37, "elements": 1000003, "spread": "ragged", "layout": 11, "param": "bf16", "grad": "bf16", "bits": 8, "copies": False},
        # all four projections of six blocks, 32-bit moments
        {"name": "adamw dense weights", "op": "adamw", "tensors": 24, "elements": 265420800, "spread": "ragged", "layout": 12, "param": "f32", "grad": "bf16", "bits": 32, "copies": False},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["forward", "forward", "train", "train", "adamw"])
    layout = rng.randrange(1000, 1 << 30)
    if op == "adamw":
        tensors = _log(rng, 1, 300)
        return {"op": op, "tensors": tensors, "elements": max(tensors, _log(rng, 3000, 150_000_000)), "spread": rng.choice(["even", "ragged"]), "layout": layout,
                "param": rng.choice(["f32", "bf16"]), "grad": rng.choice(["f32", "bf16"]), "bits": rng.choice([8, 32]), "copies": rng.random() < 0.5}
    tokens = _log(rng, 1 if op == "forward" else 17, 35000 if op == "forward" else 15000)
    requests = min(tokens, _log(rng, 1, 128 if op == "forward" else 24))
    return {"op": op, "requests": requests, "tokens": tokens, "spread": rng.choice(["even", "ragged"]), "layout": layout, "adapters": _log(rng, 1, 24 if tokens < 2000 else 4),
            "rank": 8 * rng.randint(1, 16 if op == "train" else 8), "k": 8 * _log(rng, 40, 320), "n": 8 * _log(rng, 40, 900 if op == "forward" else 320), "y": rng.choice(["bf16", "bf16", "f32"])}


def _parts(total, count, spread, rng):
    """`total` cut into `count` parts: as even as it goes, or ragged with empty and one-element parts among them (the last part is not empty)."""
    if spread == "even":
        return [total // count + (i < total % count) for i in range(count)]
    cuts = sorted(rng.randint(0, total - 1) for _ in range(count - 1))
    if count > 3:
        cuts[0] = 0
        cuts[1] = 1 if total > 1 else 0
        cuts = sorted(cuts)
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _requests(case):
    """(rows, adapter) of every request; -1: a request without an adapter."""
    rng = random.Random(case["layout"])
    lengths = _parts(case["tokens"], case["requests"], case["spread"], rng)
    adapters = [i % case["adapters"] if i < case["adapters"] else rng.randrange(case["adapters"]) for i in range(case["requests"])]
    if case["requests"] > 16:
        adapters = [-1 if i % 13 == 5 else g for i, g in enumerate(adapters)]
    if case["spread"] == "ragged":
        rng.shuffle(adapters)
    return lengths, adapters


def _sizes(case):
    """Elements of every tensor of an optimiser case."""
    rng = random.Random(case["layout"])
    return [max(1, s) for s in _parts(case["elements"], case["tensors"], case["spread"], rng)]


def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        p, g = (4 if case["param"] == "f32" else 2), (4 if case["grad"] == "f32" else 2)
        # 8-bit moments: codes and scales read and written, and their values handed out in bf16
        moments = 16 if case["bits"] == 32 else 4 + 16 / BLOCK + 4
        return {"bytes": n * (2 * p + g + moments + (2 if case["copies"] else 0)), "flops": 15 * n}
    lengths, adapters = _requests(case)
    rows = sum(t for t, g in zip(lengths, adapters) if g >= 0)
    used = len({g for t, g in zip(lengths, adapters) if g >= 0 and t})
    r, k, n, y = case["rank"], case["k"], case["n"], (4 if case["y"] == "f32" else 2)
    weights = used * r * (k + n)
    if case["op"] == "forward":
        return {"bytes": rows * (2 * k + 2 * y * n) + 2 * weights, "flops": 2 * rows * r * (k + n)}
    # forward and backward: x, dy and the weights once, y and dx read and written, both gradients written
    return {"bytes": rows * (2 * k + 2 * n + 2 * y * (k + n)) + 2 * weights + 4 * case["adapters"] * r * (k + n), "flops": 6 * rows * r * (k + n)}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(rows, cols, gen):
    """bf16 activations with a hundredth of the channels much larger, as the quantised layers meet them."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    x[:, torch.randperm(cols, device="cuda", generator=gen)[: max(1, cols // 100)]] *= 50.0
    return x.to(torch.bfloat16)


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def prepare(case, seed):
    gen = _generator(seed)
    if case["op"] == "adamw":
        return _prepare_adamw(case, gen)
    lengths, adapters = _requests(case)
    T, G, r, K, N = case["tokens"], case["adapters"], case["rank"], case["k"], case["n"]
    s = {"op": case["op"], "x": _activations(T, K, gen),
         "a": (torch.randn(G, r, K, device="cuda", generator=gen) * K ** -0.5).to(torch.bfloat16),
         "b": (torch.randn(G, N, r, device="cuda", generator=gen) * 0.02).to(torch.bfloat16),
         "scale": 0.25 + 1.5 * torch.rand(G, device="cuda", generator=gen),
         "y": torch.randn(T, N, device="cuda", generator=gen).to(_dtype(case["y"])),  # the shared projection's output
         "of_row": torch.repeat_interleave(torch.tensor(adapters), torch.tensor(lengths)).cuda()}
    if case["op"] == "train":
        s["dy"] = (torch.randn(T, N, device="cuda", generator=gen) * 0.1).to(torch.bfloat16)
        s["dx"] = (torch.randn(T, K, device="cuda", generator=gen) * 0.1).to(_dtype(case["y"]))  # the shared projection's part of it
        s["da"] = torch.empty(G, r, K, device="cuda")
        s["db"] = torch.empty(G, N, r, device="cuda")
    if own:  # what a program keeps for all layers and steps of a batch
        import int8_mixed_precision_gb300 as dit
        s["ws"] = dit.workspace()
        s["bank"] = dit.AdapterBank(s["a"], s["b"], s["scale"])
        s["plan"] = dit.AdapterPlan(lengths, adapters, G, training=case["op"] == "train")
        s["scratch"] = dit.adapter_scratch(s["plan"], s["bank"])
        s["saved"] = dit.adapter_saved(s["plan"], s["bank"]) if case["op"] == "train" else None
    return s


def _places(sizes):
    """Where each tensor begins in the flat buffers (a multiple of BLOCK), and the buffers' length."""
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // BLOCK) * BLOCK)
    return at[:-1], at[-1]


def _inside(sizes):
    """True where a flat buffer's element belongs to a tensor, not to the gap behind one."""
    rooms = torch.tensor([-(-n // BLOCK) * BLOCK for n in sizes])
    last = torch.repeat_interleave(torch.tensor(_places(sizes)[0]) + torch.tensor(sizes), rooms).cuda()
    return torch.arange(last.numel(), device="cuda") < last


def _prepare_adamw(case, gen):
    # The tensors are views of one buffer for each kind, as trainers keep them; gaps hold zeros.
    sizes = _sizes(case)
    at, total = _places(sizes)
    inside = _inside(sizes)
    new = lambda std: torch.randn(total, device="cuda", generator=gen) * std * inside  # noqa: E731
    views = lambda flat: [flat[i:i + n] for i, n in zip(at, sizes)]  # noqa: E731
    s = {"op": "adamw", "bits": case["bits"], "t": STEPS_BEFORE, "grad_scale": torch.full((1,), 0.37, device="cuda"),
         "p": new(0.02).to(_dtype(case["param"])), "g": new(0.01).to(_dtype(case["grad"]))}
    s["copies"] = s["p"].to(torch.bfloat16) if case["copies"] else None
    m, u = new(1e-3), (new(5e-3).abs() + 1e-5) * inside  # the first moment, the second one's root
    if case["bits"] == 32:
        s.update(m=m, v=u * u)
    else:
        for name, t in (("m", m), ("v", u)):
            code, scale = _encode(t)
            s.update({name: code.to(torch.float8_e4m3fn), name + "_scale": scale, name + "_values": torch.zeros(total, dtype=torch.bfloat16, device="cuda")})
    if own:  # the optimiser that a training program keeps, over its tensors
        import int8_mixed_precision_gb300 as dit
        more = {}
        if case["copies"]:
            more["copies"] = views(s["copies"])
        if case["bits"] == 8:
            for name in ("m", "v"):
                more[name + "_scale"] = [s[name + "_scale"][i // BLOCK:(i + n - 1) // BLOCK + 1] for i, n in zip(at, sizes)]
                more[name + "_values"] = views(s[name + "_values"])
        s["opt"] = dit.AdamW(views(s["p"]), views(s["g"]), views(s["m"]), views(s["v"]), step=STEPS_BEFORE, **HYPER, **more)
    return s


# ------------------------------------------------------------------------------------------
# the operators
# ------------------------------------------------------------------------------------------

def run(s):
    if s["op"] == "adamw":
        return _adamw(s)
    if own:
        import int8_mixed_precision_gb300 as dit
        dit.lora_forward(s["plan"], s["bank"], s["x"], s["y"], s["scratch"], s["ws"], saved=s["saved"])
        if s["op"] == "forward":
            return s["y"]
        dit.lora_backward(s["plan"], s["bank"], s["x"], s["dy"], s["saved"], s["da"], s["db"], s["scratch"], s["ws"], dx=s["dx"])
        return {"y": s["y"], "dx": s["dx"], "da": s["da"], "db": s["db"]}
    # All adapters side by side, and in each row the columns of its own adapter only.
    G, r, K = s["a"].shape
    N = s["b"].shape[1]
    mask = (s["of_row"][:, None] == torch.arange(G, device="cuda")).float() * s["scale"]
    a, b = s["a"].float().reshape(G * r, K), s["b"].float().permute(0, 2, 1).reshape(G * r, N)
    x = s["x"].float()
    h = ((x @ a.T).view(-1, G, r) * mask[:, :, None]).view(-1, G * r)
    s["y"].copy_(s["y"].float() + h @ b)
    if s["op"] == "forward":
        return s["y"]
    dy = s["dy"].float()
    dh = ((dy @ b.T).view(-1, G, r) * mask[:, :, None]).view(-1, G * r)
    s["dx"].copy_(s["dx"].float() + dh @ a)
    s["da"].copy_((dh.T @ x).view(G, r, K))
    s["db"].copy_((h.T @ dy).view(G, r, N).permute(0, 2, 1))
    return {"y": s["y"], "dx": s["dx"], "da": s["da"], "db": s["db"]}


def _encode(values, root=False):
    """(E4M3 values, scales) of a flat buffer in blocks of BLOCK; of roots, none but 0 becomes 0."""
    blocks = values.view(-1, BLOCK)
    amax = blocks.abs().amax(dim=1)
    fine = amax >= TINY
    to_code = torch.where(fine, torch.div(torch.full_like(amax, E4M3_MAX), torch.where(fine, amax, 1.0)), 0.0)
    code = (blocks * to_code[:, None]).to(torch.float8_e4m3fn).float()
    if root:
        code = torch.where((code == 0) & (blocks > 0) & fine[:, None], E4M3_LEAST, code)
    return code.view(-1), torch.where(fine, amax * (1.0 / E4M3_MAX), 0.0)


def _decode(code, scale):
    return (code.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _adamw(s):
    names = ("p", "m", "v") if s["bits"] == 32 else ("p", "m_values", "v_values")
    if own:
        s["opt"].step(grad_scale=s["grad_scale"])
        if s["bits"] == 8:
            s["opt"].export_moments()  # the values that the codes stand for
    else:
        _adamw_plain(s)
    return {**{name: s[name] for name in names}, "copies": s["copies"]}


def _adamw_plain(s):
    # All tensors at once over the flat buffers; the factors are scalars, as a host program has them.
    s["t"] += 1
    b1, b2 = HYPER["beta1"], HYPER["beta2"]
    keep = 1.0 - HYPER["lr"] * HYPER["weight_decay"]
    rate = HYPER["lr"] / (1.0 - b1 ** s["t"])
    root = (1.0 - b2 ** s["t"]) ** -0.5
    g = s["g"].float() * s["grad_scale"]
    if s["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m, u = _decode(s["m"], s["m_scale"]), _decode(s["v"], s["v_scale"])
        v = u * u
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    u = v.sqrt()
    s["p"].copy_(s["p"].float() * keep - (m * rate) / (u * root + HYPER["eps"]))
    if s["copies"] is not None:
        s["copies"].copy_(s["p"])
    if s["bits"] == 32:
        s["m"], s["v"] = m, v
        return
    m, s["m_scale"] = _encode(m)
    u, s["v_scale"] = _encode(u, root=True)
    s["m"], s["v"] = m.to(torch.float8_e4m3fn), u.to(torch.float8_e4m3fn)
    u = _decode(u, s["v_scale"])
    s["m_values"], s["v_values"] = _decode(m, s["m_scale"]).to(torch.bfloat16), (u * u).to(torch.bfloat16)


# ------------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(case, s)
    y, x = s["y"].double(), s["x"].double()
    got = {"y": y}
    if case["op"] == "train":
        dy = s["dy"].double()
        got.update(dx=s["dx"].double(), da=torch.zeros_like(s["da"], dtype=torch.float64), db=torch.zeros_like(s["db"], dtype=torch.float64))
    begin = 0
    for rows, g in zip(*_requests(case)):
        part = slice(begin, begin + rows)
        begin += rows
        if g < 0 or not rows:
            continue
        a, b, c = s["a"][g].double(), s["b"][g].double(), float(s["scale"][g])
        delta = torch.einsum("tr,nr->tn", torch.einsum("tk,rk->tr", x[part], a), b)
        y[part] += c * delta
        if case["op"] == "train":
            through = torch.einsum("tn,nr->tr", dy[part], b)
            got["dx"][part] += c * torch.einsum("tr,rk->tk", through, a)
            got["da"][g] += c * torch.einsum("tr,tk->rk", through, x[part])
            got["db"][g] += c * torch.einsum("tn,tr->nr", dy[part], torch.einsum("tk,rk->tr", x[part], a))
    return got if case["op"] == "train" else y


def _exact_e4m3(x):
    """The nearest E4M3 value of each element (ties to the even code)."""
    e = torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 4  # three bits behind the leading one
    step = torch.ldexp(torch.ones_like(x), e)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_held(t, root):
    """What is left of one tensor's values when they are held in 8 bits."""
    out = torch.empty_like(t)
    whole = t.numel() // BLOCK * BLOCK
    for part, width in ((slice(0, whole), BLOCK), (slice(whole, None), t.numel() - whole)):
        if not width or not t[part].numel():
            continue
        b = t[part].view(-1, width)
        top = b.abs().amax(dim=1, keepdim=True)
        z = torch.where(top >= TINY, top / 448.0, torch.zeros_like(top))
        q = _exact_e4m3(torch.where(z > 0, b / z, torch.zeros_like(b)))
        if root:
            q = torch.where((q == 0) & (b > 0) & (z > 0), torch.full_like(q, 2.0 ** -9), q)
        out[part] = (q * z).view(-1)
    return out


def _exact_adamw(case, s):
    h, t = HYPER, STEPS_BEFORE + 1
    sizes = _sizes(case)
    at, total = _places(sizes)
    names = ("p", "m", "v") if case["bits"] == 32 else ("p", "m_values", "v_values")
    got = {name: torch.zeros(total, dtype=torch.float64, device="cuda") for name in names}
    for i, n in zip(at, sizes):
        part = slice(i, i + n)
        g = s["g"][part].double() * float(s["grad_scale"])
        m, v = s["m"][part].double(), s["v"][part].double()
        if case["bits"] == 8:
            of = torch.arange(i, i + n, device="cuda") // BLOCK
            m, v = m * s["m_scale"].double()[of], (v * s["v_scale"].double()[of]) ** 2
        m = h["beta1"] * m + (1 - h["beta1"]) * g
        v = h["beta2"] * v + (1 - h["beta2"]) * g * g
        p = s["p"][part].double()
        got["p"][part] = p - h["lr"] * (h["weight_decay"] * p + m / (1 - h["beta1"] ** t) / ((v / (1 - h["beta2"] ** t)).sqrt() + h["eps"]))
        if case["bits"] == 8:
            m, v = _exact_held(m, False), _exact_held(v.sqrt(), True) ** 2
        got[names[1]][part], got[names[2]][part] = m, v
    got["copies"] = got["p"] if case["copies"] else None
    return got
