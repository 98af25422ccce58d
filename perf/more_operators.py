"""Cases that measure the operators between a block's QKV projection and its output projection.

Two operators are measured, each forward and with its backward pass.  Each has a plain form, made of
elementary torch operations in 32 bits, and the framework's calls.

* ``norm``: the norm of every query and key head (layer norm with weights and biases, or RMS norm with
  weights), then the rotation by positions with several axes.  Pair p of the rotated dimensions
  belongs to one axis a and is index i of that axis' d_a / 2 pairs; it turns by
  ``position[a] * scale[a] * theta ** (-2 i / d_a)``.
* ``attention``: softmax attention over documents packed in one batch.  A token sees its own document;
  with ``frame`` > 0 the document's first ``prefix`` tokens (text) are seen by all of it, and tokens
  behind them see the frames up to their own, each of ``frame`` tokens.  Queries may be the last tokens of a
  document whose keys and values lie in a cache.

``own`` chooses the form that ``run`` takes.  Token counts and the hidden size of 1920 (30 heads of 64)
are those of this repository's CogVideoX-2B-shaped and 1080p-shaped workloads; other sizes are generic.
"""
import random

import torch

own = False

THETA = 10000.0
EPS = 1e-6
TEXT = 226            # text tokens of a video
FRAME = (30, 45)      # rows and columns of patches of a video's frame


# ------------------------------------------------------------------------------------------
# the cases
# ------------------------------------------------------------------------------------------

def listed():
    norm = {"op": "norm", "train": False, "scale": 1.0, "offset": 0}
    attend = {"op": "attention", "train": False, "frame": 0, "prefix": 0, "cached": False}
    return [
        # one token of one request: pure latency
        {**norm, "name": "norm one token", "tokens": 1, "heads": 30, "kv_heads": 30, "dim": 64, "axes": 3, "kind": "layer", "interleaved": True},
        # one video and its text through a block
        {**norm, "name": "norm one video", "tokens": 17776, "heads": 30, "kv_heads": 30, "dim": 64, "axes": 3, "kind": "layer", "interleaved": True},
        # shared key heads, pairs half a head apart, positions far along the time axis
        {**norm, "name": "norm shared heads", "tokens": 2011, "heads": 24, "kv_heads": 8, "dim": 128, "axes": 3, "kind": "rms", "interleaved": False, "offset": 100003},
        # a 1080p video, its spatial positions scaled to the trained range
        {**norm, "name": "norm 1080p video", "tokens": 104746, "heads": 30, "kv_heads": 30, "dim": 64, "axes": 3, "kind": "rms", "interleaved": True, "scale": 0.375},
        # training on one short clip of odd length
        {**norm, "name": "norm train clip", "tokens": 1577, "heads": 12, "kv_heads": 4, "dim": 128, "axes": 2, "kind": "rms", "interleaved": False, "train": True},
        # training on one video
        {**norm, "name": "norm train video", "tokens": 17776, "heads": 30, "kv_heads": 30, "dim": 64, "axes": 3, "kind": "layer", "interleaved": True, "train": True},
        # four requests generate a token each over their caches
        {**attend, "name": "attention single tokens", "requests": 4, "tokens": 4, "keys": 23000, "heads": 16, "kv_heads": 4, "dim": 128, "layout": 1, "frame": 1, "cached": True},
        # prompts of odd lengths packed into one batch
        {**attend, "name": "attention packed prompts", "requests": 32, "tokens": 5003, "keys": 5003, "heads": 30, "kv_heads": 30, "dim": 64, "layout": 2},
        # the next frame of a video that is generated frame by frame, over the cache of the text and five frames
        {**attend, "name": "attention next frame", "requests": 1, "tokens": 1350, "keys": 226 + 6 * 1350, "heads": 30, "kv_heads": 30, "dim": 64, "layout": 3, "frame": 1350, "prefix": 226, "cached": True},
        # one video denoised as a whole
        {**attend, "name": "attention one video", "requests": 1, "tokens": 17776, "keys": 17776, "heads": 30, "kv_heads": 30, "dim": 64, "layout": 4},
        # training on clips of odd lengths, causal by short frames behind a prompt, shared key heads
        {**attend, "name": "attention train clips", "requests": 9, "tokens": 5003, "keys": 5003, "heads": 12, "kv_heads": 4, "dim": 128, "layout": 5, "frame": 60, "prefix": 33, "train": True},
        # training on one video
        {**attend, "name": "attention train video", "requests": 1, "tokens": 17776, "keys": 17776, "heads": 30, "kv_heads": 30, "dim": 64, "layout": 6, "train": True},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kv_heads = _log(rng, 1, 16)
    heads = kv_heads * rng.choice([1, 1, 2, 3, 4])
    dim = rng.choice([64, 64, 128, 128, 40, 72, 96])
    train = rng.random() < 0.4
    if rng.random() < 0.45:
        interleaved = rng.random() < 0.6
        return {"op": "norm", "train": train, "tokens": _log(rng, 1, 60000), "heads": heads, "kv_heads": kv_heads, "dim": dim, "axes": rng.randint(1, 3),
                "kind": rng.choice(["layer", "rms"]), "interleaved": interleaved, "scale": rng.choice([1.0, 1.0, 0.5, 0.375]), "offset": rng.choice([0, 0, 0, 4097, 100003, 1000003])}
    cached = not train and rng.random() < 0.4
    frame = rng.choice([0, 0, 1, _log(rng, 2, 1500)])
    requests = _log(rng, 1, 40)
    keys = max(requests, _log(rng, 5, 14000))
    if train or not cached:
        keys = max(requests, min(keys, 9000)) if train else keys
        tokens = keys
    else:
        tokens = min(keys, requests * _log(rng, 1, 1500))
    return {"op": "attention", "train": train, "requests": requests, "tokens": tokens, "keys": keys, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "layout": rng.randrange(1000, 1 << 30), "frame": frame, "prefix": rng.choice([0, _log(rng, 1, 300)]) if frame else 0, "cached": cached}


def _parts(total, count, rng):
    """`total` cut into `count` random parts; among four or more, one is empty and one has one token."""
    cuts = sorted(rng.randint(0, total) for _ in range(count - 1))
    if count > 3 and total > 1:
        cuts[0], cuts[1] = 0, 1
        cuts = sorted(cuts)
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _documents(case):
    """(query tokens, key tokens) of every document."""
    rng = random.Random(case["layout"])
    if not case["cached"]:
        lengths = _parts(case["tokens"], case["requests"], rng)
        return lengths, lengths
    n = case["requests"]
    queries = [case["tokens"] // n + (i < case["tokens"] % n) for i in range(n)]
    spare = _parts(case["keys"] - case["tokens"], n, rng)
    return queries, [q + s for q, s in zip(queries, spare)]


def _split(case):
    """Dimensions of each axis: even numbers of pairs' halves, about a quarter for the first of three axes."""
    d, axes = case["dim"], case["axes"]
    if axes == 1:
        return [d]
    if axes == 2:
        return [d // 4 * 2, d - d // 4 * 2]
    first = d // 8 * 2
    second = (d - first) // 4 * 2
    return [first, second, d - first - second]


def _visible(case):
    """Visible pairs of one head."""
    total = 0
    for n, m in zip(*_documents(case)):
        if not case["frame"]:
            total += n * m
            continue
        f, pre = case["frame"], case["prefix"]
        total += sum(min(m, pre if p < pre else pre + ((p - pre) // f + 1) * f) for p in range(m - n, m))
    return total


def work(case):
    heads, kv_heads, d, t = case["heads"], case["kv_heads"], case["dim"], case["tokens"]
    if case["op"] == "norm":
        elements = t * (heads + kv_heads) * d
        # forward reads and writes each element; backward reads it and its gradient and writes one
        return {"bytes": elements * (10 if case["train"] else 4) + 4 * t * case["axes"], "flops": elements * (40 if case["train"] else 14)}
    keys = sum(_documents(case)[1])
    q, kv = t * heads * d, keys * kv_heads * d
    pairs = _visible(case) * heads * d
    if not case["train"]:
        return {"bytes": 2 * (2 * q + 2 * kv), "flops": 4 * pairs}
    # forward and backward: q, k, v and the output's gradient read once, the output and three gradients written
    return {"bytes": 2 * (4 * q + 4 * kv), "flops": 14 * pairs}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _positions(case):
    """int32 [tokens, axes]: text tokens at the origin, then the patches of each frame."""
    t = case["tokens"]
    text = min(TEXT, t // 4)
    i = torch.arange(t - text, device="cuda")
    rows, cols = FRAME
    axes = [i // (rows * cols) + case["offset"], i // cols % rows, i % cols]
    if case["axes"] == 1:
        axes = [i + case["offset"]]
    axes = axes[: case["axes"]]
    return torch.cat([torch.zeros(text, case["axes"], dtype=torch.int64, device="cuda"), torch.stack(axes, 1)]).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    new = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
    bf16 = torch.bfloat16
    t, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    s = {"case": case}
    if case["op"] == "norm":
        # the projection's output, a few of its channels larger, with the values behind queries and keys
        x = new(t, (h + 2 * hk) * d) * (1.0 + 4.0 * (torch.rand((h + 2 * hk) * d, device="cuda", generator=g) < 0.02))
        x = (x + 0.1 * new((h + 2 * hk) * d)).to(bf16)
        s["q"], s["k"] = x[:, : h * d].view(t, h, d), x[:, h * d: (h + hk) * d].view(t, hk, d)
        s["params"] = 1.0 + 0.3 * new(4 if case["kind"] == "layer" else 2, d)
        if case["kind"] == "layer":
            s["params"][1::2] -= 1.0  # the biases
        s["positions"] = _positions(case)
        s["out"] = torch.empty(t, (h + hk) * d, dtype=bf16, device="cuda")
        if case["train"]:
            dy = new(t, (h + hk) * d).to(bf16)
            s["dy"] = dy
            s["dx"] = torch.empty_like(x[:, : (h + hk) * d], memory_format=torch.contiguous_format)
            s["dparams"] = torch.empty_like(s["params"])
        if own:  # what a program keeps for all blocks and steps
            import int8_mixed_precision_gb300 as dit
            s["norm"] = dit.QKNorm(s["params"], case["kind"], EPS)
            s["rotary"] = dit.Rotary(_split(case), d, theta=THETA, scale=case["scale"], interleaved=case["interleaved"])
            s["ws"] = dit.workspace()
            s["scratch"] = dit.qk_norm_scratch(d) if case["train"] else None
        return s
    queries, keys = _documents(case)
    s["queries"], s["keys"] = queries, keys
    gain = 0.5 + torch.rand(h, 1, device="cuda", generator=g)  # heads attend more or less sharply
    if case["cached"]:
        # a cache with room behind each document's keys
        room = max(keys) + 64
        s["q"] = (new(t, h, d) * gain).to(bf16)
        s["k"], s["v"] = new(len(keys) * room, hk, d).to(bf16), new(len(keys) * room, hk, d).to(bf16)
        s["begins"] = [i * room for i in range(len(keys))]
    else:
        x = new(t, h + 2 * hk, d)
        x[:, :h] *= gain
        x = x.to(bf16)
        s["q"], s["k"], s["v"] = x[:, :h], x[:, h: h + hk], x[:, h + hk:]
        s["begins"] = [sum(keys[:i]) for i in range(len(keys))]
    s["out"] = torch.empty(t, h, d, dtype=bf16, device="cuda")
    if case["train"]:
        s["dout"] = new(t, h, d).to(bf16)
        s["grad"] = torch.empty(t, h + 2 * hk, d, dtype=bf16, device="cuda")
    if own:  # the plan of a batch serves every block and step
        import int8_mixed_precision_gb300 as dit
        s["ws"] = dit.workspace()
        s["plan"] = dit.AttentionPlan(queries, h, d, kv_heads=hk, kv_lengths=keys, kv_begins=s["begins"] if case["cached"] else None,
                                      frame=case["frame"], prefix=case["prefix"], training=case["train"])
        s["scratch"] = dit.attention_scratch(s["plan"])
        s["saved"] = dit.attention_saved(s["plan"]) if case["train"] else None
    return s


# ------------------------------------------------------------------------------------------
# the operators
# ------------------------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return _plain_norm(s) if s["case"]["op"] == "norm" else _plain_attention(s)


def _own(s):
    import int8_mixed_precision_gb300 as dit
    case = s["case"]
    t, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "norm":
        out = s["out"].view(t, h + hk, d)
        dit.qk_norm_rope(s["q"], s["k"], out[:, :h], out[:, h:], s["norm"], s["rotary"], s["positions"])
        if not case["train"]:
            return s["out"]
        dy, dx = s["dy"].view(t, h + hk, d), s["dx"].view(t, h + hk, d)
        dit.qk_norm_rope_backward(s["q"], s["k"], dy[:, :h], dy[:, h:], dx[:, :h], dx[:, h:], s["norm"], s["rotary"], s["positions"],
                                  s["dparams"], s["scratch"], s["ws"])
        return {"out": s["out"], "dx": s["dx"], "dparams": s["dparams"]}
    dit.attention(s["plan"], s["q"], s["k"], s["v"], s["out"], s["scratch"], s["ws"], saved=s["saved"])
    if not case["train"]:
        return s["out"]
    g = s["grad"]
    dit.attention_backward(s["plan"], s["q"], s["k"], s["v"], s["out"], s["dout"], s["saved"], g[:, :h], g[:, h:h + hk], g[:, h + hk:], s["scratch"], s["ws"])
    return {"out": s["out"], "grad": g}


def _cos_sin(s):
    """[tokens, 1, pairs] each; the angles in 64 bits, far positions need them."""
    case = s["case"]
    parts = []
    for a, d in enumerate(_split(case)):
        freq = THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
        parts.append(s["positions"][:, a, None].double() * case["scale"] * freq)
    angle = torch.cat(parts, 1)[:, None]
    return angle.cos().float(), angle.sin().float()


def _turn(x, cos, sin, interleaved):
    half = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    y = a * cos - b * sin, a * sin + b * cos
    return torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)


def _plain_norm(s):
    case = s["case"]
    t, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    layer, pairs = case["kind"] == "layer", case["interleaved"]
    cos, sin = _cos_sin(s)
    out = s["out"].view(t, h + hk, d)
    for i, x, at in ((0, s["q"], slice(0, h)), (1, s["k"], slice(h, h + hk))):
        weight, bias = (s["params"][2 * i], s["params"][2 * i + 1]) if layer else (s["params"][i], 0.0)
        x = x.float()
        x = x - x.mean(-1, keepdim=True) if layer else x
        rstd = (x.square().mean(-1, keepdim=True) + EPS) ** -0.5
        hat = x * rstd
        out[:, at] = _turn(hat * weight + bias, cos, sin, pairs).to(out.dtype)
        if case["train"]:
            dn = _turn(s["dy"].view(t, h + hk, d)[:, at].float(), cos, -sin, pairs)
            if layer:
                s["dparams"][2 * i], s["dparams"][2 * i + 1] = (dn * hat).sum((0, 1)), dn.sum((0, 1))
            else:
                s["dparams"][i] = (dn * hat).sum((0, 1))
            g = dn * weight
            g = g - hat * (g * hat).mean(-1, keepdim=True) - (g.mean(-1, keepdim=True) if layer else 0.0)
            s["dx"].view(t, h + hk, d)[:, at] = (g * rstd).to(out.dtype)
    return {"out": s["out"], "dx": s["dx"], "dparams": s["dparams"]} if case["train"] else s["out"]


def _seen(case, n, m):
    """bool [n, m]: which of a document's m keys its last n tokens see; None: all."""
    f, pre = case["frame"], case["prefix"]
    if not f:
        return None
    p = torch.arange(m - n, m, device="cuda")
    upto = torch.where(p < pre, pre, pre + ((p - pre) // f + 1) * f)
    return torch.arange(m, device="cuda")[None] < upto[:, None]


def _plain_attention(s):
    case = s["case"]
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    group, scale, q0 = h // hk, d ** -0.5, 0
    for n, m, k0 in zip(s["queries"], s["keys"], s["begins"]):
        seen = _seen(case, n, m)
        # as many key heads at a time as leave the scores below 4 GB
        step = max(1, min(hk, (1 << 30) // max(1, n * m * group)))
        for j in range(0, hk, step):
            kv, qs = slice(j, min(hk, j + step)), slice(j * group, min(hk, j + step) * group)
            if not n:
                continue
            q = s["q"][q0:q0 + n, qs].float().transpose(0, 1)
            k = s["k"][k0:k0 + m, kv].float().transpose(0, 1).repeat_interleave(group, 0)
            v = s["v"][k0:k0 + m, kv].float().transpose(0, 1).repeat_interleave(group, 0)
            p = (q @ k.transpose(1, 2)) * scale
            if seen is not None:
                p.masked_fill_(~seen, float("-inf"))
            p = p.sub_(p.amax(-1, keepdim=True)).exp_()
            p /= p.sum(-1, keepdim=True)
            s["out"][q0:q0 + n, qs] = (p @ v).transpose(0, 1).to(torch.bfloat16)
            if case["train"]:
                do = s["dout"][q0:q0 + n, qs].float().transpose(0, 1)
                dv = p.transpose(1, 2) @ do
                dp = do @ v.transpose(1, 2)
                dp -= (dp * p).sum(-1, keepdim=True)
                dp *= p
                del p
                dq, dk = (dp @ k) * scale, (dp.transpose(1, 2) @ q) * scale
                g = s["grad"]
                g[q0:q0 + n, qs] = dq.transpose(0, 1).to(g.dtype)
                for at, t in ((h, dk), (h + hk, dv)):
                    g[k0:k0 + m, at + j:at + kv.stop] = t.view(-1, group, m, d).sum(1).transpose(0, 1).to(g.dtype)
        q0 += n
    return {"out": s["out"], "grad": s["grad"]} if case["train"] else s["out"]


# ------------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(case, s) if case["op"] == "norm" else _exact_attention(case, s)


def _exact_norm(case, s):
    t, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    dims, R = _split(case), sum(_split(case))
    # the rotation of each token as complex factors, one for each pair, and where a pair's two elements are
    angle = torch.empty(t, R // 2, dtype=torch.float64, device="cuda")
    at = 0
    for a, da in enumerate(dims):
        for i in range(da // 2):
            angle[:, at] = s["positions"][:, a].double() * case["scale"] / THETA ** (2.0 * i / da)
            at += 1
    factor = torch.polar(torch.ones_like(angle), angle)
    p = torch.arange(R // 2, device="cuda")
    one, two = (2 * p, 2 * p + 1) if case["interleaved"] else (p, p + R // 2)
    out, dx = torch.empty(t, h + hk, d, dtype=torch.float64, device="cuda"), torch.empty(t, h + hk, d, dtype=torch.float64, device="cuda")
    dparams = torch.zeros(s["params"].shape, dtype=torch.float64, device="cuda")
    for head in range(h + hk):
        x = (s["q"][:, head] if head < h else s["k"][:, head - h]).double()
        i = int(head >= h)
        if case["kind"] == "layer":
            w, b, row = s["params"][2 * i].double(), s["params"][2 * i + 1].double(), 2 * i
            var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        else:
            w, b, row = s["params"][i].double(), torch.zeros(d, dtype=torch.float64, device="cuda"), i
            var, mean = torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / d, torch.zeros(t, 1, dtype=torch.float64, device="cuda")
        sigma = torch.sqrt(var + EPS)
        z = (x - mean) / sigma
        n = torch.addcmul(b, z, w)
        c = torch.complex(n[:, one], n[:, two]) * factor
        out[:, head, one], out[:, head, two] = c.real, c.imag
        if case["train"]:
            dy = s["dy"].view(t, h + hk, d)[:, head].double()
            c = torch.complex(dy[:, one], dy[:, two]) * factor.conj()
            dn = torch.empty_like(dy)
            dn[:, one], dn[:, two] = c.real, c.imag
            dparams[row] += torch.einsum("td,td->d", dn, z)
            if case["kind"] == "layer":
                dparams[row + 1] += dn.sum(0)
            dz = dn * w
            back = dz - z * (torch.einsum("td,td->t", dz, z) / d)[:, None]
            if case["kind"] == "layer":
                back = back - dz.mean(1, keepdim=True)
            dx[:, head] = back / sigma
    if not case["train"]:
        return out.view(t, -1)
    return {"out": out.view(t, -1), "dx": dx.view(t, -1), "dparams": dparams}


def _exact_attention(case, s):
    if work(case)["flops"] > 1e13:  # about 20 seconds in 64 bits
        return None
    t, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    f, pre = case["frame"], case["prefix"]
    out = torch.zeros(t, h, d, dtype=torch.float64, device="cuda")
    grad = torch.zeros(t, h + 2 * hk, d, dtype=torch.float64, device="cuda") if case["train"] else None
    q0 = 0
    for n, m, k0 in zip(s["queries"], s["keys"], s["begins"]):
        for head in range(h if n else 0):
            of = head // (h // hk)
            k, v = s["k"][k0:k0 + m, of].double(), s["v"][k0:k0 + m, of].double()
            for r in range(0, n, 8192):  # some rows at a time
                rows = slice(q0 + r, q0 + min(n, r + 8192))
                q = s["q"][rows, head].double()
                scores = torch.einsum("nd,md->nm", q, k) / d ** 0.5
                if f:
                    at = torch.arange(r, min(n, r + 8192), device="cuda") + (m - n)
                    key = torch.arange(m, device="cuda")
                    # a key is seen from its own frame on, one of the prefix from the start
                    since = torch.where(key < pre, torch.zeros_like(key), pre + torch.div(key - pre, f, rounding_mode="floor") * f)
                    scores[at[:, None] < since[None]] = -torch.inf
                w = torch.exp(scores - torch.logsumexp(scores, 1, keepdim=True))
                del scores
                o = torch.einsum("nm,md->nd", w, v)
                out[rows, head] = o
                if grad is not None:
                    do = s["dout"][rows, head].double()
                    grad[k0:k0 + m, h + hk + of] += torch.einsum("nm,nd->md", w, do)
                    ds = (torch.einsum("nd,md->nm", do, v) - (do * o).sum(1, keepdim=True)) * w
                    grad[rows, head] = torch.einsum("nm,md->nd", ds, k) / d ** 0.5
                    grad[k0:k0 + m, h + of] += torch.einsum("nm,nd->md", ds, q) / d ** 0.5
        q0 += n
    return out if grad is None else {"out": out, "grad": grad}
