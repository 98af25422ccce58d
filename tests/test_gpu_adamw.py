"""The AdamW step on the GPU against its definition in 64 bits, and its 8-bit moments code by code."""
import pytest
import torch

from adapter_reference import e4m3

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import int8_mixed_precision_gb300 as dit  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
SIZES = [1, 7, 8, 255, 256, 257, 511, 4095, 4096, 4097, 9000, 0, 30720]
H = {"lr": 3e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1}


def make(sizes, p_dt, g_dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    ps = [(torch.randn(n, generator=g) * 0.02).to(p_dt) for n in sizes]
    gs = [(torch.randn(n, generator=g) * 0.01).to(g_dt) for n in sizes]
    return ps, gs, g


def step64(p, g, m, v, t, gs, h=H):
    """p, m, v after one step, from the textbook form in 64 bits."""
    g = g.double() * gs
    m = h["beta1"] * m.double() + (1 - h["beta1"]) * g
    v = h["beta2"] * v.double() + (1 - h["beta2"]) * g * g
    mh, vh = m / (1 - h["beta1"] ** t), v / (1 - h["beta2"] ** t)
    return p.double() - h["lr"] * (mh / (vh.sqrt() + h["eps"]) + h["weight_decay"] * p.double()), m, v


def near(got, want, rel, absolute, what):
    d = (got.double().cpu() - want).abs()
    assert bool((d <= rel * want.abs() + absolute).all()), (what, float((d - rel * want.abs()).max()))


@pytest.mark.parametrize("g_dt", [F32, BF16])
@pytest.mark.parametrize("p_dt", [F32, BF16])
def test_moments_in_32_bits(p_dt, g_dt):
    """Three steps.  m, v: two products and a sum, 3 roundings of 2^-24 of the larger term, each step; p: 8
    roundings of the step (at most 2 lr) and 2 of p each step, and in bf16 half a unit (8 significant bits: 2^-8) of p."""
    ps, gs, _ = make(SIZES, p_dt, g_dt)
    dp, dg = [p.cuda() for p in ps], [g.cuda() for g in gs]
    mom = dit.adamw_moments(dp, 32)
    copies = [torch.zeros(n, dtype=BF16, device="cuda") for n in SIZES]
    opt = dit.AdamW(dp, dg, **mom, copies=copies, **H)
    ms, vs = [torch.zeros(n).double() for n in SIZES], [torch.zeros(n).double() for n in SIZES]
    scale = torch.full((1,), 0.5, device="cuda")
    for t in range(1, 4):
        opt.step(grad_scale=scale)
        for i, n in enumerate(SIZES):
            # p is compared step by step from the kernel's own last value, so bf16's rounding does not add up
            want, ms[i], vs[i] = step64(ps[i], gs[i], ms[i], vs[i], t, 0.5)
            unit = 2.0 ** -8 if p_dt == BF16 else 2.0 ** -23
            near(dp[i], want, unit, 2 * H["lr"] * 24 * 2.0 ** -24, ("p", n, t))
            near(mom["m"][i], ms[i], 9 * 2.0 ** -24, 9 * 2.0 ** -24 * 0.05, ("m", n, t))
            near(mom["v"][i], vs[i], 12 * 2.0 ** -24, 0, ("v", n, t))
            ps[i] = dp[i].cpu()
            assert torch.equal(copies[i].cpu(), ps[i].to(BF16))
    assert opt.step_count == 3 and dit.device_status(opt.ws) == 0


def blocks_of(t):
    return torch.nn.functional.pad(t, (0, -t.numel() % 256)).view(-1, 256)


@pytest.mark.parametrize("p_dt,g_dt", [(F32, F32), (F32, BF16), (BF16, BF16)])
def test_moments_in_8_bits(p_dt, g_dt):
    """Steps from held moments: p as from the values that the codes stand for.  The kernel's m is off by three
    roundings of its two terms (which may cancel), u = sqrt(v) by 4 units of itself; a scale by as much as
    its block's values and 2 units more; a code is the nearest one to the exact value, or to one that is
    as far from it as that (the scaled value has the errors of the value and of its scale)."""
    ps, gs, gen = make(SIZES, p_dt, g_dt, seed=1)
    dp, dg = [p.cuda() for p in ps], [g.cuda() for g in gs]
    mom = dit.adamw_moments(dp, 8)
    values = {k: [torch.zeros(n, dtype=BF16, device="cuda") for n in SIZES] for k in ("m_values", "v_values")}
    opt = dit.AdamW(dp, dg, **mom, **values, **H)
    for t in range(1, 5):
        held = [(blocks_of(mom["m"][i].cpu().double()) * mom["m_scale"][i].cpu().double()[:, None],
                 blocks_of(mom["v"][i].cpu().double()) * mom["v_scale"][i].cpu().double()[:, None]) for i in range(len(SIZES))]
        for i, n in enumerate(SIZES):
            g = (torch.randn(n, generator=gen) * 0.01).to(g_dt)
            if n > 300:
                g[5] = 0.0
                g[290] = 3.0                        # a block of very uneven magnitudes
            gs[i] = g
            dg[i].copy_(g)
        opt.step()
        opt.export_moments()
        for i, n in enumerate(SIZES):
            m0, u0 = (h.view(-1)[:n] for h in held[i])
            want, m, v = step64(ps[i], gs[i], m0, u0 * u0, t, 1.0)
            unit = 2.0 ** -8 if p_dt == BF16 else 2.0 ** -23
            # u is the root of a small nonzero v at worst, and |m| / u at most 1 / sqrt(1 - beta2) in a step from zero;
            # from held moments it is bounded by the ratio of their scales: 16 lr covers this test's inputs
            near(dp[i], want, unit, 16 * H["lr"] * 24 * 2.0 ** -24, ("p", n, t))
            ps[i] = dp[i].cpu()
            terms = H["beta1"] * m0.abs() + (1 - H["beta1"]) * gs[i].double().abs()
            for name, x, off in (("m", m, 3 * 2.0 ** -24 * terms), ("v", v.sqrt(), 4 * 2.0 ** -24 * v.sqrt())):
                b = blocks_of(x)
                z = b.abs().amax(1) / 448
                z_off = blocks_of(off).amax(1) / 448 + 2 * 2.0 ** -24 * z
                got_z = mom[name + "_scale"][i].cpu().double()
                assert bool(((got_z - z).abs() <= z_off).all())
                z, z_off = (t.clamp(min=1e-300).repeat_interleave(256)[:n] for t in (z, z_off))
                norm = x / z
                off = off / z + norm.abs() * (z_off / z + 2 * 2.0 ** -24)
                code = e4m3(norm)
                if name == "v":
                    code = torch.where((code == 0) & (norm > 0), 2.0 ** -9 + 0 * code, code)
                got = mom[name][i].cpu().double()
                wrong = (got - norm).abs() > (code - norm).abs() + 2 * off
                assert not wrong.any(), (name, n, t, wrong.nonzero()[:3].tolist(), got[wrong][:3], code[wrong][:3], norm[wrong][:3])
                value = got * got_z.repeat_interleave(256)[:n]
                if name == "v":
                    value = value * value
                    assert bool((mom["v"][i].cpu().float()[x > 0] > 0).all())
                near(values[name + "_values"][i], value, 2.0 ** -8, 1e-38, (name, n, t))
    assert dit.device_status(opt.ws) == 0


def test_extreme_gradients():
    """A block whose moments vanish is held as zeros; a NaN or an infinity changes p and the moments of its own
    tensor's block alone."""
    n = 1024
    p = torch.full((n,), 0.5, device="cuda")
    g = torch.zeros(n, device="cuda")
    g[:256] = 1e-40
    g[300] = float("nan")
    g[600] = float("inf")
    g[768:] = 1e-3
    mom = dit.adamw_moments([p], 8)
    opt = dit.AdamW([p], [g], **mom, **H)
    opt.step()
    torch.cuda.synchronize()
    assert not mom["m_scale"][0][0].item() and not mom["m"][0][:256].float().any()
    got = p.cpu()
    keep = 0.5 * (1 - H["lr"] * H["weight_decay"])
    assert torch.isnan(got[300]) and bool(torch.isfinite(got[:300]).all())
    assert abs(float(got[301]) - keep) < 1e-6 and abs(float(got[256]) - keep) < 1e-6
    assert bool(torch.isfinite(got[768:]).all())
    assert torch.isnan(mom["m"][0][300].float()) and float(mom["m"][0][301].float()) == 0.0
    clean_p = torch.full((256,), 0.5, device="cuda")
    clean_g = torch.full((256,), 1e-3, device="cuda")
    other = dit.AdamW([clean_p], [clean_g], **dit.adamw_moments([clean_p], 8), **H)
    other.step()
    assert torch.equal(p[768:], clean_p)


def test_one_launch_gives_what_separate_steps_give():
    ps, gs, _ = make(SIZES, F32, BF16, seed=3)
    a, b = [p.cuda() for p in ps], [p.cuda() for p in ps]
    dg = [g.cuda() for g in gs]
    together = dit.AdamW(a, dg, **dit.adamw_moments(a, 8), **H)
    apart = [dit.AdamW([q], [g], **dit.adamw_moments([q], 8), **H) for q, g in zip(b, dg)]
    for _ in range(2):
        together.step()
        for o in apart:
            o.step()
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_checkpoint_resumes_bit_for_bit():
    ps, gs, _ = make([300, 5000], F32, F32, seed=4)
    for bits in (8, 32):
        a = [p.cuda() for p in ps]
        dg = [g.cuda() for g in gs]
        opt = dit.AdamW(a, dg, **dit.adamw_moments(a, bits), **H)
        opt.step()
        sd, b = opt.state_dict(), [p.clone() for p in a]
        opt.step()
        again = dit.AdamW(b, dg, **dit.adamw_moments(b, bits), **H)
        again.load_state_dict(sd)
        again.step()
        assert again.step_count == 2 and all(torch.equal(p, q) for p, q in zip(a, b))


def test_a_wrong_chunk_is_skipped_and_reported():
    p, g = torch.ones(10000, device="cuda"), torch.ones(10000, device="cuda")
    opt = dit.AdamW([p], [g], **dit.adamw_moments([p], 32), **H)
    opt._chunks[0, 0] = 5
    opt._chunks[1, 1] = 1000
    opt.step()
    torch.cuda.synchronize()
    assert dit.device_status(opt.ws) == 1 << 1
    assert torch.equal(p[:8192], torch.ones(8192, device="cuda")) and float(p[8192]) != 1.0


def test_another_stream():
    p, g = torch.ones(5000, device="cuda"), torch.ones(5000, device="cuda")
    opt = dit.AdamW([p], [g], **dit.adamw_moments([p], 8), **H)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    opt.step(stream=st)
    st.synchronize()
    assert abs(float(p[0]) - (1 - H["lr"] * 1.1)) < 1e-5


def test_a_tensor_of_more_than_2_31_elements():
    """One tensor whose last block lies past 2^31 elements, in 8 bits: its end is stepped like a small tensor's."""
    n, tail = 2 ** 31 + 600, 5000
    p = torch.zeros(n, dtype=BF16, device="cuda")
    g = torch.zeros(n, dtype=BF16, device="cuda")
    gen = torch.Generator().manual_seed(5)
    # the tail begins with a block of 256, as the small tensor's blocks do
    begin = (n - tail) // 256 * 256
    small_p, small_g = (torch.randn(n - begin, generator=gen).to(BF16).cuda() for _ in range(2))
    p[begin:], g[begin:] = small_p, small_g
    opt = dit.AdamW([p], [g], **dit.adamw_moments([p], 8), **H)
    other = dit.AdamW([small_p], [small_g], **dit.adamw_moments([small_p], 8), **H)
    for _ in range(2):
        opt.step()
        other.step()
    assert torch.equal(p[begin:], small_p)
    assert torch.equal(opt._lists["m"][0][begin:].view(torch.uint8), other._lists["m"][0].view(torch.uint8))
    assert torch.equal(opt._lists["v_scale"][0][begin // 256:], other._lists["v_scale"][0])
    assert not p[:begin:4099].any()
