"""Calls behind one another without a wait of the host: kernels start ahead of their predecessors' end and read what
earlier ones left.  Everything that a call reads ahead (the projection's y, gradients, weights that an optimiser
step has just written, h and e) is written right before it, through shared scratch and one workspace; each result has
the bits of the same call on an idle device."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import int8_mixed_precision_gb300 as dit  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def spread(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


class Layer:
    """One layer with its own batch: gemm (y), adapters, gemm (dx), their backward pass, an optimiser step."""

    def __init__(self, rng, seed, scratch, ws, cut):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        G, r = spread(rng, 1, 5), 8 * rng.randint(1, 16)
        K, N = 32 * spread(rng, 2, 60), 32 * spread(rng, 2, 60)
        lengths = [spread(rng, 1, 900) for _ in range(spread(rng, 1, 12))]
        T = sum(lengths)
        self.dtype, self.training = rng.choice([BF16, F32]), rng.random() < 0.75
        self.plan = dit.AdapterPlan(lengths, [rng.randrange(-1, G) for _ in lengths], G, training=self.training)
        self.masters = [new(G, r, K) * K ** -0.5, new(G, N, r) * 0.1]
        self.bank = dit.AdapterBank(*(m.to(BF16) for m in self.masters), torch.rand(G, device="cuda", generator=gen) + 0.5)
        self.w, self.w_t = (new(N, K) * K ** -0.5).to(BF16), (new(K, N) * K ** -0.5).to(BF16)
        self.x, self.dy = new(T, K).to(BF16), new(T, N).to(BF16)
        self.y, self.dx = torch.empty(T, N, dtype=self.dtype, device="cuda"), torch.empty(T, K, dtype=self.dtype, device="cuda")
        self.grads = [torch.empty_like(m) for m in self.masters]
        self.first = [m.clone() for m in self.masters]
        self.opt = dit.AdamW(self.masters, self.grads, **dit.adamw_moments(self.masters, 8), copies=[self.bank.a, self.bank.b], lr=1e-3)
        self.opt.ws, self.opt._tail = ws, (ws.data_ptr(), ws.numel())
        self.saved = dit.adapter_saved(self.plan, self.bank) if self.training else None
        assert dit.adapter_scratch(self.plan, self.bank).numel() <= scratch.numel()
        self.scratch, self.ws, self.cut = scratch, ws, cut

    def reset(self):
        for m, f, c in zip(self.masters, self.first, (self.bank.a, self.bank.b)):
            m.copy_(f)
            c.copy_(f)
        for name in ("m", "v", "m_scale", "v_scale"):
            for t in self.opt._lists[name]:
                t.view(torch.uint8).zero_()
        self.opt.step_count = 0

    def steps(self, env, between=lambda: None):
        """Two training steps (or two calls); `between` comes after every launch of the library."""
        env.setenv("DIT6_TEST_CUT", self.cut) if self.cut else env.delenv("DIT6_TEST_CUT", raising=False)
        for _ in range(2):
            dit.gemm_bf16(self.x, self.w, self.y, self.ws), between()
            dit.lora_forward(self.plan, self.bank, self.x, self.y, self.scratch, self.ws, saved=self.saved), between()
            if self.training:
                dit.gemm_bf16(self.dy, self.w_t, self.dx, self.ws), between()
                dit.lora_backward(self.plan, self.bank, self.x, self.dy, self.saved, *self.grads, self.scratch, self.ws, dx=self.dx)
                between()
                self.opt.step(), between()

    def results(self):
        return [self.y] + ([self.dx, *self.grads, *self.masters, self.bank.a, self.bank.b] if self.training else [])


@pytest.mark.parametrize("cut", ["", "2,0,1", "1,0,0"])
@pytest.mark.parametrize("seed", range(6))
def test_back_to_back_calls_give_the_bits_of_calls_on_an_idle_device(seed, cut, monkeypatch):
    rng = random.Random(seed)
    ws = dit.workspace()
    scratch = torch.empty(400 << 20, dtype=torch.uint8, device="cuda")
    layers = [Layer(rng, 10 * seed + i, scratch, ws, cut) for i in range(4)]
    wants = []
    for layer in layers:
        layer.reset()
        torch.cuda.synchronize()
        layer.steps(monkeypatch, torch.cuda.synchronize)
        wants.append([t.clone() for t in layer.results()])
    for _ in range(60):
        order = list(layers)
        rng.shuffle(order)
        for layer in order:
            layer.reset()
        for layer in order:
            layer.steps(monkeypatch)
        torch.cuda.synchronize()
        for layer, want in zip(layers, wants):
            assert all(torch.equal(a, b) for a, b in zip(layer.results(), want))
    assert dit.device_status(ws) == 0
