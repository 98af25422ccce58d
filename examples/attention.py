"""A block's attention part: trained through its norms and adapters, then run between quantised projections.

Several clips of different sizes, each behind its text prompt, are packed into one batch.  The frozen QKV and output projections
exist in quantised form only; low-rank adapters beside the QKV projection and the norms' weights of queries and keys are
trained to match a target, with the gradient passing back through attention, rotation and norms.  The block then
runs as it is served: QKV projection, norms and rotation, attention, output projection.

  python examples/attention.py [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import int8_mixed_precision_gb300 as dit  # noqa: E402


def grid_positions(text: int, frames: int, rows: int, cols: int):
    """(time, row, column) of a clip's tokens: the prompt at the origin, then the patches of each frame."""
    patches = torch.cartesian_prod(torch.arange(frames), torch.arange(rows), torch.arange(cols))
    return torch.cat([torch.zeros(text, 3, dtype=torch.int64), patches]).to(torch.int32)


class Trainable:
    """Attention of one block for training: adapters beside the QKV projection, norms, rotation, attention."""

    def __init__(self, layer, norm, rotary, heads, dim, adapter_plan, plan, positions):
        self.layer, self.norm, self.rotary, self.h, self.d = layer, norm, rotary, heads, dim
        self.adapters, self.plan, self.positions = adapter_plan, plan, positions
        rows, device, bf16 = plan.q_rows, positions.device, torch.bfloat16
        self.ws = layer.linear.ws
        self.qkv, self.dqkv = (torch.empty(rows, 3 * heads, dim, dtype=bf16, device=device) for _ in range(2))
        self.qk, self.dqk = (torch.empty(rows, 2 * heads, dim, dtype=bf16, device=device) for _ in range(2))
        self.out = torch.empty(rows, heads, dim, dtype=bf16, device=device)
        self.dx = torch.empty(rows, layer.bank.k, dtype=bf16, device=device)
        self.dparams = torch.empty_like(norm.params)
        self.da, self.db = torch.empty(layer.bank.a.shape, device=device), torch.empty(layer.bank.b.shape, device=device)
        self.adapter_scratch, self.adapter_saved = dit.adapter_scratch(adapter_plan, layer.bank), dit.adapter_saved(adapter_plan, layer.bank)
        self.scratch, self.saved, self.norm_scratch = dit.attention_scratch(plan), dit.attention_saved(plan), dit.qk_norm_scratch(dim, device)

    def forward(self, x):
        h = self.h
        self.layer(x, dit.ROUTE_INT8, self.qkv.view(len(x), -1), self.adapters, self.adapter_scratch, saved=self.adapter_saved)
        dit.qk_norm_rope(self.qkv[:, :h], self.qkv[:, h:2 * h], self.qk[:, :h], self.qk[:, h:], self.norm, self.rotary, self.positions)
        dit.attention(self.plan, self.qk[:, :h], self.qk[:, h:], self.qkv[:, 2 * h:], self.out, self.scratch, self.ws, saved=self.saved)
        return self.out

    def backward(self, x, dout):
        """Gradients of the adapters (da, db), the norms' weights (dparams) and the adapters' part of dx."""
        h = self.h
        dit.attention_backward(self.plan, self.qk[:, :h], self.qk[:, h:], self.qkv[:, 2 * h:], self.out, dout, self.saved, self.dqk[:, :h],
                               self.dqk[:, h:], self.dqkv[:, 2 * h:], self.scratch, self.ws)
        dit.qk_norm_rope_backward(self.qkv[:, :h], self.qkv[:, h:2 * h], self.dqk[:, :h], self.dqk[:, h:], self.dqkv[:, :h], self.dqkv[:, h:2 * h],
                                  self.norm, self.rotary, self.positions, self.dparams, self.norm_scratch, self.ws)
        self.layer.backward(x, self.dqkv.view(len(x), -1), self.adapters, self.adapter_saved, self.da, self.db, self.dx, self.adapter_scratch)


def main(steps: int = 60, heads: int = 4, dim: int = 64, rank: int = 8) -> dict:
    gen = torch.Generator(device="cuda").manual_seed(0)
    new = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    bf16, hidden = torch.bfloat16, heads * dim

    # three clips in one batch, each with its prompt
    clips = [(17, 3, 5, 7), (9, 2, 4, 4), (26, 1, 9, 6)]
    positions = torch.cat([grid_positions(*c) for c in clips]).cuda()
    lengths = [text + f * r * c for text, f, r, c in clips]
    rows = sum(lengths)

    ws = dit.workspace()
    w_qkv, w_out = new(3 * hidden, hidden) * hidden ** -0.5, new(hidden, hidden) * hidden ** -0.5
    qkv = dit.RoutedLinear(dit.QuantizedWeight(w_qkv, 64, ws), rows, ws)
    out = dit.RoutedLinear(dit.QuantizedWeight(w_out, 64, ws), rows, ws)
    params = torch.ones(2, dim, device="cuda")
    norm, rotary = dit.QKNorm(params, "rms"), dit.Rotary((16, 24, 24), dim)

    # adapters beside the QKV projection, fp32 masters and bf16 copies, and the optimiser over them and the norms' weights
    a, b = new(1, rank, hidden) * hidden ** -0.5, torch.zeros(1, 3 * hidden, rank, device="cuda")
    bank = dit.AdapterBank(a.to(bf16), b.to(bf16), torch.ones(1, device="cuda"))
    block = Trainable(dit.AdaptedLinear(qkv, bank), norm, rotary, heads, dim, dit.AdapterPlan([rows], [0], 1, training=True),
                      dit.AttentionPlan(lengths, heads, dim, training=True), positions)
    grads, masters = [block.da, block.db], [a, b]
    opt = dit.AdamW(masters, grads, **dit.adamw_moments(masters), copies=[bank.a, bank.b], lr=2e-3, weight_decay=0.0)
    opt_norm = dit.AdamW([params], [block.dparams], **dit.adamw_moments([params]), lr=1e-2, weight_decay=0.0)

    x, target = new(rows, hidden).to(bf16), new(rows, heads, dim) * 0.3
    losses = []
    for _ in range(steps):
        off = block.forward(x).float() - target
        losses.append(off.square().mean())
        block.backward(x, (off * (2.0 / rows)).to(bf16))
        opt.step()
        opt_norm.step()

    # the same part of a block as it is served, without the adapters
    part = dit.RoutedAttention(qkv, out, heads, norm=norm, rotary=rotary)
    plan = dit.AttentionPlan(lengths, heads, dim)
    y = torch.empty(rows, hidden, dtype=bf16, device="cuda")
    part(x, (dit.ROUTE_INT8, dit.ROUTE_NVFP4), y, plan, block.qkv, block.out, dit.attention_scratch(plan), positions)
    assert dit.device_status(ws) == 0
    return {"loss": [float(losses[0]), float(losses[-1])], "rows": rows, "y": y}


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    got = main(ap.parse_args().steps)
    print("%d tokens of three clips, training loss %.4f -> %.4f" % (got["rows"], *got["loss"]))
