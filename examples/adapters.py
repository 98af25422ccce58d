"""Train low-rank adapters beside a frozen quantised projection, then serve them to many requests at once.

A projection's weight exists only in its quantised forms (NVFP4 and INT8).  Two tasks want the
projection plus a low-rank change of it; each gets an adapter, trained on a batch that holds both
(one forward and one backward call for all adapters), with AdamW on fp32 masters whose moments
are held in 8 bits.  The trained adapters then serve a batch of short requests, some with either adapter
and some with none, in one launch beside the same projection.

  python examples/adapters.py [--steps 200]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import int8_mixed_precision_gb300 as dit  # noqa: E402


def main(steps: int = 200, k: int = 512, n: int = 768, rank: int = 16, rows: int = 600) -> dict:
    gen = torch.Generator(device="cuda").manual_seed(0)
    new = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    bf16, tasks = torch.bfloat16, 2

    # the frozen projection, and what each task wants of it
    weight = new(n, k) * k ** -0.5
    ws = dit.workspace()
    projection = dit.RoutedLinear(dit.QuantizedWeight(weight, 64, ws), rows, ws)
    wanted = [new(n, 8) @ new(8, k) * (0.3 / k) ** 0.5 for _ in range(tasks)]

    # fp32 masters of both adapters' factors with their bf16 copies, and the optimiser over them
    a, b = new(tasks, rank, k) * k ** -0.5, torch.zeros(tasks, n, rank, device="cuda")
    bank = dit.AdapterBank(a.to(bf16), b.to(bf16), torch.ones(tasks, device="cuda"))
    da, db = torch.empty_like(a), torch.empty_like(b)
    layer = dit.AdaptedLinear(projection, bank)
    opt = dit.AdamW([a, b], [da, db], **dit.adamw_moments([a, b], 8), copies=[bank.a, bank.b], lr=2e-3, weight_decay=0.0)

    # training: one batch holds rows of both tasks
    lengths = [rows // 2 + 7, rows - rows // 2 - 7]
    plan = dit.AdapterPlan(lengths, [0, 1], tasks, training=True)
    scratch, saved = dit.adapter_scratch(plan, bank), dit.adapter_saved(plan, bank)
    y, dx = torch.empty(rows, n, device="cuda"), torch.empty(rows, k, device="cuda")
    losses = []
    for _ in range(steps):
        x = new(rows, k).to(bf16)
        target = torch.cat([part.float() @ (weight + w).T for part, w in zip(x.split(lengths), wanted)])
        layer(x, dit.ROUTE_INT8, y, plan, scratch, saved=saved)
        off = y - target
        losses.append(off.square().mean())
        layer.backward(x, (off * (2.0 / rows)).to(bf16), plan, saved, da, db, dx, scratch)
        opt.step()

    # serving: requests of one to five rows, adapter 0, adapter 1 or none
    lengths = [1 + i % 5 for i in range(40)]
    adapters = [i % 3 - 1 for i in range(40)]
    plan = dit.AdapterPlan(lengths, adapters, tasks)
    scratch = dit.adapter_scratch(plan, bank)
    x = new(sum(lengths), k).to(bf16)
    y = torch.empty(sum(lengths), n, device="cuda")
    layer(x, dit.ROUTE_INT8, y, plan, scratch)
    of_row = torch.repeat_interleave(torch.tensor(adapters), torch.tensor(lengths)).cuda()
    errors = {}
    for g in (-1, 0, 1):
        at = of_row == g
        target = x[at].float() @ (weight + (wanted[g] if g >= 0 else 0)).T
        errors[g] = float((y[at] - target).norm() / target.norm())
    assert dit.device_status(ws) == 0
    return {"loss": [float(losses[0]), float(losses[-1])], "errors": errors, "rows": sum(lengths)}


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=200)
    got = main(ap.parse_args().steps)
    print("training loss: %.4f -> %.4f" % tuple(got["loss"]))
    print("serving %d rows, relative error: without an adapter %.4f, with the first %.4f, with the second %.4f" % (
        got["rows"], got["errors"][-1], got["errors"][0], got["errors"][1]))
