"""Synchronous data-parallel training of a small MLP, all of it in the library's
kernels: P logical workers on one GPU, each with its own batch.

Per iteration, for every worker: the forward pass (two linear layers with fused
bias, GELU and residual), the backward pass straight into the worker's flat
binary32 gradient buffer, and, as soon as the output layer's gradients are there,
the overlapped all-reduce of its bucket; then the Muon step on every worker's
copy of the weight matrices (the biases take plain SGD).

    python examples/train_mlp.py --workers 4 --steps 30

The task is synthetic: the targets come from a fixed random network.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gradient_all_reduce_ddl_gb300 import ddl  # noqa: E402


class Worker:
    """A worker's parameters (binary32 in one flat buffer, bfloat16 copies for the products), gradients and batch."""

    def __init__(self, layout, n, params, width, batch, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.layout = layout
        self.params = params.clone()
        self.grad = torch.zeros(n, device="cuda")
        self.x = torch.randn(batch, width, generator=gen, device="cuda").bfloat16()
        self.h = torch.empty(batch, layout["w1"][1][0], dtype=torch.bfloat16, device="cuda")
        self.z = torch.empty_like(self.h)
        self.y = torch.empty_like(self.x)
        self.dh, self.target = torch.empty_like(self.h), None

    def view(self, flat, name):
        offset, shape = self.layout[name]
        count = shape[0] * (shape[1] if len(shape) > 1 else 1)
        return flat[offset:offset + count].view(shape)

    def operand(self, name):
        return self.view(self.params, name).bfloat16()


def train(workers=4, width=256, hidden=768, batch=512, steps=30, lr=0.02, seed=1, report=print):
    """Trains and returns the losses and the workers."""
    shapes = {"w1": (hidden, width), "b1": (hidden,), "w2": (width, hidden), "b2": (width,)}
    layout, n = {}, 0
    for name, shape in shapes.items():  # forward order at increasing addresses, as the plan's layer list
        layout[name] = (n, shape)
        n += shape[0] * (shape[1] if len(shape) > 1 else 1)
    matrices = [(layout[k][0], *layout[k][1]) for k in ("w1", "w2")]
    tensors = [s[0] * (s[1] if len(s) > 1 else 1) for s in shapes.values()]

    gen = torch.Generator(device="cuda").manual_seed(seed)
    teacher, start = torch.randn(n, generator=gen, device="cuda"), torch.randn(n, generator=gen, device="cuda")
    for flat, scale in ((teacher, 1.5), (start, 1.0)):
        for name, (offset, shape) in layout.items():
            part = flat[offset:offset + shape[0] * (shape[1] if len(shape) > 1 else 1)]
            part.mul_(scale * shape[1] ** -0.5 if len(shape) > 1 else 0.0)
    team = [Worker(layout, n, start, width, batch, seed + 10 + r) for r in range(workers)]

    up = ddl.Linear(width, hidden, batch, "bf16", "gelu")
    down = ddl.Linear(hidden, width, batch, "bf16", "none")
    muon = ddl.Ortho(matrices, "f32")
    mom = torch.zeros(n, device="cuda")
    # a bucket per layer, the output layer's first: its all-reduce runs under the input layer's backward pass
    plan = ddl.Plan(workers, n, "f32", "ring", layers=tensors, bucket_bytes=4 * (width * hidden + width))

    def forward(w, params):
        w.params, kept = params, w.params
        up.forward(w.x, w.operand("w1"), w.h, bias=w.operand("b1"), z=w.z)
        down.forward(w.h, w.operand("w2"), w.y, bias=w.operand("b2"), residual=w.x)
        w.params = kept
        return w.y

    for w in team:
        w.target = forward(w, teacher).clone()
    losses = []
    for step in range(steps):
        plan.overlap_begin([w.grad for w in team], 1.0 / workers)
        total, pending = 0.0, []
        for w in team:
            y = forward(w, w.params)
            off = y.float() - w.target.float()
            total = total + off.square().mean()
            dy = (off * (2.0 / off.numel()) * 4096).bfloat16()  # scaled, so that small gradients keep their bits
            down.backward(dy, w.h, w.operand("w2"), dx=w.dh, dw=w.view(w.grad, "w2"), db=w.view(w.grad, "b2"))
            pending.append((w, w.dh.clone(), w.z.clone()))
        plan.bucket_ready(0)
        for w, dh, z in pending:
            up.backward(dh, w.x, z=z, dw=w.view(w.grad, "w1"), db=w.view(w.grad, "b1"))
        plan.overlap_end()
        muon.muon(team[0].grad, [w.params for w in team], mom, lr)
        for w in team:
            for name in ("b1", "b2"):
                w.view(w.params, name).sub_(w.view(w.grad, name), alpha=lr / 4096)
        losses.append(float(total) / workers)
        if report and step % 5 == 0:
            report(f"step {step:3d}  loss {losses[-1]:.5f}")
    for handle in (up, down, muon, plan):
        handle.check()
        handle.close()
    return losses, team


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--workers", type=int, default=4)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    got, _ = train(workers=a.workers, steps=a.steps)
    print(f"loss {got[0]:.5f} -> {got[-1]:.5f}")
