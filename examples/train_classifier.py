"""Synchronous data-parallel training of a classifier with a large number of
classes, all of it in the library's kernels: P logical workers on one GPU, each
with its own batch.

Per iteration, for every worker: a linear layer with fused bias and GELU, the
softmax cross entropy of a linear head (the logits are never kept), both backward
passes straight into the worker's flat binary32 gradient buffer, and, as soon as
the head's gradients are there, the overlapped all-reduce of its bucket; then the
Muon step on the hidden layer's matrix, and AdamW with 8-bit states, clipped, on the
head and the biases, which also writes the head's bfloat16 weights for the next step.

    python examples/train_classifier.py --workers 4 --steps 30

The task is synthetic: the labels come from a fixed random network.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gradient_all_reduce_ddl_gb300 import ddl  # noqa: E402


class Worker:
    """A worker's parameters (binary32, and bfloat16 for the products), gradients and batch."""

    def __init__(self, start, width, hidden, batch, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.params, self.operands, self.grad = start.clone(), start.bfloat16(), torch.zeros_like(start)
        self.x = torch.randn(batch, width, generator=gen, device="cuda").bfloat16()
        self.h = torch.empty(batch, hidden, dtype=torch.bfloat16, device="cuda")
        self.z, self.dh = torch.empty_like(self.h), torch.empty_like(self.h)
        self.loss, self.lse = torch.empty(batch, device="cuda"), torch.empty(batch, device="cuda")
        self.labels = None


def train(workers=4, width=256, hidden=512, classes=2000, batch=512, steps=30, lr=0.02, seed=1, report=print):
    """Trains and returns the losses, the workers and the layout."""
    shapes = {"w1": (hidden, width), "b1": (hidden,), "w2": (classes, hidden), "b2": (classes,)}
    layout, n = {}, 0
    for name, shape in shapes.items():  # forward order at increasing addresses, as the plan's layer list
        layout[name] = (n, shape)
        n += shape[0] * (shape[1] if len(shape) > 1 else 1)
    sizes = {k: s[0] * (s[1] if len(s) > 1 else 1) for k, s in shapes.items()}

    def view(flat, name):
        return flat[layout[name][0]:layout[name][0] + sizes[name]].view(shapes[name])

    gen = torch.Generator(device="cuda").manual_seed(seed)
    teacher, start = torch.randn(n, generator=gen, device="cuda"), torch.randn(n, generator=gen, device="cuda")
    for flat, scale in ((teacher, 3.0), (start, 1.0)):
        for name, shape in shapes.items():
            view(flat, name).mul_(scale * shape[1] ** -0.5 if len(shape) > 1 else 0.0)
    team = [Worker(start, width, hidden, batch, seed + 10 + r) for r in range(workers)]

    up = ddl.Linear(width, hidden, batch, "bf16", "gelu")
    head = ddl.CrossEntropy(hidden, classes, batch, "bf16")
    muon, mom = ddl.Ortho([(layout["w1"][0], hidden, width)], "f32"), torch.zeros(n, device="cuda")
    # the head decays, the biases do not
    adam = ddl.Adam([(layout[k][0], sizes[k], 1.0, float(k == "w2")) for k in ("b1", "w2", "b2")], "f32", "8bit")
    state, norm = adam.new_state(), torch.zeros(1, device="cuda")
    dloss = torch.full((batch,), 1.0 / batch, device="cuda")
    # a bucket per layer, the head's first: its all-reduce runs under the hidden layer's backward pass
    plan = ddl.Plan(workers, n, "f32", "ring", layers=list(sizes.values()), bucket_bytes=4 * (sizes["w2"] + sizes["b2"]))

    for w in team:
        t = teacher.bfloat16()
        up.forward(w.x, view(t, "w1"), w.h, bias=view(t, "b1"))
        w.labels = (w.h.float() @ view(t, "w2").float().t()).argmax(1)
    losses = []
    for step in range(steps):
        plan.overlap_begin([w.grad for w in team], 1.0 / workers)
        total = 0.0
        for w in team:
            o = w.operands
            up.forward(w.x, view(o, "w1"), w.h, bias=view(o, "b1"), z=w.z)
            head.forward(w.h, view(o, "w2"), w.labels, w.loss, w.lse, bias=view(o, "b2"))
            head.backward(w.h, view(o, "w2"), w.labels, w.lse, dloss=dloss, bias=view(o, "b2"), dx=w.dh,
                          dw=view(w.grad, "w2"), db=view(w.grad, "b2"))
            total = total + w.loss.mean()
        plan.bucket_ready(0)
        for w in team:
            up.backward(w.dh, w.x, z=w.z, dw=view(w.grad, "w1"), db=view(w.grad, "b1"))
        plan.overlap_end()
        params = [w.params for w in team]
        muon.muon(team[0].grad, params, mom, lr)
        adam.step(team[0].grad, params, lr=lr / 10, weight_decay=0.01, operands=[w.operands for w in team], max_norm=1.0,
                  norm=norm, **state)
        for w in team:  # the matrix that Muon has stepped
            view(w.operands, "w1").copy_(view(w.params, "w1"))
        losses.append(float(total) / workers)
        if report and step % 5 == 0:
            report(f"step {step:3d}  loss {losses[-1]:.5f}  gradient norm {float(norm):.4f}")
    for handle in (up, head, muon, plan):
        handle.check()
    for handle in (up, head, muon, adam, plan):
        handle.close()
    return losses, team, view


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--workers", type=int, default=4)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    got = train(workers=a.workers, steps=a.steps)[0]
    print(f"loss {got[0]:.5f} -> {got[-1]:.5f}")
