"""The classifier example: layer, softmax cross entropy, overlapped all-reduce, Muon and AdamW together."""
import math
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def train():
    assert torch.cuda.is_available(), "GPU test needs a CUDA device"
    import __graft_entry__
    __graft_entry__.build()
    from train_classifier import train as fn
    return fn


@pytest.mark.parametrize("workers, width, hidden, classes, batch", [(4, 256, 512, 2000, 512), (3, 72, 200, 333, 100)])
def test_it_runs_and_keeps_the_workers_equal(train, workers, width, hidden, classes, batch):
    losses, team, _ = train(workers=workers, width=width, hidden=hidden, classes=classes, batch=batch, steps=4, report=None)
    assert len(losses) == 4 and all(math.isfinite(v) for v in losses)
    for w in team:
        assert torch.equal(w.params, team[0].params) and torch.equal(w.grad, team[0].grad)
        assert torch.equal(w.operands, w.params.bfloat16())
        assert bool(torch.isfinite(w.params).all())


def test_the_averaged_gradient_is_the_whole_batchs(train):
    """One step's averaged gradient against autograd on the concatenated batch, in 64 bits.  The products see bfloat16
    parameters; activations, pre-activations, the head's dz in dh and dh are rounded to bfloat16 on the way (2^-9 of each
    on average); 3 % of the norm leaves room for all of them."""
    losses, team, view = train(workers=3, width=64, hidden=96, classes=130, batch=50, steps=1, lr=0.0, report=None)
    p = {k: view(team[0].operands, k).double().clone().requires_grad_() for k in ("w1", "b1", "w2", "b2")}
    x, y = torch.cat([w.x for w in team]).double(), torch.cat([w.labels for w in team])
    h = torch.nn.functional.gelu(x @ p["w1"].t() + p["b1"])
    loss = torch.nn.functional.cross_entropy(h @ p["w2"].t() + p["b2"], y)
    loss.backward()
    assert abs(losses[0] - float(loss.detach())) <= 0.01 * float(loss.detach())
    for k, v in p.items():
        assert (view(team[0].grad, k).double() - v.grad).norm() <= 0.03 * v.grad.norm(), k
