"""The training example: layers, overlapped all-reduce and Muon step together."""
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
    from train_mlp import train as fn
    return fn


@pytest.mark.parametrize("workers, width, hidden, batch", [(4, 256, 768, 512), (3, 72, 200, 100)])
def test_training_lowers_the_loss_and_keeps_the_workers_equal(train, workers, width, hidden, batch):
    losses, team = train(workers=workers, width=width, hidden=hidden, batch=batch, steps=25, report=None)
    assert losses[-1] < 0.5 * losses[0]
    for w in team[1:]:
        assert torch.equal(w.params, team[0].params) and torch.equal(w.grad, team[0].grad)


def test_the_averaged_gradient_is_the_whole_batchs(train):
    """One step's averaged gradient against autograd on the concatenated batch, in 64 bits.  The products see
    bfloat16 parameters, activations and dz (2^-9 of each on average); 3 % of the norm leaves room for three
    such roundings through two layers."""
    losses, team = train(workers=3, width=64, hidden=96, batch=50, steps=1, lr=0.0, report=None)
    w0 = team[0]
    p = {k: w0.operand(k).double().requires_grad_() for k in ("w1", "b1", "w2", "b2")}
    x = torch.cat([w.x for w in team]).double()
    target = torch.cat([w.target for w in team]).double()
    y = torch.nn.functional.gelu(x @ p["w1"].t() + p["b1"]) @ p["w2"].t() + p["b2"] + x
    loss = (y - target).square().mean()
    loss.backward()
    for k, v in p.items():
        got = w0.view(w0.grad, k).double() / 4096
        assert (got - v.grad).norm() <= 0.03 * v.grad.norm(), k
