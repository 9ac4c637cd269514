"""The 8-bit operators run together (examples/train_block8.py): the gradients
of a network against torch's on the same formulas, and training with Muon."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_block8.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("train_block8", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_follow_the_formulas(ex):
    hidden, ffn, tokens = 192, 320, 130
    net = ex.Net(hidden, ffn, 2, seed=3)
    x = torch.randn(tokens, hidden, device="cuda", dtype=torch.bfloat16)
    target = torch.randn(tokens, hidden, device="cuda")
    loss = net.loss_and_gradients(x, target)
    # the same network in 64 bits, without the 8-bit rounding
    ws = [w.detach().double().requires_grad_() for w in net.matrices]
    gs = [b.norm.double().requires_grad_() for b in net.blocks]
    out, h = torch.zeros(tokens, hidden, device="cuda", dtype=torch.float64), x.double()
    for i in range(2):
        h = h + out
        y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + 1e-6) * gs[i]
        out = torch.relu(y @ ws[2 * i].t().contiguous()).square() @ ws[2 * i + 1].t().contiguous()
    ref = (h + out - target.double()).square().mean()
    ref.backward()
    # 8-bit rows of Gaussian values: a step of 2^e with 127 * 2^e >= max, so at
    # most max / 63.5, max about 3.3 sigma over 192 values: rounding noise of at
    # most 3.3 / 63.5 / sqrt(12) = 1.5 % per operand; squared activations have
    # about twice the range (3 %).  A gradient passes at most eight such
    # operands; their noises are independent: 3 % * sqrt(8) = 8.5 %.
    assert abs(float(loss) - float(ref.detach())) <= 0.085 * float(ref.detach())
    got = [g for b in net.blocks for g in (b.dw1, b.dw2)] + [b.dnorm for b in net.blocks]
    for g, r in zip(got, [w.grad for w in ws] + [g.grad for g in gs]):
        rel = float((g.double() - r).norm() / r.norm())
        assert rel <= 0.085, rel


@pytest.mark.parametrize("refresh_period", [0, 4])
def test_training_lowers_the_loss(ex, refresh_period):
    losses = ex.train(steps=24, tokens=512, hidden=256, ffn=512, blocks=2, refresh_period=refresh_period)
    assert all(v == v for v in losses)
    assert losses[-1] < 0.7 * losses[0], losses
    again = ex.train(steps=24, tokens=512, hidden=256, ffn=512, blocks=2, refresh_period=refresh_period)
    assert losses == again  # nothing depends on timing
