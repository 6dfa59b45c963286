"""The training example: its gradients against differences of its loss, and
its loss over some steps."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_follow_differences(example):
    # The loss is read through bfloat16 fields and weights, so the comparison is
    # along each gradient itself, with a step that should change the loss by half
    # a percent: rounding moves the mean over 7e4 values by 2^-9 / sqrt(7e4) of
    # it, 7e-6, or 0.15 percent of the change.  The difference's own error falls
    # with the square of the step (along beta, the most curved: 39 percent at a
    # step ten times as long).  3 percent allowed.
    sdc = example.sdc
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    psi = sdc.psi_build(17, 32, 17, 32, (3, 3), 4 * math.pi / 16).to_device()
    net = example.Stack(psi, 2, 64, gen)
    x = torch.randn((2, 64, 17, 32), generator=gen, device="cuda").to(torch.bfloat16)
    target = torch.randn((2, 64, 17, 32), generator=gen, device="cuda")

    def loss():
        out, saved = net.forward(x)
        return out.float() - target, saved

    diff, saved = loss()
    base = float(diff.square().mean())
    gw, gg, gb = net.backward(saved, (2.0 / diff.numel() * diff).to(torch.bfloat16))
    for tensors, grads in ((net.w, gw), (net.gamma, gg), (net.beta, gb)):
        norm2 = sum(float(g.double().square().sum()) for g in grads)
        h = 0.005 * base / norm2
        got = []
        for sign in (1.0, -1.0):
            for t, g in zip(tensors, grads):
                t += sign * h * g
            net.w16 = [w.to(torch.bfloat16) for w in net.w]
            got.append(float(loss()[0].square().mean()))
            for t, g in zip(tensors, grads):
                t -= sign * h * g
        net.w16 = [w.to(torch.bfloat16) for w in net.w]
        assert abs((got[0] - got[1]) / (2 * h) / norm2 - 1) <= 0.03


def test_the_loss_falls(example):
    losses = example.train(steps=30)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.5 * losses[0]
