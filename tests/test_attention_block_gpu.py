"""The block of the example: layer norm, projection, norm and rotation of queries and
keys, attention with quadrature weights, projection, dropout joined to the stream,
forward and backward, against float64 automatic differentiation and differences."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")
from attention_reference import BF16, F32, halves, rotate, turns  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def block(example, dtype, seed=1, batch=2):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    points = example.Points(9, 16, 16)
    b = example.Block(points, batch, 96, 4, 2, 32, 0.25, dtype, gen)
    for n in ("gamma", "q", "k"):
        b.w[n] += 0.2 * torch.randn(b.w[n].shape, generator=gen, device="cuda")
    x = torch.randn((batch * points.count, 96), generator=gen, device="cuda").to(dtype)
    gout = torch.randn(x.shape, generator=gen, device="cuda").to(dtype)
    return b, x, gout


def reference(b, x, gout, seed, offset):
    """The same in float64 on the CPU, gradients by automatic differentiation."""
    w = {n: t.double().cpu().requires_grad_() for n, t in b.w.items()}
    x = x.double().cpu().requires_grad_()
    n, hq, hkv, d, per = x.shape[0], b.hq, b.hkv, b.d, b.points.count
    mu = x.mean(1, keepdim=True)
    y = (x - mu) / torch.sqrt((x - mu).square().mean(1, keepdim=True) + 1e-5) * w["gamma"] + w["beta"]
    qkv = y @ w["qkv"]
    q, k, v = qkv.split((hq * d, hkv * d, hkv * d), dim=1)
    angle = turns(b.rope["positions"], b.rope["inv_freq"], 2)

    def turned(t, heads, weight):
        t = t.reshape(n, heads, d)
        return rotate(t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-6) * weight, angle, False)

    q, k, v = turned(q, hq, w["q"]), turned(k, hkv, w["k"]), v.reshape(n, hkv, d)
    rows = []
    for s in range(b.batch):
        part = slice(s * per, (s + 1) * per)
        heads = [torch.softmax(q[part, h] @ k[part, h // (hq // hkv)].T / math.sqrt(d) + b.bias[part].double().cpu(), 1)
                 @ v[part, h // (hq // hkv)] for h in range(hq)]
        rows.append(torch.cat(heads, dim=1))
    branch = torch.cat(rows) @ w["out"]
    t = math.floor(b.p * 65536 + 0.5)
    keep = torch.from_numpy(halves(branch.numel(), seed, offset) >= t).view(branch.shape)
    out = x + torch.where(keep, branch * (65536.0 / (65536 - t)), 0.0)
    (out * gout.double().cpu()).sum().backward()
    return out.detach(), x.grad, {m: t.grad for m, t in w.items()}


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_forward_and_backward(example, dtype):
    b, x, gout = block(example, dtype)
    out, saved = b.forward(x, 11, 7)
    gx, g = b.backward(saved, gout)
    want, wgx, wg = reference(b, x, gout, 11, 7)
    # relative to the whole tensor.  float32: a chain of about ten operators with sums of
    # up to 288 terms, each off by up to 300 * 2^-24 = 2e-5 where errors add up, a tenth
    # where they are random.  bfloat16: twelve roundings of half a step (2^-8) on the way
    # there and back, of which about a third is the mean over a binade, random: sqrt(12)
    # 2^-8 / sqrt(3) = 0.8 percent; twice that is allowed.
    tol = 2e-5 if dtype == F32 else 0.016
    pairs = [("out", out, want), ("x", gx, wgx)] + [(n, g[n], wg[n]) for n in wg]
    for n, a, e in pairs:
        err = float((a.double().cpu() - e).norm() / e.norm())
        assert err <= tol, (n, err)


def test_in_a_graph(example):
    b, x, gout = block(example, BF16)

    def step():
        out, saved = b.forward(x, 3, 1)
        gx, g = b.backward(saved, gout)
        return [out, gx] + [g[n] for n in sorted(g)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        want = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want))
        _ = float(step()[0].float().abs().sum())


def test_gradients_follow_differences(example):
    # Along each gradient, float32, with a step of at most half a percent of the loss and
    # of 2 percent of the weights' norm.  A central difference is off by the square of the
    # relative step times a number of order one: 4e-4 (a step for half a percent of the
    # loss alone would move the weights of the queries' norm, whose gradient is small, by
    # 0.24 of their norm: 0.24^2 / 6 = 1 percent times that number).  The loss, a mean over
    # 27648 values, is off by about 2^-22 / sqrt(27648) = 1.4e-9 of it, and the smallest
    # change is 4e-4 of it.  One percent allowed.
    b, x, gout = block(example, F32)
    target = torch.randn(x.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))

    def loss():
        out, saved = b.forward(x, 2, 9)
        return out.double() - target.double(), saved

    diff, saved = loss()
    base = float(diff.square().mean())
    _, g = b.backward(saved, (2.0 / diff.numel() * diff).float())
    for n, grad in g.items():
        norm2 = float(grad.double().square().sum())
        h = min(0.005 * base / norm2, 0.02 * float(b.w[n].norm()) / norm2 ** 0.5 if float(b.w[n].norm()) else 1e30)
        keep = b.w[n].clone()
        got = []
        for sign in (1.0, -1.0):
            b.w[n].copy_(keep + sign * h * grad)
            got.append(float(loss()[0].square().mean()))
        b.w[n].copy_(keep)
        assert abs((got[0] - got[1]) / (2 * h) / norm2 - 1) <= 0.01, n


def test_the_example_runs(example):
    losses = example.train(steps=3)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)
