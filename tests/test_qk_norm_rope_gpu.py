"""Norm and rotation of queries and keys, and their gradients, against float64."""
import pytest

torch = pytest.importorskip("torch")
from attention_reference import BF16, F32, half_step, rotate, turns  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def sdc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import spherical_disco_convolution_amd as m
    return m


def randn(seed, shape, dtype=F32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def bounded(name, got, want, bound):
    far = (got.double().cpu() - want).abs() - bound
    assert bool(got.isfinite().all()), name
    assert float(far.max()) <= 0, f"{name}: {float(far.max()):.3g} over the bound"


def reference(x, w, angle, interleaved, eps, gy=None):
    """Values and bounds: with A the magnitudes that a pair's sum is made of, the
    float32 steps (norm of d terms, weight, cosine and sine to 2^-22, two products)
    cost (d + 16) u A + 2^-21 A."""
    x, d = x.double().cpu(), x.shape[-1]
    w = torch.ones(d, dtype=torch.float64) if w is None else w.double().cpu()
    r = 1.0 / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    small = (d + 16) * U + 2.0 ** -21

    def both(t):   # magnitudes of a pair, for either of its elements
        return rotate(t.abs(), torch.zeros_like(angle), interleaved) + swap(t.abs())

    def swap(t):
        y, n = torch.zeros_like(t), angle.shape[1]
        for p in range(n):
            a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + n)
            y[..., a], y[..., b] = t[..., b], t[..., a]
        return y

    n = x * r * w
    y = rotate(n, angle, interleaved)
    if gy is None:
        return y, small * both(n)
    gy = gy.double().cpu()
    gn = rotate(gy, -angle, interleaved)
    t = gn * w
    dot = (t * x).mean(-1, keepdim=True)
    gx = r * (t - x * r * r * dot)
    m = both(gy) * w.abs()
    e = small * r * (m + x.abs() * r * r * (m * x.abs()).mean(-1, keepdim=True)) * 3
    gw = (gn * x * r).sum((0, 1))
    rows = x.shape[0] * x.shape[1]
    ew = (small * 2 + (min(rows, 4096) + 64) * U) * (both(gy) * x.abs() * r).sum((0, 1))
    return gx, e, gw, ew


def case(sdc, tokens, hq, hkv, d, rot, axes, interleaved, dtype, weights=True, eps=1e-6, far=False, views=False):
    if views:
        buf = randn(1, (tokens, (hq + hkv) * d + 3), dtype)
        q, k = buf[:, 3:3 + hq * d].unflatten(1, (hq, d)), buf[:, 3 + hq * d:].unflatten(1, (hkv, d))
    else:
        q, k = randn(1, (tokens, hq, d), dtype), randn(2, (tokens, hkv, d), dtype)
    qw, kw = (1.0 + 0.3 * randn(3, (d,)), 1.0 + 0.3 * randn(4, (d,))) if weights else (None, None)
    opt = {}
    angle = torch.zeros((tokens, 0), dtype=torch.float64)
    if rot:
        inv = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float()
        if axes == 1:
            pos = torch.arange(tokens, dtype=torch.int32, device="cuda") * 7 + (2 ** 31 - 1 - 7 * tokens if far else 0)
        else:
            pos = 6.3 * torch.rand((tokens, axes), device="cuda")
        angle = turns(pos, inv, axes)
        opt = dict(positions=pos, inv_freq=inv, interleaved=interleaved)
    qo, ko = sdc.qk_norm_rope_fwd(q, k, qw, kw, eps=eps, **opt)
    gqo, gko = randn(5, (tokens, hq, d), dtype), randn(6, (tokens, hkv, d), dtype)
    gq, gk, gqw, gkw = sdc.qk_norm_rope_bwd(q, k, gqo, gko, qw, kw, eps=eps, **opt)
    torch.cuda.synchronize()
    # a float64 angle is off by 2^-53 of it, and the turn that is left by 2^-24 of half a turn
    half = half_step(dtype)
    for n, x, w, y, gy, gx, gw in (("q", q, qw, qo, gqo, gq, gqw), ("k", k, kw, ko, gko, gk, gkw)):
        want, e = reference(x, w, angle, interleaved, eps)
        bounded(n, y, want, e + half * want.abs())
        want, e, ww, ew = reference(x, w, angle, interleaved, eps, gy)
        bounded("g" + n, gx, want, e + half * want.abs())
        bounded("gw" + n, gw, ww, ew)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(1, 0), (2, 2), (3, 2), (8, 8), (16, 8), (24, 24), (32, 12), (33, 32), (40, 40), (63, 10),
                                   (64, 64), (64, 32), (100, 96), (128, 128), (128, 64), (128, 0), (200, 200), (255, 254),
                                   (256, 256), (256, 6)])
def test_head_sizes(sdc, d, rot, interleaved, dtype):
    case(sdc, 37, 3, 2, d, rot, 1, interleaved, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 2, 63, 65, 1000, 5003])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (12, 4), (7, 7)])
def test_tokens_and_heads(sdc, tokens, hq, hkv, dtype):
    case(sdc, tokens, hq, hkv, 64, 64, 1, False, dtype)


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_axes(sdc, axes, interleaved):
    case(sdc, 50, 4, 2, 64, 40, axes, interleaved, F32)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_far_positions(sdc, dtype):
    case(sdc, 50, 4, 2, 64, 64, 1, False, dtype, far=True)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_views_and_no_weights(sdc, dtype):
    case(sdc, 45, 4, 2, 64, 64, 1, False, dtype, views=True)
    case(sdc, 45, 4, 2, 64, 64, 1, True, dtype, weights=False, eps=0.0)


def test_rows_of_zeros_and_nan(sdc):
    q, k = randn(1, (9, 2, 32)), randn(2, (9, 1, 32))
    q[3, 1] = 0.0
    clean = sdc.qk_norm_rope_fwd(q, k)[0].clone()
    assert not bool(clean[3, 1].any())
    q[5, 0, 7] = float("nan")
    got = sdc.qk_norm_rope_fwd(q, k)[0]
    assert bool(got[5, 0].isnan().all())
    got[5, 0] = clean[5, 0]
    assert torch.equal(got, clean)


def test_no_tokens(sdc):
    q, k = torch.zeros((0, 4, 32), device="cuda"), torch.zeros((0, 2, 32), device="cuda")
    sdc.qk_norm_rope_fwd(q, k)
    gq, gk, gqw, gkw = sdc.qk_norm_rope_bwd(q, k, q, k)
    torch.cuda.synchronize()
    assert gq.numel() == 0 and not bool(gqw.any()) and not bool(gkw.any()) and gqw.shape == (32,)


def test_gradients_follow_differences(sdc):
    q, k, w = randn(1, (20, 2, 16)), randn(2, (20, 1, 16)), 1.0 + 0.1 * randn(3, (16,))
    pos, inv = torch.arange(20, dtype=torch.int32, device="cuda"), torch.rand(8, device="cuda")
    gq, gk = randn(4, q.shape), randn(5, k.shape)
    opt = dict(positions=pos, inv_freq=inv)

    def loss(q, k, w):
        a, b = sdc.qk_norm_rope_fwd(q, k, w, w, **opt)
        return float((a.double() * gq.double()).sum() + (b.double() * gk.double()).sum())

    dq, dk, dqw, dkw = sdc.qk_norm_rope_bwd(q, k, gq, gk, w, w, **opt)
    h = 1e-2    # off by h^2 / 6 of the third derivative and by 1e-6 / h of rounding
    for i, g in enumerate((dq, dk, dqw + dkw)):
        args = [q, k, w]
        d = randn(10 + i, g.shape)
        d /= d.norm()
        args[i] = (q, k, w)[i] + h * d
        up = loss(*args)
        args[i] = (q, k, w)[i] - h * d
        want = float((g.double() * d.double()).sum())
        assert abs((up - loss(*args)) / (2 * h) - want) <= 2e-3 * max(1.0, abs(want))


def test_the_same_bits_again_and_in_a_graph(sdc):
    q, k = randn(1, (3000, 8, 64), BF16), randn(2, (3000, 2, 64), BF16)
    w = randn(3, (64,))
    pos, inv = torch.arange(3000, dtype=torch.int32, device="cuda"), torch.rand(32, device="cuda")
    opt = dict(positions=pos, inv_freq=inv)

    def step():
        a = sdc.qk_norm_rope_fwd(q, k, w, w, **opt)
        return a + sdc.qk_norm_rope_bwd(q, k, q, k, w, w, **opt)

    want = step()
    assert all(torch.equal(a, b) for a, b in zip(step(), want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        _ = float(step()[2].float().abs().sum())
