"""Layer norm over every combination of types, on each of its paths, against the
formulas in float64.

Tolerances as for the other shapes: relative L2 of 1e-5 for float32 results and
2^-8 for bfloat16 ones (their rounding of at most 2^-9 an element, twice);
parameter sums within 2e-6 of the sums of their terms' magnitudes.
"""
import itertools

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
BAR = {F32: 1e-5, BF16: 2.0 ** -8}
# a lane of one point, of several, 32 channels a wave, channel walks; rows of a part of
# a wave, of waves, of a workgroup, row walks
SHAPES = [((2, 24, 9, 13), 1), ((4, 64, 181, 360), 1), ((1, 400, 45, 90), 1), ((1, 700, 20, 31), 1),
          ((70, 40), -1), ((3000, 777), -1), ((300, 9000), -1), ((4, 20001), -1)]


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


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def statistics64(s, axis):
    m = s.double().mean(axis, keepdim=True)
    return m, ((s.double() - m).square().mean(axis, keepdim=True) + 1e-5).rsqrt()


@pytest.mark.parametrize("shape,axis", SHAPES)
def test_forward_types(sdc, shape, axis):
    C = shape[axis]
    per_c = [-1 if d == axis % len(shape) else 1 for d in range(len(shape))]
    gamma, beta = 1 + 0.1 * randn(1, (C,)), 0.1 * randn(2, (C,))
    for tx, ty, with_res in itertools.product((F32, BF16), (F32, BF16), (False, True)):
        x = (1.5 * randn(3, shape) + 0.7).to(tx)
        res = randn(4, shape, tx) if with_res else None
        y, s, mean, rstd = sdc.layer_norm_fwd(x, gamma, beta, residual=res, axis=axis, out_dtype=ty)
        if with_res:
            assert torch.equal(s, (x.float() + res.float()).to(tx))
        m64, r64 = statistics64(s if with_res else x, axis)
        want = ((s if with_res else x).double() - m64) * r64 * gamma.double().view(per_c) + beta.double().view(per_c)
        assert y.dtype == ty and rel(y, want) <= BAR[ty], (tx, ty, with_res)
        assert rel(rstd.unsqueeze(axis), r64) <= 1e-5 and rel(mean.unsqueeze(axis), m64) <= 1e-5


@pytest.mark.parametrize("shape,axis", SHAPES)
def test_backward_types(sdc, shape, axis):
    C = shape[axis]
    per_c = [-1 if d == axis % len(shape) else 1 for d in range(len(shape))]
    dims = [d for d in range(len(shape)) if d != axis % len(shape)]
    gamma = 1 + 0.1 * randn(1, (C,))
    for tx, tg, to, with_sum in itertools.product((F32, BF16), (F32, BF16), (F32, BF16, None), (False, True)):
        x, gy = (1.5 * randn(3, shape) + 0.7).to(tx), randn(4, shape, tg)
        gsum = randn(5, shape, tg) if with_sum else None
        m64, r64 = statistics64(x, axis)
        mean, rstd = m64.float().squeeze(axis), r64.float().squeeze(axis)
        gx, gg, gb = sdc.layer_norm_bwd(x, gy, mean, rstd, gamma, gsum=gsum, axis=axis, gx_dtype=to)
        r = rstd.double().unsqueeze(axis)
        h = (x.double() - mean.double().unsqueeze(axis)) * r
        g = gy.double()
        t = g * gamma.double().view(per_c)
        want = r * (t - t.mean(axis, keepdim=True) - h * (t * h).mean(axis, keepdim=True))
        if with_sum:
            want = want + gsum.double()
        assert gx.dtype == (F32 if to is None else to) and rel(gx, want) <= BAR[gx.dtype], (tx, tg, to, with_sum)
        assert float(((gg.double() - (g * h).sum(dims)).abs() - 2e-6 * (g * h).abs().sum(dims)).max()) <= 1e-30
        assert float(((gb.double() - g.sum(dims)).abs() - 2e-6 * g.abs().sum(dims)).max()) <= 1e-30
