"""Layer norm over more channels than one launch has workgroups for."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


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


# 2^24 channels make 2^32 threads in workgroups of 256 for each, 2^25 in the reduction
@pytest.mark.parametrize("shape,axis", [((1, 2 ** 24 + 3, 2), 1), ((2, 2 ** 24 - 1, 3), 1), ((2, 2 ** 25 + 5), -1),
                                        ((1, 2 ** 26 + 1), -1)])
def test_gradients_of_many_channels(sdc, shape, axis):
    # The sums run over two to six points; 2e-6 of the terms' magnitudes is allowed as
    # for other shapes, and the error of rstd: half that of a variance summed in 16
    # float32 chains of C / 16 terms, 2^-24 a term in a random walk
    C = shape[axis]
    bar = 2e-6 + 2.0 ** -25 * (C / 16) ** 0.5
    x, gy, gamma = randn(1, shape, BF16), randn(2, shape, BF16), 1 + 0.1 * randn(3, (C,))
    y, _, mean, rstd = sdc.layer_norm_fwd(x, gamma, axis=axis)
    gx, gg, gb = sdc.layer_norm_bwd(x, gy, mean, rstd, gamma, axis=axis, gx_dtype=BF16)
    dims = [d for d in range(x.dim()) if d != axis % x.dim()]
    per_c = [-1 if d == axis % x.dim() else 1 for d in range(x.dim())]
    xd = x.double()
    m64 = xd.mean(axis, keepdim=True)
    r64 = ((xd - m64).square().mean(axis, keepdim=True) + 1e-5).rsqrt()
    h = (xd - m64) * r64
    del xd
    g = gamma.double().view(per_c)
    assert float((y.double() - h * g).norm() / (h * g).norm()) <= 2.0 ** -8
    gyd = gy.double()
    assert float(((gg.double() - (gyd * h).sum(dims)).abs() - bar * (gyd * h).abs().sum(dims)).max()) <= 1e-6
    assert float(((gb.double() - gyd.sum(dims)).abs() - 2e-6 * gyd.abs().sum(dims)).max()) <= 1e-30
    t = gyd * g
    want = r64 * (t - t.mean(axis, keepdim=True) - h * (t * h).mean(axis, keepdim=True))
    assert float((gx.double() - want).norm() / want.norm()) <= 2.0 ** -8
