"""Statistics and gradients over millions of channels: sums of that many terms
keep float32 accuracy."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import spherical_disco_convolution_amd as m
    return m


@pytest.mark.parametrize("shape,axis", [((1, 2 ** 24 - 1, 2), 1), ((1, 2 ** 22, 5), 1), ((2, 2 ** 24 - 1), -1)])
def test_sums_over_millions_of_channels(sdc, shape, axis):
    # the float32 bar of every other shape, 1e-5 (relative L2)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn(shape, generator=g, device="cuda") + 0.5
    gy = torch.randn(shape, generator=g, device="cuda") + 0.5 * x
    y, _, mean, rstd = sdc.layer_norm_fwd(x, axis=axis)
    gx = sdc.layer_norm_bwd(x, gy, mean, rstd, axis=axis, need_gparams=False)[0]
    m64 = x.double().mean(axis, keepdim=True)
    r64 = ((x.double() - m64).square().mean(axis, keepdim=True) + 1e-5).rsqrt()
    h = (x.double() - m64) * r64
    t = gy.double()
    want = r64 * (t - t.mean(axis, keepdim=True) - h * (t * h).mean(axis, keepdim=True))
    assert float(((mean.double().unsqueeze(axis) - m64) / m64).abs().max()) <= 1e-5
    assert float(((rstd.double().unsqueeze(axis) - r64) / r64).abs().max()) <= 1e-5
    assert float((y.double() - h).norm() / h.norm()) <= 1e-5
    assert float((gx.double() - want).norm() / want.norm()) <= 1e-5
