"""Tensors of more than 2^31 elements: zeros but for their first and last points,
rows or matrices, whose results are compared and which no other place may take
part in.  Offsets cut to 32 bits, signed or not, would land among the zeros.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def sdc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import spherical_disco_convolution_amd as m
    yield m
    torch.cuda.empty_cache()


def randn(seed, shape, dtype=F32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


# registers and walks, of fields and of rows; k points or rows at either end
@pytest.mark.parametrize("shape,axis,k", [((2, 128, 9_000_001), 1, 700), ((2, 600, 1_800_001), 1, 300),
                                          ((530_001, 4096), -1, 60), ((131_101, 16400), -1, 20)])
def test_layer_norm(sdc, shape, axis, k):
    C = shape[axis]
    if axis == 1:
        ends = [(slice(0, 1), slice(None), slice(0, k)), (slice(1, 2), slice(None), slice(-k, None))]
        part, sums, per_c = (1, C, k), (0, 2), (1, C, 1)
    else:
        ends = [(slice(0, k),), (slice(-k, None),)]
        part, sums, per_c = (k, C), (0,), (1, C)
    gamma = 1 + 0.1 * randn(9, (C,))
    x, gy = (torch.zeros(shape, device="cuda", dtype=BF16) for _ in range(2))
    for n, e in enumerate(ends):
        x[e], gy[e] = randn(1 + n, part, BF16) + 0.5, randn(3 + n, part, BF16)
    y, _, mean, rstd = sdc.layer_norm_fwd(x, gamma, axis=axis)
    gx, gg, gb = sdc.layer_norm_bwd(x, gy, mean, rstd, gamma, axis=axis, gx_dtype=BF16)
    rg = rb = mg = mb = 0.0
    for e in ends:
        f, g = x[e].double(), gy[e].double()
        m64 = f.mean(axis, keepdim=True)
        r64 = ((f - m64).square().mean(axis, keepdim=True) + 1e-5).rsqrt()
        h = (f - m64) * r64
        t = g * gamma.double().view(per_c)
        want = r64 * (t - t.mean(axis, keepdim=True) - h * (t * h).mean(axis, keepdim=True))
        wy = h * gamma.double().view(per_c)
        assert float((y[e].double() - wy).norm() / wy.norm()) <= 2.0 ** -8
        assert float((gx[e].double() - want).norm() / want.norm()) <= 2.0 ** -8
        rg, rb = rg + (g * h).sum(sums), rb + g.sum(sums)
        mg, mb = mg + (g * h).abs().sum(sums), mb + g.abs().sum(sums)
        y[e], gx[e] = 0, 0
    # the statistics of these points come from float32: 1e-5 of the terms' magnitudes
    assert float(((gg.double() - rg).abs() - 1e-5 * mg).max()) <= 1e-30
    assert float(((gb.double() - rb).abs() - 2e-6 * mb).max()) <= 1e-30
    assert not y.any() and not gx.any()


# one workgroup a matrix (2^32 bytes; 65535 matrices are the most), flat, tiled
@pytest.mark.parametrize("batch,rows,cols,dtype", [(65535, 32, 512, F32), (4100, 64, 8192, BF16),
                                                   (2050, 256, 4096, BF16)])
def test_orthogonalize(sdc, batch, rows, cols, dtype):
    m = torch.zeros((batch, rows, cols), device="cuda", dtype=dtype)
    m[0], m[-1] = randn(1, (rows, cols), dtype), randn(2, (rows, cols), dtype)
    o = sdc.orthogonalize(m)
    for k in (0, -1):
        assert torch.equal(o[k], sdc.orthogonalize(m[k].clone())) and bool(o[k].any())
        o[k] = 0
    assert not o.any()


def test_muon_step(sdc):
    groups, rows, cols = 4100, 64, 8192
    w, grad = (torch.zeros((groups * rows, cols), device="cuda", dtype=BF16) for _ in range(2))
    buf = torch.zeros((groups * rows, cols), device="cuda")
    ends = slice(0, rows), slice(-rows, None)
    want = []
    for n, e in enumerate(ends):
        w[e], grad[e] = randn(1 + n, (rows, cols), BF16), randn(3 + n, (rows, cols), BF16)
        buf[e] = randn(5 + n, (rows, cols))
        want.append(sdc.muon_step(w[e].clone(), grad[e].clone(), buf[e].clone(), 0.1)[:2])
    sdc.muon_step(w, grad, buf, 0.1, groups=groups)
    for e, (ww, wb) in zip(ends, want):
        assert torch.equal(w[e], ww) and torch.equal(buf[e], wb)
        w[e], buf[e] = 0, 0
    assert not w.any() and not buf.any()
