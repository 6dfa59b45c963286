"""Coefficients whose last step leaves singular values far above one: only what a
further step reads has to stay in the range of the products' operands."""
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


def ns64(m, steps, coeffs):
    x = m.double() / m.double().square().sum(dim=(-2, -1), keepdim=True).sqrt()
    for _ in range(steps):
        g = x @ x.mT.contiguous()
        x = coeffs[0] * x + (coeffs[1] * g + coeffs[2] * (g @ g)) @ x
    return x


# matrices of one workgroup (one and two tile rows), flat ones and tiled ones; the
# result's largest singular value is 16 to 23.5
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 17), (32, 512), (40, 41), (64, 256), (64, 448), (128, 896), (150, 200)])
@pytest.mark.parametrize("steps,coeffs", [(1, (16.0, 0.0, 0.0)), (1, (20.0, 0.0, 0.0)), (1, (23.5, 0.0, 0.0)),
                                          (2, (2.2, 0.3, 0.1)), (2, (2.2, -0.3, 0.3))])
def test_the_last_step_may_leave_the_operands_range(sdc, rows, cols, steps, coeffs):
    # one strong direction, so that entries come near the largest singular value
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + cols)
    u = torch.zeros(rows, 1, device="cuda")
    v = torch.zeros(1, cols, device="cuda")
    u[rows // 2] = v[0, cols // 3] = 1.0
    m = u * v + 1e-3 * torch.randn((3, rows, cols), generator=g, device="cuda")
    ref = ns64(m, steps, coeffs)
    o = sdc.orthogonalize(m, steps=steps, coeffs=coeffs, eps=0.0)
    assert float((o.double() - ref).norm() / ref.norm()) <= 1e-5
    assert torch.equal(sdc.orthogonalize(m, steps=steps, coeffs=coeffs, eps=0.0, out_dtype=BF16), o.to(BF16))
    w, grad, buf = torch.zeros_like(m[0]), m[0].clone(), torch.zeros_like(m[0])
    sdc.muon_step(w, grad, buf, 1.0, steps=steps, coeffs=coeffs, scale=1.0, eps=0.0, beta=0.0)
    assert float((w.double() + ref[0]).norm() / ref[0].norm()) <= 1e-5
