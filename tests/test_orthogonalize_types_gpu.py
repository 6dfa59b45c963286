"""Results of the orthogonalisation in bfloat16 against those in float32 and
against float64, over spectra and numbers of steps.

A bfloat16 result is the float32 result rounded once: the bits are compared.
Against float64 its error is then at most the rounding, 2^-9 of each element
and so of the norm, and the float32 result's own: 1e-5 for five default steps,
and with more steps a rounding is amplified by a = 3.4445 a step at most.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
A, B, C = 3.4445, -4.7750, 2.0315


@pytest.fixture(scope="module")
def sdc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import spherical_disco_convolution_amd as m
    return m


def spectrum(kind, rows, cols, seed=0):
    """A matrix whose singular values are `kind`: "gauss" (of a random matrix),
    "flat", "power" (1/i), or a number (one strong direction, the others that far below)."""
    g = torch.Generator()
    g.manual_seed(seed)
    r = min(rows, cols)
    if kind == "gauss":
        return torch.randn(rows, cols, generator=g, dtype=torch.float64)
    u = torch.linalg.qr(torch.randn(rows, r, generator=g, dtype=torch.float64))[0]
    v = torch.linalg.qr(torch.randn(cols, r, generator=g, dtype=torch.float64))[0]
    s = torch.ones(r, dtype=torch.float64)
    if kind == "power":
        s /= torch.arange(1, r + 1)
    elif kind != "flat":
        s[1:] = kind
    return (u * s) @ v.T


def ns64(m, steps):
    x = m / m.square().sum().sqrt()
    if x.shape[0] > x.shape[1]:
        return ns64(m.T, steps).T
    for _ in range(steps):
        g = x @ x.T
        x = A * x + (B * g + C * (g @ g)) @ x
    return x


KINDS = ["gauss", "flat", "power", 0.3, 0.1, 0.001]


@pytest.mark.parametrize("rows,cols", [(20, 50), (60, 300), (128, 500), (300, 500), (700, 200), (333, 1001), (150, 4000)])
@pytest.mark.parametrize("steps", [1, 5, 8])
def test_bfloat16_is_within_its_rounding(sdc, rows, cols, steps):
    for kind in KINDS:
        m = spectrum(kind, rows, cols).float()
        ref = ns64(m.double(), steps)
        o = sdc.orthogonalize(m.cuda(), out_dtype=BF16, eps=0.0, steps=steps).double().cpu()
        bar = 2.0 ** -9 + 1e-5 * max(1.0, A ** (steps - 5))
        assert float((o - ref).norm() / ref.norm()) <= bar, kind


@pytest.mark.parametrize("batch,rows,cols", [(3, 20, 50), (2, 60, 300), (1, 128, 500), (2, 300, 500), (3, 333, 1001),
                                             (1, 256, 4096), (1, 900, 1100), (1, 2048, 2048)])
def test_bfloat16_is_the_rounded_float32_result(sdc, batch, rows, cols):
    for tin in (F32, BF16):
        m = torch.stack([spectrum("gauss", rows, cols, k) for k in range(batch)]).to(tin).cuda()
        for steps in (1, 2, 5, 16):
            o32 = sdc.orthogonalize(m, out_dtype=F32, steps=steps)
            o16 = sdc.orthogonalize(m, out_dtype=BF16, steps=steps)
            assert torch.equal(o16, o32.to(BF16)), (tin, steps)


@pytest.mark.parametrize("shape,groups", [((64, 20, 7), 1), ((128, 128, 7), 1), ((600, 400), 2)])
def test_bfloat16_weights_take_the_rounded_float32_update(sdc, shape, groups):
    w = spectrum("gauss", shape[0], 1).expand(shape[0], 1).reshape(-1, *([1] * (len(shape) - 1)))
    w = (w * torch.linspace(0.5, 1.5, shape[-1], dtype=torch.float64)).expand(shape).to(BF16).cuda().contiguous()
    n = w.numel() // shape[0]
    grad = spectrum("power", shape[0], n).float().view(shape).cuda()
    buf = spectrum(0.1, shape[0], n, 1).float().view(shape).cuda()
    args = dict(lr=0.1, weight_decay=0.01, groups=groups, momentum_out=torch.empty_like(buf))
    w16, _, _ = sdc.muon_step(w, grad, buf, w_out=torch.empty_like(w), **args)
    w32, _, _ = sdc.muon_step(w.float(), grad, buf, w_out=torch.empty_like(grad), **args)
    assert torch.equal(w16, w32.to(BF16))
