"""Newton-Schulz orthogonalisation and the optimiser step on the GPU against
the formulas in float64 on the same inputs.

Tolerances.  A float32 result is held to the float32 bar, 1e-5 (relative L2):
an input or product rounding of 2^-24 is amplified by at most a^5 = 485 in the
directions of the smallest singular values, 2.9e-5 there in the worst case and
far less in the norm of the whole; with other coefficients or step counts the
bar is scaled by (a^steps / 485).  A bfloat16 result adds its own rounding
(2^-9 an element at most, 1.7e-3 in norm) to single float16 products (2^-12 an
operand) in the early steps, whose errors later steps damp to the level of one
or two such roundings times the gain of the last steps (|f'| <= 3.5): 4e-3 in
all, as 2^-8.  Below 64 rows there is less averaging: 2^-7.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEFAULT = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def sdc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import spherical_disco_convolution_amd as m
    return m


def bar(dtype, rows, cols):
    return 1e-5 if dtype == F32 else 2.0 ** (-8 if min(rows, cols) >= 64 else -7)


def randn(seed, shape, dtype=F32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def update(seed, batch, rows, cols, dtype=F32):
    """Strong directions over a noise floor, as gradients have."""
    r = max(1, min(rows, cols) // 4)
    s = torch.arange(1, r + 1, device="cuda", dtype=F32) ** -0.5
    g = torch.matmul(randn(seed, (batch, rows, r)) * s, randn(seed + 1, (batch, r, cols)))
    return ((g + 0.5 * randn(seed + 2, (batch, rows, cols))) * 1e-3).to(dtype)


def ns64(m, steps=5, coeffs=DEFAULT, eps=1e-7):
    a, b, c = coeffs
    x = m.double()
    x = x / (x.square().sum(dim=(-2, -1), keepdim=True).sqrt() + eps)
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT.contiguous()
    for _ in range(steps):
        g = x @ x.mT.contiguous()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.mT.contiguous() if tall else x


def rel(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm().clamp_min(1e-300))


SHAPES = [(1, 1, 1), (1, 1, 17), (256, 1, 17), (3, 17, 1), (2, 4, 12), (5, 2, 5000), (1, 32, 224), (2, 31, 33),
          (1, 64, 64), (1, 64, 448), (2, 63, 449), (1, 65, 64), (1, 128, 896), (1, 896, 128), (3, 127, 257),
          (1, 129, 130), (3, 1001, 333), (1, 256, 256), (2, 200, 3000), (1, 512, 777), (1, 1024, 1024),
          (1, 1300, 1100), (1, 640, 4096), (70, 40, 41), (300, 5, 9), (1, 100, 9000), (1, 2048, 2050)]


@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_against_float64(sdc, batch, rows, cols):
    for tin, tout in ((F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)):
        m = update(7, batch, rows, cols, tin)
        o = sdc.orthogonalize(m, out_dtype=tout)
        assert o.dtype == tout and o.shape == m.shape
        assert rel(o, ns64(m)) <= bar(tout, rows, cols), (tin, tout)
        assert torch.equal(o, sdc.orthogonalize(m, out_dtype=tout))   # reproducible
        if batch > 1:
            # each matrix by itself gives the same bits (two dimensions: one matrix)
            k = batch - 1
            assert torch.equal(o[k], sdc.orthogonalize(m[k].clone(), out_dtype=tout))


@pytest.mark.parametrize("rows,cols", [(40, 200), (150, 150), (300, 100)])
@pytest.mark.parametrize("steps,coeffs", [(1, DEFAULT), (2, DEFAULT), (3, DEFAULT), (8, DEFAULT),
                                          (6, (2.0, -1.5, 0.5)), (5, (1.875, -1.25, 0.375))])
def test_steps_and_coefficients(sdc, rows, cols, steps, coeffs):
    m = update(3, 2, rows, cols)
    o = sdc.orthogonalize(m, steps=steps, coeffs=coeffs)
    assert rel(o, ns64(m, steps, coeffs)) <= 1e-5 * max(1.0, coeffs[0] ** steps / 485)
    o16 = sdc.orthogonalize(m, out_dtype=BF16, steps=steps, coeffs=coeffs)
    assert rel(o16, ns64(m, steps, coeffs)) <= 2.0 ** -7


@pytest.mark.parametrize("rows,cols", [(48, 100), (128, 300), (400, 150)])
def test_the_result_is_near_orthogonal(sdc, rows, cols):
    # the map sends singular values in [0.01, 1] into [0.68, 1.13] after five steps
    q = torch.linalg.qr(randn(1, (max(rows, cols), min(rows, cols))).double().cpu())[0]
    s = torch.linspace(0.05, 1.0, min(rows, cols), dtype=torch.float64)
    v = torch.linalg.qr(randn(2, (min(rows, cols),) * 2).double().cpu())[0]
    m = (q * s) @ v.mT
    m = (m if rows > cols else m.mT).float().cuda().contiguous()
    sv = torch.linalg.svdvals(sdc.orthogonalize(m).double().cpu())
    assert 0.6 < float(sv.min()) and float(sv.max()) < 1.25


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1.0, 1e12, 1e30])
def test_scale_invariance(sdc, scale):
    # eps = 0: the result does not depend on the scale, even where squares of the
    # entries leave float32's range
    m = update(5, 1, 70, 300) * 1e3
    ref = ns64(m, eps=0.0)
    o = sdc.orthogonalize((m.double() * scale).float(), eps=0.0)
    assert rel(o, ref) <= 2e-5


def test_rows_of_very_different_size(sdc):
    # entries from 1 to 1e-6 of the largest: float16's range alone would not hold them
    m = randn(1, (96, 400)) * torch.logspace(0, -6, 96, device="cuda").unsqueeze(1)
    o = sdc.orthogonalize(m)
    ref = ns64(m)
    assert rel(o, ref) <= 1e-5
    # the small rows by themselves: 2^-24 absolute in X, amplified at most 485 times
    assert float((o.double() - ref).abs().max()) <= 485 * 2.0 ** -23


@pytest.mark.parametrize("rows,cols", [(60, 200), (64, 448), (128, 896), (128, 128), (300, 500), (1024, 600)])
def test_no_single_entry_is_off(sdc, rows, cols):
    # Two steps amplify by at most a^2 = 12; an operand is off by 2^-22 of its
    # entry at most, the largest entry is some five times the root mean square:
    # 12 * 2^-22 * 5 = 1.4e-5 of that.  A hi and a lo part that do not belong
    # together would put single entries 1e-4 to 1e-3 off, unseen in the norm.
    m = update(7, 1, rows, cols)
    d = (sdc.orthogonalize(m, steps=2).double() - ns64(m, 2)).abs()
    assert float(d.max() / ns64(m, 2).square().mean().sqrt()) <= 2e-5


def test_zero_nan_infinity(sdc):
    for rows, cols in ((5, 9), (64, 448), (130, 200), (300, 40)):
        m = update(1, 4, rows, cols)
        clean = sdc.orthogonalize(m)
        m[1].zero_()
        m[2, rows // 2, cols // 3] = float("nan")
        m[3, rows - 1, 0] = float("inf")
        o = sdc.orthogonalize(m)
        assert torch.equal(o[0], clean[0])
        assert not o[1].any()
        assert torch.isnan(o[2]).all() and torch.isnan(o[3]).all()


def step64(w, g, buf, lr, beta, nesterov, wd, scale, groups, steps=5):
    rows = w.shape[0] // groups
    b = beta * buf.double() + g.double()
    u = g.double() + beta * b if nesterov else b
    o = ns64(u.view(groups, rows, -1), steps).view(w.shape)
    return w.double() * (1 - lr * wd) - lr * scale * o, b


@pytest.mark.parametrize("shape,groups", [((4, 4, 3), 1), ((256, 1, 17), 256), ((64, 64, 7), 1), ((128, 128, 7), 1),
                                          ((96, 10, 7), 4), ((500, 33), 1), ((6, 40), 6), ((1024, 1500), 1),
                                          ((300, 20), 2)])
def test_step(sdc, shape, groups):
    rows, cols = shape[0] // groups, math.prod(shape[1:])
    for tw, tg, nesterov, wd, scale in ((F32, F32, True, 0.01, None), (F32, BF16, False, 0.0, 0.2),
                                        (BF16, BF16, True, 0.1, None), (BF16, F32, False, 0.1, 1.0)):
        w = (randn(1, shape) / math.sqrt(cols)).to(tw)
        g = update(2, groups, rows, cols, tg).view(shape)
        buf = 5 * update(9, groups, rows, cols).view(shape)
        s = math.sqrt(max(1.0, rows / cols)) if scale is None else scale
        rw, rb = step64(w, g, buf, 0.02, 0.95, nesterov, wd, s, groups)
        w0, b0 = w.clone(), buf.clone()
        w2, b2, w16 = sdc.muon_step(w, g, buf, 0.02, nesterov=nesterov, weight_decay=wd, scale=scale,
                                    groups=groups, w_out=torch.empty_like(w),
                                    momentum_out=torch.empty_like(buf), need_bf16_copy=tw == F32)
        assert torch.equal(w, w0) and torch.equal(buf, b0)
        # the step moves w by 0.02 s |o|, so the update itself is what is compared:
        # its bar plus the rounding of w
        du, dr = w2.double() - w0.double() * (1 - 0.02 * wd), rw - w0.double() * (1 - 0.02 * wd)
        wround = float(w0.double().norm()) * (2.0 ** -23 if tw == F32 else 2.0 ** -8)
        assert float((du - dr).norm()) <= bar(tw, rows, cols) * float(dr.norm()) + wround
        assert rel(b2, rb) <= 2.0 ** -23
        if tw == F32:
            assert torch.equal(w16, w2.to(BF16))
        else:
            assert w16 is None
        # in place: the same bits
        w3, b3, _ = sdc.muon_step(w, g, buf, 0.02, nesterov=nesterov, weight_decay=wd, scale=scale,
                                  groups=groups)
        assert w3 is w and b3 is buf and torch.equal(w, w2) and torch.equal(buf, b2)


def test_several_steps_follow_float64(sdc):
    shape, groups = (48, 20, 7), 2
    w, buf = randn(1, shape) / 10, torch.zeros(shape, device="cuda")
    w64, b64 = w.double(), buf.double()
    for k in range(6):
        g = update(20 + 3 * k, groups, 24, 140).view(shape)
        sdc.muon_step(w, g, buf, 0.05, weight_decay=0.1, groups=groups)
        w64, b64 = step64(w64, g, b64, 0.05, 0.95, True, 0.1, 1.0, groups)
    assert rel(w, w64) <= 1e-5 and rel(buf, b64) <= 1e-6


def test_views_that_start_anywhere(sdc):
    for t in (F32, BF16):
        for rows, cols in ((33, 65), (130, 257), (7, 5)):
            n = rows * cols
            m = update(1, 1, 1, n + 8, t).view(-1)[3:3 + n].view(rows, cols)
            o = torch.full((n + 8,), 7.0, device="cuda", dtype=t)
            sdc.orthogonalize(m, out=o[1:1 + n].view(rows, cols))
            assert rel(o[1:1 + n].view(rows, cols), ns64(m)) <= bar(t, rows, cols)
            assert (o[:1] == 7).all() and (o[1 + n:] == 7).all()


def test_empty(sdc):
    for shape in ((0, 4, 5), (2, 0, 5), (2, 4, 0), (0, 7)):
        m = torch.empty(shape, device="cuda")
        assert sdc.orthogonalize(m).shape == m.shape
        if len(shape) == 2:
            sdc.muon_step(m, m.clone(), m.clone(), 0.1)


@pytest.mark.parametrize("rows,cols", [(64, 448), (128, 896), (150, 200)])
def test_another_stream_and_graph(sdc, rows, cols):
    m = update(1, 2, rows, cols)
    ref = sdc.orthogonalize(m)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sdc.orthogonalize(m, stream=side)
    side.synchronize()
    assert torch.equal(got, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = sdc.orthogonalize(m)
    for _ in range(4):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, ref)
        _ = float(o.sum())


def test_refusals(sdc):
    m = update(1, 2, 8, 12)
    with pytest.raises(ValueError):
        sdc.orthogonalize(m.half())
    with pytest.raises(ValueError):
        sdc.orthogonalize(m.mT)
    with pytest.raises(ValueError):
        sdc.orthogonalize(m.view(-1))
    with pytest.raises(ValueError):
        sdc.orthogonalize(m, steps=0)
    with pytest.raises(ValueError):
        sdc.orthogonalize(m, eps=-1.0)
    with pytest.raises(ValueError):
        sdc.orthogonalize(m, out=m)
    with pytest.raises(ValueError):
        sdc.orthogonalize(m, coeffs=(1.0, 2.0))
    with pytest.raises(ValueError):
        sdc.orthogonalize(m, coeffs=(float("nan"), 0.0, 0.0))
    with pytest.raises(NotImplementedError):
        sdc.orthogonalize(m, coeffs=(50.0, 0.0, 0.0))
    with pytest.raises(NotImplementedError):
        sdc.orthogonalize(m, steps=1, coeffs=(50.0, 0.0, 0.0))
    with pytest.raises(ValueError):
        sdc.orthogonalize(m.cpu())
    w = randn(1, (8, 12))
    g, b = w.clone(), torch.zeros_like(w)
    with pytest.raises(ValueError):
        sdc.muon_step(w, g, b, 0.1, groups=3)
    with pytest.raises(ValueError):
        sdc.muon_step(w, g[:4], b, 0.1)
    with pytest.raises(ValueError):
        sdc.muon_step(w, g, b.to(BF16), 0.1)
    with pytest.raises(ValueError):
        sdc.muon_step(w, g, None, 0.1)
    with pytest.raises(ValueError):
        sdc.muon_step(w, g, b, float("inf"))
    with pytest.raises(ValueError):
        sdc.muon_step(w, g, b, 0.1, beta=1.0)
    with pytest.raises(ValueError):
        sdc.muon_step(w, w, b, 0.1)                      # grad is what is overwritten
    with pytest.raises(ValueError):
        sdc.muon_step(w, g, b, 0.1, w_out=b)
    with pytest.raises(ValueError):
        sdc.muon_step(w.to(BF16), g, b, 0.1, need_bf16_copy=True)
    lib = sdc._lib
    m = update(1, 2, 200, 300)   # small matrices need no workspace
    o = torch.empty_like(m)
    need = lib.disco_orthogonalize_workspace(2, 200, 300)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert lib.disco_orthogonalize(m.data_ptr(), 0, o.data_ptr(), 0, 2, 200, 300, 5, None, 1e-7,
                                   ws.data_ptr(), need - 1, None) == sdc.DISCO_EINVAL
    assert "workspace" in lib.disco_last_error().decode()
