"""Layer norm forward and backward on the GPU against the formulas in float64
on the same inputs.

Tolerances.  float32 results: the statistics are sums of at most C float32
terms in chains of at most a few hundred, so a result's relative error stays
below a few hundred times 2^-24; the bar is the layer's float32 bar, 1e-5
(relative L2).  bfloat16 results add one rounding of at most 2^-9 of each
element: relative L2 at most 2^-9, with a factor of two in hand 2^-8.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
BAR = {F32: 1e-5, BF16: 2.0 ** -8}


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
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm().clamp_min(1e-300))


def fwd64(s, gamma, beta, axis, eps):
    f = s.double()
    mean = f.mean(dim=axis, keepdim=True)
    rstd = ((f - mean).square().mean(dim=axis, keepdim=True) + eps).rsqrt()
    shape = [1] * s.dim()
    shape[axis] = -1
    y = (f - mean) * rstd
    if gamma is not None:
        y = y * gamma.double().view(shape)
    if beta is not None:
        y = y + beta.double().view(shape)
    return y, mean.squeeze(axis), rstd.squeeze(axis)


def bwd64(x, gy, mean, rstd, gamma, gsum, axis):
    shape = [1] * x.dim()
    shape[axis] = -1
    r = rstd.double().unsqueeze(axis)
    h = (x.double() - mean.double().unsqueeze(axis)) * r
    g = gy.double()
    t = g if gamma is None else g * gamma.double().view(shape)
    gx = r * (t - t.mean(axis, keepdim=True) - h * (t * h).mean(axis, keepdim=True))
    if gsum is not None:
        gx = gx + gsum.double()
    dims = [d for d in range(x.dim()) if d != axis % x.dim()]
    return gx, (g * h).sum(dims), g.sum(dims)


FIELDS = [(1, 4, 33, 64), (1, 1, 5, 7), (2, 3, 9, 16), (3, 8, 1, 2), (1, 17, 12, 31), (4, 32, 129, 256),
          (1, 100, 37, 72), (2, 128, 33, 65), (1, 130, 20, 41), (1, 256, 61, 120), (1, 300, 9, 17),
          (1, 512, 45, 91), (2, 600, 7, 9), (300, 6, 3, 1), (1, 128, 361, 720), (1, 16, 721, 1439),
          (5, 24, 181, 359)]
ROWS = [(1, 1), (3, 5), (1, 7), (300, 8), (2, 16), (70, 63), (5, 64), (129, 129), (1, 1000), (9, 2048),
        (5000, 96), (2500, 2049), (4100, 31), (2, 4099), (3000, 4100), (600, 8192), (520, 8200), (1, 16384), (3, 16385), (2, 40001), (1, 1)]
CASES = [(s, 1) for s in FIELDS] + [(s, -1) for s in ROWS]
TYPES = [(F32, F32, False), (F32, BF16, True), (BF16, BF16, True), (BF16, F32, False), (BF16, BF16, False)]


@pytest.mark.parametrize("shape,axis", CASES)
def test_forward(sdc, shape, axis):
    C = shape[axis]
    gamma, beta = 1 + 0.1 * randn(1, (C,)), 0.1 * randn(2, (C,))
    for k, (tx, ty, with_res) in enumerate(TYPES):
        x = (randn(3 + k, shape) * 1.5 + 0.7).to(tx)
        res = randn(30 + k, shape, tx) if with_res else None
        y, s, mean, rstd = sdc.layer_norm_fwd(x, gamma, beta, residual=res, axis=axis, out_dtype=ty)
        assert y.dtype == ty and mean.dtype == rstd.dtype == F32
        if with_res:
            assert torch.equal(s, (x.float() + res.float()).to(tx))
        else:
            assert s is None
        ry, rmean, rrstd = fwd64(s if with_res else x, gamma, beta, axis, 1e-5)
        assert mean.shape == rmean.shape
        assert rel(y, ry) <= BAR[ty], (tx, ty)
        assert float((mean.double() - rmean).abs().max()) <= 1e-5 * float(x.float().abs().max() + 1)
        assert rel(rstd, rrstd) <= 1e-5
        # without statistics, weights and offsets the same values come out
        y2, _, m2, r2 = sdc.layer_norm_fwd(x, gamma, beta, residual=res, axis=axis, out_dtype=ty,
                                           need_stats=False)
        assert m2 is None and r2 is None and torch.equal(y, y2)
        y3 = sdc.layer_norm_fwd(x, residual=res, axis=axis, out_dtype=ty)[0]
        assert rel(y3, fwd64(s if with_res else x, None, None, axis, 1e-5)[0]) <= BAR[ty]


@pytest.mark.parametrize("shape,axis", CASES)
def test_backward(sdc, shape, axis):
    C = shape[axis]
    gamma = 1 + 0.1 * randn(1, (C,))
    for k, (tx, tg, to, with_sum) in enumerate([(F32, F32, F32, False), (BF16, BF16, BF16, True),
                                                (F32, BF16, BF16, True), (BF16, F32, F32, False)]):
        x = (randn(3 + k, shape) * 1.5 + 0.7).to(tx)
        gy = randn(40 + k, shape, tg)
        gsum = randn(50 + k, shape, tg) if with_sum else None
        _, mean, rstd = fwd64(x, None, None, axis, 1e-5)
        mean, rstd = mean.float(), rstd.float()
        gx, gg, gb = sdc.layer_norm_bwd(x, gy, mean, rstd, gamma, gsum=gsum, axis=axis, gx_dtype=to)
        rx, rg, rb = bwd64(x, gy, mean, rstd, gamma, gsum, axis)
        # C == 1: h = 0 and gx = 0 + gsum up to rounding of t - t
        scale = max(float(rx.norm()), float((gy.double() * rstd.double().unsqueeze(axis)).norm()) * 1e-2)
        assert float((gx.double() - rx).norm()) <= BAR[to] * scale, (tx, tg, to)
        # the sums run over points of both signs: their error is measured against
        # the sums of the magnitudes
        dims = [d for d in range(x.dim()) if d != axis % x.dim()]
        h = ((x.double() - mean.double().unsqueeze(axis)) * rstd.double().unsqueeze(axis)).abs()
        mag_g, mag_b = (gy.double().abs() * h).sum(dims), gy.double().abs().sum(dims)
        assert float(((gg.double() - rg).abs() - 2e-6 * mag_g).max()) <= 1e-30
        assert float(((gb.double() - rb).abs() - 2e-6 * mag_b).max()) <= 1e-30
        again = sdc.layer_norm_bwd(x, gy, mean, rstd, gamma, gsum=gsum, axis=axis, gx_dtype=to)
        assert torch.equal(gx, again[0]) and torch.equal(gg, again[1]) and torch.equal(gb, again[2])
        only = sdc.layer_norm_bwd(x, gy, mean, rstd, gamma, gsum=gsum, axis=axis, gx_dtype=to,
                                  need_gparams=False)
        assert torch.equal(only[0], gx) and only[1] is None and only[2] is None
        par = sdc.layer_norm_bwd(x, gy, mean, rstd, gamma, axis=axis, need_gx=False)
        assert par[0] is None and torch.equal(par[1], gg) and torch.equal(par[2], gb)


# one, two, four and more rows a workgroup, one and several rounds, a last round that is not full
@pytest.mark.parametrize("rows,C", [(1031, 4096), (511, 4097), (1025, 8192), (1300, 2400), (2600, 777), (2049, 513),
                                    (9000, 129), (260, 12345)])
def test_backward_rows_of_a_workgroup(sdc, rows, C):
    test_backward(sdc, (rows, C), -1)


@pytest.mark.parametrize("shape,axis", [((2, 12, 9, 14), 1), ((40, 24), -1)])
def test_gradient_against_differences(sdc, shape, axis):
    # central differences of L = sum(gy y + gs s) along random directions; step
    # h = 1/64: truncation O(h^2) ~ 2e-4, rounding 2^-23 sqrt(n) / h ~ 5e-4 of
    # the gradient's norm along the direction
    C = shape[axis]
    gamma, beta = 1 + 0.1 * randn(1, (C,)), 0.1 * randn(2, (C,))
    x, gy, gs = randn(3, shape) + 0.5, randn(4, shape), randn(5, shape)
    _, _, mean, rstd = sdc.layer_norm_fwd(x, gamma, beta, axis=axis)
    gx, gg, gb = sdc.layer_norm_bwd(x, gy, mean, rstd, gamma, gsum=gs, axis=axis)

    def loss(xx, ga, be):
        y = sdc.layer_norm_fwd(xx, ga, be, axis=axis)[0]
        return float((y.double() * gy.double()).sum() + (xx.double() * gs.double()).sum())

    h = 1.0 / 64
    for k in range(4):
        d, dg, db = randn(10 + k, shape), randn(20 + k, (C,)), randn(30 + k, (C,))
        for got, num in (((gx.double() * d.double()).sum(),
                          (loss(x + h * d, gamma, beta) - loss(x - h * d, gamma, beta)) / (2 * h)),
                         ((gg.double() * dg.double()).sum(),
                          (loss(x, gamma + h * dg, beta) - loss(x, gamma - h * dg, beta)) / (2 * h)),
                         ((gb.double() * db.double()).sum(),
                          (loss(x, gamma, beta + h * db) - loss(x, gamma, beta - h * db)) / (2 * h))):
            bound = 2e-3 * float(gx.norm()) * float(d.norm()) / (x.numel() ** 0.5)
            assert abs(float(got) - num) <= max(bound, 2e-3 * abs(num)) + 1e-2, k


@pytest.mark.parametrize("shape,axis", [((2, 64, 19, 33), 1), ((7, 600), -1)])
def test_a_large_offset_keeps_its_spread(sdc, shape, axis):
    # x = 1000 + N(0, 1) in float32: a mean that is off by some ulps of 1000
    # (6.1e-5) moves y by as much; 8 ulps allowed.  E[x^2] - mean^2 would lose
    # every digit of the variance.
    x = 1000 + randn(1, shape)
    y = sdc.layer_norm_fwd(x, axis=axis)[0]
    assert float((y.double() - fwd64(x, None, None, axis, 1e-5)[0]).abs().max()) <= 8 * 6.1e-5


@pytest.mark.parametrize("shape,axis", [((2, 24, 11, 37), 1), ((40, 96), -1), ((1, 128, 181, 360), 1)])
def test_a_nan_or_infinity_stays_in_its_point(sdc, shape, axis):
    x = randn(1, shape, BF16)
    gy = randn(2, shape, BF16)
    clean, _, mean, rstd = sdc.layer_norm_fwd(x, axis=axis)
    gclean = sdc.layer_norm_bwd(x, gy, mean, rstd, axis=axis, gx_dtype=BF16)[0]
    for bad in (float("nan"), float("inf"), -float("inf")):
        xb, gb = x.clone(), gy.clone()
        where = (0, 3, 5, 17) if axis == 1 else (5, 3)
        xb[where] = bad
        y, _, m2, r2 = sdc.layer_norm_fwd(xb, axis=axis)
        hit = torch.zeros(shape, dtype=torch.bool, device="cuda")
        hit[(where[0], slice(None)) + where[2:]] = True
        assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], clean[~hit])
        gb[where] = bad
        gx = sdc.layer_norm_bwd(x, gb, mean, rstd, axis=axis, gx_dtype=BF16)[0]
        assert not torch.isfinite(gx[hit]).any() and torch.equal(gx[~hit], gclean[~hit])


def test_constant_points_give_beta(sdc):
    # the float32 mean of C equal values v is off by at most some ulps of v;
    # 1/sqrt(eps) = 316 magnifies that
    beta = randn(1, (48,))
    for shape, axis in (((2, 48, 5, 9), 1), ((6, 48), -1)):
        x = torch.full(shape, 2.5, device="cuda")
        y = sdc.layer_norm_fwd(x, None, beta, axis=axis)[0]
        want = beta.view([-1 if d == axis % len(shape) else 1 for d in range(len(shape))])
        assert float((y - want).abs().max()) <= 316 * 4 * 2.5 * 2.0 ** -24


@pytest.mark.parametrize("tx", [F32, BF16])
def test_views_that_start_anywhere(sdc, tx):
    # contiguous tensors at storage offsets that are multiples of the element only
    for shape, axis in (((2, 20, 7, 33), 1), ((1, 64, 40, 901), 1), ((31, 257), -1)):
        n = 1
        for d in shape:
            n *= d
        for off in (1, 3):
            x = randn(1, (n + 8,), tx)[off:off + n].view(shape)
            gy = randn(2, (n + 8,), tx)[off:off + n].view(shape)
            y = torch.full((n + 8,), 7.0, device="cuda", dtype=tx)
            out = y[off:off + n].view(shape)
            _, _, mean, rstd = sdc.layer_norm_fwd(x, axis=axis, y=out)
            assert rel(out, fwd64(x, None, None, axis, 1e-5)[0]) <= BAR[tx]
            assert (y[:off] == 7).all() and (y[off + n:] == 7).all()
            gx = sdc.layer_norm_bwd(x, gy, mean, rstd, axis=axis, gx_dtype=tx)[0]
            assert rel(gx, bwd64(x, gy, mean, rstd, None, None, axis)[0]) <= BAR[tx]


def test_offsets_past_32_bits(sdc):
    # 2.3e9 elements: zeros but for the first and last points
    shape, k = (2, 128, 9_000_001), 700
    x = torch.zeros(shape, device="cuda", dtype=BF16)
    x[0, :, :k], x[1, :, -k:] = randn(1, (128, k), BF16), randn(2, (128, k), BF16)
    y, _, mean, rstd = sdc.layer_norm_fwd(x)
    for part in ((slice(0, 1), slice(None), slice(0, k)), (slice(1, 2), slice(None), slice(-k, None))):
        ry, rm, rr = fwd64(x[part], None, None, 1, 1e-5)
        assert rel(y[part], ry) <= BAR[BF16]
    assert not y[0, :, k:].any() and not y[1, :, :-k].any()
    gx, gg, gb = sdc.layer_norm_bwd(x, y, mean, rstd, gx_dtype=BF16)
    part = (slice(1, 2), slice(None), slice(-k, None))
    rx, _, _ = bwd64(x[part], y[part], mean[1:, -k:], rstd[1:, -k:], None, None, 1)
    # gx cancels t against its projections here (y is t's own direction): what is
    # left is bounded by the bf16 rounding of t
    assert float((gx[part].double() - rx).abs().max()) <= 2.0 ** -8 * float(y[part].float().abs().max())
    assert not gx[0, :, k:].any() and not gx[1, :, :-k].any()
    assert torch.isfinite(gg).all() and torch.isfinite(gb).all()


def test_empty_tensors(sdc):
    for shape, axis in (((0, 8, 3, 4), 1), ((2, 8, 0, 4), 1), ((0, 8), -1)):
        x = torch.empty(shape, device="cuda")
        y, _, mean, rstd = sdc.layer_norm_fwd(x, axis=axis)
        assert y.shape == x.shape and mean.numel() == 0
        gx, gg, gb = sdc.layer_norm_bwd(x, x, mean, rstd, axis=axis)
        assert gx.shape == x.shape and not gg.any() and not gb.any()


def test_another_stream_and_graph(sdc):
    x, gy = randn(1, (2, 32, 33, 64)), randn(2, (2, 32, 33, 64))
    ref = sdc.layer_norm_fwd(x)
    gref = sdc.layer_norm_bwd(x, gy, ref[2], ref[3])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sdc.layer_norm_fwd(x, stream=side)
    ggot = sdc.layer_norm_bwd(x, gy, got[2], got[3], stream=side)
    side.synchronize()
    assert torch.equal(got[0], ref[0])
    assert all(torch.equal(a, b) for a, b in zip(ggot, gref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _, mean, rstd = sdc.layer_norm_fwd(x)
        out = sdc.layer_norm_bwd(x, gy, mean, rstd)
    for _ in range(4):
        y.zero_()
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref[0]) and all(torch.equal(a, b) for a, b in zip(out, gref))
        _ = float(y.sum())


def test_refusals(sdc):
    x = randn(1, (2, 8, 5, 6))
    y, _, mean, rstd = sdc.layer_norm_fwd(x)
    with pytest.raises(ValueError):
        sdc.layer_norm_fwd(x.half())
    with pytest.raises(ValueError):
        sdc.layer_norm_fwd(x.transpose(2, 3))
    with pytest.raises(ValueError):
        sdc.layer_norm_fwd(x, gamma=torch.ones(7, device="cuda"))
    with pytest.raises(ValueError):
        sdc.layer_norm_fwd(x, gamma=torch.ones(8, device="cuda", dtype=BF16))
    with pytest.raises(ValueError):
        sdc.layer_norm_fwd(x, residual=x.to(BF16))
    with pytest.raises(ValueError):
        sdc.layer_norm_fwd(x, axis=4)
    with pytest.raises(ValueError):
        sdc.layer_norm_fwd(x, eps=-1.0)
    with pytest.raises(ValueError):
        sdc.layer_norm_fwd(x, eps=float("nan"))
    with pytest.raises(ValueError):
        sdc.layer_norm_fwd(x, y=x)                       # in place
    with pytest.raises(ValueError):
        sdc.layer_norm_fwd(x.cpu())
    with pytest.raises(ValueError):
        sdc.layer_norm_bwd(x, y, None, None)
    with pytest.raises(ValueError):
        sdc.layer_norm_bwd(x, y, mean[:1], rstd)
    with pytest.raises(ValueError):
        sdc.layer_norm_bwd(x, y, mean, rstd, gsum=y.to(BF16))
    with pytest.raises(ValueError):
        sdc.layer_norm_bwd(x, y, mean, rstd, need_gx=False, need_gparams=False)
    gg = torch.empty(8, device="cuda")
    lib = sdc._lib
    args = (x.data_ptr(), 0, y.data_ptr(), 0, mean.data_ptr(), rstd.data_ptr(), None, None, None, 0,
            gg.data_ptr(), None)
    need = lib.disco_layer_norm_bwd_workspace(2, 8, 30)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert lib.disco_layer_norm_bwd(*args, ws.data_ptr(), need - 1, 2, 8, 30, None) == sdc.DISCO_EINVAL
    assert "workspace" in lib.disco_last_error().decode()
    assert lib.disco_layer_norm_bwd(*args, None, 0, 2, 8, 30, None) == sdc.DISCO_EINVAL
