"""Dropout: the mask against the generator's definition, values against float64."""
import math

import pytest

torch = pytest.importorskip("torch")
from attention_reference import BF16, F32, half_step, halves  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import spherical_disco_convolution_amd as m
    return m


def randn(seed, n, dtype=F32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(n, generator=g, device="cuda").to(dtype)


def kept(n, p, seed, offset):
    return torch.from_numpy(halves(n, seed, offset) >= math.floor(p * 65536 + 0.5))


def scale(p):
    return 65536.0 / (65536 - math.floor(p * 65536 + 0.5))


@pytest.mark.parametrize("tx", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("ty", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2047, 2048, 2049, 100003])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999])
def test_values(sdc, n, p, tx, ty):
    x, res = randn(n, n, tx), randn(n + 1, n, tx)
    seed, offset = 0xfedcba9876543210, 2 ** 33 + 5
    mask = kept(n, p, seed, offset)
    want = torch.where(mask, x.double().cpu() * scale(p), 0.0)
    # the scale and two operations in float32, then the result's rounding
    for r, y in ((None, sdc.dropout_fwd(x, p, seed, offset, out_dtype=ty)),
                 (res, sdc.dropout_fwd(x, p, seed, offset, residual=res, out_dtype=ty)),
                 (None, sdc.dropout_bwd(x, p, seed, offset, gx_dtype=ty))):
        w = want if r is None else want + r.double().cpu()
        bound = 3 * 2.0 ** -24 * (want.abs() + w.abs()) + half_step(ty) * w.abs()
        assert y.dtype == ty and y.shape == x.shape
        assert bool(((y.double().cpu() - w).abs() <= bound).all())
        if r is None:
            assert bool((y.cpu()[~mask] == 0.0).all())


@pytest.mark.parametrize("seed,offset", [(0, 0), (-1, -1), (2 ** 64 - 1, 2 ** 64 - 1), (1, 2 ** 32), (2 ** 32, 1)])
def test_masks_of_seeds_and_offsets(sdc, seed, offset):
    x = torch.ones(5000, device="cuda")
    y = sdc.dropout_fwd(x, 0.5, seed, offset)
    assert torch.equal(y.cpu() != 0, kept(5000, 0.5, seed, offset))


def test_what_is_dropped_is_zero(sdc):
    x = torch.full((4096,), math.nan, device="cuda")
    y = sdc.dropout_fwd(x, 0.5, 3)
    mask = kept(4096, 0.5, 3, 0)
    assert bool((y.cpu()[~mask] == 0).all()) and bool(y.cpu()[mask].isnan().all())


def test_odd_addresses_and_in_place(sdc):
    for dtype in (F32, BF16):
        buf = randn(1, 10001, dtype)
        x = buf[3:9004]
        want = sdc.dropout_fwd(x.clone(), 0.3, 9)
        before = buf.clone()
        assert sdc.dropout_fwd(x, 0.3, 9, y=x) is x
        assert torch.equal(x, want)
        assert torch.equal(buf[:3], before[:3]) and torch.equal(buf[9004:], before[9004:])
        g = sdc.dropout_bwd(want.clone(), 0.3, 9, gx_dtype=dtype)
        assert torch.equal(g != 0, want != 0)


def test_the_share_and_the_mean(sdc):
    # of n draws of probability q the share is off by 6 sqrt(q (1 - q) / n) in one of 10^9 cases
    n, p = 1 << 24, 0.1
    y = sdc.dropout_fwd(torch.ones(n, device="cuda"), p, 12345)
    q = 1 - math.floor(p * 65536 + 0.5) / 65536
    assert abs(float((y != 0).double().mean()) - q) <= 6 * math.sqrt(q * (1 - q) / n)


def test_a_step_counter_in_a_graph(sdc):
    x = torch.ones(4096, device="cuda")
    step = torch.zeros((), dtype=torch.int64, device="cuda")
    sdc.dropout_fwd(x, 0.5, 7, 100, step=step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = sdc.dropout_fwd(x, 0.5, 7, 100, step=step)
        g = sdc.dropout_bwd(x, 0.5, 7, 100, step=step)
        step.add_(1)
    for i in range(4):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu() != 0, kept(4096, 0.5, 7, 100 + i))
        assert torch.equal(y, g)
        assert torch.equal(y, sdc.dropout_fwd(x, 0.5, 7, 100 + i))


@pytest.mark.parametrize("n", [(1 << 31) + 4099, (1 << 34) + 4099])   # the last takes two launches
def test_past_2_31_elements(sdc, n):
    x = torch.ones(n, dtype=BF16, device="cuda")
    y = sdc.dropout_fwd(x, 0.5, 5, 6, y=x)
    # blocks at the far end, by a call whose counters the definition gives
    import numpy as np
    from attention_reference import philox
    blocks = np.arange((n - 4096) // 8, (n + 7) // 8, dtype=np.uint64)
    words = philox(blocks, blocks * 0, blocks * 0 + 6, blocks * 0, 5, 0)
    h = np.stack([v for w in words for v in (w & np.uint64(0xffff), w >> np.uint64(16))], axis=1).reshape(-1)
    first = int(blocks[0]) * 8
    want = torch.from_numpy(h[:n - first].astype(np.int64) >= 32768)
    assert torch.equal(y[first:].cpu() != 0, want)
    del x, y
    torch.cuda.empty_cache()
