"""Attention under large finite biases and scores: masks made of
-1e4 to -1e30 on a few keys, on tiles and on whole rows, large positive biases, large
products.

Queries and keys are small integers times a power of two, chosen so that every float32
score is either exact or the bias alone (all of q.k is below half its last place).  The
scores are then known whatever the order of the sums, and the formulas in float64 hold
for the kernels' own scores."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from attention_reference import BF16, F32, half_step  # noqa: E402

pytestmark = pytest.mark.gpu
INF = math.inf
U = 2.0 ** -24
FAR = 45000.0     # |lse| up to which a gradient's weights may carry the rounding of lse
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


@pytest.fixture(scope="module")
def sdc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import spherical_disco_convolution_amd as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def unit(b):
    """Largest entry of q and k under a bias of b: products are multiples of the last
    place of b / scale for heads of up to 128 (|b| of 1e8 and 1e9), or lost in it."""
    return 16 if 1e7 < abs(b) < 5e8 else 32 if 5e8 < abs(b) < 5e9 else 1


def inputs(seed, lq, lk, hq, hkv, d, dtype, size=1, most=1):
    g = gen(seed)

    def whole(*shape):
        return (size * torch.randint(-most, most + 1, shape, generator=g, device="cuda")).to(dtype)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    return whole(lq, hq, d), whole(lk, hkv, d), normal(lk, hkv, d), normal(lq, hq, d)


def scores(q, k, bias, scale):
    """Scores of one head as float32 holds them, in units of the scale: [Lq, Lk]"""
    raw = (q.double().cpu() @ k.double().cpu().T).numpy()
    if bias is not None:
        per = np.float32(1.0) / np.float32(scale)
        b = (bias.cpu().numpy() * per).astype(np.float32).astype(np.float64)
        raw = np.where(np.isinf(b), -INF, (raw + np.where(np.isinf(b), 0.0, b)).astype(np.float32).astype(np.float64))
    return torch.from_numpy(raw) * float(np.float32(scale))


def reference(q, k, v, bias, causal, scale, go):
    """{name: (value, bound)}, float64.  The bounds count: the exponent, a float32 product
    of at most 128 that matters, and its exponential; in gradients of ordinary rows the
    rounding of lse and of the scores, 16 u of their size; sums; half a step of each
    weight and each ds in bfloat16, and of each result."""
    dtype = q.dtype
    half = half_step(dtype)
    low = half if dtype == BF16 else 0.0
    (lq, hq, _), (lk, hkv, d) = q.shape, v.shape
    g = hq // hkv
    q64, k64, v64, go64 = (t.double().cpu() for t in (q, k, v, go))
    res = {n: (torch.zeros(s, dtype=torch.float64), torch.zeros(s, dtype=torch.float64))
           for n, s in (("o", (lq, hq, d)), ("lse", (lq, hq)), ("gq", q.shape), ("gk", k.shape), ("gv", v.shape))}

    def add(name, at, value, bound):
        res[name][0][at] += value
        res[name][1][at] += bound

    for h in range(hq):
        j = h // g
        qs, ks, vs, gs = q64[:, h], k64[:, j], v64[:, j], go64[:, h]
        x = scores(q[:, h], k[:, j], bias, scale)
        if causal:
            x = torch.where(torch.arange(lk) <= torch.arange(lq)[:, None] + lk - lq, x, -INF)
        l = torch.logsumexp(x, 1)
        fin = l.isfinite()
        size = torch.where(fin, l, 0.0).abs()[:, None]
        p = torch.softmax(x, 1).nan_to_num(0.0)   # of l, float64 too would have lost the sum's digits
        ax = scale * (qs.abs() @ ks.abs().T).max(1, keepdim=True).values
        dw = (lk + 16) * U + 16 * U * 128
        o = p @ vs
        add("o", (slice(None), h), o, (dw + low) * (p @ vs.abs()) + half * o.abs())
        res["lse"][0][:, h], res["lse"][1][:, h] = l, 6 * U * size[:, 0] + (lk + 16) * U
        dp, delta = gs @ vs.T, (gs * o).sum(1, keepdim=True)
        # delta comes from the rounded o
        err = (d + 2) * U * (gs.abs() @ vs.abs().T + (gs * o).abs().sum(1, keepdim=True)) + (
            gs.abs() * res["o"][1][:, h]).sum(1, keepdim=True)
        ds = p * (dp - delta)
        dw = dw + torch.where(size < FAR, 16 * U * (size + ax), 0.0)
        es = p * (dw * (dp.abs() + delta.abs()) + err) + low * ds.abs()
        add("gq", (slice(None), h), scale * ds @ ks, scale * (es + (lk + 4) * U * ds.abs()) @ ks.abs())
        add("gk", (slice(None), j), scale * ds.T @ qs, scale * (es + (g * lq + 4) * U * ds.abs()).T @ qs.abs())
        add("gv", (slice(None), j), p.T @ gs, (p * (dw + low + (g * lq + 4) * U)).T @ gs.abs())
    for n in ("gq", "gk", "gv"):
        res[n] = (res[n][0], res[n][1] + half * res[n][0].abs())
    return res


def check(got, want):
    for name, t in zip(("o", "lse", "gq", "gk", "gv"), got):
        w, bound = want[name]
        t, inf = t.double().cpu(), w.isinf()
        assert torch.equal(t[inf], w[inf]), name
        assert bool(t[~inf].isfinite().all()), f"{name}: not finite"
        far = ((t - w).abs() - bound)[~inf]
        assert float(far.max()) <= 1e-30, (
            f"{name}: {float(far.max()):.3g} over the bound; largest difference {float((t - w).abs()[~inf].max()):.3g}")


BIASES = [-1e4, -1e5, -1e8, -1e9, -1e10, -1e20, -1e29, -1e30, 1e8, 1e9, 1e10, 1e29]
WHERE = {"some": lambda n: torch.arange(n) % 3 == 0, "leading": lambda n: torch.arange(n) < 40,
         "tiles": lambda n: torch.arange(n) < 128, "inside": lambda n: (torch.arange(n) >= 128) & (torch.arange(n) < 256),
         "all": lambda n: torch.arange(n) >= 0}


def biased(lq, lk, hq, hkv, d, b, where, causal=False):
    """(q, k, v, go, bias, causal) of a type, with b on the keys of `where`"""
    def make(dtype):
        bias = torch.where(WHERE[where](lk), b, 0.0).cuda()
        return inputs(lq + d, lq, lk, hq, hkv, d, dtype, unit(b)) + (bias, causal)
    return make


def large(lq, lk, d, causal):
    # no bias: products are multiples of 2^18 of at most 2^26, exact in float32
    return lambda dtype: inputs(5, lq, lk, 2, 1, d, dtype, 512, 2) + (None, causal)


CASES = {f"{lq}x{lk} {b:g} {w}": biased(lq, lk, 4, 2, 64, b, w)
         for lq, lk in ((150, 300), (3, 5000)) for b in BIASES for w in WHERE}
CASES.update({f"heads of {d} {b:g}": biased(70, 200, 3, 1, d, b, "all")
              for d in (16, 32, 33, 40, 96, 128) for b in (-1e8, -1e9, -1e10, -1e29, 1e10)})
# the first rows see biased keys alone, later ones of the same tile ordinary keys too
CASES.update({f"{lq}x{lk} {b:g} behind padding": biased(lq, lk, 4, 2, 64, b, "leading", True)
              for lq, lk in ((260, 260), (1500, 1500), (5, 3000)) for b in (-1e5, -1e9, -1e10, -1e30, 1e9)})
CASES.update({f"{lq}x{lk} in parts": biased(lq, lk, 4, 2, 64, -1e8, "all") for lq, lk in ((1500, 1500), (2000, 40))})
CASES.update({f"{lq}x{lk} products of {d}{' causal' * c}": large(lq, lk, d, c)
              for lq, lk in ((150, 300), (4, 4000), (1100, 1100)) for d in (16, 64) for c in (False, True)})


@TYPES
@pytest.mark.parametrize("name", list(CASES))
def test_values(sdc, name, dtype):
    q, k, v, go, bias, causal = CASES[name](dtype)
    got = sdc.attention_fwd(q, k, v, key_bias=bias, causal=causal)
    check(got, reference(q, k, v, bias, causal, q.shape[2] ** -0.5, go))


def masked(lq, lk, hidden, dtype):
    """(q, k, v, go, bias): every row has ordinary keys; the others are for a mask"""
    q, k, v, go = inputs(6, lq, lk, 4, 2, 64, dtype)
    q, k = (torch.randn(t.shape, generator=gen(7), device="cuda").to(dtype) for t in (q, k))
    return q, k, v, go, torch.rand(lk, generator=gen(8), device="cuda").log()


HIDDEN = [(150, 300, slice(0, 40)), (150, 300, slice(0, 128)), (150, 300, slice(128, 256)), (150, 300, slice(200, 300)),
          (3, 5000, slice(0, 4000)), (3, 5000, slice(700, 5000))]


@TYPES
@pytest.mark.parametrize("b", [-1e4, -1e9, -1e10, -1e20, -1e30])
@pytest.mark.parametrize("lq,lk,hidden", HIDDEN)
def test_a_finite_mask_is_a_mask(sdc, lq, lk, hidden, b, dtype):
    # the same bits as with -inf
    q, k, v, go, bias = masked(lq, lk, hidden, dtype)
    bias[hidden] = b
    got = sdc.attention_fwd(q, k, v, key_bias=bias)
    bias[hidden] = -INF
    assert all(torch.equal(a, c) for a, c in zip(got, sdc.attention_fwd(q, k, v, key_bias=bias)))


def padded(dtype):
    """Three packed sequences, the keys of the second all carry the mask."""
    cu = torch.tensor([0, 90, 230, 300], dtype=torch.int32, device="cuda")
    bias = torch.zeros(300, device="cuda")
    bias[90:230] = -1e9
    return inputs(12, 300, 300, 4, 2, 64, dtype, unit(-1e9)) + (bias, cu)


@TYPES
def test_one_sequence_of_padding_among_others(sdc, dtype):
    q, k, v, go, bias, cu = padded(dtype)
    got = sdc.attention_fwd(q, k, v, key_bias=bias, cu_q=cu, cu_k=cu)
    for at in (slice(0, 90), slice(90, 230), slice(230, 300)):
        check([t[at] for t in got], reference(q[at], k[at], v[at], bias[at], False, 0.125, go[at]))
