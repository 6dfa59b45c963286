"""Attention forward and backward on the GPU against float64 formulas, with the
bounds of attention_reference: lengths from none to thousands, head layouts, types,
strides, masks that leave rows empty, and what lies where nothing may be read."""
import itertools
import math

import pytest

torch = pytest.importorskip("torch")
from attention_reference import BF16, F32, attention, check  # noqa: E402

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


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


def randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def cu_of(lens):
    return list(itertools.accumulate(lens, initial=0))


def dev(cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def run(sdc, q, k, v, go, bias=None, cu_q=None, cu_k=None, causal=False, scale=None, **kw):
    """Forward and backward, checked; returns (o, lse, gq, gk, gv)."""
    lists = [list(range(0, n + 1, n)) if cu is None else cu for cu, n in ((cu_q, max(q.shape[0], 1)), (cu_k, max(k.shape[0], 1)))]
    opt = dict(key_bias=bias, cu_q=None if cu_q is None else dev(cu_q), cu_k=None if cu_k is None else dev(cu_k),
               causal=causal, scale=scale)
    o, lse = sdc.attention_fwd(q, k, v, **opt, **{n: t for n, t in kw.items() if n == "out"})
    s = q.shape[-1] ** -0.5 if scale is None else scale
    gq, gk, gv = sdc.attention_bwd(q, k, v, o, lse, go, **opt, **{n: t for n, t in kw.items() if n != "out"})
    torch.cuda.synchronize()
    want = attention(q, k, v, bias, *lists, causal, s, go, o, lse, dtype=q.dtype)
    got = dict(o=o, lse=lse, gq=gq, gk=gk, gv=gv)
    for n, t in got.items():
        check(n, t, *want[n])
    return o, lse, gq, gk, gv


def inputs(seed, tq, tk, hq, hkv, dk, dv, dtype, spread=1.0):
    g = gen(seed)
    return (spread * randn(g, (tq, hq, dk), F32)).to(dtype), randn(g, (tk, hkv, dk), dtype), \
        randn(g, (tk, hkv, dv), dtype), randn(g, (tq, hq, dv), dtype)


# (queries, keys) of one sequence: ends and middles of tiles, one, few rows over many keys, many over few
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("lq,lk", [(1, 1), (1, 64), (3, 65), (31, 63), (33, 129), (128, 128), (129, 200), (257, 191),
                                   (1, 3001), (7, 4097), (2500, 5), (300, 1)])
def test_lengths(sdc, lq, lk, dtype):
    q, k, v, go = inputs(lq * 7 + lk, lq, lk, 4, 2, 64, 64, dtype)
    run(sdc, q, k, v, go)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dk,dv", [(1, 1), (8, 8), (16, 32), (24, 24), (32, 32), (33, 20), (40, 72), (64, 64), (65, 65),
                                   (80, 80), (96, 96), (100, 128), (127, 127), (128, 16), (128, 128)])
def test_head_sizes(sdc, dk, dv, dtype, causal):
    q, k, v, go = inputs(dk + dv, 150, 170, 3, 1, dk, dv, dtype)
    run(sdc, q, k, v, go, causal=causal)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 2), (6, 3), (8, 1), (5, 1), (16, 8), (12, 4), (24, 8), (33, 11), (70, 1)])
def test_heads(sdc, hq, hkv, dtype):
    q, k, v, go = inputs(hq, 45, 77, hq, hkv, 32, 32, dtype)
    run(sdc, q, k, v, go, causal=True)


PACKED = {
    "mixed": ([5, 1, 0, 130, 64, 65, 0, 200], [5, 1, 0, 130, 64, 65, 0, 200]),
    "no keys": ([5, 3, 70], [64, 0, 9]),
    "no queries": ([0, 0, 4], [70, 3, 0]),
    "longer queries": ([200, 65, 300], [100, 1, 299]),
    "longer keys": ([1, 2, 17], [900, 64, 333]),
    "many short": ([1, 2, 3] * 40, [1, 2, 3] * 40),
}


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("name", list(PACKED))
def test_packed(sdc, name, causal, dtype):
    cu_q, cu_k = (cu_of(x) for x in PACKED[name])
    q, k, v, go = inputs(3, cu_q[-1], cu_k[-1], 6, 2, 64, 64, dtype)
    run(sdc, q, k, v, go, cu_q=cu_q, cu_k=cu_k, causal=causal)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_tokens_of_no_sequence(sdc, dtype):
    # 7 tokens before the first sequence and 20 behind the last: not read, left as they were
    cu = [7, 40, 40, 140]
    q, k, v, go = inputs(5, 160, 160, 4, 2, 64, 64, dtype)
    for t in (q, k, v, go):
        t[:7], t[140:] = NAN, NAN
    out, gq, gk, gv = (torch.full_like(t, 5.0) for t in (go, q, k, v))
    run(sdc, q, k, v, go, cu_q=cu, cu_k=cu, causal=True, out=out, gq=gq, gk=gk, gv=gv)
    for t in (out, gq, gk, gv):
        assert bool((t[:7] == 5.0).all()) and bool((t[140:] == 5.0).all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("lq", [3, 200])
def test_boundaries_out_of_order(sdc, lq, dtype):
    # cut to what the tensors hold: no access outside, no claim on the values
    q, k, v, go = inputs(6, lq, 900, 4, 2, 64, 64, dtype)
    for cu_q, cu_k in (([0, 10 ** 9], [-5, 10 ** 9]), ([-100, lq, 2], [900, 0, 10 ** 9]), ([5, 1, 0], [3, 2, 1]),
                       ([lq, lq, lq], [900, 900, 900])):
        o, lse = sdc.attention_fwd(q, k, v, cu_q=dev(cu_q), cu_k=dev(cu_k))
        sdc.attention_bwd(q, k, v, o, lse, go, cu_q=dev(cu_q), cu_k=dev(cu_k), causal=True)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_neighbours_stay_out(sdc, dtype):
    # the second sequence holds NaN; the first and third are those of a call of their own
    cu = [0, 50, 90, 190]
    q, k, v, go = inputs(7, 190, 190, 4, 2, 32, 32, dtype)
    clean = run(sdc, q, k, v, go, cu_q=cu, cu_k=cu)
    for t in (q, k, v, go):
        t[50:90] = NAN
    o, lse = sdc.attention_fwd(q, k, v, cu_q=dev(cu), cu_k=dev(cu))
    got = (o, lse) + sdc.attention_bwd(q, k, v, o, lse, go, cu_q=dev(cu), cu_k=dev(cu))
    for a, b in zip(got, clean):
        assert torch.equal(a[:50], b[:50]) and torch.equal(a[90:], b[90:])
        assert bool(a[50:90].isnan().all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("lq", [3, 150])
@pytest.mark.parametrize("low", [-INF, torch.finfo(F32).min, -1e31])
def test_keys_left_out(sdc, low, lq, dtype):
    q, k, v, go = inputs(8, lq, 1000, 4, 2, 64, 64, dtype)
    bias = torch.rand(1000, generator=gen(9), device="cuda").log()
    out = torch.rand(1000, generator=gen(10), device="cuda") < 0.3
    out[128:320] = True     # whole tiles
    bias[out] = low
    clean = run(sdc, q, k, v, go, bias=bias)
    k[out], v[out] = NAN, INF
    got = run(sdc, q, k, v, go, bias=bias)
    for a, b in zip(got, clean):
        assert torch.equal(a, b)
    assert not bool(got[3][out].any()) and not bool(got[4][out].any())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("lq", [1, 140])
def test_rows_that_see_nothing(sdc, lq, dtype):
    q, k, v, go = inputs(11, lq, 300, 4, 4, 32, 32, dtype)
    o, lse, gq, gk, gv = run(sdc, q, k, v, go, bias=torch.full((300,), -INF, device="cuda"))
    assert bool((lse == -INF).all())
    assert not any(bool(t.any()) for t in (o, gq, gk, gv))
    # a causal first row whose only key is left out
    bias = torch.zeros(300, device="cuda")
    bias[:300 - lq + 1] = -INF
    o, lse, gq, gk, gv = run(sdc, q, k, v, go, bias=bias, causal=True)
    assert bool((lse[0] == -INF).all()) and not bool(o[0].any())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_nan_stays_in_its_row(sdc, dtype):
    q, k, v, go = inputs(12, 100, 100, 2, 1, 64, 64, dtype)
    clean = run(sdc, q, k, v, go)
    q[17, 1, 3] = NAN
    o, lse = sdc.attention_fwd(q, k, v)
    assert bool(o[17, 1].isnan().all()) and bool(lse[17, 1].isnan())
    for a, b in ((o, clean[0]), (lse, clean[1])):
        a[17, 1] = b[17, 1]
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_scores_of_every_size(sdc, dtype):
    # growing scores make each tile's maximum a new one; falling ones leave it behind
    for sign in (1.0, -1.0):
        q, k, v, go = inputs(13, 130, 700, 2, 2, 32, 32, dtype)
        k = (k.float() + sign * torch.linspace(0, 6, 700, device="cuda")[:, None, None] * q[:1].float().mean(0)).to(dtype)
        run(sdc, (4 * q.float()).to(dtype), k, v, go, scale=0.5)
    # all scores far below zero, and far above
    bias = torch.full((700,), -30000.0, device="cuda")
    run(sdc, q, k, v, go, bias=bias)
    run(sdc, q, k, v, go, bias=-bias)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_large_values_under_growing_scores(sdc, dtype):
    # each tile's scores are larger than the last one's, by 2^9 a tile in the weights
    q, k, v, go = inputs(25, 70, 900, 2, 2, 32, 32, dtype)
    bias = torch.linspace(0, 100, 900, device="cuda")
    v = (1e25 * v.float()).to(dtype)
    opt = dict(key_bias=bias)
    o, lse = sdc.attention_fwd(q, k, v, **opt)
    want = attention(q, k, v, bias, [0, 70], [0, 900], False, 32 ** -0.5, dtype=dtype)
    check("o", o, *want["o"])
    check("lse", lse, *want["lse"])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("off", [0, 1, 3])
def test_columns_of_one_buffer(sdc, off, dtype):
    # q, k, v side by side in a projection's output, gradients side by side too; odd starts
    hq, hkv, d, t = 6, 2, 32, 170
    width = (hq + 2 * hkv) * d + 8
    g = gen(14)
    buf = randn(g, (t, width), dtype)
    gbuf = torch.full((t, width), 7.0, dtype=dtype, device="cuda")

    def parts(b):
        return (b[:, off:off + hq * d].unflatten(1, (hq, d)), b[:, off + hq * d:off + (hq + hkv) * d].unflatten(1, (hkv, d)),
                b[:, off + (hq + hkv) * d:off + (hq + 2 * hkv) * d].unflatten(1, (hkv, d)))

    q, k, v = parts(buf)
    go = randn(g, (t, hq, d), dtype)
    gq, gk, gv = parts(gbuf)
    run(sdc, q, k, v, go, causal=True, gq=gq, gk=gk, gv=gv)
    assert bool((gbuf[:, :off] == 7.0).all()) and bool((gbuf[:, off + (hq + 2 * hkv) * d:] == 7.0).all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_heads_first(sdc, dtype):
    g = gen(15)
    q, k, v, go = (randn(g, (h, t, 64), dtype).transpose(0, 1) for h, t in ((4, 90), (2, 150), (2, 150), (4, 90)))
    out = torch.zeros((4, 90, 64), dtype=dtype, device="cuda").transpose(0, 1)
    gk = torch.zeros((2, 150, 64), dtype=dtype, device="cuda").transpose(0, 1)
    run(sdc, q, k, v, go, out=out, gk=gk)
    # one key head for all, by a stride of zero
    k1, v1 = (t[:, :1].expand(150, 2, 64) for t in (k, v))
    run(sdc, q, k1, v1, go)


# causal: tiles of few and of many steps, in parts
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("lq,lk", [(1, 1), (1, 3001), (5, 5000), (700, 2900), (1500, 1500), (2500, 5), (2500, 1)])
def test_causal_lengths(sdc, lq, lk, dtype):
    q, k, v, go = inputs(lq * 5 + lk, lq, lk, 4, 2, 64, 64, dtype)
    run(sdc, q, k, v, go, causal=True)


# 64 sequences are counted, more are searched; causal tiles go by their steps
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,causal", [(63, True), (64, True), (65, True), (64, False), (300, True), (300, False)])
def test_many_sequences(sdc, n, causal, dtype):
    r = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 60, (2, n), generator=r) * (torch.rand(2, n, generator=r) < 0.8)
    lens[:, 2] = 300
    cu_q, cu_k = ([0] + x.cumsum(0).tolist() for x in lens)
    q, k, v, go = inputs(n, cu_q[-1], cu_k[-1], 3, 1, 32, 32, dtype)
    run(sdc, q, k, v, go, cu_q=cu_q, cu_k=cu_k, causal=causal)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("b,t,s", [(3, 77, 131), (40, 130, 130)])
def test_a_batch_is_its_sequences(sdc, b, t, s, dtype):
    # with boundaries the sums may be cut up for sequences of other lengths, so that each
    # of the two is held against the formula, not against the other's bits
    q, k, v, go = inputs(16, b * t, b * s, 4, 2, 64, 64, dtype)
    bias = torch.rand(b * s, generator=gen(17), device="cuda")
    cu_q, cu_k = list(range(0, b * t + 1, t)), list(range(0, b * s + 1, s))
    run(sdc, q, k, v, go, bias=bias, cu_q=cu_q, cu_k=cu_k)
    q4, k4, v4, go4 = (x.unflatten(0, (b, -1)) for x in (q, k, v, go))
    o, lse = sdc.attention_fwd(q4, k4, v4, key_bias=bias.view(b, s))
    got = (o, lse) + sdc.attention_bwd(q4, k4, v4, o, lse, go4, key_bias=bias)
    want = attention(q, k, v, bias, cu_q, cu_k, False, 64 ** -0.5, go, o.flatten(0, 1), lse.flatten(0, 1), dtype=dtype)
    for n, x in zip(("o", "lse", "gq", "gk", "gv"), got):
        check(n, x.flatten(0, 1), *want[n])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_the_same_bits_again(sdc, dtype):
    for lq, lk in ((300, 300), (5, 6000), (6000, 70)):
        q, k, v, go = inputs(18, lq, lk, 4, 1, 64, 64, dtype)
        runs = []
        for _ in range(2):
            o, lse = sdc.attention_fwd(q, k, v)
            runs.append((o, lse) + sdc.attention_bwd(q, k, v, o, lse, go))
        assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_gradients_skipped(sdc):
    q, k, v, go = inputs(19, 100, 120, 2, 2, 32, 32, BF16)
    o, lse = sdc.attention_fwd(q, k, v)
    gq, gk, gv = sdc.attention_bwd(q, k, v, o, lse, go)
    a = sdc.attention_bwd(q, k, v, o, lse, go, need_gkv=False)
    b = sdc.attention_bwd(q, k, v, o, lse, go, need_gq=False)
    assert a[1] is None and a[2] is None and b[0] is None
    assert torch.equal(a[0], gq) and torch.equal(b[1], gk) and torch.equal(b[2], gv)
    o2, none = sdc.attention_fwd(q, k, v, need_lse=False)
    assert none is None and torch.equal(o2, o)


def test_empty_tensors(sdc):
    for tq, tk in ((0, 5), (5, 0), (0, 0)):
        q, k, v, go = inputs(20, tq, tk, 4, 2, 32, 32, BF16)
        o, lse = sdc.attention_fwd(q, k, v)
        gq, gk, gv = sdc.attention_bwd(q, k, v, o, lse, go)
        torch.cuda.synchronize()
        assert not any(bool(t.any()) for t in (o, gq, gk, gv)) and bool((lse == -INF).all())


def test_gradients_follow_differences(sdc):
    # float32, a loss of sum(go * o) along random directions.  Central differences
    # with step h are off by h^2/6 times the third derivative (of order 1 for
    # unit-size directions) and by the loss's rounding over h: 1e-4 + 1e-7 * 40 / 1e-2
    # of a derivative of order 1..10.
    q, k, v, go = (t.double() for t in inputs(21, 40, 50, 4, 2, 16, 16, F32))
    h = 1e-2

    def loss(q, k, v):
        return float((sdc.attention_fwd(q.float(), k.float(), v.float(), causal=True)[0].double() * go).sum())

    o, lse = sdc.attention_fwd(q.float(), k.float(), v.float(), causal=True)
    grads = sdc.attention_bwd(q.float(), k.float(), v.float(), o, lse, go.float(), causal=True)
    for i, t in enumerate((q, k, v)):
        d = randn(gen(30 + i), t.shape, F32).double()
        d /= d.norm()
        a = [q, k, v]
        a[i] = t + h * d
        up = loss(*a)
        a[i] = t - h * d
        down = loss(*a)
        want = float((grads[i].double() * d).sum())
        assert abs((up - down) / (2 * h) - want) <= 2e-3 * max(1.0, abs(want))


@pytest.mark.parametrize("lq,lk", [(200, 200), (6, 5000)])
def test_graph_replays(sdc, lq, lk):
    q, k, v, go = inputs(22, lq, lk, 4, 2, 64, 64, BF16)

    def step():
        o, lse = sdc.attention_fwd(q, k, v)
        return (o, lse) + sdc.attention_bwd(q, k, v, o, lse, go)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.cuda.graph(second):
        again = step()
    for _ in range(3):
        for g, r in ((graph, got), (second, again)):
            for t in r:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(r, want))
            _ = float(step()[0].float().abs().sum())


def test_two_streams_at_once(sdc):
    sets = [inputs(23 + i, 500 if i else 9, 4000, 4, 2, 64, 64, BF16) for i in range(2)]
    want = []
    for q, k, v, go in sets:
        o, lse = sdc.attention_fwd(q, k, v)
        want.append((o, lse) + sdc.attention_bwd(q, k, v, o, lse, go))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for i, (q, k, v, go) in enumerate(sets):
            s = side if i else None
            o, lse = sdc.attention_fwd(q, k, v, stream=s)
            got.append((o, lse) + sdc.attention_bwd(q, k, v, o, lse, go, stream=s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_far_rows(sdc, dtype):
    # tokens 2^23 elements apart: offsets past 2^31 elements
    t, ts = 300, 1 << 23
    small = inputs(24, t, t, 2, 2, 32, 32, dtype)
    big = torch.empty(t * ts, dtype=dtype, device="cuda").view(t, ts)
    wide = []
    for i, x in enumerate(small):
        view = big[:, 128 * i:128 * i + 64].unflatten(1, (2, 32))
        view.copy_(x)
        wide.append(view)
    out = big[:, 1024:1088].unflatten(1, (2, 32))
    gq, gk, gv = (big[:, 2048 + 64 * i:2112 + 64 * i].unflatten(1, (2, 32)) for i in range(3))
    q, k, v, go = wide
    o, lse = sdc.attention_fwd(q, k, v, causal=True, out=out)
    got = (o, lse) + sdc.attention_bwd(q, k, v, o, lse, go, causal=True, gq=gq, gk=gk, gv=gv)
    o, lse = sdc.attention_fwd(*small[:3], causal=True)
    want = (o, lse) + sdc.attention_bwd(*small[:3], o, lse, small[3], causal=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_host_memory_is_refused(sdc):
    q, k, v, go = inputs(3, 20, 30, 2, 2, 32, 32, F32)
    cu_q, cu_k, bias = dev([0, 20]), dev([0, 30]), torch.zeros(30, device="cuda")
    o, lse = sdc.attention_fwd(q, k, v, bias, cu_q, cu_k)
    calls = [lambda: sdc.attention_fwd(q, k, v, bias, cu_q.cpu(), cu_k),
             lambda: sdc.attention_fwd(q, k, v, bias, cu_q, cu_k.cpu()),
             lambda: sdc.attention_fwd(q, k, v, bias.cpu(), cu_q, cu_k),
             lambda: sdc.attention_fwd(q, k.cpu(), v, bias, cu_q, cu_k),
             lambda: sdc.attention_bwd(q, k, v, o, lse.cpu(), go, bias, cu_q, cu_k),
             lambda: sdc.attention_bwd(q, k, v, o, lse, go.cpu(), bias, cu_q, cu_k),
             lambda: sdc.qk_norm_rope_fwd(q, q, positions=torch.zeros(20, dtype=torch.int32),
                                          inv_freq=torch.ones(16, device="cuda")),
             lambda: sdc.qk_norm_rope_fwd(q, q, torch.ones(32)),
             lambda: sdc.dropout_fwd(q, 0.5, 1, step=torch.zeros(1, dtype=torch.int64))]
    for call in calls:
        with pytest.raises(ValueError, match="device"):
            call()
    torch.cuda.synchronize()
