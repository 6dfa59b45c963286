"""Gradients of attention under large finite biases and scores: the cases, the formulas
and the bounds of test_attention_far_scores_gpu."""
import pytest

torch = pytest.importorskip("torch")
from attention_reference import BF16, half_step  # noqa: E402
from test_attention_far_scores_gpu import (CASES, HIDDEN, INF, TYPES, U, check, gen, inputs, masked,  # noqa: E402
                                           padded, reference, sdc)  # noqa: F401

pytestmark = pytest.mark.gpu


def run(sdc, q, k, v, go, bias, causal=False, **kw):  # noqa: F811
    o, lse = sdc.attention_fwd(q, k, v, key_bias=bias, causal=causal)
    return (o, lse) + sdc.attention_bwd(q, k, v, o, lse, go, key_bias=bias, causal=causal, **kw)


@TYPES
@pytest.mark.parametrize("name", list(CASES))
def test_values(sdc, name, dtype):  # noqa: F811
    q, k, v, go, bias, causal = CASES[name](dtype)
    got = run(sdc, q, k, v, go, bias, causal)
    check(got, reference(q, k, v, bias, causal, q.shape[2] ** -0.5, go))


@TYPES
@pytest.mark.parametrize("name", ["1500x1500 in parts", "3x5000 -1e+09 all", "1500x1500 -1e+09 behind padding"])
def test_gradients_skipped(sdc, name, dtype):  # noqa: F811
    case = CASES[name](dtype)
    got = run(sdc, *case)
    alone = run(sdc, *case, need_gq=False)
    assert torch.equal(alone[3], got[3]) and torch.equal(alone[4], got[4])
    assert torch.equal(run(sdc, *case, need_gkv=False)[2], got[2])


@TYPES
@pytest.mark.parametrize("b", [-1e4, -1e9, -1e10, -1e20, -1e30])
@pytest.mark.parametrize("lq,lk,hidden", HIDDEN)
def test_a_finite_mask_is_a_mask(sdc, lq, lk, hidden, b, dtype):  # noqa: F811
    q, k, v, go, bias = masked(lq, lk, hidden, dtype)
    bias[hidden] = b
    got = run(sdc, q, k, v, go, bias)
    bias[hidden] = -INF
    assert all(torch.equal(a, c) for a, c in zip(got, run(sdc, q, k, v, go, bias)))


@TYPES
@pytest.mark.parametrize("b", [-1e6, -1e7, -1e8, -1e9, -1e12, 1e8])
@pytest.mark.parametrize("lq,lk", [(150, 300), (900, 900), (3, 5000)])
def test_weights_of_any_scores_add_up(sdc, lq, lk, b, dtype):  # noqa: F811
    # scores that round: whichever they are, a row's weights sum to 1 and its ds to 0, in
    # the gradient too.  Each weight is off by dw, and in bfloat16 by half a step.
    q, k, v, go = inputs(9, lq, lk, 4, 2, 64, dtype)
    q, k = (torch.randn(t.shape, generator=gen(10 + i), device="cuda").to(dtype) for i, t in enumerate((q, k)))
    bias = torch.full((lk,), b, device="cuda")
    o, lse, gq, gk, gv = (t.double().cpu() for t in run(sdc, q, k, v, go, bias))
    q, k, v, go = (t.double().cpu() for t in (q, k, v, go))
    half = half_step(dtype)
    low = half if dtype == BF16 else 0.0
    dw = (4 * lq + lk + 16) * U + 16 * U * 128
    assert bool((o.amax(0) <= v.amax() * 1.01).all()) and bool((o.amin(0) >= v.amin() * 1.01).all())
    assert float((lse - b).abs().max()) <= 6 * U * abs(b) + 40
    groups = go.view(lq, 2, 2, 64)
    bound = (dw + low + half) * groups.abs().sum((0, 2)) + half * gv.abs().sum(0)
    assert bool(((gv.sum(0) - groups.sum((0, 2))).abs() <= bound).all())
    most = 2 * go.abs().sum(2).max() * v.abs().max()      # of dp and delta
    bound = 0.125 * (4 * dw + 3 * low + 2 * half + 64 * U) * most * q.abs().view(lq, 2, 2, 64).sum((0, 2))
    assert bool((gk.sum(0).abs() <= bound + half * gk.abs().sum(0)).all())


@TYPES
def test_one_sequence_of_padding_among_others(sdc, dtype):  # noqa: F811
    q, k, v, go, bias, cu = padded(dtype)
    o, lse = sdc.attention_fwd(q, k, v, key_bias=bias, cu_q=cu, cu_k=cu)
    got = (o, lse) + sdc.attention_bwd(q, k, v, o, lse, go, key_bias=bias, cu_q=cu, cu_k=cu)
    for at in (slice(0, 90), slice(90, 230), slice(230, 300)):
        check([t[at] for t in got], reference(q[at], k[at], v[at], bias[at], False, 0.125, go[at]))


def test_in_a_graph(sdc):  # noqa: F811
    case = CASES["260x260 -1e+09 behind padding"](BF16)
    want = run(sdc, *case)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(sdc, *case)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        _ = run(sdc, *case)
