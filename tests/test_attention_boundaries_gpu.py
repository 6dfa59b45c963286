"""Boundaries out of order and out of range: cut to what the tensors hold.  There is no
claim on the values, but nothing around the results is written, and a list in order that
follows gives its usual results.  Up to 64 sequences are counted, more are searched."""
import random

import pytest

torch = pytest.importorskip("torch")
from attention_reference import BF16, F32  # noqa: E402

pytestmark = pytest.mark.gpu
MARK = 5.0


@pytest.fixture(scope="module")
def sdc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import spherical_disco_convolution_amd as m
    return m


def randn(seed, shape, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def lists(n, total):
    """Boundaries of n sequences: at random, falling, all at the end, all past it, in order but for two."""
    r = random.Random(n + total)
    at = sorted(r.randrange(total + 1) for _ in range(n + 1))
    turned = list(at)
    turned[n // 3], turned[n // 2] = turned[n // 2], turned[n // 3]
    return [[r.randrange(-50, total + 50) for _ in range(n + 1)], at[::-1], [total] * (n + 1), [10 ** 9 + i for i in range(n + 1)],
            [-10 ** 9] * n + [10 ** 9], turned]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n,lq,lk", [(1, 3, 900), (2, 200, 900), (64, 700, 650), (65, 700, 650), (300, 500, 2100)])
def test_nothing_around_the_results_is_written(sdc, n, lq, lk, causal, dtype):
    hq, hkv, d, edge = 4, 2, 32, 40
    q, k, v, go = (randn(i, (t, h, d), dtype) for i, (t, h) in enumerate(((lq, hq), (lk, hkv), (lk, hkv), (lq, hq))))
    whole = [torch.full((t + 2 * edge, h, d), MARK, dtype=dtype, device="cuda") for t, h in ((lq, hq), (lq, hq), (lk, hkv), (lk, hkv))]
    out, gq, gk, gv = (w[edge:-edge] for w in whole)
    # the same list in order first and last
    r = random.Random(7)
    cu = [torch.tensor([0] + sorted(r.randrange(t + 1) for _ in range(n - 1)) + [t], dtype=torch.int32, device="cuda")
          for t in (lq, lk)]

    def step(cu_q, cu_k):
        opt = dict(cu_q=cu_q, cu_k=cu_k, causal=causal)
        _, lse = sdc.attention_fwd(q, k, v, out=out, **opt)
        sdc.attention_bwd(q, k, v, out, lse, go, gq=gq, gk=gk, gv=gv, **opt)
        return [t.clone() for t in (out, lse, gq, gk, gv)]

    want = step(*cu)
    for a, b in zip(lists(n, lq), reversed(lists(n, lk))):
        step(*(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (a, b)))
        torch.cuda.synchronize()
        for w in whole:
            assert bool((w[:edge] == MARK).all()) and bool((w[-edge:] == MARK).all())
    assert all(torch.equal(a, b) for a, b in zip(step(*cu), want))
