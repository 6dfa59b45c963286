"""Calls on two streams at once, and calls whose results or inputs are let go of
at once, against the same calls one after another: equal bits."""
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


def randn(seed, shape, dtype=F32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def check(got, want):
    assert all(torch.equal(a, b) for a, b in zip(got, want) if a is not None)


def test_scratch_of_two_streams(sdc):
    # the same sizes on both streams, inputs ready beforehand, no order between them
    x = [randn(k, (2, 64, 181, 360), BF16) for k in range(2)]
    gy = [randn(5 + k, (2, 64, 181, 360), BF16) for k in range(2)]
    m = [randn(10 + k, (600, 900)) for k in range(2)]
    fwd = [sdc.layer_norm_fwd(v) for v in x]
    want = [sdc.layer_norm_bwd(x[k], gy[k], fwd[k][2], fwd[k][3]) for k in range(2)]
    owant = [sdc.orthogonalize(v) for v in m]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a = [sdc.layer_norm_bwd(x[k], gy[k], fwd[k][2], fwd[k][3], stream=side if k else None) for k in range(2)]
        b = [sdc.orthogonalize(m[k], stream=side if k else None) for k in range(2)]
        torch.cuda.synchronize()
        for k in range(2):
            check(a[k], want[k])
            check([b[k]], [owant[k]])


def test_results_and_inputs_let_go_of(sdc):
    shape = (1, 64, 181, 360)
    x, res = randn(1, shape), randn(2, shape)
    y, s, mean, rstd = sdc.layer_norm_fwd(x, residual=res)
    m = randn(3, (700, 700))
    o = sdc.orthogonalize(m)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        xs, ms = x.clone(), m.clone()
        side.wait_stream(torch.cuda.current_stream())
        got = sdc.layer_norm_fwd(xs, residual=res, stream=side)[0]
        oo = sdc.orthogonalize(ms, stream=side)
        del xs, ms
        # memory of every size that was just let go of, written on the current stream
        fills = [torch.full_like(t, 7.0) for t in (x, s, mean, rstd, m)]
        torch.cuda.synchronize()
        check([got, oo], [y, o])
        assert all(bool((t == 7.0).all()) for t in fills)


def test_a_graph_with_a_branch(sdc):
    x, m = randn(1, (2, 32, 65, 128)), randn(2, (300, 400))
    y, o = sdc.layer_norm_fwd(x)[0], sdc.orthogonalize(m)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        oo = sdc.orthogonalize(m, stream=side)
        yy = sdc.layer_norm_fwd(x)[0]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(4):
        oo.zero_()
        yy.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check([yy, oo], [y, o])
        _ = float(yy.abs().max())
