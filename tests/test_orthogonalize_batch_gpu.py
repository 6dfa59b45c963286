"""A matrix has the same bits in a batch of any size as by itself, over shapes
whose batches take other tiles than one matrix does, and whose X X^T is shared
among workgroups along the summed index."""
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


@pytest.mark.parametrize("rows,cols", [(256, 4096), (512, 2048), (512, 4096), (384, 3456), (1024, 4096), (1500, 1100),
                                       (200, 10000), (700, 900)])
def test_bits_do_not_depend_on_the_batch(sdc, rows, cols):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    m = torch.randn((9, rows, cols), generator=g, device="cuda")
    want = [sdc.orthogonalize(v) for v in m]
    for batch in (2, 3, 4, 5, 9):
        o = sdc.orthogonalize(m[:batch].contiguous())
        assert all(torch.equal(o[k], want[k]) for k in range(batch)), batch
        o = sdc.orthogonalize(m[:batch].contiguous(), out_dtype=BF16)
        assert all(torch.equal(o[k], want[k].to(BF16)) for k in range(batch)), batch
    w, buf = torch.randn((9 * rows, cols), generator=g, device="cuda"), torch.zeros((9 * rows, cols), device="cuda")
    sdc.muon_step(w.clone(), m.view(9 * rows, cols), buf, 0.1, groups=9, w_out=w.clone())
    w9 = sdc.muon_step(w, m.view(9 * rows, cols), buf, 0.1, groups=9, w_out=torch.empty_like(w),
                       momentum_out=torch.empty_like(w))[0].view(9, rows, cols)
    w1 = sdc.muon_step(w[:rows].clone(), m[0].clone(), buf[:rows].clone(), 0.1)[0]
    assert torch.equal(w9[0], w1)
