"""Sizes at the ends of 32 bits: refused before any device work, in the C entry
points and in the binding, which hands them over as 32-bit integers.  No GPU."""
import ctypes

import pytest

import spherical_disco_convolution_amd as sdc

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("rows,cols", [(1, TOP), (TOP, 1), (40, TOP), (1, TOP - 30), (TOP - 62, 3)])
def test_orthogonalize_refuses_sides_that_do_not_round_up(rows, cols):
    # sides are rounded up to 64 in 32 bits
    lib, fake = sdc._lib, ctypes.c_void_p(0x1000)
    assert lib.disco_orthogonalize_workspace(1, rows, cols) == sdc.DISCO_EUNSUPPORTED
    assert "2147483584" in lib.disco_last_error().decode()
    assert lib.disco_orthogonalize(fake, 1, fake, 1, 1, rows, cols, 5, None, 1e-7, fake, 1 << 60,
                                   None) == sdc.DISCO_EUNSUPPORTED
    assert lib.disco_muon_step(fake, 1, fake, fake, fake, 1, fake, None, 0.1, 0.9, 1, 0.0, 1.0, 1, rows, cols, 5, None,
                               1e-7, fake, 1 << 60, None) == sdc.DISCO_EUNSUPPORTED


def test_orthogonalize_takes_the_largest_side():
    # six planes of 64 rows, float16
    assert sdc._lib.disco_orthogonalize_workspace(1, 1, TOP - 63) >= 6 * 2 * 64 * (TOP - 63)


@pytest.mark.parametrize("C", [TOP, TOP - 1023, 2 ** 30 + 1])
@pytest.mark.parametrize("inner", [1, 2])
def test_layer_norm_refuses_channel_counts_that_leave_no_room_to_stride(C, inner):
    # a lane's next channel is up to 2^16 further on, in 32 bits
    lib, fake = sdc._lib, ctypes.c_void_p(0x1000)
    assert lib.disco_layer_norm_bwd_workspace(1, C, inner) == sdc.DISCO_EUNSUPPORTED
    assert "1073741824" in lib.disco_last_error().decode()
    assert lib.disco_layer_norm_fwd(fake, 1, None, None, None, fake, 1, None, None, None, 1, C, inner, 1e-5,
                                    None) == sdc.DISCO_EUNSUPPORTED
    assert lib.disco_layer_norm_bwd(fake, 1, fake, 1, fake, fake, None, None, fake, 1, None, None, None, 0, 1, C,
                                    inner, None) == sdc.DISCO_EUNSUPPORTED
    assert lib.disco_layer_norm_bwd_workspace(1, 2 ** 30, inner) > 0


def test_binding_refuses_what_32_bits_would_cut_off():
    torch = pytest.importorskip("torch")
    n = 2 ** 32 + 8   # 8 in 32 bits; the memory is never touched
    big = torch.empty((1, n), dtype=torch.bfloat16)
    f32 = torch.empty((1, n))
    stat = torch.zeros(1)
    for call in (lambda: sdc.layer_norm_fwd(big, axis=-1, need_stats=False, y=big),
                 lambda: sdc.layer_norm_bwd(big, big, stat, stat, axis=-1, need_gparams=False),
                 lambda: sdc.orthogonalize(big, out=big),
                 lambda: sdc.orthogonalize(big.view(n, 1), out=big.view(n, 1)),
                 lambda: sdc.orthogonalize(big.view(n, 1, 1), out=big.view(n, 1, 1)),
                 lambda: sdc.muon_step(big, big, f32, 0.1),
                 lambda: sdc.muon_step(big.view(n, 1), big.view(n, 1), f32.view(n, 1), 0.1, groups=n),
                 lambda: sdc.orthogonalize(torch.zeros(4, 5), steps=2 ** 32 + 5)):
        with pytest.raises(NotImplementedError, match="32 bits"):
            call()
