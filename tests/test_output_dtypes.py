"""A result tensor and an out_dtype that contradicts it are refused, not taken
one over the other.  No GPU: the refusal comes before any device work."""
import pytest

import spherical_disco_convolution_amd as sdc

torch = pytest.importorskip("torch")

F32, BF16 = torch.float32, torch.bfloat16


def test_layer_norm_refuses_a_contradicting_dtype():
    x = torch.zeros(2, 4, 5, 6)
    for y, dt in ((torch.zeros_like(x), BF16), (torch.zeros_like(x, dtype=BF16), F32)):
        with pytest.raises(ValueError, match="out_dtype"):
            sdc.layer_norm_fwd(x, y=y, out_dtype=dt)


def test_orthogonalize_refuses_a_contradicting_dtype():
    m = torch.zeros(4, 5)
    for o, dt in ((torch.zeros_like(m), BF16), (torch.zeros_like(m, dtype=BF16), F32)):
        with pytest.raises(ValueError, match="out_dtype"):
            sdc.orthogonalize(m, out=o, out_dtype=dt)
