"""Checks of the layer norm's and the weight update's C entry points that need
no GPU: their argument checks under AddressSanitizer and
UndefinedBehaviorSanitizer (training_api.cpp with stub launchers, driven by
tests/host/training_driver.cpp), and the Python binding's own refusals."""
import ctypes
import os
import shutil
import subprocess

import pytest

import spherical_disco_convolution_amd as sdc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "spherical_disco_convolution_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_argument_checks_are_sanitizer_clean(tmp_path):
    exe = str(tmp_path / "training_driver")
    r = subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                        "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
                        os.path.join(ROOT, "tests", "host", "training_driver.cpp"),
                        os.path.join(CSRC, "training_api.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60,
                       env=dict(os.environ, ASAN_OPTIONS="verify_asan_link_order=0"))
    assert r.returncode == 0 and "training-driver ok" in r.stdout, (r.stdout + r.stderr)[-4000:]


def test_real_library_refuses_before_device_work():
    lib = sdc._lib
    fake = ctypes.c_void_p(0x1000)
    assert lib.disco_layer_norm_fwd(fake, 5, None, None, None, fake, 0, None, None, None, 1, 4, 8, 1e-5,
                                    None) == sdc.DISCO_EINVAL
    assert "dtype" in lib.disco_last_error().decode()
    assert lib.disco_layer_norm_bwd_workspace(4, -1, 8) == sdc.DISCO_EINVAL
    assert lib.disco_layer_norm_bwd_workspace(0, 4, 8) == 0
    assert lib.disco_layer_norm_bwd_workspace(4, 128, 721 * 1440) > 0
    assert lib.disco_orthogonalize_workspace(1, 4, -1) == sdc.DISCO_EINVAL
    assert lib.disco_orthogonalize_workspace(70000, 1, 17) == sdc.DISCO_EUNSUPPORTED
    assert lib.disco_orthogonalize_workspace(256, 1, 17) == 0       # in one workgroup each
    assert lib.disco_orthogonalize_workspace(1, 1000, 3000) > 0
    assert lib.disco_orthogonalize(fake, 0, fake, 0, 1, 8, 8, 99, None, 1e-7, None, 0, None) == sdc.DISCO_EINVAL
    # a workspace grows with the matrix and never falls short of its operands
    last = 0
    for n in (600, 1000, 2000, 4000):
        need = lib.disco_orthogonalize_workspace(1, n, n)
        assert need > last and need >= 10 * n * n
        last = need


def test_binding_refuses_shapes_and_types():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 8, 5, 6)
    with pytest.raises(ValueError):
        sdc.layer_norm_fwd(torch.zeros(8))
    with pytest.raises(ValueError):
        sdc.layer_norm_fwd(x, axis=7)
    with pytest.raises(ValueError):
        sdc.layer_norm_fwd(x, gamma=torch.zeros(7))
    with pytest.raises(ValueError):
        sdc.layer_norm_fwd(x, residual=x.to(torch.bfloat16))
    with pytest.raises(ValueError):
        sdc.layer_norm_bwd(x, x[:1], torch.zeros(2, 5, 6), torch.zeros(2, 5, 6))
    with pytest.raises(ValueError):
        sdc.layer_norm_bwd(x, x, torch.zeros(2, 5, 7), torch.zeros(2, 5, 6))
    with pytest.raises(ValueError):
        sdc.orthogonalize(torch.zeros(3))
    with pytest.raises(ValueError):
        sdc.orthogonalize(torch.zeros(4, 5).T)
    w = torch.zeros(8, 12)
    with pytest.raises(ValueError):
        sdc.muon_step(w, w[:, :6], w, 0.1)
    with pytest.raises(ValueError):
        sdc.muon_step(w, w, w.double(), 0.1)
    with pytest.raises(ValueError):
        sdc.muon_step(w, w, w.clone(), 0.1, groups=5)
