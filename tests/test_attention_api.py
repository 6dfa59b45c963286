"""Checks of the attention's, the query/key norm's and dropout's entry points that
need no GPU: the C calls' argument checks under AddressSanitizer and
UndefinedBehaviorSanitizer (attention_api.cpp with stub launchers, driven by
tests/host/attention_driver.cpp), the real library's and the binding's refusals,
where a call on a stream takes its memory from, and the tests' own generator."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import spherical_disco_convolution_amd as sdc

torch = pytest.importorskip("torch")
import test_streams  # noqa: E402
from attention_reference import philox  # noqa: E402
from test_streams import world  # noqa: E402,F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "spherical_disco_convolution_amd", "csrc")
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_argument_checks_are_sanitizer_clean(tmp_path):
    exe = str(tmp_path / "attention_driver")
    r = subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                        "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
                        os.path.join(ROOT, "tests", "host", "attention_driver.cpp"),
                        os.path.join(CSRC, "attention_api.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60,
                       env=dict(os.environ, ASAN_OPTIONS="verify_asan_link_order=0"))
    assert r.returncode == 0 and "attention-driver ok" in r.stdout, (r.stdout + r.stderr)[-4000:]


def test_the_generator_of_the_tests():
    # the published known answers of Philox4x32 with ten rounds
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
            ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
            ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
             (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        assert tuple(int(w) for w in philox(*(np.uint64(c) for c in counter), *key)) == want


def test_real_library_refuses_before_device_work():
    lib, fake = sdc._lib, ctypes.c_void_p(0x1000)
    d = sdc._AttentionDesc()
    d.total_q, d.total_k, d.n_seq, d.hq, d.hkv, d.dk, d.dv, d.scale = 8, 8, 1, 4, 3, 16, 16, 1.0
    ref = ctypes.byref(d)
    assert lib.disco_attention_fwd_workspace(ref) == sdc.DISCO_EINVAL
    assert "divide" in lib.disco_last_error().decode()
    assert lib.disco_attention_fwd(ref, fake, fake, fake, None, None, None, fake, None, None, 0, None) == sdc.DISCO_EINVAL
    d.hkv, d.dk = 2, 129
    assert lib.disco_attention_bwd_workspace(ref) == sdc.DISCO_EUNSUPPORTED
    d.dk, d.total_q = 16, 2 ** 30
    assert lib.disco_attention_bwd_workspace(ref) == sdc.DISCO_EUNSUPPORTED
    # few rows over many keys need room for their parts, many rows none
    d.total_q, d.total_k = 8, 30000
    assert lib.disco_attention_fwd_workspace(ref) > 0
    d.total_q = 30000
    assert lib.disco_attention_fwd_workspace(ref) == 0
    assert lib.disco_attention_bwd_workspace(ref) >= 30000 * 4 * 4
    assert lib.disco_attention_fwd_workspace(None) == sdc.DISCO_EINVAL
    assert lib.disco_qk_norm_rope_bwd_workspace(257) == sdc.DISCO_EUNSUPPORTED
    assert lib.disco_qk_norm_rope_bwd_workspace(0) == sdc.DISCO_EINVAL
    for p in (-0.1, 1.0, 1.0 - 2.0 ** -18, float("nan"), float("inf")):
        assert lib.disco_dropout_fwd(fake, 0, None, fake, 0, 8, p, 1, 0, None, None) == sdc.DISCO_EINVAL
    assert lib.disco_dropout_fwd(fake, 3, None, fake, 0, 8, 0.1, 1, 0, None, None) == sdc.DISCO_EINVAL
    assert lib.disco_dropout_bwd(fake, 0, fake, 0, -1, 0.1, 1, 0, None, None) == sdc.DISCO_EINVAL
    assert lib.disco_dropout_bwd(fake, 0, fake, 0, 2 ** 40 + 1, 0.1, 1, 0, None, None) == sdc.DISCO_EUNSUPPORTED
    assert lib.disco_dropout_bwd(None, 0, None, 0, 0, 0.1, 1, 0, None, None) == sdc.DISCO_OK


def z(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype)


Q, K = (10, 4, 16), (12, 2, 16)


@pytest.mark.parametrize("what,call", {
    "dimensions": lambda: sdc.attention_fwd(z(10, 64), z(12, 32), z(12, 32)),
    "mixed dimensions": lambda: sdc.attention_fwd(z(1, *Q), z(*K), z(*K)),
    "mixed types": lambda: sdc.attention_fwd(z(*Q), z(*K, dtype=BF16), z(*K)),
    "float16": lambda: sdc.attention_fwd(*(z(*s, dtype=torch.float16) for s in (Q, K, K))),
    "head sizes": lambda: sdc.attention_fwd(z(*Q), z(12, 2, 8), z(*K)),
    "heads": lambda: sdc.attention_fwd(z(*Q), z(12, 3, 16), z(12, 3, 16)),
    "v tokens": lambda: sdc.attention_fwd(z(*Q), z(*K), z(11, 2, 16)),
    "batch sizes": lambda: sdc.attention_fwd(z(2, *Q), z(3, *K), z(3, *K)),
    "batch of views": lambda: sdc.attention_fwd(z(2, 12, 4, 16)[:, :10], z(2, *K), z(2, *K)),
    "strided elements": lambda: sdc.attention_fwd(z(10, 4, 32)[..., ::2], z(*K), z(*K)),
    "bias size": lambda: sdc.attention_fwd(z(*Q), z(*K), z(*K), key_bias=z(10)),
    "bias of a batch turned": lambda: sdc.attention_fwd(z(2, 5, 4, 16), z(2, 6, 2, 16), z(2, 6, 2, 16), key_bias=z(6, 2)),
    "weight of two dimensions": lambda: sdc.qk_norm_rope_fwd(z(*Q), z(10, 2, 16), q_weight=z(4, 4)),
    "bias type": lambda: sdc.attention_fwd(z(*Q), z(*K), z(*K), key_bias=z(12, dtype=BF16)),
    "boundary type": lambda: sdc.attention_fwd(z(*Q), z(*K), z(*K), cu_q=torch.tensor([0, 10])),
    "boundary counts": lambda: sdc.attention_fwd(z(*Q), z(*K), z(*K), cu_q=torch.tensor([0, 10], dtype=torch.int32),
                                                 cu_k=torch.tensor([0, 6, 12], dtype=torch.int32)),
    "unequal shares": lambda: sdc.attention_fwd(z(*Q), z(*K), z(*K), cu_k=torch.tensor([0, 3, 6, 12], dtype=torch.int32)),
    "boundaries of a batch": lambda: sdc.attention_fwd(z(1, *Q), z(1, *K), z(1, *K),
                                                       cu_q=torch.tensor([0, 10], dtype=torch.int32)),
    "scale": lambda: sdc.attention_fwd(z(*Q), z(*K), z(*K), scale=0.0),
    "scale nan": lambda: sdc.attention_fwd(z(*Q), z(*K), z(*K), scale=float("nan")),
    "out shape": lambda: sdc.attention_fwd(z(*Q), z(*K), z(*K), out=z(10, 4, 8)),
    "out type": lambda: sdc.attention_fwd(z(*Q), z(*K), z(*K), out=z(*Q, dtype=BF16)),
    "o shape": lambda: sdc.attention_bwd(z(*Q), z(*K), z(*K), z(9, 4, 16), z(10, 4), z(*Q)),
    "go type": lambda: sdc.attention_bwd(z(*Q), z(*K), z(*K), z(*Q), z(10, 4), z(*Q, dtype=BF16)),
    "lse shape": lambda: sdc.attention_bwd(z(*Q), z(*K), z(*K), z(*Q), z(10, 2), z(*Q)),
    "lse missing": lambda: sdc.attention_bwd(z(*Q), z(*K), z(*K), z(*Q), None, z(*Q)),
    "gq shape": lambda: sdc.attention_bwd(z(*Q), z(*K), z(*K), z(*Q), z(10, 4), z(*Q), gq=z(*K)),
    "nothing": lambda: sdc.attention_bwd(z(*Q), z(*K), z(*K), z(*Q), z(10, 4), z(*Q), need_gq=False, need_gkv=False),
    "qk tokens": lambda: sdc.qk_norm_rope_fwd(z(*Q), z(*K)),
    "qk sizes": lambda: sdc.qk_norm_rope_fwd(z(*Q), z(10, 2, 8)),
    "qk types": lambda: sdc.qk_norm_rope_fwd(z(*Q), z(10, 2, 16, dtype=BF16)),
    "qk weight": lambda: sdc.qk_norm_rope_fwd(z(*Q), z(10, 2, 16), q_weight=z(8)),
    "positions alone": lambda: sdc.qk_norm_rope_fwd(z(*Q), z(10, 2, 16), positions=z(10)),
    "positions type": lambda: sdc.qk_norm_rope_fwd(z(*Q), z(10, 2, 16), positions=torch.zeros(10, dtype=torch.int64),
                                                   inv_freq=z(8)),
    "positions count": lambda: sdc.qk_norm_rope_fwd(z(*Q), z(10, 2, 16), positions=z(9), inv_freq=z(8)),
    "axes": lambda: sdc.qk_norm_rope_fwd(z(*Q), z(10, 2, 16), positions=z(10, 5), inv_freq=z(8)),
    "frequencies": lambda: sdc.qk_norm_rope_fwd(z(*Q), z(10, 2, 16), positions=z(10), inv_freq=z(9)),
    "qk eps": lambda: sdc.qk_norm_rope_fwd(z(*Q), z(10, 2, 16), eps=-1.0),
    "gradient shape": lambda: sdc.qk_norm_rope_bwd(z(*Q), z(10, 2, 16), z(*Q), z(*Q)),
    "p": lambda: sdc.dropout_fwd(z(8), 1.0, 1),
    "p below zero": lambda: sdc.dropout_bwd(z(8), -0.5, 1),
    "seed": lambda: sdc.dropout_fwd(z(8), 0.5, 2 ** 64),
    "offset": lambda: sdc.dropout_fwd(z(8), 0.5, 1, -2 ** 63 - 1),
    "step type": lambda: sdc.dropout_fwd(z(8), 0.5, 1, step=torch.zeros(1, dtype=torch.int32)),
    "step count": lambda: sdc.dropout_fwd(z(8), 0.5, 1, step=torch.zeros(2, dtype=torch.int64)),
    "residual type": lambda: sdc.dropout_fwd(z(8), 0.5, 1, residual=z(8, dtype=BF16)),
    "residual shape": lambda: sdc.dropout_fwd(z(8), 0.5, 1, residual=z(9)),
    "y against out_dtype": lambda: sdc.dropout_fwd(z(8), 0.5, 1, y=z(8), out_dtype=BF16),
    "gx against gx_dtype": lambda: sdc.dropout_bwd(z(8), 0.5, 1, gx=z(8), gx_dtype=BF16),
    "strided x": lambda: sdc.dropout_fwd(z(8, 8).T[:4], 0.5, 1),
}.items(), ids=lambda v: v if isinstance(v, str) else "")
def test_binding_refuses(what, call, monkeypatch):
    monkeypatch.setattr(sdc, "_raw_current_stream", lambda: 0)
    with pytest.raises(ValueError):
        call()


def test_binding_refuses_what_is_not_built(monkeypatch):
    monkeypatch.setattr(sdc, "_raw_current_stream", lambda: 0)
    with pytest.raises(NotImplementedError, match="128"):
        sdc.attention_fwd(z(4, 1, 160), z(4, 1, 160), z(4, 1, 160))
    with pytest.raises(NotImplementedError, match="256"):
        sdc.qk_norm_rope_fwd(z(4, 1, 300), z(4, 1, 300))


# every entry point that takes a stream: a call of its inputs, and the inputs
I32 = torch.int32
CALLS = {
    "attention_fwd": (lambda a, s: sdc.attention_fwd(*a[:3], key_bias=a[3], cu_q=a[4], cu_k=a[5], stream=s),
                      lambda: [z(*Q), z(*K), z(*K), z(12), z(3, dtype=I32), z(3, dtype=I32)]),
    "attention_fwd_out": (lambda a, s: sdc.attention_fwd(*a[:3], out=a[3], need_lse=False, stream=s),
                          lambda: [z(*Q), z(*K), z(*K), z(*Q)]),
    "attention_bwd": (lambda a, s: sdc.attention_bwd(*a, stream=s),
                      lambda: [z(*Q), z(*K), z(*K), z(*Q), z(10, 4), z(*Q)]),
    "attention_bwd_out": (lambda a, s: sdc.attention_bwd(*a[:6], gq=a[6], gk=a[7], gv=a[8], stream=s),
                          lambda: [z(*Q), z(*K), z(*K), z(*Q), z(10, 4), z(*Q), z(*Q), z(*K), z(*K)]),
    "qk_norm_rope_fwd": (lambda a, s: sdc.qk_norm_rope_fwd(*a, stream=s),
                         lambda: [z(*Q), z(10, 2, 16), z(16), z(16), z(10), z(8)]),
    "qk_norm_rope_bwd": (lambda a, s: sdc.qk_norm_rope_bwd(*a, stream=s),
                         lambda: [z(*Q), z(10, 2, 16), z(*Q), z(10, 2, 16), z(16), z(16), z(10), z(8)]),
    "qk_norm_rope_bwd_out": (lambda a, s: sdc.qk_norm_rope_bwd(*a[:4], need_gweights=False, gq=a[4], gk=a[5], stream=s),
                             lambda: [z(*Q), z(10, 2, 16), z(*Q), z(10, 2, 16), z(*Q), z(10, 2, 16)]),
    "dropout_fwd": (lambda a, s: sdc.dropout_fwd(a[0], 0.5, 1, residual=a[1], step=a[2], stream=s),
                    lambda: [z(9), z(9), z(1, dtype=torch.int64)]),
    "dropout_fwd_out": (lambda a, s: sdc.dropout_fwd(a[0], 0.5, 1, y=a[1], stream=s), lambda: [z(9), z(9)]),
    "dropout_bwd": (lambda a, s: sdc.dropout_bwd(a[0], 0.5, 1, stream=s), lambda: [z(9)]),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_memory_of_a_call_on_another_stream(world, name, monkeypatch):  # noqa: F811
    monkeypatch.setitem(test_streams.CALLS, name, CALLS[name])
    test_streams.test_memory_of_a_call_on_another_stream(world, name)


@pytest.mark.parametrize("name", list(CALLS))
def test_memory_of_a_call_on_the_current_stream(world, name, monkeypatch):  # noqa: F811
    monkeypatch.setitem(test_streams.CALLS, name, CALLS[name])
    test_streams.test_memory_of_a_call_on_the_current_stream(world, name)
