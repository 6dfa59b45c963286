"""Where the binding's calls take their memory from when they are given a
stream, without a GPU: the library and torch's streams are stubs.

A block of the caching allocator belongs to the stream that was current when it
was taken, and work that used it before is ordered on that stream only.  So
what a call makes for kernels on `side` has to be taken under `side`, and kept
until the stream that the caller works on is through with it too; what the
caller hands over has to be kept until `side` is through with it.
"""
import contextlib
import types

import pytest

import spherical_disco_convolution_amd as sdc

torch = pytest.importorskip("torch")
from torch.utils._python_dispatch import TorchDispatchMode  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
PSI = types.SimpleNamespace(handle=None, K=3, nlat_in=5, nlon_in=8, nlat_out=5, nlon_out=8)


def z(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype)


def field():
    return z(2, 4, 5, 8)


# every entry point that takes a stream: a call of its inputs, and the inputs
CALLS = {
    "contract": (lambda a, s: sdc.contract(PSI, *a, stream=s), lambda: [field()]),
    "einsum": (lambda a, s: sdc.einsum(a[0], a[1], bias=a[2], stream=s),
               lambda: [z(2, 4, 3, 5, 8), z(6, 4, 3), z(6)]),
    "fused_fwd": (lambda a, s: sdc.fused_fwd(PSI, a[0], a[1], bias=a[2], stream=s),
                  lambda: [field(), z(6, 4, 3), z(6)]),
    "fused_fwd_noalloc": (lambda a, s: sdc.fused_fwd_noalloc(PSI, *a, stream=s),
                          lambda: [field(), z(6, 4, 3), z(2, 6, 5, 8)]),
    "contract_transpose": (lambda a, s: sdc.contract_transpose(PSI, *a, stream=s), lambda: [z(2, 4, 3, 5, 8)]),
    "einsum_grad_xk": (lambda a, s: sdc.einsum_grad_xk(*a, stream=s), lambda: [z(2, 6, 5, 8), z(6, 4, 3)]),
    "einsum_grad_w": (lambda a, s: sdc.einsum_grad_w(*a, stream=s), lambda: [z(2, 4, 3, 5, 8), z(2, 6, 5, 8)]),
    "fused_bwd": (lambda a, s: sdc.fused_bwd(PSI, *a, need_gbias=True, stream=s),
                  lambda: [field(), z(6, 4, 3), z(2, 6, 5, 8)]),
    "layer_norm_fwd": (lambda a, s: sdc.layer_norm_fwd(a[0], a[1], a[2], residual=a[3], stream=s),
                       lambda: [field(), z(4), z(4), field()]),
    "layer_norm_fwd_out": (lambda a, s: sdc.layer_norm_fwd(a[0], y=a[1], stream=s), lambda: [field(), field()]),
    "layer_norm_bwd": (lambda a, s: sdc.layer_norm_bwd(*a[:5], gsum=a[5], stream=s),
                       lambda: [field(), field(), z(2, 5, 8), z(2, 5, 8), z(4), field()]),
    "orthogonalize": (lambda a, s: sdc.orthogonalize(*a, stream=s), lambda: [z(2, 70, 90)]),
    "orthogonalize_out": (lambda a, s: sdc.orthogonalize(a[0], out=a[1], stream=s),
                          lambda: [z(2, 70, 90), z(2, 70, 90)]),
    "muon_step": (lambda a, s: sdc.muon_step(*a, 0.1, need_bf16_copy=True, stream=s),
                  lambda: [z(70, 90), z(70, 90), z(70, 90)]),
    "muon_step_out": (lambda a, s: sdc.muon_step(*a[:3], 0.1, w_out=a[3], momentum_out=a[4], w16=a[5], stream=s),
                      lambda: [z(70, 90), z(70, 90), z(70, 90), z(70, 90), z(70, 90), z(70, 90, dtype=BF16)]),
}


class Library:
    """Every call succeeds; workspaces have 4096 bytes."""

    def __getattr__(self, name):
        return (lambda *a: 4096) if name.endswith("_workspace") else (lambda *a: 0)


class Allocations(TorchDispatchMode):
    """(tensor, stream it was made under) of every new empty tensor."""

    def __init__(self, streams):
        super().__init__()
        self.streams, self.made = streams, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if "empty" in func.__name__:
            self.made.append((out, self.streams[-1]))
        return out


@pytest.fixture
def world(monkeypatch):
    """Stub streams: `current`, `side`; .under lists the streams made current."""
    w = types.SimpleNamespace(current=types.SimpleNamespace(cuda_stream=1), side=types.SimpleNamespace(cuda_stream=2),
                              records=[])
    w.under = [w.current]

    @contextlib.contextmanager
    def stream(s):
        w.under.append(s)
        yield
        w.under.pop()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w.under[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: w.records.append((t.data_ptr(), s)))
    monkeypatch.setattr(sdc, "_raw_current_stream", lambda: 1)
    monkeypatch.setattr(sdc, "_lib", Library())
    return w


def tensors(out):
    return [t for t in (out if isinstance(out, (tuple, list)) else [out]) if t is not None]


@pytest.mark.parametrize("name", list(CALLS))
def test_memory_of_a_call_on_another_stream(world, name):
    call, make = CALLS[name]
    inputs = make()
    with Allocations(world.under) as seen:
        out = tensors(call(inputs, world.side))
    given = {t.data_ptr() for t in inputs}
    for t, under in seen.made:
        assert under is world.side, (name, t.shape)
    made = {t.data_ptr() for t, _ in seen.made}
    assert {t.data_ptr() for t in out} <= made | given
    for t in inputs:                      # the kernels on `side` read or write them
        assert (t.data_ptr(), world.side) in world.records, (name, t.shape)
    for t in out:                         # the caller goes on with them
        if t.data_ptr() not in given:
            assert (t.data_ptr(), world.current) in world.records, (name, t.shape)


@pytest.mark.parametrize("name", list(CALLS))
def test_memory_of_a_call_on_the_current_stream(world, name):
    call, make = CALLS[name]
    with Allocations(world.under) as seen:
        call(make(), None)
    assert all(under is world.current for _, under in seen.made)
    assert not world.records
