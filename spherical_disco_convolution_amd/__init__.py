"""Python binding of libdisco.so, the gfx950 forward DISCO convolution on S^2.

Thin ctypes layer: it marshals torch tensors (device memory and the current
HIP stream) into the C-ABI calls declared in include/disco.h and turns status
codes into exceptions.  All arithmetic runs in the library's HIP kernels;
there is no Python or CPU fallback, and importing fails loudly when the
library is missing.

Entry points (same names as the C ABI, without the ``disco_`` prefix):
    psi_build(...)      -> Psi          host float64 build of the sparse tensor
    contract(psi, x)    -> xk           [B, C, K, nlat_out, nlon_out]
    einsum(xk, w, ...)  -> y            [B, Co, nlat_out, nlon_out]
    fused_fwd(psi, x, w, ...) -> y      same result without storing xk
  gradients (gy: gradient of the loss with respect to y):
    contract_transpose(psi, gxk) -> gx          adjoint of contract
    einsum_grad_xk(gy, w, ...)   -> gxk         adjoint of einsum in xk
    einsum_grad_w(xk, gy, ...)   -> gw          adjoint of einsum in w
    fused_bwd(psi, x, w, gy, ...) -> (gx, gw, gbias)   X_K recomputed, never whole
  around the layer in a training step:
    layer_norm_fwd(x, gamma, beta, residual=...) -> (y, sum, mean, rstd)
    layer_norm_bwd(x, gy, mean, rstd, gamma, gsum=...) -> (gx, ggamma, gbeta)
    orthogonalize(m, ...) -> o                  Newton-Schulz products
    muon_step(w, grad, momentum, lr, ...) -> (w, momentum, w16)   one optimiser step

With stream=s a call's kernels run on s, and its results are there once s has
come to them.  Inputs have to be ready on s (s.wait_stream where another stream
makes them); they may be let go of as soon as the call returns, and so may the
results by the stream that was current at the call.
"""
from __future__ import annotations

import ctypes
import math
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdisco.so")

DISCO_OK = 0
DISCO_EINVAL = -1
DISCO_EUNSUPPORTED = -2
DISCO_ENOMEM = -3
DISCO_EHIP = -4

F32 = 0
BF16 = 1

GRIDS = {"equiangular": 0, "legendre-gauss": 1, "lobatto": 2, "equiangular-trapezoidal": 3}
BASES = {"piecewise linear": 0}
NORMS = {"none": 0}


class _Desc(ctypes.Structure):
    _fields_ = [
        ("nlat_in", ctypes.c_int32), ("nlon_in", ctypes.c_int32),
        ("nlat_out", ctypes.c_int32), ("nlon_out", ctypes.c_int32),
        ("grid_in", ctypes.c_int32), ("grid_out", ctypes.c_int32),
        ("basis_type", ctypes.c_int32), ("basis_norm", ctypes.c_int32),
        ("kernel_shape", ctypes.c_int32 * 2),
        ("theta_cutoff", ctypes.c_double),
    ]


def _load():
    # PyTorch ships its own HIP runtime (SONAME libamdhip64.so.7).  Loading
    # torch first makes libdisco.so bind to that same runtime, so the device
    # pointers and stream handles torch hands over are valid in the library.
    # Loading libdisco.so first would pull in a second HIP runtime.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python spherical_disco_convolution_amd/build_lib.py` (hipcc, gfx950)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, D = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double
    sig = {
        "disco_psi_build": (ctypes.c_int, [ctypes.POINTER(_Desc), ctypes.POINTER(P)]),
        "disco_psi_query": (ctypes.c_int, [P, ctypes.POINTER(I32), ctypes.POINTER(I64),
                                           ctypes.POINTER(I64), ctypes.POINTER(D)]),
        "disco_psi_export": (ctypes.c_int, [P, P, P, P, P]),
        "disco_psi_to_device": (ctypes.c_int, [P]),
        "disco_psi_free": (None, [P]),
        "disco_contract": (ctypes.c_int, [P, P, ctypes.c_int, P, ctypes.c_int, I32, I32, P]),
        "disco_einsum": (ctypes.c_int, [P, ctypes.c_int, P, ctypes.c_int, P, P, ctypes.c_int,
                                        I32, I32, I32, I32, I32, I32, I32, P]),
        "disco_fused_fwd": (ctypes.c_int, [P, P, ctypes.c_int, P, ctypes.c_int, P, P,
                                           ctypes.c_int, I32, I32, I32, I32, P]),
        "disco_fused_fwd_noalloc": (ctypes.c_int, [P, P, ctypes.c_int, P, ctypes.c_int, P, P,
                                                   ctypes.c_int, I32, I32, I32, I32, P]),
        "disco_fused_is_spectral": (ctypes.c_int, [P, ctypes.c_int, I32, I32, I32]),
        "disco_contract_transpose": (ctypes.c_int, [P, P, ctypes.c_int, P, ctypes.c_int, I32, I32,
                                                    P]),
        "disco_einsum_grad_xk": (ctypes.c_int, [P, ctypes.c_int, P, ctypes.c_int, P, ctypes.c_int,
                                                I32, I32, I32, I32, I32, I32, I32, P]),
        "disco_einsum_grad_w": (ctypes.c_int, [P, ctypes.c_int, P, ctypes.c_int, P, I32, I32, I32,
                                               I32, I32, I32, I32, P]),
        "disco_fused_bwd": (ctypes.c_int, [P, P, ctypes.c_int, P, ctypes.c_int, P, ctypes.c_int, P,
                                           ctypes.c_int, P, P, I32, I32, I32, I32, P]),
        "disco_layer_norm_fwd": (ctypes.c_int, [P, ctypes.c_int, P, P, P, P, ctypes.c_int, P, P, P,
                                                I64, I32, I64, ctypes.c_float, P]),
        "disco_layer_norm_bwd_workspace": (I64, [I64, I32, I64]),
        "disco_layer_norm_bwd": (ctypes.c_int, [P, ctypes.c_int, P, ctypes.c_int, P, P, P, P, P,
                                                ctypes.c_int, P, P, P, I64, I64, I32, I64, P]),
        "disco_orthogonalize_workspace": (I64, [I32, I32, I32]),
        "disco_orthogonalize": (ctypes.c_int, [P, ctypes.c_int, P, ctypes.c_int, I32, I32, I32, I32, P,
                                               ctypes.c_float, P, I64, P]),
        "disco_muon_step": (ctypes.c_int, [P, ctypes.c_int, P, P, P, ctypes.c_int, P, P, ctypes.c_float,
                                           ctypes.c_float, ctypes.c_int, ctypes.c_float,
                                           ctypes.c_float, I32, I32, I32, I32, P, ctypes.c_float, P,
                                           I64, P]),
        "disco_kernel_timing": (ctypes.c_int, [ctypes.c_int]),
        "disco_kernel_timing_read": (ctypes.c_int, [ctypes.c_char_p, I32, ctypes.POINTER(D),
                                                    ctypes.POINTER(I64), I32]),
        "disco_last_error": (ctypes.c_char_p, []),
        "disco_version": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()
EXPORTED = ("disco_psi_build", "disco_psi_query", "disco_psi_export", "disco_psi_to_device",
            "disco_psi_free", "disco_contract", "disco_einsum", "disco_fused_fwd",
            "disco_fused_fwd_noalloc",
            "disco_fused_is_spectral", "disco_contract_transpose", "disco_einsum_grad_xk",
            "disco_einsum_grad_w", "disco_fused_bwd", "disco_layer_norm_fwd",
            "disco_layer_norm_bwd_workspace", "disco_layer_norm_bwd", "disco_orthogonalize_workspace",
            "disco_orthogonalize", "disco_muon_step", "disco_kernel_timing", "disco_kernel_timing_read",
            "disco_last_error", "disco_version")


def version() -> str:
    return _lib.disco_version().decode()


def _check(rc: int, what: str):
    if rc == DISCO_OK:
        return
    msg = f"{what}: {_lib.disco_last_error().decode()}"
    if rc == DISCO_EINVAL:
        raise ValueError(msg)
    if rc == DISCO_EUNSUPPORTED:
        raise NotImplementedError(msg)
    if rc == DISCO_ENOMEM:
        raise MemoryError(msg)
    raise RuntimeError(msg)


def _kernel_shape(ks):
    if isinstance(ks, int):
        return (ks, 0)
    ks = tuple(int(v) for v in ks)
    if len(ks) == 1:
        return (ks[0], 0)
    if len(ks) == 2:
        return ks
    raise ValueError(f"kernel_shape must be an int or a tuple of one or two ints, got {ks}")


class Psi:
    """Handle of a built Psi tensor (library-owned)."""

    def __init__(self, handle, desc: _Desc):
        self._h = ctypes.c_void_p(handle)
        self.desc = desc
        K = ctypes.c_int32()
        nnz = ctypes.c_int64()
        nzz = ctypes.c_int64()
        cut = ctypes.c_double()
        _check(_lib.disco_psi_query(self._h, ctypes.byref(K), ctypes.byref(nnz),
                                    ctypes.byref(nzz), ctypes.byref(cut)), "psi_query")
        self.K = K.value
        self.nnz = nnz.value
        self.nnz_nonzero = nzz.value
        self.theta_cutoff = cut.value
        self.nlat_in, self.nlon_in = desc.nlat_in, desc.nlon_in
        self.nlat_out, self.nlon_out = desc.nlat_out, desc.nlon_out
        self.on_device = False

    @property
    def handle(self):
        return self._h

    def export(self):
        """Canonical CSR as numpy arrays (row_ptr, in_lat, lon_off, vals[nnz, K])."""
        row_ptr = np.zeros(self.nlat_out + 1, dtype=np.int64)
        in_lat = np.zeros(self.nnz, dtype=np.int32)
        lon_off = np.zeros(self.nnz, dtype=np.int32)
        vals = np.zeros((self.nnz, self.K), dtype=np.float64)
        _check(_lib.disco_psi_export(self._h, row_ptr.ctypes.data, in_lat.ctypes.data,
                                     lon_off.ctypes.data, vals.ctypes.data), "psi_export")
        return row_ptr, in_lat, lon_off, vals

    def to_device(self):
        """Copy the device form to the current HIP device (once)."""
        _check(_lib.disco_psi_to_device(self._h), "psi_to_device")
        self.on_device = True
        return self

    def __del__(self):
        h = getattr(self, "_h", None)
        # at interpreter exit the module's globals may already be cleared:
        # the process is ending and the handle goes with it
        if h is not None and h.value and _lib is not None:
            _lib.disco_psi_free(h)
            self._h = ctypes.c_void_p(0)


def psi_build(nlat_in: int, nlon_in: int, nlat_out: int, nlon_out: int, kernel_shape,
              theta_cutoff: float | None = None, grid_in: str = "equiangular",
              grid_out: str = "equiangular", basis_type: str = "piecewise linear",
              basis_norm_mode: str = "none") -> Psi:
    """Build Psi on the host (float64).  Arguments follow the layer's
    constructor: in_shape/out_shape as (nlat, nlon), kernel_shape, theta_cutoff
    (None selects (nr+1)*pi/(nlat_out-1)), grids, basis type and norm."""
    d = _Desc()
    d.nlat_in, d.nlon_in, d.nlat_out, d.nlon_out = nlat_in, nlon_in, nlat_out, nlon_out
    for key, table, val in (("grid_in", GRIDS, grid_in), ("grid_out", GRIDS, grid_out),
                            ("basis_type", BASES, basis_type), ("basis_norm", NORMS, basis_norm_mode)):
        if val not in table:
            raise NotImplementedError(f"{key}={val!r} is not implemented (supported: {list(table)})")
        setattr(d, key, table[val])
    nr, nphi = _kernel_shape(kernel_shape)
    d.kernel_shape[0], d.kernel_shape[1] = nr, nphi
    if theta_cutoff is None:
        d.theta_cutoff = 0.0
    else:
        if not (theta_cutoff > 0.0):
            raise ValueError(f"theta_cutoff must be positive, got {theta_cutoff}")
        d.theta_cutoff = float(theta_cutoff)
    h = ctypes.c_void_p()
    _check(_lib.disco_psi_build(ctypes.byref(d), ctypes.byref(h)), "psi_build")
    return Psi(h.value, d)


# ----------------------------------------------------------------------------
# compute entry points (torch tensors on the current HIP device)
# ----------------------------------------------------------------------------
def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise ValueError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _torch_dtype(code: int):
    torch = _torch()
    return torch.float32 if code == F32 else torch.bfloat16


def _raw_current_stream():
    """Handle of the current device's current stream.  torch.cuda.current_stream()
    builds a Stream object each time (2.7 us, against 0.1 us for the handle)."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None:
        return torch.cuda.current_stream().cuda_stream
    return raw(torch.cuda.current_device())


def _stream():
    return ctypes.c_void_p(_raw_current_stream())


def _on(stream, f, *args):
    """f(*args) on `stream`.  A block of the allocator's is free as far as the stream
    goes that it was taken under, so the call takes its results and its scratch under
    `stream`.  What it was given is kept, should the caller let go of it, until
    `stream` is through with it, and the results until the current stream is."""
    torch = _torch()
    current = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        out = f(*args)
    given = [t for t in args if isinstance(t, torch.Tensor)]
    for t in given:
        t.record_stream(stream)
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None and not any(t is g for g in given):
            t.record_stream(current)
    return out


def _need(t, name, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def contract(psi: Psi, x, xk=None, xk_dtype=None, stream=None):
    """xk[b,c,k,j,q] = sum_(i,p) Psi[k,j,(i,p)] x[b,c,i,(q*s+p) mod nlon_in]."""
    if stream is not None:
        return _on(stream, contract, psi, x, xk, xk_dtype)
    torch = _torch()
    if x.dim() != 4:
        raise ValueError("x must be [B, C, nlat_in, nlon_in]")
    B, C = x.shape[:2]
    _need(x, "x", (B, C, psi.nlat_in, psi.nlon_in))
    if xk is None:
        dt = x.dtype if xk_dtype is None else xk_dtype
        xk = torch.empty((B, C, psi.K, psi.nlat_out, psi.nlon_out), dtype=dt, device=x.device)
    _need(xk, "xk", (B, C, psi.K, psi.nlat_out, psi.nlon_out))
    _check(_lib.disco_contract(psi.handle, x.data_ptr(), _dtype_code(x), xk.data_ptr(),
                               _dtype_code(xk), B, C, _stream()), "contract")
    return xk


def einsum(xk, w, groups: int = 1, bias=None, y=None, out_dtype=None, stream=None):
    """y[b,co,j,q] = bias[co] + sum_(ci',k) w[co,ci',k] xk[b, G(co)*Ci/G+ci', k, j, q]."""
    if stream is not None:
        return _on(stream, einsum, xk, w, groups, bias, y, out_dtype)
    torch = _torch()
    if xk.dim() != 5 or w.dim() != 3:
        raise ValueError("xk must be [B, Ci, K, nlat_out, nlon_out] and w [Co, Ci/groups, K]")
    B, Ci, K, H, W = xk.shape
    Co = w.shape[0]
    _need(xk, "xk", (B, Ci, K, H, W))
    if groups < 1 or Ci % groups or Co % groups:
        raise ValueError(f"groups ({groups}) must divide in_channels ({Ci}) and out_channels ({Co})")
    _need(w, "w", (Co, Ci // groups, K))
    if y is None:
        dt = torch.float32 if out_dtype is None else out_dtype
        y = torch.empty((B, Co, H, W), dtype=dt, device=xk.device)
    _need(y, "y", (B, Co, H, W))
    bptr = None
    if bias is not None:
        _need(bias, "bias", (Co,))
        if bias.dtype != torch.float32:
            raise ValueError("bias must be float32")
        bptr = bias.data_ptr()
    _check(_lib.disco_einsum(xk.data_ptr(), _dtype_code(xk), w.data_ptr(), _dtype_code(w), bptr,
                             y.data_ptr(), _dtype_code(y), B, Ci, Co, groups, K, H, W,
                             _stream()), "einsum")
    return y


def fused_is_spectral(psi: Psi, x_dtype, Ci: int, Co: int, groups: int = 1) -> bool:
    """Whether fused_fwd takes the longitude-spectral path for these arguments
    (x_dtype: a torch dtype)."""
    torch = _torch()
    code = BF16 if x_dtype == torch.bfloat16 else F32
    rc = _lib.disco_fused_is_spectral(psi.handle, code, Ci, Co, groups)
    if rc < 0:
        _check(rc, "fused_is_spectral")
    return rc == 1


def kernel_timing(enable: bool) -> None:
    """Start (True) or stop (False) recording a HIP event pair around every
    kernel the library launches, on its launch stream."""
    _check(_lib.disco_kernel_timing(1 if enable else 0), "kernel_timing")


def kernel_timing_read(max_kernels: int = 64) -> dict:
    """Drain the recorded events: {kernel name: (total milliseconds, launches)},
    in order of first launch.  Waits for the recorded launches to finish."""
    names = ctypes.create_string_buffer(64 * max_kernels)
    tot = (ctypes.c_double * max_kernels)()
    cnt = (ctypes.c_int64 * max_kernels)()
    n = _lib.disco_kernel_timing_read(names, len(names), tot, cnt, max_kernels)
    if n < 0:
        _check(n, "kernel_timing_read")
    out, off = {}, 0
    raw = names.raw
    for i in range(n):
        end = raw.index(b"\0", off)
        out[raw[off:end].decode()] = (tot[i], cnt[i])
        off = end + 1
    return out


def fused_fwd(psi: Psi, x, w, groups: int = 1, bias=None, y=None, out_dtype=None, stream=None):
    """The forward DISCO convolution without storing the K-expanded tensor."""
    if stream is not None:
        return _on(stream, fused_fwd, psi, x, w, groups, bias, y, out_dtype)
    torch = _torch()
    if x.dim() != 4 or w.dim() != 3:
        raise ValueError("x must be [B, Ci, nlat_in, nlon_in] and w [Co, Ci/groups, K]")
    B, Ci = x.shape[:2]
    Co = w.shape[0]
    _need(x, "x", (B, Ci, psi.nlat_in, psi.nlon_in))
    if groups < 1 or Ci % groups or Co % groups:
        raise ValueError(f"groups ({groups}) must divide in_channels ({Ci}) and out_channels ({Co})")
    _need(w, "w", (Co, Ci // groups, psi.K))
    if y is None:
        dt = torch.float32 if out_dtype is None else out_dtype
        y = torch.empty((B, Co, psi.nlat_out, psi.nlon_out), dtype=dt, device=x.device)
    _need(y, "y", (B, Co, psi.nlat_out, psi.nlon_out))
    bptr = None
    if bias is not None:
        _need(bias, "bias", (Co,))
        if bias.dtype != torch.float32:
            raise ValueError("bias must be float32")
        bptr = bias.data_ptr()
    _check(_lib.disco_fused_fwd(psi.handle, x.data_ptr(), _dtype_code(x), w.data_ptr(),
                                _dtype_code(w), bptr, y.data_ptr(), _dtype_code(y), B, Ci, Co,
                                groups, _stream()), "fused_fwd")
    return y



def fused_fwd_noalloc(psi: Psi, x, w, y, groups: int = 1, bias=None, stream=None):
    """fused_fwd for callers that cannot allocate device memory: the direct
    algorithms with the library's fixed scratch; y must be given."""
    if stream is not None:
        return _on(stream, fused_fwd_noalloc, psi, x, w, y, groups, bias)
    if x.dim() != 4 or w.dim() != 3:
        raise ValueError("x must be [B, Ci, nlat_in, nlon_in] and w [Co, Ci/groups, K]")
    B, Ci = x.shape[:2]
    Co = w.shape[0]
    _need(x, "x", (B, Ci, psi.nlat_in, psi.nlon_in))
    if groups < 1 or Ci % groups or Co % groups:
        raise ValueError(f"groups ({groups}) must divide in_channels ({Ci}) and out_channels ({Co})")
    _need(w, "w", (Co, Ci // groups, psi.K))
    _need(y, "y", (B, Co, psi.nlat_out, psi.nlon_out))
    bptr = None
    if bias is not None:
        _need(bias, "bias", (Co,))
        bptr = bias.data_ptr()
    _check(_lib.disco_fused_fwd_noalloc(psi.handle, x.data_ptr(), _dtype_code(x), w.data_ptr(),
                                        _dtype_code(w), bptr, y.data_ptr(), _dtype_code(y), B, Ci,
                                        Co, groups, _stream()), "fused_fwd_noalloc")
    return y


# ----------------------------------------------------------------------------
# gradients
# ----------------------------------------------------------------------------
def contract_transpose(psi: Psi, gxk, gx=None, gx_dtype=None, stream=None):
    """gx[b,c,i,(q*s+p) mod nlon_in] = sum over windows of Psi[k,j,(i,p)] gxk[b,c,k,j,q]
    (the adjoint of contract)."""
    if stream is not None:
        return _on(stream, contract_transpose, psi, gxk, gx, gx_dtype)
    torch = _torch()
    if gxk.dim() != 5:
        raise ValueError("gxk must be [B, C, K, nlat_out, nlon_out]")
    B, C = gxk.shape[:2]
    _need(gxk, "gxk", (B, C, psi.K, psi.nlat_out, psi.nlon_out))
    if gx is None:
        dt = torch.float32 if gx_dtype is None else gx_dtype
        gx = torch.empty((B, C, psi.nlat_in, psi.nlon_in), dtype=dt, device=gxk.device)
    _need(gx, "gx", (B, C, psi.nlat_in, psi.nlon_in))
    _check(_lib.disco_contract_transpose(psi.handle, gxk.data_ptr(), _dtype_code(gxk),
                                         gx.data_ptr(), _dtype_code(gx), B, C, _stream()),
           "contract_transpose")
    return gx


def einsum_grad_xk(gy, w, groups: int = 1, gxk=None, out_dtype=None, stream=None):
    """gxk[b, G*Ci/G+ci', k, j, q] = sum_{co in G} w[co,ci',k] gy[b,co,j,q]."""
    if stream is not None:
        return _on(stream, einsum_grad_xk, gy, w, groups, gxk, out_dtype)
    torch = _torch()
    if gy.dim() != 4 or w.dim() != 3:
        raise ValueError("gy must be [B, Co, nlat_out, nlon_out] and w [Co, Ci/groups, K]")
    B, Co, H, W = gy.shape
    _need(gy, "gy", (B, Co, H, W))
    if groups < 1 or Co % groups or w.shape[0] != Co:
        raise ValueError(f"w must have {Co} rows and groups ({groups}) must divide them")
    Ci, K = w.shape[1] * groups, w.shape[2]
    _need(w, "w", (Co, Ci // groups, K))
    if gxk is None:
        dt = torch.float32 if out_dtype is None else out_dtype
        gxk = torch.empty((B, Ci, K, H, W), dtype=dt, device=gy.device)
    _need(gxk, "gxk", (B, Ci, K, H, W))
    _check(_lib.disco_einsum_grad_xk(gy.data_ptr(), _dtype_code(gy), w.data_ptr(), _dtype_code(w),
                                     gxk.data_ptr(), _dtype_code(gxk), B, Ci, Co, groups, K, H, W,
                                     _stream()), "einsum_grad_xk")
    return gxk


def einsum_grad_w(xk, gy, groups: int = 1, gw=None, stream=None):
    """gw[co,ci',k] = sum_{b,j,q} gy[b,co,j,q] xk[b, G(co)*Ci/G+ci', k, j, q] (float32)."""
    if stream is not None:
        return _on(stream, einsum_grad_w, xk, gy, groups, gw)
    torch = _torch()
    if xk.dim() != 5 or gy.dim() != 4:
        raise ValueError("xk must be [B, Ci, K, nlat_out, nlon_out] and gy [B, Co, nlat_out, nlon_out]")
    B, Ci, K, H, W = xk.shape
    Co = gy.shape[1]
    _need(xk, "xk", (B, Ci, K, H, W))
    _need(gy, "gy", (B, Co, H, W))
    if groups < 1 or Ci % groups or Co % groups:
        raise ValueError(f"groups ({groups}) must divide in_channels ({Ci}) and out_channels ({Co})")
    if gw is None:
        gw = torch.empty((Co, Ci // groups, K), dtype=torch.float32, device=xk.device)
    _need(gw, "gw", (Co, Ci // groups, K))
    if gw.dtype != torch.float32:
        raise ValueError("gw must be float32")
    _check(_lib.disco_einsum_grad_w(xk.data_ptr(), _dtype_code(xk), gy.data_ptr(), _dtype_code(gy),
                                    gw.data_ptr(), B, Ci, Co, groups, K, H, W, _stream()),
           "einsum_grad_w")
    return gw


def fused_bwd(psi: Psi, x, w, gy, groups: int = 1, need_gx: bool = True, need_gw: bool = True,
              need_gbias: bool = False, gx_dtype=None, stream=None):
    """Gradients (gx, gw, gbias) of sum(gy * fused_fwd(psi, x, w)) with X_K
    recomputed slab by slab; entries not asked for are None."""
    if stream is not None:
        return _on(stream, fused_bwd, psi, x, w, gy, groups, need_gx, need_gw, need_gbias, gx_dtype)
    torch = _torch()
    if x.dim() != 4 or w.dim() != 3 or gy.dim() != 4:
        raise ValueError("x must be [B, Ci, nlat_in, nlon_in], w [Co, Ci/groups, K] and gy "
                         "[B, Co, nlat_out, nlon_out]")
    B, Ci = x.shape[:2]
    Co = w.shape[0]
    _need(x, "x", (B, Ci, psi.nlat_in, psi.nlon_in))
    if groups < 1 or Ci % groups or Co % groups:
        raise ValueError(f"groups ({groups}) must divide in_channels ({Ci}) and out_channels ({Co})")
    _need(w, "w", (Co, Ci // groups, psi.K))
    _need(gy, "gy", (B, Co, psi.nlat_out, psi.nlon_out))
    gx = gw = gb = None
    if need_gx:
        gx = torch.empty((B, Ci, psi.nlat_in, psi.nlon_in),
                         dtype=torch.float32 if gx_dtype is None else gx_dtype, device=x.device)
    if need_gw:
        gw = torch.empty((Co, Ci // groups, psi.K), dtype=torch.float32, device=x.device)
    if need_gbias:
        gb = torch.empty((Co,), dtype=torch.float32, device=x.device)
    _check(_lib.disco_fused_bwd(psi.handle, x.data_ptr(), _dtype_code(x), w.data_ptr(),
                                _dtype_code(w), gy.data_ptr(), _dtype_code(gy),
                                gx.data_ptr() if gx is not None else None,
                                _dtype_code(gx) if gx is not None else F32,
                                gw.data_ptr() if gw is not None else None,
                                gb.data_ptr() if gb is not None else None,
                                B, Ci, Co, groups, _stream()), "fused_bwd")
    return gx, gw, gb


# ----------------------------------------------------------------------------
# layer norm
# ----------------------------------------------------------------------------
def _int32(*sizes):
    """The library takes these as 32-bit integers; ctypes would cut them off."""
    for n in sizes:
        if not -0x80000000 <= n <= 0x7fffffff:
            raise NotImplementedError(f"a size or count of {n} does not fit 32 bits")


def _norm_view(x, axis):
    """(outer, C, inner, shape without the channel axis) of x's channel axis."""
    if x.dim() < 2:
        raise ValueError("x must have at least two dimensions")
    if not -x.dim() <= axis < x.dim():
        raise ValueError(f"axis {axis} is out of range for {x.dim()} dimensions")
    axis %= x.dim()
    shape = x.shape
    before, after = shape[:axis], shape[axis + 1:]
    _int32(shape[axis])
    return math.prod(before), shape[axis], math.prod(after), before + after


def _same_dtype(t, name, out_dtype):
    if out_dtype is not None and t.dtype != out_dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, out_dtype is {out_dtype}")


def _f32_ptr(t, name, shape):
    """Pointer of an optional float32 tensor."""
    if t is None:
        return None
    _need(t, name, shape)
    if t.dtype != _torch().float32:
        raise ValueError(f"{name} must be float32")
    return t.data_ptr()


def _workspace(nbytes, like):
    """Scratch for one call on like's device (None for no bytes).  Let go of when the
    call returns, it goes to later work on the current stream only."""
    return like.new_empty(nbytes, dtype=_torch().uint8) if nbytes else None


def layer_norm_fwd(x, gamma=None, beta=None, residual=None, eps: float = 1e-5, axis: int = 1,
                   y=None, out_dtype=None, need_stats: bool = True, stream=None):
    """Layer norm over `axis` (1: the channels of a field [B, C, nlat, nlon];
    -1: channel-last rows): y = (s - mean) * rstd * gamma + beta with s = x, or
    s = x + residual rounded to x's dtype.

    Returns (y, s, mean, rstd): s is None without a residual, the statistics
    (float32, x's shape without the axis) None with need_stats=False.  y has
    out_dtype, or x's dtype."""
    if stream is not None:
        return _on(stream, layer_norm_fwd, x, gamma, beta, residual, eps, axis, y, out_dtype, need_stats)
    torch = _torch()
    outer, C, inner, points = _norm_view(x, axis)
    _need(x, "x", x.shape)
    gptr, bptr = _f32_ptr(gamma, "gamma", (C,)), _f32_ptr(beta, "beta", (C,))
    s = mean = rstd = None
    if residual is not None:
        _need(residual, "residual", x.shape)
        if residual.dtype != x.dtype:
            raise ValueError(f"residual must have x's dtype ({x.dtype})")
        s = torch.empty_like(x)
    if y is None:
        y = torch.empty_like(x, dtype=x.dtype if out_dtype is None else out_dtype)
    else:
        _need(y, "y", x.shape)
        _same_dtype(y, "y", out_dtype)
    if need_stats:
        mean = x.new_empty(points, dtype=torch.float32)
        rstd = torch.empty_like(mean)
    _check(_lib.disco_layer_norm_fwd(
        x.data_ptr(), _dtype_code(x), residual.data_ptr() if s is not None else None, gptr, bptr,
        y.data_ptr(), _dtype_code(y), s.data_ptr() if s is not None else None,
        mean.data_ptr() if need_stats else None, rstd.data_ptr() if need_stats else None,
        outer, C, inner, eps, _stream()), "layer_norm_fwd")
    return y, s, mean, rstd


def layer_norm_bwd(x, gy, mean, rstd, gamma=None, gsum=None, axis: int = 1, need_gx: bool = True,
                   need_gparams: bool = True, gx_dtype=None, stream=None):
    """Gradients (gx, ggamma, gbeta) of sum(gy * layer_norm_fwd(x)); entries not
    asked for are None.  x is what was normalised (the forward's s where it had
    a residual).  gsum (gy's dtype): the gradient that reaches x past the norm,
    added to gx.  gx has gx_dtype, or float32."""
    if stream is not None:
        return _on(stream, layer_norm_bwd, x, gy, mean, rstd, gamma, gsum, axis, need_gx, need_gparams,
                   gx_dtype)
    torch = _torch()
    outer, C, inner, points = _norm_view(x, axis)
    _need(x, "x", x.shape)
    _need(gy, "gy", x.shape)
    if mean is None or rstd is None:
        raise ValueError("mean and rstd of the forward pass are needed")
    mptr, rptr = _f32_ptr(mean, "mean", points), _f32_ptr(rstd, "rstd", points)
    gptr = _f32_ptr(gamma, "gamma", (C,))
    if gsum is not None:
        _need(gsum, "gsum", x.shape)
        if gsum.dtype != gy.dtype:
            raise ValueError(f"gsum must have gy's dtype ({gy.dtype})")
    gx = gg = gb = None
    if need_gx:
        gx = torch.empty_like(x, dtype=torch.float32 if gx_dtype is None else gx_dtype)
    ws, nws = None, 0
    if need_gparams:
        gg = x.new_empty((C,), dtype=torch.float32)
        gb = torch.empty_like(gg)
        nws = _lib.disco_layer_norm_bwd_workspace(outer, C, inner)
        if nws < 0:
            _check(nws, "layer_norm_bwd")
        ws = _workspace(nws, x)
    _check(_lib.disco_layer_norm_bwd(
        x.data_ptr(), _dtype_code(x), gy.data_ptr(), _dtype_code(gy), mptr, rptr, gptr,
        gsum.data_ptr() if gsum is not None else None,
        gx.data_ptr() if need_gx else None, _dtype_code(gx) if need_gx else F32,
        gg.data_ptr() if need_gparams else None, gb.data_ptr() if need_gparams else None,
        ws.data_ptr() if ws is not None else None, nws, outer, C, inner, _stream()),
        "layer_norm_bwd")
    return gx, gg, gb


# ----------------------------------------------------------------------------
# orthogonalised weight updates
# ----------------------------------------------------------------------------
def _coeffs(coeffs):
    if coeffs is None:
        return None
    coeffs = tuple(float(c) for c in coeffs)
    if len(coeffs) != 3:
        raise ValueError("coeffs must be three numbers (a, b, c)")
    return (ctypes.c_float * 3)(*coeffs)


def _ortho_workspace(batch, rows, cols, like, what):
    n = _lib.disco_orthogonalize_workspace(batch, rows, cols)
    if n < 0:
        _check(n, what)
    return _workspace(n, like), n


def orthogonalize(m, out=None, out_dtype=None, steps: int = 5, coeffs=None, eps: float = 1e-7,
                  stream=None):
    """Newton-Schulz orthogonalisation of a matrix [rows, cols] or of each
    matrix of a batch [batch, rows, cols]: singular values near one, singular
    vectors kept.  The result is computed to float32 accuracy and rounded to
    out_dtype, or m's dtype.  coeffs: (a, b, c) of the step X <- a X + (b A + c A^2) X."""
    if stream is not None:
        return _on(stream, orthogonalize, m, out, out_dtype, steps, coeffs, eps)
    torch = _torch()
    if m.dim() not in (2, 3):
        raise ValueError("m must be [rows, cols] or [batch, rows, cols]")
    _need(m, "m", m.shape)
    batch = m.shape[0] if m.dim() == 3 else 1
    rows, cols = m.shape[-2:]
    _int32(batch, rows, cols, steps)
    if out is None:
        out = torch.empty_like(m, dtype=m.dtype if out_dtype is None else out_dtype)
    else:
        _need(out, "out", m.shape)
        _same_dtype(out, "out", out_dtype)
    ws, nws = _ortho_workspace(batch, rows, cols, m, "orthogonalize")
    _check(_lib.disco_orthogonalize(m.data_ptr(), _dtype_code(m), out.data_ptr(), _dtype_code(out),
                                    batch, rows, cols, steps, _coeffs(coeffs), eps,
                                    ws.data_ptr() if ws is not None else None, nws,
                                    _stream()), "orthogonalize")
    return out


def muon_step(w, grad, momentum, lr: float, beta: float = 0.95, nesterov: bool = True,
              weight_decay: float = 0.0, scale: float | None = None, steps: int = 5, coeffs=None,
              eps: float = 1e-7, groups: int = 1, w_out=None, momentum_out=None,
              need_bf16_copy: bool = False, w16=None, stream=None):
    """One step of the optimiser that orthogonalises the momentum:

        momentum <- beta momentum + grad
        u = grad + beta momentum (nesterov), or momentum
        w <- w (1 - lr weight_decay) - lr scale orthogonalize(u)

    w [Co, ...] is seen as `groups` matrices of Co/groups rows (the layer's
    weight [Co, Ci/groups, K] with its groups); grad and momentum (float32)
    have its shape.  scale None: sqrt(max(1, rows/cols)).  w and momentum are
    updated in place unless w_out / momentum_out are given.  need_bf16_copy:
    also return (in w16, if given) the bfloat16 copy of a float32 w.
    Returns (w, momentum, w16)."""
    if stream is not None:
        return _on(stream, muon_step, w, grad, momentum, lr, beta, nesterov, weight_decay, scale, steps, coeffs,
                   eps, groups, w_out, momentum_out, need_bf16_copy, w16)
    torch = _torch()
    if w.dim() < 2:
        raise ValueError("w must have at least two dimensions")
    if groups < 1 or w.shape[0] % groups:
        raise ValueError(f"groups ({groups}) must divide w's {w.shape[0]} rows")
    _need(w, "w", w.shape)
    _need(grad, "grad", w.shape)
    mptr = _f32_ptr(momentum, "momentum", w.shape)
    if mptr is None:
        raise ValueError("momentum is needed (zeros at first)")
    w_out = w if w_out is None else w_out
    momentum_out = momentum if momentum_out is None else momentum_out
    _need(w_out, "w_out", w.shape)
    if w_out.dtype != w.dtype:
        raise ValueError(f"w_out must have w's dtype ({w.dtype})")
    rows, cols = w.shape[0] // groups, math.prod(w.shape[1:])
    _int32(groups, rows, cols, steps)
    if scale is None:
        scale = max(1.0, rows / cols) ** 0.5 if cols else 1.0
    if w16 is None and need_bf16_copy:
        w16 = torch.empty_like(w, dtype=torch.bfloat16)
    if w16 is not None:
        _need(w16, "w16", w.shape)
        if w16.dtype != torch.bfloat16:
            raise ValueError("w16 must be bfloat16")
    ws, nws = _ortho_workspace(groups, rows, cols, w, "muon_step")
    _check(_lib.disco_muon_step(
        grad.data_ptr(), _dtype_code(grad), mptr, _f32_ptr(momentum_out, "momentum_out", w.shape),
        w.data_ptr(), _dtype_code(w), w_out.data_ptr(), w16.data_ptr() if w16 is not None else None,
        lr, beta, int(nesterov), weight_decay, scale, groups, rows, cols, steps, _coeffs(coeffs), eps,
        ws.data_ptr() if ws is not None else None, nws, _stream()), "muon_step")
    return w_out, momentum_out, w16
