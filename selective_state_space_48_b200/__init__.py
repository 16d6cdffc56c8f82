"""Python binding of the B200 selective-scan (S6) library.

Argument marshalling only: torch tensors supply device memory and the
current CUDA stream; every step of the computation runs in the CUDA kernels
of ``_lib/libsss48.so`` behind the C ABI declared in
``include/selective_scan.h``.  There is no CPU fallback: if the library is
missing or no CUDA device is present, the calls raise.

Functions mirror the C entry points:
  mamba_selective_scan_fwd  -> selective_scan_fwd(...)
  selective_state_update    -> selective_state_update(...)
  mss_scan_workspace_size   -> scan_workspace_size(...)
  mss_scan_status           -> scan_status(...)
  mamba2_ssd_fwd            -> ssd_fwd(...)         (include/ssd.h)
  mss_ssd_workspace_size    -> ssd_workspace_size(...)
  gated_delta_fwd           -> gated_delta_fwd(...)       (include/gated_delta.h)
  gated_delta_update        -> gated_delta_update(...)
  gated_rmsnorm_fwd / _bwd  -> gated_rmsnorm_fwd / _bwd / _fn(...)  (include/norm.h)
  add_rmsnorm_fwd / _bwd    -> add_rmsnorm_fwd / _bwd / _fn(...)
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct as _struct
import threading

import torch

from . import builder as _build

LIB_PATH = _build.LIB_PATH

ABI_VERSION = 11  # MSS_ABI_VERSION of include/selective_scan.h

MSS_OK = 0
MSS_ERR_INVALID_ARG = 1
MSS_ERR_UNSUPPORTED = 2
MSS_ERR_CUDA = 3
MSS_ERR_TIMEOUT = 4
MSS_ERR_WORKSPACE = 5
MSS_F32 = 0
MSS_BF16 = 1
MSS_TESTFLAG_DROP_PUBLISH = 0x1
MSS_TESTFLAG_DEBUG_OOB = 0x2  # checked build only: one planted out-of-range y store

MSS_DELTA_AUTO = 0
MSS_DELTA_RECURRENT = 1
MSS_DELTA_CHUNKED = 2

# every symbol the headers in include/ declare
EXPORTED_SYMBOLS = (
    "mss_scan_workspace_size",
    "mamba_selective_scan_fwd",
    "mss_scan_status",
    "mamba_selective_scan_fwd_noalloc",
    "mss_scan_noalloc_status",
    "selective_state_update",
    "mss_scan_bwd_workspace_size",
    "mamba_selective_scan_bwd",
    "mss_status_string",
    "mss_abi_version",
    "mss_ssd_workspace_size",
    "mamba2_ssd_fwd",
    "mss_ssd_status",
    "gated_delta_fwd",
    "gated_delta_update",
    "mss_gated_delta_status",
    "mss_gated_delta_workspace_size",
    "gated_rmsnorm_fwd",
    "gated_rmsnorm_bwd",
    "mss_gated_rmsnorm_bwd_workspace_size",
    "add_rmsnorm_fwd",
    "add_rmsnorm_bwd",
    "mss_add_rmsnorm_bwd_workspace_size",
)


class ScanArgs(ctypes.Structure):
    """Mirror of ``mss_scan_args``."""
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("dim", ctypes.c_int64),
        ("dstate", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("in_dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int),
        ("u", ctypes.c_void_p),
        ("delta", ctypes.c_void_p),
        ("A", ctypes.c_void_p),
        ("B", ctypes.c_void_p),
        ("C", ctypes.c_void_p),
        ("D", ctypes.c_void_p),
        ("z", ctypes.c_void_p),
        ("delta_bias", ctypes.c_void_p),
        ("delta_softplus", ctypes.c_int),
        ("h0", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("last_state", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("plan_splits", ctypes.c_int),
        ("plan_chunk_steps", ctypes.c_int),
        ("test_flags", ctypes.c_uint),
        ("spin_timeout_ns", ctypes.c_int64),
        ("stride_u", ctypes.c_int64 * 2),
        ("stride_delta", ctypes.c_int64 * 2),
        ("stride_z", ctypes.c_int64 * 2),
        ("stride_B", ctypes.c_int64 * 2),
        ("stride_C", ctypes.c_int64 * 2),
        ("stride_y", ctypes.c_int64 * 2),
        ("cu_seqlens", ctypes.c_void_p),
        ("num_seqs", ctypes.c_int64),
        ("trapezoid", ctypes.c_int),
        ("checkpoints", ctypes.c_void_p),
    ]


class UpdateArgs(ctypes.Structure):
    """Mirror of ``mss_update_args``."""
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("dim", ctypes.c_int64),
        ("dstate", ctypes.c_int64),
        ("in_dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int),
        ("state", ctypes.c_void_p),
        ("x", ctypes.c_void_p),
        ("dt", ctypes.c_void_p),
        ("A", ctypes.c_void_p),
        ("B", ctypes.c_void_p),
        ("C", ctypes.c_void_p),
        ("D", ctypes.c_void_p),
        ("z", ctypes.c_void_p),
        ("dt_bias", ctypes.c_void_p),
        ("dt_softplus", ctypes.c_int),
        ("y", ctypes.c_void_p),
    ]


class ScanBwdArgs(ctypes.Structure):
    """Mirror of ``mss_scan_bwd_args``."""
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("dim", ctypes.c_int64),
        ("dstate", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("in_dtype", ctypes.c_int),
    ] + [(name, ctypes.c_void_p) for name in (
        "u", "delta", "A", "B", "C", "D", "z", "delta_bias")] + [
        ("delta_softplus", ctypes.c_int),
    ] + [(name, ctypes.c_void_p) for name in (
        "h0", "dy", "d_last", "du", "ddelta", "dA", "dB", "dC", "dD", "dz",
        "ddelta_bias", "dh0", "checkpoints", "workspace")] + [
        ("workspace_bytes", ctypes.c_size_t),
    ] + [("stride_" + name, ctypes.c_int64 * 2) for name in (
        "u", "delta", "z", "B", "C", "dy")] + [
        ("cu_seqlens", ctypes.c_void_p),
        ("num_seqs", ctypes.c_int64),
    ]


class SsdArgs(ctypes.Structure):
    """Mirror of ``mss_ssd_args``."""
    _fields_ = [(name, ctypes.c_int64) for name in (
        "batch", "seqlen", "nheads", "headdim", "ngroups", "dstate")] + [
        ("in_dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int),
    ] + [(name, ctypes.c_void_p) for name in (
        "x", "dt", "A", "B", "C", "D", "z", "dt_bias")] + [
        ("dt_softplus", ctypes.c_int),
    ] + [(name, ctypes.c_void_p) for name in ("h0", "y", "last_state")] + [
        ("spin_timeout_ns", ctypes.c_uint64),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class DeltaArgs(ctypes.Structure):
    """Mirror of ``mss_delta_args``."""
    _fields_ = [(name, ctypes.c_int64) for name in (
        "batch", "seqlen", "nheads", "headdim", "ngroups", "dstate")] + [
        ("in_dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int),
    ] + [(name, ctypes.c_void_p) for name in (
        "q", "k", "v", "dt", "A", "beta", "dt_bias")] + [
        ("dt_softplus", ctypes.c_int),
        ("beta_sigmoid", ctypes.c_int),
        ("scale", ctypes.c_float),
    ] + [(name, ctypes.c_void_p) for name in ("h0", "y", "last_state")] + [
        ("stride_" + name, ctypes.c_int64 * 3) for name in (
            "q", "k", "v", "dt", "beta", "y")] + [
        ("cu_seqlens", ctypes.c_void_p),
        ("num_seqs", ctypes.c_int64),
        ("plan", ctypes.c_int),
        ("spin_timeout_ns", ctypes.c_uint64),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class DeltaUpdateArgs(ctypes.Structure):
    """Mirror of ``mss_delta_update_args``."""
    _fields_ = [(name, ctypes.c_int64) for name in (
        "batch", "nheads", "headdim", "ngroups", "dstate")] + [
        ("in_dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int),
    ] + [(name, ctypes.c_void_p) for name in (
        "state", "q", "k", "v", "dt", "A", "beta", "dt_bias")] + [
        ("dt_softplus", ctypes.c_int),
        ("beta_sigmoid", ctypes.c_int),
        ("scale", ctypes.c_float),
        ("y", ctypes.c_void_p),
    ] + [("stride_" + name, ctypes.c_int64 * 2) for name in (
        "q", "k", "v", "dt", "beta", "y")]


class GatedNormArgs(ctypes.Structure):
    """Mirror of ``mss_gated_norm_args``."""
    _fields_ = [(name, ctypes.c_int64) for name in ("rows", "width", "group_size")] + [
        ("dtype", ctypes.c_int),
        ("norm_before_gate", ctypes.c_int),
        ("shared_weight", ctypes.c_int),
        ("eps", ctypes.c_float),
    ] + [(name, ctypes.c_void_p) for name in (
        "x", "z", "weight", "y", "dy", "dx", "dz", "dweight")] + [
        ("stride_" + name, ctypes.c_int64) for name in ("x", "z", "y", "dy", "dx", "dz")] + [
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class AddNormArgs(ctypes.Structure):
    """Mirror of ``mss_add_norm_args``."""
    _fields_ = [(name, ctypes.c_int64) for name in ("rows", "width")] + [
        ("dtype", ctypes.c_int),
        ("res_dtype", ctypes.c_int),
        ("eps", ctypes.c_float),
    ] + [(name, ctypes.c_void_p) for name in (
        "x", "residual", "scale", "weight", "y", "residual_out", "dy", "dresidual_out",
        "dx", "dresidual", "dweight", "dscale")] + [
        ("stride_" + name, ctypes.c_int64) for name in (
            "x", "residual", "y", "residual_out", "dy", "dresidual_out", "dx", "dresidual")] + [
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class MssError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)}")


_lib = None
_lock = threading.Lock()


def _bind(lib):
    P = ctypes.POINTER
    lib.mss_scan_workspace_size.argtypes = [P(ScanArgs), P(ctypes.c_size_t)]
    lib.mss_scan_workspace_size.restype = ctypes.c_int
    lib.mamba_selective_scan_fwd.argtypes = [P(ScanArgs), ctypes.c_void_p]
    lib.mamba_selective_scan_fwd.restype = ctypes.c_int
    lib.mss_scan_status.argtypes = [P(ScanArgs), ctypes.c_void_p]
    lib.mss_scan_status.restype = ctypes.c_int
    lib.mamba_selective_scan_fwd_noalloc.argtypes = [P(ScanArgs), ctypes.c_void_p]
    lib.mamba_selective_scan_fwd_noalloc.restype = ctypes.c_int
    lib.mss_scan_noalloc_status.argtypes = [P(ScanArgs), ctypes.c_void_p]
    lib.mss_scan_noalloc_status.restype = ctypes.c_int
    lib.selective_state_update.argtypes = [P(UpdateArgs), ctypes.c_void_p]
    lib.selective_state_update.restype = ctypes.c_int
    lib.mss_scan_bwd_workspace_size.argtypes = [P(ScanBwdArgs), P(ctypes.c_size_t)]
    lib.mss_scan_bwd_workspace_size.restype = ctypes.c_int
    lib.mamba_selective_scan_bwd.argtypes = [P(ScanBwdArgs), ctypes.c_void_p]
    lib.mamba_selective_scan_bwd.restype = ctypes.c_int
    lib.mss_status_string.argtypes = [ctypes.c_int]
    lib.mss_status_string.restype = ctypes.c_char_p
    lib.mss_ssd_workspace_size.argtypes = [P(SsdArgs), P(ctypes.c_size_t)]
    lib.mss_ssd_workspace_size.restype = ctypes.c_int
    lib.mamba2_ssd_fwd.argtypes = [P(SsdArgs), ctypes.c_void_p]
    lib.mamba2_ssd_fwd.restype = ctypes.c_int
    lib.mss_ssd_status.argtypes = [ctypes.c_void_p]
    lib.mss_ssd_status.restype = ctypes.c_int
    for name, args in (("gated_delta_fwd", DeltaArgs), ("gated_delta_update", DeltaUpdateArgs),
                       ("gated_rmsnorm_fwd", GatedNormArgs), ("gated_rmsnorm_bwd", GatedNormArgs),
                       ("add_rmsnorm_fwd", AddNormArgs), ("add_rmsnorm_bwd", AddNormArgs)):
        getattr(lib, name).argtypes = [P(args), ctypes.c_void_p]
        getattr(lib, name).restype = ctypes.c_int
    lib.mss_gated_delta_status.argtypes = [ctypes.c_void_p]
    lib.mss_gated_delta_status.restype = ctypes.c_int
    for name, args in (("mss_gated_delta_workspace_size", DeltaArgs),
                       ("mss_gated_rmsnorm_bwd_workspace_size", GatedNormArgs),
                       ("mss_add_rmsnorm_bwd_workspace_size", AddNormArgs)):
        getattr(lib, name).argtypes = [P(args), P(ctypes.c_size_t)]
        getattr(lib, name).restype = ctypes.c_int
    lib.mss_abi_version.argtypes = []
    lib.mss_abi_version.restype = ctypes.c_int
    return lib


def _open(path: str):
    if not os.path.exists(path):
        raise RuntimeError(
            f"CUDA library {path} is missing; build it with "
            "`python -m selective_state_space_48_b200.builder`")
    lib = _bind(ctypes.CDLL(path))
    if lib.mss_abi_version() != ABI_VERSION:
        raise RuntimeError(
            f"{path} has ABI version {lib.mss_abi_version()}, "
            f"this binding expects {ABI_VERSION}; rebuild it")
    return lib


def load_library():
    """Load libsss48.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            _lib = _open(LIB_PATH)
    return _lib


_debug_lib = None


def load_debug_library():
    """Load the checked build libsss48_debug.so (``builder --debug``): the
    same entry points with device-side bounds checks that report an access
    outside its tensor as MSS_ERR_INVALID_ARG through the status calls."""
    global _debug_lib
    with _lock:
        if _debug_lib is None:
            _debug_lib = _open(_build.DEBUG_LIB_PATH)
    return _debug_lib


def status_string(code: int) -> str:
    return load_library().mss_status_string(int(code)).decode()


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return MSS_F32
    if t == torch.bfloat16:
        return MSS_BF16
    raise TypeError(f"unsupported dtype {t}; use float32 or bfloat16")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_cuda(name, t, dtype=None, shape=None, strided=False):
    """Type, dtype and shape checks; ``strided`` tensors may be views whose
    last (time) dimension is contiguous, all others must be contiguous."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if strided:
        if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
            raise ValueError(f"{name} must be a 3-d view with a contiguous last dimension")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _under(stream, like, call, *args, **kw):
    """``call`` with ``stream`` as the current one.  What it allocates is then
    that stream's own memory, in that stream's order: from the current
    stream's, it could be a block that its kernels still read or write.  The
    results are recorded on the caller's stream, which is to use and drop
    them."""
    if not isinstance(like, torch.Tensor) or not like.is_cuda:
        return call(*args, **kw)  # refuses them
    if stream.device != like.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {like.device}")
    caller = torch.cuda.current_stream(like.device)
    with torch.cuda.stream(stream):
        out = call(*args, **kw)
    if caller != stream:
        outs = out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else [out]
        for t in outs:
            if t is not None:
                t.record_stream(caller)
    return out


def make_scan_args(u, delta, A, B, C, D=None, z=None, delta_bias=None,
                   delta_softplus=True, h0=None, y=None, last_state=None,
                   workspace=None, plan_splits=0, test_flags=0,
                   spin_timeout_ns=0, cu_seqlens=None, trapezoid=False,
                   checkpoints=None) -> ScanArgs:
    batch, dim, L = u.shape
    N = A.shape[1]
    ind = u.dtype
    _check_cuda("u", u, ind, strided=True)
    _check_cuda("delta", delta, ind, (batch, dim, L), strided=True)
    _check_cuda("A", A, torch.float32, (dim, N))
    _check_cuda("B", B, ind, (batch, N, L), strided=True)
    _check_cuda("C", C, ind, (batch, N, L), strided=True)
    _check_cuda("D", D, torch.float32, (dim,))
    _check_cuda("z", z, ind, (batch, dim, L), strided=True)
    _check_cuda("delta_bias", delta_bias, torch.float32, (dim,))
    _check_cuda("h0", h0, torch.float32, (batch, dim, N))
    _check_cuda("last_state", last_state, torch.float32, (batch, dim, N))
    if y is not None:
        _check_cuda("y", y, None, (batch, dim, L), strided=True)
    a = ScanArgs()
    a.batch, a.dim, a.dstate, a.seqlen = batch, dim, N, L
    a.in_dtype = _dtype_code(ind)
    a.out_dtype = _dtype_code(y.dtype) if y is not None else MSS_F32
    a.u, a.delta, a.A, a.B, a.C = (_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C))
    a.D, a.z, a.delta_bias = _ptr(D), _ptr(z), _ptr(delta_bias)
    a.delta_softplus = 1 if delta_softplus else 0
    a.h0, a.y, a.last_state = _ptr(h0), _ptr(y), _ptr(last_state)
    if workspace is not None:
        a.workspace = workspace.data_ptr()
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    a.plan_splits = int(plan_splits)
    a.plan_chunk_steps = 0
    a.test_flags = int(test_flags)
    a.spin_timeout_ns = int(spin_timeout_ns)
    a.trapezoid = 1 if trapezoid else 0
    if checkpoints is not None:
        _check_cuda("checkpoints", checkpoints, torch.float32)
        a.checkpoints = checkpoints.data_ptr()
    if cu_seqlens is not None:
        _check_cuda("cu_seqlens", cu_seqlens, torch.int32)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must hold num_seqs + 1 >= 2 offsets")
        a.cu_seqlens = cu_seqlens.data_ptr()
        a.num_seqs = cu_seqlens.numel() - 1
    for name, t in (("u", u), ("delta", delta), ("z", z), ("B", B), ("C", C), ("y", y)):
        if t is not None:
            getattr(a, "stride_" + name)[0] = t.stride(0)
            getattr(a, "stride_" + name)[1] = t.stride(1)
    return a


def scan_workspace_size(args: ScanArgs) -> int:
    n = ctypes.c_size_t(0)
    rc = load_library().mss_scan_workspace_size(ctypes.byref(args), ctypes.byref(n))
    if rc != MSS_OK:
        raise MssError(rc, "mss_scan_workspace_size")
    return int(n.value)


def alloc_workspace(nbytes: int, device) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    # torch allocations are 512-byte aligned, above the 256 the ABI needs
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def selective_scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None,
                       delta_softplus=True, h0=None, return_last_state=False,
                       out_dtype=torch.float32, y=None, last_state=None,
                       workspace=None, stream=None, plan_splits=0,
                       test_flags=0, spin_timeout_ns=0, check_status=False,
                       cu_seqlens=None, trapezoid=False, checkpoints=None):
    """Forward selective scan through ``mamba_selective_scan_fwd``.

    u, delta, z: (batch, dim, L); B, C: (batch, N, L) (float32 or bfloat16,
    all the same dtype); A: (dim, N), D, delta_bias: (dim,), h0:
    (batch, dim, N) float32.  u, delta, z, B, C and y may be views whose
    last dimension is contiguous.  ``cu_seqlens`` (int32 CUDA tensor of
    num_seqs + 1 offsets, 0 ... L) packs independent sequences into every
    row.  ``trapezoid`` selects the three-term trapezoidal update.
    ``checkpoints`` (from ``scan_checkpoints``) receives the states the
    backward pass starts from.  Returns
    y (batch, dim, L) in ``out_dtype`` (and the final state when
    ``return_last_state``).
    """
    if stream is not None:
        return _under(stream, u, selective_scan_fwd, u, delta, A, B, C, D, z, delta_bias,
                      delta_softplus, h0, return_last_state, out_dtype, y, last_state, workspace,
                      None, plan_splits, test_flags, spin_timeout_ns, check_status, cu_seqlens,
                      trapezoid, checkpoints)
    batch, dim, L = u.shape
    N = A.shape[1]
    if y is None:
        y = torch.empty((batch, dim, L), dtype=out_dtype, device=u.device)
    if return_last_state and last_state is None:
        last_state = torch.empty((batch, dim, N), dtype=torch.float32,
                                 device=u.device)
    args = make_scan_args(u, delta, A, B, C, D, z, delta_bias, delta_softplus,
                          h0, y, last_state, None, plan_splits, test_flags,
                          spin_timeout_ns, cu_seqlens, trapezoid, checkpoints)
    if workspace is None:
        workspace = alloc_workspace(scan_workspace_size(args), u.device)
    if workspace is not None:
        args.workspace = workspace.data_ptr()
        args.workspace_bytes = workspace.numel() * workspace.element_size()
    lib = load_library()
    rc = lib.mamba_selective_scan_fwd(ctypes.byref(args), _stream_handle(None))
    if rc != MSS_OK:
        raise MssError(rc, "mamba_selective_scan_fwd")
    if check_status:
        rc = lib.mss_scan_status(ctypes.byref(args), _stream_handle(None))
        if rc != MSS_OK:
            raise MssError(rc, "mss_scan_status")
    # keep the workspace alive until the stream has used it
    if workspace is not None:
        workspace.record_stream(torch.cuda.current_stream())
    return (y, last_state) if return_last_state else y


def scan_status(args: ScanArgs, stream=None) -> int:
    """Raw status code of the last scan that used ``args.workspace``."""
    return load_library().mss_scan_status(ctypes.byref(args), _stream_handle(stream))


def selective_state_update(state, x, dt, A, B, C, D=None, z=None, dt_bias=None,
                           dt_softplus=True, out_dtype=torch.float32, y=None,
                           stream=None):
    """One decode step through ``selective_state_update``; ``state``
    (batch, dim, N) float32 is updated in place.  x, dt, z: (batch, dim);
    B, C: (batch, N).  Returns y (batch, dim)."""
    if stream is not None:
        return _under(stream, state, selective_state_update, state, x, dt, A, B, C, D, z, dt_bias,
                      dt_softplus, out_dtype, y)
    batch, dim, N = state.shape
    ind = x.dtype
    _check_cuda("state", state, torch.float32)
    _check_cuda("x", x, ind, (batch, dim))
    _check_cuda("dt", dt, ind, (batch, dim))
    _check_cuda("A", A, torch.float32, (dim, N))
    _check_cuda("B", B, ind, (batch, N))
    _check_cuda("C", C, ind, (batch, N))
    _check_cuda("D", D, torch.float32, (dim,))
    _check_cuda("z", z, ind, (batch, dim))
    _check_cuda("dt_bias", dt_bias, torch.float32, (dim,))
    if y is None:
        y = torch.empty((batch, dim), dtype=out_dtype, device=state.device)
    _check_cuda("y", y, None, (batch, dim))
    a = UpdateArgs()
    a.batch, a.dim, a.dstate = batch, dim, N
    a.in_dtype, a.out_dtype = _dtype_code(ind), _dtype_code(y.dtype)
    a.state, a.x, a.dt = _ptr(state), _ptr(x), _ptr(dt)
    a.A, a.B, a.C, a.D, a.z = _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z)
    a.dt_bias = _ptr(dt_bias)
    a.dt_softplus = 1 if dt_softplus else 0
    a.y = _ptr(y)
    rc = load_library().selective_state_update(ctypes.byref(a), _stream_handle(None))
    if rc != MSS_OK:
        raise MssError(rc, "selective_state_update")
    return y


def make_ssd_args(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True,
                  h0=None, y=None, last_state=None, spin_timeout_ns=0) -> SsdArgs:
    batch, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    ind = x.dtype
    _check_cuda("x", x, ind)
    _check_cuda("dt", dt, ind, (batch, L, H))
    _check_cuda("A", A, torch.float32, (H,))
    _check_cuda("B", B, ind, (batch, L, G, N))
    _check_cuda("C", C, ind, (batch, L, G, N))
    _check_cuda("D", D, torch.float32, (H,))
    _check_cuda("z", z, ind, (batch, L, H, P))
    _check_cuda("dt_bias", dt_bias, torch.float32, (H,))
    _check_cuda("h0", h0, torch.float32, (batch, H, P, N))
    _check_cuda("last_state", last_state, torch.float32, (batch, H, P, N))
    if y is not None:
        _check_cuda("y", y, None, (batch, L, H, P))
    a = SsdArgs()
    a.batch, a.seqlen, a.nheads, a.headdim, a.ngroups, a.dstate = batch, L, H, P, G, N
    a.in_dtype = _dtype_code(ind)
    a.out_dtype = _dtype_code(y.dtype) if y is not None else MSS_F32
    a.x, a.dt, a.A, a.B, a.C = _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C)
    a.D, a.z, a.dt_bias = _ptr(D), _ptr(z), _ptr(dt_bias)
    a.dt_softplus = 1 if dt_softplus else 0
    a.h0, a.y, a.last_state = _ptr(h0), _ptr(y), _ptr(last_state)
    a.spin_timeout_ns = int(spin_timeout_ns)
    return a


def ssd_workspace_size(args: SsdArgs) -> int:
    """``mss_ssd_workspace_size``: bytes that let the SSD scan cut the last
    wave's sequences in two on the current device (0: nothing to cut)."""
    n = ctypes.c_size_t(0)
    rc = load_library().mss_ssd_workspace_size(ctypes.byref(args), ctypes.byref(n))
    if rc != MSS_OK:
        raise MssError(rc, "mss_ssd_workspace_size")
    return int(n.value)


def ssd_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, h0=None,
            return_last_state=False, out_dtype=torch.float32, y=None, last_state=None,
            stream=None, check_status=False, workspace=None):
    """Mamba-2 (SSD) chunked scan through ``mamba2_ssd_fwd``.

    x, z: (batch, L, nheads, headdim); dt: (batch, L, nheads); B, C:
    (batch, L, ngroups, dstate), all bfloat16; A, D, dt_bias: (nheads,)
    float32; h0: (batch, nheads, headdim, dstate) float32.  Returns y
    (batch, L, nheads, headdim) in ``out_dtype`` (and the final state when
    ``return_last_state``).  ``workspace``: None allocates what
    ``ssd_workspace_size`` asks for; False runs every sequence whole; a
    uint8 CUDA tensor is used as given.
    """
    if stream is not None:
        return _under(stream, x, ssd_fwd, x, dt, A, B, C, D, z, dt_bias, dt_softplus, h0,
                      return_last_state, out_dtype, y, last_state, None, check_status, workspace)
    batch, L, H, P = x.shape
    N = B.shape[3]
    if y is None:
        y = torch.empty((batch, L, H, P), dtype=out_dtype, device=x.device)
    if return_last_state and last_state is None:
        last_state = torch.empty((batch, H, P, N), dtype=torch.float32, device=x.device)
    args = make_ssd_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, h0, y, last_state)
    if workspace is None:
        workspace = alloc_workspace(ssd_workspace_size(args), x.device)
    if workspace is not None and workspace is not False:
        args.workspace = workspace.data_ptr()
        args.workspace_bytes = workspace.numel() * workspace.element_size()
    lib = load_library()
    rc = lib.mamba2_ssd_fwd(ctypes.byref(args), _stream_handle(None))
    if rc != MSS_OK:
        raise MssError(rc, "mamba2_ssd_fwd")
    # keep the workspace alive until the stream has used it
    if workspace is not None and workspace is not False:
        workspace.record_stream(torch.cuda.current_stream())
    if check_status:
        rc = lib.mss_ssd_status(_stream_handle(None))
        if rc != MSS_OK:
            raise MssError(rc, "mss_ssd_status")
    return (y, last_state) if return_last_state else y


def build(force: bool = False) -> str:
    return _build.build(force=force)


__all__ = [
    "selective_scan_fwd", "selective_state_update", "scan_workspace_size",
    "scan_status", "make_scan_args", "load_library", "status_string",
    "MssError", "ScanArgs", "UpdateArgs", "EXPORTED_SYMBOLS", "build",
    "ssd_fwd", "make_ssd_args", "SsdArgs", "ssd_workspace_size",
    "gated_delta_fwd", "gated_delta_update", "make_gated_delta_args", "gated_delta_status",
    "DeltaArgs", "DeltaUpdateArgs", "gated_rmsnorm_fwd", "gated_rmsnorm_bwd",
    "gated_rmsnorm_fn", "add_rmsnorm_fwd", "add_rmsnorm_bwd", "add_rmsnorm_fn",
    "GatedNormArgs", "AddNormArgs",
]


def selective_scan_bwd(u, delta, A, B, C, dy, D=None, z=None, delta_bias=None,
                       delta_softplus=True, h0=None, d_last=None, stream=None,
                       workspace=None, checkpoints=None, cu_seqlens=None):
    """Gradients of sum(dy * y) + sum(d_last * last_state) for the forward
    scan on the same inputs (and the same ``cu_seqlens`` packing), through
    ``mamba_selective_scan_bwd``.

    Inputs as for ``selective_scan_fwd`` (u, delta, z, B, C and dy may be
    3-d views with a contiguous last dimension); dy (batch, dim, L) and
    d_last (batch, dim, N) float32.  ``checkpoints`` written by the forward
    scan of the same inputs let the backward skip its forward sweep.
    ``workspace``: None allocates what ``mss_scan_bwd_workspace_size`` asks
    for (the checkpoints and the cut schedule's area); False passes none
    (valid with ``checkpoints``; every tile then runs whole); a uint8 CUDA
    tensor is used as given.  Returns a dict of float32 tensors du, ddelta,
    dA, dB, dC, dD, dz, ddelta_bias, dh0 (None for absent inputs).
    """
    if stream is not None:
        return _under(stream, u, selective_scan_bwd, u, delta, A, B, C, dy, D, z, delta_bias,
                      delta_softplus, h0, d_last, None, workspace, checkpoints, cu_seqlens)
    batch, dim, L = u.shape
    N = A.shape[1]
    ind = u.dtype
    rows = ("u", "delta", "B", "C", "z", "dy")  # may be strided views
    for name, t, dt, shape in (
            ("u", u, ind, None), ("delta", delta, ind, (batch, dim, L)),
            ("A", A, torch.float32, (dim, N)), ("B", B, ind, (batch, N, L)),
            ("C", C, ind, (batch, N, L)), ("D", D, torch.float32, (dim,)),
            ("z", z, ind, (batch, dim, L)),
            ("delta_bias", delta_bias, torch.float32, (dim,)),
            ("h0", h0, torch.float32, (batch, dim, N)),
            ("dy", dy, torch.float32, (batch, dim, L)),
            ("d_last", d_last, torch.float32, (batch, dim, N))):
        _check_cuda(name, t, dt, shape, strided=name in rows)
    dev = u.device
    f32 = dict(dtype=torch.float32, device=dev)
    g = {
        "du": torch.empty((batch, dim, L), **f32),
        "ddelta": torch.empty((batch, dim, L), **f32),
        "dA": torch.empty((dim, N), **f32),
        "dB": torch.empty((batch, N, L), **f32),
        "dC": torch.empty((batch, N, L), **f32),
        "dD": torch.empty((dim,), **f32) if D is not None else None,
        "dz": torch.empty((batch, dim, L), **f32) if z is not None else None,
        "ddelta_bias": torch.empty((dim,), **f32) if delta_bias is not None else None,
        "dh0": torch.empty((batch, dim, N), **f32),
    }
    a = ScanBwdArgs()
    a.batch, a.dim, a.dstate, a.seqlen = batch, dim, N, L
    a.in_dtype = _dtype_code(ind)
    a.u, a.delta, a.A, a.B, a.C = _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C)
    a.D, a.z, a.delta_bias = _ptr(D), _ptr(z), _ptr(delta_bias)
    a.delta_softplus = 1 if delta_softplus else 0
    a.h0, a.dy, a.d_last = _ptr(h0), _ptr(dy), _ptr(d_last)
    a.checkpoints = _ptr(checkpoints)
    for k, v in g.items():
        setattr(a, k, _ptr(v))
    for name, t in (("u", u), ("delta", delta), ("z", z), ("B", B), ("C", C), ("dy", dy)):
        if t is not None:
            getattr(a, "stride_" + name)[0] = t.stride(0)
            getattr(a, "stride_" + name)[1] = t.stride(1)
    if cu_seqlens is not None:
        _check_cuda("cu_seqlens", cu_seqlens, torch.int32)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must hold num_seqs + 1 >= 2 offsets")
        a.cu_seqlens = cu_seqlens.data_ptr()
        a.num_seqs = cu_seqlens.numel() - 1
    lib = load_library()
    n = ctypes.c_size_t(0)
    rc = lib.mss_scan_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n))
    if rc != MSS_OK:
        raise MssError(rc, "mss_scan_bwd_workspace_size")
    if workspace is None:
        # the checkpoints (without given ones) and the cut schedule's area
        workspace = alloc_workspace(int(n.value), dev)
    if workspace is False:  # no workspace (valid with checkpoints): no cut
        workspace = None
    if workspace is not None:
        a.workspace = workspace.data_ptr()
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    rc = lib.mamba_selective_scan_bwd(ctypes.byref(a), _stream_handle(None))
    if rc != MSS_OK:
        raise MssError(rc, "mamba_selective_scan_bwd")
    if workspace is not None:
        workspace.record_stream(torch.cuda.current_stream())
    return g


def scan_checkpoints(batch, dim, dstate, seqlen, device):
    """A buffer for the forward scan's checkpoints (float32, the checkpoint
    part of what ``mss_scan_bwd_workspace_size`` reports)."""
    groups = (dstate + 3) // 4
    groups = 1 if groups <= 1 else (2 if groups == 2 else 4)
    tiles = batch * ((dim + 31) // 32)
    nblk = (seqlen + 15) // 16
    # two arrays: the states at every block's start and entering its step 8
    return torch.empty(2 * tiles * nblk * 4 * groups * 32, dtype=torch.float32,
                       device=device)


class _NoSecond(torch.autograd.Function):
    @staticmethod
    def forward(ctx, t, *sources):
        return t.view_as(t)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the backward passes of selective_scan_fn, gated_rmsnorm_fn and "
                           "add_rmsnorm_fn cannot be differentiated again")


def _first_order(backward):
    """A backward whose gradients raise when they are differentiated: they
    hang on every tensor they were computed from.  (With torch's
    once_differentiable they hang on nothing when the upstream gradient is a
    constant, and a gradient penalty misses them without a word.)"""
    @functools.wraps(backward)
    def run(ctx, *grads):
        saved = ctx.saved_tensors  # (once: checkpointing allows no more)
        with torch.no_grad():
            out = backward(ctx, saved, *grads)
        if not torch.is_grad_enabled():
            return out
        sources = [t for t in (*saved, *grads) if t is not None and t.requires_grad]
        return tuple(None if t is None else _NoSecond.apply(t, *sources) for t in out)
    return run


class _SelectiveScanFn(torch.autograd.Function):
    """Autograd wrapper: forward through mamba_selective_scan_fwd (writing
    the backward's state checkpoints), backward through
    mamba_selective_scan_bwd starting from them."""

    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, z, delta_bias, delta_softplus, h0, cu_seqlens):
        batch, dim, L = u.shape
        # packed sequences: no forward checkpoints, the backward sweeps itself
        ck = (scan_checkpoints(batch, dim, A.shape[1], L, u.device)
              if cu_seqlens is None else None)
        y = selective_scan_fwd(u, delta, A, B, C, D=D, z=z, delta_bias=delta_bias,
                               delta_softplus=delta_softplus, h0=h0, checkpoints=ck,
                               cu_seqlens=cu_seqlens)
        ctx.delta_softplus = delta_softplus
        ctx.save_for_backward(u, delta, A, B, C, D, z, delta_bias, h0, ck, cu_seqlens)
        return y

    @staticmethod
    @_first_order
    def backward(ctx, saved, dy):
        u, delta, A, B, C, D, z, delta_bias, h0, ck, cu = saved
        g = selective_scan_bwd(u, delta, A, B, C, _rows_view(dy.float()), D=D, z=z,
                               delta_bias=delta_bias, delta_softplus=ctx.delta_softplus,
                               h0=h0, checkpoints=ck, cu_seqlens=cu)
        cast = lambda t, like: None if t is None else t.to(like.dtype)
        return (cast(g["du"], u), cast(g["ddelta"], delta), g["dA"], cast(g["dB"], B),
                cast(g["dC"], C), g["dD"], cast(g["dz"], z) if z is not None else None,
                g["ddelta_bias"], None, g["dh0"] if h0 is not None else None, None)


def _rows_view(t):
    """t itself when its last (time) dimension is contiguous, else a copy."""
    return t if t.dim() == 3 and (t.shape[2] <= 1 or t.stride(2) == 1) else t.contiguous()


def selective_scan_fn(u, delta, A, B, C, D=None, z=None, delta_bias=None,
                      delta_softplus=True, h0=None, cu_seqlens=None):
    """Differentiable selective scan: y (batch, dim, L) float32, with
    gradients for every tensor input through the CUDA backward pass.
    Inputs as for ``selective_scan_fwd``: u, delta, B, C and z may be views
    with a contiguous time dimension (the halves of an input projection,
    say), which both passes read in place; ``cu_seqlens`` packs independent
    sequences as for ``selective_scan_fwd``.  Gradients come back packed, in
    the inputs' dtypes (computed in float32)."""
    return _SelectiveScanFn.apply(_rows_view(u), _rows_view(delta), A, _rows_view(B),
                                  _rows_view(C), D, None if z is None else _rows_view(z),
                                  delta_bias, delta_softplus, h0, cu_seqlens)


# ------------------------------------------------------- gated delta rule


def _check_views(device, named):
    """CUDA tensors on `device` of the given dtype and shape, each with a
    contiguous last dimension (no shape: strides are free)."""
    for name, t, dtype, shape, inner in named:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if inner == "dense" and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if inner == "rows" and t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must have a contiguous last dimension")


# The calls below fill their argument structs with one struct.pack and look
# tensors over with plain comparisons, since a decode step's kernel takes a few
# microseconds and ctypes fields one each; whatever does not compare equal goes
# through the checks that say what is wrong.

_PACK = {ctypes.c_int64: "q", ctypes.c_int: "i", ctypes.c_float: "f", ctypes.c_void_p: "P",
         ctypes.c_uint64: "Q", ctypes.c_size_t: "N"}


def _packer(args_type):
    """``struct.pack`` of an argument struct's fields in order (native
    alignment, as in C)."""
    fmt = "@"
    for _, t in args_type._fields_:
        n = getattr(t, "_length_", None)
        fmt += _PACK[t] if n is None else f"{n}{_PACK[t._type_]}"
    pad = ctypes.sizeof(args_type) - _struct.calcsize(fmt)
    return _struct.Struct(fmt + (f"{pad}x" if pad else "")).pack


_entries = {}


def _entry(name):
    """The library function `name`, taking packed arguments."""
    fn = _entries.get(name)
    if fn is None:
        fn = load_library()[name]  # a handle of its own, apart from lib.<name>
        fn.argtypes, fn.restype = [ctypes.c_char_p, ctypes.c_void_p], ctypes.c_int
        _entries[name] = fn
    return fn


def _enqueue(name, packed, device):
    """On the device's current stream, with the device as the current one."""
    if torch._C._cuda_getDevice() == device.index:
        rc = _entry(name)(packed, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            rc = _entry(name)(packed, torch._C._cuda_getCurrentRawStream(device.index))
    if rc != MSS_OK:
        raise MssError(rc, name)


_Tensor = torch.Tensor


def _tensors(a, b, c, d):
    return (isinstance(a, _Tensor) and isinstance(b, _Tensor) and isinstance(c, _Tensor)
            and isinstance(d, _Tensor))


def _dense(t, dtype, device, shape):
    return t is None or (isinstance(t, _Tensor) and t.dtype is dtype and t.device == device
                         and t.shape == shape and t.is_contiguous())


def _new(like, dtype=None):
    """An uninitialised contiguous tensor of the shape and device of `like`."""
    if dtype is None or dtype is like.dtype:
        if like.is_contiguous():  # (half the time of torch.empty)
            return torch.empty_like(like)
        dtype = like.dtype
    return torch.empty(like.shape, dtype=dtype, device=like.device)


def _refuse_gradients(call, *inputs):
    """Raises where a gradient would be expected of a forward-only call."""
    for t in inputs:
        if t is not None and t.requires_grad:
            raise RuntimeError(f"{call} is forward only and an input requires a gradient: detach "
                               "it, or call under torch.no_grad()")


def _same(t, dtype, device, shape):
    return (isinstance(t, _Tensor) and t.dtype is dtype and t.device == device
            and t.shape == shape)


def _packed_sequences(cu_seqlens, device):
    """Their number, from the offsets."""
    _check_views(device, [("cu_seqlens", cu_seqlens, torch.int32, None, "dense")])
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must hold num_seqs + 1 >= 2 offsets")
    return cu_seqlens.shape[0] - 1


def _delta_values(q, k, v, dt, A, beta, dt_bias, dt_softplus, beta_sigmoid, scale, h0, y,
                  last_state, cu_seqlens, plan, spin_timeout_ns, workspace):
    """The values of ``mss_delta_args`` in order, after the checks."""
    if not isinstance(v, torch.Tensor) or not isinstance(q, torch.Tensor):
        raise TypeError("q and v must be CUDA tensors")
    if v.dim() != 4 or q.dim() != 4:
        raise ValueError("q, k and v must have the dimensions (batch, seqlen, heads, width)")
    batch, L, H, P = values = v.shape
    G, N = q.shape[2], q.shape[3]
    ind, dev, f32, cu = q.dtype, q.device, torch.float32, 0
    keys, heads, seqs = (batch, L, G, N), (batch, L, H), batch
    if cu_seqlens is not None:
        seqs, cu = _packed_sequences(cu_seqlens, dev), cu_seqlens.data_ptr()
        if batch != 1:
            raise ValueError("packed sequences need batch 1")
    states = (seqs, H, P, N)
    if not (_tensors(k, dt, beta, A) and q.is_cuda
            and ind is k.dtype is v.dtype is dt.dtype is beta.dtype
            and dev == k.device == v.device == dt.device == beta.device
            and q.shape == keys == k.shape and dt.shape == heads == beta.shape
            and q.stride()[3] == k.stride()[3] == v.stride()[3] == 1
            and (y is None or (_same(y, y.dtype, dev, values) and y.stride()[3] == 1))
            and _dense(A, f32, dev, (H,)) and _dense(dt_bias, f32, dev, (H,))
            and _dense(h0, f32, dev, states) and _dense(last_state, f32, dev, states)):
        _check_views(dev, [
            ("q", q, ind, keys, "rows"), ("k", k, ind, keys, "rows"),
            ("v", v, ind, values, "rows"), ("dt", dt, ind, heads, None),
            ("beta", beta, ind, heads, None), ("A", A, f32, (H,), "dense"),
            ("dt_bias", dt_bias, f32, (H,), "dense"), ("h0", h0, f32, states, "dense"),
            ("last_state", last_state, f32, states, "dense"), ("y", y, None, values, "rows")])
    return (
        batch, L, H, P, G, N, _dtype_code(ind), MSS_F32 if y is None else _dtype_code(y.dtype),
        q.data_ptr(), k.data_ptr(), v.data_ptr(), dt.data_ptr(), A.data_ptr(), beta.data_ptr(),
        0 if dt_bias is None else dt_bias.data_ptr(), bool(dt_softplus), bool(beta_sigmoid),
        N ** -0.5 if scale is None else float(scale), 0 if h0 is None else h0.data_ptr(),
        0 if y is None else y.data_ptr(), 0 if last_state is None else last_state.data_ptr(),
        *q.stride()[:3], *k.stride()[:3], *v.stride()[:3], *dt.stride(), *beta.stride(),
        *((0, 0, 0) if y is None else y.stride()[:3]), cu, seqs if cu else 0, int(plan),
        int(spin_timeout_ns), *workspace)


def _workspace(nbytes, device):
    if not nbytes:
        return None, 0
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr()


def _delta_room(a, device_index):
    """Workspace bytes of a call on this device (0 also for one that the call
    itself refuses)."""
    n = ctypes.c_size_t(0)
    with torch.cuda.device(device_index):
        load_library().mss_gated_delta_workspace_size(ctypes.byref(a), ctypes.byref(n))
    return int(n.value)


@functools.lru_cache(maxsize=1024)
def _delta_workspace_bytes(batch, seqlen, nheads, headdim, ngroups, dstate, seqs, plan,
                           device_index):
    """Workspace bytes of a call of dense bf16 tensors of these sizes."""
    a = DeltaArgs()
    a.batch, a.seqlen, a.nheads, a.headdim, a.ngroups = batch, seqlen, nheads, headdim, ngroups
    a.dstate, a.in_dtype, a.plan = dstate, MSS_BF16, plan
    a.cu_seqlens, a.num_seqs = (1 << 20, seqs) if seqs else (None, 0)
    for n, heads, width in (("q", ngroups, dstate), ("k", ngroups, dstate),
                            ("v", nheads, headdim)):
        getattr(a, "stride_" + n)[:] = (seqlen * heads * width, heads * width, width)
    return _delta_room(a, device_index)


_pack_delta = _packer(DeltaArgs)


def make_gated_delta_args(q, k, v, dt, A, beta, dt_bias=None, dt_softplus=True,
                          beta_sigmoid=True, scale=None, h0=None, y=None, last_state=None,
                          cu_seqlens=None, plan=MSS_DELTA_AUTO, spin_timeout_ns=0,
                          workspace=None) -> DeltaArgs:
    if workspace is not None:
        _check_views(q.device, [("workspace", workspace, torch.uint8, None, "dense")])
    return DeltaArgs.from_buffer_copy(_pack_delta(*_delta_values(
        q, k, v, dt, A, beta, dt_bias, dt_softplus, beta_sigmoid, scale, h0, y, last_state,
        cu_seqlens, plan, spin_timeout_ns,
        (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel()))))


def gated_delta_fwd(q, k, v, dt, A, beta, dt_bias=None, dt_softplus=True, beta_sigmoid=True,
                    scale=None, h0=None, return_last_state=False, out_dtype=torch.float32,
                    y=None, last_state=None, cu_seqlens=None, stream=None, check_status=False,
                    plan=MSS_DELTA_AUTO):
    """Gated delta rule over whole sequences through ``gated_delta_fwd``.

    q, k: (batch, L, ngroups, dstate); v: (batch, L, nheads, headdim); dt,
    beta: (batch, L, nheads), float32 or bfloat16, all the same; A, dt_bias:
    (nheads,) float32.  q, k, v and y may be views with a contiguous last
    dimension, dt and beta any views.  ``scale`` multiplies the readout
    (default dstate ** -0.5).  ``cu_seqlens`` (int32 CUDA tensor of
    num_seqs + 1 ascending offsets within 0 ... L) packs independent
    sequences into one row (batch 1); rows of y outside them are not
    written.  h0 and last_state: (sequences, nheads, headdim, dstate)
    float32, and may be one tensor; y must not overlap the inputs.  ``plan``:
    MSS_DELTA_AUTO goes by the length (of packed sequences by the average),
    MSS_DELTA_CHUNKED suits a pack of a long sequence and many short ones too,
    MSS_DELTA_RECURRENT keeps fp32 throughout.  With ``stream`` the call runs,
    and allocates, on that stream; the inputs have to be ready there.  Returns
    y (batch, L, nheads, headdim) in
    ``out_dtype`` (and the final states when ``return_last_state``).  Forward
    only: an input that requires a gradient is refused outside of
    ``torch.no_grad()``.
    """
    if stream is not None:
        return _under(stream, q, gated_delta_fwd, q, k, v, dt, A, beta, dt_bias, dt_softplus,
                      beta_sigmoid, scale, h0, return_last_state, out_dtype, y, last_state,
                      cu_seqlens, None, check_status, plan)
    if not isinstance(v, _Tensor) or not isinstance(q, _Tensor):
        raise TypeError("q and v must be CUDA tensors")
    if v.dim() != 4 or q.dim() != 4:
        raise ValueError("q, k and v must have the dimensions (batch, seqlen, heads, width)")
    if y is None:
        y = _new(v, out_dtype)
    if return_last_state and last_state is None:
        seqs = v.shape[0] if cu_seqlens is None else _packed_sequences(cu_seqlens, q.device)
        last_state = torch.empty((seqs, v.shape[2], v.shape[3], q.shape[-1]),
                                 dtype=torch.float32, device=v.device)
    values = _delta_values(q, k, v, dt, A, beta, dt_bias, dt_softplus, beta_sigmoid, scale, h0, y,
                           last_state, cu_seqlens, plan, 0, (0, 0))
    if torch.is_grad_enabled():
        _refuse_gradients("gated_delta_fwd", q, k, v, dt, A, beta, dt_bias, h0)
    ws = None
    if v.dtype is torch.bfloat16 and plan != MSS_DELTA_RECURRENT:
        at = q.data_ptr() | k.data_ptr() | v.data_ptr()
        for t in (h0, last_state):
            at |= 0 if t is None else t.data_ptr()
        if at & 15 == 0 and q.is_contiguous() and k.is_contiguous() and v.is_contiguous():
            nbytes = _delta_workspace_bytes(
                *v.shape, q.shape[2], q.shape[3],
                0 if cu_seqlens is None else cu_seqlens.shape[0] - 1, plan, v.device.index)
        else:
            nbytes = _delta_room(DeltaArgs.from_buffer_copy(_pack_delta(*values)), v.device.index)
        if nbytes:
            ws, pws = _workspace(nbytes, v.device)
            values = (*values[:-2], pws, nbytes)
    _enqueue("gated_delta_fwd", _pack_delta(*values), q.device)
    if check_status:
        with torch.cuda.device(q.device):
            rc = gated_delta_status()
        if rc != MSS_OK:
            raise MssError(rc, "mss_gated_delta_status")
    return (y, last_state) if return_last_state else y


def gated_delta_status(stream=None) -> int:
    """Raw status code of the chunked calls completed on this device since
    the last read (``mss_gated_delta_status``)."""
    return load_library().mss_gated_delta_status(_stream_handle(stream))


def gated_delta_update(state, q, k, v, dt, A, beta, dt_bias=None, dt_softplus=True,
                       beta_sigmoid=True, scale=None, out_dtype=torch.float32, y=None,
                       stream=None):
    """One decode step through ``gated_delta_update``; ``state`` (batch,
    nheads, headdim, dstate) float32 is updated in place.  q, k: (batch,
    ngroups, dstate); v: (batch, nheads, headdim); dt, beta: (batch, nheads);
    views, and inputs that require gradients, as for ``gated_delta_fwd``.
    Returns y (batch, nheads, headdim)."""
    if stream is not None:
        return _under(stream, q, gated_delta_update, state, q, k, v, dt, A, beta, dt_bias,
                      dt_softplus, beta_sigmoid, scale, out_dtype, y)
    if not _tensors(state, q, v, state):
        raise TypeError("state, q and v must be CUDA tensors")
    if state.dim() != 4 or q.dim() != 3:
        raise ValueError("state must be (batch, heads, headdim, dstate), q (batch, groups, dstate)")
    batch, H, P, N = shape = state.shape
    G, ind, dev, f32 = q.shape[1], q.dtype, q.device, torch.float32
    if y is None:
        y = _new(v, out_dtype)
    keys, values, heads = (batch, G, N), (batch, H, P), (batch, H)
    if not (_tensors(k, dt, beta, A) and isinstance(y, _Tensor) and q.is_cuda
            and ind is k.dtype is v.dtype is dt.dtype is beta.dtype
            and dev == k.device == v.device == dt.device == beta.device == y.device
            and q.shape == keys == k.shape and v.shape == values == y.shape
            and dt.shape == heads == beta.shape
            and q.stride()[2] == k.stride()[2] == v.stride()[2] == y.stride()[2] == 1
            and _dense(state, f32, dev, shape) and _dense(A, f32, dev, (H,))
            and _dense(dt_bias, f32, dev, (H,))):
        _check_views(dev, [
            ("state", state, f32, None, "dense"), ("q", q, ind, keys, "rows"),
            ("k", k, ind, keys, "rows"), ("v", v, ind, values, "rows"),
            ("dt", dt, ind, heads, None), ("beta", beta, ind, heads, None),
            ("A", A, f32, (H,), "dense"), ("dt_bias", dt_bias, f32, (H,), "dense"),
            ("y", y, None, values, "rows")])
    if torch.is_grad_enabled():
        _refuse_gradients("gated_delta_update", state, q, k, v, dt, A, beta, dt_bias)
    packed = _pack_update(
        batch, H, P, G, N, _dtype_code(ind), _dtype_code(y.dtype), state.data_ptr(),
        q.data_ptr(), k.data_ptr(), v.data_ptr(), dt.data_ptr(), A.data_ptr(), beta.data_ptr(),
        0 if dt_bias is None else dt_bias.data_ptr(), bool(dt_softplus), bool(beta_sigmoid),
        N ** -0.5 if scale is None else float(scale), y.data_ptr(), *q.stride()[:2],
        *k.stride()[:2], *v.stride()[:2], *dt.stride(), *beta.stride(), *y.stride()[:2])
    _enqueue("gated_delta_update", packed, dev)
    return y


_pack_update = _packer(DeltaUpdateArgs)


# ------------------------------------------- norms before and after a block


def _rows_of(name, t):
    """(rows, row stride) of a tensor (..., width) whose leading dimensions
    step evenly through memory."""
    if t.dim() < 1 or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must have a contiguous last dimension")
    rows, stride = 1, None
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride = st
        elif st != rows * stride:
            raise ValueError(f"the leading dimensions of {name} must be one run of rows at an "
                             "even stride")
        rows *= n
    return rows, (t.shape[-1] if stride is None else stride)


def _norm_rows(device, shape, named):
    """[pointer, ...] and [row stride, ...] of the (..., width) tensors of a
    norm call (0 for None)."""
    ptrs, strides, width = [], [], shape[-1]
    for name, t, dtype in named:
        if t is None:
            ptrs.append(0)
            strides.append(0)
            continue
        if not (isinstance(t, _Tensor) and t.is_cuda and t.dtype is dtype and t.device == device
                and t.shape == shape):
            _check_views(device, [(name, t, dtype, shape, "rows")])
        ptrs.append(t.data_ptr())
        strides.append(width if t.is_contiguous() else _rows_of(name, t)[1])
    return ptrs, strides


@functools.lru_cache(maxsize=1024)
def _norm_workspace_bytes(name, rows, width, group, sums, device_index):
    """Workspace bytes of a norm's backward of these sizes on this device."""
    a = GatedNormArgs() if name == "gated" else AddNormArgs()
    a.rows, a.width = rows, width
    if name == "gated":
        a.group_size, a.dweight = group, 1 if sums else None
    else:
        a.dweight, a.dscale = (1 if sums & 1 else None), (1 if sums & 2 else None)
    fn = f"mss_{name}_rmsnorm_bwd_workspace_size"
    n = ctypes.c_size_t(0)
    with torch.cuda.device(device_index):
        rc = getattr(load_library(), fn)(ctypes.byref(a), ctypes.byref(n))
    if rc != MSS_OK:
        raise MssError(rc, fn)
    return int(n.value)


def _gated_norm_sizes(x, weight, group_size):
    """rows, width, group size, and whether the groups share the weight."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise TypeError("x must be a CUDA tensor with at least one dimension")
    width = x.shape[-1]
    gs = width if group_size is None else int(group_size)
    if gs < 1 or width % gs:
        raise ValueError(f"group_size {gs} must divide the width {width}")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 1 or \
            weight.shape[0] not in (width, gs):
        raise ValueError(f"weight must have {width} or {gs} entries")
    if not _dense(weight, torch.float32, x.device, weight.shape):
        _check_views(x.device, [("weight", weight, torch.float32, None, "dense")])
    return x.numel() // max(width, 1), width, gs, weight.shape[0] == gs


_pack_gated_norm = _packer(GatedNormArgs)
_pack_add_norm = _packer(AddNormArgs)


def gated_rmsnorm_fwd(x, z, weight, eps=1e-5, group_size=None, norm_before_gate=False, y=None,
                      stream=None):
    """RMS norm after a block, gated by silu(z), through ``gated_rmsnorm_fwd``.

    x, z: (..., width) float32 or bfloat16, rows contiguous and evenly
    spaced; weight float32 with ``width`` entries, or ``group_size`` entries
    shared by every group.  The norm is taken over each group of
    ``group_size`` channels (default: the width), of x o silu(z), or of x
    with the gate applied after it (``norm_before_gate``).  Returns y like x.
    """
    if stream is not None:
        return _under(stream, x, gated_rmsnorm_fwd, x, z, weight, eps, group_size,
                      norm_before_gate, y)
    rows, width, gs, shared = _gated_norm_sizes(x, weight, group_size)
    dev, kind, shape = x.device, x.dtype, x.shape
    if y is None:
        y = _new(x)
    (px, pz, py), (sx, sz, sy) = _norm_rows(dev, shape, (("x", x, kind), ("z", z, kind),
                                                         ("y", y, kind)))
    _enqueue("gated_rmsnorm_fwd", _pack_gated_norm(
        rows, width, gs, _dtype_code(kind), bool(norm_before_gate), shared, eps, px, pz,
        weight.data_ptr(), py, 0, 0, 0, 0, sx, sz, sy, 0, 0, 0, 0, 0), dev)
    return y


def gated_rmsnorm_bwd(x, z, weight, dy, eps=1e-5, group_size=None, norm_before_gate=False,
                      need_dweight=True, stream=None):
    """Gradients of sum(dy * y) for ``gated_rmsnorm_fwd`` on the same inputs.
    Returns a dict of dx, dz (x's dtype) and dweight (float32, like weight,
    None unless ``need_dweight``)."""
    if stream is not None:
        return _under(stream, x, gated_rmsnorm_bwd, x, z, weight, dy, eps, group_size,
                      norm_before_gate, need_dweight)
    rows, width, gs, shared = _gated_norm_sizes(x, weight, group_size)
    dev, kind, shape = x.device, x.dtype, x.shape
    dx, dz = _new(x), _new(x)
    dw = torch.empty_like(weight) if need_dweight else None
    (px, pz, pdy, pdx, pdz), (sx, sz, sdy, sdx, sdz) = _norm_rows(dev, shape, (
        ("x", x, kind), ("z", z, kind), ("dy", dy, kind), ("dx", dx, kind), ("dz", dz, kind)))
    nbytes = _norm_workspace_bytes("gated", rows, width, gs, 1, dev.index) if need_dweight else 0
    ws, pws = _workspace(nbytes, dev)
    _enqueue("gated_rmsnorm_bwd", _pack_gated_norm(
        rows, width, gs, _dtype_code(kind), bool(norm_before_gate), shared, eps, px, pz,
        weight.data_ptr(), 0, pdy, pdx, pdz, dw.data_ptr() if need_dweight else 0, sx, sz, 0, sdy,
        sdx, sdz, pws, nbytes), dev)
    return {"dx": dx, "dz": dz, "dweight": dw}


def _add_norm_sizes(like, weight, scale):
    if not isinstance(like, torch.Tensor) or like.dim() < 1:
        raise TypeError("x and the residual must be CUDA tensors with at least one dimension")
    width, dev, f32 = like.shape[-1], like.device, torch.float32
    if weight is None or not _dense(weight, f32, dev, (width,)) or \
            not _dense(scale, f32, dev, (width,)):
        if not isinstance(weight, torch.Tensor):
            raise TypeError("weight must be a CUDA tensor")
        _check_views(dev, [("weight", weight, f32, (width,), "dense"),
                           ("scale", scale, f32, (width,), "dense")])
    return like.numel() // max(width, 1), width


def add_rmsnorm_fwd(x, residual, weight, scale=None, eps=1e-5, residual_dtype=None, y=None,
                    residual_out=None, stream=None):
    """Residual sum and RMS norm before a block, through ``add_rmsnorm_fwd``:
    r = residual + scale o x and y = r / sqrt(mean(r^2) + eps) o weight.

    x: (..., width) float32 or bfloat16; residual: the same shape, float32
    or x's dtype, or None (a stream's first block; r then has
    ``residual_dtype``, default float32); weight, scale (optional):
    (width,) float32.  ``residual_out`` may be the residual itself.  Returns
    (y in x's dtype, r in the residual's dtype).
    """
    if stream is not None:
        return _under(stream, x, add_rmsnorm_fwd, x, residual, weight, scale, eps,
                      residual_dtype, y, residual_out)
    rows, width = _add_norm_sizes(x, weight, scale)
    dev, kind, shape = x.device, x.dtype, x.shape
    if residual_out is None:
        rd = residual.dtype if residual is not None else residual_dtype or torch.float32
        residual_out = _new(x, rd)
    rd = residual_out.dtype
    if y is None:
        y = _new(x)
    (px, pr, py, po), (sx, sr, sy, so) = _norm_rows(dev, shape, (
        ("x", x, kind), ("residual", residual, rd), ("y", y, kind),
        ("residual_out", residual_out, rd)))
    _enqueue("add_rmsnorm_fwd", _pack_add_norm(
        rows, width, _dtype_code(kind), _dtype_code(rd), eps, px, pr,
        0 if scale is None else scale.data_ptr(), weight.data_ptr(), py, po, 0, 0, 0, 0, 0, 0,
        sx, sr, sy, so, 0, 0, 0, 0, 0, 0), dev)
    return y, residual_out


def add_rmsnorm_bwd(residual_out, weight, dy, dresidual_out=None, x=None, scale=None, eps=1e-5,
                    need_dweight=True, need_dscale=True, stream=None):
    """Gradients for ``add_rmsnorm_fwd`` from its stored sum ``residual_out``:
    of sum(dy * y) + sum(dresidual_out * residual_out).  x is needed for
    dscale only.  Returns a dict of dx (dy's dtype), dresidual (the
    residual's dtype), dweight and dscale (float32; None where not asked for
    or there is no scale)."""
    if stream is not None:
        return _under(stream, residual_out, add_rmsnorm_bwd, residual_out, weight, dy,
                      dresidual_out, x, scale, eps, need_dweight, need_dscale)
    rows, width = _add_norm_sizes(residual_out, weight, scale)
    if not isinstance(dy, torch.Tensor):
        raise TypeError("dy must be a CUDA tensor")
    rd, kind, shape, dev = residual_out.dtype, dy.dtype, residual_out.shape, residual_out.device
    need_dscale = need_dscale and scale is not None
    if need_dscale and x is None:
        raise ValueError("dscale needs x")
    dx, dres = _new(residual_out, kind), _new(residual_out)
    dw = torch.empty_like(weight) if need_dweight else None
    ds = torch.empty_like(scale) if need_dscale else None
    (po, pdy, pdo, px, pdx, pdr), (so, sdy, sdo, sx, sdx, sdr) = _norm_rows(dev, shape, (
        ("residual_out", residual_out, rd), ("dy", dy, kind), ("dresidual_out", dresidual_out, rd),
        ("x", x if need_dscale else None, kind), ("dx", dx, kind), ("dresidual", dres, rd)))
    sums = (1 if need_dweight else 0) + (2 if need_dscale else 0)
    nbytes = _norm_workspace_bytes("add", rows, width, 0, sums, dev.index) if sums else 0
    ws, pws = _workspace(nbytes, dev)
    _enqueue("add_rmsnorm_bwd", _pack_add_norm(
        rows, width, _dtype_code(kind), _dtype_code(rd), eps, px, 0,
        0 if scale is None else scale.data_ptr(), weight.data_ptr(), 0, po, pdy, pdo, pdx, pdr,
        dw.data_ptr() if need_dweight else 0, ds.data_ptr() if need_dscale else 0,
        sx, 0, 0, so, sdy, sdo, sdx, sdr, pws, nbytes), dev)
    return {"dx": dx, "dresidual": dres, "dweight": dw, "dscale": ds}


def _even_rows(t):
    """t itself when its rows are contiguous and evenly spaced, else a copy."""
    try:
        _rows_of("t", t)
        return t
    except ValueError:
        return t.contiguous()


class _GatedRmsNormFn(torch.autograd.Function):
    """Autograd wrapper of gated_rmsnorm_fwd and gated_rmsnorm_bwd."""

    @staticmethod
    def forward(ctx, x, z, weight, eps, group_size, norm_before_gate):
        ctx.kw = dict(eps=eps, group_size=group_size, norm_before_gate=norm_before_gate)
        ctx.save_for_backward(x, z, weight)
        return gated_rmsnorm_fwd(x, z, weight, **ctx.kw)

    @staticmethod
    @_first_order
    def backward(ctx, saved, dy):
        x, z, weight = saved
        g = gated_rmsnorm_bwd(x, z, weight, _even_rows(dy), need_dweight=ctx.needs_input_grad[2],
                              **ctx.kw)
        return g["dx"], g["dz"], g["dweight"], None, None, None


def gated_rmsnorm_fn(x, z, weight, eps=1e-5, group_size=None, norm_before_gate=False):
    """Differentiable ``gated_rmsnorm_fwd``, with gradients for x, z and
    weight through the CUDA backward pass."""
    return _GatedRmsNormFn.apply(_even_rows(x), _even_rows(z), weight, eps, group_size,
                                 norm_before_gate)


class _AddRmsNormFn(torch.autograd.Function):
    """Autograd wrapper of add_rmsnorm_fwd and add_rmsnorm_bwd."""

    @staticmethod
    def forward(ctx, x, residual, weight, scale, eps, residual_dtype):
        y, res = add_rmsnorm_fwd(x, residual, weight, scale, eps, residual_dtype)
        ctx.eps, ctx.x_dtype = eps, x.dtype
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x if scale is not None else None, weight, scale, res)
        return y, res

    @staticmethod
    @_first_order
    def backward(ctx, saved, dy, dres):
        x, weight, scale, res = saved
        if dy is None:
            dy = torch.zeros(res.shape, dtype=ctx.x_dtype, device=res.device)
        g = add_rmsnorm_bwd(res, weight, _even_rows(dy),
                            None if dres is None else _even_rows(dres), x, scale, ctx.eps,
                            need_dweight=ctx.needs_input_grad[2],
                            need_dscale=ctx.needs_input_grad[3])
        return (g["dx"], g["dresidual"] if ctx.needs_input_grad[1] else None, g["dweight"],
                g["dscale"], None, None)


def add_rmsnorm_fn(x, residual, weight, scale=None, eps=1e-5, residual_dtype=None):
    """Differentiable ``add_rmsnorm_fwd``: (y, residual_out), with gradients
    for x, residual, weight and scale through the CUDA backward pass."""
    return _AddRmsNormFn.apply(_even_rows(x), None if residual is None else _even_rows(residual),
                               weight, scale, eps, residual_dtype)
