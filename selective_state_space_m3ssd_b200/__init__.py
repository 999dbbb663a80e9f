"""B200-native Mamba-3 SISO selective scan: Python binding of ``libm3ssd``.

The binding only marshals arguments (device pointers, sizes, the current CUDA
stream) into the C ABI declared in ``include/m3ssd.h``; every step of the scan
runs in the library's CUDA kernels.  Importing this package does not load the
library; the first call does, and raises ``LibraryMissing`` if it has not been
built (``python -m selective_state_space_m3ssd_b200.build``).  There is no
other implementation behind these functions.

Beside the scan, its step and its block: the residual addition and RMS norm
(:func:`add_rmsnorm`), microscaled tensors and their product (:func:`mx_quant`,
:func:`gemm_mx`) and the decode step on a cache held in 8 bits (:func:`quant_cache`,
:func:`step_q8`).
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libm3ssd.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_NONFINITE, ERR_TIMEOUT = range(7)
F32, BF16 = 0, 1
CHECK_FINITE = 1  # m3ssd_dims.flags: scan the outputs for NaN / infinity

_lib = None
_lock = threading.Lock()


class LibraryMissing(RuntimeError):
    pass


class M3SSDError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


class M3SSDInvalidArgument(M3SSDError, ValueError):
    pass


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("chunk", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class FwdExtra(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("angle0", "xprev0", "bprev0", "angleT", "xprevT", "bprevT")]


GRAD_NAMES = ("dX", "dlogdecay", "dbeta", "dgamma", "dB", "dC", "dtheta", "dD", "dh0",
              "dangle0", "dxprev0", "dbprev0")


class BwdGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in GRAD_NAMES]


class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("angle", "ssm", "x_prev", "b_prev")]


class NormDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("width", ctypes.c_int64), ("x_dtype", ctypes.c_int32),
                ("res_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_uint32)]


class Mx(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("reserved", ctypes.c_uint32),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class CacheQ8(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("angle", "ssm", "scale", "x_prev", "b_prev")]


class BlockDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("batch", "seqlen", "d_model", "nheads", "headdim", "dstate", "ngroups")]


BLOCK_WEIGHT_NAMES = ("W_in", "W_out", "dt_bias", "A_log", "D", "B_norm_w", "C_norm_w",
                      "B_bias", "C_bias")


class BlockWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in BLOCK_WEIGHT_NAMES] + [("eps", ctypes.c_float)]


def load(path: str | None = None):
    """Load ``libm3ssd.so`` (once) and declare the C signatures.

    With ``path``, load that build of the library and return its handle with
    the signatures declared; the module's own calls keep using the in-tree
    library (assign the handle to ``_lib`` to route them to the other build).
    """
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise LibraryMissing(
                f"{p} is not built; run `python -m selective_state_space_m3ssd_b200.build`")
        lib = ctypes.CDLL(p)
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        lib.m3ssd_fwd_workspace_size.argtypes = [ctypes.POINTER(Dims)]
        lib.m3ssd_fwd_workspace_size.restype = sz
        lib.m3ssd_fwd.argtypes = [ctypes.POINTER(Dims)] + [vp] * 11 + \
            [ctypes.POINTER(FwdExtra), vp, sz, vp]
        lib.m3ssd_fwd.restype = ctypes.c_int
        lib.m3ssd_step.argtypes = [ctypes.POINTER(Dims)] + [vp] * 8 + \
            [ctypes.POINTER(Cache), vp, vp]
        lib.m3ssd_step.restype = ctypes.c_int
        lib.m3ssd_mimo_fwd.argtypes = [ctypes.POINTER(Dims), ctypes.c_int32] + [vp] * 11 + \
            [ctypes.POINTER(FwdExtra), vp]
        lib.m3ssd_mimo_fwd.restype = ctypes.c_int
        lib.m3ssd_mimo_step.argtypes = [ctypes.POINTER(Dims), ctypes.c_int32] + [vp] * 8 + \
            [ctypes.POINTER(Cache), vp, vp]
        lib.m3ssd_mimo_step.restype = ctypes.c_int
        lib.m3ssd_bwd_workspace_size.argtypes = [ctypes.POINTER(Dims)]
        lib.m3ssd_bwd_workspace_size.restype = sz
        lib.m3ssd_bwd.argtypes = [ctypes.POINTER(Dims)] + [vp] * 9 + \
            [ctypes.POINTER(FwdExtra), vp, vp, ctypes.POINTER(BwdGrads), vp, sz, vp]
        lib.m3ssd_bwd.restype = ctypes.c_int
        lib.m3ssd_bwd_noalloc.argtypes = [ctypes.POINTER(Dims)] + [vp] * 9 + \
            [ctypes.POINTER(FwdExtra), vp, vp, ctypes.POINTER(BwdGrads), vp]
        lib.m3ssd_bwd_noalloc.restype = ctypes.c_int
        lib.m3ssd_block_workspace_size.argtypes = [ctypes.POINTER(BlockDims)]
        lib.m3ssd_block_workspace_size.restype = sz
        lib.m3ssd_block_fwd.argtypes = [ctypes.POINTER(BlockDims), ctypes.POINTER(BlockWeights),
                                        vp, vp, ctypes.POINTER(Cache), ctypes.POINTER(Cache),
                                        vp, sz, vp]
        lib.m3ssd_block_fwd.restype = ctypes.c_int
        lib.m3ssd_block_step.argtypes = [ctypes.POINTER(BlockDims), ctypes.POINTER(BlockWeights),
                                         vp, vp, ctypes.POINTER(Cache), vp, sz, vp]
        lib.m3ssd_block_step.restype = ctypes.c_int
        lib.m3ssd_gemm_bf16.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_int64, ctypes.c_void_p]
        lib.m3ssd_gemm_bf16.restype = ctypes.c_int
        lib.m3ssd_status_string.argtypes = [ctypes.c_int]
        lib.m3ssd_status_string.restype = ctypes.c_char_p
        lib.m3ssd_abi_version.argtypes = []
        lib.m3ssd_abi_version.restype = ctypes.c_int
        lib.m3ssd_device_wait_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
        lib.m3ssd_device_wait_timeouts.restype = ctypes.c_int
        lib.m3ssd_nonfinite_outputs.argtypes = []
        lib.m3ssd_nonfinite_outputs.restype = ctypes.c_int
        lib.m3ssd_test_set_wait_limit.argtypes = [ctypes.c_uint64]
        lib.m3ssd_test_set_wait_limit.restype = ctypes.c_int
        lib.m3ssd_test_drop_next_gram_signal.argtypes = []
        lib.m3ssd_test_drop_next_gram_signal.restype = ctypes.c_int
        i64, i32p = ctypes.c_int64, ctypes.POINTER(ctypes.c_int32)
        lib.m3ssd_test_fwd_split_plan.argtypes = [i64, i64, i64, ctypes.c_int32, i32p, i32p]
        lib.m3ssd_test_fwd_split_plan.restype = ctypes.c_int
        i32, mxp = ctypes.c_int32, ctypes.POINTER(Mx)
        lib.m3ssd_mx_codes_size.argtypes = [i32, i64, i64]
        lib.m3ssd_mx_codes_size.restype = sz
        lib.m3ssd_mx_scales_size.argtypes = [i64, i64]
        lib.m3ssd_mx_scales_size.restype = sz
        for f in (lib.m3ssd_mx_quant, lib.m3ssd_mx_dequant):
            f.argtypes, f.restype = [mxp, i32, vp, i64, vp], ctypes.c_int
        lib.m3ssd_gemm_mx.argtypes = [mxp, mxp, vp, i64, vp]
        lib.m3ssd_gemm_mx.restype = ctypes.c_int
        ndp = ctypes.POINTER(NormDims)
        lib.m3ssd_add_rmsnorm.argtypes = [ndp, vp, vp, vp, vp, mxp, vp, vp, vp]
        lib.m3ssd_add_rmsnorm.restype = ctypes.c_int
        lib.m3ssd_add_rmsnorm_bwd_workspace_size.argtypes = [ndp]
        lib.m3ssd_add_rmsnorm_bwd_workspace_size.restype = sz
        lib.m3ssd_add_rmsnorm_bwd.argtypes = [ndp] + [vp] * 8 + [sz, vp]
        lib.m3ssd_add_rmsnorm_bwd.restype = ctypes.c_int
        lib.m3ssd_test_gemm_mx_plan.argtypes = [i32, i64, i64, i64, i32, i32p, i32p, i32p]
        lib.m3ssd_test_gemm_mx_plan.restype = ctypes.c_int
        lib.m3ssd_test_give_up_next_waits.argtypes = [ctypes.c_uint32]
        lib.m3ssd_test_give_up_next_waits.restype = ctypes.c_int
        lib.m3ssd_test_norm_access.argtypes = [ndp, i64, i32, i32p]
        lib.m3ssd_test_norm_access.restype = ctypes.c_int
        for f in (lib.m3ssd_quant_state, lib.m3ssd_dequant_state):
            f.argtypes, f.restype = [ctypes.POINTER(Dims), vp, vp, vp, vp], ctypes.c_int
        lib.m3ssd_step_q8.argtypes = [ctypes.POINTER(Dims)] + [vp] * 8 + \
            [ctypes.POINTER(CacheQ8), ctypes.POINTER(CacheQ8), vp, vp]
        lib.m3ssd_step_q8.restype = ctypes.c_int
        if path is None:
            _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().m3ssd_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status == OK:
        return
    if status == ERR_INVALID_ARG:
        raise M3SSDInvalidArgument(status, what)
    raise M3SSDError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(device):
    import torch
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(device.index))


def _xdtype(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise ValueError(f"X/B/C must be bf16 or fp32, got {t.dtype}")


def _need_shape(t, name, dtype=None, shape=None):
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _need(t, name, dtype=None, shape=None, device=None):
    if t is None:
        return
    # one pass over what a valid tensor has; what is wrong is found below
    if (dtype is None or t.dtype == dtype) and (shape is None or t.shape == shape) and \
            (device is None or t.device == device) and t.is_cuda and t.is_contiguous():
        return
    _need_shape(t, name, dtype, shape)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def device_wait_timeouts() -> int:
    """Bounded device-side waits that ran out since the last call (synchronises)."""
    n = ctypes.c_uint32(0)
    _check(load().m3ssd_device_wait_timeouts(ctypes.byref(n)), "m3ssd_device_wait_timeouts")
    return int(n.value)


def nonfinite_outputs() -> bool:
    """Whether any output checked under CHECK_FINITE since the last call held a
    NaN or an infinity (synchronises; clears the record)."""
    st = load().m3ssd_nonfinite_outputs()
    if st == ERR_NONFINITE:
        return True
    _check(st, "m3ssd_nonfinite_outputs")
    return False


def set_wait_limit_for_tests(nanoseconds: int):
    """Testing hook: the chunked forward's bounded waits give up after this many
    nanoseconds (0 restores the default 2 s).  Synchronous; not while work is
    in flight."""
    _check(load().m3ssd_test_set_wait_limit(int(nanoseconds)), "m3ssd_test_set_wait_limit")


def drop_next_gram_signal_for_tests():
    """Testing hook: the next chunked-forward sequence leaves out one completion
    signal, so one of its bounded waits runs out (reported by
    device_wait_timeouts; that launch's outputs are undefined)."""
    _check(load().m3ssd_test_drop_next_gram_signal(), "m3ssd_test_drop_next_gram_signal")


def give_up_next_waits_for_tests(lanes: int):
    """Testing hook: in the next launch that has such waits (include/m3ssd.h), the lanes of
    this mask in every warp that waits for a result give up at once (reported by
    device_wait_timeouts; that launch's outputs are undefined)."""
    _check(load().m3ssd_test_give_up_next_waits(int(lanes)), "m3ssd_test_give_up_next_waits")


def fwd_split_plan(batch: int, seqlen: int, nheads: int, sms: int) -> tuple:
    """(segments, chunks per segment) of the chunked bf16 forward's sequence
    split for this shape on a device with ``sms`` SMs; (1, 0) means no split."""
    nseg, segc = ctypes.c_int32(), ctypes.c_int32()
    _check(load().m3ssd_test_fwd_split_plan(int(batch), int(seqlen), int(nheads), int(sms),
                                            ctypes.byref(nseg), ctypes.byref(segc)),
           "m3ssd_test_fwd_split_plan")
    return nseg.value, segc.value


def make_dims(batch, seqlen, nheads, headdim, dstate, ngroups, x_dtype, chunk=0, flags=0) -> Dims:
    return Dims(batch, seqlen, nheads, headdim, dstate, ngroups, chunk, x_dtype, flags, 0)


def _workspace(workspace, need: int, device):
    """A call's device scratch, allocated where the caller gave none: the tensor, its
    address and its bytes.  A caller's is one contiguous run of memory on ``device``."""
    if workspace is None and need:
        import torch
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    _need(workspace, "workspace", device=device)
    if workspace is None:
        return None, None, 0
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def fwd_workspace_size(dims: Dims) -> int:
    return int(load().m3ssd_fwd_workspace_size(ctypes.byref(dims)))


def fwd(X, logdecay, beta, gamma, B, C, theta=None, D=None, h0=None, *, Y=None,
        want_hT: bool = True, hT=None, angle0=None, xprev0=None, bprev0=None,
        want_cache: bool = False, chunk: int = 0, workspace=None, check_finite: bool = False):
    """Forward scan through ``m3ssd_fwd`` on the current CUDA stream.

    Shapes as in ``include/m3ssd.h``.  Returns ``(Y, hT, cache_out)`` where
    ``cache_out`` is a dict with angleT/xprevT/bprevT when ``want_cache``.
    Output tensors are allocated by torch unless passed in.  ``check_finite``
    sets CHECK_FINITE (see :func:`nonfinite_outputs`).
    """
    import torch
    b, L, H, P = X.shape
    G, N = B.shape[2], B.shape[3]
    dev = X.device
    f32 = torch.float32
    _need(X, "X", device=dev)
    xd = X.dtype
    _need(logdecay, "logdecay", f32, (b, L, H), dev)
    _need(beta, "beta", f32, (b, L, H), dev)
    _need(gamma, "gamma", f32, (b, L, H), dev)
    _need(B, "B", xd, (b, L, G, N), dev)
    _need(C, "C", xd, (b, L, G, N), dev)
    _need(theta, "theta", f32, (b, L, H, N // 2), dev)
    _need(D, "D", f32, (H,), dev)
    _need(h0, "h0", f32, (b, H, N, P), dev)
    _need(angle0, "angle0", f32, (b, H, N // 2), dev)
    _need(xprev0, "xprev0", f32, (b, H, P), dev)
    _need(bprev0, "bprev0", f32, (b, G, N), dev)
    if Y is None:
        Y = torch.empty_like(X)
    _need(Y, "Y", xd, (b, L, H, P), dev)
    if hT is None and want_hT:
        hT = torch.empty(b, H, N, P, dtype=f32, device=dev)
    _need(hT, "hT", f32, (b, H, N, P), dev)
    cache_out = None
    extra = None
    if want_cache or angle0 is not None or xprev0 is not None or bprev0 is not None:
        if want_cache:
            cache_out = {"angle": torch.empty(b, H, N // 2, dtype=f32, device=dev),
                         "x_prev": torch.empty(b, H, P, dtype=f32, device=dev),
                         "b_prev": torch.empty(b, G, N, dtype=f32, device=dev)}
        extra = FwdExtra(
            *(None if t is None else t.data_ptr() for t in (angle0, xprev0, bprev0)),
            *(None if cache_out is None else cache_out[k].data_ptr()
              for k in ("angle", "x_prev", "b_prev")))
    dims = make_dims(b, L, H, P, N, G, _xdtype(X), chunk, CHECK_FINITE if check_finite else 0)
    workspace, ws, ws_bytes = _workspace(workspace, fwd_workspace_size(dims), dev)
    st = load().m3ssd_fwd(ctypes.byref(dims), _ptr(X), _ptr(logdecay), _ptr(beta), _ptr(gamma),
                          _ptr(B), _ptr(C), _ptr(theta), _ptr(D), _ptr(h0), _ptr(Y), _ptr(hT),
                          None if extra is None else ctypes.byref(extra), ws, ws_bytes,
                          _stream_handle(dev))
    _check(st, "m3ssd_fwd")
    return Y, hT, cache_out


def bwd_workspace_size(dims: Dims) -> int:
    return int(load().m3ssd_bwd_workspace_size(ctypes.byref(dims)))


def _bwd_args(X, logdecay, beta, gamma, B, C, theta, D, h0, dY, dhT, angle0, xprev0, bprev0,
              grads):
    """Validates every backward input (dtype, shape, device) and marshals the C
    arguments shared by :func:`bwd` and :func:`bwd_noalloc`."""
    import torch
    b, L, H, P = X.shape
    G, N = B.shape[2], B.shape[3]
    dev = X.device
    f32 = torch.float32
    xd = X.dtype
    checks = [(X, "X", None, None), (logdecay, "logdecay", f32, (b, L, H)),
              (beta, "beta", f32, (b, L, H)), (gamma, "gamma", f32, (b, L, H)),
              (B, "B", xd, (b, L, G, N)), (C, "C", xd, (b, L, G, N)),
              (theta, "theta", f32, (b, L, H, N // 2)), (D, "D", f32, (H,)),
              (h0, "h0", f32, (b, H, N, P)), (angle0, "angle0", f32, (b, H, N // 2)),
              (xprev0, "xprev0", f32, (b, H, P)), (bprev0, "bprev0", f32, (b, G, N)),
              (dY, "dY", xd, (b, L, H, P)), (dhT, "dhT", f32, (b, H, N, P))]
    for t, name, dt, shape in checks:  # every shape and dtype first, then placement
        if t is not None:
            _need_shape(t, name, dt, shape)
    for t, name, dt, shape in checks:
        _need(t, name, dt, shape, dev)
    shapes = {"dX": (b, L, H, P), "dlogdecay": (b, L, H), "dbeta": (b, L, H),
              "dgamma": (b, L, H), "dB": (b, L, G, N), "dC": (b, L, G, N),
              "dtheta": (b, L, H, N // 2), "dD": (H,), "dh0": (b, H, N, P),
              "dangle0": (b, H, N // 2), "dxprev0": (b, H, P), "dbprev0": (b, G, N)}
    if grads is None:
        grads = {k: torch.empty(v, dtype=f32, device=dev) for k, v in shapes.items()}
    for k in GRAD_NAMES:
        _need(grads.get(k), k, f32, shapes[k], dev)
    gs = BwdGrads(*(None if grads.get(k) is None else grads[k].data_ptr() for k in GRAD_NAMES))
    extra = None
    if angle0 is not None or xprev0 is not None or bprev0 is not None:
        extra = FwdExtra(*(None if t is None else t.data_ptr() for t in (angle0, xprev0, bprev0)),
                         None, None, None)
    dims = make_dims(b, L, H, P, N, G, _xdtype(X), 0)
    ptrs = [_ptr(t) for t in (X, logdecay, beta, gamma, B, C, theta, D, h0)]
    return dims, ptrs, extra, gs, grads


def bwd(X, logdecay, beta, gamma, B, C, theta=None, D=None, h0=None, *, dY, dhT=None,
        angle0=None, xprev0=None, bprev0=None, grads=None, workspace=None):
    """Backward of :func:`fwd` through ``m3ssd_bwd`` on the current CUDA stream.

    Takes the forward's inputs and the upstream gradients ``dY`` (dtype of X)
    and ``dhT`` (fp32 or None).  Returns a dict of fp32 gradients named as in
    ``GRAD_NAMES``, each shaped like its input (allocated by torch unless
    ``grads`` supplies them).
    """
    dims, ptrs, extra, gs, grads = _bwd_args(X, logdecay, beta, gamma, B, C, theta, D, h0, dY,
                                             dhT, angle0, xprev0, bprev0, grads)
    workspace, ws, ws_bytes = _workspace(workspace, bwd_workspace_size(dims), X.device)
    st = load().m3ssd_bwd(ctypes.byref(dims), *ptrs,
                          None if extra is None else ctypes.byref(extra), _ptr(dY), _ptr(dhT),
                          ctypes.byref(gs), ws, ws_bytes,
                          _stream_handle(X.device))
    _check(st, "m3ssd_bwd")
    return grads


def bwd_noalloc(X, logdecay, beta, gamma, B, C, theta=None, D=None, h0=None, *, dY,
                dhT=None, angle0=None, xprev0=None, bprev0=None, grads=None):
    """:func:`bwd` through ``m3ssd_bwd_noalloc`` (scratch inside the library;
    calls must not overlap).  Validates its inputs exactly as :func:`bwd` does
    and returns the same dict of fp32 gradients."""
    dims, ptrs, extra, gs, grads = _bwd_args(X, logdecay, beta, gamma, B, C, theta, D, h0, dY,
                                             dhT, angle0, xprev0, bprev0, grads)
    st = load().m3ssd_bwd_noalloc(ctypes.byref(dims), *ptrs,
                                  None if extra is None else ctypes.byref(extra), _ptr(dY),
                                  _ptr(dhT), ctypes.byref(gs), _stream_handle(X.device))
    _check(st, "m3ssd_bwd_noalloc")
    return grads


def new_cache(batch, nheads, headdim, dstate, ngroups, device):
    """A zeroed fp32 decode cache (angle, ssm, x_prev, b_prev) allocated by torch."""
    import torch
    z = dict(dtype=torch.float32, device=device)
    return {"angle": torch.zeros(batch, nheads, dstate // 2, **z),
            "ssm": torch.zeros(batch, nheads, dstate, headdim, **z),
            "x_prev": torch.zeros(batch, nheads, headdim, **z),
            "b_prev": torch.zeros(batch, ngroups, dstate, **z)}


def step(cache: dict, x_t, logdecay_t, beta_t, gamma_t, B_t, C_t, theta_t=None, D=None, *,
         y_t=None, check_finite: bool = False):
    """One decode step through ``m3ssd_step``; updates ``cache`` in place and
    returns y_t (b, H, P) in the dtype of x_t.  ``check_finite`` sets
    CHECK_FINITE on y_t (see :func:`nonfinite_outputs`)."""
    import torch
    b, H, P = x_t.shape
    G, N = B_t.shape[1], B_t.shape[2]
    dev = x_t.device
    f32 = torch.float32
    xd = x_t.dtype
    _need(x_t, "x_t", device=dev)
    _need(logdecay_t, "logdecay_t", f32, (b, H), dev)
    _need(beta_t, "beta_t", f32, (b, H), dev)
    _need(gamma_t, "gamma_t", f32, (b, H), dev)
    _need(B_t, "B_t", xd, (b, G, N), dev)
    _need(C_t, "C_t", xd, (b, G, N), dev)
    _need(theta_t, "theta_t", f32, (b, H, N // 2), dev)
    _need(D, "D", f32, (H,), dev)
    _need(cache["angle"], "cache.angle", f32, (b, H, N // 2), dev)
    _need(cache["ssm"], "cache.ssm", f32, (b, H, N, P), dev)
    _need(cache["x_prev"], "cache.x_prev", f32, (b, H, P), dev)
    _need(cache["b_prev"], "cache.b_prev", f32, (b, G, N), dev)
    if y_t is None:
        y_t = torch.empty_like(x_t)
    _need(y_t, "y_t", xd, (b, H, P), dev)
    c = Cache(cache["angle"].data_ptr(), cache["ssm"].data_ptr(), cache["x_prev"].data_ptr(),
              cache["b_prev"].data_ptr())
    dims = make_dims(b, 1, H, P, N, G, _xdtype(x_t), 0, CHECK_FINITE if check_finite else 0)
    st = load().m3ssd_step(ctypes.byref(dims), _ptr(x_t), _ptr(logdecay_t), _ptr(beta_t),
                           _ptr(gamma_t), _ptr(B_t), _ptr(C_t), _ptr(theta_t), _ptr(D),
                           ctypes.byref(c), _ptr(y_t), _stream_handle(dev))
    _check(st, "m3ssd_step")
    return y_t


def mimo_fwd(X, logdecay, beta, gamma, B, C, theta=None, D=None, h0=None, *, Y=None,
             want_hT: bool = True, angle0=None, xprev0=None, bprev0=None,
             want_cache: bool = False, check_finite: bool = False):
    """MIMO rank-R forward through ``m3ssd_mimo_fwd``: X (b,L,H,P,R), B, C
    (b,L,G,N,R).  Returns ``(Y, hT, cache_out)`` like :func:`fwd`, with the
    cache's x_prev (b,H,P,R) and b_prev (b,G,N,R)."""
    import torch
    b, L, H, P, R = X.shape
    G, N = B.shape[2], B.shape[3]
    dev, f32, xd = X.device, torch.float32, X.dtype
    _need(X, "X", device=dev)
    for name, t, dt, shape in (("logdecay", logdecay, f32, (b, L, H)), ("beta", beta, f32, (b, L, H)),
                               ("gamma", gamma, f32, (b, L, H)), ("B", B, xd, (b, L, G, N, R)),
                               ("C", C, xd, (b, L, G, N, R)), ("theta", theta, f32, (b, L, H, N // 2)),
                               ("D", D, f32, (H,)), ("h0", h0, f32, (b, H, N, P)),
                               ("angle0", angle0, f32, (b, H, N // 2)),
                               ("xprev0", xprev0, f32, (b, H, P, R)),
                               ("bprev0", bprev0, f32, (b, G, N, R))):
        _need(t, name, dt, shape, dev)
    Y = torch.empty_like(X) if Y is None else Y
    _need(Y, "Y", xd, (b, L, H, P, R), dev)
    hT = torch.empty(b, H, N, P, dtype=f32, device=dev) if want_hT else None
    cache_out = None
    extra = None
    if want_cache or angle0 is not None or xprev0 is not None or bprev0 is not None:
        if want_cache:
            cache_out = {"angle": torch.empty(b, H, N // 2, dtype=f32, device=dev),
                         "x_prev": torch.empty(b, H, P, R, dtype=f32, device=dev),
                         "b_prev": torch.empty(b, G, N, R, dtype=f32, device=dev)}
        extra = FwdExtra(
            *(None if t is None else t.data_ptr() for t in (angle0, xprev0, bprev0)),
            *(None if cache_out is None else cache_out[k].data_ptr()
              for k in ("angle", "x_prev", "b_prev")))
    dims = make_dims(b, L, H, P, N, G, _xdtype(X), 0, CHECK_FINITE if check_finite else 0)
    st = load().m3ssd_mimo_fwd(ctypes.byref(dims), R, _ptr(X), _ptr(logdecay), _ptr(beta),
                               _ptr(gamma), _ptr(B), _ptr(C), _ptr(theta), _ptr(D), _ptr(h0),
                               _ptr(Y), _ptr(hT), None if extra is None else ctypes.byref(extra),
                               _stream_handle(dev))
    _check(st, "m3ssd_mimo_fwd")
    return Y, hT, cache_out


def new_mimo_cache(batch, nheads, headdim, dstate, ngroups, rank, device):
    """A zeroed fp32 MIMO decode cache: angle, ssm, x_prev (b,H,P,R), b_prev (b,G,N,R)."""
    import torch
    z = dict(dtype=torch.float32, device=device)
    return {"angle": torch.zeros(batch, nheads, dstate // 2, **z),
            "ssm": torch.zeros(batch, nheads, dstate, headdim, **z),
            "x_prev": torch.zeros(batch, nheads, headdim, rank, **z),
            "b_prev": torch.zeros(batch, ngroups, dstate, rank, **z)}


def mimo_step(cache: dict, x_t, logdecay_t, beta_t, gamma_t, B_t, C_t, theta_t=None, D=None, *,
              y_t=None, check_finite: bool = False):
    """One MIMO decode step through ``m3ssd_mimo_step``: x_t (b,H,P,R), B_t, C_t
    (b,G,N,R); updates ``cache`` in place and returns y_t (b,H,P,R)."""
    import torch
    b, H, P, R = x_t.shape
    G, N = B_t.shape[1], B_t.shape[2]
    dev, f32, xd = x_t.device, torch.float32, x_t.dtype
    _need(x_t, "x_t", device=dev)
    for name, t, dt, shape in (("logdecay_t", logdecay_t, f32, (b, H)), ("beta_t", beta_t, f32, (b, H)),
                               ("gamma_t", gamma_t, f32, (b, H)), ("B_t", B_t, xd, (b, G, N, R)),
                               ("C_t", C_t, xd, (b, G, N, R)), ("theta_t", theta_t, f32, (b, H, N // 2)),
                               ("D", D, f32, (H,)),
                               ("cache.angle", cache["angle"], f32, (b, H, N // 2)),
                               ("cache.ssm", cache["ssm"], f32, (b, H, N, P)),
                               ("cache.x_prev", cache["x_prev"], f32, (b, H, P, R)),
                               ("cache.b_prev", cache["b_prev"], f32, (b, G, N, R))):
        _need(t, name, dt, shape, dev)
    y_t = torch.empty_like(x_t) if y_t is None else y_t
    _need(y_t, "y_t", xd, (b, H, P, R), dev)
    c = Cache(cache["angle"].data_ptr(), cache["ssm"].data_ptr(), cache["x_prev"].data_ptr(),
              cache["b_prev"].data_ptr())
    dims = make_dims(b, 1, H, P, N, G, _xdtype(x_t), 0, CHECK_FINITE if check_finite else 0)
    st = load().m3ssd_mimo_step(ctypes.byref(dims), R, _ptr(x_t), _ptr(logdecay_t), _ptr(beta_t),
                                _ptr(gamma_t), _ptr(B_t), _ptr(C_t), _ptr(theta_t), _ptr(D),
                                ctypes.byref(c), _ptr(y_t), _stream_handle(dev))
    _check(st, "m3ssd_mimo_step")
    return y_t


# ---- the Mamba-3 SISO block around the scan --------------------------------------

def block_in_proj_width(nheads, headdim, dstate, ngroups) -> int:
    """Rows of W_in: z, x (H P each), B, C (G N each), dt, lam (H each), theta (H N/2)."""
    return 2 * nheads * headdim + 2 * ngroups * dstate + 2 * nheads + nheads * (dstate // 2)


def _block_args(u, wts, seqlen):
    import torch
    b, dm = u.shape[0], u.shape[-1]
    H = wts["A_log"].shape[0]
    N = wts["B_norm_w"].shape[0]
    HP = wts["W_out"].shape[1]
    if HP % H:
        raise ValueError("W_out's columns must be H * P")
    P = HP // H
    width = wts["W_in"].shape[0]
    rest = width - 2 * HP - 2 * H - H * (N // 2)
    if rest <= 0 or rest % (2 * N):
        raise ValueError("W_in's rows do not match any group count")
    G = rest // (2 * N)
    dev = u.device
    f32, bf = torch.float32, torch.bfloat16
    _need(u, "u", bf, device=dev)
    _need(wts["W_in"], "W_in", bf, (width, dm), dev)
    _need(wts["W_out"], "W_out", bf, (dm, HP), dev)
    for k, shape in (("dt_bias", (H,)), ("A_log", (H,)), ("B_norm_w", (N,)), ("C_norm_w", (N,)),
                     ("B_bias", (H, N)), ("C_bias", (H, N))):
        _need(wts[k], k, f32, shape, dev)
    _need(wts.get("D"), "D", f32, (H,), dev)
    dims = BlockDims(b, seqlen, dm, H, P, N, G)
    w = BlockWeights(*[(None if wts.get(k) is None else wts[k].data_ptr())
                       for k in BLOCK_WEIGHT_NAMES], float(wts.get("eps", 1e-6)))
    return dims, w, (H, P, N, G)


def new_block_cache(batch, nheads, headdim, dstate, ngroups, device):
    """A zeroed block cache: angle (b,H,N/2), ssm (b,H,N,P), x_prev (b,H,P) and
    b_prev (b,G,N) (the normed group vector, the head bias added at use), all fp32."""
    return new_cache(batch, nheads, headdim, dstate, ngroups, device)


def _cache_struct(cache, b, H, P, N, G, dev, name):
    import torch
    f32 = torch.float32
    _need(cache["angle"], name + ".angle", f32, (b, H, N // 2), dev)
    _need(cache["ssm"], name + ".ssm", f32, (b, H, N, P), dev)
    _need(cache["x_prev"], name + ".x_prev", f32, (b, H, P), dev)
    _need(cache["b_prev"], name + ".b_prev", f32, (b, G, N), dev)
    return Cache(cache["angle"].data_ptr(), cache["ssm"].data_ptr(), cache["x_prev"].data_ptr(),
                 cache["b_prev"].data_ptr())


def block_workspace_size(dims: BlockDims) -> int:
    return int(load().m3ssd_block_workspace_size(ctypes.byref(dims)))


def block_fwd(u, wts: dict, *, cache_in=None, cache_out=None, out=None, workspace=None):
    """Forward of the Mamba-3 SISO block through ``m3ssd_block_fwd``: u (b, L,
    d_model) bf16 -> out (b, L, d_model) bf16.  ``cache_in`` / ``cache_out``
    (dicts as from :func:`new_block_cache`, may be the same dict) continue from
    and hand back the decode state.  ``workspace`` (uint8, 256-byte aligned) is
    allocated by torch when not given."""
    import torch
    b, L, dm = u.shape
    dims, w, (H, P, N, G) = _block_args(u, wts, L)
    dev = u.device
    out = torch.empty_like(u) if out is None else out
    _need(out, "out", torch.bfloat16, (b, L, dm), dev)
    ci = None if cache_in is None else _cache_struct(cache_in, b, H, P, N, G, dev, "cache_in")
    co = None if cache_out is None else _cache_struct(cache_out, b, H, P, N, G, dev, "cache_out")
    workspace, ws, ws_bytes = _workspace(workspace, block_workspace_size(dims), dev)
    st = load().m3ssd_block_fwd(ctypes.byref(dims), ctypes.byref(w), _ptr(u), _ptr(out),
                                None if ci is None else ctypes.byref(ci),
                                None if co is None else ctypes.byref(co), ws, ws_bytes,
                                _stream_handle(dev))
    _check(st, "m3ssd_block_fwd")
    return out


def gemm_bf16(A, W, *, out=None):
    """``m3ssd_gemm_bf16``: A (M, K) @ W (N, K)^T in bf16 with fp32 accumulation
    on the current stream; returns out (M, N) bf16."""
    import torch
    _need(A, "A", torch.bfloat16, device=A.device)
    M, K = A.shape
    _need(W, "W", torch.bfloat16, (W.shape[0], K), A.device)
    N = W.shape[0]
    out = torch.empty(M, N, dtype=torch.bfloat16, device=A.device) if out is None else out
    _need(out, "out", torch.bfloat16, (M, N), A.device)
    st = load().m3ssd_gemm_bf16(M, N, K, _ptr(A), _ptr(W), _ptr(out), N, _stream_handle(A.device))
    _check(st, "m3ssd_gemm_bf16")
    return out


def block_step(cache: dict, u_t, wts: dict, *, out_t=None, workspace=None):
    """One decode step of the block through ``m3ssd_block_step``: u_t (b,
    d_model) bf16 -> out_t; ``cache`` is advanced in place."""
    import torch
    b, dm = u_t.shape
    dims, w, (H, P, N, G) = _block_args(u_t, wts, 1)
    dev = u_t.device
    out_t = torch.empty_like(u_t) if out_t is None else out_t
    _need(out_t, "out_t", torch.bfloat16, (b, dm), dev)
    c = _cache_struct(cache, b, H, P, N, G, dev, "cache")
    workspace, ws, ws_bytes = _workspace(workspace, block_workspace_size(dims), dev)
    st = load().m3ssd_block_step(ctypes.byref(dims), ctypes.byref(w), _ptr(u_t), _ptr(out_t),
                                 ctypes.byref(c), ws, ws_bytes, _stream_handle(dev))
    _check(st, "m3ssd_block_step")
    return out_t


def _launch(name: str, dev, *args):
    """Calls a C entry point whose last argument is the stream, with the tensors'
    device current (a stream, a workspace size and a launch all go by it)."""
    import torch
    f = getattr(_lib or load(), name)
    index = dev.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        st = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = f(*args, stream)
    if st != OK:
        _check(st, name)


def _need_all(dev, *checks):
    """:func:`_need` for (tensor, name, dtype, shape) on the CUDA device ``dev``, in one
    loop: a decode step checks some twenty tensors."""
    index = dev.index  # of a CUDA device; a CPU tensor's is -1
    for t, name, dtype, shape in checks:
        if t is not None and (t.dtype != dtype or t.shape != shape or t.get_device() != index or
                              not t.is_contiguous()):
            _need(t, name, dtype, shape, dev)


def _addr(t):
    return None if t is None else t.data_ptr()


# ---- microscaled tensors and their product ------------------------------------------

MXFP4, MXFP8 = 0, 1
_MX_FORMATS = {"mxfp4": MXFP4, "mxfp8": MXFP8}


def _pad128(n: int) -> int:
    return (n + 127) // 128 * 128


class MXTensor:
    """A microscaled tensor (``m3ssd_mx``): ``fmt`` "mxfp4" or "mxfp8", ``rows`` x
    ``cols`` values in blocks of 32; ``codes`` (rows, Kp / 2 or Kp) and ``scales``
    (flat, tiles of 128 rows x 4 blocks), uint8, as laid out in ``include/m3ssd.h``."""

    __slots__ = ("fmt", "rows", "cols", "codes", "scales")

    def __init__(self, fmt: str, rows: int, cols: int, codes, scales):
        self.fmt, self.rows, self.cols, self.codes, self.scales = fmt, rows, cols, codes, scales

    @classmethod
    def empty(cls, fmt: str, rows: int, cols: int, device):
        """Unwritten storage for a tensor of this size."""
        import torch
        kp = _pad128(cols)
        return cls(fmt, rows, cols,
                   torch.empty(rows, kp if _mx_format(fmt) == MXFP8 else kp // 2,
                               dtype=torch.uint8, device=device),
                   torch.empty(_pad128(rows) * (kp // 32), dtype=torch.uint8, device=device))


def _mx_format(fmt) -> int:
    if fmt not in _MX_FORMATS:
        raise ValueError(f"format must be one of {sorted(_MX_FORMATS)}, got {fmt!r}")
    return _MX_FORMATS[fmt]


def _mx_of(t: MXTensor) -> Mx:
    return Mx(_MX_FORMATS[t.fmt], 0, t.rows, t.cols, t.codes.data_ptr(), t.scales.data_ptr())


def _mx_struct(t: MXTensor, name: str, device) -> Mx:
    """The C descriptor of a caller's tensor, its storage checked."""
    import torch
    f, kp, u8 = _mx_format(t.fmt), _pad128(t.cols), torch.uint8
    codes, scales = t.codes, t.scales
    _need(codes, name + ".codes", u8, (t.rows, kp if f == MXFP8 else kp // 2), device)
    _need(scales, name + ".scales", u8, (_pad128(t.rows) * (kp // 32),), device)
    return Mx(f, 0, t.rows, t.cols, codes.data_ptr(), scales.data_ptr())


def _rows_stride(x, name):
    """A (rows, cols) CUDA tensor with unit column stride; returns its row stride."""
    if x.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {tuple(x.shape)}")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    rows, cols = x.shape
    if (cols > 1 and x.stride(1) != 1) or (rows > 1 and x.stride(0) < cols):
        raise ValueError(f"{name} must have contiguous rows")
    return x.stride(0) if rows > 1 else max(cols, 1)


def mx_quant(x, fmt: str, *, out: MXTensor | None = None) -> MXTensor:
    """x (rows, cols), bf16 or fp32, rows contiguous (any row stride), to the
    microscaled format ``fmt`` through ``m3ssd_mx_quant``."""
    ldx = _rows_stride(x, "x")
    rows, cols = x.shape
    if out is None:
        out = MXTensor.empty(fmt, rows, cols, x.device)
        o = _mx_of(out)
    elif not isinstance(out, MXTensor) or (out.fmt, out.rows, out.cols) != (fmt, rows, cols):
        raise ValueError(f"out must be {fmt} of {rows} x {cols}")
    else:
        o = _mx_struct(out, "out", x.device)
    _launch("m3ssd_mx_quant", x.device, ctypes.byref(o), _xdtype(x), _addr(x), ldx)
    return out


def mx_dequant(t: MXTensor, dtype=None, *, out=None):
    """The values of a microscaled tensor (rows, cols) through ``m3ssd_mx_dequant``,
    in ``dtype`` (bf16 unless given) or into ``out`` (rows contiguous)."""
    import torch
    dev = t.codes.device
    if out is None:
        out, ldx = torch.empty(t.rows, t.cols, dtype=dtype or torch.bfloat16, device=dev), t.cols
    else:
        _need_shape(out, "out", dtype, (t.rows, t.cols))
        ldx = _rows_stride(out, "out")
    m = _mx_struct(t, "t", out.device)
    _launch("m3ssd_mx_dequant", dev, ctypes.byref(m), _xdtype(out), _addr(out), ldx)
    return out


def gemm_mx(A: MXTensor, W: MXTensor, *, out=None):
    """A (M, K) @ W (N, K)^T of microscaled operands through ``m3ssd_gemm_mx`` (W in
    "mxfp4", A in either format) -> out (M, N) bf16, rows contiguous."""
    import torch
    dev = A.codes.device
    if out is None:
        out, ldd = torch.empty(A.rows, W.rows, dtype=torch.bfloat16, device=dev), W.rows
    else:
        _need_shape(out, "out", torch.bfloat16, (A.rows, W.rows))
        ldd = _rows_stride(out, "out")
    a, w = _mx_struct(A, "A", out.device), _mx_struct(W, "W", out.device)
    _launch("m3ssd_gemm_mx", dev, ctypes.byref(a), ctypes.byref(w), _addr(out), ldd)
    return out


def gemm_mx_plan(M: int, N: int, K: int, fmt: str, sms: int) -> tuple:
    """(split, tile, part) of :func:`gemm_mx` with A (M, K) in ``fmt`` and W (N, K) on a device
    with ``sms`` SMs: the CTAs that share a tile's K (0: none), the tile's tokens there, else
    its columns, and the columns of the parts that the last tiles go out in (0: whole)."""
    out = [ctypes.c_int32() for _ in range(3)]
    _check(load().m3ssd_test_gemm_mx_plan(_mx_format(fmt), int(M), int(N), int(K), int(sms),
                                          *(ctypes.byref(v) for v in out)),
           "m3ssd_test_gemm_mx_plan")
    return tuple(v.value for v in out)


# ---- the residual addition with the RMS norm -------------------------------------------

def add_rmsnorm(x, w, *, residual=None, eps: float = 1e-6, fmt: str | None = None,
                want_rstd: bool = False, y=None, residual_out=None):
    """r = x + residual, y = r / sqrt(mean r^2 + eps) * w over the last axis, through
    ``m3ssd_add_rmsnorm``.  x (..., d) bf16 or fp32; residual (its shape) bf16 or fp32;
    w (d) fp32.  ``fmt`` ("mxfp8" or "mxfp4") returns y as an :class:`MXTensor` of the
    flattened rows, the A operand of :func:`gemm_mx`; else y has x's type.  Returns ``(y,
    residual_out, rstd)``; residual_out (residual's type; pass ``residual`` to write it in
    place) is None without a residual, rstd (fp32, rows) None unless ``want_rstd``."""
    import torch
    dev, f32 = x.device, torch.float32
    d = x.shape[-1]
    rows = x.numel() // d if d else 0
    _need(x, "x", device=dev)
    _need(w, "w", f32, (d,), dev)
    xd = rd = _xdtype(x)
    if residual is not None:
        rd = _xdtype(residual)
        _need(residual, "residual", None, x.shape, dev)
        if residual_out is None:
            residual_out = torch.empty_like(residual)
        else:
            _need(residual_out, "residual_out", residual.dtype, x.shape, dev)
    elif residual_out is not None:
        raise ValueError("residual_out is only written with a residual")
    mx = None
    if fmt is None and y is None:
        y = torch.empty_like(x)
    elif fmt is None:
        _need(y, "y", x.dtype, x.shape, dev)
    elif y is None:
        y = MXTensor.empty(fmt, rows, d, dev)
        mx = _mx_of(y)
    elif not isinstance(y, MXTensor) or (y.fmt, y.rows, y.cols) != (fmt, rows, d):
        raise ValueError(f"y must be {fmt} of {rows} x {d}")
    else:
        mx = _mx_struct(y, "y", dev)
    rstd = torch.empty(rows, dtype=f32, device=dev) if want_rstd else None
    dims = NormDims(rows, d, xd, rd, eps, 0)
    _launch("m3ssd_add_rmsnorm", dev, ctypes.byref(dims), _addr(x), _addr(residual), _addr(w),
            None if mx is not None else _addr(y), None if mx is None else ctypes.byref(mx),
            _addr(residual_out), _addr(rstd))
    return y, residual_out, rstd


def add_rmsnorm_bwd_workspace_size(dims: NormDims) -> int:
    """Bytes on the current device."""
    return int(load().m3ssd_add_rmsnorm_bwd_workspace_size(ctypes.byref(dims)))


def add_rmsnorm_bwd(dy, r, w, rstd, *, dres=None, dr=None, dw=None, workspace=None):
    """Backward of :func:`add_rmsnorm` through ``m3ssd_add_rmsnorm_bwd``: dy (..., d) bf16
    or fp32, r the forward's residual_out (or x without a residual), rstd its rstd, dres
    the fp32 gradient of residual_out (None = 0).  Returns ``(dr, dw)`` in fp32: dr is the
    gradient of x and of residual alike."""
    import torch
    dev, f32 = dy.device, torch.float32
    d = dy.shape[-1]
    rows = dy.numel() // d if d else 0
    _need(dy, "dy", device=dev)
    _need_all(dev, (r, "r", r.dtype, dy.shape), (w, "w", f32, (d,)),
              (rstd, "rstd", f32, (rows,)), (dres, "dres", f32, dy.shape))
    if dr is None:
        dr = torch.empty(dy.shape, dtype=f32, device=dev)
    else:
        _need(dr, "dr", f32, dy.shape, dev)
    if dw is None:
        dw = torch.empty(d, dtype=f32, device=dev)
    else:
        _need(dw, "dw", f32, (d,), dev)
    dims = NormDims(rows, d, _xdtype(dy), _xdtype(r), 0.0, 0)
    if torch._C._cuda_getDevice() == dev.index:
        need = add_rmsnorm_bwd_workspace_size(dims)
    else:
        with torch.cuda.device(dev):
            need = add_rmsnorm_bwd_workspace_size(dims)
    workspace, ws, ws_bytes = _workspace(workspace, need, dev)
    _launch("m3ssd_add_rmsnorm_bwd", dev, ctypes.byref(dims), _addr(dy), _addr(r), _addr(w),
            _addr(rstd), _addr(dres), _addr(dr), _addr(dw), ws, ws_bytes)
    return dr, dw


# ---- the decode cache with its state in 8 bits -------------------------------------------

def quant_state(ssm, *, codes=None, scale=None):
    """An fp32 state (b, H, N, P) as E4M3 codes (uint8, same shape) and scales (b, H, N)
    fp32, through ``m3ssd_quant_state``; returns ``(codes, scale)``."""
    import torch
    _need(ssm, "ssm", torch.float32, device=ssm.device)
    b, H, N, P = ssm.shape
    dev = ssm.device
    codes = torch.empty(b, H, N, P, dtype=torch.uint8, device=dev) if codes is None else codes
    scale = torch.empty(b, H, N, dtype=torch.float32, device=dev) if scale is None else scale
    _need(codes, "codes", torch.uint8, (b, H, N, P), dev)
    _need(scale, "scale", torch.float32, (b, H, N), dev)
    dims = make_dims(b, 1, H, P, N, 1, F32)
    _launch("m3ssd_quant_state", dev, ctypes.byref(dims), _addr(ssm), _addr(codes), _addr(scale))
    return codes, scale


def dequant_state(codes, scale, *, ssm=None):
    """The fp32 state (b, H, N, P) that codes and scales stand for, through
    ``m3ssd_dequant_state``."""
    import torch
    dev = codes.device
    _need(codes, "codes", torch.uint8, device=dev)
    b, H, N, P = codes.shape
    _need(scale, "scale", torch.float32, (b, H, N), dev)
    ssm = torch.empty(b, H, N, P, dtype=torch.float32, device=dev) if ssm is None else ssm
    _need(ssm, "ssm", torch.float32, (b, H, N, P), dev)
    dims = make_dims(b, 1, H, P, N, 1, F32)
    _launch("m3ssd_dequant_state", dev, ctypes.byref(dims), _addr(codes), _addr(scale), _addr(ssm))
    return ssm


def new_cache_q8(batch, nheads, headdim, dstate, ngroups, device):
    """A zeroed decode cache with its state in 8 bits: angle, ssm (uint8 E4M3 codes,
    b,H,N,P), scale (b,H,N), x_prev, b_prev."""
    import torch
    c = {k: v for k, v in new_cache(batch, nheads, 1, dstate, ngroups, device).items()}
    c["x_prev"] = torch.zeros(batch, nheads, headdim, dtype=torch.float32, device=device)
    c["ssm"] = torch.zeros(batch, nheads, dstate, headdim, dtype=torch.uint8, device=device)
    c["scale"] = torch.zeros(batch, nheads, dstate, dtype=torch.float32, device=device)
    return c


def quant_cache(cache: dict) -> dict:
    """An fp32 decode cache (:func:`new_cache`, or prefill's) with its state in 8 bits;
    the other parts are copied."""
    codes, scale = quant_state(cache["ssm"])
    return {"angle": cache["angle"].clone(), "ssm": codes, "scale": scale,
            "x_prev": cache["x_prev"].clone(), "b_prev": cache["b_prev"].clone()}


def dequant_cache(cache: dict) -> dict:
    """The fp32 decode cache that an 8-bit one stands for."""
    return {"angle": cache["angle"].clone(), "ssm": dequant_state(cache["ssm"], cache["scale"]),
            "x_prev": cache["x_prev"].clone(), "b_prev": cache["b_prev"].clone()}


def _cache_q8_struct(c, b, H, P, N, G, dev, name):
    import torch
    f32 = torch.float32
    angle, ssm, scale, xp, bp = c["angle"], c["ssm"], c["scale"], c["x_prev"], c["b_prev"]
    _need_all(dev, (angle, name + ".angle", f32, (b, H, N // 2)),
              (ssm, name + ".ssm", torch.uint8, (b, H, N, P)),
              (scale, name + ".scale", f32, (b, H, N)), (xp, name + ".x_prev", f32, (b, H, P)),
              (bp, name + ".b_prev", f32, (b, G, N)))
    return CacheQ8(angle.data_ptr(), ssm.data_ptr(), scale.data_ptr(), xp.data_ptr(),
                   bp.data_ptr())


def step_q8(cache: dict, x_t, logdecay_t, beta_t, gamma_t, B_t, C_t, theta_t=None, D=None, *,
            cache_out: dict | None = None, y_t=None, check_finite: bool = False):
    """:func:`step` on a cache whose state is held in 8 bits (:func:`quant_cache`,
    :func:`new_cache_q8`), through ``m3ssd_step_q8``.  The new cache is written to
    ``cache_out`` (the old one stays), or over ``cache``; returns y_t (b, H, P)."""
    import torch
    b, H, P = x_t.shape
    G, N = B_t.shape[1], B_t.shape[2]
    dev, f32, xd = x_t.device, torch.float32, x_t.dtype
    _need(x_t, "x_t", device=dev)
    _need_all(dev, (logdecay_t, "logdecay_t", f32, (b, H)), (beta_t, "beta_t", f32, (b, H)),
              (gamma_t, "gamma_t", f32, (b, H)), (B_t, "B_t", xd, (b, G, N)),
              (C_t, "C_t", xd, (b, G, N)), (theta_t, "theta_t", f32, (b, H, N // 2)),
              (D, "D", f32, (H,)))
    ci = _cache_q8_struct(cache, b, H, P, N, G, dev, "cache")
    co = None if cache_out is None else \
        _cache_q8_struct(cache_out, b, H, P, N, G, dev, "cache_out")
    if y_t is None:
        y_t = torch.empty_like(x_t)
    else:
        _need(y_t, "y_t", xd, (b, H, P), dev)
    dims = make_dims(b, 1, H, P, N, G, _xdtype(x_t), 0, CHECK_FINITE if check_finite else 0)
    _launch("m3ssd_step_q8", dev, ctypes.byref(dims), _addr(x_t), _addr(logdecay_t), _addr(beta_t),
            _addr(gamma_t), _addr(B_t), _addr(C_t), _addr(theta_t), _addr(D), ctypes.byref(ci),
            None if co is None else ctypes.byref(co), _addr(y_t))
    return y_t


class PreparedFwd:
    """A forward call with its C arguments marshalled once, for loops that
    launch the same problem many times (benchmarks, graph capture).  Calling
    it enqueues ``m3ssd_fwd`` on the current stream of the tensors' device."""

    def __init__(self, X, logdecay, beta, gamma, B, C, theta=None, D=None, h0=None, *,
                 Y=None, hT=None, chunk: int = 0):
        import torch
        b, L, H, P = X.shape
        G, N = B.shape[2], B.shape[3]
        self.Y = torch.empty_like(X) if Y is None else Y
        self.hT = hT
        self._keep = (X, logdecay, beta, gamma, B, C, theta, D, h0, self.Y, hT)
        self._dims = make_dims(b, L, H, P, N, G, _xdtype(X), chunk)
        self._args = [_ptr(t) for t in self._keep]
        self.device = X.device
        ws = fwd_workspace_size(self._dims)
        self._ws = torch.empty(ws, dtype=torch.uint8, device=X.device) if ws else None
        self._lib = load()

    def __call__(self):
        st = self._lib.m3ssd_fwd(ctypes.byref(self._dims), *self._args, None, _ptr(self._ws),
                                 0 if self._ws is None else self._ws.numel(),
                                 _stream_handle(self.device))
        _check(st, "m3ssd_fwd")
        return self.Y
