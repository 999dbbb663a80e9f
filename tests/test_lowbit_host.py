"""Host-side validation of the low-bit and norm entry points (CPU: every call fails
its checks or has nothing to do, so no kernel is reached), and the binding's refusals."""
import ctypes

import pytest
import torch

import selective_state_space_m3ssd_b200 as m3

A, B = 0x10000, 0x20000  # aligned, never dereferenced
PA = ctypes.c_void_p(A)
OK, BAD, UNSUP, WS = m3.OK, m3.ERR_INVALID_ARG, m3.ERR_UNSUPPORTED, m3.ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return m3.load()


def mx(fmt=0, rows=4, cols=64, codes=A, scales=B, reserved=0):
    return m3.Mx(fmt, reserved, rows, cols, codes, scales)


BAD_MX = [(dict(fmt=2), BAD), (dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(codes=None), BAD),
          (dict(scales=None), BAD), (dict(codes=A + 64), BAD), (dict(scales=B + 16), BAD),
          (dict(reserved=1), BAD), (dict(rows=2 ** 31 - 1), UNSUP),
          (dict(rows=2 ** 24, cols=2 ** 20), UNSUP)]


@pytest.mark.parametrize("kw,status", BAD_MX)
def test_mx_tensor_is_checked_everywhere(lib, kw, status):
    t, ok = mx(**kw), mx()
    r = ctypes.byref
    assert lib.m3ssd_mx_quant(r(t), m3.BF16, PA, 64, None) == status
    assert lib.m3ssd_mx_dequant(r(t), m3.BF16, PA, 64, None) == status
    assert lib.m3ssd_gemm_mx(r(t), r(ok), PA, 4, None) == status
    assert lib.m3ssd_gemm_mx(r(ok), r(t), PA, 4, None) == status
    n = m3.NormDims(4, 64, m3.BF16, m3.F32, 1e-6, 0)
    assert lib.m3ssd_add_rmsnorm(r(n), PA, None, PA, None, r(t), None, None, None) == status


def test_mx_and_gemm_arguments(lib):
    r, t = ctypes.byref, mx()
    assert lib.m3ssd_mx_quant(None, m3.BF16, PA, 64, None) == BAD
    assert lib.m3ssd_mx_quant(r(t), 7, PA, 64, None) == BAD
    assert lib.m3ssd_mx_quant(r(t), m3.BF16, PA, 63, None) == BAD       # stride < cols
    assert lib.m3ssd_mx_quant(r(t), m3.BF16, None, 64, None) == BAD
    assert lib.m3ssd_mx_quant(r(t), m3.F32, ctypes.c_void_p(A + 2), 64, None) == BAD
    assert lib.m3ssd_mx_quant(r(mx(rows=0, codes=None, scales=None)), m3.F32, None, 64, None) == OK
    assert lib.m3ssd_gemm_mx(r(t), r(mx(cols=96)), PA, 4, None) == BAD  # K differs
    assert lib.m3ssd_gemm_mx(r(t), r(t), PA, 3, None) == BAD            # ldd < N
    assert lib.m3ssd_gemm_mx(r(t), r(mx(fmt=1)), PA, 4, None) == UNSUP  # W in 8 bits
    assert lib.m3ssd_gemm_mx(r(t), r(t), None, 4, None) == BAD
    assert lib.m3ssd_gemm_mx(r(t), r(t), ctypes.c_void_p(A + 1), 4, None) == BAD
    assert lib.m3ssd_gemm_mx(r(mx(rows=0)), r(t), None, 4, None) == OK
    assert lib.m3ssd_mx_codes_size(0, 3, 130) == 3 * 128
    assert lib.m3ssd_mx_codes_size(1, 3, 130) == 3 * 256
    assert lib.m3ssd_mx_scales_size(129, 130) == 256 * 8
    assert lib.m3ssd_mx_codes_size(2, 3, 130) == 0 and lib.m3ssd_mx_scales_size(3, 0) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), BAD), (dict(width=0), BAD), (dict(x_dtype=2), BAD), (dict(res_dtype=2), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(reserved=1), BAD),
    (dict(width=16385), UNSUP), (dict(rows=2 ** 31), UNSUP)])
def test_norm_dims(lib, kw, status):
    d = dict(rows=4, width=64, x_dtype=m3.BF16, res_dtype=m3.F32, eps=1e-6, reserved=0)
    n = ctypes.byref(m3.NormDims(*{**d, **kw}.values()))
    assert lib.m3ssd_add_rmsnorm(n, PA, None, PA, PA, None, None, None, None) == status
    assert lib.m3ssd_add_rmsnorm_bwd(n, PA, PA, PA, PA, None, PA, PA, PA, 1 << 30, None) == status
    assert lib.m3ssd_add_rmsnorm_bwd_workspace_size(n) == 0


def test_norm_arguments(lib):
    n, r = ctypes.byref(m3.NormDims(4, 64, m3.BF16, m3.F32, 1e-6, 0)), ctypes.byref
    f = lib.m3ssd_add_rmsnorm
    assert f(None, PA, None, PA, PA, None, None, None, None) == BAD
    assert f(n, PA, None, PA, None, None, None, None, None) == BAD          # no output
    assert f(n, PA, None, PA, PA, r(mx()), None, None, None) == BAD         # two outputs
    assert f(n, PA, PA, PA, PA, None, None, None, None) == BAD              # residual alone
    assert f(n, PA, None, PA, PA, None, PA, None, None) == BAD              # residual_out alone
    assert f(n, None, None, PA, PA, None, None, None, None) == BAD
    assert f(n, PA, PA, PA, ctypes.c_void_p(B), None, ctypes.c_void_p(B), None, None) == BAD  # y = r
    assert f(n, PA, None, None, PA, None, None, None, None) == BAD
    assert f(n, PA, None, PA, None, r(mx(rows=5)), None, None, None) == BAD
    assert f(n, PA, None, PA, None, r(mx(cols=65)), None, None, None) == BAD
    odd = ctypes.c_void_p(A + 2)
    assert f(n, PA, odd, PA, PA, None, PA, None, None) == BAD               # fp32 residual
    assert f(n, PA, None, PA, PA, None, None, odd, None) == BAD             # rstd
    zero = ctypes.byref(m3.NormDims(0, 64, m3.BF16, m3.F32, 1e-6, 0))
    assert f(zero, None, None, None, None, None, None, None, None) == OK
    b = lib.m3ssd_add_rmsnorm_bwd
    assert b(n, PA, PA, PA, PA, None, PA, None, PA, 1 << 30, None) == BAD   # dw
    assert b(n, None, PA, PA, PA, None, PA, PA, PA, 1 << 30, None) == BAD
    assert b(n, PA, PA, PA, PA, odd, PA, PA, PA, 1 << 30, None) == BAD
    need = lib.m3ssd_add_rmsnorm_bwd_workspace_size(n)
    assert need >= 4 * 64 * 4
    assert b(n, PA, PA, PA, PA, None, PA, PA, PA, need - 1, None) == WS
    assert b(n, PA, PA, PA, PA, None, PA, PA, None, need, None) == WS
    assert b(n, PA, PA, PA, PA, None, PA, PA, ctypes.c_void_p(A + 4), need, None) == WS


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), BAD), (dict(nheads=0), BAD), (dict(headdim=0), BAD), (dict(dstate=7), BAD),
    (dict(ngroups=2, nheads=3), BAD), (dict(x_dtype=3), BAD), (dict(flags=2), UNSUP),
    (dict(headdim=257), UNSUP), (dict(dstate=258), UNSUP), (dict(dstate=256, headdim=65), UNSUP),
    (dict(batch=2 ** 20, nheads=2 ** 12), UNSUP)])
def test_state_dims(lib, kw, status):
    d = dict(batch=1, seqlen=1, nheads=2, headdim=8, dstate=8, ngroups=1, x_dtype=m3.F32, chunk=0,
             flags=0)
    n = ctypes.byref(m3.make_dims(**{**d, **kw}))
    c = ctypes.byref(m3.CacheQ8(A, A, A, A, A))
    assert lib.m3ssd_quant_state(n, PA, PA, PA, None) == status
    assert lib.m3ssd_dequant_state(n, PA, PA, PA, None) == status
    assert lib.m3ssd_step_q8(n, PA, PA, None, PA, PA, PA, None, None, c, None, PA, None) == status


def test_step_arguments(lib):
    n = ctypes.byref(m3.make_dims(1, 1, 2, 8, 8, 1, m3.F32))
    c = m3.CacheQ8(A, A, A, A, A)
    r = ctypes.byref
    f = lib.m3ssd_step_q8
    assert f(None, PA, PA, None, PA, PA, PA, None, None, r(c), None, PA, None) == BAD
    assert f(n, PA, PA, None, PA, PA, PA, None, None, None, None, PA, None) == BAD
    for i in (0, 1, 3, 4, 5):  # a required tensor missing
        a = [PA, PA, None, PA, PA, PA, None, None]
        a[i] = None
        assert f(n, *a, r(c), None, PA, None) == BAD
    assert f(n, PA, PA, None, PA, PA, PA, None, None, r(c), None, None, None) == BAD
    for k in ("angle", "ssm", "ssm_scale", "x_prev", "b_prev"):
        parts = dict(angle=A, ssm=A, ssm_scale=A, x_prev=A, b_prev=A)
        bad = m3.CacheQ8(*{**parts, k: None}.values())
        assert f(n, PA, PA, None, PA, PA, PA, None, None, r(bad), None, PA, None) == BAD
        assert f(n, PA, PA, None, PA, PA, PA, None, None, r(c), r(bad), PA, None) == BAD
    odd = ctypes.c_void_p(A + 2)
    assert f(n, PA, PA, odd, PA, PA, PA, None, None, r(c), None, PA, None) == BAD
    assert f(n, odd, PA, None, PA, PA, PA, None, None, r(c), None, PA, None) == BAD
    flagged = ctypes.byref(m3.make_dims(1, 1, 2, 8, 8, 1, m3.F32, 0, m3.CHECK_FINITE))
    assert lib.m3ssd_quant_state(flagged, PA, PA, PA, None) == UNSUP
    empty = ctypes.byref(m3.make_dims(0, 1, 2, 8, 8, 1, m3.F32))
    assert f(empty, None, None, None, None, None, None, None, None, r(c), None, None, None) == OK
    assert lib.m3ssd_quant_state(empty, None, None, None, None) == OK


def test_binding_refusals():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        m3.mx_quant(x, "mxfp4")
    with pytest.raises(ValueError, match="CUDA tensor"):
        m3.add_rmsnorm(x, torch.ones(64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        m3.quant_state(torch.zeros(1, 2, 8, 8))
    with pytest.raises(ValueError, match="format must be"):
        m3.MXTensor.empty("int4", 4, 64, "cpu")
    t = m3.MXTensor.empty("mxfp4", 4, 64, "cpu")
    assert t.codes.shape == (4, 64) and t.scales.shape == (128 * 4,)
    with pytest.raises(ValueError, match="CUDA tensor"):
        m3.mx_dequant(t, out=torch.zeros(4, 64))
    with pytest.raises(ValueError, match="shape"):
        m3.gemm_mx(t, t, out=torch.zeros(4, 5, dtype=torch.bfloat16))
