"""Host validation of the operators around the scan (no GPU: nothing here reaches a kernel)."""
import ctypes

import pytest
import torch

import selective_state_space_m3ssd_b200 as m3
from selective_state_space_m3ssd_b200 import build as m3build

P = ctypes.c_void_p
A, ODD = P(0x10000), P(0x10001)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    m3build.build()
    return m3.load()


def glr_dims(**kw):
    d = dict(batch=2, seqlen=8, width=6, ldx=6, ldr=6, ldi=6, x_dtype=m3.F32, c=8.0, reserved=0)
    d.update(kw)
    return m3.GlrDims(*(d[n] for n, _ in m3.GlrDims._fields_))


GLR_FWD = ("x", "r", "i", "rate", "bias_r", "bias_i", "h0", "reset", "lengths", "y", "hT")


def glr_fwd(lib, dims, ws=A, nbytes=1 << 20, **kw):
    a = {n: A for n in GLR_FWD}
    a.update(kw)
    return lib.m3ssd_glr_fwd(ctypes.byref(dims), *(a[n] for n in GLR_FWD), ws, nbytes, None)


def glr_bwd(lib, dims, grads=None, ws=A, nbytes=1 << 20, **kw):
    names = GLR_FWD[:9] + ("y", "dy", "dhT")
    a = {n: A for n in names}
    a.update(kw)
    g = grads if grads is not None else m3.GlrGrads(6, m3.F32, 0, *[0x10000] * 7)
    return lib.m3ssd_glr_bwd(ctypes.byref(dims), *(a[n] for n in names), ctypes.byref(g), ws, nbytes, None)


def glr_step(lib, dims, **kw):
    names = ("x", "r", "i", "rate", "bias_r", "bias_i", "h", "h_out", "y")
    a = {n: A for n in names}
    a.update(kw)
    return lib.m3ssd_glr_step(ctypes.byref(dims), *(a[n] for n in names), None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), m3.ERR_INVALID_ARG), (dict(width=0), m3.ERR_INVALID_ARG),
    (dict(ldx=5), m3.ERR_INVALID_ARG), (dict(ldr=5), m3.ERR_INVALID_ARG),
    (dict(ldi=0), m3.ERR_INVALID_ARG), (dict(x_dtype=5), m3.ERR_INVALID_ARG),
    (dict(c=0.0), m3.ERR_INVALID_ARG), (dict(c=-1.0), m3.ERR_INVALID_ARG),
    (dict(c=float("nan")), m3.ERR_INVALID_ARG), (dict(c=float("inf")), m3.ERR_INVALID_ARG),
    (dict(reserved=1), m3.ERR_INVALID_ARG), (dict(ldx=1 << 31), m3.ERR_UNSUPPORTED),
    (dict(batch=1 << 30, width=64, ldx=64, ldr=64, ldi=64), m3.ERR_UNSUPPORTED),
    (dict(batch=1 << 40), m3.ERR_UNSUPPORTED),
    (dict(width=1 << 32, ldx=1 << 32, ldr=1 << 32, ldi=1 << 32), m3.ERR_UNSUPPORTED)])
def test_glr_rejects_bad_dims(lib, kw, status):
    d = glr_dims(**kw)
    assert glr_fwd(lib, d) == glr_bwd(lib, d) == glr_step(lib, d) == status
    assert lib.m3ssd_glr_bwd_workspace_size(ctypes.byref(d)) == 0


def test_glr_rejects_bad_lengths_and_null_dims(lib):
    assert glr_fwd(lib, glr_dims(seqlen=-1)) == m3.ERR_INVALID_ARG
    assert glr_fwd(lib, glr_dims(seqlen=1 << 31)) == m3.ERR_UNSUPPORTED
    assert lib.m3ssd_glr_bwd_workspace_size(None) == 0


def test_glr_rejects_null_and_misaligned_pointers(lib):
    d = glr_dims()
    for n in ("x", "r", "i", "rate", "y"):
        assert glr_fwd(lib, d, **{n: None}) == m3.ERR_INVALID_ARG, n
    for n in GLR_FWD:
        if n != "reset":
            assert glr_fwd(lib, d, **{n: ODD}) == m3.ERR_INVALID_ARG, n
    for n in ("x", "r", "i", "rate", "h", "y"):
        assert glr_step(lib, d, **{n: None}) == m3.ERR_INVALID_ARG, n
        assert glr_step(lib, d, **{n: ODD}) == m3.ERR_INVALID_ARG, n
    assert glr_step(lib, d, h_out=ODD) == m3.ERR_INVALID_ARG
    for n in ("x", "r", "i", "rate", "y", "dy"):
        assert glr_bwd(lib, d, **{n: None}) == m3.ERR_INVALID_ARG, n
        assert glr_bwd(lib, d, **{n: ODD}) == m3.ERR_INVALID_ARG, n
    assert glr_bwd(lib, d, dhT=ODD) == m3.ERR_INVALID_ARG
    for j, n in enumerate(m3.GLR_GRAD_NAMES):
        p = [0x10000] * 7
        p[j] = 0x10001
        assert glr_bwd(lib, d, m3.GlrGrads(6, m3.F32, 0, *p)) == m3.ERR_INVALID_ARG, n
        if n in ("dx", "dr", "di", "drate"):
            p[j] = None
            assert glr_bwd(lib, d, m3.GlrGrads(6, m3.F32, 0, *p)) == m3.ERR_INVALID_ARG, n


def test_glr_rejects_bad_gradients_and_workspaces(lib):
    d, p = glr_dims(), [0x10000] * 7
    assert glr_bwd(lib, d, m3.GlrGrads(5, m3.F32, 0, *p)) == m3.ERR_INVALID_ARG
    assert glr_bwd(lib, d, m3.GlrGrads(1 << 31, m3.F32, 0, *p)) == m3.ERR_UNSUPPORTED
    assert glr_bwd(lib, d, m3.GlrGrads(6, 9, 0, *p)) == m3.ERR_INVALID_ARG
    assert glr_bwd(lib, d, m3.GlrGrads(6, m3.F32, 1, *p)) == m3.ERR_INVALID_ARG
    assert glr_bwd(lib, d, m3.GlrGrads(6, m3.BF16, 0, *p)) == m3.ERR_UNSUPPORTED  # fp32 inputs
    long = glr_dims(batch=1, seqlen=4096)  # few sequences: cut into parts
    need = lib.m3ssd_glr_fwd_workspace_size(ctypes.byref(long))
    assert need > 0 and lib.m3ssd_glr_fwd_workspace_size(ctypes.byref(d)) == 0
    assert glr_fwd(lib, long, nbytes=need - 1) == m3.ERR_WORKSPACE
    assert glr_fwd(lib, long, ws=None) == m3.ERR_WORKSPACE
    assert glr_fwd(lib, long, ws=P(0x10010)) == m3.ERR_WORKSPACE
    need = lib.m3ssd_glr_bwd_workspace_size(ctypes.byref(d))
    assert need > 0
    assert glr_bwd(lib, d, nbytes=need - 1) == m3.ERR_WORKSPACE
    assert glr_bwd(lib, d, ws=None) == m3.ERR_WORKSPACE
    assert glr_bwd(lib, d, ws=P(0x10080)) == m3.ERR_WORKSPACE


def test_glr_without_sequences_is_a_no_op(lib):
    d = glr_dims(batch=0)
    none = {n: None for n in GLR_FWD if n != "rate"}
    assert glr_fwd(lib, d, **none) == m3.OK
    assert glr_step(lib, d, x=None, r=None, i=None, h=None, h_out=None, y=None) == m3.OK


def test_glr_binding_refuses_on_the_host():
    x, v = torch.zeros(2, 3, 8), torch.zeros(8)
    for f, a in ((m3.glr_fwd, (x, x, x, v)), (m3.glr_bwd, (x, x, x, v, x, x)),
                 (m3.glr_step, (x[:, 0], x[:, 0], x[:, 0], x[:, 0], v))):
        with pytest.raises(ValueError):
            f(*a)
    with pytest.raises(ValueError):
        m3.glr_fwd(x[0], x[0], x[0], v)


def test_row_strides_of_token_tensors():
    """The binding's rule for rows a fixed distance apart (device -1 is the host)."""
    f = lambda t, lead, *w: m3._tokens_stride(t, "t", t.dtype, lead, w, -1)  # noqa: E731
    p = torch.zeros(3, 5, 40)
    assert f(p[..., 8:16], (3, 5), 8) == 40 and f(p, (3, 5), 40) == 40
    assert f(p[:1, :, 8:16], (1, 5), 8) == 40 and f(p[:, :1, 8:16], (3, 1), 8) == 200
    assert f(p[:1, :1, 8:16], (1, 1), 8) == 8 and f(p[:, 0, 8:16], (3,), 8) == 200
    assert f(p[..., 8:20].unflatten(-1, (3, 4)), (3, 5), 3, 4) == 40
    assert f(p[..., 8:20].unflatten(-1, (3, 4))[..., :1, :], (3, 5), 1, 4) == 40
    with pytest.raises(ValueError):  # a token's heads apart
        f(p[..., 8:20].unflatten(-1, (3, 4))[..., :2], (3, 5), 3, 2)
    for bad in (p[:, :4, 8:16], p[..., ::5], p[:, :, :1].expand(3, 5, 8), p[:, ::2, :8][:, :2],
                torch.zeros(5, 3, 8).transpose(0, 1), torch.zeros(5, 8).expand(3, 5, 8)):
        with pytest.raises(ValueError):
            f(bad, tuple(bad.shape[:-1]), 8)


def rot_dims(**kw):
    d = dict(rows=4, q_heads=3, k_heads=2, width=8, pairs=4, ldq=24, ldk=16, x_dtype=m3.F32, eps=1e-6,
             reserved=0)
    d.update(kw)
    return m3.RotateDims(*(d[n] for n, _ in m3.RotateDims._fields_))


ROT_IN = ("q", "k", "q_w", "k_w", "positions", "freqs")


def rot_fwd(lib, dims, **kw):
    a = {n: A for n in ROT_IN + ("q_out", "k_out")}
    a.update(kw)
    return lib.m3ssd_norm_rotate(ctypes.byref(dims), *(a[n] for n in ROT_IN + ("q_out", "k_out")), None)


def rot_bwd(lib, dims, grads=None, up=m3.F32, ws=A, nbytes=1 << 24, **kw):
    a = {n: A for n in ROT_IN + ("dq_out", "dk_out")}
    a.update(kw)
    g = grads if grads is not None else m3.RotateGrads(24, 16, m3.F32, 0, *[0x10000] * 4)
    return lib.m3ssd_norm_rotate_bwd(ctypes.byref(dims), *(a[n] for n in ROT_IN), up, a["dq_out"],
                                     a["dk_out"], ctypes.byref(g), ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), m3.ERR_INVALID_ARG), (dict(q_heads=0), m3.ERR_INVALID_ARG),
    (dict(k_heads=-1), m3.ERR_INVALID_ARG), (dict(width=7), m3.ERR_INVALID_ARG),
    (dict(width=0), m3.ERR_INVALID_ARG), (dict(pairs=5), m3.ERR_INVALID_ARG),
    (dict(pairs=-1), m3.ERR_INVALID_ARG), (dict(ldq=23), m3.ERR_INVALID_ARG),
    (dict(ldk=15), m3.ERR_INVALID_ARG), (dict(x_dtype=2), m3.ERR_INVALID_ARG),
    (dict(eps=-1.0), m3.ERR_INVALID_ARG), (dict(eps=float("nan")), m3.ERR_INVALID_ARG),
    (dict(reserved=1), m3.ERR_INVALID_ARG), (dict(width=258, ldq=1000, ldk=1000), m3.ERR_UNSUPPORTED),
    (dict(rows=1 << 31), m3.ERR_UNSUPPORTED), (dict(rows=(1 << 31) // 5 + 1), m3.ERR_UNSUPPORTED),
    (dict(ldq=1 << 31), m3.ERR_UNSUPPORTED),
    (dict(rows=((1 << 31) - (1 << 16)) // 5 + 1), m3.ERR_UNSUPPORTED),
    (dict(rows=(1 << 31) - 2, q_heads=1, k_heads=0), m3.ERR_UNSUPPORTED),
    (dict(q_heads=65536, ldq=1 << 20), m3.ERR_UNSUPPORTED)])
def test_rotate_rejects_bad_dims(lib, kw, status):
    d = rot_dims(**kw)
    assert rot_fwd(lib, d) == rot_bwd(lib, d) == status
    assert lib.m3ssd_norm_rotate_bwd_workspace_size(ctypes.byref(d)) == 0


def test_rotate_rejects_null_and_misaligned_pointers(lib):
    d = rot_dims()
    for n in ("q", "k", "positions", "freqs", "q_out", "k_out"):
        assert rot_fwd(lib, d, **{n: None}) == m3.ERR_INVALID_ARG, n
    for n in ROT_IN + ("q_out", "k_out"):
        assert rot_fwd(lib, d, **{n: ODD}) == m3.ERR_INVALID_ARG, n
    for n in ("q", "k", "positions", "freqs", "dq_out", "dk_out"):
        assert rot_bwd(lib, d, **{n: None}) == m3.ERR_INVALID_ARG, n
        assert rot_bwd(lib, d, **{n: ODD}) == m3.ERR_INVALID_ARG, n
    p = [0x10000] * 4
    for j in range(4):
        bad = list(p)
        bad[j] = 0x10002
        assert rot_bwd(lib, d, m3.RotateGrads(24, 16, m3.F32, 0, *bad)) == m3.ERR_INVALID_ARG
    for j in range(2):
        bad = list(p)
        bad[j] = None
        assert rot_bwd(lib, d, m3.RotateGrads(24, 16, m3.F32, 0, *bad)) == m3.ERR_INVALID_ARG
    assert rot_bwd(lib, d, m3.RotateGrads(23, 16, m3.F32, 0, *p)) == m3.ERR_INVALID_ARG
    assert rot_bwd(lib, d, m3.RotateGrads(24, 15, m3.F32, 0, *p)) == m3.ERR_INVALID_ARG
    assert rot_bwd(lib, d, m3.RotateGrads(24, 16, m3.BF16, 0, *p)) == m3.ERR_UNSUPPORTED
    assert rot_bwd(lib, d, up=m3.BF16) == m3.ERR_UNSUPPORTED
    assert rot_bwd(lib, d, up=9) == m3.ERR_INVALID_ARG
    need = lib.m3ssd_norm_rotate_bwd_workspace_size(ctypes.byref(d))
    assert need > 0 and rot_bwd(lib, d, nbytes=need - 1) == m3.ERR_WORKSPACE
    assert rot_bwd(lib, d, ws=None) == rot_bwd(lib, d, ws=P(0x10040)) == m3.ERR_WORKSPACE


def test_rotate_without_tokens_is_a_no_op(lib):
    none = {n: None for n in ("q", "k", "positions", "q_out", "k_out")}
    assert rot_fwd(lib, rot_dims(rows=0), **none) == m3.OK


def test_rotate_binding_refuses_on_the_host():
    q, w = torch.zeros(2, 3, 8), torch.zeros(8)
    with pytest.raises(ValueError):
        m3.norm_rotate(q, q, w, w)
    with pytest.raises(ValueError):
        m3.norm_rotate_bwd(q, q, w, w, q, q)
    with pytest.raises(ValueError):
        m3.norm_rotate(w)


def w4(**kw):
    d = dict(rows=4, cols=100, group=32, reserved=0, codes=0x10000, scales=0x10000, zeros=None)
    d.update(kw)
    return m3.W4(*(d[n] for n, _ in m3.W4._fields_))


def gemv(lib, W, tokens=2, xd=m3.F32, x=A, ldx=100, od=m3.F32, out=A, ldd=4):
    return lib.m3ssd_gemv_w4(tokens, xd, x, ldx, ctypes.byref(W), od, out, ldd, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), m3.ERR_INVALID_ARG), (dict(cols=0), m3.ERR_INVALID_ARG),
    (dict(group=0), m3.ERR_INVALID_ARG), (dict(group=16), m3.ERR_INVALID_ARG),
    (dict(group=96), m3.ERR_INVALID_ARG), (dict(group=160), m3.ERR_INVALID_ARG),
    (dict(reserved=1), m3.ERR_INVALID_ARG), (dict(codes=None), m3.ERR_INVALID_ARG),
    (dict(scales=None), m3.ERR_INVALID_ARG), (dict(codes=0x10008), m3.ERR_INVALID_ARG),
    (dict(scales=0x10001), m3.ERR_INVALID_ARG), (dict(rows=1 << 31), m3.ERR_UNSUPPORTED),
    (dict(cols=1 << 30), m3.ERR_UNSUPPORTED), (dict(rows=1 << 30, cols=1 << 14), m3.ERR_UNSUPPORTED)])
def test_w4_rejects_bad_weights(lib, kw, status):
    W = w4(**kw)
    big = 1 << 31
    assert gemv(lib, W, ldx=big, ldd=big) == status
    assert lib.m3ssd_w4_quant(ctypes.byref(W), m3.F32, A, big, None) == status
    assert lib.m3ssd_w4_dequant(ctypes.byref(W), m3.F32, A, big, None) == status


def test_w4_rejects_bad_arguments(lib):
    assert gemv(lib, w4(), tokens=-1) == m3.ERR_INVALID_ARG
    assert gemv(lib, w4(), tokens=17) == m3.ERR_UNSUPPORTED
    for kw in (dict(xd=5), dict(od=5), dict(ldx=99), dict(ldd=3), dict(x=None), dict(out=None), dict(x=ODD),
               dict(out=ODD)):
        assert gemv(lib, w4(), **kw) == m3.ERR_INVALID_ARG, kw
    for f in (lib.m3ssd_w4_quant, lib.m3ssd_w4_dequant):
        for dt, p, ld in ((5, A, 100), (m3.F32, None, 100), (m3.F32, ODD, 100), (m3.F32, A, 99)):
            assert f(ctypes.byref(w4()), dt, p, ld, None) == m3.ERR_INVALID_ARG
        assert f(None, m3.F32, A, 100, None) == m3.ERR_INVALID_ARG
        assert f(ctypes.byref(w4(rows=0, codes=None, scales=None)), m3.F32, None, 100, None) == m3.OK
    assert gemv(lib, w4(), tokens=0, x=None, out=None) == m3.OK
    assert gemv(lib, w4(rows=0, codes=None, scales=None), x=None, out=None) == m3.OK
    assert lib.m3ssd_w4_codes_size(17, 129) == 2 * 2 * 1024 and lib.m3ssd_w4_codes_size(1, 0) == 0


def test_w4_binding_refuses_on_the_host():
    W = m3.W4Tensor.empty(8, 64, 32, device="cpu")
    for f in (lambda: m3.gemv_w4(torch.zeros(1, 64), W), lambda: m3.w4_quant(torch.zeros(8, 64)),
              lambda: m3.w4_dequant(W), lambda: m3.W4Tensor.empty(8, 64, 48, device="cpu")):
        with pytest.raises(ValueError):
            f()


@pytest.mark.parametrize("rows,cols,group", [(1, 1, 32), (16, 128, 128), (19, 333, 64), (40, 700, 256)])
def test_w4_codes_from_elsewhere_are_laid_out(rows, cols, group):
    from oracle import layer as ly
    g = torch.Generator().manual_seed(1)
    codes = torch.randint(0, 16, (rows, cols), generator=g, dtype=torch.uint8)
    n = -(-cols // group)
    scales, zeros = torch.rand(rows, n, generator=g), torch.randint(0, 16, (rows, n), dtype=torch.uint8)
    W = m3.W4Tensor.from_codes(codes, scales, zeros, group=group)
    assert (ly.w4_codes(W.codes.numpy(), rows, cols) == codes.numpy()).all()
    assert torch.equal(W.scales, scales.bfloat16().t()) and torch.equal(W.zeros, zeros.t())
    assert W.codes.numel() == m3._w4_codes(rows, cols)
    with pytest.raises(ValueError):
        m3.W4Tensor.from_codes(codes, scales[:, :-1], group=group)


def test_w4_codes_from_elsewhere_are_checked():
    """A code above 15 would run into its neighbour's byte half, or lose bits."""
    codes = torch.full((20, 200), 15, dtype=torch.uint8)
    scales, zeros = torch.ones(20, 2), torch.full((20, 2), 15, dtype=torch.uint8)
    m3.W4Tensor.from_codes(codes, scales, zeros)
    for r, k in ((0, 0), (19, 199), (7, 33)):
        bad = codes.clone()
        bad[r, k] = 16
        with pytest.raises(ValueError, match="codes must be 0 to 15, got 16"):
            m3.W4Tensor.from_codes(bad, scales, zeros)
    zeros[3, 1] = 255
    with pytest.raises(ValueError, match="zeros must be 0 to 15, got 255"):
        m3.W4Tensor.from_codes(codes, scales, zeros)
    empty = m3.W4Tensor.from_codes(codes[:0], scales[:0])
    assert empty.rows == 0 and empty.codes.numel() == 0
