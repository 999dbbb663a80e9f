"""The norm of heads with their rotation against the fp64 oracle.

Tolerances, e = 2^-24.  A mean of N squares in fp32 is off by (N / 8 + 8) e of itself (eight a lane,
then a tree), rstd by half of that and 4 e more, v = u rstd w by 2 e more; sine and cosine
by 4 e and by the angle's 2^-25 turns, 4 e: so a rotated value by (N / 16 + 24) e of |v_re| + |v_im|.
Backward: dv by 12 e of |d_re| + |d_im|, the mean of g uh by (N / 8 + 40) e of the mean of magnitudes; so du by
rstd ((N + 60) e (|g| + mean |g uh| |uh|)) with |g| from |d_re| + |d_im|.  dw sums rows x heads terms
in any order: one e a term and 20 e each.  All doubled; bf16 outputs add half a step.
"""
import numpy as np
import pytest
import torch

import selective_state_space_m3ssd_b200 as m3
from oracle import layer as ly
from tests.gpu_util import np64

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32


def make(rows, Hq, Hk, N, R, dtype, seed=0, far=False, up=F32):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    head = lambda H: (2 * rn(rows, H, N) * torch.exp(0.5 * rn(rows, H, 1))).to(dtype)  # noqa: E731
    d = dict(q=head(Hq), k=head(Hk) if Hk else None, q_w=0.5 + torch.rand(N, generator=g),
             k_w=0.5 + torch.rand(N, generator=g) if Hk else None)
    if R:
        lo, hi = (-2 ** 31, 2 ** 31) if far else (-50, 5000)
        d["positions"] = torch.randint(lo, hi, (rows,), generator=g).to(torch.int32)
        d["freqs"] = 10000.0 ** (-torch.arange(R).float() * 2 / N)
    d["dq"] = rn(rows, Hq, N).to(up)
    d["dk"] = rn(rows, Hk, N).to(up) if Hk else None
    return d


def gpu(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def pos_of(d):
    return (d["positions"].numpy(), d["freqs"].double().numpy()) if "positions" in d else (None, None)


def both(v, R):
    """|re| + |im| of every rotated component, |v| of the others."""
    a = np.abs(v)
    o = a.copy()
    if R:
        p = a[..., :2 * R].reshape(*a.shape[:-1], R, 2).sum(-1, keepdims=True)
        o[..., :2 * R] = np.broadcast_to(p, (*p.shape[:-1], 2)).reshape(*a.shape[:-1], 2 * R)
    return o


def check(got, ref, tol, dtype, name):
    err = np.abs(np64(got) - ref)
    bad = ~(err <= 2 * tol + HALF[dtype] * (np.abs(ref) + 2 * tol) + 1e-37)
    assert not bad.any(), (name, float(np.max(err)), np.argwhere(bad)[:4])


def fwd(c, **kw):
    return m3.norm_rotate(c["q"], c["k"], c["q_w"], c["k_w"], positions=c.get("positions"),
                          freqs=c.get("freqs"), **kw)


def bwd(c, **kw):
    return m3.norm_rotate_bwd(c["q"], c["k"], c["q_w"], c["k_w"], c["dq"], c["dk"],
                              positions=c.get("positions"), freqs=c.get("freqs"), **kw)


def check_fwd(d, out, eps=1e-6):
    pos, f = pos_of(d)
    R = 0 if f is None else len(f)
    for n, o in zip("qk", out):
        if d[n] is None:
            assert o is None
            continue
        u = np64(d[n])
        w = 1.0 if d[n + "_w"] is None else np64(d[n + "_w"])
        v = ly.norm_rotate(u, w, None, None, eps)
        tol = (u.shape[-1] / 16 + 24) * E * both(v, R)
        check(o, ly.norm_rotate(u, w, pos, f, eps), tol, d[n].dtype, n)


def check_bwd(d, got, grad, eps=1e-6):
    pos, f = pos_of(d)
    R = 0 if f is None else len(f)
    for n in "qk":
        if d[n] is None:
            assert got["d" + n] is None and got["d" + n + "_w"] is None
            continue
        u, up = np64(d[n]), np64(d["d" + n])
        N = u.shape[-1]
        w = np.ones(N) if d[n + "_w"] is None else np64(d[n + "_w"])
        du, dw = ly.norm_rotate_bwd(u, w, up, pos, f, eps)
        rstd = 1 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
        m, uh = both(up, R), np.abs(u) * rstd
        g = m * w
        tol = rstd * (N + 60) * E * (g + (g * uh).mean(-1, keepdims=True) * uh)
        check(got["d" + n], du, tol, grad, "d" + n)
        tol = (u.shape[0] * u.shape[1] + N + 40) * E * (m * uh).sum((0, 1))
        check(got["d" + n + "_w"], dw, tol, F32, "d" + n + "_w")


SHAPES = [(1, 1, 1, 2, 1), (5, 1, 1, 8, 4), (3, 2, 1, 10, 3), (7, 3, 2, 64, 32), (2, 32, 8, 128, 64),
          (33, 4, 4, 128, 20), (9, 5, 3, 96, 48), (4, 7, 2, 256, 128), (11, 1, 2, 250, 125),
          (6, 33, 1, 18, 9), (700, 1, 1, 128, 64), (1300, 3, 1, 40, 0), (2, 40, 0, 72, 36),
          (300, 17, 5, 16, 8)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,Hq,Hk,N,R", SHAPES)
def test_forward(rows, Hq, Hk, N, R, dtype):
    d = make(rows, Hq, Hk, N, R, dtype, seed=rows + N)
    check_fwd(d, fwd(gpu(d)))
    d = make(rows, Hq, Hk, N, R, dtype, seed=N, far=True)
    d["q_w"] = d["k_w"] = None
    check_fwd(d, fwd(gpu(d), eps=0.5), 0.5)


@pytest.mark.parametrize("dtype,up,grad", [(BF, BF, BF), (BF, BF, F32), (BF, F32, BF), (BF, F32, F32),
                                           (F32, F32, F32)])
@pytest.mark.parametrize("rows,Hq,Hk,N,R", SHAPES)
def test_backward(rows, Hq, Hk, N, R, dtype, up, grad):
    d = make(rows, Hq, Hk, N, R, dtype, seed=rows + N, up=up)
    check_bwd(d, bwd(gpu(d), grad_dtype=grad), grad)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off,N", [(0, 64), (8, 64), (1, 64), (2, 10), (3, 10), (4, 24)])
def test_a_projections_rows_are_read_in_place(dtype, off, N):
    """q and k as column ranges of a projection, gradients into one; every alignment."""
    b, L, Hq, Hk = 3, 11, 3, 2
    d = make(b * L, Hq, Hk, N, N // 2, dtype, seed=2, up=dtype)
    width = off + (Hq + Hk) * N + 3
    zx = torch.randn(b, L, width).to(dtype)
    zx[..., off:off + Hq * N] = d["q"].view(b, L, -1)
    zx[..., off + Hq * N:-3] = d["k"].view(b, L, -1)
    z = zx.cuda()
    c = gpu(d)
    c["q"] = z[..., off:off + Hq * N].unflatten(-1, (Hq, N))
    c["k"] = z[..., off + Hq * N:-3].unflatten(-1, (Hk, N))
    c["positions"] = c["positions"].view(b, L)
    out = fwd(c)
    check_fwd(d, [o.flatten(0, 1) for o in out])
    c["dq"], c["dk"] = c["dq"].view(b, L, Hq, N), c["dk"].view(b, L, Hk, N)
    buf = torch.full((b, L, width), 7.0, device="cuda", dtype=dtype)
    grads = {"dq": buf[..., off:off + Hq * N].unflatten(-1, (Hq, N)),
             "dk": buf[..., off + Hq * N:-3].unflatten(-1, (Hk, N))}
    got = bwd(c, grad_dtype=dtype, grads=grads)
    check_bwd(d, {k: (v.reshape(b * L, -1, N) if v.dim() == 4 else v) for k, v in got.items()}, dtype)
    assert (buf[..., :off] == 7).all() and (buf[..., -3:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place_and_queries_alone(dtype):
    d = make(50, 6, 2, 128, 64, dtype, seed=3)
    c = gpu(d)
    q, k = fwd(c)
    q2, k2 = fwd(c, q_out=c["q"], k_out=c["k"])
    assert q2 is c["q"] and torch.equal(q, q2) and torch.equal(k, k2)
    only = gpu(dict(d, k=None, k_w=None, dk=None))
    q3, none = fwd(only)
    assert none is None and torch.equal(q3, q)
    g = bwd(gpu(d))
    g3 = bwd(only)
    assert g3["dk"] is None and torch.equal(g3["dq"], g["dq"])
    if dtype == F32:  # the gradient over the upstream one
        c = gpu(d)
        g4 = bwd(c, grads={"dq": c["dq"], "dk": c["dk"]})
        assert g4["dq"] is c["dq"] and all(torch.equal(g[n], g4[n]) for n in g)


def test_far_positions_keep_their_angle():
    """Positions of 10^9 at one radian each: the angle is good to 2^-25 of a turn."""
    pos = torch.tensor([0, 1, 10 ** 6, 10 ** 9, -10 ** 9, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    d = dict(q=torch.tensor([[[1.0, 0.0]]]).repeat(7, 1, 1), k=None, q_w=None, k_w=None, positions=pos,
             freqs=torch.tensor([1.0]))
    out = np64(fwd(gpu(d), eps=0.0)[0])[:, 0] / np.sqrt(2)
    ref = [(np.cos(v), np.sin(v)) for v in
           np.asarray(np.remainder(pos.numpy().astype(np.longdouble),
                                   2 * np.longdouble("3.14159265358979323846")), np.float64)]
    # 2^31 / 2 pi turns in fp64: 2^-25 of a turn; 8 e of sine, cosine, norm
    assert np.abs(out - ref).max() <= 2 * np.pi * (2.0 ** -25 + 2.0 ** -24) + 16 * E


def test_values_that_are_not_finite_stay_in_their_head():
    d = make(4, 3, 2, 64, 32, F32, seed=4)
    d["q"][1, 2, 5], d["k"][2, 0, 0] = float("nan"), float("inf")
    q, k = (t.cpu() for t in fwd(gpu(d)))
    assert torch.isnan(q[1, 2]).all() and torch.isnan(k[2, 0]).any()
    q[1, 2], k[2, 0] = 0, 0
    assert torch.isfinite(q).all() and torch.isfinite(k).all()
    zero = torch.zeros(2, 1, 16, device="cuda")
    assert not m3.norm_rotate(zero)[0].any()
    g = m3.norm_rotate_bwd(zero, None, None, None, zero + 1, None)
    assert torch.allclose(g["dq"], torch.full_like(zero, 1e3)) and not g["dq_w"].any()


def test_same_bits_again_and_in_a_graph():
    d = make(900, 5, 2, 128, 64, BF, seed=5, up=BF)
    c = gpu(d)
    out, g = fwd(c), bwd(c, grad_dtype=BF)
    q, k = torch.empty_like(out[0]), torch.empty_like(out[1])
    gr = {n: torch.empty_like(v) for n, v in g.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            fwd(c, q_out=q, k_out=k)
            bwd(c, grad_dtype=BF, grads=gr)
    for _ in range(2):
        for t in (q, k, *gr.values()):
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, out[0]) and torch.equal(k, out[1])
        assert all(torch.equal(g[n], gr[n]) for n in g)


def test_gradients_against_differences():
    """Along random directions.  The loss sums 20 x 5 x 64 products within 40 e of themselves:
    below 1e-3 in all; over a step of 2 x 2e-2 that leaves 3e-2 of some 100, and the third
    derivative of a norm at a distance of 2e-2 of some 16 less."""
    d = make(20, 4, 1, 64, 32, F32, seed=6)
    c = gpu(d)
    got = bwd(c)
    loss = lambda e: sum(float((o.double() * c["d" + n].double()).sum())  # noqa: E731
                         for n, o in zip("qk", fwd(e)))
    g = torch.Generator().manual_seed(7)
    for k, n in (("q", "dq"), ("k", "dk"), ("q_w", "dq_w"), ("k_w", "dk_w")):
        v = torch.randn(c[k].shape, generator=g).cuda()
        v /= v.norm()
        hi, lo = (loss(dict(c, **{k: c[k] + sgn * 2e-2 * v})) for sgn in (1, -1))
        want, scale = float((got[n].double() * v.double()).sum()), float(got[n].double().norm())
        assert abs((hi - lo) / 4e-2 - want) <= 3e-2 + 1e-3 * scale, (k, hi - lo, want)


def test_empty_calls():
    q = torch.empty(0, 2, 8, device="cuda")
    out, _ = m3.norm_rotate(q)
    assert out.shape == q.shape
    g = m3.norm_rotate_bwd(q, q, None, None, q, q)
    assert not g["dq_w"].any() and not g["dk_w"].any()
