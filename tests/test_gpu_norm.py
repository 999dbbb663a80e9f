"""The residual addition with the RMS norm and its backward against the fp64 oracle.

Forward: r is one fp32 sum rounded once, so it is compared bit for bit.  y carries at most
2^-19 of relative fp32 error: the sum of squares runs over at most 32 terms a thread, 5
shuffles and 16 partial sums (53 roundings of 2^-24, halved by the square root), and six
more roundings; 33 2^-24 < 2^-18.9 is rounded up to 2^-18.  In bf16 half a step (2^-8) is
added; quantised, half a step of the code and a scale that fits the same bound.
Backward: dr's terms to 96 2^-24 of their magnitudes (the row's dot product has as many
roundings as the forward's sum, not halved, and about 30 more); dw to (rows + 32) 2^-24 of
the sum of magnitudes."""
import numpy as np
import pytest
import torch

import selective_state_space_m3ssd_b200 as m3
from oracle import lowbit as ol

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
FP = 2.0 ** -18
SHAPES = [(1, 1), (1, 7), (3, 32), (2, 100), (37, 64), (130, 257), (300, 768), (5, 1024),
          (700, 1000), (4, 4096), (3, 4097), (2, 8200), (2, 16384)]


def inputs(rows, d, dtype, res, seed=0):
    g = torch.Generator().manual_seed(rows + 31 * d + seed)
    x = torch.randn(rows, d, generator=g).to(dtype)
    r = None if res is None else (3 * torch.randn(rows, d, generator=g) *
                                  torch.exp(torch.randn(rows, 1, generator=g))).to(res)
    return x, r, 0.5 + torch.rand(d, generator=g)


def cu(*ts):
    return [None if t is None else t.cuda() for t in ts]


def np64(t):
    return t.detach().cpu().double().numpy()


def summed(x, res):
    return x if res is None else (x.float() + res.float()).to(res.dtype)


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("dtype,res", [(F32, None), (BF16, None), (BF16, F32), (BF16, BF16),
                                       (F32, F32), (F32, BF16)])
def test_forward(rows, d, dtype, res):
    x, r, w = inputs(rows, d, dtype, res)
    xc, rc, wc = cu(x, r, w)
    y, out, rstd = m3.add_rmsnorm(xc, wc, residual=rc, eps=1e-5, want_rstd=True)
    s = summed(x, r)
    if r is None:
        assert out is None
    else:
        assert torch.equal(out.cpu(), s)
    ref, ref_rstd = ol.rmsnorm(np64(s), np64(w), 1e-5)
    assert y.dtype == dtype and np.all(np.abs(np64(rstd) - ref_rstd) <= FP * ref_rstd)
    tol = FP + (2.0 ** -8 if dtype == BF16 else 0)
    assert np.all(np.abs(np64(y) - ref) <= tol * np.abs(ref) + 1e-38)


# more rows than walkers at the end, unaligned and aligned
@pytest.mark.parametrize("rows,d", SHAPES + [(9001, 100), (2501, 512)])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype,res", [(BF16, F32), (F32, None)])
def test_quantised_output(rows, d, fmt, dtype, res):
    x, r, w = inputs(rows, d, dtype, res)
    t = m3.MXTensor.empty(fmt, rows, d, "cuda")
    t.codes.fill_(0x5A)
    t.scales.fill_(0xA5)
    xc, rc, wc = cu(x, r, w)
    y, out, _ = m3.add_rmsnorm(xc, wc, residual=rc, fmt=fmt, y=t)
    assert y is t and (r is None or torch.equal(out.cpu(), summed(x, r)))
    ref = ol.rmsnorm(np64(summed(x, r)), np64(w), 1e-6)[0]
    codes, tiles = t.codes.cpu().numpy(), t.scales.cpu().numpy()
    got = ol.mx_load(codes, tiles, rows, d, fmt)
    # scales that stand for 2^E as the definition chooses it, up to the fp32 error of amax
    _, s = ol.mx_encode(ref, fmt)
    lo, hi = (ol.mx_encode(ref * f, fmt)[1] for f in (1 - FP, 1 + FP))
    nb = s.shape[1]
    want = ol.mx_store(np.zeros((rows, 32 * nb), np.uint8), s, "mxfp8")[1]
    low, high = (ol.mx_store(np.zeros((rows, 32 * nb), np.uint8), v, "mxfp8")[1] for v in (lo, hi))
    assert np.all((tiles >= low) & (tiles <= high)), (tiles != want).sum()
    # values within half a step of their code
    half, floor = (0.25, 0.25) if fmt == "mxfp4" else (2.0 ** -4, 2.0 ** -10)
    unit = np.repeat(2.0 ** (hi.astype(float) - 127), 32, -1)[:, :d]
    assert np.all(np.abs(got - ref) <= np.maximum(half * np.abs(ref), floor * unit) * (1 + 4 * FP))
    # the padding is zero
    kp = codes.shape[1] * (2 if fmt == "mxfp4" else 1)
    assert not codes[:, (d + 1) // 2 if fmt == "mxfp4" else d:].any() or kp == d


# every offset of a row inside an access; rows that end in the last access of their padding
@pytest.mark.parametrize("rows,d", [(5000, 33), (1301, 257), (640, 1021), (900, 1049), (150, 4093),
                                    (160, 8191), (150, 9001), (60, 16377), (60, 16383)])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype,res", [(BF16, BF16), (F32, F32), (F32, BF16)])
def test_quantised_odd_widths(rows, d, fmt, dtype, res):
    test_quantised_output(rows, d, fmt, dtype, res)


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("dtype,res", [(BF16, F32), (BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("dres", [False, True])
def test_backward(rows, d, dtype, res, dres):
    dy, r, w = inputs(rows, d, dtype, res, 7)
    g = torch.Generator().manual_seed(3)
    up = torch.randn(rows, d, generator=g) if dres else None
    rstd = torch.from_numpy(ol.rmsnorm(np64(r), np64(w), 1e-6)[1]).float()
    dr, dw = m3.add_rmsnorm_bwd(*cu(dy, r, w, rstd), dres=None if up is None else up.cuda())
    a = [np64(t) for t in (dy, r, w, rstd)]
    ref_dr, ref_dw = ol.rmsnorm_bwd(*a, None if up is None else np64(up))
    gm, rh, s = np.abs(a[0] * a[2]), np.abs(a[1]) * a[3][:, None], a[3][:, None]
    mag = s * (gm + rh * (gm * rh).mean(-1, keepdims=True)) + (0 if up is None else np.abs(np64(up)))
    assert np.all(np.abs(np64(dr) - ref_dr) <= 96 * 2.0 ** -24 * mag + 1e-38)
    mag = (np.abs(a[0]) * rh).sum(0)
    assert np.all(np.abs(np64(dw) - ref_dw) <= (rows + 32) * 2.0 ** -24 * mag + 1e-38)
    again = m3.add_rmsnorm_bwd(*cu(dy, r, w, rstd), dres=None if up is None else up.cuda())
    assert torch.equal(again[0], dr) and torch.equal(again[1], dw)  # fixed order of sums


def test_gradient_of_the_kernels_against_differences():
    """Differences of the fp32 forward kernel itself: y moves by h dr . e along e; with h =
    2^-7 the truncation is below 2 h^2 and the fp32 rounding of the two sums below
    d 2^-23 / h of the terms."""
    rows, d = 4, 96
    r, _, w = inputs(rows, d, F32, None, 5)
    dy, _, e = inputs(rows, d, F32, None, 6)
    e = torch.randn(rows, d, generator=torch.Generator().manual_seed(1))
    _, _, rstd = m3.add_rmsnorm(*cu(r, w), want_rstd=True)
    dr, dw = m3.add_rmsnorm_bwd(*cu(dy, r, w), rstd)
    h = 2.0 ** -7
    loss = lambda r, w: (m3.add_rmsnorm(*cu(r, w))[0].double().cpu() * dy.double()).sum()  # noqa: E731
    got = (loss(r + h * e, w) - loss(r - h * e, w)) / (2 * h)
    want = (dr.double().cpu() * e.double()).sum()
    scale = (dy.double() * w.double()).norm() * e.double().norm()
    assert abs(got - want) <= (2 * h * h + d * 2.0 ** -23 / h) * scale
    ew = torch.randn(d, generator=torch.Generator().manual_seed(2))
    got = (loss(r, w + h * ew) - loss(r, w - h * ew)) / (2 * h)
    assert abs(got - (dw.double().cpu() * ew.double()).sum()) <= d * 2.0 ** -23 / h * scale


def test_many_rows_walk_the_grid():
    """More rows than CTAs, so a CTA walks several (and sums their dw)."""
    rows, d = 20011, 256
    x, r, w = inputs(rows, d, BF16, F32)
    xc, rc, wc = cu(x, r, w)
    y, out, rstd = m3.add_rmsnorm(xc, wc, residual=rc, want_rstd=True)
    assert torch.equal(out.cpu(), summed(x, r))
    ref = ol.rmsnorm(np64(out), np64(w), 1e-6)[0]
    assert np.all(np.abs(np64(y) - ref) <= (FP + 2.0 ** -8) * np.abs(ref))
    dr, dw = m3.add_rmsnorm_bwd(xc, out, wc, rstd)
    ref_dr, ref_dw = ol.rmsnorm_bwd(np64(x), np64(out), np64(w), np64(rstd))
    rh = np.abs(np64(out)) * np64(rstd)[:, None]
    gm = np.abs(np64(x) * np64(w))
    mag = np64(rstd)[:, None] * (gm + rh * (gm * rh).mean(-1, keepdims=True))
    assert np.all(np.abs(np64(dr) - ref_dr) <= 96 * 2.0 ** -24 * mag)
    # a CTA's chain is at most rows / 300 long (2 CTAs an SM or more), then 300 / 8 + 8 sums
    assert np.all(np.abs(np64(dw) - ref_dw) <= 256 * 2.0 ** -24 * (np.abs(np64(x)) * rh).sum(0))


def test_unaligned_tensors_and_in_place():
    rows, d = 33, 512
    x, r, w = inputs(rows, d, BF16, F32)
    want = [t.clone() for t in m3.add_rmsnorm(*cu(x, w), residual=r.cuda(), want_rstd=True)]
    buf = torch.empty(rows * d + 1, dtype=BF16, device="cuda")
    xo = buf[1:].view(rows, d).copy_(x)
    rbuf = torch.empty(rows * d + 1, device="cuda")
    ro = rbuf[1:].view(rows, d).copy_(r)
    y, out, rstd = m3.add_rmsnorm(xo, w.cuda(), residual=ro, residual_out=ro, y=xo, want_rstd=True)
    assert y is xo and out is ro and torch.equal(out, want[1])
    # rows that are not aligned are summed in another order: both are within FP (and half a
    # step of bf16) of the exact value, so within twice that of each other
    assert np.all(np.abs(np64(rstd) - np64(want[2])) <= 2 * FP * np64(rstd))
    assert np.all(np.abs(np64(y) - np64(want[0])) <= 2 * (FP + 2.0 ** -8) * np.abs(np64(y)))
    rstd = want[2]
    up = torch.randn(rows, d, device="cuda")
    a = m3.add_rmsnorm_bwd(x.cuda(), want[1], w.cuda(), rstd, dres=up)
    b = m3.add_rmsnorm_bwd(x.cuda(), want[1], w.cuda(), rstd, dres=up, dr=up)
    assert b[0] is up and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# widths that are no multiple of eight, walkers of several rows: every offset of a row inside
# an access, the widest rows there are
@pytest.mark.parametrize("rows,d", [(5000, 33), (1301, 257), (2003, 1049), (700, 4103), (333, 9001),
                                    (200, 16377), (200, 16383)])
@pytest.mark.parametrize("dtype,res", [(BF16, F32), (BF16, BF16), (F32, F32), (F32, BF16)])
def test_odd_widths(rows, d, dtype, res):
    """Forward in place and backward against fp64, nothing written behind the tensors' ends, and
    a NaN stays in its row."""
    def guarded(t):
        buf = torch.full((rows * d + 64,), 7.0, dtype=t.dtype, device="cuda")
        buf[:rows * d] = t.reshape(-1).cuda()
        return buf, buf[:rows * d].view(rows, d)
    x, r, w = inputs(rows, d, dtype, res, 1)
    wc, s = w.cuda(), summed(x, r)
    (xb, xc), (rb, rc) = guarded(x), guarded(r)
    y, out, rstd = m3.add_rmsnorm(xc, wc, residual=rc, residual_out=rc, y=xc, want_rstd=True)
    assert torch.equal(out.cpu(), s)
    ref, ref_rstd = ol.rmsnorm(np64(s), np64(w), 1e-6)
    assert np.all(np.abs(np64(rstd) - ref_rstd) <= FP * ref_rstd)
    tol = FP + (2.0 ** -8 if dtype == BF16 else 0)
    assert np.all(np.abs(np64(y) - ref) <= tol * np.abs(ref) + 1e-38)
    assert torch.all(xb[rows * d:] == 7) and torch.all(rb[rows * d:] == 7)
    up = torch.randn(rows, d, generator=torch.Generator().manual_seed(4))
    (ub, uc), dy = guarded(up), x.cuda()
    dr, dw = m3.add_rmsnorm_bwd(dy, out, wc, rstd, dres=uc, dr=uc)
    a = [np64(t) for t in (x, s, w, rstd)]
    ref_dr, ref_dw = ol.rmsnorm_bwd(*a, np64(up))
    gm, rh, sc = np.abs(a[0] * a[2]), np.abs(a[1]) * a[3][:, None], a[3][:, None]
    mag = sc * (gm + rh * (gm * rh).mean(-1, keepdims=True)) + np.abs(np64(up))
    assert np.all(np.abs(np64(dr) - ref_dr) <= 96 * 2.0 ** -24 * mag + 1e-38)
    assert np.all(np.abs(np64(dw) - ref_dw) <=
                  (rows + 32) * 2.0 ** -24 * (np.abs(a[0]) * rh).sum(0) + 1e-38)
    assert torch.all(ub[rows * d:] == 7)
    bad = rows // 2
    dy[bad] = float("nan")
    assert torch.isnan(m3.add_rmsnorm(dy, wc, residual=out)[0]).any(1).nonzero().flatten().tolist() \
        == [bad]
    dr, dw2 = m3.add_rmsnorm_bwd(dy, out, wc, rstd)
    assert torch.isnan(dr).any(1).nonzero().flatten().tolist() == [bad] and torch.isnan(dw2).all()


def test_nonfinite_and_zero_rows():
    x, _, w = inputs(4, 96, F32, None)
    x[0] = 0
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    y = m3.add_rmsnorm(*cu(x, w), eps=1e-6)[0].cpu()
    assert not y[0].any() and torch.isnan(y[1]).all() and torch.isnan(y[2, 7])
    assert torch.isfinite(y[3]).all()
    t = m3.add_rmsnorm(*cu(x, w), fmt="mxfp8")[0]
    v = m3.mx_dequant(t, dtype=F32).cpu()
    assert not v[0].any() and torch.isnan(v[1]).all() and torch.isfinite(v[3]).all()


def test_no_rows():
    w = torch.ones(64, device="cuda")
    x = torch.zeros(0, 64, device="cuda")
    y, r, rstd = m3.add_rmsnorm(x, w, residual=x, want_rstd=True)
    assert y.shape == r.shape == (0, 64) and rstd.shape == (0,)
    dr, dw = m3.add_rmsnorm_bwd(x, x, w, rstd)
    assert dr.shape == (0, 64) and not dw.any()


def test_captured_backward_beside_a_second_graph():
    """Forward and backward captured into two graphs with a workspace each, replayed on two
    streams at once on new inputs."""
    x, r, w = cu(*inputs(500, 320, BF16, F32))
    dy = torch.randn(500, 320, device="cuda").to(BF16)
    def run():
        y, out, rstd = m3.add_rmsnorm(x, w, residual=r, want_rstd=True)
        return (y, *m3.add_rmsnorm_bwd(dy, out, w, rstd, dres=out))
    run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = run()
        graphs.append((g, outs))
    x.mul_(2)
    dy.neg_()
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for st, (g, _) in zip(streams, graphs):
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    for _, outs in graphs:
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
