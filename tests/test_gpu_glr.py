"""The gated linear recurrence against the fp64 oracle.

Tolerances.  e = 2^-24, one rounding of fp32.  With w = |r| + |bias_r| and the same of i:
exp(-(r + bias)) is off by (3 w + 8) e of its value (the exponent's rounding times ln 2, twice
over, and the hardware exponential's 2^-22), so the gates by eta = (3 w + 16) e (reciprocal and
products), log a by tau = eta + 16 e (softplus included), a by |log a| tau + 6 e, and
sqrt(1 - a^2) by tau / 2 + 12 e, since |d log(1 - a^2)| <= 2 |d log a| / |log a| |log a| a^2 /
(1 - a^2) <= tau.  So u = s iota x is off by (eta_r + eta_i + 40 e) |u|, and the state by what the
recurrence makes of that: err_t = a err_{t-1} + a M_{t-1} (|log a| tau + 8 e) + ... + 2 e M_t, the
8 covering one product more a token that a scan in pieces does.  M_t = a M_{t-1} + |u_t| stands in
for |h_t|: a scan in pieces adds A h and B of whole runs of tokens, whose roundings go by the size
of those, and they may cancel (in the backward, |dy_t| + a_{t+1} M_{t+1} for |g_t|; at one token
A h + B is a (back + dy) as a back + a dy).  Every bound is doubled.
Where 1 - a^2 is below 1e-37, the kernels' root of it is off by up to sqrt(1e-37) = 3.2e-19 and
(log a) / s, about s / 2 there, by no more: S0 = 4e-19 of iota x (or g iota x) is allowed for.
An a that is no normal number counts as zero: A0 = 2^-126 of |h_{t-1}| (or g, g |log a| |h_{t-1}|).
bf16 outputs add half a step, 2^-8 of the value's power of two at most.
"""
import numpy as np
import pytest
import torch

import selective_state_space_m3ssd_b200 as m3
from oracle import layer as ly
from tests.gpu_util import np64

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
S0 = 4e-19
A0 = 2.0 ** -126
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def make(b, L, D, dtype, seed=0, h0=True, bias=True, reset=None, lengths=None):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(x=rn(b, L, D).to(dtype), r=(1.5 * rn(b, L, D)).to(dtype), i=(1.5 * rn(b, L, D)).to(dtype),
             rate=torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(D, generator=g)))),
             bias_r=rn(D) if bias else None, bias_i=rn(D) if bias else None,
             h0=rn(b, D) if h0 else None)
    if reset is not None:
        d["reset"] = torch.rand(b, L, generator=g) < reset
    if lengths is not None:
        d["lengths"] = torch.tensor(lengths, dtype=torch.int32)
    d["dy"], d["dhT"] = rn(b, L, D).to(dtype), rn(b, D)
    return d


def gpu(d):
    return {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in d.items()}


def host(d):
    return {k: (None if v is None else v.numpy() if v.dtype in (torch.bool, torch.int32) else np64(v))
            for k, v in d.items()}


def bounds(h):
    """(relative error of u, of a, tau) of every token, before doubling."""
    w = lambda g, bias: np.abs(g) + (0 if bias is None else np.abs(bias))  # noqa: E731
    er, ei = ((3 * w(h[k], h[n]) + 16) * E for k, n in (("r", "bias_r"), ("i", "bias_i")))
    _, _, la, _, _ = ly.glr_gates(h["r"], h["i"], h["rate"], h["bias_r"], h["bias_i"])
    tau = er + 16 * E
    return er + ei + 40 * E, np.abs(la) * tau + 8 * E, tau, er, ei


FWD = ("x", "r", "i", "rate", "bias_r", "bias_i", "h0", "reset", "lengths")


def fwd_tolerance(h, y, hT):
    """The state's error after every token, and after the last."""
    _, iota, _, a, s = ly.glr_gates(h["r"], h["i"], h["rate"], h["bias_r"], h["bias_i"], 8.0,
                                    h.get("reset"))
    ru, ra, *_ = bounds(h)
    err, out = np.zeros_like(hT), np.zeros_like(y)
    M = np.zeros_like(hT) if h["h0"] is None else np.abs(h["h0"])
    n = ly._lens(h.get("lengths"), *y.shape[:2])
    for t in range(y.shape[1]):
        u = np.abs(s * iota * h["x"])[:, t]
        new = a[:, t] * err + M * (a[:, t] * ra[:, t] + A0) + u * ru[:, t] + \
            np.abs(iota * h["x"])[:, t] * S0 + 2 * E * (u + 2 * a[:, t] * M)
        live = (t < n)[:, None]
        err, M = np.where(live, new, err), np.where(live, a[:, t] * M + u, M)
        out[:, t] = np.where(live, err, 0)
    return 2 * out, 2 * err


def check(got, ref, tol, dtype, name):
    err = np.abs(np64(got) - ref)
    bad = ~(err <= tol * (1 + 1e-3) + HALF[dtype] * (np.abs(ref) + tol) + 1e-37)
    assert not bad.any(), (name, float(np.max(err)), np.argwhere(bad)[:4])


def call(f, d, *a, **kw):
    return f(d["x"], d["r"], d["i"], d["rate"], *a, bias_r=d["bias_r"], bias_i=d["bias_i"], h0=d["h0"],
             reset=d.get("reset"), lengths=d.get("lengths"), **kw)


def run_fwd(d):
    h = host(d)
    y, hT = ly.glr_fwd(**{k: h[k] for k in FWD if k in h})
    ty, tT = fwd_tolerance(h, y, hT)
    gy, gT = call(m3.glr_fwd, gpu(d))
    check(gy, y, ty, d["x"].dtype, "y")
    check(gT, hT, tT, torch.float32, "hT")
    return gy, gT


def run_bwd(d, grad_dtype=torch.float32, **kw):
    """The gradients from the forward's own y, against the oracle's from the same y."""
    c = gpu(d)
    c["y"] = call(m3.glr_fwd, c)[0]
    got = call(m3.glr_bwd, c, c["y"], c["dy"], dhT=c["dhT"], grad_dtype=grad_dtype, **kw)
    check_bwd(d, np64(c["y"]), got, grad_dtype)
    return got


def check_bwd(d, y, got, grad_dtype):
    h = host(d)
    o = ly.glr_bwd(**{k: h[k] for k in FWD if k in h}, y=y, dy=h["dy"], dhT=h["dhT"])
    rho, iota, la, a, s = ly.glr_gates(h["r"], h["i"], h["rate"], h["bias_r"], h["bias_i"], 8.0,
                                       h.get("reset"))
    b, L, D = y.shape
    ru, ra, tau, er, ei = bounds(h)
    n = ly._lens(h.get("lengths"), b, L)
    eg, nxt, M = np.zeros((b, L, D)), np.zeros((b, D)), np.abs(h["dhT"])
    for t in range(L - 1, -1, -1):
        live = (t < n)[:, None]
        Mg = np.where(live, M + np.abs(h["dy"][:, t]), 0)
        eg[:, t] = np.where(live, nxt + 2 * E * Mg, 0)
        nxt = np.where(live, a[:, t] * eg[:, t] + Mg * (a[:, t] * ra[:, t] + A0), nxt)
        M = np.where(live, a[:, t] * Mg, M)
    first = np.zeros((b, 1, D)) if h["h0"] is None else h["h0"][:, None]
    prev = np.abs(np.concatenate((first, y[:, :-1]), 1))
    g, x = np.abs(o["g"]), np.abs(h["x"])
    with np.errstate(divide="ignore", invalid="ignore"):
        terms = a * np.abs(la) * prev + a * a * np.abs(np.where(s > 0, la / s, 0)) * iota * x
    tE = terms * (eg + g * (3 * tau + ra + ei + 40 * E)) + S0 * g * iota * x + \
        A0 * g * np.abs(la) * prev
    if "reset" in h:
        tE = np.where(h["reset"][..., None], 0, tE)
    tdx = s * iota * (eg + g * (ru + 8 * E)) + S0 * g * iota
    tol = {"dx": tdx, "di": x * (1 - iota) * (tdx + s * iota * g * (ei + 16 * E)),
           "dr": (1 - rho) * (tE + np.abs(o["E"]) * (er + 16 * E))}
    # sums in pieces of any order: at most one rounding a term of what is summed
    m = b * L * E
    k = np.where(h["rate"] < -40, 1.0, ly.sigmoid(h["rate"]) / ly.softplus(h["rate"]))
    live = np.arange(L)[None, :, None] < n[:, None, None]
    tol = {k2: np.where(live, v, 0) for k2, v in tol.items()}
    tE = np.where(live, tE, 0)
    tol["drate"] = k * (tE.sum((0, 1)) + (m + 16 * E) * np.abs(o["E"]).sum((0, 1)))
    tol["dbias_r"] = tol["dr"].sum((0, 1)) + m * np.abs(o["dr"]).sum((0, 1))
    tol["dbias_i"] = tol["di"].sum((0, 1)) + m * np.abs(o["di"]).sum((0, 1))
    tol["dh0"] = nxt
    for name in m3.GLR_GRAD_NAMES:
        check(got[name], o[name], 2 * tol[name],
              grad_dtype if name in ("dx", "dr", "di") else torch.float32, name)


# one token, ends around whole tiles, several tiles; widths around whole groups of channels; from
# L = 512 on these few sequences are cut into parts, backward from 256 in bf16 and 128 in fp32
SHAPES = [(1, 1, 1), (2, 1, 64), (1, 2, 2), (3, 7, 63), (2, 16, 65), (1, 63, 130), (2, 64, 128), (1, 65, 8),
          (2, 129, 72), (1, 300, 200), (5, 33, 4), (1, 1025, 40), (2, 517, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b,L,D", SHAPES)
def test_forward(b, L, D, dtype):
    run_fwd(make(b, L, D, dtype, seed=b + L + D))
    run_fwd(make(b, L, D, dtype, seed=L, h0=False, bias=False))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b,L,D", SHAPES)
def test_backward(b, L, D, dtype):
    run_bwd(make(b, L, D, dtype, seed=b + L + D))
    run_bwd(make(b, L, D, dtype, seed=L, h0=False, bias=False), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rate", [0.02, 0.3, 1.0])
def test_resets(dtype, rate):
    d = make(2, 200, 70, dtype, seed=5, reset=rate)
    run_fwd(d)
    run_bwd(d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("L", [512, 1100, 2311])
def test_parts_of_a_long_sequence(L, dtype):
    # both directions in parts: resets in some parts only, ends inside, between and before the parts
    run_fwd(make(1, L, 70, dtype, seed=L, reset=0.002))
    run_bwd(make(1, L, 70, dtype, seed=L, reset=0.002))
    d = make(4, L, 33, dtype, seed=L + 1, reset=0.01, lengths=[0, L, 1, L // 2 + 3])
    run_fwd(d)
    run_bwd(d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_lengths_of_padded_batches(dtype):
    d = make(7, 150, 66, dtype, seed=6, lengths=[0, 1, 64, 65, 150, 149, 8])
    for k in ("x", "r", "i", "dy"):  # what lies behind an end is not looked at
        for j, n in enumerate((0, 1, 64, 65, 150, 149, 8)):
            d[k][j, n:] = float("nan")
    clean = {k: (torch.nan_to_num(v) if torch.is_tensor(v) and v.dtype.is_floating_point else v)
             for k, v in d.items()}
    c = gpu(d)
    y, hT = call(m3.glr_fwd, c)
    ry, rT = run_fwd(clean)
    assert torch.equal(y, ry) and torch.equal(hT, rT)
    assert torch.equal(hT[0], c["h0"][0])
    got = call(m3.glr_bwd, c, y, c["dy"], dhT=c["dhT"])
    check_bwd(clean, np64(y), got, torch.float32)
    for k in ("dx", "dr", "di"):
        assert not got[k][0].any() and not got[k][6, 8:].any()
    # and with resets, lengths past the end or below zero
    d = make(4, 90, 64, dtype, seed=8, reset=0.1, lengths=[-5, 90, 1000, 31])
    run_fwd(d)
    run_bwd(d)


def test_a_reset_cuts_nan_and_infinity():
    """What came before a reset, a state that is not finite or such a token, ends there; in the
    backward a gradient that is not finite does not pass it."""
    for bad in (float("nan"), float("inf")):
        d = make(2, 400, 64, torch.float32, seed=9, reset=0.0)
        d["reset"][:, [5, 64, 130]] = True
        d["h0"][0, 3], d["x"][1, 60, 4], d["x"][0, 129, 7] = bad, bad, bad
        y, hT = call(m3.glr_fwd, gpu(d))
        ok = torch.isfinite(y).cpu()
        assert ok[0, 5:, 3].all() and not ok[0, :5, 3].any()
        assert ok[1, 64:, 4].all() and not ok[1, 60:64, 4].any()
        assert ok[0, 130:, 7].all() and not ok[0, 129, 7]
        d = make(2, 400, 64, torch.float32, seed=9, reset=0.0)
        d["reset"][:, [5, 64, 130]] = True
        d["dhT"][0, 3], d["dy"][1, 70, 4] = bad, bad
        c = gpu(d)
        got = call(m3.glr_bwd, c, call(m3.glr_fwd, c)[0], c["dy"], dhT=c["dhT"])
        ok = torch.isfinite(got["dx"]).cpu()
        assert ok[0, :130, 3].all() and not ok[0, 130:, 3].any()
        assert ok[1, :64, 4].all() and not ok[1, 64:71, 4].any() and ok[1, 71:, 4].all()


def test_without_a_reset_nan_stays():
    d = make(1, 100, 64, torch.float32, seed=10)
    d["x"][0, 40, 5] = float("nan")
    d["r"][0, 50, 6] = float("nan")
    d["i"][0, 60, 7] = float("nan")
    y = call(m3.glr_fwd, gpu(d))[0].cpu()
    for t, ch in ((40, 5), (50, 6), (60, 7)):
        assert torch.isfinite(y[0, :t, ch]).all() and torch.isnan(y[0, t:, ch]).all()


def test_gates_and_rates_at_their_ends():
    """Saturated gates and rates from none to a state that is gone in a token: a = 1 keeps the
    state bit for bit, a = 0 takes the token alone, and the gradients stay finite."""
    D = 64
    d = make(1, 140, D, torch.float32, seed=11, bias=False)
    d["rate"] = torch.linspace(-120, 60, D)
    d["r"][0, :, ::3] = 90.0
    d["r"][0, :, 1::3] = -40.0
    d["i"][0, ::2] = -40.0
    d["i"][0, 1::4] = 200.0
    run_fwd(d)
    got = run_bwd(d)
    assert all(torch.isfinite(v).all() for v in got.values())
    # further down a gate counts as 2^-63, so s as sqrt(2 k 2^-63) <= 1.1e-8 where it is less
    d["r"][0, :, 1::3] = -300.0
    d["i"][0, ::2] = -float("inf")
    d["i"][0, 1::4] = float("inf")
    y, hT = call(m3.glr_fwd, gpu(d))
    h = host(d)
    with np.errstate(invalid="ignore"):
        ref, refT = ly.glr_fwd(**{k: h[k] for k in FWD if k in h})
    assert np.abs(np64(y) - ref).max() <= 140 * 1.1e-8 * np.abs(h["x"]).max() + \
        140 * 20 * E * np.abs(ref).max()
    got = call(m3.glr_bwd, gpu(d), y, d["dy"].cuda(), dhT=d["dhT"].cuda())
    assert all(torch.isfinite(v).all() for v in got.values())
    d["rate"][:] = -200.0
    y, _ = call(m3.glr_fwd, gpu(d))
    assert torch.equal(y.cpu(), d["h0"][:, None].expand(1, 140, D))


def test_a_projections_rows_are_read_in_place():
    """x, r, i as column ranges of one projection, and gradients written into one."""
    b, L, D = 2, 77, 72
    for dtype in (torch.bfloat16, torch.float32):
        for off in (0, 1, 8):  # ranges that start off the 16-byte grid
            d = make(b, L, D, dtype, seed=12)
            c = gpu(d)
            zx = torch.randn(b, L, 4 * D + off + 8, device="cuda").to(dtype)
            for j, k in enumerate(("x", "r", "i")):
                zx[..., off + j * D:off + (j + 1) * D] = c[k]
            v = dict(c, **{k: zx[..., off + j * D:off + (j + 1) * D] for j, k in enumerate(("x", "r", "i"))})
            y, hT = call(m3.glr_fwd, v)
            ry, rT = run_fwd(d)
            assert torch.equal(y, ry) and torch.equal(hT, rT)
            buf = torch.full((b, L, 4 * D + off), 7.0, device="cuda", dtype=dtype)
            g = {k: buf[..., off + j * D:off + (j + 1) * D] for j, k in enumerate(("dx", "dr", "di"))}
            got = call(m3.glr_bwd, v, y, c["dy"], dhT=c["dhT"], grad_dtype=dtype, grads=g)
            check_bwd(d, np64(y), got, dtype)
            assert (buf[..., :off] == 7).all() and (buf[..., off + 3 * D:] == 7).all()


@pytest.mark.parametrize("b,L,cut", [(3, 210, 100), (2, 3000, 1700)])
def test_state_in_place_and_continuation(b, L, cut):
    """hT may be h0's tensor, dh0 dhT's (also where few sequences are cut into parts); two pieces
    equal the whole."""
    d = make(b, L, 96, torch.float32, seed=13)
    c = gpu(d)
    y, hT = call(m3.glr_fwd, c)
    h = c["h0"].clone()
    half = lambda lo, hi: {k: (v[:, lo:hi].contiguous() if k in ("x", "r", "i") else v)  # noqa: E731
                           for k, v in dict(c, h0=h).items()}
    y1, h1 = call(m3.glr_fwd, half(0, cut), hT=h)
    assert h1 is h
    y2, _ = call(m3.glr_fwd, half(cut, L), hT=h)
    hh = host(d)
    ref, refT = ly.glr_fwd(**{k: hh[k] for k in FWD if k in hh})
    ty, tT = fwd_tolerance(hh, ref, refT)
    check(torch.cat((y1, y2), 1), ref, ty, torch.float32, "y")
    check(h, refT, tT, torch.float32, "h")
    g1 = call(m3.glr_bwd, c, y, c["dy"], dhT=c["dhT"])
    dh = c["dhT"].clone()
    g2 = call(m3.glr_bwd, c, y, c["dy"], dhT=dh, grads={"dh0": dh})
    assert g2["dh0"] is dh and torch.equal(dh, g1["dh0"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b,D", [(1, 1), (3, 64), (256, 200), (1, 4096), (5, 33)])
def test_step(b, D, dtype):
    d = make(b, 1, D, dtype, seed=b + D)
    h = host(d)
    y, hT = ly.glr_fwd(**{k: h[k] for k in FWD if k in h})
    ty, tT = fwd_tolerance(h, y, hT)
    c = gpu(d)
    one = {k: c[k][:, 0] for k in ("x", "r", "i")}
    keep = c["h0"].clone()
    out = torch.empty_like(keep)
    gy, gh = m3.glr_step(keep, one["x"], one["r"], one["i"], c["rate"], bias_r=c["bias_r"],
                         bias_i=c["bias_i"], h_out=out)
    assert gh is out and torch.equal(keep, c["h0"])
    check(gy, y[:, 0], ty[:, 0], dtype, "y")
    check(gh, hT, tT, torch.float32, "h")
    gy2, gh2 = m3.glr_step(keep, one["x"], one["r"], one["i"], c["rate"], bias_r=c["bias_r"],
                           bias_i=c["bias_i"])
    assert gh2 is keep and torch.equal(gh2, gh) and torch.equal(gy2, gy)
    # rows of a projection, off the grid
    zx = torch.randn(b, 3 * D + 1, device="cuda").to(dtype)
    v = [zx[:, 1 + j * D:1 + (j + 1) * D] for j in range(3)]
    for t, k in zip(v, ("x", "r", "i")):
        t.copy_(one[k])
    gy3, gh3 = m3.glr_step(c["h0"], *v, c["rate"], bias_r=c["bias_r"], bias_i=c["bias_i"])
    assert torch.equal(gy3, gy) and torch.equal(gh3, gh)


def test_forward_then_steps():
    """Prefill hands its state to single tokens: the same as one forward."""
    d = make(2, 60, 136, torch.float32, seed=15)
    h = host(d)
    y, hT = ly.glr_fwd(**{k: h[k] for k in FWD if k in h})
    ty, tT = fwd_tolerance(h, y, hT)
    c = gpu(d)
    _, st = call(m3.glr_fwd, {k: (v[:, :50].contiguous() if k in ("x", "r", "i") else v)
                              for k, v in c.items()})
    for t in range(50, 60):
        yt, st = m3.glr_step(st, c["x"][:, t], c["r"][:, t], c["i"][:, t], c["rate"],
                             bias_r=c["bias_r"], bias_i=c["bias_i"])
        check(yt, y[:, t], ty[:, t], torch.float32, t)
    check(st, hT, tT, torch.float32, "h")


def test_gradients_against_differences():
    """Central differences of the library's own fp32 forward, along random directions.  The
    loss sums some 5000 terms, each within about 1e-6 of itself (the tolerances above), so it is
    within 1e-4; over a step of 2 x 1e-2 that leaves 5e-3, and the third derivatives, about the
    gradient's own size times 1e-4, less."""
    d = make(2, 40, 66, torch.float32, seed=16)
    c = gpu(d)
    y, _ = call(m3.glr_fwd, c)
    got = call(m3.glr_bwd, c, y, c["dy"], dhT=c["dhT"])

    def loss(e):
        yy, hh = call(m3.glr_fwd, e)
        return float((yy.double() * c["dy"].double()).sum() + (hh.double() * c["dhT"].double()).sum())
    g = torch.Generator().manual_seed(1)
    for k, n in (("x", "dx"), ("r", "dr"), ("i", "di"), ("rate", "drate"), ("bias_r", "dbias_r"),
                 ("bias_i", "dbias_i"), ("h0", "dh0")):
        v = torch.randn(c[k].shape, generator=g).cuda()
        v /= v.norm()
        hi, lo = (loss(dict(c, **{k: c[k] + sgn * 1e-2 * v})) for sgn in (1, -1))
        want = float((got[n].double() * v.double()).sum())
        scale = float(got[n].double().norm())
        assert abs((hi - lo) / 2e-2 - want) <= 5e-3 + 1e-3 * scale, (k, hi - lo, want)


def test_same_bits_again_and_in_a_graph():
    d = make(4, 700, 128, torch.bfloat16, seed=17, reset=0.01)
    c = gpu(d)
    y, hT = call(m3.glr_fwd, c)
    g = call(m3.glr_bwd, c, y, c["dy"], dhT=c["dhT"])
    y2, hT2 = torch.empty_like(y), torch.empty_like(hT)
    out = {k: torch.empty_like(v) for k, v in g.items()}
    ws = torch.empty(m3.glr_bwd_workspace_size(m3.GlrDims(4, 700, 128, 128, 128, 128, m3.BF16, 8.0, 0)),
                     dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call(m3.glr_fwd, c, y=y2, hT=hT2)
            call(m3.glr_bwd, c, y2, c["dy"], dhT=c["dhT"], grads=out, workspace=ws)
    for _ in range(3):
        y2.fill_(9), hT2.fill_(9), ws.fill_(255)
        for v in out.values():
            v.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(hT, hT2)
        assert all(torch.equal(g[k], out[k]) for k in g)


def test_empty_calls():
    for b, L in ((0, 5), (2, 0)):
        x = torch.empty(b, L, 8, device="cuda")
        rate = torch.zeros(8, device="cuda")
        h0 = torch.randn(b, 8, device="cuda")
        y, hT = m3.glr_fwd(x, x, x, rate, h0=h0)
        assert y.shape == (b, L, 8) and torch.equal(hT, h0)
        g = m3.glr_bwd(x, x, x, rate, y, x, dhT=h0)
        assert torch.equal(g["dh0"], h0) and not g["drate"].any() and not g["dbias_i"].any()
    y, h = m3.glr_step(h0[:0], x[:0, 0] if L else torch.empty(0, 8, device="cuda"),
                       torch.empty(0, 8, device="cuda"), torch.empty(0, 8, device="cuda"), rate)
    assert y.shape == (0, 8)


def test_far_rows():
    """Offsets of more than 2^31 elements: a token's rows lie 2^31 / 64 apart."""
    ld, D = (1 << 25) + 64, 64
    buf = torch.empty(80 * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((1, 80, D), (80 * ld, ld, 1))
    d = make(1, 80, D, torch.bfloat16, seed=18)
    x.copy_(d["x"])
    c = dict(gpu(d))
    y, hT = call(m3.glr_fwd, c)
    y2, hT2 = call(m3.glr_fwd, dict(c, x=x))
    assert torch.equal(y, y2) and torch.equal(hT, hT2)
    del buf
