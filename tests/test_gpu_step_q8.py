"""The 8-bit state and the decode step on it, against the fp64 oracle.

quant_state is a fixed sequence of correctly rounded fp32 operations, so its bytes equal
the same sequence in numpy.  The step: with the same held state, a new value h carries
about 8 2^-24 of the magnitude m of its three terms (products, sums, exp and sincos to an
ulp or two each) plus the angle's fp32 error (4 2^-23 absolute: the sum and the reduction
near pi) on the two rotated ones: 24 2^-24 m in all, rounded up to EH = 2^-19.  y sums N such values: (N +
40) 2^-24 of sum |Cbar| m, and half a step in bf16.  The held new value is within half a
step of its code, 2^-4 |h| or 2^-10 s, of h."""
import numpy as np
import pytest
import torch

import selective_state_space_m3ssd_b200 as m3
from oracle import lowbit as ol
from selective_state_space_m3ssd_b200.synth import WORKLOADS, make_inputs
from tests.gpu_util import angle_err, np64

pytestmark = pytest.mark.gpu
EH = 2.0 ** -19


def state(b, H, N, P, seed):
    g = torch.Generator().manual_seed(seed)
    return 0.3 * torch.randn(b, H, N, P, generator=g) * \
        torch.exp(torch.randn(b, H, N, 1, generator=g))


def make(b, H, G, N, P, dtype, beta=True, theta=True, D=True, seed=3):
    w = WORKLOADS["tiny"].with_(batch=b, nheads=H, ngroups=G, headdim=P, dstate=N, seqlen=1,
                                dtype=dtype, has_beta=beta, has_theta=theta, seed=seed)
    inp = {k: None if v is None else v for k, v in make_inputs(w).items()}
    step = {k: None if inp[k] is None else inp[k][:, 0].contiguous()
            for k in ("X", "logdecay", "beta", "gamma", "B", "C", "theta")}
    step["D"] = inp["D"] if D else None
    g = torch.Generator().manual_seed(seed + 1)
    codes, scale = ol.state_encode(state(b, H, N, P, seed).double().numpy())
    cache = {"angle": torch.rand(b, H, N // 2, generator=g) * 6.28 - 3.14,
             "ssm": torch.from_numpy(codes), "scale": torch.from_numpy(scale).float(),
             "x_prev": torch.randn(b, H, P, generator=g),
             "b_prev": torch.randn(b, G, N, generator=g) / N ** 0.5}
    return step, cache


ORDER = ("X", "logdecay", "beta", "gamma", "B", "C", "theta", "D")


def to_cuda(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def pair_norm(v):
    """Per component, the magnitude a rotation can give it."""
    n = np.sqrt(v[..., 0::2] ** 2 + v[..., 1::2] ** 2)
    return np.repeat(n, 2, -1)


def check(step, cache, y, out, bf16):
    args = [None if step[k] is None else np64(step[k]) for k in ORDER]
    host = {k: v.cpu().numpy() for k, v in cache.items()}
    ref_y, ref = ol.step_q8(host, *args)
    b, H, P = args[0].shape
    rep = H // args[4].shape[1]
    heads = lambda v: np.repeat(pair_norm(v), rep, 1)  # noqa: E731
    Bm, Cm, Bp = heads(args[4]), heads(args[5]), heads(np64(cache["b_prev"]))
    mag = np.exp(args[1])[..., None, None] * np.abs(ol.state_decode(host["ssm"], np64(cache["scale"])))
    mag += np.abs(args[3])[..., None, None] * Bm[..., None] * np.abs(args[0])[:, :, None]
    if args[2] is not None:
        mag += np.abs(args[2])[..., None, None] * Bp[..., None] * np.abs(np64(cache["x_prev"]))[:, :, None]
    N = mag.shape[2]
    my = (Cm[..., None] * mag).sum(2)
    if args[7] is not None:
        my += np.abs(args[7])[:, None] * np.abs(args[0])
    err = np.abs(np64(y) - ref_y)
    assert np.all(err <= (N + 40) * 2.0 ** -24 * my + (2.0 ** -8 * np.abs(ref_y) if bf16 else 0))
    # the new state
    s = np64(out["scale"])
    amax, eh = np.abs(ref["ssm"]).max(-1), EH * mag.max(-1)
    assert np.all(np.abs(s - amax / 448) <= eh / 448 + 2.0 ** -22 * s)
    got = ol.state_decode(out["ssm"].cpu().numpy(), s)
    h = np.abs(ref["ssm"])
    half = np.maximum(2.0 ** -4 * h, 2.0 ** -10 * s[..., None]) * (1 + 2.0 ** -18)
    assert np.all(np.abs(got - ref["ssm"]) <= half + 1.1 * EH * mag)
    # the small parts
    assert angle_err(np64(out["angle"]), ref["angle"]) <= 2.0 ** -20
    np.testing.assert_array_equal(np64(out["x_prev"]), ref["x_prev"])
    np.testing.assert_array_equal(np64(out["b_prev"]), ref["b_prev"])


CASES = [(1, 1, 1, 128, 64), (3, 24, 1, 128, 64), (2, 4, 2, 128, 64), (2, 4, 4, 128, 64),
         (7, 48, 1, 128, 64), (40, 32, 2, 128, 64), (1, 2, 1, 2, 1), (2, 4, 2, 10, 12),
         (3, 2, 1, 6, 3), (1, 3, 3, 256, 64), (2, 2, 1, 64, 256), (1, 2, 1, 128, 63), (2, 6, 1, 128, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("b,H,G,N,P", CASES)
def test_step(b, H, G, N, P, dtype):
    step, cache = make(b, H, G, N, P, dtype)
    sd, cd = to_cuda(step), to_cuda(cache)
    out = {k: torch.full_like(v, 77) for k, v in cd.items()}
    y = m3.step_q8(cd, *[sd[k] for k in ORDER], cache_out=out)
    check(step, cache, y, out, dtype == "bf16")
    for k in cd:  # the old cache stays
        assert torch.equal(cd[k].cpu(), cache[k]), k
    y2 = m3.step_q8(cd, *[sd[k] for k in ORDER])  # in place: the same bits
    assert torch.equal(y2, y)
    for k in cd:
        assert torch.equal(cd[k], out[k]), k


# rows that start inside an access, of one column to the most; states in and out that lie alike
# in an access and otherwise; the cache written over; whole rows of other widths
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,P", [(2, 1), (64, 7), (34, 17), (128, 75), (130, 121), (128, 125), (64, 249),
                                 (62, 250), (64, 255), (64, 64), (256, 32), (100, 72), (64, 256)])
@pytest.mark.parametrize("shift_in,shift_out", [(0, 0), (3, 3), (3, 6)])
def test_rows_inside_an_access(N, P, dtype, shift_in, shift_out):
    step, cache = make(3, 4, 2, N, P, dtype)
    sd, cd = to_cuda(step), to_cuda(cache)
    n = cd["ssm"].numel()
    out = {k: torch.full_like(v, 77) for k, v in cd.items()}
    bi = torch.full((n + 16,), 0x7F, dtype=torch.uint8, device="cuda")  # NaN codes around the state
    bo = torch.full((n + 16,), 0x55, dtype=torch.uint8, device="cuda")
    bi[shift_in:shift_in + n] = cd["ssm"].reshape(-1)
    cd["ssm"] = bi[shift_in:shift_in + n].view(cd["ssm"].shape)
    out["ssm"] = bo[shift_out:shift_out + n].view(out["ssm"].shape)
    y = m3.step_q8(cd, *[sd[k] for k in ORDER], cache_out=out)
    check(step, cache, y, out, dtype == "bf16")
    assert torch.all(bo[:shift_out] == 0x55) and torch.all(bo[shift_out + n:] == 0x55)
    if shift_in == shift_out:  # in place: the same bits
        y2 = m3.step_q8(cd, *[sd[k] for k in ORDER])
        assert torch.equal(y2, y)
        for k in out:
            assert torch.equal(cd[k], out[k]), k
        assert torch.all(bi[:shift_in] == 0x7F) and torch.all(bi[shift_in + n:] == 0x7F)


@pytest.mark.parametrize("b,H,N,P", [(3, 4, 128, 64), (30, 32, 128, 64), (2, 3, 10, 12)])
@pytest.mark.parametrize("beta,theta,D", [(False, True, True), (True, False, True),
                                          (True, True, False), (False, False, False)])
def test_absent_inputs(b, H, N, P, beta, theta, D):
    step, cache = make(b, H, 1, N, P, "f32", beta, theta, D)
    sd, cd = to_cuda(step), to_cuda(cache)
    out = {k: torch.empty_like(v) for k, v in cd.items()}
    y = m3.step_q8(cd, *[sd[k] for k in ORDER], cache_out=out)
    check(step, cache, y, out, False)


@pytest.mark.parametrize("P,N", [(64, 128), (1, 2), (3, 6), (63, 128), (200, 64), (256, 64), (8, 4)])
def test_state_round_trip(P, N):
    h = state(3, 5, N, P, 11)
    h[0, 1] = 0
    h[1, 2, 1] *= 1e-35  # below 2^-100: held as zeros
    h[2, 0, 0, 0] = float("inf")
    h[2, 1, 1, P - 1] = float("nan")
    codes, scale = m3.quant_state(h.cuda())
    back = m3.dequant_state(codes, scale).cpu()
    v = h.numpy()
    with np.errstate(all="ignore"):
        amax = np.abs(v).max(-1)  # NaN where the row holds one
        s = np.where(np.isfinite(amax), np.where(amax >= 2.0 ** -100, amax * np.float32(1 / 448), 0),
                     np.nan).astype(np.float32)
        inv = np.where(s > 0, np.float32(1) / s, np.float32(0)).astype(np.float32)
    np.testing.assert_array_equal(scale.cpu().numpy(), s)
    ok = np.isfinite(s)
    q = torch.from_numpy(v[ok] * inv[ok][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    np.testing.assert_array_equal(codes.cpu().numpy()[ok], q.numpy())
    want = q.view(torch.float8_e4m3fn).float().numpy() * s[ok][..., None]
    np.testing.assert_array_equal(back.numpy()[ok], want)
    assert np.isnan(back.numpy()[~ok]).all()


# every place a row can start at inside an access, in tensors that are aligned and not
@pytest.mark.parametrize("P,N", [(1, 34), (7, 64), (17, 64), (75, 128), (121, 64), (130, 64),
                                 (249, 62), (250, 64), (255, 64)])
def test_odd_states(P, N):
    test_state_round_trip(P, N)
    h = state(3, 5, N, P, 12)
    want_codes, want_scale = m3.quant_state(h.cuda())
    want = m3.dequant_state(want_codes, want_scale)
    n = h.numel()
    for oh, oc in ((0, 0), (1, 0), (0, 3)):
        hb = torch.full((n + 16,), float("nan"), device="cuda")
        cb = torch.full((n + 16,), 0x55, dtype=torch.uint8, device="cuda")
        hb[oh:oh + n] = h.reshape(-1).cuda()
        hv, cv = hb[oh:oh + n].view(h.shape), cb[oc:oc + n].view(h.shape)
        codes, scale = m3.quant_state(hv, codes=cv)
        assert torch.equal(codes, want_codes) and torch.equal(scale, want_scale)
        assert torch.all(cb[:oc] == 0x55) and torch.all(cb[oc + n:] == 0x55)
        hb.fill_(7)
        assert torch.equal(m3.dequant_state(cv, scale, ssm=hv), want)
        assert torch.all(hb[:oh] == 7) and torch.all(hb[oh + n:] == 7)


def test_nonfinite_state_rows():
    """A NaN or infinite input poisons the rows it reaches, reported by the check."""
    step, cache = make(2, 3, 1, 128, 64, "f32")
    sd, cd = to_cuda(step), to_cuda(cache)
    m3.nonfinite_outputs()
    m3.step_q8(cd, *[sd[k] for k in ORDER], check_finite=True)
    assert not m3.nonfinite_outputs()
    sd["X"][1, 2, 5] = float("inf")
    y = m3.step_q8(cd, *[sd[k] for k in ORDER], check_finite=True)
    assert m3.nonfinite_outputs()
    h = m3.dequant_state(cd["ssm"], cd["scale"])
    assert torch.isnan(h[1, 2]).any(-1).all() and torch.isfinite(h[0]).all() and \
        torch.isfinite(h[1, :2]).all() and torch.isfinite(y[0]).all()


def test_unaligned_state_takes_the_general_kernel():
    step, cache = make(2, 3, 1, 128, 64, "f32")
    sd, cd = to_cuda(step), to_cuda(cache)
    buf = torch.empty(cd["ssm"].numel() + 1, dtype=torch.uint8, device="cuda")
    cd["ssm"] = buf[1:].view(cd["ssm"].shape).copy_(cd["ssm"])
    out = {k: torch.empty_like(v) for k, v in cd.items()}
    check(step, cache, m3.step_q8(cd, *[sd[k] for k in ORDER], cache_out=out), out, False)


@pytest.mark.parametrize("b,H", [(2, 4), (40, 24)])
def test_graph_replays_the_eager_steps(b, H):
    step, cache = make(b, H, 1, 128, 64, "bf16")
    sd = to_cuda(step)
    eager, cd = to_cuda(cache), to_cuda(cache)
    ys = [m3.step_q8(eager, *[sd[k] for k in ORDER]) for _ in range(3)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = m3.step_q8(cd, *[sd[k] for k in ORDER])
    for t in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ys[t])
    for k in cd:
        assert torch.equal(cd[k], eager[k]), k


def test_prefill_then_decode_in_8_bits():
    """A prompt through the forward, its state quantised, then steps: the outputs stay within
    the noise that rounding the state to 2^-4 (uniform in a step: 2^-4 / sqrt(3) rms at most)
    puts on them.  Each token's rounding error enters h once and fades with it, and the sum
    over the past of its squared decays is at most the number of steps, so the error of y is
    below sqrt(steps) 2^-4 / sqrt(3) of the rms that the state's part of y has."""
    w = WORKLOADS["siso"].with_(batch=2, nheads=4, seqlen=140, seed=12)
    inp = make_inputs(w)
    d = to_cuda(inp)
    cut = 128
    names = ("X", "logdecay", "beta", "gamma", "B", "C", "theta")
    full, _, _ = m3.fwd(*[d[k] for k in names], d["D"], d["h0"])
    _, hT, c = m3.fwd(*[d[k][:, :cut].contiguous() for k in names], d["D"], d["h0"], want_cache=True)
    cache = m3.quant_cache({**c, "ssm": hT})
    assert torch.equal(m3.dequant_cache(cache)["b_prev"], c["b_prev"])
    got = torch.stack([m3.step_q8(cache, *[d[k][:, t].contiguous() for k in names], d["D"])
                       for t in range(cut, 140)], 1)
    state_part = (full - d["D"][:, None] * d["X"])[:, cut:].float()
    err = (got - full[:, cut:]).float()
    rms = lambda v: v.square().mean().sqrt().item()  # noqa: E731
    steps = 140 - cut
    assert rms(err) <= steps ** 0.5 * 2.0 ** -4 / 3 ** 0.5 * rms(state_part) + 2.0 ** -8 * rms(full.float())


def test_empty_batch():
    c = m3.new_cache_q8(0, 2, 64, 128, 1, "cuda")
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    y = m3.step_q8(c, z(0, 2, 64), z(0, 2), None, z(0, 2), z(0, 1, 128), z(0, 1, 128))
    assert y.shape == (0, 2, 64)
    assert m3.quant_state(z(0, 2, 128, 64))[0].shape == (0, 2, 128, 64)


def test_two_steps_at_once():
    """Two batches on two streams at the same time, each as it is alone (a walk and a small
    launch share nothing)."""
    made = [make(40, 24, 1, 128, 64, "f32", seed=21), make(3, 4, 2, 128, 64, "f32", seed=22)]
    dev = [(to_cuda(s), to_cuda(c)) for s, c in made]
    alone = []
    for s, c in dev:
        out = {k: torch.empty_like(v) for k, v in c.items()}
        alone.append((m3.step_q8(c, *[s[k] for k in ORDER], cache_out=out), out))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dev]
    both = []
    for st, (s, c) in zip(streams, dev):
        with torch.cuda.stream(st):
            out = {k: torch.empty_like(v) for k, v in c.items()}
            both.append([(m3.step_q8(c, *[s[k] for k in ORDER], cache_out=out), out)
                         for _ in range(5)])
    torch.cuda.synchronize()
    for (y, out), runs in zip(alone, both):
        for y2, out2 in runs:
            assert torch.equal(y, y2) and all(torch.equal(out[k], out2[k]) for k in out)


def test_large_batch_of_states():
    """More (b, h) than the walkers take in a few rounds; sampled against the oracle."""
    b, H = 300, 32
    step, cache = make(b, H, 2, 128, 64, "f32", seed=31)
    sd, cd = to_cuda(step), to_cuda(cache)
    y = m3.step_q8(cd, *[sd[k] for k in ORDER])
    rows = [0, 1, 149, 298, 299]
    cut = lambda v, d: None if v is None else (v if d == "D" else v[rows])  # noqa: E731
    check({k: cut(v, k) for k, v in step.items()}, {k: v[rows] for k, v in cache.items()}, y[rows],
          {k: v[rows] for k, v in cd.items()}, False)
