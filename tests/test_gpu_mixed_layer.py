"""The gated recurrence, the heads' norm with rotation and the 4-bit products together, beside the
operators that were there, as a layer with both kinds of mixers is trained and served: residual
addition and norm, in_proj, the scan on queries and keys normed and rotated by position (no theta) next
to the recurrence, out_proj; the gradients back into one projection's gradient; and single
tokens with the projections in 4 bits, captured in a graph.  Each operator is checked from its own
inputs with the bounds of its own tests, so a rounding upstream is not counted twice."""
import numpy as np
import pytest
import torch

import oracle
import selective_state_space_m3ssd_b200 as m3
from oracle import layer as ly
from tests import test_gpu_gemv_w4 as tw
from tests import test_gpu_glr as tg
from tests import test_gpu_rotate as tr
from tests.gpu_util import np64, rel_max_err, rel_max_err_out

pytestmark = pytest.mark.gpu
DM, H, P, N, R = 256, 4, 64, 128, 200
HP = H * P
# in_proj's columns: x | C | B | dt, lam | the recurrence's x, r, i
PARTS = {"x": HP, "C": N, "B": N, "dt": H, "lam": H, "xr": R, "r": R, "i": R}
WIDTH = sum(PARTS.values())
FREQS = 10000.0 ** (-torch.arange(N // 2).float() * 2 / N)


def weights(seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    u = lambda *s: torch.rand(*s, generator=g)  # noqa: E731
    w = {"norm": 0.5 + u(DM), "W_in": r(WIDTH, DM) / DM ** 0.5, "W_out": r(DM, HP + R) / (HP + R) ** 0.5,
         "Cw": (0.5 + u(N)) / N ** 0.5, "Bw": (0.5 + u(N)) / N ** 0.5, "dt_bias": -4 + 2 * u(H),
         "A": 1 + 15 * u(H), "D": r(H),
         "rate": torch.log(torch.expm1(-torch.log(0.9 + 0.099 * u(R)))), "bias_r": r(R), "bias_i": r(R),
         "freqs": FREQS}
    w = {k: v.cuda() for k, v in w.items()}
    w["q_in"], w["q_out"] = m3.w4_quant(w["W_in"], 128), m3.w4_quant(w["W_out"], 64, zeros=True)
    # the same weights as a prompt's products take them
    w["b_in"], w["b_out"] = m3.w4_dequant(w["q_in"]), m3.w4_dequant(w["q_out"])
    return w


def split(zx):
    return dict(zip(PARTS, torch.split(zx, list(PARTS.values()), -1)))


def scan_inputs(s, w):
    """logdecay, beta, gamma of the projection's dt and lam, as a caller forms them."""
    delta = torch.nn.functional.softplus(s["dt"].float() + w["dt_bias"])
    ld, lm = -w["A"] * delta, torch.sigmoid(s["lam"].float())
    return ld, (1 - lm) * delta * ld.exp(), lm * delta


def gates(w):
    return dict(bias_r=w["bias_r"], bias_i=w["bias_i"])


def heads(t):
    return t.unflatten(-1, (1, N))


def host_glr(s, w, h0=None, **kw):
    """The recurrence's inputs as the oracle's checks take them."""
    d = {"x": s["xr"], "r": s["r"], "i": s["i"], "rate": w["rate"], "h0": h0, **gates(w), **kw}
    return {k: None if v is None else v.cpu() for k, v in d.items()}


def test_training_pass():
    w = weights()
    b, L = 2, 150
    g = torch.Generator().manual_seed(7)
    x = torch.randn(b * L, DM, generator=g).bfloat16().cuda()
    res = 3 * torch.randn(b * L, DM, generator=g).cuda()
    pos = torch.arange(L, dtype=torch.int32).expand(b, L).contiguous().cuda()

    y, r, rstd = m3.add_rmsnorm(x, w["norm"], residual=res, want_rstd=True)
    zx = m3.gemm_bf16(y, w["b_in"]).view(b, L, WIDTH)
    s = split(zx)
    C, B = m3.norm_rotate(heads(s["C"]), heads(s["B"]), w["Cw"], w["Bw"], positions=pos, freqs=w["freqs"])
    rot = {"q": s["C"].reshape(b * L, 1, N).cpu(), "k": s["B"].reshape(b * L, 1, N).cpu(), "q_w": w["Cw"].cpu(),
           "k_w": w["Bw"].cpu(), "positions": pos.flatten().cpu(), "freqs": FREQS}
    tr.check_fwd(rot, [t.flatten(0, 1) for t in (C, B)])
    ld, be, ga = scan_inputs(s, w)
    X = s["x"].reshape(b, L, H, P).contiguous()
    Y, hT, _ = m3.fwd(X, ld, be, ga, B, C, None, w["D"])
    scan = dict(X=X, logdecay=ld, beta=be, gamma=ga, B=B, C=C, theta=None, D=w["D"], h0=None)
    scan = {k: None if v is None else v.cpu() for k, v in scan.items()}
    ref = oracle.oracle_fwd(**scan)
    assert rel_max_err_out(np64(Y), ref["Y"], True) <= 2e-2 and rel_max_err(np64(hT), ref["hT"]) <= 2e-2
    yr, _ = m3.glr_fwd(s["xr"], s["r"], s["i"], w["rate"], **gates(w))
    d = host_glr(s, w)
    h = tg.host(d)
    yo, hTo = ly.glr_fwd(**{k: h[k] for k in tg.FWD if k in h})
    tg.check(yr, yo, tg.fwd_tolerance(h, yo, hTo)[0], torch.bfloat16, "yr")
    out = m3.gemm_bf16(torch.cat((Y.flatten(2), yr), -1).view(b * L, HP + R), w["b_out"])
    assert torch.isfinite(out).all()

    # and back, every operator's gradient into its columns of one fp32 gradient of zx
    dout = torch.randn(b * L, DM, generator=g).cuda()
    dcat = (dout @ w["b_out"].float()).bfloat16().view(b, L, HP + R)
    dY, dyr = dcat[..., :HP].reshape(b, L, H, P).contiguous(), dcat[..., HP:].contiguous()
    sg = m3.bwd(X, ld, be, ga, B, C, None, w["D"], dY=dY)
    dzx = torch.full((b, L, WIDTH), float("nan"), device="cuda")
    ds = split(dzx)
    rg = m3.norm_rotate_bwd(heads(s["C"]), heads(s["B"]), w["Cw"], w["Bw"], sg["dC"], sg["dB"], positions=pos,
                            freqs=w["freqs"], grads={"dq": heads(ds["C"]), "dk": heads(ds["B"])})
    gg = m3.glr_bwd(s["xr"], s["r"], s["i"], w["rate"], yr, dyr, **gates(w),
                    grads={"dx": ds["xr"], "dr": ds["r"], "di": ds["i"]})
    tg.check_bwd(host_glr(s, w, dy=dyr, dhT=torch.zeros(b, R)), np64(yr), gg, torch.float32)
    rot.update(dq=sg["dC"].flatten(0, 1).cpu(), dk=sg["dB"].flatten(0, 1).cpu())
    tr.check_bwd(rot, {k: v.reshape(b * L, 1, N) if v.dim() > 1 else v for k, v in rg.items()}, torch.float32)
    ds["x"].copy_(sg["dX"].flatten(2))
    for k in ("dt", "lam"):
        ds[k].zero_()
    assert torch.isfinite(dzx).all()
    dy = (dzx.view(-1, WIDTH).bfloat16().float() @ w["b_in"].float()).bfloat16()
    dr, dw = m3.add_rmsnorm_bwd(dy, r, w["norm"], rstd, dres=dout)
    assert torch.isfinite(dr).all() and torch.isfinite(dw).all()
    ob = oracle.oracle_bwd(**scan, dY=dY.cpu())
    for k in ("dX", "dB", "dC"):
        assert rel_max_err(np64(sg[k]), ob[k]) <= 1e-3, k


def test_prompt_then_tokens():
    w = weights(2)
    b, L, steps = 3, 40, 5
    g = torch.Generator().manual_seed(8)
    xs = torch.randn(b, L + steps, DM, generator=g).bfloat16().cuda()
    rs = 3 * torch.randn(b, L + steps, DM, generator=g).cuda()
    lens = torch.tensor([L, L - 7, 5], dtype=torch.int32)  # a padded batch of prompts
    pos = torch.arange(L, dtype=torch.int32).expand(b, L).contiguous().cuda()

    y, _, _ = m3.add_rmsnorm(xs[:, :L].reshape(-1, DM), w["norm"], residual=rs[:, :L].reshape(-1, DM))
    zx = m3.gemm_bf16(y, w["b_in"]).view(b, L, WIDTH)
    s = split(zx)
    C, B = m3.norm_rotate(heads(s["C"]), heads(s["B"]), w["Cw"], w["Bw"], positions=pos, freqs=w["freqs"])
    ld, be, ga = scan_inputs(s, w)
    cache = m3.new_cache(b, H, P, N, 1, "cuda")
    h = torch.empty(b, R, device="cuda")
    for k in range(b):  # the scan takes no lengths: a sequence at a time
        n = int(lens[k])
        one = [t[k:k + 1, :n].contiguous() for t in (s["x"].reshape(b, L, H, P), ld, be, ga, B, C)]
        _, hT, c = m3.fwd(*one, None, w["D"], want_cache=True)
        for name, v in (("ssm", hT), *((n, c[n]) for n in ("angle", "x_prev", "b_prev"))):
            cache[name][k:k + 1] = v
    m3.glr_fwd(s["xr"], s["r"], s["i"], w["rate"], **gates(w), lengths=lens.cuda(), hT=h)
    hh = tg.host(host_glr(s, w, lengths=lens))
    yo, hTo = ly.glr_fwd(**{k: hh[k] for k in tg.FWD if k in hh})
    tg.check(h, hTo, tg.fwd_tolerance(hh, yo, hTo)[1], torch.float32, "h")

    x_t, r_t, p_t = xs[:, L].clone(), rs[:, L].clone(), lens.cuda()

    def token():
        y, _, _ = m3.add_rmsnorm(x_t, w["norm"], residual=r_t)
        zx = m3.gemv_w4(y, w["q_in"])
        s = split(zx)
        C, B = m3.norm_rotate(heads(s["C"]), heads(s["B"]), w["Cw"], w["Bw"], positions=p_t, freqs=w["freqs"])
        ld, be, ga = scan_inputs(s, w)
        X = s["x"].reshape(b, H, P).contiguous()
        Y = m3.step(cache, X, ld, be, ga, B, C, None, w["D"])
        yr, _ = m3.glr_step(h, s["xr"], s["r"], s["i"], w["rate"], **gates(w))
        cat = torch.cat((Y.flatten(1), yr), -1)
        return dict(y=y, zx=zx, C=C, B=B, X=X, ld=ld, be=be, ga=ga, Y=Y, yr=yr, cat=cat,
                    out=m3.gemv_w4(cat, w["q_out"], out_dtype=torch.float32))
    keep = {k: v.clone() for k, v in {**cache, "h": h}.items()}
    token()  # warms up what a first call sets
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = token()
    for k, v in keep.items():
        (h if k == "h" else cache[k]).copy_(v)
    win, wout = (np64(m3.w4_dequant(w[k], torch.float32)) for k in ("q_in", "q_out"))
    for t in range(steps):
        x_t.copy_(xs[:, L + t])
        r_t.copy_(rs[:, L + t])
        old_h, old = h.clone(), {k: v.clone() for k, v in cache.items()}
        graph.replay()
        torch.cuda.synchronize()
        tw.check(o["zx"], o["y"], win, DM)
        tw.check(o["out"], o["cat"], wout, HP + R)
        s = split(o["zx"])
        tr.check_fwd({"q": heads(s["C"]).cpu(), "k": heads(s["B"]).cpu(), "q_w": w["Cw"].cpu(),
                      "k_w": w["Bw"].cpu(), "positions": p_t.cpu(), "freqs": FREQS}, (o["C"], o["B"]))
        d = host_glr({k: v.unsqueeze(1) for k, v in s.items()}, w, h0=old_h)
        hd = tg.host(d)
        yo, hTo = ly.glr_fwd(**{k: hd[k] for k in tg.FWD if k in hd})
        ty, tT = tg.fwd_tolerance(hd, yo, hTo)
        tg.check(o["yr"], yo[:, 0], ty[:, 0], torch.bfloat16, "yr")
        tg.check(h, hTo, tT, torch.float32, "h")
        c64 = {k: np64(v) for k, v in old.items()}  # the oracle advances it
        ref = oracle.oracle_step(c64, *[np64(o[k]) for k in ("X", "ld", "be", "ga", "B", "C")], None,
                                 np64(w["D"]))
        assert rel_max_err_out(np64(o["Y"]), ref, True) <= 1e-4
        assert rel_max_err(np64(cache["ssm"]), c64["ssm"]) <= 1e-4
        p_t += 1
    assert m3.device_wait_timeouts() == 0
