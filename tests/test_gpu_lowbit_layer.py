"""The low-bit operators together, as a layer is served with them: residual addition and norm
into the 8-bit operand, in_proj with 4-bit weights, the scan (a prompt) or the step on the
8-bit cache (single tokens), the gated output quantised, out_proj with 4-bit weights.  The
small parts between them (the split of the in_proj row, QK-norm, SiLU) are plain torch here.
Every operator's output is checked against fp64 from its own inputs, so a rounding next to
a border upstream is not counted twice; the tolerances are those of the operators' tests."""
import math

import numpy as np
import pytest
import torch

import selective_state_space_m3ssd_b200 as m3
from oracle import lowbit as ol
from tests.gpu_util import np64

pytestmark = pytest.mark.gpu
DM, H, P, N = 256, 8, 64, 128
HP = H * P
WIDTH = 2 * HP + 2 * N + 2 * H + H * (N // 2)


def weights(seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    u = lambda *s: torch.rand(*s, generator=g)  # noqa: E731
    return {"norm": 0.5 + u(DM), "W_in": r(WIDTH, DM) / DM ** 0.5, "W_out": r(DM, HP) / HP ** 0.5,
            "dt_bias": -4 + 2 * u(H), "A": 1 + 15 * u(H), "D": r(H), "Bw": 0.5 + u(N),
            "Cw": 0.5 + u(N)}


def front(x, res, w):
    """norm and in_proj of (tokens, DM): the in_proj rows and the new residual."""
    y, res, _ = m3.add_rmsnorm(x, w["norm"], residual=res, fmt="mxfp8")
    return y, m3.gemm_mx(y, w["q_in"]), res


def split(zx, w):
    """The in_proj rows (..., WIDTH) to the scan's inputs."""
    z, x, B, C, dt, lam, th = torch.split(zx, [HP, HP, N, N, H, H, H * (N // 2)], -1)
    norm = lambda v, g: (v.float() * torch.rsqrt(v.float().square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
                         * g).to(torch.bfloat16)
    delta = torch.nn.functional.softplus(dt.float() + w["dt_bias"])
    ld = -w["A"] * delta
    lm = torch.sigmoid(lam.float())
    lead = zx.shape[:-1]
    theta = (delta.unsqueeze(-1) * th.float().view(*lead, H, N // 2)).contiguous()
    return z, dict(X=x.reshape(*lead, H, P).contiguous(), logdecay=ld, gamma=lm * delta,
                   beta=(1 - lm) * delta * ld.exp(), B=norm(B, w["Bw"]).view(*lead, 1, N),
                   C=norm(C, w["Cw"]).view(*lead, 1, N), theta=theta)


def back(y, z, w):
    g = (y.float().reshape(-1, HP) * torch.nn.functional.silu(z.float().reshape(-1, HP)))
    q = m3.mx_quant(g.to(torch.bfloat16), "mxfp8")
    return q, m3.gemm_mx(q, w["q_out"])


ORDER = ("X", "logdecay", "beta", "gamma", "B", "C", "theta")


def check_gemm(D, A, W):
    a, v = (m3.mx_dequant(t, dtype=torch.float32).double() for t in (A, W))
    ref = a @ v.t()
    bound = 2.0 ** -8 * ref.abs() + A.cols * 2.0 ** -23 * (a.abs() @ v.abs().t()) + 1e-30
    assert ((D.double() - ref).abs() <= bound).all()


def test_prompt_then_tokens():
    w = {k: v.cuda() for k, v in weights().items()}
    w["q_in"], w["q_out"] = (m3.mx_quant(w[k], "mxfp4") for k in ("W_in", "W_out"))
    b, L, steps = 3, 37, 5
    g = torch.Generator().manual_seed(7)
    xs = torch.randn(b, L + steps, DM, generator=g).to(torch.bfloat16).cuda()
    rs = 3 * torch.randn(b, L + steps, DM, generator=g).cuda()

    # the prompt: the forward hands its cache to the 8-bit form
    yq, zx, r = front(xs[:, :L].reshape(-1, DM), rs[:, :L].reshape(-1, DM), w)
    assert torch.equal(r, xs[:, :L].reshape(-1, DM).float() + rs[:, :L].reshape(-1, DM))
    check_gemm(zx, yq, w["q_in"])
    z, s = split(zx.view(b, L, WIDTH), w)
    Y, hT, c = m3.fwd(*[s[k] for k in ORDER], w["D"], want_cache=True)
    cache = m3.quant_cache({**c, "ssm": hT})
    held = m3.dequant_cache(cache)["ssm"]
    amax = hT.abs().amax(-1, keepdim=True)
    assert ((held - hT).abs() <= torch.maximum(2.0 ** -4 * hT.abs(), 2.0 ** -10 / 448 * amax) * 1.001).all()
    yq, out = back(Y, z, w)
    check_gemm(out, yq, w["q_out"])
    assert torch.isfinite(out).all()

    # single tokens, captured once and replayed; the cache advances in place
    x_t, r_t = xs[:, L].clone(), rs[:, L].clone()
    def token():
        yq, zx, r = front(x_t, r_t, w)
        z, s = split(zx, w)
        y = m3.step_q8(cache, *[s[k] for k in ORDER], w["D"])
        gq, out = back(y, z, w)
        return yq, zx, r, s, y, gq, out
    before = {k: v.clone() for k, v in cache.items()}
    token()  # warms up what a first call sets
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yq, zx, r, s, y, gq, out = token()
    for k, v in before.items():
        cache[k].copy_(v)
    for t in range(steps):
        x_t.copy_(xs[:, L + t])
        r_t.copy_(rs[:, L + t])
        old = {k: v.cpu().numpy().copy() for k, v in cache.items()}
        graph.replay()
        torch.cuda.synchronize()
        check_gemm(zx, yq, w["q_in"])
        check_gemm(out, gq, w["q_out"])
        ref_y, ref = ol.step_q8(old, *[np64(s[k]) for k in ORDER], np64(w["D"]))
        # the step's bound, with every magnitude taken at its largest: h below its row's amax
        hmax = np.abs(ref["ssm"]).max()
        cmax = np.abs(np64(s["C"])).max() * math.sqrt(2)
        tol = (N + 40) * 2.0 ** -24 * N * cmax * (3 * hmax + 1) + 2.0 ** -8 * np.abs(ref_y)
        assert np.all(np.abs(np64(y) - ref_y) <= tol)
        new = ol.state_decode(cache["ssm"].cpu().numpy(), np64(cache["scale"]))
        half = np.maximum(2.0 ** -4 * np.abs(ref["ssm"]), 2.0 ** -10 * np64(cache["scale"])[..., None])
        assert np.all(np.abs(new - ref["ssm"]) <= half * 1.001 + 2.0 ** -18 * hmax)
    assert m3.device_wait_timeouts() == 0
