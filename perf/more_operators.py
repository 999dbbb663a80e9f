"""Timed cases of libm3ssd's gated linear recurrence, head norm with rotation and 4-bit products.

One pass is one of: the gated linear recurrence over a sequence (``glr_fwd``), its
backward (``glr_bwd``) and a decode step of it (``glr_step``); the norm of every head
of queries and keys with the rotation by position (``rot_fwd``) and its backward
(``rot_bwd``); the product of a few tokens with 4-bit weights in groups (``gemv``).

``run`` computes the plain form (elementary torch operations in fp32) while ``own`` is
false and calls the library while it is true; ``exact`` computes the definition in fp64.

The recurrence, per channel, with k = c softplus(rate):
    rho = sigmoid(r + bias_r),  iota = sigmoid(i + bias_i),  a = exp(-k rho), 0 at a reset,
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) iota_t x_t,  y_t = h_t.
Tokens at or past lengths[b] do not exist: y is zero there, as are the gradients.  The
backward reads h_{t-1} as the stored y_{t-1}.

The rotation turns pair (2i, 2i + 1) of a normed head by positions * freqs[i].

4-bit weights W (N, K): W = (code - zero) scale, codes 0 to 15, a bf16 scale and a zero
(8 unless given) for each row and group of columns.  K is padded to Kp, a multiple of
128, N to a multiple of 16.  Tiles of 16 rows by 128 columns take 1024 bytes, row
blocks outermost: byte 512 (r / 8) + 64 (r % 8) + 16 l + 4 j + m of row r of the tile
holds columns 32 j + 8 l + 2 m (low half) and the next one (high half).  Scales and
zeros are (groups, N).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESZ = {"bf16": 2, "f32": 4}
RATE_C = 8.0  # the recurrence's constant c
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # prefill or a training forward: 8 sequences of 4096 tokens, 32 x 64 channels
        {"name": "glr_fwd_8x4096", "op": "glr_fwd", "b": 8, "L": 4096, "D": 2048, "dtype": "bf16",
         "bias": True, "h0": False, "reset": False, "lengths": False},
        # prompts of unlike lengths in a padded batch, continued from a state, odd width, fp32
        {"name": "glr_fwd_ragged_f32", "op": "glr_fwd", "b": 3, "L": 1777, "D": 513, "dtype": "f32",
         "bias": True, "h0": True, "reset": False, "lengths": True},
        # the gradient of the training forward
        {"name": "glr_bwd_8x4096", "op": "glr_bwd", "b": 8, "L": 4096, "D": 2048, "dtype": "bf16",
         "grad": "bf16", "bias": True, "h0": False, "reset": False, "lengths": False},
        # few long sequences of packed documents, fp32 gradients
        {"name": "glr_bwd_2x32768", "op": "glr_bwd", "b": 2, "L": 32768, "D": 768, "dtype": "bf16",
         "grad": "f32", "bias": True, "h0": True, "reset": True, "lengths": False},
        # batched decoding: 256 sequences, one token each
        {"name": "glr_step_b256", "op": "glr_step", "b": 256, "D": 2048, "dtype": "bf16", "bias": True},
        # one sequence decoding
        {"name": "glr_step_b1", "op": "glr_step", "b": 1, "D": 1024, "dtype": "bf16", "bias": True},
        # decoding 256 sequences at positions of their own, 32 query and 8 key heads
        {"name": "rot_fwd_decode", "op": "rot_fwd", "rows": 256, "Hq": 32, "Hk": 8, "N": 128, "R": 64,
         "dtype": "bf16", "far": True},
        # the same heads over 8 x 4096 tokens
        {"name": "rot_fwd_32k", "op": "rot_fwd", "rows": 32768, "Hq": 32, "Hk": 8, "N": 128, "R": 64,
         "dtype": "bf16", "far": False},
        # gradients for the scan's one group of C and B (its backward returns fp32), a ragged
        # batch, half of the head rotated
        {"name": "rot_bwd_ragged", "op": "rot_bwd", "rows": 1777, "Hq": 1, "Hk": 1, "N": 128, "R": 32,
         "dtype": "bf16", "up": "f32", "grad": "f32", "far": False},
        # a training step's gradient at 32 query and 8 key heads, kept in bf16
        {"name": "rot_bwd_32k", "op": "rot_bwd", "rows": 32768, "Hq": 32, "Hk": 8, "N": 128, "R": 64,
         "dtype": "bf16", "up": "bf16", "grad": "bf16", "far": False},
        # in_proj of one decoding sequence
        {"name": "gemv_in_proj_m1", "op": "gemv", "M": 1, "N": 6464, "K": 1024, "group": 128,
         "zeros": False, "dtype": "bf16", "out": "bf16"},
        # logits of eight decoding sequences: a wide head, groups of 64 with zero points
        {"name": "gemv_head_m8", "op": "gemv", "M": 8, "N": 65536, "K": 4096, "group": 64,
         "zeros": True, "dtype": "bf16", "out": "f32"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["glr_fwd", "glr_bwd", "glr_step", "rot_fwd", "rot_bwd", "gemv"])
    dt = rng.choice(["bf16", "f32"])
    flag = lambda p: rng.random() < p  # noqa: E731
    if op == "glr_step":
        return {"op": op, "b": _log(rng, 1, 512), "D": _log(rng, 16, 4096), "dtype": dt,
                "bias": flag(0.7)}
    if op in ("glr_fwd", "glr_bwd"):
        D = _log(rng, 16, 4096)
        if flag(0.6):
            D = max(8, D // 8 * 8)
        c = {"op": op, "b": 1, "L": _log(rng, 1, 32768), "D": D, "dtype": dt, "bias": flag(0.7),
             "h0": flag(0.5), "reset": flag(0.4), "lengths": flag(0.4)}
        most = 67108864 if dt == "bf16" else 16777216
        if op == "glr_bwd":
            c["grad"] = dt if flag(0.5) else "f32"
            if c["grad"] != dt:
                most //= 2
        c["L"] = min(c["L"], most // D)
        c["b"] = _log(rng, 1, max(1, min(64, most // (D * c["L"]))))
        return c
    if op in ("rot_fwd", "rot_bwd"):
        N = 128 if flag(0.5) else 2 * rng.randint(4, 128)
        Hq, Hk = _log(rng, 1, 32), _log(rng, 1, 8)
        most = (32768 * 40 * 128) // (1 if dt == "bf16" else 4)
        c = {"op": op, "rows": _log(rng, 1, min(32768, most // (N * (Hq + Hk)))), "Hq": Hq,
             "Hk": Hk, "N": N, "R": N // 2 if flag(0.7) else rng.randint(1, N // 2), "dtype": dt,
             "far": flag(0.5)}
        if op == "rot_bwd":
            c["up"] = dt if flag(0.5) else "f32"
            c["grad"] = dt if flag(0.5) else "f32"
            if dt == "bf16" and "f32" in (c["up"], c["grad"]):
                c["rows"] = max(1, c["rows"] // 2)
        return c
    K = _log(rng, 32, 16384)
    if flag(0.6):
        K = max(32, K // 32 * 32)
    return {"op": op, "M": rng.randint(1, 16), "N": _log(rng, 1, min(65536, 268435456 // K)), "K": K,
            "group": rng.choice([32, 64, 128]), "zeros": flag(0.5), "dtype": dt,
            "out": rng.choice(["bf16", "f32"])}


# ---- inputs ---------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ru = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    s, dt = {"case": case}, DTYPES[case["dtype"]]
    if op.startswith("glr"):
        b, D = case["b"], case["D"]
        lead = (b, D) if op == "glr_step" else (b, case["L"], D)
        s["x"], s["r"], s["i"] = rn(*lead).to(dt), (1.5 * rn(*lead)).to(dt), (1.5 * rn(*lead)).to(dt)
        # exp(-softplus(rate)) between 0.9 and 0.999, the range such rates are started in
        s["rate"] = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * ru(D))))
        s["bias_r"], s["bias_i"] = (rn(D), rn(D)) if case["bias"] else (None, None)
        if op == "glr_step":
            s["h"] = rn(b, D)
            return s
        L = case["L"]
        s["h0"] = rn(b, D) if case["h0"] else None
        # packed documents of some 500 tokens
        s["reset"] = (ru(b, L) < 0.002) if case["reset"] else None
        s["lengths"] = (ru(b) * (L + 1)).to(torch.int32).clamp(max=L) if case["lengths"] else None
        if op == "glr_bwd":
            s["y"] = _glr_fwd(s)[0]
            s["dy"], s["dhT"] = rn(b, L, D).to(dt), rn(b, D) if case["h0"] else None
    elif op.startswith("rot"):
        rows, Hq, Hk, N = (case[k] for k in ("rows", "Hq", "Hk", "N"))
        s["q"] = (2 * rn(rows, Hq, N) * torch.exp(0.5 * rn(rows, Hq, 1))).to(dt)
        s["k"] = (2 * rn(rows, Hk, N) * torch.exp(0.5 * rn(rows, Hk, 1))).to(dt)
        s["q_w"], s["k_w"] = 0.5 + ru(N), 0.5 + ru(N)
        s["freqs"] = 10000.0 ** (-torch.arange(case["R"], device="cuda").float() * 2 / N)
        # sequences far into their caches, or prompts from the first token on
        s["positions"] = (ru(rows) * 500000).to(torch.int32) if case["far"] else \
            torch.arange(rows, device="cuda", dtype=torch.int32) % 4096
        if op == "rot_bwd":
            up = DTYPES[case["up"]]
            s["dq"], s["dk"] = rn(rows, Hq, N).to(up), rn(rows, Hk, N).to(up)
    else:
        M, N, K, gr = (case[k] for k in ("M", "N", "K", "group"))
        Kp, groups = (K + 127) // 128 * 128, (K + gr - 1) // gr
        s["x"] = (rn(M, K) * torch.exp(0.5 * rn(M, 1))).to(dt)
        codes = torch.randint(0, 16, (N, K), generator=g, device="cuda", dtype=torch.uint8)
        s["codes"] = _tile_codes(codes, Kp)
        s["scales"] = (K ** -0.5 / 4 * torch.exp(0.3 * rn(groups, N))).to(torch.bfloat16)
        s["zeros"] = torch.randint(4, 12, (groups, N), generator=g, device="cuda",
                                   dtype=torch.uint8) if case["zeros"] else None
    return s


def _tile_codes(codes, Kp):
    """(N, K) codes -> the tiled bytes, flat."""
    N, K = codes.shape
    Np = (N + 15) // 16 * 16
    p = torch.zeros(Np, Kp, dtype=torch.uint8, device=codes.device)
    p[:N, :K] = codes
    p = p[:, 0::2] | (p[:, 1::2] << 4)
    # (row block, r, k block, j, l, m) -> (row block, k block, r, l, j, m)
    return p.view(Np // 16, 16, Kp // 128, 4, 4, 4).permute(0, 2, 1, 4, 3, 5).reshape(-1)


def _untile_codes(t, N, K):
    Kp = (K + 127) // 128 * 128
    Np = (N + 15) // 16 * 16
    p = t.view(Np // 16, Kp // 128, 16, 4, 4, 4).permute(0, 2, 1, 4, 3, 5).reshape(Np, Kp // 2)
    return torch.stack((p & 15, p >> 4), -1).view(Np, Kp)[:N, :K]


# ---- one pass ---------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import selective_state_space_m3ssd_b200 as m3
    c, op = s["case"], s["case"]["op"]
    if op == "glr_fwd":
        y, hT = m3.glr_fwd(s["x"], s["r"], s["i"], s["rate"], bias_r=s["bias_r"], bias_i=s["bias_i"],
                           c=RATE_C, h0=s["h0"], reset=s["reset"], lengths=s["lengths"])
        return {"y": y, "hT": hT}
    if op == "glr_bwd":
        return m3.glr_bwd(s["x"], s["r"], s["i"], s["rate"], s["y"], s["dy"], bias_r=s["bias_r"],
                          bias_i=s["bias_i"], c=RATE_C, h0=s["h0"], reset=s["reset"],
                          lengths=s["lengths"], dhT=s["dhT"], grad_dtype=DTYPES[c["grad"]])
    if op == "glr_step":
        # the state goes to a buffer of its own, so that a pass can be repeated
        y, h = m3.glr_step(s["h"], s["x"], s["r"], s["i"], s["rate"], bias_r=s["bias_r"],
                           bias_i=s["bias_i"], c=RATE_C, h_out=torch.empty_like(s["h"]))
        return {"y": y, "h": h}
    if op == "rot_fwd":
        q, k = m3.norm_rotate(s["q"], s["k"], s["q_w"], s["k_w"], positions=s["positions"],
                              freqs=s["freqs"], eps=EPS)
        return {"q": q, "k": k}
    if op == "rot_bwd":
        return m3.norm_rotate_bwd(s["q"], s["k"], s["q_w"], s["k_w"], s["dq"], s["dk"],
                                  positions=s["positions"], freqs=s["freqs"], eps=EPS,
                                  grad_dtype=DTYPES[c["grad"]])
    W = m3.W4Tensor(c["N"], c["K"], c["group"], s["codes"], s["scales"], s["zeros"])
    return m3.gemv_w4(s["x"], W, out_dtype=DTYPES[c["out"]])


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _glr_gates(s):
    """x, k, rho, iota, log a, a and sqrt(1 - a^2) in fp32."""
    r, i = s["r"].float(), s["i"].float()
    if s["bias_r"] is not None:
        r, i = r + s["bias_r"], i + s["bias_i"]
    rho, iota = _sigmoid(r), _sigmoid(i)
    la = -RATE_C * torch.log1p(torch.exp(s["rate"])) * rho
    return s["x"].float(), rho, iota, la, torch.exp(la), torch.sqrt(-torch.expm1(2 * la))


def _alive(s):
    """(b, L, 1): whether a token exists."""
    t = torch.arange(s["case"]["L"], device="cuda")
    return (t < s["lengths"].unsqueeze(-1)).unsqueeze(-1)


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t along axis 1, by doubling."""
    d, L = 1, a.shape[1]
    while d < L:
        u = torch.cat((u[:, :d], u[:, d:] + a[:, d:] * u[:, :-d]), 1)
        a = torch.cat((a[:, :d], a[:, d:] * a[:, :-d]), 1)
        d *= 2
    return u


def _glr_fwd(s):
    x, _, iota, _, a, sq = _glr_gates(s)
    if s["reset"] is not None:
        a, sq = a.masked_fill(s["reset"].unsqueeze(-1), 0), sq.masked_fill(s["reset"].unsqueeze(-1), 1)
    u = sq * iota * x
    if s["lengths"] is not None:
        on = _alive(s)
        a, u = a.masked_fill(~on, 1), u.masked_fill(~on, 0)
    if s["h0"] is not None:
        u[:, 0] += a[:, 0] * s["h0"]
    h = _scan(a, u)
    hT = h[:, -1].contiguous()
    if s["lengths"] is not None:
        h = h.masked_fill(~on, 0)
    return h.to(s["x"].dtype), hT


def _glr_bwd(s):
    gd = DTYPES[s["case"]["grad"]]
    x, rho, iota, la, a, sq = _glr_gates(s)
    if s["reset"] is not None:
        cut = s["reset"].unsqueeze(-1)
        a, sq = a.masked_fill(cut, 0), sq.masked_fill(cut, 1)
    dy = s["dy"].float()
    if s["lengths"] is not None:
        on = _alive(s)
        a, dy = a.masked_fill(~on, 1), dy.masked_fill(~on, 0)
    # time reversed: g_t = dy_t + a_{t+1} g_{t+1}
    dy = dy.flip(1)
    if s["dhT"] is not None:
        dy[:, 0] += s["dhT"]
    nxt = torch.cat((torch.ones_like(a[:, :1]), a[:, 1:].flip(1)), 1)
    g = _scan(nxt, dy).flip(1)
    dh0 = a[:, 0] * g[:, 0]
    first = torch.zeros_like(x[:, 0]) if s["h0"] is None else s["h0"]
    prev = torch.cat((first.unsqueeze(1), s["y"][:, :-1].float()), 1)
    ratio = torch.where(sq > 0, la / sq, 0)
    E = g * (a * la * prev - a * a * ratio * iota * x)
    if s["reset"] is not None:
        E = E.masked_fill(cut, 0)
    dx = g * sq * iota
    di, dr = dx * x * (1 - iota), E * (1 - rho)
    if s["lengths"] is not None:
        dx, di, dr, E = (v.masked_fill(~on, 0) for v in (dx, di, dr, E))
    total = lambda v: v.sum((0, 1), dtype=torch.float64).float()  # noqa: E731
    slope = _sigmoid(s["rate"]) / torch.log1p(torch.exp(s["rate"]))
    return {"dx": dx.to(gd), "dr": dr.to(gd), "di": di.to(gd), "drate": total(E) * slope,
            "dbias_r": total(dr), "dbias_i": total(di), "dh0": dh0}


def _turns(s):
    """cos and sin of every (row, pair), from angles in fp64."""
    ang = s["positions"].double().unsqueeze(-1) * s["freqs"].double()
    return torch.cos(ang).float().unsqueeze(1), torch.sin(ang).float().unsqueeze(1)


def _rotate(v, c, sn):
    R = c.shape[-1]
    p, rest = v[..., :2 * R].unflatten(-1, (R, 2)), v[..., 2 * R:]
    re, im = p[..., 0], p[..., 1]
    return torch.cat((torch.stack((c * re - sn * im, sn * re + c * im), -1).flatten(-2), rest), -1)


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "glr_fwd":
        y, hT = _glr_fwd(s)
        return {"y": y, "hT": hT}
    if op == "glr_bwd":
        return _glr_bwd(s)
    if op == "glr_step":
        x, _, iota, _, a, sq = _glr_gates(s)
        h = a * s["h"] + sq * iota * x
        return {"y": h.to(s["x"].dtype), "h": h}
    if op == "rot_fwd":
        cs, out = _turns(s), {}
        for n in ("q", "k"):
            u = s[n].float()
            v = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS) * s[n + "_w"]
            out[n] = _rotate(v, *cs).to(s[n].dtype)
        return out
    if op == "rot_bwd":
        (co, si), out = _turns(s), {}
        for n in ("q", "k"):
            u = s[n].float()
            rstd = torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)
            dv, uh = _rotate(s["d" + n].float(), co, -si), u * rstd
            gw = dv * s[n + "_w"]
            out["d" + n] = (rstd * (gw - uh * (gw * uh).mean(-1, keepdim=True))).to(DTYPES[c["grad"]])
            out["d" + n + "_w"] = (dv * uh).sum((0, 1), dtype=torch.float64).float()
        return out
    W = _weights(s, torch.float32)
    return torch.matmul(s["x"].float(), W.t()).to(DTYPES[c["out"]])


def _weights(s, dtype):
    c = s["case"]
    g = torch.arange(c["K"], device="cuda") // c["group"]
    zero = 8 if s["zeros"] is None else s["zeros"].to(dtype)[g].t()
    return (_untile_codes(s["codes"], c["N"], c["K"]).to(dtype) - zero) * s["scales"].to(dtype)[g].t()


# ---- the definition in fp64 ----------------------------------------------------------

def exact(case, seed):
    """run()'s outputs in fp64."""
    s, op = prepare(case, seed), case["op"]
    return {"glr_fwd": _exact_glr_fwd, "glr_bwd": _exact_glr_bwd, "glr_step": _exact_glr_step,
            "rot_fwd": _exact_rot_fwd, "rot_bwd": _exact_rot_bwd,
            "gemv": _exact_gemv}[op](s)


def _exact_token(s, pick):
    """(x, rho, iota, log a, a, scale of the input) of the tokens that pick() takes, fp64."""
    br = 0 if s["bias_r"] is None else s["bias_r"].double()
    bi = 0 if s["bias_i"] is None else s["bias_i"].double()
    rho = torch.special.expit(pick(s["r"]).double() + br)
    iota = torch.special.expit(pick(s["i"]).double() + bi)
    la = -RATE_C * torch.nn.functional.softplus(s["rate"].double(), threshold=40.0) * rho
    a = la.exp()
    return pick(s["x"]).double(), rho, iota, la, a, ((1 - a) * (1 + a)).sqrt()


def _exact_glr_step(s):
    x, _, iota, _, a, sq = _exact_token(s, lambda v: v)
    h = a * s["h"].double() + sq * iota * x
    return {"y": h, "h": h}


def _exact_glr_fwd(s):
    """Token by token."""
    c = s["case"]
    h = torch.zeros(c["b"], c["D"], dtype=torch.float64, device="cuda") if s["h0"] is None \
        else s["h0"].double()
    ys = torch.zeros(c["b"], c["L"], c["D"], dtype=torch.float64, device="cuda")
    for t in range(c["L"]):
        x, _, iota, _, a, sq = _exact_token(s, lambda v: v[:, t])
        new = a * h + sq * iota * x
        if s["reset"] is not None:
            new = torch.where(s["reset"][:, t, None], iota * x, new)
        if s["lengths"] is None:
            h = ys[:, t] = new
        else:
            live = (t < s["lengths"])[:, None]
            h = torch.where(live, new, h)
            ys[:, t] = torch.where(live, new, 0)
    return {"y": ys, "hT": h}


def _exact_glr_bwd(s):
    """Token by token from the last: g, the gradient of h_t, goes back through
    h_t = a h_{t-1} + sqrt(1 - a^2) iota x with h_{t-1} as stored."""
    c, f64 = s["case"], torch.float64
    b, L, D = c["b"], c["L"], c["D"]
    back = torch.zeros(b, D, dtype=f64, device="cuda") if s["dhT"] is None else s["dhT"].double()
    out = {k: torch.zeros(b, L, D, dtype=f64, device="cuda") for k in ("dx", "dr", "di")}
    sums = {k: torch.zeros(D, dtype=f64, device="cuda") for k in ("rate", "r", "i")}
    for t in range(L - 1, -1, -1):
        x, rho, iota, la, a, sq = _exact_token(s, lambda v: v[:, t])
        if t > 0:
            prev = s["y"][:, t - 1].double()
        else:
            prev = 0 if s["h0"] is None else s["h0"].double()
        cut = None if s["reset"] is None else s["reset"][:, t, None]
        g = s["dy"][:, t].double() + back
        if cut is not None:
            a, sq = torch.where(cut, 0, a), torch.where(cut, 1, sq)
        dla = g * (a * prev - a.square() / sq * iota * x)
        if cut is not None:
            dla = torch.where(cut, 0, dla)
        one = {"dx": g * sq * iota, "di": g * sq * x * iota * (1 - iota), "dr": dla * la * (1 - rho)}
        rate, new = dla * la, a * g
        if s["lengths"] is not None:
            live = (t < s["lengths"])[:, None]
            one = {k: torch.where(live, v, 0) for k, v in one.items()}
            rate, new = torch.where(live, rate, 0), torch.where(live, new, back)
        back = new
        for k, v in one.items():
            out[k][:, t] = v
        sums["rate"] += rate.sum(0)
        sums["r"] += one["dr"].sum(0)
        sums["i"] += one["di"].sum(0)
    k = s["rate"].double()
    slope = torch.special.expit(k) / torch.nn.functional.softplus(k, threshold=40.0)
    return {**out, "drate": sums["rate"] * slope, "dbias_r": sums["r"], "dbias_i": sums["i"],
            "dh0": back}


def _exact_turn(s, sign):
    """exp(i sign angle), 1 for the pairs that are not turned; (rows, 1, N / 2)."""
    c = s["case"]
    ang = torch.zeros(c["rows"], c["N"] // 2, dtype=torch.float64, device="cuda")
    ang[:, :c["R"]] = torch.outer(s["positions"].double(), s["freqs"].double())
    return torch.polar(torch.ones_like(ang), sign * ang).unsqueeze(1)


def _exact_turned(v, z):
    # a few rows at a time: complex pairs take eight times a bf16 tensor
    out = torch.empty_like(v)
    for lo in range(0, v.shape[0], 4096):
        part = torch.view_as_complex(v[lo:lo + 4096].unflatten(-1, (-1, 2)).contiguous())
        out[lo:lo + 4096] = torch.view_as_real(part * z[lo:lo + 4096]).flatten(-2)
    return out


def _exact_rot_fwd(s):
    z, out = _exact_turn(s, 1), {}
    for n in ("q", "k"):
        u = s[n].double()
        inv = (torch.einsum("rhn,rhn->rh", u, u) / u.shape[-1] + EPS) ** -0.5
        out[n] = _exact_turned(u * inv[..., None] * s[n + "_w"].double(), z)
    return out


def _exact_rot_bwd(s):
    z, out = _exact_turn(s, -1), {}
    for n in ("q", "k"):
        u, w = s[n].double(), s[n + "_w"].double()
        inv = (torch.einsum("rhn,rhn->rh", u, u) / u.shape[-1] + EPS) ** -0.5
        dv = _exact_turned(s["d" + n].double(), z)
        # the quotient rule on u inv(u) w
        dot = torch.einsum("rhn,n,rhn->rh", dv, w, u)
        out["d" + n] = inv[..., None] * dv * w - (inv ** 3 * dot / u.shape[-1])[..., None] * u
        out["d" + n + "_w"] = torch.einsum("rhn,rhn,rh->n", dv, u, inv)
    return out


def _exact_gemv(s):
    """Group by group: the codes' integer products first, then the group's scale."""
    c = s["case"]
    x, K, gr = s["x"].double(), c["K"], c["group"]
    codes = _untile_codes(s["codes"], c["N"], K)
    out = torch.zeros(c["M"], c["N"], dtype=torch.float64, device="cuda")
    for j in range((K + gr - 1) // gr):
        cols = slice(j * gr, min(K, (j + 1) * gr))
        part = x[:, cols] @ codes[:, cols].double().t()
        zero = 8.0 if s["zeros"] is None else s["zeros"][j].double()
        out += (part - x[:, cols].sum(1, keepdim=True) * zero) * s["scales"][j].double()
    return out


# ---- what a pass cannot do without -------------------------------------------------------

def work(case):
    op, e = case["op"], ESZ[case["dtype"]]
    if op == "glr_step":
        n = case["b"] * case["D"]
        return {"bytes": n * (4 * e + 8) + 4 * case["D"] * (3 if case["bias"] else 1), "flops": 25 * n}
    if op in ("glr_fwd", "glr_bwd"):
        b, D = case["b"], case["D"]
        n = b * case["L"] * D
        side = 4 * D * (3 if case["bias"] else 1) + 4 * b * D * (1 + case["h0"]) + \
            b * case["L"] * case["reset"]
        if op == "glr_fwd":
            return {"bytes": 4 * n * e + side, "flops": 25 * n}
        return {"bytes": n * (5 * e + 3 * ESZ[case["grad"]]) + 2 * side, "flops": 45 * n}
    if op in ("rot_fwd", "rot_bwd"):
        n = case["rows"] * (case["Hq"] + case["Hk"]) * case["N"]
        side = 4 * case["rows"] + 4 * case["R"] + 8 * case["N"]
        if op == "rot_fwd":
            return {"bytes": 2 * n * e + side, "flops": 8 * n}
        return {"bytes": n * (e + ESZ[case["up"]] + ESZ[case["grad"]]) + side + 8 * case["N"],
                "flops": 16 * n}
    M, N, K = case["M"], case["N"], case["K"]
    groups = (K + case["group"] - 1) // case["group"]
    return {"bytes": N * K / 2 + N * groups * (2 + case["zeros"]) + M * K * e + M * N * ESZ[case["out"]],
            "flops": 2 * M * N * K}
