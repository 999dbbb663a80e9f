"""Timed cases of the low-bit and normalisation operators of libm3ssd.

One pass is one of: the residual addition with the root-mean-square norm
(``norm``, output in bf16, fp32, MXFP8 or MXFP4) and its backward
(``norm_bwd``); a tensor quantised to a microscaled format and read back
(``mx``); the product of two microscaled operands (``gemm``); a decode step on
a cache whose state is held in 8 bits (``step``); and the hand-over of an fp32
state to such a cache and back (``cache``).

``run`` computes the plain form (elementary torch operations in fp32) while
``own`` is false and calls the library while it is true; ``exact`` computes the
definition in fp64.

Formats.  An MX tensor holds blocks of 32 values along its last axis, each
block with a power-of-two scale 2^E, the least with amax <= maxval 2^E (maxval
6 for E2M1 codes, 448 for E4M3 codes; E clamped to [-127, 127], byte E + 127;
a block of zeros takes byte 0).  Codes are value / 2^E rounded to nearest even.  The
last axis is padded with zeros to a multiple of 128; E2M1 codes are packed two a
byte, the even index in the low half.  The scales of 128 rows by 4 blocks
form a 512-byte tile: byte (r % 32) * 16 + (r / 32) * 4 + k for row r and block k
of the tile, tiles row-block-major, missing rows with byte 0.  The 8-bit state
holds E4M3 codes and one fp32 scale for each row of headdim values, s = amax /
448 (zero below 2^-100), code = value * (1 / s) rounded to nearest even.
"""
import math

import torch

own = False

FMT_MAX = {"mxfp4": 6.0, "mxfp8": 448.0}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # the layer's entry in batched decoding: 256 sequences, one token each, fp32 residual
        # stream, the in_proj operand in 8 bits
        {"name": "norm_decode_b256", "op": "norm", "rows": 256, "d": 1024, "dtype": "bf16",
         "res": "f32", "fmt": "mxfp8"},
        # the same at the forward's workload (8 x 4096 tokens), output in bf16
        {"name": "norm_prefill_32k", "op": "norm", "rows": 32768, "d": 1024, "dtype": "bf16",
         "res": "f32", "fmt": "none"},
        # a training step's norm gradient over a ragged batch at d_model 768, bf16 residual stream
        {"name": "norm_bwd_ragged", "op": "norm_bwd", "rows": 1777, "d": 768, "dtype": "bf16",
         "res": "bf16", "dres": True},
        # the same at the training workload
        {"name": "norm_bwd_32k", "op": "norm_bwd", "rows": 32768, "d": 1024, "dtype": "bf16",
         "res": "f32", "dres": True},
        # gated outputs before out_proj, quantised to 4 bits and read back (prefill)
        {"name": "mx4_prefill", "op": "mx", "rows": 32768, "cols": 2048, "dtype": "bf16",
         "fmt": "mxfp4"},
        # an fp32 activation of odd sizes in 8 bits
        {"name": "mx8_odd", "op": "mx", "rows": 333, "cols": 1049, "dtype": "f32", "fmt": "mxfp8"},
        # in_proj of 16 decoding sequences: 8-bit activations, 4-bit weights streamed once
        {"name": "gemm_decode_m16", "op": "gemm", "M": 16, "N": 6464, "K": 1024, "a": "mxfp8"},
        # in_proj of a prompt of 8 x 4096 tokens, both operands in 4 bits
        {"name": "gemm_in_proj_44", "op": "gemm", "M": 32768, "N": 6464, "K": 1024, "a": "mxfp4"},
        # out_proj of a ragged prompt, 8-bit activations, 4-bit weights
        {"name": "gemm_out_proj_84", "op": "gemm", "M": 20011, "N": 1024, "K": 2048, "a": "mxfp8"},
        # batched decode: 256 sequences, 32 heads
        {"name": "step_b256", "op": "step", "b": 256, "H": 32, "G": 1, "N": 128, "P": 64,
         "dtype": "f32", "beta": True, "theta": True, "D": True},
        # a few sequences decoding, bf16 inputs
        {"name": "step_b3_h24", "op": "step", "b": 3, "H": 24, "G": 1, "N": 128, "P": 64,
         "dtype": "bf16", "beta": True, "theta": True, "D": True},
        # the state of 64 sequences handed from prefill to the 8-bit cache, and read back
        {"name": "cache_b64", "op": "cache", "b": 64, "H": 32, "N": 128, "P": 64},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "mx", "gemm", "step", "cache"])
    dt = rng.choice(["bf16", "f32"])
    if op in ("norm", "norm_bwd"):
        d = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            d = max(8, d // 8 * 8)
        rows = _log(rng, 1, min(32768, 32768 * 1024 // d))
        c = {"op": op, "rows": rows, "d": d, "dtype": dt}
        if op == "norm":
            return {**c, "res": rng.choice(["none", "f32", "bf16"]),
                    "fmt": rng.choice(["none", "mxfp8", "mxfp4"])}
        return {**c, "res": rng.choice(["f32", "bf16"]), "dres": rng.random() < 0.7}
    if op == "mx":
        cols = _log(rng, 32, 8192)
        rows = _log(rng, 1, min(32768, 32768 * 1024 // cols))
        return {"op": op, "rows": rows, "cols": cols, "dtype": dt,
                "fmt": rng.choice(["mxfp8", "mxfp4"])}
    if op == "gemm":
        n, k = _log(rng, 16, 8192), _log(rng, 32, 8192)
        if rng.random() < 0.6:
            n, k = max(8, n // 8 * 8), max(32, k // 32 * 32)
        m = _log(rng, 1, min(32768, max(1, 32768 * 6464 * 1024 // (n * k))))
        return {"op": op, "M": m, "N": n, "K": k, "a": rng.choice(["mxfp8", "mxfp4"])}
    if rng.random() < 0.6:
        n, p = 128, 64
    else:
        n = 2 * rng.randint(1, 128)
        p = rng.randint(1, min(256, 16384 // n))
    h = rng.choice([2, 6, 8, 24, 32, 48])
    b = _log(rng, 1, max(1, min(256, 256 * 32 * 128 * 64 // (h * n * p))))
    if op == "cache":
        return {"op": op, "b": b, "H": h, "N": n, "P": p}
    return {"op": op, "b": b, "H": h, "G": rng.choice([1, 2, h]), "N": n, "P": p, "dtype": dt,
            "beta": rng.random() < 0.8, "theta": rng.random() < 0.8, "D": rng.random() < 0.8}


# ---- the formats, elementary ------------------------------------------------------

def _pad128(k):
    return (k + 127) // 128 * 128


def _scale_exp(amax, fmt):
    """E of the least power of two with amax <= maxval 2^E, clamped (int32; fp32 or fp64 amax)."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1)
    E = e - (3 if fmt == "mxfp4" else 9) + (m > (0.75 if fmt == "mxfp4" else 0.875)).to(e.dtype)
    return torch.where(amax > 0, E, torch.full_like(E, -127)).clamp(-127, 127)


def _round_e2m1(v):
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(v.dtype)
    return torch.copysign(torch.round(a / step) * step, v)


def _pow2(e, dtype):
    return ((e.long() + 1023) << 52).view(torch.float64).to(dtype)


def _mx_values(x, fmt):
    """x (rows, cols) floating -> (rounded codes' values, E), both padded: (rows, Kp), (rows, Kp/32)."""
    rows, cols = x.shape
    xp = torch.zeros(rows, _pad128(cols), dtype=x.dtype, device=x.device)
    xp[:, :cols] = x
    blk = xp.view(rows, -1, 32)
    E = _scale_exp(blk.abs().amax(-1), fmt)
    v = (blk.double() * _pow2(-E, torch.float64).unsqueeze(-1)).to(x.dtype)
    q = _round_e2m1(v) if fmt == "mxfp4" else v.float().to(torch.float8_e4m3fn).to(x.dtype)
    return q.view(rows, -1), E


def _pack_codes(q, fmt):
    """Code values (rows, Kp) -> stored codes."""
    if fmt == "mxfp8":
        return q.float().to(torch.float8_e4m3fn).view(torch.uint8)
    a = q.abs()
    idx = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c = idx | (torch.signbit(q).to(torch.uint8) << 3)
    return c[:, 0::2] | (c[:, 1::2] << 4)


def _tile_scales(E):
    """(rows, blocks) exponents -> scale bytes in 128 x 4 tiles."""
    rows, nb = E.shape
    rp = _pad128(rows)
    s = torch.zeros(rp, nb, dtype=torch.uint8, device=E.device)
    s[:rows] = (E + 127).to(torch.uint8)
    return s.view(rp // 128, 4, 32, nb // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile_scales(s, rows, nb):
    t = s.view(-1, nb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, nb)
    return t[:rows].to(torch.int32) - 127


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _decode(codes, scales, rows, cols, fmt, dtype):
    """Stored codes and tiled scales -> values (rows, cols)."""
    if fmt == "mxfp8":
        q = codes.view(torch.float8_e4m3fn).to(dtype)
    else:
        table = torch.tensor(_E2M1, dtype=dtype, device=codes.device)
        q = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1)
        q = q.view(rows, -1)
    E = _untile_scales(scales, rows, q.shape[1] // 32)
    return (q.view(rows, -1, 32) * _pow2(E, dtype).unsqueeze(-1)).view(rows, -1)[:, :cols]


# ---- inputs ---------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ru = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    s = {"case": case}
    if op == "norm":
        rows, d = case["rows"], case["d"]
        s["x"] = rn(rows, d).to(DTYPES[case["dtype"]])
        # a residual stream grows with depth: a few times the new branch, rows of unlike size
        s["res"] = None if case["res"] == "none" else \
            (3 * rn(rows, d) * torch.exp(0.5 * rn(rows, 1))).to(DTYPES[case["res"]])
        s["w"] = 0.5 + ru(d)
    elif op == "norm_bwd":
        rows, d = case["rows"], case["d"]
        s["r"] = (3 * rn(rows, d) * torch.exp(0.5 * rn(rows, 1))).to(DTYPES[case["res"]])
        s["dy"] = rn(rows, d).to(DTYPES[case["dtype"]])
        s["dres"] = rn(rows, d) if case["dres"] else None
        s["w"] = 0.5 + ru(d)
        s["rstd"] = (1 / torch.sqrt(s["r"].double().square().mean(-1) + 1e-6)).float()
    elif op == "mx":
        # heavy-tailed activations: a few channels ten times the rest, some rows near zero
        x = rn(case["rows"], case["cols"]) * torch.exp(1.5 * rn(case["rows"], 1))
        x *= torch.where(ru(case["cols"]) < 0.02, 10.0, 1.0)
        s["x"] = x.to(DTYPES[case["dtype"]])
    elif op == "gemm":
        for name, rows, fmt, mag in (("A", case["M"], case["a"], 1.0),
                                     ("W", case["N"], "mxfp4", case["K"] ** -0.5)):
            x = rn(rows, case["K"]) * (mag * torch.exp(0.5 * rn(rows, 1)))
            q, E = _mx_values(x, fmt)
            s[name] = (_pack_codes(q, fmt), _tile_scales(E))
    else:
        b, H, N, P = (case[k] for k in ("b", "H", "N", "P"))
        ssm = 0.3 * rn(b, H, N, P) * torch.exp(0.7 * rn(b, H, N, 1))
        if op == "cache":
            s["ssm"] = ssm
            return s
        G, xd = case["G"], DTYPES[case["dtype"]]
        q, scale = _state_codes(ssm)
        del ssm
        pi = math.pi
        s["cache"] = {"angle": ru(b, H, N // 2) * (2 * pi) - pi, "ssm": q, "scale": scale,
                      "x_prev": rn(b, H, P).to(xd).float(),
                      "b_prev": (rn(b, G, N) * N ** -0.5).to(xd).float()}
        # the step sizes and decays of the scan's inputs
        delta = torch.log1p(torch.exp(rn(b, H) - 2))
        ld = -delta * (1 + 15 * ru(H))
        lam = torch.sigmoid(rn(b, H))
        s["logdecay"], s["gamma"] = ld, lam * delta
        s["beta"] = (1 - lam) * delta * torch.exp(ld) if case["beta"] else None
        s["theta"] = delta.unsqueeze(-1) * rn(b, H, N // 2) if case["theta"] else None
        s["D"] = rn(H) if case["D"] else None
        s["x"] = rn(b, H, P).to(xd)
        s["B"] = (rn(b, G, N) * N ** -0.5).to(xd)
        s["C"] = (rn(b, G, N) * N ** -0.5).to(xd)
        s["out"] = {k: torch.empty_like(v) for k, v in s["cache"].items()}
    return s


# ---- one pass ---------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import selective_state_space_m3ssd_b200 as m3
    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        fmt = None if c["fmt"] == "none" else c["fmt"]
        y, r, rstd = m3.add_rmsnorm(s["x"], s["w"], residual=s["res"], eps=1e-6, fmt=fmt,
                                    want_rstd=True)
        if fmt == "mxfp8":
            y = (y.codes.view(torch.float8_e4m3fn), y.scales.view(torch.float8_e8m0fnu))
        elif fmt == "mxfp4":
            y = m3.mx_dequant(y, dtype=torch.bfloat16)
        return {"y": y, "r": r, "rstd": rstd}
    if op == "norm_bwd":
        dr, dw = m3.add_rmsnorm_bwd(s["dy"], s["r"], s["w"], s["rstd"], dres=s["dres"])
        return {"dr": dr, "dw": dw}
    if op == "mx":
        return m3.mx_dequant(m3.mx_quant(s["x"], c["fmt"]), dtype=s["x"].dtype)
    if op == "gemm":
        A = m3.MXTensor(c["a"], c["M"], c["K"], *s["A"])
        W = m3.MXTensor("mxfp4", c["N"], c["K"], *s["W"])
        return m3.gemm_mx(A, W)
    if op == "cache":
        q, scale = m3.quant_state(s["ssm"])
        return {"q": q.view(torch.float8_e4m3fn), "scale": scale, "ssm": m3.dequant_state(q, scale)}
    y, o = m3.step_q8(s["cache"], s["x"], s["logdecay"], s["beta"], s["gamma"], s["B"], s["C"],
                      s["theta"], s["D"], cache_out=s["out"]), s["out"]
    return {"y": y, **{k: o[k] for k in ("angle", "scale", "x_prev", "b_prev")},
            "q": o["ssm"].view(torch.float8_e4m3fn)}


def _state_codes(h):
    """fp32 state (..., P) -> (codes as uint8, scales): s = amax / 448, code = h (1 / s)."""
    amax = h.abs().amax(-1)
    scale = torch.where(amax >= 2.0 ** -100, amax / 448, 0)
    inv = torch.where(scale > 0, 1 / scale, 0)
    return (h * inv.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        x, r = s["x"].float(), None
        if s["res"] is not None:
            r = (x + s["res"].float()).to(s["res"].dtype)
            x = r.float()
        rstd = 1 / torch.sqrt((x * x).mean(-1) + 1e-6)
        y = x * rstd.unsqueeze(-1) * s["w"]
        if c["fmt"] == "none":
            y = y.to(s["x"].dtype)
        else:
            q, E = _mx_values(y, c["fmt"])
            if c["fmt"] == "mxfp8":
                y = (q.to(torch.float8_e4m3fn), _tile_scales(E).view(torch.float8_e8m0fnu))
            else:
                y = (q.view(c["rows"], -1, 32) * _pow2(E, torch.float32).unsqueeze(-1)) \
                    .view(c["rows"], -1)[:, :c["d"]].to(torch.bfloat16)
        return {"y": y, "r": r, "rstd": rstd}
    if op == "norm_bwd":
        r, dy, rstd = s["r"].float(), s["dy"].float(), s["rstd"].unsqueeze(-1)
        rh, wdy = r * rstd, dy * s["w"]
        dr = rstd * (wdy - rh * (wdy * rh).mean(-1, keepdim=True))
        if s["dres"] is not None:
            dr = dr + s["dres"]
        return {"dr": dr, "dw": (dy * rh).sum(0, dtype=torch.float64).float()}
    if op == "mx":
        x = s["x"].float()
        q, E = _mx_values(x, c["fmt"])
        v = (q.view(c["rows"], -1, 32).double() * _pow2(E, torch.float64).unsqueeze(-1))
        return v.view(c["rows"], -1)[:, :c["cols"]].to(s["x"].dtype).contiguous()
    if op == "gemm":
        A = _decode(*s["A"], c["M"], c["K"], c["a"], torch.float32)
        W = _decode(*s["W"], c["N"], c["K"], "mxfp4", torch.float32)
        return torch.matmul(A, W.t()).to(torch.bfloat16)
    if op == "cache":
        q, scale = _state_codes(s["ssm"])
        q = q.view(torch.float8_e4m3fn)
        return {"q": q, "scale": scale, "ssm": q.float() * scale.unsqueeze(-1)}
    y, new, h = _step(s, torch.float32)
    q, scale = _state_codes(h)
    return {"y": y.to(s["x"].dtype), "angle": new["angle"].float(), "scale": scale,
            "x_prev": new["x_prev"], "b_prev": new["b_prev"], "q": q.view(torch.float8_e4m3fn)}


def _rot(v, ang):
    """Pairs of v (b, H, N) rotated by ang (b, H, N/2)."""
    c, s, a, b = torch.cos(ang), torch.sin(ang), v[..., 0::2], v[..., 1::2]
    return torch.stack((c * a - s * b, s * a + c * b), -1).flatten(-2)


def _wrapped(angle, theta):
    """angle + theta reduced to [-pi, pi], in fp64; the turn is counted on the fp32 sum."""
    t = angle if theta is None else angle + theta
    k = torch.round(t * 0.159154943091895336)
    return t.double() - k.double() * (2 * math.pi)


def _step(s, dtype):
    """(y, new small cache parts, new state) of a step on the 8-bit cache."""
    c, o = s["case"], s["cache"]
    rep = lambda v: v.to(dtype).repeat_interleave(c["H"] // c["G"], 1)  # noqa: E731
    new = _wrapped(o["angle"], s["theta"])
    Bb, Cb = _rot(rep(s["B"]), new.to(dtype)), _rot(rep(s["C"]), new.to(dtype))
    x = s["x"].to(dtype)
    h = o["ssm"].view(torch.float8_e4m3fn).to(dtype) * o["scale"].to(dtype).unsqueeze(-1)
    h = h * torch.exp(s["logdecay"].to(dtype))[..., None, None]
    h = h + (s["gamma"].to(dtype)[..., None] * Bb).unsqueeze(-1) * x.unsqueeze(-2)
    if s["beta"] is not None:
        Bp = _rot(rep(o["b_prev"]), o["angle"].to(dtype))
        h = h + (s["beta"].to(dtype)[..., None] * Bp).unsqueeze(-1) * \
            o["x_prev"].to(dtype).unsqueeze(-2)
    y = (Cb.unsqueeze(-1) * h).sum(-2)
    if s["D"] is not None:
        y = y + s["D"].to(dtype)[:, None] * x
    return y, {"angle": new, "x_prev": s["x"].float(), "b_prev": s["B"].float()}, h


# ---- the definition in fp64 ----------------------------------------------------------

def exact(case, seed):
    """run()'s floating outputs in fp64; None where an output was rounded to 8 or 4 bits from a
    computed value (the rounding of a value next to a border has no single answer)."""
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        r = None
        v = s["x"].double()
        if s["res"] is not None:
            r = (s["x"].double() + s["res"].double()).float().to(s["res"].dtype).double()
            v = r
        inv = (v.pow(2).sum(1) / case["d"] + 1e-6).pow(-0.5)
        y = v * inv[:, None] * s["w"].double() if case["fmt"] == "none" else \
            (None, None) if case["fmt"] == "mxfp8" else None
        return {"y": y, "r": r, "rstd": inv}
    if op == "norm_bwd":
        # the derivative of sum(dy . (r rstd(r) w)) written out by the quotient rule
        r, dy, w, q = (s[k].double() for k in ("r", "dy", "w", "rstd"))
        g = dy * w
        dr = q[:, None] * g - (q ** 3 / case["d"] * torch.einsum("ij,ij->i", g, r))[:, None] * r
        if s["dres"] is not None:
            dr += s["dres"].double()
        return {"dr": dr, "dw": torch.einsum("ij,ij,i->j", dy, r, q)}
    if op == "mx":
        x = s["x"].double()
        rows, cols = x.shape
        x = torch.nn.functional.pad(x, (0, -cols % 32)).view(rows, -1, 32)
        top = FMT_MAX[case["fmt"]]
        # 1e-9: less than the distance of a value above the border, more than log2's error
        E = torch.ceil(torch.log2((x.abs().amax(-1) / top).clamp(min=2.0 ** -127)) - 1e-9)
        E = E.clamp(-127, 127)
        unit = torch.exp2(E)[..., None]
        grid = torch.tensor(_grid(case["fmt"]), dtype=torch.float64, device=x.device)
        a = (x / unit).abs().contiguous()
        hi = torch.searchsorted(grid, a).clamp(1, grid.numel() - 1)
        lo = hi - 1
        up = a - grid[lo] > grid[hi] - a
        tie = a - grid[lo] == grid[hi] - a
        q = grid[torch.where(up | (tie & (hi % 2 == 0)), hi, lo)]
        return (torch.sign(x) * q * unit).view(rows, -1)[:, :cols].contiguous()
    if op == "gemm":
        A = _decode(*s["A"], case["M"], case["K"], case["a"], torch.float64)
        W = _decode(*s["W"], case["N"], case["K"], "mxfp4", torch.float64)
        return A @ W.t()
    if op == "cache":
        amax = s["ssm"].double().abs().amax(-1)
        return {"q": None, "scale": amax / 448, "ssm": None}
    return _exact_step(s, case)


def _grid(fmt):
    """The non-negative values of the code, ascending (an even place has an even mantissa)."""
    if fmt == "mxfp4":
        return _E2M1[:8]
    return [m * 2.0 ** -9 for m in range(8)] + \
        [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)]


def _exact_step(s, case):
    """The step with the state as complex pairs: a rotation is a product with exp(i phi)."""
    o, f64 = s["cache"], torch.float64
    rep = case["H"] // case["G"]
    new = _wrapped(o["angle"], s["theta"])
    pairs = lambda v: torch.view_as_complex(  # noqa: E731
        v.to(f64).unflatten(-1, (-1, 2)).contiguous()).repeat_interleave(rep, 1)
    turn = lambda phi: torch.polar(torch.ones_like(phi), phi)  # noqa: E731
    back = lambda z: torch.view_as_real(z).flatten(-2)  # noqa: E731
    Bb, Cb = back(pairs(s["B"]) * turn(new)), back(pairs(s["C"]) * turn(new))
    x = s["x"].to(f64)
    h = torch.exp(s["logdecay"].to(f64))[..., None, None] * \
        (o["ssm"].view(torch.float8_e4m3fn).to(f64) * o["scale"].to(f64)[..., None])
    h += torch.einsum("bh,bhn,bhp->bhnp", s["gamma"].to(f64), Bb, x)
    if s["beta"] is not None:
        Bp = back(pairs(o["b_prev"]) * turn(o["angle"].to(f64)))
        h += torch.einsum("bh,bhn,bhp->bhnp", s["beta"].to(f64), Bp, o["x_prev"].to(f64))
    y = torch.einsum("bhn,bhnp->bhp", Cb, h)
    if s["D"] is not None:
        y += s["D"].to(f64)[:, None] * x
    amax = h.abs().amax(-1)
    return {"y": y, "angle": new, "scale": amax / 448, "x_prev": None, "b_prev": None, "q": None}


# ---- what a pass cannot do without -------------------------------------------------------

def _mx_bytes(rows, cols, fmt):
    return rows * cols * (0.5 if fmt == "mxfp4" else 1.0) + rows * cols / 32


def work(case):
    op = case["op"]
    esz = {"bf16": 2, "f32": 4, "none": 0}
    if op == "norm":
        n = case["rows"] * case["d"]
        out = n * esz[case["dtype"]] if case["fmt"] == "none" else \
            _mx_bytes(case["rows"], case["d"], case["fmt"])
        return {"bytes": n * (esz[case["dtype"]] + 2 * esz[case["res"]]) + out +
                4 * (case["rows"] + case["d"]), "flops": 6 * n}
    if op == "norm_bwd":
        n = case["rows"] * case["d"]
        return {"bytes": n * (esz[case["dtype"]] + esz[case["res"]] + 4 + 4 * case["dres"]) +
                4 * (case["rows"] + 2 * case["d"]), "flops": 10 * n}
    if op == "mx":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * esz[case["dtype"]] +
                2 * _mx_bytes(case["rows"], case["cols"], case["fmt"]), "flops": 6 * n}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": _mx_bytes(M, K, case["a"]) + _mx_bytes(N, K, "mxfp4") + 2 * M * N,
                "flops": 2 * M * N * K}
    b, H, N, P = (case[k] for k in ("b", "H", "N", "P"))
    if op == "cache":
        return {"bytes": b * H * N * (10 * P + 8), "flops": 5 * b * H * N * P}
    e = esz[case["dtype"]]
    return {"bytes": b * H * (2 * N * P + 8 * N + 4 * N + 2 * N * case["theta"] + 8 * P +
                              2 * e * P + 4 * (2 + case["beta"])) +
            b * case["G"] * N * (2 * e + 8), "flops": 9 * b * H * N * P}
