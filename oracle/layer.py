"""fp64 oracle of the operators that a layer has around the scan: plain numpy, written
from their definitions (include/m3ssd.h), sharing no code with the library.

The gated linear recurrence walks token by token, forward and in reverse.  The heads' norm with
its rotation is written with complex pairs.  4-bit weights are looked up byte by byte.
"""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def glr_gates(r, i, rate, bias_r=None, bias_i=None, c=8.0, reset=None):
    """rho, iota, log a, a, s of every token; a = 0 and s = 1 at a reset."""
    rho = sigmoid(r + (0 if bias_r is None else bias_r))
    iota = sigmoid(i + (0 if bias_i is None else bias_i))
    la = -c * softplus(rate) * rho
    a, s = np.exp(la), np.sqrt(-np.expm1(2 * la))
    if reset is not None:
        cut = np.asarray(reset, bool)[..., None]
        a, s = np.where(cut, 0.0, a), np.where(cut, 1.0, s)
    return rho, iota, la, a, s


def _lens(lengths, b, L):
    return np.full(b, L) if lengths is None else np.clip(np.asarray(lengths), 0, L)


def glr_fwd(x, r, i, rate, bias_r=None, bias_i=None, c=8.0, h0=None, reset=None, lengths=None):
    """(y, hT) of x, r, i (b, L, D)."""
    b, L, D = x.shape
    _, iota, _, a, s = glr_gates(r, i, rate, bias_r, bias_i, c, reset)
    h = np.zeros((b, D)) if h0 is None else np.array(h0, np.float64)
    n, y = _lens(lengths, b, L), np.zeros((b, L, D))
    for k in range(b):
        for t in range(n[k]):
            u = s[k, t] * iota[k, t] * x[k, t]
            h[k] = u if reset is not None and reset[k, t] else a[k, t] * h[k] + u
            y[k, t] = h[k]
    return y, h


def glr_bwd(x, r, i, rate, y, dy, bias_r=None, bias_i=None, c=8.0, h0=None, reset=None,
            lengths=None, dhT=None):
    """Gradients by the header's formulas, with h_{t-1} = y_{t-1}; also g (b, L, D)."""
    b, L, D = x.shape
    rho, iota, la, a, s = glr_gates(r, i, rate, bias_r, bias_i, c, reset)
    back = np.zeros((b, D)) if dhT is None else np.array(dhT, np.float64)
    n = _lens(lengths, b, L)
    o = {k: np.zeros((b, L, D)) for k in ("dx", "dr", "di", "E", "g")}
    for k in range(b):
        for t in range(n[k] - 1, -1, -1):
            prev = y[k, t - 1] if t > 0 else (0.0 if h0 is None else h0[k])
            g = dy[k, t] + back[k]
            cut = reset is not None and reset[k, t]
            o["g"][k, t] = g
            o["dx"][k, t] = g * s[k, t] * iota[k, t]
            o["di"][k, t] = g * s[k, t] * x[k, t] * iota[k, t] * (1 - iota[k, t])
            if not cut:
                with np.errstate(divide="ignore", invalid="ignore"):
                    slope = np.where(s[k, t] > 0, la[k, t] / s[k, t], 0.0)
                E = g * (a[k, t] * la[k, t] * prev - a[k, t] ** 2 * slope * iota[k, t] * x[k, t])
                o["E"][k, t] = E
                o["dr"][k, t] = E * (1 - rho[k, t])
            back[k] = 0.0 if cut else a[k, t] * g
    # sigma / softplus is 1 - exp(rate) / 2 + ... far down
    slope = np.where(rate < -40, 1.0, sigmoid(rate) / np.maximum(softplus(rate), 1e-300))
    o["drate"] = o["E"].sum((0, 1)) * slope
    o["dbias_r"], o["dbias_i"], o["dh0"] = o["dr"].sum((0, 1)), o["di"].sum((0, 1)), back
    return o


def _turn(positions, freqs, N, sign):
    """exp(i sign angle) of every (token, pair), 1 past the rotated ones; angles in long double."""
    if positions is None:
        return np.ones((1, 1, N // 2))
    rows = len(positions)
    ang = np.asarray(positions, np.longdouble)[:, None] * np.asarray(freqs, np.longdouble)[None]
    whole = 2 * np.longdouble("3.14159265358979323846264338327950288")
    ang = np.asarray(np.remainder(ang, whole), np.float64)
    z = np.ones((rows, 1, N // 2), complex)
    z[:, 0, :ang.shape[1]] = np.exp(1j * sign * ang)
    return z


def _turned(v, z):
    p = v.reshape(*v.shape[:-1], -1, 2)
    c = (p[..., 0] + 1j * p[..., 1]) * z
    return np.stack((c.real, c.imag), -1).reshape(v.shape)


def norm_rotate(u, w, positions, freqs, eps):
    """u (rows, H, N) -> its normed, weighted and rotated heads."""
    v = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)
    return _turned(v, _turn(positions, freqs, u.shape[-1], 1))


def norm_rotate_bwd(u, w, d, positions, freqs, eps):
    """(du, dw) from the gradient d of the output."""
    rstd = 1 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    dv, uh = _turned(d, _turn(positions, freqs, u.shape[-1], -1)), u * rstd
    g = dv * (1.0 if w is None else w)
    return rstd * (g - uh * (g * uh).mean(-1, keepdims=True)), (dv * uh).sum((0, 1))


def w4_codes(tiled, rows, cols):
    """The codes (rows, cols) from the tiled bytes, one at a time by the header's formula."""
    kb = (cols + 127) // 128
    r, k = np.meshgrid(np.arange(rows), np.arange(cols), indexing="ij")
    rr, c = r % 16, k % 128
    j, l, m = c // 32, c % 32 // 8, c % 8 // 2
    byte = (r // 16 * kb + k // 128) * 1024 + 512 * (rr // 8) + 64 * (rr % 8) + 16 * l + 4 * j + m
    v = np.asarray(tiled)[byte]
    return np.where(k % 2 == 0, v & 15, v >> 4)


def w4_weights(codes, scales, zeros, group):
    """Values of codes (rows, cols), scales and zeros (groups, rows; zeros may be None)."""
    j = np.arange(codes.shape[1]) // group
    z = 8.0 if zeros is None else np.asarray(zeros, np.float64)[j].T
    return (codes - z) * np.asarray(scales, np.float64)[j].T


def w4_quant(w, group, zeros, bf16):
    """(codes, scales, zeros) of fp32 weights by the header's rules, in fp32 as it says; ``bf16``
    rounds an fp32 array to bf16."""
    w = np.asarray(w, np.float32)
    rows, cols = w.shape
    n = -(-cols // group)
    codes = np.zeros((rows, cols), np.uint8)
    scales, zs = np.zeros((n, rows), np.float32), np.zeros((n, rows), np.uint8)
    f = np.float32
    for j in range(n):
        v = w[:, j * group:(j + 1) * group]
        ok = np.isfinite(v).all(1)
        v = np.where(ok[:, None], v, f(0))
        lo, hi = np.minimum(v.min(1), f(0)), np.maximum(v.max(1), f(0))
        s = f(2) * ((f(0.5) * hi - f(0.5) * lo) / f(15)) if zeros else np.maximum(hi, -lo) / f(7)
        s = bf16(np.where(ok, s, f("nan")))
        some = s > 0
        d = np.where(some, s, f(1))
        z = np.where(some, np.clip(np.rint(-lo / d), 0, 15), 0) if zeros else np.full(rows, 8.0)
        q = np.where(some[:, None], np.rint(v / d[:, None]), 0) + z[:, None]
        codes[:, j * group:(j + 1) * group] = np.clip(q, 0, 15).astype(np.uint8)
        scales[j], zs[j] = s, z.astype(np.uint8)
    return codes, scales, zs if zeros else None
