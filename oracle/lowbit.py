"""fp64 oracle of the low-bit and normalisation operators: plain numpy, written
from their definitions (include/m3ssd.h), sharing no code with the library.

MX tensors: blocks of 32 along the last axis, the least power-of-two scale with
amax <= maxval 2^E, codes rounded to nearest even by looking a value up in the
sorted list of representable ones.  The 8-bit state: E4M3 codes and a scale per
row, s = amax / 448.
"""
from __future__ import annotations

import numpy as np

from . import oracle_step

# Non-negative values by code; a code with an even number has an even mantissa.
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)
                 if (e, m) != (15, 7)])
GRID = {"mxfp4": E2M1, "mxfp8": E4M3}


def round_to_grid(v, grid):
    """Codes (indices into grid) of |v| rounded to nearest, ties to the even code,
    values past the end to the last one."""
    a = np.minimum(np.abs(v), grid[-1])
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - a, a - grid[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def pad(n, m=128):
    return (n + m - 1) // m * m


def mx_encode(x, fmt):
    """(rows, cols) -> (code bytes with the sign bit, unpacked (rows, Kp); scale bytes
    (rows, Kp / 32))."""
    rows, cols = x.shape
    grid = GRID[fmt]
    xp = np.zeros((rows, pad(cols)))
    xp[:, :cols] = x
    blk = xp.reshape(rows, -1, 32)
    bad = ~np.isfinite(blk).all(-1)
    blk = np.where(bad[..., None], 0.0, blk)
    amax = np.abs(blk).max(-1)
    E = np.full(amax.shape, -127)
    for e in range(-127, 128):  # the least E that fits (written out; no logarithm)
        E = np.where((amax > grid[-1] * 2.0 ** (e - 1)) & (e > -127), e, E)
    idx = round_to_grid(blk / 2.0 ** E[..., None].astype(np.float64), grid)
    sign = np.signbit(blk)
    codes = idx | (sign * (8 if fmt == "mxfp4" else 128))
    codes = np.where(bad[..., None], 0, codes)
    return codes.reshape(rows, -1).astype(np.uint8), np.where(bad, 255, E + 127).astype(np.uint8)


def mx_store(codes, scales, fmt):
    """Unpacked codes and (rows, blocks) scale bytes as they are stored."""
    rows, nb = scales.shape
    if fmt == "mxfp4":
        codes = codes[:, 0::2] | (codes[:, 1::2] << 4)
    tiles = np.zeros(pad(rows) * nb, np.uint8)
    r, k = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    at = ((r // 128) * (nb // 4) + k // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + k % 4
    tiles[at] = scales
    return codes, tiles


def mx_load(codes, tiles, rows, cols, fmt):
    """Stored codes and scale tiles -> fp64 values (rows, cols)."""
    nb = pad(cols) // 32
    r, k = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    at = ((r // 128) * (nb // 4) + k // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + k % 4
    b = tiles[at]
    scale = np.where(b == 255, np.nan, 2.0 ** (b.astype(np.float64) - 127))
    if fmt == "mxfp4":
        full = np.empty((rows, 2 * codes.shape[1]), np.uint8)
        full[:, 0::2], full[:, 1::2] = codes & 15, codes >> 4
        v = np.where(full & 8, -1.0, 1.0) * E2M1[full & 7]
    else:
        grid = np.append(E4M3, np.nan)
        v = np.where(codes & 128, -1.0, 1.0) * grid[codes & 127]
    return (v.reshape(rows, nb, 32) * scale[..., None]).reshape(rows, -1)[:, :cols]


def rmsnorm(r, w, eps):
    """(y, rstd) of rows r."""
    rstd = 1.0 / np.sqrt((r ** 2).sum(-1) / r.shape[-1] + eps)
    return r * rstd[:, None] * w, rstd


def rmsnorm_bwd(dy, r, w, rstd, dres=None):
    """(dr, dw); the mean over a row written as a sum over its elements."""
    d = r.shape[-1]
    g = dy * w
    dot = (g * r).sum(-1)
    dr = rstd[:, None] * g - (rstd ** 3 * dot / d)[:, None] * r
    if dres is not None:
        dr = dr + dres
    return dr, (dy * r * rstd[:, None]).sum(0)


def state_encode(h):
    """State rows (..., P) -> (code bytes, scales)."""
    amax = np.abs(h).max(-1)
    scale = np.where(amax >= 2.0 ** -100, amax / 448.0, 0.0)
    inv = np.where(scale > 0, 1.0 / np.where(scale > 0, scale, 1.0), 0.0)
    v = h * inv[..., None]
    return (round_to_grid(v, E4M3) | (np.signbit(v) * 128)).astype(np.uint8), scale


def state_decode(codes, scale):
    v = np.where(codes & 128, -1.0, 1.0) * np.append(E4M3, np.nan)[codes & 127]
    return v * scale[..., None]


def step_q8(cache, *args):
    """A step on the cache {angle, ssm codes, scale, x_prev, b_prev}: the fp64 step on
    the state the codes stand for.  Returns (y, the fp64 cache after it, unrounded)."""
    c = {k: np.array(cache[k], dtype=np.float64) for k in ("angle", "x_prev", "b_prev")}
    c["ssm"] = state_decode(cache["ssm"], np.asarray(cache["scale"], dtype=np.float64))
    return oracle_step(c, *args), c
