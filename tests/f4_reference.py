"""Plain numpy statement of the microscaled 4-bit floating-point format and its
operators, in 64 bits: element by element from the definitions in
``include/w4.h``, sharing no code with the CUDA path.  Scales are numbers of
their own types (fp32, e4m3, powers of two), so their roundings are part of the
definition and are made here by rounding exact 64-bit quotients.
"""
from __future__ import annotations

import numpy as np

MX, NV = "mx", "nv"
BLOCK = {MX: 32, NV: 16}
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
NAN_BYTE = {MX: 255, NV: 127}


def e4m3_value(byte):
    byte = np.asarray(byte, np.int64) & 0x7F
    e, f = byte >> 3, byte & 7
    v = np.where(e == 0, f * 2.0 ** -9, (1.0 + f / 8.0) * 2.0 ** (e - 7.0))
    return np.where(byte == 0x7F, np.nan, v)


E4M3 = e4m3_value(np.arange(127))  # 0 .. 448, ascending


def scale_value(byte, fmt):
    byte = np.asarray(byte, np.int64)
    if fmt == MX:
        return np.where(byte == 255, np.nan, np.ldexp(1.0, byte - 127))
    return e4m3_value(byte)


def _nearest(v, grid):
    """Index of the grid value nearest to each v >= 0, ties to the even index,
    the last value for anything beyond it."""
    v = np.minimum(v, grid[-1])
    hi = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo = hi - 1
    down, up = v - grid[lo], grid[hi] - v
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def e2m1_codes(v):
    return (_nearest(np.abs(v), LEVELS) + 8 * np.signbit(v)).astype(np.uint8)


def e2m1_values(codes):
    codes = np.asarray(codes)
    return np.where(codes & 8, -1.0, 1.0) * LEVELS[codes & 7]


def f32(v):
    return np.asarray(v, np.float64).astype(np.float32).astype(np.float64)


def tensor_scale(x):
    a = np.abs(np.asarray(x, np.float64))
    a = a[np.isfinite(a)]
    return max(float(f32((a.max() if a.size else 0.0) / 2688.0)), 2.0 ** -100)


def quantize(x, fmt, g=None):
    """codes [R][K] (one a byte) and row-major scale bytes [R][K / block] of
    float64 values x."""
    R, K = x.shape
    b = x.reshape(R, K // BLOCK[fmt], BLOCK[fmt])
    amax = np.abs(b).max(-1) if b.size else np.zeros(b.shape[:2])
    bad = ~np.isfinite(amax)
    amax = np.where(bad, 0.0, amax)
    b = np.where(bad[..., None], 0.0, b)
    if fmt == MX:
        e = np.where(amax > 0, np.frexp(amax)[1] - 1 - 2, -127)
        e = np.maximum(e, -127)
        scales = (e + 127).astype(np.uint8)
        v = np.ldexp(b, -e[..., None])
    else:
        with np.errstate(over="ignore"):  # quotients beyond fp32 saturate at 448
            s = _nearest(f32(amax / f32(6.0 * g)), E4M3)
        scales = s.astype(np.uint8)
        den = f32(E4M3[s] * g)
        inv = f32(np.divide(1.0, den, out=np.zeros_like(den), where=den != 0))
        with np.errstate(over="ignore"):  # infinity saturates
            v = f32(b * inv[..., None])
    scales = np.where(bad, NAN_BYTE[fmt], scales).astype(np.uint8)
    return e2m1_codes(v).reshape(R, K), scales


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def tile(scales, fmt):
    """Scale tiles [row tiles][tiles along K][512] of row-major scale bytes."""
    R, nb = scales.shape
    out = np.zeros((-(-R // 128), -(-nb // 4), 512), np.uint8)
    for r in range(R):
        for b in range(nb):
            out[r // 128, b // 4, r % 32 * 16 + r % 128 // 32 * 4 + b % 4] = scales[r, b]
    return out


def values(codes, scales, fmt):
    """q * s in 64 bits (exact) from one-a-byte codes and row-major scales."""
    R, K = codes.shape
    s = scale_value(scales, fmt)
    v = e2m1_values(codes).reshape(R, K // BLOCK[fmt], BLOCK[fmt])
    return (v * s[..., None]).reshape(R, K)


def block_amax(x, fmt):
    """Largest magnitude of each element's block, element by element."""
    b = np.abs(x).reshape(x.shape[0], -1, BLOCK[fmt])
    return np.broadcast_to(b.max(-1, keepdims=True), b.shape).reshape(x.shape)


# ---------------------------------------------------------------------------
# error bounds
# ---------------------------------------------------------------------------

def accumulation(K):
    """Largest relative error of an fp32 accumulation on the tensor cores, as a
    factor of the sum of the products' magnitudes.  An MMA adds 64 exact
    products to its accumulator; every one of its ceil(K / 64) steps rounds or
    cuts the running sum, which is never above that sum of magnitudes, by at
    most 2 units of 2^-23 (a cut of the aligned addends and one of the result),
    hence 2^-22 a step.  Eight more such steps cover the joining of K slices
    (at most 7 fp32 additions, 2^-24 each), the factor g (two roundings) and
    the last product's own rounding."""
    return (-(-K // 64) + 8) * 2.0 ** -22


def mm_bound(a, w, K):
    return accumulation(K) * (np.abs(a) @ np.abs(w).T)


def gemv_bound(x, w, K, fmt):
    """f4_gemv: the fixed-point x of a block is off by at most half a unit of
    2^-21 2^E, with 2^E <= the block's largest magnitude (NV: or 2^-17 of the
    token's); its digits -4..3 at 8^0, 8^-1, ... sum to at most 32 / 7 2^E in
    magnitude, which takes the place of |x| in the accumulation; the joining of
    the 8 digit columns adds 7 fp32 steps, counted as two of 2^-22 each."""
    top = block_amax(x, fmt)
    if fmt == NV:
        top = np.maximum(top, np.abs(x).max(-1, keepdims=True) * 2.0 ** -16)
    s = top @ np.abs(w).T
    return (2.0 ** -22 + (32.0 / 7.0) * (accumulation(K) + 2 * 2.0 ** -22)) * s
