"""CPU float64 definitions of the block-scaled formats: E4M3 with a power-of-two scale for each 32
values of a row, and E2M1 as mxfp4 (a power of two for each 32) or nvfp4 (an E4M3 scale for each
16, and a power of two for the row). Written from the formats; test infrastructure only."""
from __future__ import annotations

import math

import numpy as np


def grid(mantissa_bits: int, lowest: int, count: int) -> np.ndarray:
    """The first `count` non-negative values of a format; value k has code k. Codes below
    2^mantissa_bits are subnormal, with the exponent `lowest`."""
    out = []
    for k in range(count):
        e, m = divmod(k, 2 ** mantissa_bits)
        significand = m if e == 0 else 2 ** mantissa_bits + m
        out.append(math.ldexp(significand, lowest + max(e - 1, 0) - mantissa_bits))
    return np.array(out)


E4M3 = grid(3, -6, 127)   # up to 448; 127 is NaN
E2M1 = grid(1, 0, 8)      # 0 0.5 1 1.5 2 3 4 6


def nearest_code(x, values) -> np.ndarray:
    """The code of the value nearest to |x|; halfway, the even code."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    mid = (values[1:] + values[:-1]) / 2
    low, high = np.searchsorted(mid, a, "left"), np.searchsorted(mid, a, "right")
    return np.where(low % 2 == 0, low, high)


def power_of_two(amax: float, most: float) -> int:
    """The smallest e >= -127 with amax <= most 2^e."""
    e = -127
    while amax > most * math.ldexp(1.0, e):
        e += max(1, int(math.log2(amax / (most * math.ldexp(1.0, e)))))   # never past the smallest
    return e


def _blocks(row, size):
    for i in range(0, len(row), size):
        yield i, row[i:i + size]


def pack_e4m3(x):
    """(codes with the sign in bit 7 [N, D], scale bytes [N, blocks], values [N, D])."""
    x = np.asarray(x, dtype=np.float64)
    N, D = x.shape
    codes, values = np.zeros((N, D), np.uint8), np.zeros((N, D))
    scales = np.zeros((N, -(-D // 32)), np.uint8)
    for r in range(N):
        for i, b in _blocks(x[r], 32):
            amax = np.max(np.abs(b)) if np.isfinite(b).all() else np.inf
            if not np.isfinite(amax):
                codes[r, i:i + 32], scales[r, i // 32], values[r, i:i + 32] = 0x7F, 255, np.nan
                continue
            e = power_of_two(amax, 448.0)
            q = nearest_code(b / math.ldexp(1.0, e), E4M3)
            codes[r, i:i + 32] = q | np.where(np.signbit(b), 0x80, 0)
            scales[r, i // 32] = e + 127
            values[r, i:i + 32] = np.copysign(E4M3[q] * math.ldexp(1.0, e), b)
    return codes, scales, values


def quantize_fp4(x, fmt):
    """(codes with the sign in bit 3 [N, D], scale bytes [N, blocks], row scales [N], values [N, D]).
    mxfp4: bytes e + 127; nvfp4: E4M3 codes. A block with an infinity or a NaN has the
    format's NaN for a scale and codes 0."""
    x = np.asarray(x, dtype=np.float64)
    N, D = x.shape
    size = 16 if fmt == "nvfp4" else 32
    codes, values = np.zeros((N, D), np.uint8), np.zeros((N, D))
    scales, rows = np.zeros((N, -(-D // size)), np.uint8), np.ones(N)
    for r in range(N):
        if fmt == "nvfp4":
            finite = np.abs(x[r][np.isfinite(x[r])])
            top = finite.max() if finite.size else 0.0
            rows[r] = math.ldexp(1.0, max(power_of_two(top, 2688.0), -126)) if top > 0 else 1.0
        for i, b in _blocks(x[r], size):
            if not np.isfinite(b).all():
                scales[r, i // size], values[r, i:i + size] = 0x7F if fmt == "nvfp4" else 255, np.nan
                continue
            amax = np.max(np.abs(b))
            if fmt == "nvfp4":
                s = int(nearest_code(amax / 6.0 / rows[r], E4M3))
                scale = E4M3[s] * rows[r]
            else:
                s = power_of_two(amax, 6.0) + 127
                scale = math.ldexp(1.0, s - 127)
            q = nearest_code(b / scale, E2M1) if scale > 0 else np.zeros(len(b), np.int64)
            codes[r, i:i + size] = q | np.where(np.signbit(b), 8, 0)
            scales[r, i // size] = s
            values[r, i:i + size] = np.copysign(E2M1[q] * scale, b)
    return codes, scales, rows, values
