"""64-bit reference of the microscaled 4-bit formats and of the 4-bit grouped product,
from the formats' definitions (numpy, shares nothing with the CUDA path)."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"nvfp4": 16, "mxfp4": 32}


def pitch(K, fmt):
    return -(-(K // BLOCK[fmt]) // 16) * 16


def e4m3_values():
    """The value of every e4m3 code (NaN for 0x7F and 0xFF)."""
    c = np.arange(256)
    ex, m = (c >> 3) & 15, c & 7
    v = np.where(ex == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (ex.astype(float) - 7))
    v = np.where(c & 0x7F == 0x7F, np.nan, v)
    return np.where(c >= 128, -v, v)


def e8m0_values():
    v = 2.0 ** (np.arange(256).astype(float) - 127)
    v[255] = np.nan
    return v


SCALES = {"nvfp4": e4m3_values(), "mxfp4": e8m0_values()}


def round_to(x, grid):
    """Index of the nearest grid value (ascending, index 0 even), ties to the even index, saturating."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(grid, x, side="left"), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def scale_codes(amax, fmt, g=1.0):
    """Scale codes of finite block maxima."""
    if fmt == "nvfp4":
        return round_to(amax / (6.0 * g), SCALES["nvfp4"][:127])
    _, ex = np.frexp(np.where(amax == 0, 1.0, amax))        # amax = m 2^ex, m in [0.5, 1)
    return np.where(amax == 0, 0, np.clip(ex - 1 - 2 + 127, 0, 254)).astype(np.int64)


def codes(x, d):
    """e2m1 codes (sign in bit 3) of x over the block scales' values d, both broadcast."""
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(d == 0, 0.0, np.abs(x) / d)
    return round_to(y, E2M1) | (np.signbit(x).astype(np.int64) << 3)


def unpack(packed):
    """uint8 [..., K / 2] -> codes [..., K]."""
    p = np.asarray(packed).astype(np.int64)
    return np.stack([p & 15, p >> 4], -1).reshape(*p.shape[:-1], p.shape[-1] * 2)


def pack(c):
    c = np.asarray(c).astype(np.uint8)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def pad_scales(s, K, fmt, fill=0):
    out = np.full((*s.shape[:-1], pitch(K, fmt)), fill, np.uint8)
    out[..., : s.shape[-1]] = s
    return out


def values(packed, scales, fmt, g=1.0):
    c = unpack(packed)
    K = c.shape[-1]
    q = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = SCALES[fmt][np.asarray(scales)[..., : K // BLOCK[fmt]].astype(np.int64)]
    return q * np.repeat(s, BLOCK[fmt], -1) * g


def random_operand(rng, lead, K, fmt, sigma=1.0):
    """Quantised normal values: (packed, scales)."""
    x = rng.standard_normal((*lead, K)) * sigma
    b = BLOCK[fmt]
    blocks = x.reshape(*lead, K // b, b)
    s = scale_codes(np.abs(blocks).max(-1), fmt)
    d = SCALES[fmt][s]
    return pack(codes(blocks, d[..., None]).reshape(x.shape)), pad_scales(s.astype(np.uint8), K, fmt)


def product(a, a_scales, offsets, b, b_scales, ids, fmt, ga=None, gb=None):
    """(C in 64 bits, sum of magnitudes, active-row mask) of the grouped product."""
    A = values(a, a_scales, fmt, 1.0 if ga is None else float(ga))
    rows, N, E = A.shape[0], b.shape[1], b.shape[0]
    C, S, live = np.zeros((rows, N)), np.zeros((rows, N)), np.zeros(rows, bool)
    for g, e in enumerate(ids):
        r0, r1 = int(offsets[g]), int(offsets[g + 1])
        if 0 <= e < E and r1 > r0:
            W = values(b[e], b_scales[e], fmt, 1.0 if gb is None else float(gb[e]))
            C[r0:r1] = A[r0:r1] @ W.T
            S[r0:r1] = np.abs(A[r0:r1]) @ np.abs(W).T
            live[r0:r1] = True
    return C, S, live
