"""64-bit reference of the 8-bit quantisers and of the weight gradient, from the formats'
definitions (numpy, shares nothing with the CUDA path)."""
from __future__ import annotations

import numpy as np

from tests.fp4_util import e4m3_values, e8m0_values, round_to

BLOCK = 128
E4M3 = e4m3_values()
E8M0 = e8m0_values()
GRID = E4M3[:127]           # the codes without a sign, ascending


def pitch(rows, groups):
    return (rows // BLOCK + groups) * BLOCK


def scale_of(amax, pow2):
    """fp32 scale of blocks with the largest magnitudes `amax` (fp32 values): amax / 448 rounded to fp32, or
    the smallest power of two from 2^-127 up that is at least that; NaN for what is not finite."""
    amax = np.asarray(amax, np.float32)
    fine = np.where(np.isfinite(amax), amax, 1).astype(np.float32)
    if pow2:
        m, ex = np.frexp(fine.astype(np.float64) / 448.0)           # m in [0.5, 1)
        s = np.ldexp(1.0, np.maximum(np.where(m == 0.5, ex - 1, ex), -127))
    else:
        s = (fine / np.float32(448)).astype(np.float64)
    return np.where(np.isfinite(amax), np.where(amax == 0, 0.0, s), np.nan)


def codes(x, s):
    """e4m3 codes of fp32 values x over scales s, the quotient rounded to fp32 first; zero codes for s of 0 or NaN."""
    x, s = np.broadcast_arrays(np.asarray(x, np.float32), np.asarray(s, np.float64))
    ok = np.isfinite(s) & (s > 0)
    with np.errstate(over="ignore", under="ignore"):
        y = (np.where(ok, x, 0).astype(np.float64) / np.where(ok, s, 1.0)).astype(np.float32).astype(np.float64)
    c = round_to(np.minimum(np.abs(y), 448.0), GRID)
    return np.where(ok, c | (np.signbit(y).astype(np.int64) << 7), 0).astype(np.uint8)


def blocks_of(x, axis):
    """x padded with zeros along `axis` to whole blocks, that axis split in two."""
    n = x.shape[axis]
    pad = [(0, 0)] * x.ndim
    pad[axis] = (0, -n % BLOCK)
    y = np.pad(x, pad)
    return y.reshape(*x.shape[:axis], -1, BLOCK, *x.shape[axis + 1:])


def amax_of(b, axis):
    with np.errstate(invalid="ignore"):
        return np.max(np.abs(b), axis=axis)      # NaN wins


def rows(x, pow2):
    """(codes, scales) of x [rows, K], a scale for each 128 of a row."""
    b = blocks_of(np.asarray(x, np.float32), 1)
    s = scale_of(amax_of(b, 2), pow2)
    return codes(b, s[:, :, None]).reshape(x.shape[0], -1)[:, :x.shape[1]], s


def tiles(w, pow2):
    """(codes, scales) of w [E, N, K], a scale for each 128 x 128."""
    w = np.asarray(w, np.float32)
    b = blocks_of(blocks_of(w, 1), 3)
    s = scale_of(amax_of(amax_of(b, 4), 2), pow2)
    c = codes(b, s[:, :, None, :, None])
    return c.reshape(w.shape[0], c.shape[1] * BLOCK, -1)[:, :w.shape[1], :w.shape[2]], s


def cols(x, offsets, n_rows, q_t, t_scales):
    """(q_t, t_scales) of x [n_rows, width] along each group's rows, written over what is given."""
    x = np.asarray(x, np.float32)
    q_t, t_scales = q_t.copy(), t_scales.copy()
    for g in range(len(offsets) - 1):
        r0, r1 = int(offsets[g]), int(offsets[g + 1])
        if r1 == r0:
            continue
        at = r0 // BLOCK + g
        b = blocks_of(x[r0:r1], 0)
        s = scale_of(amax_of(b, 1), True)
        c = codes(b, s[:, None, :])
        n = b.shape[0]
        q_t[:, at * BLOCK:(at + n) * BLOCK] = c.reshape(n * BLOCK, -1).T
        t_scales[at:at + n] = np.where(np.isnan(s), 255, np.where(s == 0, 0, np.log2(np.where(s > 0, s, 1.0)) + 127)).astype(np.uint8)
    return q_t, t_scales


def decode_cols(q_t, t_scales):
    """The values that transposed codes and their exponent codes stand for, in 64 bits."""
    return E4M3[q_t] * np.repeat(E8M0[t_scales].T, BLOCK, axis=1)


def weight_grad(d_t, d_scales, a_t, a_scales, offsets):
    """(gradient, sum of the products' magnitudes) [G, N, K] in 64 bits."""
    d, a = decode_cols(d_t, d_scales), decode_cols(a_t, a_scales)
    G = len(offsets) - 1
    out, mag = np.zeros((G, d.shape[0], a.shape[0])), np.zeros((G, d.shape[0], a.shape[0]))
    for g in range(G):
        r0, r1 = int(offsets[g]), int(offsets[g + 1])
        c = (r0 // BLOCK + g) * BLOCK
        cut = slice(c, c + r1 - r0)
        out[g] = d[:, cut] @ a[:, cut].T
        mag[g] = np.abs(d[:, cut]) @ np.abs(a[:, cut]).T
    return out, mag
