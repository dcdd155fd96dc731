"""Block-scaled FP8 weights and rows, and their products, in fp64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

E4M3: 1 sign, 4 exponent bits (bias 7), 3 mantissa bits, no infinities, NaN
at 0x7F and 0xFF, largest value 448.  One fp32 scale per 128 columns of a row
or per 128 x 128 block: fl32(max|x| / 448), at least 2^-100; the code is the
one nearest to fl32(x / scale), ties to the even code.
"""

import numpy as np

BLOCK = 128
FLOOR = np.float32(2.0 ** -100)


def e4m3_values():
    """fp64 value of each of the 256 codes (NaN at 0x7F, 0xFF)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = np.nan if c & 0x7F == 0x7F else v
        if c & 0x80:
            out[c] = -out[c]
    return out


def e4m3_codes(v):
    """Nearest code of fp32 values in [-448, 448], ties to the even code."""
    pos = e4m3_values()[:0x7F]                 # ascending, codes 0 .. 0x7E
    a = np.abs(v.astype(np.float64))
    hi = np.clip(np.searchsorted(pos, a), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dh, dl = pos[hi] - a, a - pos[lo]
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    pick = np.where(pos[hi] == a, hi, pick)
    return (pick | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def group_scale(amax):
    """NaN where a group has an infinity or NaN: its codes mean nothing."""
    s = np.maximum((amax.astype(np.float32) / np.float32(448)).astype(np.float32), FLOOR)
    return np.where(np.isfinite(amax), s, np.float32(np.nan)).astype(np.float32)


def _codes(x, s):
    v = (x.astype(np.float32) / s).astype(np.float32)
    return e4m3_codes(np.clip(v, np.float32(-448), np.float32(448)))


def _amax_columns(x):
    """Max |x| over runs of 128 columns: [rows, ceil(cols / 128)]."""
    n = -(-x.shape[1] // BLOCK)
    return np.stack([np.abs(x[:, b * BLOCK:(b + 1) * BLOCK]).max(axis=1) for b in range(n)], 1)


def quantize_rows(x):
    """(codes uint8 [M, K], scale fp32 [ceil(K/128), M]) of fp32 x [M, K]."""
    s = group_scale(_amax_columns(x))
    full = np.repeat(s, BLOCK, axis=1)[:, :x.shape[1]]
    return _codes(x, full), np.ascontiguousarray(s.T)


def quantize_blocks(w):
    """(codes uint8 [N, K], scale fp32 [ceil(N/128), ceil(K/128)])."""
    col = _amax_columns(w)
    s = group_scale(_amax_columns(np.ascontiguousarray(col.T)).T)
    return _codes(w, block_scales(s, *w.shape)), s


def block_scales(s, N, K):
    return np.repeat(np.repeat(s, BLOCK, axis=0), BLOCK, axis=1)[:N, :K]


def weight_values(codes, s):
    """fp64 values of a weight (exact products of codes and fp32 scales)."""
    return e4m3_values()[codes] * block_scales(s, *codes.shape).astype(np.float64)


def row_values(codes, s):
    return e4m3_values()[codes] * np.repeat(s.T.astype(np.float64), BLOCK, 1)[:, :codes.shape[1]]
