"""Microscaled 4-bit matrices, and the rows that their products take, in fp64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

32 consecutive values of a row share one power of two 2^(byte - 127), byte 255
meaning NaN.  E2M1: 1 sign, 2 exponent bits (bias 1), 1 mantissa bit: 0, 0.5,
1, 1.5, 2, 3, 4, 6.  The power is the least one, from 2^-127, for which the
group's largest magnitude rounds to the largest code or less.  Gradients take
E4M3 codes (largest 448) by the same rule.
"""

from fractions import Fraction

import numpy as np

from oracle import fp8

GROUP = 32
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def e2m1_values():
    """fp64 value of each of the 16 codes."""
    return np.concatenate([E2M1, -E2M1])


def _nearest(pos, a):
    """Index of the number of pos nearest to a >= 0, ties to the even index,
    the last one for all above it."""
    hi = np.clip(np.searchsorted(pos, a), 0, len(pos) - 1)
    lo = np.maximum(hi - 1, 0)
    dh, dl = np.abs(pos[hi] - a), np.abs(a - pos[lo])
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def _scale_bytes(amax, pos, following):
    """The least byte whose power times the border between the largest number
    and the one that would follow is not reached (a tie goes to the even one of
    the two)."""
    top, border = pos[-1], (pos[-1] + following) / 2
    even = len(pos) % 2 == 1                 # the largest number's index is even
    out = np.full(amax.shape, 255, np.uint8)
    ok = np.isfinite(amax)
    a = np.where(ok, amax, 0).astype(np.float64)
    e = np.maximum(np.frexp(a / top)[1] - 3, -127)
    for _ in range(6):                       # from two powers too low upwards
        q = np.ldexp(a, -e)
        e = np.where((q > border) | ((q == border) & (not even)), e + 1, e)
    out[ok] = (np.where(a > 0, np.maximum(e, -127), -127) + 127)[ok]
    return out


def _amax(x):
    n = -(-x.shape[1] // GROUP)
    p = np.zeros((x.shape[0], n * GROUP))
    p[:, :x.shape[1]] = np.abs(x)
    return p.reshape(x.shape[0], n, GROUP).max(axis=2)


def powers(byte):
    return np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))


def _spread(byte, cols):
    return np.repeat(byte, GROUP, axis=1)[:, :cols]


def quantize(x):
    """(codes uint8 [R, K], a byte each; scale bytes [R, K / 32]) of fp32 x."""
    x = x.astype(np.float64)
    byte = _scale_bytes(_amax(x), E2M1, 8.0)
    q = np.abs(x) / powers(_spread(byte, x.shape[1]))
    codes = _nearest(E2M1, np.nan_to_num(q, nan=0.0, posinf=0.0))
    return (codes | np.where(np.signbit(x), 8, 0)).astype(np.uint8), byte


def values(codes, byte):
    return e2m1_values()[codes] * powers(_spread(byte, codes.shape[1]))


def pack(codes):
    return codes[:, 0::2] | codes[:, 1::2] << 4


def tiles(byte, R, K):
    """Scale bytes [R, K / 32] in the library's order, padding 0."""
    out = np.zeros((-(-K // 256), -(-R // 32), 256), np.uint8)
    for r in range(R):
        for g in range(K // GROUP):
            out[g // 8, r // 32, 4 * (16 * (g % 4) + r % 16) + 2 * (r // 16 % 2) + g // 4 % 2] = \
                byte[r, g]
    return out.reshape(-1)


def row_values8(x):
    """fp64 values of rows in E4M3 codes with one power of two per 32 columns."""
    x = x.astype(np.float64)
    pos = fp8.e4m3_values()[:0x7F]
    byte = _scale_bytes(_amax(x), pos, 480.0)
    s = powers(_spread(byte, x.shape[1]))
    v = pos[_nearest(pos, np.nan_to_num(np.abs(x) / s, nan=0.0, posinf=0.0))]
    return np.where(np.signbit(x), -v, v) * s


def turned_values(v, byte):
    """What the backward reads of a weight's values v [N, K]: those whose
    scale lies more than 2^26 below the largest of its 32 rows are 0."""
    v = v.copy()
    full = _spread(byte, v.shape[1]).astype(int)
    for n in range(0, v.shape[0], GROUP):
        b = full[n:n + GROUP]
        base = np.maximum(b.max(axis=0) - 13, 0)
        v[n:n + GROUP][b - base < -13] = 0
    return v


def exact_scale_byte(amax):
    """The scale byte of one finite E2M1 group from its definition, in exact
    rationals."""
    a = Fraction(float(amax))
    for byte in range(255):
        if a < 7 * Fraction(2) ** (byte - 127):
            return byte
    raise ValueError(amax)
