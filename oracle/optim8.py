"""AdamW with 8-bit states, dithered rounding (fp32 and integers, bit-exact).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

[rkmt] §3.5 and [czcl] §3.2 train the adapter with AdamW whose states are in
32 or 8 bits.  A state of n elements is kept in blocks of 256 with one fp32
scale: m as E4M3 codes (top 448), v as E5M2 codes (top 57344).  The rounding
to codes is decided by integers, so it is restated here by arithmetic on the
values of the codes, one element at a time in the exact rationals that fp64
holds: q = n / step with step the spacing of the codes at n, code value
floor(q + f) step, f the dither's fraction.  A value that is not finite takes
no part in its block's scale: an m is the NaN code, a v the code of infinity or
NaN.
"""

import numpy as np

BLOCK = 256
FLOOR = np.float32(2.0 ** -100)
C_I, C_T = 0x6A09E667, 0x9E3779B9


def _dither(n, step):
    i = np.arange(n, dtype=np.uint64) % BLOCK
    return (i * np.uint64(C_I) + np.uint64(step * C_T % 2 ** 32)) & np.uint64(0xFFFFFFFF)


def _codes(a, frac, mant, min_exp, bias, most):
    """Codes of fp32 a >= 0 with the dither's fractions frac in [0, 1)."""
    a64 = a.astype(np.float64)
    e = np.maximum(np.frexp(a64)[1] - 1, min_exp)
    step = np.exp2(e.astype(np.float64) - mant)
    k = np.floor(a64 / step + frac)                 # exact: 24 + 21 bits
    v = np.minimum(k * step, most)
    # the code of value v: exponent field and mantissa, subnormals below
    ev = np.maximum(np.frexp(v)[1] - 1, min_exp)
    m = v / np.exp2(ev.astype(np.float64) - mant)   # 0 .. 2^(mant+1) - 1
    normal = m >= 2 ** mant
    code = np.where(normal, (ev + bias) * 2 ** mant + m - 2 ** mant, m)
    return code.astype(np.int64)


def e5m2_values():
    out = np.empty(128)
    for c in range(128):
        e, m = c >> 2, c & 3
        out[c] = m * 2.0 ** -16 if e == 0 else (4 + m) * 2.0 ** (e - 17)
    return out


def _per_block(x, fn):
    return np.array([fn(x[b:b + BLOCK]) for b in range(0, x.size, BLOCK)], dtype=np.float32)


def _scales(x, top):
    a = np.where(np.isfinite(x), np.abs(x), np.float32(0))
    s = _per_block(a, np.max) / np.float32(top)
    return np.maximum(s.astype(np.float32), FLOOR)


def _spread(s, n):
    return np.repeat(s, BLOCK)[:n]


def encode_m(m, step):
    """(codes uint8, scales) of fp32 m."""
    s = _scales(m, 448)
    lost, m = ~np.isfinite(m), np.where(np.isnan(m), np.float32(0), m)
    sign = np.where(m < 0, 0x80, 0)
    m = np.where(lost, np.float32(0), m)
    inv = _spread((np.float32(1) / s).astype(np.float32), m.size)
    n = np.minimum((np.abs(m) * inv).astype(np.float32), np.float32(448))
    frac = (_dither(m.size, step) >> np.uint64(12)).astype(np.float64) / 2.0 ** 20
    # the fraction is added below the last mantissa bit of a 24-bit number, so
    # a subnormal's bits below 2^-20 of its step are cut before the addition
    c = _codes(_cut(n, 3, -6, 20), frac, 3, -6, 7, 448.0)
    return (np.where(lost, 0x7F, c) | sign).astype(np.uint8), s


def encode_v(v, step):
    """(codes uint8, scales) of fp32 v >= 0; a positive v is at least code 1."""
    s = _scales(v, 57344)
    inf, nan = np.isinf(v), np.isnan(v)
    v = np.where(inf | nan, np.float32(0), v)
    inv = _spread((np.float32(1) / s).astype(np.float32), v.size)
    n = np.minimum((v * inv).astype(np.float32), np.float32(57344))
    frac = ((np.uint64(0xFFFFFFFF) - _dither(v.size, step)) >> np.uint64(11)).astype(np.float64)
    c = _codes(_cut(n, 2, -14, 21), frac / 2.0 ** 21, 2, -14, 15, 57344.0)
    c = np.where(v > 0, np.maximum(c, 1), 0)
    return np.where(inf, 0x7C, np.where(nan, 0x7F, c)).astype(np.uint8), s


def _cut(n, mant, min_exp, bits):
    n64 = n.astype(np.float64)
    grid = 2.0 ** (min_exp - mant - bits)
    return np.where(n64 < 2.0 ** min_exp, np.floor(n64 / grid) * grid, n64)


def moments(g, m, v, beta1, beta2):
    """New fp32 m and v, every operation rounded (the bits of the codes hang
    on them); all arguments fp32."""
    f = np.float32
    b1, b2 = f(beta1), f(beta2)
    c1, c2 = f(1.0 - float(b1)), f(1.0 - float(b2))
    m = (b1 * m).astype(f) + (c1 * g).astype(f)
    v = (b2 * v).astype(f) + (c2 * (g * g).astype(f)).astype(f)
    return m.astype(f), v.astype(f)
