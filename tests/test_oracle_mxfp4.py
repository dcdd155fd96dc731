"""The oracle of the microscaled 4-bit format against its definition."""

import numpy as np
import pytest

from oracle import fp8, mxfp4


def test_values_are_the_formats():
    v = mxfp4.e2m1_values()
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        want = m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
        assert v[c] == (-want if c & 8 else want)


def test_scale_bytes_in_exact_rationals():
    rng = np.random.default_rng(0)
    a = np.concatenate([np.exp2(rng.uniform(-149, 127, 300)), [1.75, np.nextafter(1.75, 0), 7, 6,
                        448, 2.0 ** -149, 2.0 ** -125, 3.4e38, 0]]).astype(np.float32)
    got = mxfp4._scale_bytes(a.astype(np.float64), mxfp4.E2M1, 8.0)
    assert got.tolist() == [mxfp4.exact_scale_byte(x) for x in a]


def test_nearest_code_of_every_border():
    """Midpoints go to the even code, their neighbours to the nearer one."""
    pos = mxfp4.E2M1
    for i, m in enumerate((pos[1:] + pos[:-1]) / 2):
        x = np.zeros((3, 32), np.float32)
        x[:, 0] = 6
        x[:, 1] = [m, np.nextafter(np.float32(m), np.float32(0)),
                   np.nextafter(np.float32(m), np.float32(8))]
        c, b = mxfp4.quantize(x)
        assert (b == 127).all()
        assert c[:, 1].tolist() == [i + (i & 1), i, i + 1]


def test_rows_of_gradients_keep_three_mantissa_bits():
    x = np.zeros((4, 40), np.float32)
    x[0, 0], x[1, 0], x[2, 39], x[3, 3] = 464, 465, -448, 1.0
    v = mxfp4.row_values8(x)
    assert v[0, 0] == 448 and v[1, 0] == 480 and v[2, 39] == -448 and v[3, 3] == 1.0
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 70)).astype(np.float32)
    v = mxfp4.row_values8(x)
    big = np.repeat(mxfp4._amax(x), 32, axis=1)[:, :70]
    # half a step of the number, or of the least exponent, 2^-6 of a scale that
    # is at most amax / 232
    assert (np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, big / 232 * 2.0 ** -10)).all()


def test_groups_that_are_not_finite_and_empty_ones():
    x = np.zeros((3, 64), np.float32)
    x[0, 3], x[1, 40] = np.nan, -np.inf
    _, b = mxfp4.quantize(x)
    assert b.tolist() == [[255, 0], [0, 255], [0, 0]]


def test_tiles_hold_every_byte_once():
    rng = np.random.default_rng(2)
    R, K = 70, 544
    byte = rng.integers(1, 255, (R, K // 32)).astype(np.uint8)
    t = mxfp4.tiles(byte, R, K)
    assert t.size == 3 * 3 * 256
    assert np.array_equal(np.sort(t[t > 0]), np.sort(byte.reshape(-1)))


@pytest.mark.parametrize("spread", [26, 27, 60])
def test_turned_values_drop_what_lies_far_below(spread):
    v, byte = np.ones((32, 32)), np.full((32, 1), 100, np.uint8)
    byte[5] = 100 - spread
    got = mxfp4.turned_values(v, byte)
    assert (got[5] == (1 if spread <= 26 else 0)).all() and (got[6] == 1).all()


def test_e4m3_border_is_the_tie_between_448_and_480():
    pos = fp8.e4m3_values()[:0x7F]
    assert pos[-1] == 448 and (len(pos) - 1) % 2 == 0
