"""Pins of the FP8 oracle and of the 8-bit optimizer states' oracle (CPU):
the code tables against torch's float8 types, rounding against torch's
conversion, the dither's mean."""

import numpy as np
import torch

from oracle import fp8, optim8


def test_e4m3_values_are_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, fp8.e4m3_values(), equal_nan=True)


def test_e5m2_values_are_torchs():
    t = torch.arange(124, dtype=torch.uint8).view(torch.float8_e5m2).double().numpy()
    assert np.array_equal(t, optim8.e5m2_values()[:124])


def test_codes_are_torchs_rounding():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.standard_normal(20000) * 2.0 ** rng.integers(-14, 8, 20000),
                        fp8.e4m3_values()[:0x7F],
                        (fp8.e4m3_values()[:0x7E] + fp8.e4m3_values()[1:0x7F]) / 2])
    v = np.clip(np.concatenate([v, -v]), -448, 448).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.e4m3_codes(v), want)


def test_quantised_values_are_within_half_a_step():
    rng = np.random.default_rng(1)
    w = (rng.standard_normal((144, 272)) * 0.02).astype(np.float32)
    codes, s = fp8.quantize_blocks(w)
    assert s.shape == (2, 3)
    val = fp8.weight_values(codes, s)
    full = fp8.block_scales(s, 144, 272)
    # half a step: 2^-4 of the value, or half of a subnormal step 2^-9 scale
    assert np.all(np.abs(val - w) <= np.maximum(np.abs(w) * 2.0 ** -4, full * 2.0 ** -10) * 1.001)
    codes_r, sr = fp8.quantize_rows(w)
    assert sr.shape == (3, 144)
    assert np.all(np.abs(fp8.row_values(codes_r, sr) - w) <= np.abs(w).max() * 2.0 ** -4)


def test_zero_blocks_have_a_positive_scale():
    codes, s = fp8.quantize_blocks(np.zeros((16, 16), np.float32))
    assert not codes.any() and s[0, 0] == np.float32(2.0 ** -100)


def test_dithered_codes_follow_the_value_on_average():
    # a value between two codes: the mean over 256 elements x 64 steps of the
    # decoded values is the value to 1% of a code's step
    for enc, vals, top, x in ((optim8.encode_m, fp8.e4m3_values(), 448.0, 100.3),
                              (optim8.encode_v, optim8.e5m2_values(), 57344.0, 9000.7)):
        a = np.full(256, x, np.float32)
        a[0] = top                                  # fixes the scale at 1
        got = []
        for t in range(1, 65):
            c, s = enc(a, t)
            assert s[0] == 1.0 and c[0] == (0x7E if top == 448.0 else 0x7B)
            got.append(vals[c[1:]])
        step = 8.0 if top == 448.0 else 2048.0
        assert abs(np.mean(got) - x) <= 0.01 * step
        assert set(np.unique(got)) == {np.floor(x / step) * step, np.ceil(x / step) * step}


def test_smallest_positive_v_keeps_code_one():
    v = np.zeros(256, np.float32)
    v[0], v[1] = 1.0, 1e-30
    c, _ = optim8.encode_v(v, 5)
    assert c[1] == 1 and c[2] == 0


def test_a_group_that_is_not_finite_has_no_scale():
    x = np.ones((3, 300), np.float32)
    x[0, 130], x[1, 0], x[2, 299] = np.nan, -np.inf, np.inf
    _, s = fp8.quantize_rows(x)
    bad = np.zeros((3, 3), bool)
    bad[1, 0] = bad[0, 1] = bad[2, 2] = True
    assert np.array_equal(np.isnan(s), bad)
    assert np.isnan(fp8.quantize_blocks(x)[1]).all()
