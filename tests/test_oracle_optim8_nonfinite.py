"""The oracle's codes of optimizer states that are not finite (CPU)."""

import numpy as np
import torch

from oracle import optim8


def value(codes, scales, dtype):
    t = torch.from_numpy(codes).view(dtype).float().numpy()
    return t * np.repeat(scales, 256)[:codes.size]


def test_what_is_not_finite_keeps_its_place_alone():
    rng = np.random.default_rng(0)
    m = rng.standard_normal(700).astype(np.float32)
    v = (m * m).astype(np.float32)
    bad_m, bad_v = m.copy(), v.copy()
    bad_m[[3, 300, 699]] = np.nan, np.inf, -np.inf
    bad_v[[3, 300, 699]] = np.nan, np.inf, np.nan
    m[[3, 300, 699]] = 0
    v[[3, 300, 699]] = 0
    rest = np.ones(700, bool)
    rest[[3, 300, 699]] = False
    for enc, a, b, dtype in ((optim8.encode_m, bad_m, m, torch.float8_e4m3fn),
                             (optim8.encode_v, bad_v, v, torch.float8_e5m2)):
        (ca, sa), (cb, sb) = enc(a, 7), enc(b, 7)
        assert np.array_equal(sa, sb) and np.array_equal(ca[rest], cb[rest])
        got = value(ca, sa, dtype)
        assert not np.isfinite(got[~rest]).any() and np.isfinite(got[rest]).all()
    c, s = optim8.encode_v(bad_v, 7)
    assert np.isinf(value(c, s, torch.float8_e5m2)[300])
    assert np.isnan(value(c, s, torch.float8_e5m2)[[3, 699]]).all()


def test_a_block_of_nothing_finite_has_the_least_scale():
    x = np.full(256, np.nan, np.float32)
    for enc in (optim8.encode_m, optim8.encode_v):
        c, s = enc(x, 1)
        assert s[0] == optim8.FLOOR and np.all(c == 0x7F)
