"""Values that are not finite in the 8-bit optimizer states (GPU).

States in 8 bits keep what 32-bit states keep, as far as their formats can:
an m that is not finite is E4M3's NaN, a v is E5M2's infinity or NaN, the
block's scales are those of its finite elements, and no other element of the
block is touched.  Codes and scales must be the oracle's bit for bit.
"""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_22_amd as qn
from oracle import optim8
from tests.test_gpu_adamw_multi import B1, B2, HYPER, bits32, check, make, table_of, upload

pytestmark = pytest.mark.gpu

# element -> gradient: a NaN, infinities, a finite gradient whose square is
# none, two in one block, the last of a partial block
BAD = {5: np.nan, 300: np.inf, 301: -np.inf, 700: 1e30, 1100: np.nan, 1101: -1e25, 2999: np.nan}
N = 3000


def after(bits, bad, steps=(4,)):
    state = make([N], bits, steps[0], False, seed=6)
    for i, v in bad.items():
        state[0]["g"][i] = v
    t = upload(state, bits, False)
    tab = table_of(t, bits)
    for step in steps:
        qn.lora_adamw_multi_step(tab, step, **HYPER)
    torch.cuda.synchronize()
    return state[0], t[0]


def decoded(e, k):
    return e[k].float().cpu().numpy() * np.repeat(e[k + "s"].cpu().numpy(), 256)[:N]


@pytest.mark.parametrize("whole_block", [False, True])
def test_codes_and_scales_are_the_oracles(whole_block):
    bad = dict(BAD)
    if whole_block:
        bad.update({i: np.nan for i in range(512, 768)})
    d, t = after(8, bad)
    with np.errstate(all="ignore"):
        m, v = optim8.moments(d["g"], d["m"], d["v"], B1, B2)
    for x, s, enc, y in ((t["m"], t["ms"], optim8.encode_m, m),
                         (t["v"], t["vs"], optim8.encode_v, v)):
        codes, scales = enc(y, 4)
        assert np.array_equal(bits32(s.cpu().numpy()), bits32(scales))
        assert np.array_equal(x.view(torch.uint8).cpu().numpy(), codes)


def test_what_is_kept_is_what_32_bit_states_keep():
    _, wide = after(32, BAD)
    _, t = after(8, BAD)
    for k in ("m", "v"):
        want, got = wide[k].cpu().numpy(), decoded(t, k)
        assert np.array_equal(np.isfinite(got), np.isfinite(want))
    assert np.array_equal(np.isinf(decoded(t, "v")), np.isinf(wide["v"].cpu().numpy()))
    p, pw = (e["p"].cpu().numpy() for e in (t, wide))
    assert np.array_equal(np.isfinite(p), np.isfinite(pw))


def test_elements_beside_them_step_on():
    """A second step of all other elements is the oracle's step from their
    states, with the bits of a run without the bad gradients outside the
    blocks that had them."""
    _, clean = after(8, {}, (4, 5))
    _, t = after(8, BAD, (4, 5))
    ok = np.ones(N, bool)
    ok[list(BAD)] = False
    assert np.all(np.isfinite(t["p"].cpu().numpy()[ok]))
    assert np.all(np.isfinite(decoded(t, "m")[ok])) and np.all(np.isfinite(decoded(t, "v")[ok]))
    outside = np.ones(N, bool)
    for i in BAD:
        outside[i // 256 * 256:(i // 256 + 1) * 256] = False
    for k in ("p", "b", "m", "v"):
        a, b = (e[k].view(torch.uint8).view(N, -1).cpu().numpy() for e in (t, clean))
        assert np.array_equal(a[outside], b[outside])


def test_a_restored_parameter_is_told_of_its_states():
    """p put back, the states kept: the next step of a lost element says so
    again, as it does with 32-bit states, and does not move p by the block's
    largest m."""
    for bits in (32, 8):
        state = make([N], bits, 4, False, seed=6)
        p0 = state[0]["p"].copy()
        state[0]["g"][5] = np.nan
        t = upload(state, bits, False)
        tab = table_of(t, bits)
        qn.lora_adamw_multi_step(tab, 4, **HYPER)
        t[0]["p"].copy_(torch.from_numpy(p0))
        t[0]["g"].fill_(1e-6)
        qn.lora_adamw_multi_step(tab, 5, **HYPER)
        torch.cuda.synchronize()
        p = t[0]["p"].cpu().numpy()
        assert np.isnan(p[5]) and np.isfinite(np.delete(p, 5)).all()


def test_a_step_after_it_is_the_oracles_for_the_others():
    """The states that a step with a NaN left, decoded, taken as a start."""
    d, t = after(8, {40: np.nan})
    keep = np.arange(N) != 40
    m, v = decoded(t, "m").astype(np.float32), decoded(t, "v").astype(np.float32)
    assert np.isnan(m[40]) and np.isnan(v[40])
    # the same states with zeros in the place of the lost element
    mc, vc = (t[k].view(torch.uint8).cpu().numpy().copy() for k in ("m", "v"))
    mc[40] = vc[40] = 0
    m[40] = v[40] = 0
    rng = np.random.default_rng(3)
    g = (rng.standard_normal(N) * 1e-4).astype(np.float32)
    g[40] = 0
    p = t["p"].cpu().numpy().copy()
    p[40] = 0
    start = {"p": p, "g": g, "m": m, "v": v, "mc": mc, "vc": vc,
             "ms": t["ms"].cpu().numpy(), "vs": t["vs"].cpu().numpy()}
    a = upload([start], 8, False)
    qn.lora_adamw_multi_step(table_of(a, 8), 5, **HYPER)
    torch.cuda.synchronize()
    check([start], a, 8, 5)
    t["g"].copy_(torch.from_numpy(g))
    qn.lora_adamw_multi_step(table_of([t], 8), 5, **HYPER)
    torch.cuda.synchronize()
    for k in ("p", "m", "v"):
        x, y = (e[k].view(torch.uint8).view(N, -1).cpu().numpy() for e in (t, a[0]))
        assert np.array_equal(x[keep], y[keep])
    for k in ("ms", "vs"):
        assert np.array_equal(bits32(t[k].cpu().numpy()), bits32(a[0][k].cpu().numpy()))
