"""How many Newton-Schulz steps the Muon step takes (CPU: nothing here launches
a kernel).

The library runs the steps on S0 = X0 X0^T, with X = T X0.  Rounding leaves S0
eigenvalues of +-2^-53 or so where u has no direction, and each step multiplies
them with ns[0]^2; one that is negative and near 1 runs away, which X X^T, never
negative, cannot.  Counts with ns[0]^(2 steps) past 2^43 are refused."""

import ctypes

import numpy as np
import pytest

import bit_nf4_quantized_22_amd as qn
from oracle import muon
from tests.test_abi import lib  # noqa: F401
from tests.muon_bounds import LARGEST, steps_bound
from tests.test_abi_muon import build, hyper, tensors

# more coefficients with the largest count that is taken
MORE = [((1.0, 0.0, 0.0), 32), ((0.5, 0.2, 0.1), 32), ((0.0, 1.0, 0.0), 32),
        ((2.0 ** 21.5, 0.0, 0.0), 1)]


@pytest.mark.parametrize("ns,most", LARGEST + MORE)
def test_counts_that_64_bits_do_not_hold_are_refused(lib, ns, most):  # noqa: F811
    _, empty, _, _ = build(tensors((0, 5)))      # no matrix: no launch

    def status(steps):
        return lib.lora_muon_multi_step(ctypes.byref(empty), None,
                                        ctypes.byref(hyper(ns=ns, ns_steps=steps)), None, 0, None)

    assert [status(n) for n in range(1, most + 1)] == [qn.QN_OK] * most
    assert [status(n) for n in range(most + 1, 33)] == [qn.QN_ERR_UNSUPPORTED] * (32 - most)
    assert status(0) == status(33) == qn.QN_ERR_SHAPE


def on_the_gram_matrix(u, ns, steps, eps=1e-7):
    """The library's form in 64 bits, symmetric matrices by their upper half."""
    def sym(m):
        return np.triu(m) + np.triu(m, 1).T

    s = sym(u @ u.T)
    inv = 1 / (np.sqrt(np.trace(s)) + eps)
    s, t = s * (inv * inv), None
    for _ in range(steps):
        q = sym(ns[2] * (s @ s) + ns[1] * s + ns[0] * np.eye(len(s)))
        t = q if t is None else sym(t @ q)
        s = sym(sym(s @ q) @ q)
    return t @ (u * inv)


def update(shape, kind, seed=1):
    rng = np.random.default_rng(seed)
    a, b = shape
    if kind == "steep":
        left, _ = np.linalg.qr(rng.standard_normal((a, a)))
        right, _ = np.linalg.qr(rng.standard_normal((b, a)))
        g = (left * 10.0 ** -np.linspace(0, 10, a)) @ right.T
    else:
        g = rng.standard_normal((a, kind)) @ rng.standard_normal((kind, b))
    return (1e-3 * g).astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("ns,most", LARGEST)
@pytest.mark.parametrize("kind", [1, 5, "steep"])
@pytest.mark.parametrize("shape", [(16, 700), (64, 1500), (128, 300)])
def test_the_form_is_the_definition_up_to_the_largest_count(shape, kind, ns, most):
    u = update(shape, kind)
    for steps in (5, most // 2, most):
        off = on_the_gram_matrix(u, ns, steps) - muon.orthogonalised(u, 1e-7, ns, steps)
        bound = steps_bound(u, ns, steps, chain=shape[1])
        assert np.linalg.norm(off) <= bound, steps
        assert bound <= (2.0 ** -24 if steps == 5 else 1), steps     # of X's about sqrt(r)


def test_the_form_runs_away_past_it():
    """The reason for the refusal."""
    u = update((16, 700), 1)
    with np.errstate(all="ignore"):
        wrong = on_the_gram_matrix(u, muon.COEFFICIENTS, 20)
    assert not np.abs(wrong).max() < 1e3
    assert np.abs(muon.orthogonalised(u, 1e-7, steps=20)).max() < 1
