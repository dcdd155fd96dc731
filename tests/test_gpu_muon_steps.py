"""The Muon step at the largest counts of Newton-Schulz steps that it takes, on
updates that have no part in most directions, or parts over 10 decades (GPU)."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_22_amd as qn
from oracle import muon
from tests.gpu_helpers import to_np
from tests.muon_bounds import LARGEST, steps_bound
from tests.test_gpu_muon import Case, U

pytestmark = pytest.mark.gpu

# every class of smaller sides, wide and tall
SHAPES = [(16, 700), (700, 16), (5, 300), (31, 500), (64, 1500), (1000, 48), (128, 300), (333, 97)]


@pytest.mark.parametrize("kind", ["rank one", "steep", "zero", "falling"])
@pytest.mark.parametrize("ns,most", LARGEST)
def test_largest_counts(ns, most, kind):
    """The fp32 bounds of the step, and on X what 64 bits leave of S0: a sum has at
    most 64 elements of a chunk's 256 in a wave, 4 waves and 12 chunks."""
    f = np.float32
    lr, mu, eps = np.float64(f(2e-3)), np.float64(f(0.95)), np.float64(f(1e-7))
    om = np.float64(f(1 - mu))
    for steps in (5, most // 2, most):
        c = Case(SHAPES, 21, kinds=(kind,), momentum=kind != "rank one")
        qn.lora_muon_multi_step(c.table, lr=2e-3, weight_decay=0.0, ns_coefficients=ns,
                                ns_steps=steps)
        torch.cuda.synchronize()
        for i, (rows, cols) in enumerate(SHAPES):
            m1, p1 = (to_np(t).astype(np.float64) for t in (c.m[i], c.p[i]))
            p0 = c.p0[i].astype(np.float64)
            gs = (c.g[i].astype(f) * f(om)).astype(np.float64)
            u = (m1 * mu + gs).astype(f).astype(np.float64)
            x = muon.orthogonalised(u, eps, ns, steps)
            size = lr * muon.factor("original", rows, cols)
            want = p0 - size * x
            bound = np.linalg.norm(U * (2 * np.abs(p0) + np.abs(want) + 2 * size * np.abs(x)))
            bound += size * steps_bound(u, ns, steps, chain=64 + 4 + 12, eps=eps)
            assert np.linalg.norm(p1 - want) <= bound, (rows, cols, steps)


@pytest.mark.parametrize("ns,most", LARGEST)
def test_updates_of_exactly_rank_one(ns, most):
    """Products of integers: u is its own fp32 number, and X = f(1) u / |u| has no
    part in any other direction, whatever T makes of these."""
    rng = np.random.default_rng(23)
    eps = np.float64(np.float32(1e-7))
    for shape in SHAPES + [(1, 40), (2, 4096), (16, 4096), (4096, 16), (100, 16), (17, 900)]:
        g = np.outer(rng.integers(1, 2 ** 11, shape[0]), rng.integers(1, 2 ** 12, shape[1]))
        g = (g * 2.0 ** -30).astype(np.float32)
        p = torch.zeros(shape, device="cuda:0")
        table = qn.lora_muon_table([p], [torch.from_numpy(g).to(p.device)], [torch.zeros_like(p)])
        u = g.astype(np.float64)
        for steps in (5, 8, most):
            p.zero_()
            table.tensors[2][0].zero_()
            qn.lora_muon_multi_step(table, lr=1.0, momentum=0.0, weight_decay=0.0,
                                    ns_coefficients=ns, ns_steps=steps)
            torch.cuda.synchronize()
            size = muon.factor("original", *shape)
            want = -size * muon.orthogonalised(u, eps, ns, steps)
            bound = 3 * U * np.linalg.norm(want)
            bound += size * steps_bound(u, ns, steps, chain=64 + 4 + 32, eps=eps)
            assert np.linalg.norm(to_np(p) - want) <= bound, (shape, steps)


def test_more_steps_are_refused_and_change_nothing():
    c = Case([(16, 700)], 22, kinds=("rank one",))
    for kw in ({"ns_steps": 13}, {"ns_steps": 32},
               {"ns_steps": 24, "ns_coefficients": (1.875, -1.25, 0.375)}):
        with pytest.raises(qn.QnError) as e:
            qn.lora_muon_multi_step(c.table, **kw)
        assert e.value.status == qn.QN_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert np.array_equal(to_np(c.p[0]), c.p0[0]) and np.array_equal(to_np(c.m[0]), c.m0[0])
