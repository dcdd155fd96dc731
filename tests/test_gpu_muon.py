"""The Muon step over many LoRA matrices against the fp64 oracle (GPU).

Bounds per element, derived from the arithmetic (fp32 unit 2^-24 of a rounded
value):
  * the momentum rounds (1 - mu) g, the fused sum, and 1 - mu itself: 2^-24
    (2 |(1 - mu) g| + |m|);
  * the update is the oracle's orthogonalisation of the fp32 u that follows from
    the device's own m (its fused sum taken in fp64 and rounded): 64-bit steps add
    nothing that counts, X is rounded to fp32 once, f lr and 1 - lr wd are fp32,
    the product p (1 - lr wd) and the sum round: 2^-24 (2 |p| + |p'| + 2 lr f |X|);
  * from the oracle's own u in fp64, X may differ by the steps' largest slope,
    a^5 = 485 on either side, times what u's roundings are of its norm: 3 2^-24
    (|(1 - mu) g| + |m|) / |u| in the Frobenius norm.
"""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_22_amd as qn
from oracle import muon, mxfp4
from tests.gpu_helpers import bf16_dev, f64, synth, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24 * 1.01


def gradient(shape, rng, kind="falling"):
    a, b = shape
    g = rng.standard_normal(shape)
    if kind == "falling":             # a few strong directions over noise
        k = min(a, b, 5)
        g = 0.1 * g + (rng.standard_normal((a, k)) * 2.0 ** -np.arange(k)) @ rng.standard_normal((k, b))
    elif kind == "rank one":
        g = np.outer(rng.standard_normal(a), rng.standard_normal(b))
    elif kind == "steep":             # singular values over 10 decades
        k = min(a, b)
        q, _ = np.linalg.qr(rng.standard_normal((a, k)))
        w, _ = np.linalg.qr(rng.standard_normal((b, k)))
        g = (q * 10.0 ** -np.linspace(0, 10, k)) @ w.T
    elif kind == "zero":
        g = np.zeros(shape)
    return (g * 1e-3).astype(np.float32)


class Case:
    """Matrices on the device, with a guard behind each."""

    def __init__(self, shapes, seed=0, bf16_grad=False, kinds=("falling",), bf16_out=True,
                 momentum=True):
        rng = np.random.default_rng(seed)
        self.shapes = shapes
        gs = [gradient(s, rng, kinds[i % len(kinds)]) for i, s in enumerate(shapes)]
        self.p0 = [(rng.standard_normal(s) * 0.02).astype(np.float32) for s in shapes]
        self.m0 = [(gradient(s, rng, kinds[i % len(kinds)]) * momentum).astype(np.float32)
                   for i, s in enumerate(shapes)]
        self.g, self.gd = [], []
        for g in gs:
            t = torch.from_numpy(g).to(DEV)
            t = t.bfloat16() if bf16_grad else t
            self.gd.append(t)
            self.g.append(to_np(t).astype(np.float64))
        self.p, self.pg = zip(*[self.guarded(a, torch.float32) for a in self.p0])
        self.m, self.mg = zip(*[self.guarded(a, torch.float32) for a in self.m0])
        self.b, self.bg = zip(*[self.guarded(a, torch.bfloat16) for a in self.p0])
        self.table = qn.lora_muon_table(list(self.p), self.gd, list(self.m),
                                        p_bf16s=list(self.b) if bf16_out else None)

    @staticmethod
    def guarded(a, dtype):
        buf = torch.full((a.size + 64,), 7.0, dtype=dtype, device=DEV)
        t = buf[:a.size].view(a.shape)
        t.copy_(torch.from_numpy(a))
        return t, buf[a.size:]

    def check(self, lr=2e-3, momentum=0.95, nesterov=True, weight_decay=0.1, eps=1e-7,
              adjust="original", ns=muon.COEFFICIENTS, steps=5, bf16_out=True):
        f = np.float32
        mu, om = np.float64(f(momentum)), np.float64(f(1.0 - np.float64(f(momentum))))
        for guard in self.pg + self.mg + self.bg:
            assert (guard == 7.0).all()
        worst = 0.0
        for i, (rows, cols) in enumerate(self.shapes):
            g, p0, m0 = self.g[i], self.p0[i].astype(np.float64), self.m0[i].astype(np.float64)
            m1, p1 = to_np(self.m[i]).astype(np.float64), to_np(self.p[i]).astype(np.float64)
            ref_p, ref_m = muon.step(p0, g, m0, lr, momentum, nesterov, weight_decay, eps, adjust,
                                     ns, steps)
            assert (np.abs(m1 - ref_m) <= U * (2 * np.abs((1 - mu) * g) + np.abs(ref_m)) + 1e-45
                    ).all()
            # from the device's own momentum: u as its fp32 number
            gs = (g.astype(f) * f(om)).astype(np.float64)
            u = (m1 * mu + gs).astype(f).astype(np.float64) if nesterov else m1
            x = muon.orthogonalised(u, np.float64(f(eps)), ns, steps)
            size = np.float64(f(lr)) * muon.factor(adjust, rows, cols)
            decay = 1 - np.float64(f(lr)) * np.float64(f(weight_decay))
            want = p0 * decay - size * x
            bound = U * (2 * np.abs(p0) + np.abs(want) + 2 * size * np.abs(x)) + 1e-45
            assert (np.abs(p1 - want) <= bound).all(), (rows, cols)
            worst = max(worst, float(np.max(np.abs(p1 - want) / bound)))
            # and from the formula alone
            un = np.linalg.norm(u)
            if un > 0 and ns == muon.COEFFICIENTS and steps == 5:
                off = 2 * 485 * 3 * U * (np.linalg.norm((1 - mu) * g) + np.linalg.norm(ref_m)) / un
                assert (np.abs(p1 - ref_p) <= bound + size * off).all()
            if bf16_out:
                assert torch.equal(self.b[i], self.p[i].bfloat16())
        return worst


SHAPES = [(1, 1), (1, 50), (50, 1), (2, 2), (16, 16), (16, 4096), (4096, 16), (15, 257), (257, 15),
          (17, 300), (300, 17), (32, 33), (3, 1026), (1026, 3), (5, 7), (31, 128), (48, 500),
          (64, 1000), (1000, 64), (63, 65), (65, 129), (128, 128), (128, 2000), (2000, 100),
          (127, 333), (333, 97), (8, 8192), (16, 255), (16, 256), (64, 63), (1, 4099), (4099, 2)]


@pytest.mark.parametrize("bf16_grad", [False, True])
@pytest.mark.parametrize("nesterov", [False, True])
def test_step_against_the_oracle(bf16_grad, nesterov):
    c = Case(SHAPES, 1, bf16_grad)
    qn.lora_muon_multi_step(c.table, lr=2e-3, nesterov=nesterov)
    torch.cuda.synchronize()
    c.check(nesterov=nesterov)


@pytest.mark.parametrize("shape", SHAPES)
def test_one_matrix_alone(shape):
    c = Case([shape], 2, kinds=("falling",))
    qn.lora_muon_multi_step(c.table, lr=1e-2, adjust="match_rms_adamw", weight_decay=0.0)
    torch.cuda.synchronize()
    c.check(lr=1e-2, adjust="match_rms_adamw", weight_decay=0.0)


@pytest.mark.parametrize("kinds", [("rank one",), ("steep",), ("zero", "falling"), ("noise",)])
def test_spectra(kinds):
    c = Case([(16, 700), (700, 16), (64, 600), (128, 300), (31, 40)], 3, kinds=kinds)
    qn.lora_muon_multi_step(c.table, lr=2e-3)
    torch.cuda.synchronize()
    c.check()


def test_first_step_with_a_gradient_of_zero():
    """A of a fresh adapter: B = 0 gives A no gradient; p only decays, and
    without decay stays as it is."""
    c = Case([(16, 4096), (40, 100)], 4, kinds=("zero",), momentum=False)
    before = [p.clone() for p in c.p]
    qn.lora_muon_multi_step(c.table, weight_decay=0.0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, c.p))
    assert all((m == 0).all() for m in c.m)
    qn.lora_muon_multi_step(c.table, lr=1.0, weight_decay=0.5)
    torch.cuda.synchronize()
    assert all(torch.equal(a * 0.5, b) for a, b in zip(before, c.p))


@pytest.mark.parametrize("kw", [{"momentum": 0.0}, {"eps": 1.0}, {"eps": 1e-30}, {"steps": 1},
                                {"steps": 2}, {"steps": 12}, {"ns": (1.5, -0.5, 0.0)}, {"lr": 0.0}])
def test_hyperparameters(kw):
    c = Case([(16, 700), (300, 40), (100, 120)], 5)
    call = {{"steps": "ns_steps", "ns": "ns_coefficients"}.get(k, k): v for k, v in kw.items()}
    qn.lora_muon_multi_step(c.table, **{"lr": 2e-3, **call})
    torch.cuda.synchronize()
    c.check(**kw)


@pytest.mark.parametrize("size", [1e-30, 1e30])
def test_gradients_of_any_size(size):
    """Squares far outside fp32's range: the update does not depend on the size
    (eps far below it)."""
    rng = np.random.default_rng(6)
    g = rng.standard_normal((20, 500))
    out = []
    for s in (1.0, size):
        p = torch.zeros(20, 500, device=DEV)
        t = torch.from_numpy((g * s).astype(np.float32)).to(DEV)
        table = qn.lora_muon_table([p], [t], [torch.zeros_like(p)])
        qn.lora_muon_multi_step(table, lr=1.0, eps=1e-40)
        out.append(to_np(p))
    x = muon.orthogonalised(g)
    for o in out:
        # fp32 inputs: 485 times their rounding, as above
        assert np.abs(o + x).max() <= 2 * 485 * 4 * U + U * np.abs(x).max()


def test_an_infinite_or_nan_gradient_spoils_its_matrix_alone():
    shapes = [(16, 700), (700, 16), (64, 600), (100, 300)]
    good = Case(shapes, 7)
    qn.lora_muon_multi_step(good.table)
    for bad in range(4):
        for v in (float("nan"), float("inf")):
            c = Case(shapes, 7)
            c.gd[bad][3, 5] = v
            qn.lora_muon_multi_step(c.table)
            torch.cuda.synchronize()
            for i in range(4):
                if i == bad:
                    assert torch.isnan(c.p[i]).all()
                else:
                    assert torch.equal(c.p[i], good.p[i]) and torch.equal(c.m[i], good.m[i])


def test_long_matrices_in_many_chunks():
    c = Case([(8, 300_000), (200_001, 5), (20, 70_000)], 8)
    assert max(c.table.plan.chunks) > 200
    qn.lora_muon_multi_step(c.table, lr=2e-3)
    torch.cuda.synchronize()
    c.check()


def test_several_steps_match_single_tables_bit_for_bit():
    """A matrix's chunks depend on the table, its result only on them: the same
    table gives the same bits again, and follows the oracle over steps."""
    shapes = [(16, 700), (33, 500), (500, 64)]
    a, b = Case(shapes, 9), Case(shapes, 9)
    for step in range(3):
        for c in (a, b):
            qn.lora_muon_multi_step(c.table, lr=2e-3)
            torch.cuda.synchronize()
            c.check()
            c.p0 = [to_np(p) for p in c.p]
            c.m0 = [to_np(m) for m in c.m]
        for x, y in zip(a.p + a.m, b.p + b.m):
            assert torch.equal(x, y)


def test_without_bf16_copies_and_with_some():
    shapes = [(16, 700), (700, 16)]
    want = Case(shapes, 10)
    qn.lora_muon_multi_step(want.table)
    c = Case(shapes, 10, bf16_out=False)
    before = [b.clone() for b in c.b]
    qn.lora_muon_multi_step(c.table)
    assert all(torch.equal(x, y) for x, y in zip(c.b, before))
    d = Case(shapes, 10, bf16_out=False)
    table = qn.lora_muon_table(list(d.p), d.gd, list(d.m), p_bf16s=[None, d.b[1]])
    qn.lora_muon_multi_step(table)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(c.p + d.p, want.p + want.p))
    assert torch.equal(d.b[0], before[0]) and torch.equal(d.b[1], want.b[1])


def test_streams_and_captured_graphs():
    shapes = [(16, 4096), (4096, 16), (64, 2000), (100, 200)]
    want, c = Case(shapes, 11), Case(shapes, 11)
    qn.lora_muon_multi_step(want.table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for t, v in zip(c.p + c.m, c.p0 + c.m0):
            t.copy_(torch.from_numpy(v))
        torch.cuda.synchronize()
        qn.lora_muon_multi_step(c.table, stream=side)
        torch.full((qn.lora_muon_workspace_bytes(c.table),), 255, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(c.p + c.m, want.p + want.m))
    ws = qn.workspace(qn.lora_muon_workspace_bytes(c.table), DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qn.lora_muon_multi_step(c.table, ws=ws)
    eager = Case(shapes, 11)
    for t, v in zip(c.p + c.m, c.p0 + c.m0):
        t.copy_(torch.from_numpy(v))
    for i in range(4):
        for x, y in zip(c.gd, eager.gd):
            y.mul_(0.7).add_(1e-4 * i)
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        qn.lora_muon_multi_step(eager.table)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(c.p + c.m + c.b, eager.p + eager.m + eager.b))


def test_workspace_is_not_overrun_and_need_not_be_clean():
    c, want = Case(SHAPES, 12), Case(SHAPES, 12)
    qn.lora_muon_multi_step(want.table)
    need = qn.lora_muon_workspace_bytes(c.table)
    buf = torch.full((need + 4096,), 255, dtype=torch.uint8, device=DEV)   # NaN as doubles
    qn.lora_muon_multi_step(c.table, ws=buf[:need])
    torch.cuda.synchronize()
    assert (buf[need:] == 255).all()
    assert all(torch.equal(x, y) for x, y in zip(c.p + c.m, want.p + want.m))


def test_binding_refusals():
    p, g, m = (torch.zeros(4, 64, device=DEV) for _ in range(3))
    b = p.bfloat16()
    make = qn.lora_muon_table
    bad = [lambda: make([], [], []), lambda: make([p], [g], [None]), lambda: make([p], [g], []),
           lambda: make([p], [g], [m], p_bf16s=[]), lambda: make([p], [g.half()], [m]),
           lambda: make([b], [g], [m]), lambda: make([p], [g], [b]),
           lambda: make([p], [g], [m], p_bf16s=[p]), lambda: make([p], [g[:2]], [m]),
           lambda: make([p], [g.view(64, 4)], [m]), lambda: make([p.flatten()], [g], [m]),
           lambda: make([p.t()], [g], [m]), lambda: make([p.cpu()], [g], [m]),
           lambda: make([p], [g], [m.cpu()]), lambda: make([p, p], [g, b], [m, m])]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f, status in ((lambda: make([p], [g], [p]), qn.QN_ERR_SHAPE),
                      (lambda: make([p, p], [g, g], [m, m.clone()]), qn.QN_ERR_SHAPE),
                      (lambda: make(*[[torch.zeros(130, 129, device=DEV)] for _ in range(3)]),
                       qn.QN_ERR_UNSUPPORTED)):
        with pytest.raises(qn.QnError) as e:
            f()
        assert e.value.status == status
    table = make([p], [g], [m])
    with pytest.raises(ValueError):
        qn.lora_muon_multi_step(table, adjust="other")
    for kw, status in (({"lr": -1.0}, qn.QN_ERR_SHAPE), ({"ns_steps": 0}, qn.QN_ERR_SHAPE),
                       ({"ws": torch.empty(8, dtype=torch.uint8, device=DEV)},
                        qn.QN_ERR_WORKSPACE)):
        with pytest.raises(qn.QnError) as e:
            qn.lora_muon_multi_step(table, **kw)
        assert e.value.status == status
    assert (p == 0).all() and (m == 0).all()


def test_a_training_step_on_a_microscaled_weight():
    """The operators as a program uses them: the weight quantised, a layer's
    forward and backward, the adapter's gradients, the Muon step on A and B, and
    the next forward with the new adapter."""
    M, N, K, r, alpha, lr = 96, 320, 448, 16, 32.0, 0.02
    rng = np.random.default_rng(13)
    w = (rng.standard_normal((N, K)) * 0.05).astype(np.float32)
    xb, dyb = (synth.bf16_bits(rng.standard_normal(s).astype(np.float32) * k)
               for s, k in (((M, K), 1.0), ((M, N), 0.01)))
    A32, B32 = ((rng.standard_normal(s) * 0.02).astype(np.float32) for s in ((r, K), (N, r)))
    mw = qn.mxfp4_quantize_weight(torch.from_numpy(w).to(DEV))
    x, dy = bf16_dev(xb), bf16_dev(dyb)
    ps = [torch.from_numpy(a).to(DEV) for a in (A32, B32)]
    low = [p.bfloat16() for p in ps]
    gs, ms = [torch.zeros_like(p) for p in ps], [torch.zeros_like(p) for p in ps]
    table = qn.lora_muon_table(ps, gs, ms, p_bf16s=low)
    u = torch.empty((M, r), dtype=torch.bfloat16, device=DEV)
    t = torch.empty_like(u)
    y = qn.mxfp4_linear_fwd(mw, x, *low, r, alpha, u_out=u)
    dx = qn.mxfp4_linear_bwd_dx(mw, dy, *low, r, alpha, t_out=t)
    A0, B0 = (to_np(v).astype(np.float64) for v in low)
    qn.lora_grads(x, dy, *low, r, alpha, u=u, t=t, dA=gs[0], dB=gs[1])
    qn.lora_muon_multi_step(table, lr=lr)
    y2 = qn.mxfp4_linear_fwd(mw, x, *low, r, alpha)
    torch.cuda.synchronize()

    wv = mxfp4.values(*mxfp4.quantize(w))
    xf, dyf, s = f64(xb), f64(dyb), alpha / r
    xv, dv = mxfp4.values(*mxfp4.quantize(xf.astype(np.float32))), mxfp4.row_values8(dyf)

    def close(got, ref, tol):
        got = got if isinstance(got, np.ndarray) else to_np(got)
        assert np.linalg.norm(got - ref) <= tol * np.linalg.norm(ref)

    # 2^-8 of rounding to bf16 an element, and twice as much for the cuts of the
    # 8-bit sums and the roundings of u and t on the way
    close(y, xv @ wv.T + s * (xf @ A0.T) @ B0.T, 2.0 ** -7)
    close(dx, dv @ wv + s * (dyf @ B0) @ A0, 2.0 ** -7)
    dA, dB = s * (dyf @ B0).T @ xf, s * dyf.T @ (xf @ A0.T)
    close(gs[0], dA, 2.0 ** -7)
    close(gs[1], dB, 2.0 ** -7)
    for p, p0, g in zip(ps, (A32, B32), gs):
        want, _ = muon.step(p0, to_np(g), 0 * p0, lr, 0.95, True, 0.1)
        close(p, want, 1e-5)
    A1, B1 = (to_np(v).astype(np.float64) for v in low)
    assert np.abs(A1 - A0).max() > 1e-4 and np.abs(B1 - B0).max() > 1e-4
    close(y2, xv @ wv.T + s * (xf @ A1.T) @ B1.T, 2.0 ** -7)
