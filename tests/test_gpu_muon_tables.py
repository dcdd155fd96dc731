"""Tables of the Muon step: a matrix alone and among others, matrices whose
bytes pass 2^32, and calls that are refused (GPU)."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_22_amd as qn
from oracle import muon
from tests.test_gpu_muon import DEV, U, Case

pytestmark = pytest.mark.gpu


def test_a_matrix_alone_and_among_few():
    """Few matrices are chunked alike in any table: the same bits."""
    shapes = [(16, 700), (33, 500), (500, 64), (1000, 5), (100, 300)]
    c = Case(shapes, 31)
    qn.lora_muon_multi_step(c.table, lr=2e-3)
    for i in range(len(shapes)):
        d = Case(shapes, 31)
        table = qn.lora_muon_table([d.p[i]], [d.gd[i]], [d.m[i]], p_bf16s=[d.b[i]])
        qn.lora_muon_multi_step(table, lr=2e-3)
        torch.cuda.synchronize()
        for x, y in ((c.p, d.p), (c.m, d.m), (c.b, d.b)):
            assert torch.equal(x[i], y[i])


@pytest.mark.parametrize("shape", [(16, 4096), (4096, 20)])
def test_a_matrix_among_many(shape):
    """Chunks of several runs: the same within the step's bounds."""
    c, n = Case([shape], 32), 700
    fill = [torch.full((n,) + shape, v, device=DEV) for v in (0.01, 1e-3, 0.0)]
    table = qn.lora_muon_table(*[list(t) + [x[0]] for t, x in zip(fill, (c.p, c.gd, c.m))],
                               p_bf16s=[None] * n + [c.b[0]])
    assert sum(table.plan.chunks) < (n + 1) * 16
    qn.lora_muon_multi_step(table, lr=2e-3)
    torch.cuda.synchronize()
    c.check()
    assert (fill[0] == fill[0][0]).all()


@pytest.mark.parametrize("rows,cols,bf16_grad", [(128, 2 ** 24 - 4, True), (2 ** 24 - 1, 126, False)])
def test_offsets_past_32_bits(rows, cols, bf16_grad):
    """8 GB a matrix: the definition by torch in 64 bits, a part of the long side
    at a time, on the update as the step rounds it."""
    g = torch.Generator(device=DEV).manual_seed(1)
    tall = rows > cols
    r, length = min(rows, cols), max(rows, cols)
    p = torch.empty(rows, cols, device=DEV).normal_(generator=g).mul_(0.02)
    m = torch.zeros_like(p)
    grad = torch.empty(rows, cols, device=DEV, dtype=torch.bfloat16 if bf16_grad else
                       torch.float32).normal_(generator=g)
    # rows and columns of other sizes, so that a wrong address is seen
    grad.mul_(torch.linspace(1, 2, r, device=DEV).to(grad.dtype).view((1, r) if tall else (r, 1)))
    grad.mul_(torch.linspace(1, 3, length, device=DEV).to(grad.dtype).view(
        (length, 1) if tall else (1, length)))
    p0 = p.clone()
    lr, mu = 1.0, 0.0                            # u = g
    step = 2 ** 19

    def part(t, k):
        t = t[k:k + step].t() if tall else t[:, k:k + step]
        return t.double().contiguous()

    table = qn.lora_muon_table([p], [grad], [m])
    qn.lora_muon_multi_step(table, lr=lr, momentum=mu, weight_decay=0.0)
    torch.cuda.synchronize()
    s = torch.zeros(r, r, dtype=torch.float64, device=DEV)
    for k in range(0, length, step):
        u = part(grad, k)
        s += u @ u.t().contiguous()
    s = s.cpu().numpy()
    inv = 1 / (np.sqrt(np.trace(s)) + np.float64(np.float32(1e-7)))
    s, t, (a, b, c) = s * inv * inv, np.eye(r), muon.COEFFICIENTS
    for _ in range(muon.STEPS):
        q = a * np.eye(r) + b * s + c * s @ s
        t, s = t @ q, s @ q @ q
    t = torch.from_numpy(t * inv).to(DEV)
    f = muon.factor("original", rows, cols)
    for k in range(0, length, step):
        x = t @ part(grad, k)
        want = part(p0, k) - lr * f * x
        bound = U * (2 * part(p0, k).abs() + want.abs() + 2 * lr * f * x.abs())
        assert ((part(p, k) - want).abs() <= bound).all(), k
        assert torch.equal(part(m, k), part(grad, k))


def test_three_coefficients():
    c = Case([(16, 700)], 33)
    for ns in ((), (1.5,), (1.5, -0.5), (1.5, -0.5, 0.0, 0.0)):
        with pytest.raises(ValueError):
            qn.lora_muon_multi_step(c.table, ns_coefficients=ns)
    torch.cuda.synchronize()
    assert np.array_equal(c.p[0].cpu().numpy(), c.p0[0])
