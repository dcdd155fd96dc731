"""AdamW over many matrices, states in 32 and 8 bits, and the gradient norm
(GPU).

The moments are fp32 with every operation rounded, so m, v (32-bit), the
8-bit codes and their scales must be the oracle's bit for bit; the bf16 copy
is the device's own p rounded, bit for bit.  p against fp64, with e = 2^-24
(half an fp32 step, relative):
  * p's own roundings: the factor 1 - lr wd, its product with p and the final
    subtraction, e |p| each: 3 e |p|;
  * m's two products and their sum: 2 e (|b1 m| + |(1 - b1) g|), which does
    not shrink with m where the two terms cancel, times the step over the
    denominator;
  * relative errors of the update itself: v 3 e (all terms positive), halved
    by the square root, the root, 1 / sqrt(1 - b2^t) and the product with
    it, the sum with eps, the division, the step size and its product, e
    each: 8.5 e, and 10 e with the second-order terms.
"""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_22_amd as qn
from oracle import fp8, optim, optim8
from tests.gpu_helpers import to_bits16, synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def f32(x):
    return float(np.float32(x))


LR, B1, B2, EPS, WD = f32(2e-4), f32(0.9), f32(0.999), f32(1e-8), f32(0.01)
HYPER = dict(lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def make(sizes, bits, step, bf16_grad, seed):
    """Host state of matrices of the given sizes (flat arrays)."""
    rng = np.random.default_rng(seed)
    out = []
    for n in sizes:
        size = np.exp(2 * rng.standard_normal(n)) * 1e-4
        g = (rng.standard_normal(n) * size).astype(np.float32)
        if bf16_grad:
            g = synth.bf16_to_f32(synth.bf16_bits(g))
        d = {"p": (rng.standard_normal(n) * 0.02).astype(np.float32), "g": g}
        m = (rng.standard_normal(n) * size * 0.3).astype(np.float32)
        v = ((rng.standard_normal(n) * size) ** 2 * 0.4).astype(np.float32)
        if step == 1:
            m[:], v[:] = 0, 0
        if bits == 8:
            d["mc"], d["ms"] = optim8.encode_m(m, 0)
            d["vc"], d["vs"] = optim8.encode_v(v, 0)
            m = (fp8.e4m3_values()[d["mc"]].astype(np.float32) * np.repeat(d["ms"], 256)[:n])
            v = (optim8.e5m2_values()[d["vc"]].astype(np.float32) * np.repeat(d["vs"], 256)[:n])
        d["m"], d["v"] = m.astype(np.float32), v.astype(np.float32)
        out.append(d)
    return out


def upload(state, bits, bf16_grad):
    t = []
    for d in state:
        e = {"p": dev(d["p"]), "g": dev(d["g"])}
        if bf16_grad:
            e["g"] = e["g"].bfloat16()
        if bits == 8:
            e["m"] = dev(d["mc"]).view(torch.float8_e4m3fn)
            e["v"] = dev(d["vc"]).view(torch.float8_e5m2)
            e["ms"], e["vs"] = dev(d["ms"]), dev(d["vs"])
        else:
            e["m"], e["v"], e["ms"], e["vs"] = dev(d["m"]), dev(d["v"]), None, None
        e["b"] = torch.zeros(d["p"].size, dtype=torch.bfloat16, device=DEV)
        t.append(e)
    return t


def table_of(t, bits):
    col = lambda k: [e[k] for e in t]
    return qn.lora_adamw_table(col("p"), col("g"), col("m"), col("v"),
                               m_scales=col("ms") if bits == 8 else None,
                               v_scales=col("vs") if bits == 8 else None, p_bf16s=col("b"))


def bits32(a):
    return np.ascontiguousarray(a, np.float32).view(np.uint32)


E = 2.0 ** -24


def p_bound(p0, p64, g, m0, v64, step):
    """The bound on |p - p64| derived above."""
    p0, g, m0 = (np.asarray(a, np.float64) for a in (p0, g, m0))
    den = np.sqrt(v64 / (1 - B2 ** step)) + EPS
    size = LR / (1 - B1 ** step)
    upd = np.abs(p64 - p0 * (1 - LR * WD))
    return (3 * E * np.maximum(np.abs(p0), np.abs(p64)) * 1.01
            + size / den * 2 * E * (B1 * np.abs(m0) + (1 - B1) * np.abs(g)) * 1.01
            + 10 * E * upd + 1e-37)


def check(state, t, bits, step, c=1.0):
    for d, e in zip(state, t):
        g = (d["g"] * np.float32(c)).astype(np.float32)
        m, v = optim8.moments(g, d["m"], d["v"], B1, B2)
        p64, _, v64 = optim.adamw_step(d["p"], g, d["m"], d["v"], LR, B1, B2, EPS, WD, step)
        p = e["p"].cpu().numpy()
        assert np.all(np.abs(p - p64) <= p_bound(d["p"], p64, g, d["m"], v64, step))
        assert np.array_equal(to_bits16(e["b"]), synth.bf16_bits(p))
        if bits == 32:
            assert np.array_equal(bits32(e["m"].cpu().numpy()), bits32(m))
            assert np.array_equal(bits32(e["v"].cpu().numpy()), bits32(v))
            continue
        for x, s, enc, y in ((e["m"], e["ms"], optim8.encode_m, m),
                             (e["v"], e["vs"], optim8.encode_v, v)):
            codes, scales = enc(y, step)
            assert np.array_equal(bits32(s.cpu().numpy()), bits32(scales))
            assert np.array_equal(x.view(torch.uint8).cpu().numpy(), codes)


SIZES = [[1], [7, 8, 9], [255, 256, 257], [2047, 2048, 2049, 0, 5], [65536, 10001, 3, 4096]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bf16_grad", [False, True])
@pytest.mark.parametrize("step", [1, 2, 1000])
def test_step_is_the_oracles(sizes, bits, bf16_grad, step):
    state = make(sizes, bits, step, bf16_grad, seed=sum(sizes) + step)
    t = upload(state, bits, bf16_grad)
    qn.lora_adamw_multi_step(table_of(t, bits), step, **HYPER)
    torch.cuda.synchronize()
    check(state, t, bits, step)


@pytest.mark.parametrize("bits", [32, 8])
def test_special_values_of_gradients_and_states(bits):
    """All-zero blocks, one element in a block, tiny and large gradients."""
    state = make([2048], bits, 5, False, seed=1)
    d = state[0]
    g = d["g"]
    g[:256] = 0
    g[256:512] = 0
    g[300] = 1e-3
    g[512:768] = 1e-30
    g[768:1024] *= np.float32(1e12)
    g[1024:1280] = 1e-21
    for a in range(0, 512, 256):
        d["m"][a:a + 256] = 0
        d["v"][a:a + 256] = 0
        if bits == 8:
            d["mc"][a:a + 256] = 0
            d["vc"][a:a + 256] = 0
    t = upload(state, bits, False)
    qn.lora_adamw_multi_step(table_of(t, bits), 5, **HYPER)
    torch.cuda.synchronize()
    check(state, t, bits, 5)


def test_bf16_copy_is_optional_per_matrix():
    state = make([300, 4000], 32, 2, False, seed=3)
    t = upload(state, 32, False)
    col = lambda k: [e[k] for e in t]
    tab = qn.lora_adamw_table(col("p"), col("g"), col("m"), col("v"), p_bf16s=[None, t[1]["b"]])
    qn.lora_adamw_multi_step(tab, 2, **HYPER)
    torch.cuda.synchronize()
    assert not t[0]["b"].any()
    assert np.array_equal(to_bits16(t[1]["b"]), synth.bf16_bits(t[1]["p"].cpu().numpy()))


@pytest.mark.parametrize("bf16_grad", [False, True])
@pytest.mark.parametrize("sizes", SIZES + [[5_000_011, 70_000]])
def test_gradient_norm(sizes, bf16_grad):
    state = make(sizes, 32, 2, bf16_grad, seed=8)
    t = upload(state, 32, bf16_grad)
    tab = table_of(t, 32)
    norm = np.sqrt(sum(np.sum(d["g"].astype(np.float64) ** 2) for d in state))
    for max_norm in (0.5 * float(norm), 1e6):
        out = qn.lora_grad_norm(tab, max_norm).cpu().numpy()
        # fp64 sums, one rounding to fp32
        assert abs(out[0] - norm) <= 2.0 ** -23 * norm
        want = min(1.0, f32(max_norm) / (norm + 1e-6))
        assert abs(out[1] - want) <= 2.0 ** -23 * want


@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_step(bits):
    state = make([70001, 513], bits, 9, False, seed=2)
    t = upload(state, bits, False)
    tab = table_of(t, bits)
    norm = qn.lora_grad_norm(tab, 1e-3)
    qn.lora_adamw_multi_step(tab, 9, grad_scale=norm[1:], **HYPER)
    torch.cuda.synchronize()
    c = float(norm[1])
    assert 0 < c < 1
    check(state, t, bits, 9, c)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_norm_that_is_not_finite_skips_the_step(bad):
    for bits in (32, 8):
        state = make([3000], bits, 4, False, seed=6)
        t = upload(state, bits, False)
        t[0]["g"][1234] = bad
        tab = table_of(t, bits)
        before = {k: t[0][k].clone() for k in ("p", "m", "v", "b")}
        norm = qn.lora_grad_norm(tab, 1.0)
        qn.lora_adamw_multi_step(tab, 4, grad_scale=norm[1:], **HYPER)
        torch.cuda.synchronize()
        assert not np.isfinite(norm[0].item()) and np.isnan(norm[1].item())
        for k, was in before.items():
            assert torch.equal(t[0][k].view(torch.uint8), was.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_many_steps_follow_the_32_bit_states(bits):
    """Steady gradients of one size: after 400 steps v's expectation is the
    mean square, and the 8-bit states have not stuck on the way.  Mean over
    4096 elements of v / (1 - b2^t) against g^2: each element's dithered codes
    are unbiased with a standard deviation of at most a code (25% of v), and
    their errors are averaged over the steps and the elements; 2% is kept."""
    n = 4096
    rng = np.random.default_rng(0)
    t = upload(make([n], bits, 1, False, seed=1), bits, False)[0]
    mag = (np.exp(rng.standard_normal(n)) * 1e-3).astype(np.float32)
    tab = table_of([t], bits)
    for step in range(1, 401):
        sign = (rng.integers(0, 2, n) * 2 - 1).astype(np.float32)
        t["g"].copy_(dev(sign * mag))
        qn.lora_adamw_multi_step(tab, step, **HYPER)
    torch.cuda.synchronize()
    v = t["v"].float().cpu().numpy().astype(np.float64)
    if bits == 8:
        v = v * np.repeat(t["vs"].cpu().numpy(), 256)[:n]
    ratio = v / (1 - B2 ** 400) / mag.astype(np.float64) ** 2
    assert abs(ratio.mean() - 1) <= 0.02


def test_captured_step_repeats_itself():
    state = make([5000, 300], 8, 7, False, seed=12)
    t = upload(state, 8, False)
    eager = upload(state, 8, False)
    tab, etab = table_of(t, 8), table_of(eager, 8)
    norm = torch.empty(2, device=DEV)
    ws = qn.workspace(qn.lora_grad_norm_workspace_bytes(tab), DEV)

    def one(table):
        qn.lora_grad_norm(table, 1e-3, out=norm, ws=ws)
        qn.lora_adamw_multi_step(table, 7, grad_scale=norm[1:], **HYPER)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(tab)
    for i in range(4):
        g = torch.randn(5000, device=DEV) * 1e-3
        t[0]["g"].copy_(g)
        eager[0]["g"].copy_(g)
        one(etab)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(t, eager):
            for k in ("p", "m", "v", "ms", "vs", "b"):
                assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), (i, k)


def test_a_training_step_of_an_8_bit_layer():
    """The operators together, as a step uses them: quantise the frozen
    weight, forward, backward to the input, LoRA gradients, clip, one AdamW
    launch for A and B, forward with the new bf16 adapter.  The new adapter
    must be the oracle's step on the gradients that lora_grads gave, and the
    forward the one of the new adapter."""
    M, N, K, r, alpha = 96, 192, 320, 16, 32.0
    rng = np.random.default_rng(0)
    bf = lambda a: synth.bf16_to_f32(synth.bf16_bits(a.astype(np.float32)))
    w = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    A0, B0 = bf(rng.standard_normal((r, K)) * 0.02), bf(rng.standard_normal((N, r)) * 0.02)
    x, dy = bf(rng.standard_normal((M, K))), bf(rng.standard_normal((M, N)) * 1e-2)
    fw = qn.fp8_quantize_weight(dev(w))
    xd, dyd = dev(x).bfloat16(), dev(dy).bfloat16()
    A, B = dev(A0), dev(B0)
    Ab, Bb = A.bfloat16(), B.bfloat16()
    dA, dB = torch.empty_like(A), torch.empty_like(B)
    z8 = lambda t, d: torch.zeros(t.numel(), dtype=torch.uint8, device=DEV).view(d)
    zs = lambda t: torch.zeros(-(-t.numel() // 256), device=DEV)
    ms, vs = [zs(A), zs(B)], [zs(A), zs(B)]
    m = [z8(t, torch.float8_e4m3fn) for t in (A, B)]
    v = [z8(t, torch.float8_e5m2) for t in (A, B)]
    tab = qn.lora_adamw_table([A, B], [dA, dB], m, v, ms, vs, [Ab, Bb])
    u = torch.empty((M, r), dtype=torch.bfloat16, device=DEV)
    t = torch.empty((M, r), dtype=torch.bfloat16, device=DEV)
    y0 = qn.fp8_linear_fwd(fw, xd, Ab, Bb, r, alpha, u_out=u)
    dx = qn.fp8_linear_bwd_dx(fw, dyd, Ab, Bb, r, alpha, t_out=t)
    qn.lora_grads(xd, dyd, Ab, Bb, r, alpha, u=u, t=t, dA=dA, dB=dB)
    norm = qn.lora_grad_norm(tab, 0.3)
    qn.lora_adamw_multi_step(tab, 1, grad_scale=norm[1:], **HYPER)
    y1 = qn.fp8_linear_fwd(fw, xd, Ab, Bb, r, alpha)
    torch.cuda.synchronize()
    gA, gB = dA.cpu().numpy().astype(np.float64), dB.cpu().numpy().astype(np.float64)
    s = alpha / r
    wv = fp8.weight_values(*fp8.quantize_blocks(w))
    ref_gA, ref_gB = s * (dy @ B0).T.astype(np.float64) @ x, s * dy.T.astype(np.float64) @ (x @ A0.T)
    assert np.linalg.norm(gA - ref_gA) <= 1e-2 * np.linalg.norm(ref_gA)
    assert np.linalg.norm(gB - ref_gB) <= 1e-2 * np.linalg.norm(ref_gB)
    want = np.sqrt((gA ** 2).sum() + (gB ** 2).sum())
    assert abs(norm[0].item() - want) <= 2.0 ** -23 * want
    c = norm[1].item()
    for p0, p, g, b in ((A0, A, gA, Ab), (B0, B, gB, Bb)):
        g = (g.astype(np.float32) * np.float32(c)).astype(np.float32)
        z = np.zeros_like(p0)
        ref, _, v64 = optim.adamw_step(p0, g, z, z, LR, B1, B2, EPS, WD, 1)
        got = p.cpu().numpy()
        assert np.all(np.abs(got - ref) <= p_bound(p0, ref, g, z, v64, 1))
        assert np.array_equal(to_bits16(b), synth.bf16_bits(got))
    qx = fp8.row_values(*fp8.quantize_rows(x))
    for y, Af, Bf in ((y0, A0, B0), (y1, Ab.float().cpu().numpy(), Bb.float().cpu().numpy())):
        ref = qx @ wv.T + s * (x.astype(np.float64) @ Af.T) @ Bf.T
        e = np.linalg.norm(y.float().cpu().numpy() - ref) / np.linalg.norm(ref)
        assert e <= 2.0 ** -8
    qd = fp8.row_values(*fp8.quantize_rows(dy))
    ref = qd @ wv + s * (dy.astype(np.float64) @ B0) @ A0
    assert np.linalg.norm(dx.float().cpu().numpy() - ref) <= 2.0 ** -8 * np.linalg.norm(ref)


def test_table_refuses_the_same_matrix_twice():
    t = upload(make([300], 32, 2, False, seed=1), 32, False)[0]
    two = lambda k: [t[k], t[k]]
    with pytest.raises(qn.QnError) as e:
        qn.lora_adamw_table(two("p"), two("g"), two("m"), two("v"))
    assert e.value.status == qn.QN_ERR_SHAPE
    with pytest.raises(ValueError):
        qn.lora_adamw_table([t["p"]], [t["g"]], [t["m"].cpu()], [t["v"]])
    with pytest.raises(ValueError):
        qn.lora_adamw_table([t["p"]], [t["g"]], [t["m"][:299]], [t["v"]])
    with pytest.raises(qn.QnError) as e:
        qn.lora_adamw_table([t["p"][1:]], [t["g"][1:]], [t["m"][1:]], [t["v"][1:]])
    assert e.value.status == qn.QN_ERR_ALIGN


def test_steps_on_another_stream():
    state = make([5000, 70], 8, 3, False, seed=4)
    t = upload(state, 8, False)
    tab = table_of(t, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm = qn.lora_grad_norm(tab, 1e9, stream=side)
    qn.lora_adamw_multi_step(tab, 3, grad_scale=norm[1:], stream=side, **HYPER)
    torch.cuda.synchronize()
    check(state, t, 8, 3)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_gradient_that_is_not_finite_without_clipping(bits, bad):
    """p of its element is NaN, and nothing outside its block of 256 differs."""
    state = make([3000], bits, 4, False, seed=6)
    clean, t = upload(state, bits, False), upload(state, bits, False)
    t[0]["g"][700] = bad
    for e in (clean, t):
        tab = table_of(e, bits)
        qn.lora_adamw_multi_step(tab, 4, **HYPER)
        qn.lora_adamw_multi_step(tab, 5, **HYPER)
    torch.cuda.synchronize()
    assert torch.isnan(t[0]["p"][700])
    for k in ("p", "b", "m", "v"):
        same = t[0][k].view(torch.uint8).view(3000, -1) == clean[0][k].view(torch.uint8).view(3000, -1)
        same[512:768] = True
        assert same.all(), k


def test_offsets_past_32_bits():
    """A matrix whose fp32 values take more than 2^32 bytes: its end steps as
    a small matrix of the same values does."""
    n, n0 = 2 ** 30 + 2125, 2 ** 30 - 2048
    g = torch.Generator(device=DEV).manual_seed(1)
    p = torch.randn(n, generator=g, device=DEV)
    grad = torch.randn(n, generator=g, device=DEV).bfloat16()
    blocks = -(-n // 256)
    ms = torch.rand(blocks, generator=g, device=DEV) * 1e-4
    vs = torch.rand(blocks, generator=g, device=DEV) * 1e-4
    m = torch.randint(0, 0x7F, (n,), generator=g, device=DEV, dtype=torch.uint8)
    v = torch.randint(0, 0x7C, (n,), generator=g, device=DEV, dtype=torch.uint8)
    b = torch.empty(n, dtype=torch.bfloat16, device=DEV)
    whole = [p, grad, m.view(torch.float8_e4m3fn), v.view(torch.float8_e5m2), ms, vs, b]
    first = [n0 // 256 if i in (4, 5) else n0 for i in range(7)]
    end = [t[a:].clone() for a, t in zip(first, whole)]
    norms = []
    for cols in (whole, end):
        tab = qn.lora_adamw_table(*[[t] for t in cols])
        norms.append(qn.lora_grad_norm(tab, 1e9))
        qn.lora_adamw_multi_step(tab, 100, **HYPER)
    torch.cuda.synchronize()
    want = sum(float(grad[i:i + 2 ** 27].double().square().sum()) for i in range(0, n, 2 ** 27))
    assert abs(norms[0][0].item() - want ** 0.5) <= 2.0 ** -23 * want ** 0.5
    for a, t, e in zip(first, whole, end):
        assert torch.equal(t[a:].view(torch.uint8), e.view(torch.uint8))
