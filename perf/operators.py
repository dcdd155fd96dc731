"""The 8-bit operators as cases to measure: the block-scaled FP8 linear layer
(quantisation, forward, backward to the input) and the AdamW step over many
LoRA matrices at once (states in 32 or in 8 bits, gradient clipping).

``listed()`` and ``draw()`` give cases, ``prepare()`` what a program holds
before the call, ``run()`` one pass (in elementary torch operations, or
through the library where ``own`` is true), ``work()`` the bytes and
operations a pass cannot do without, ``exact()`` the result in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda:0"
BLOCK = 128          # one FP8 scale per 128 columns of a row, or per 128 x 128 weights
STATE_BLOCK = 256    # one scale per 256 optimizer-state values
FLOOR = 2.0 ** -100  # least scale
F8_MAX, F5_MAX = 448.0, 57344.0
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
# dither of the 8-bit optimizer states: element i of a block at step t
DITHER_I, DITHER_T = 0x6A09E667, 0x9E3779B9

# (N, K) of the seven projections of a 7B-shaped decoder layer
LAYER_7B = [(4096, 4096)] * 4 + [(11008, 4096)] * 2 + [(4096, 11008)]


def listed():
    return [
        # one token through an attention projection: latency
        {"name": "fwd 1 token 4096x4096", "op": "fwd", "M": 1, "N": 4096, "K": 4096, "r": 16},
        # a small batch of decoded sequences through the MLP's down projection
        {"name": "fwd 16 tokens 4096x11008", "op": "fwd", "M": 16, "N": 4096, "K": 11008, "r": 16},
        # the training step's gate projection, 7B shapes
        {"name": "fwd 2048 tokens 11008x4096", "op": "fwd", "M": 2048, "N": 11008, "K": 4096,
         "r": 16},
        # the same of a 65B-shaped layer: the largest product
        {"name": "fwd 4096 tokens 22016x8192", "op": "fwd", "M": 4096, "N": 22016, "K": 8192,
         "r": 64},
        # gradient to the input of the gate projection
        {"name": "bwd 2048 tokens 11008x4096", "op": "bwd", "M": 2048, "N": 11008, "K": 4096,
         "r": 64},
        # a ragged micro-batch on sizes that end inside a scale block
        {"name": "bwd 333 tokens 1088x2112", "op": "bwd", "M": 333, "N": 1088, "K": 2112, "r": 24},
        # a weight at load time
        {"name": "quantise 11008x4096 bf16", "op": "quantise", "N": 11008, "K": 4096,
         "bf16": True},
        # a small fp32 weight whose last blocks are partial
        {"name": "quantise 1088x2112 fp32", "op": "quantise", "N": 1088, "K": 2112, "bf16": False},
        # the adapters of one 7B layer, 32-bit states, clipped gradients: latency
        {"name": "adamw32 one layer r=16", "op": "adamw", "bits": 32, "tensors": 14, "layers": 1,
         "r": 16, "size": 0, "clip": True, "bf16_grad": False, "step": 100},
        # all adapters of a 7B model, 8-bit states, clipped gradients
        {"name": "adamw8 7B r=16", "op": "adamw", "bits": 8, "tensors": 448, "layers": 32, "r": 16,
         "size": 0, "clip": True, "bf16_grad": False, "step": 1000},
        # all adapters of a 7B model at rank 64, 32-bit states
        {"name": "adamw32 7B r=64", "op": "adamw", "bits": 32, "tensors": 448, "layers": 32,
         "r": 64, "size": 0, "clip": False, "bf16_grad": False, "step": 3},
        # tensors of odd sizes with bf16 gradients, 8-bit states
        {"name": "adamw8 odd sizes", "op": "adamw", "bits": 8, "tensors": 61, "layers": 0, "r": 0,
         "size": 50021, "clip": False, "bf16_grad": True, "step": 17},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "quantise", "adamw", "adamw"])
    if op == "adamw":
        return {"op": "adamw", "bits": rng.choice([8, 32]), "tensors": _log_uniform(rng, 1, 448),
                "layers": 0, "r": 0, "size": _log_uniform(rng, 1, 300000),
                "clip": rng.random() < 0.5, "bf16_grad": rng.random() < 0.3,
                "step": _log_uniform(rng, 1, 20000)}
    N, K = (16 * _log_uniform(rng, 8, 700) for _ in range(2))
    if op == "quantise":
        return {"op": op, "N": N, "K": K, "bf16": rng.random() < 0.7}
    return {"op": op, "M": _log_uniform(rng, 1, 4096), "N": N, "K": K,
            "r": rng.choice([0, 8, 16, 16, 24, 64, 128])}


# --- cases of the optimizer: the sizes of the tensors ------------------------

def _sizes(case):
    if case["layers"]:
        per = [n for N, K in LAYER_7B for n in (case["r"] * K, N * case["r"])]
        return per * case["layers"]
    # odd sizes between 1 and twice `size`, the same for every seed
    t = case["tensors"]
    return [1 + (2 * case["size"] * (i * 7919 % t) // t + 37 * i) % (2 * case["size"])
            for i in range(t)]


def _padded(n):
    return -(-n // STATE_BLOCK) * STATE_BLOCK


# --- inputs ------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _weight(g, N, K):
    """Normal weights of std 0.02 with rows and outliers of other sizes."""
    w = _normal(g, N, K).mul_(0.02)
    w.mul_(_normal(g, N, 1).mul_(0.3).exp_())
    w.flatten()[:: 4099].mul_(8.0)
    return w


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "quantise":
        w = _weight(g, case["N"], case["K"])
        return {"case": case, "w": w.bfloat16() if case["bf16"] else w}
    if case["op"] == "adamw":
        return _prepare_adamw(case, g)
    M, N, K, r = case["M"], case["N"], case["K"], case["r"]
    L = K if case["op"] == "fwd" else N
    codes, scale = _quantise_blocks(_weight(g, N, K))
    # activations (or gradients) whose columns and rows differ in size
    x = _normal(g, M, L).mul_(_normal(g, 1, L).exp_()).mul_(_normal(g, M, 1).mul_(0.5).exp_())
    if case["op"] == "bwd":
        x.mul_(1e-3)
    s = {"case": case, "codes": codes, "scale": scale, "x": x.bfloat16(), "r": r,
         "alpha": 16.0 if r >= 64 else 32.0,
         "A": _normal(g, r, K).mul_(0.02).bfloat16() if r else None,
         "B": _normal(g, N, r).mul_(0.02).bfloat16() if r else None}
    if own:
        import bit_nf4_quantized_22_amd as qn
        s["weight"] = qn.Fp8Weight(codes, scale)
        op = qn.QN_OP_FP8_FWD if case["op"] == "fwd" else qn.QN_OP_FP8_BWD_DX
        s["ws"] = qn.workspace(qn.qn_workspace_bytes(op, M, N, K, r), DEV)
    return s


def _prepare_adamw(case, g):
    sizes = _sizes(case)
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += _padded(n)
    real = torch.zeros(total, device=DEV)   # 1 where an element belongs to a tensor
    for o, n in zip(starts, sizes):
        real[o:o + n] = 1
    p = _normal(g, total).mul_(0.02).mul_(real)
    # gradients whose size changes from block to block, and a state that has
    # seen such gradients for some steps
    size = _normal(g, total // STATE_BLOCK, 1).mul_(1.5).exp_().mul_(1e-4)
    def like_grad():
        return (_normal(g, total // STATE_BLOCK, STATE_BLOCK) * size).flatten().mul_(real)
    grad = like_grad()
    if case["bf16_grad"]:
        grad = grad.bfloat16()
    first = case["step"] == 1
    m = like_grad().mul_(0.3).mul_(0.0 if first else 1.0)
    v = like_grad().square_().add_(like_grad().square_()).mul_(0.0 if first else 0.4)
    s = {"case": case, "p": p, "g": grad, "b": p.bfloat16(), "ms": None, "vs": None,
         "hyper": {"lr": 2e-4, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 0.01},
         "max_norm": 0.3}
    if case["bits"] == 8:
        s["m"], s["ms"] = _encode_m(m.view(-1, STATE_BLOCK), 0)
        s["v"], s["vs"] = _encode_v(v.view(-1, STATE_BLOCK), 0)
    else:
        s["m"], s["v"] = m, v
    if own:
        import bit_nf4_quantized_22_amd as qn
        part = lambda t: [t[o:o + n] for o, n in zip(starts, sizes)]
        blocks = lambda t: [t[o // STATE_BLOCK:(o + _padded(n)) // STATE_BLOCK]
                            for o, n in zip(starts, sizes)]
        eight = case["bits"] == 8
        s["table"] = qn.lora_adamw_table(
            part(s["p"]), part(s["g"]), part(s["m"]), part(s["v"]),
            m_scales=blocks(s["ms"]) if eight else None,
            v_scales=blocks(s["vs"]) if eight else None, p_bf16s=part(s["b"]))
        s["norm"] = torch.empty(2, device=DEV)
        s["ws"] = qn.workspace(qn.lora_grad_norm_workspace_bytes(s["table"]), DEV)
    return s


# --- one pass ----------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if op == "quantise":
        if own:
            import bit_nf4_quantized_22_amd as qn
            return qn.fp8_quantize_blocks(state["w"])
        return _quantise_blocks(state["w"])
    if op == "adamw":
        return _adamw_own(state) if own else _adamw_plain(state)
    return _linear_own(state) if own else _linear_plain(state)


def _linear_own(s):
    import bit_nf4_quantized_22_amd as qn
    x, r = s["x"], s["r"]
    saved = torch.empty((x.shape[0], r), dtype=torch.bfloat16, device=DEV) if r else None
    if s["case"]["op"] == "fwd":
        out = qn.fp8_linear_fwd(s["weight"], x, s["A"], s["B"], r, s["alpha"], u_out=saved,
                                ws=s["ws"])
    else:
        out = qn.fp8_linear_bwd_dx(s["weight"], x, s["A"], s["B"], r, s["alpha"], t_out=saved,
                                   ws=s["ws"])
    return [out, saved] if r else [out]


def _adamw_own(s):
    import bit_nf4_quantized_22_amd as qn
    coef = None
    if s["case"]["clip"]:
        qn.lora_grad_norm(s["table"], s["max_norm"], out=s["norm"], ws=s["ws"])
        coef = s["norm"][1:]
    qn.lora_adamw_multi_step(s["table"], s["case"]["step"], grad_scale=coef, **s["hyper"])
    return _adamw_outputs(s, s["norm"][0] if s["case"]["clip"] else None)


def _adamw_outputs(s, norm):
    return {"p": s["p"], "b": s["b"], "m": s["m"], "v": s["v"], "ms": s["ms"], "vs": s["vs"],
            "norm": norm}


# --- plain forms -------------------------------------------------------------

def _pad_to(t, rows, cols):
    return torch.nn.functional.pad(t, (0, cols - t.shape[1], 0, rows - t.shape[0]))


def _up(n, b):
    return -(-n // b) * b


def _scale(amax, top):
    """fl32(amax / top), at least FLOOR (a quotient of two tensors: by a plain
    number the device multiplies with its reciprocal, another rounding)."""
    return (amax / torch.full_like(amax, top)).clamp_min(FLOOR)


def _ratio(t, s):
    """fl32(t / s) within the codes' range.  The quotient is taken in 64 bits:
    bf16 values often lie exactly between two codes, where the last bit of a
    32-bit quotient decides."""
    return (t.double() / s.double()).float().clamp(-F8_MAX, F8_MAX)


def _quantise_blocks(w):
    """E4M3 codes [N, K] and the scale of each 128 x 128 block."""
    N, K = w.shape
    nb, kb = _up(N, BLOCK) // BLOCK, _up(K, BLOCK) // BLOCK
    t = _pad_to(w.float(), nb * BLOCK, kb * BLOCK).view(nb, BLOCK, kb, BLOCK)
    s = _scale(t.abs().amax(dim=(1, 3)), F8_MAX)
    q = _ratio(t, s[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)
    return q[:N, :K].to(E4M3).contiguous(), s


def _quantised_rows(x):
    """x as the values that its E4M3 codes, scaled per row and 128 columns, stand for."""
    M, K = x.shape
    kb = _up(K, BLOCK) // BLOCK
    t = _pad_to(x.float(), M, kb * BLOCK).view(M, kb, BLOCK)
    s = _scale(t.abs().amax(dim=2, keepdim=True), F8_MAX)
    q = _ratio(t, s).to(E4M3).float()
    return (q * s).view(M, kb * BLOCK)[:, :K]


def _weight_values(codes, scale):
    s = scale.repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
    return codes.float() * s[:codes.shape[0], :codes.shape[1]]


def _linear_plain(s):
    x, r = s["x"], s["r"]
    w = _weight_values(s["codes"], s["scale"])
    fwd = s["case"]["op"] == "fwd"
    out = _quantised_rows(x) @ (w.t() if fwd else w)
    if not r:
        return [out.bfloat16()]
    A, B, xf = s["A"].float(), s["B"].float(), x.float()
    low = xf @ A.t() if fwd else xf @ B
    up = low @ (B.t() if fwd else A)
    return [(out + (s["alpha"] / r) * up).bfloat16(), low.bfloat16()]


def _dither(step):
    i = torch.arange(STATE_BLOCK, device=DEV, dtype=torch.int64)
    return (i * DITHER_I + step * DITHER_T) & 0xFFFFFFFF


def _encode(n, d, shift, offset, least, sub, most):
    """Codes of n >= 0: the fp32 bits plus the dither d, cut to the code's
    mantissa; below the least normal number the same on a fixed grid."""
    normal = ((n.view(torch.int32) + d) >> shift) - offset
    small = ((n * sub).to(torch.int32) + d) >> shift
    return torch.where(n >= least, normal, small).clamp_max(most)


def _encode_m(m, step):
    s = _scale(m.abs().amax(dim=1, keepdim=True), F8_MAX)
    n = (m.abs() * (1.0 / s)).clamp_max(F8_MAX)
    c = _encode(n, (_dither(step) >> 12).int(), 20, 960, 2.0 ** -6, 2.0 ** 29, 0x7E)
    c = c + 128 * (m < 0).int()
    return c.to(torch.uint8).view(E4M3).flatten(), s.flatten()


def _encode_v(v, step):
    s = _scale(v.amax(dim=1, keepdim=True), F5_MAX)
    n = (v * (1.0 / s)).clamp_max(F5_MAX)
    c = _encode(n, ((_dither(step) ^ 0xFFFFFFFF) >> 11).int(), 21, 448, 2.0 ** -14, 2.0 ** 37,
                0x7B)
    c = torch.where(v > 0, c.clamp_min(1), torch.zeros_like(c))
    return c.to(torch.uint8).view(E5M2).flatten(), s.flatten()


def _adamw_plain(s):
    case, h = s["case"], s["hyper"]
    f32 = lambda a: float(torch.tensor(a, dtype=torch.float32))
    lr, wd, eps = f32(h["lr"]), f32(h["weight_decay"]), f32(h["eps"])
    b1, b2 = f32(h["betas"][0]), f32(h["betas"][1])
    g, norm = s["g"].float(), None
    if case["clip"]:
        norm = g.double().square().sum().sqrt()
        g = g * (s["max_norm"] / (norm + 1e-6)).clamp_max(1.0).float()
        norm = norm.float()
    m, v = s["m"], s["v"]
    if case["bits"] == 8:
        m = (m.float().view(-1, STATE_BLOCK) * s["ms"][:, None]).flatten()
        v = (v.float().view(-1, STATE_BLOCK) * s["vs"][:, None]).flatten()
    m = m * b1 + g * f32(1.0 - b1)
    v = v * b2 + (g * g) * f32(1.0 - b2)
    den = v.sqrt() * f32(1.0 / math.sqrt(1.0 - b2 ** case["step"])) + eps
    s["p"].mul_(f32(1.0 - lr * wd)).sub_((m / den) * f32(lr / (1.0 - b1 ** case["step"])))
    s["b"].copy_(s["p"])
    if case["bits"] == 8:
        (mc, ms), (vc, vs) = (_encode_m(m.view(-1, STATE_BLOCK), case["step"]),
                              _encode_v(v.view(-1, STATE_BLOCK), case["step"]))
        for old, new in ((s["m"], mc), (s["v"], vc), (s["ms"], ms), (s["vs"], vs)):
            old.copy_(new)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adamw_outputs(s, norm)


# --- bytes and operations ----------------------------------------------------

def work(case):
    if case["op"] == "quantise":
        n = case["N"] * case["K"]
        return {"bytes": n * (2 if case["bf16"] else 4) + n + 4 * n / BLOCK ** 2, "flops": 4 * n}
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        state = 16 if case["bits"] == 32 else 4 + 16 / STATE_BLOCK
        grad = 2 if case["bf16_grad"] else 4
        # p read and written, its bf16 copy written, g read, both states read and written
        return {"bytes": n * (8 + 2 + grad + state), "flops": n * (20 if case["clip"] else 18)}
    M, N, K, r = case["M"], case["N"], case["K"], case["r"]
    scales = 4 * _up(N, BLOCK) * _up(K, BLOCK) / BLOCK ** 2
    return {"bytes": 2 * M * (K + N) + N * K + scales + 2 * r * (N + K + M),
            "flops": 2 * M * N * K + 2 * M * r * (N + K)}


# --- the definitions in 64 bits ----------------------------------------------

def _round8(x, mant, least_exp, u):
    """|x| cut to `mant` mantissa bits, exponents from least_exp: nearest with
    ties to even where u is None, else up where the fraction reaches 1 - u."""
    e = torch.frexp(x)[1].double() - 1
    step = torch.exp2(e.clamp_min(least_exp) - mant)
    k = x / step
    return (torch.round(k) if u is None else torch.floor(k + u)) * step


def _exact_scale(amax, top):
    """A scale is a stored fp32 number: its rounding is part of the definition."""
    return (amax.double() / top).float().double().clamp_min(FLOOR)


def _exact_codes(t, s):
    # the code is defined as the one nearest to the quotient's fp32 rounding
    return torch.sign(t) * _round8((t.abs() / s).float().double(), 3, -6, None).clamp_max(F8_MAX)


def _exact_rows(x):
    M, K = x.shape
    out = torch.zeros(M, K, dtype=torch.float64, device=DEV)
    for k in range(0, K, BLOCK):
        t = x[:, k:k + BLOCK].double()
        s = _exact_scale(t.abs().max(dim=1, keepdim=True)[0], F8_MAX)
        out[:, k:k + BLOCK] = _exact_codes(t, s) * s
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        w = s["w"].double()
        codes = torch.empty_like(w)
        scale = torch.empty(_up(w.shape[0], BLOCK) // BLOCK, _up(w.shape[1], BLOCK) // BLOCK,
                            dtype=torch.float64, device=DEV)
        for i in range(scale.shape[0]):
            for j in range(scale.shape[1]):
                at = (slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
                scale[i, j] = _exact_scale(w[at].abs().max(), F8_MAX)
                codes[at] = _exact_codes(w[at], scale[i, j])
        return codes, scale
    if case["op"] == "adamw":
        return _exact_adamw(s)
    codes, scale, r = s["codes"].double(), s["scale"].double(), s["r"]
    for i in range(scale.shape[0]):
        rows = slice(i * BLOCK, (i + 1) * BLOCK)
        codes[rows] *= scale[i].repeat_interleave(BLOCK)[:codes.shape[1]]
    fwd = case["op"] == "fwd"
    out = _exact_rows(s["x"]).matmul(codes.t().contiguous() if fwd else codes)
    if not r:
        return [out]
    x, A, B = s["x"].double(), s["A"].double(), s["B"].double()
    low = x.matmul(A.t().contiguous() if fwd else B)
    out += (s["alpha"] / r) * low.matmul(B.t().contiguous() if fwd else A)
    return [out, low]


def _exact_adamw(s):
    case, t = s["case"], s["case"]["step"]
    # the hyperparameters are fp32 numbers of the call; all else is in 64 bits
    f32 = lambda a: torch.tensor(a, dtype=torch.float32).item()
    h = {k: f32(a) for k, a in s["hyper"].items() if k != "betas"}
    b1, b2 = (f32(b) for b in s["hyper"]["betas"])
    g, norm = s["g"].double(), None
    if case["clip"]:
        norm = torch.linalg.vector_norm(g)
        g = g * min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    m, v = s["m"].double(), s["v"].double()
    if case["bits"] == 8:
        m = m * s["ms"].double().repeat_interleave(STATE_BLOCK)
        v = v * s["vs"].double().repeat_interleave(STATE_BLOCK)
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    p = s["p"].double() * (1 - h["lr"] * h["weight_decay"])
    p -= h["lr"] * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + h["eps"])
    got = {"p": p, "b": p, "m": m, "v": v, "ms": None, "vs": None, "norm": norm}
    if case["bits"] == 8:
        u = (_dither(t) >> 12).double() / 2.0 ** 20
        w = ((0xFFFFFFFF - _dither(t)) >> 11).double() / 2.0 ** 21
        mb, vb = m.view(-1, STATE_BLOCK), v.view(-1, STATE_BLOCK)
        ms = (mb.abs().max(dim=1, keepdim=True)[0] / F8_MAX).clamp_min(FLOOR)
        vs = (vb.max(dim=1, keepdim=True)[0] / F5_MAX).clamp_min(FLOOR)
        got["m"] = (torch.sign(mb) * _round8(mb.abs() / ms, 3, -6, u).clamp_max(F8_MAX)).flatten()
        vq = _round8(vb / vs, 2, -14, w).clamp_max(F5_MAX)
        got["v"] = torch.where(vb > 0, vq.clamp_min(2.0 ** -16), vq).flatten()
        got["ms"], got["vs"] = ms.flatten(), vs.flatten()
    return got
