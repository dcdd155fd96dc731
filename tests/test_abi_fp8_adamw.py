"""Host-side checks of the FP8 layer and of AdamW over many matrices (CPU:
nothing here launches a kernel)."""

import ctypes

import numpy as np
import pytest

import bit_nf4_quantized_22_amd as qn
from tests.test_abi import FAKE, ODD, lib  # noqa: F401

BIG = 1 << 40


def fp8_w(codes=0x100000, scale=0x100000, N=128, K=128):
    return ctypes.byref(qn.qn_fp8_weight(codes, scale, N, K))


def test_fp8_quantiser_argument_errors(lib):  # noqa: F811
    f = lib.fp8_quantize_blocks
    assert f(FAKE, 2, 16, 16, FAKE, FAKE, None) == qn.QN_ERR_UNSUPPORTED
    for n, k in ((8, 16), (16, 24), (-16, 16), (16, -16), (1 << 24, 16), (1 << 23, 1 << 23)):
        assert f(FAKE, qn.QN_F32, n, k, FAKE, FAKE, None) == qn.QN_ERR_SHAPE
    for a in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None)):
        assert f(a[0], qn.QN_BF16, 16, 16, a[1], a[2], None) == qn.QN_ERR_NULL
    assert f(ODD, qn.QN_BF16, 16, 16, FAKE, FAKE, None) == qn.QN_ERR_ALIGN
    assert f(FAKE, qn.QN_BF16, 16, 16, ODD, FAKE, None) == qn.QN_ERR_ALIGN
    assert f(FAKE, qn.QN_BF16, 16, 16, FAKE, ODD, None) == qn.QN_ERR_ALIGN
    assert f(None, qn.QN_BF16, 0, 16, None, None, None) == qn.QN_OK
    f = lib.fp8_quantize_rows
    for m, k in ((-1, 16), (1, 8), (1, -16), (1 << 32, 16), (1 << 20, 1 << 20)):
        assert f(FAKE, m, k, FAKE, FAKE, None) == qn.QN_ERR_SHAPE
    assert f(None, 1, 16, FAKE, FAKE, None) == qn.QN_ERR_NULL
    assert f(FAKE, 1, 16, ODD, FAKE, None) == qn.QN_ERR_ALIGN
    assert f(None, 0, 16, None, None, None) == qn.QN_OK


def test_fp8_weight_checks(lib):  # noqa: F811
    need = qn.qn_workspace_bytes(qn.QN_OP_FP8_FWD, 32, 128, 128, 8)
    bad = [(fp8_w(codes=None), qn.QN_ERR_NULL), (fp8_w(scale=None), qn.QN_ERR_NULL),
           (fp8_w(codes=0x100008), qn.QN_ERR_ALIGN), (fp8_w(scale=0x100001), qn.QN_ERR_ALIGN),
           (fp8_w(N=0), qn.QN_ERR_SHAPE), (fp8_w(K=0), qn.QN_ERR_SHAPE),
           (fp8_w(N=120), qn.QN_ERR_SHAPE), (fp8_w(K=-16), qn.QN_ERR_SHAPE),
           (fp8_w(N=(1 << 23) + 16), qn.QN_ERR_SHAPE), (None, qn.QN_ERR_NULL)]
    for w, status in bad:
        assert lib.fp8_dequant(w, qn.QN_F32, FAKE, None) == status
        assert lib.fp8_matmul(w, FAKE, FAKE, 1, 0, FAKE, FAKE, need, None) == status
        for f in (lib.fp8_linear_fwd, lib.fp8_linear_bwd_dx):
            assert f(w, FAKE, 32, FAKE, FAKE, 8, 16.0, FAKE, None, FAKE, need, None) == status


def test_fp8_product_argument_errors(lib):  # noqa: F811
    need = qn.qn_workspace_bytes(qn.QN_OP_FP8_BWD_DX, 80, 128, 128, 0)

    def f(x=FAKE, s=FAKE, M=80, tr=1, out=FAKE, ws=FAKE, n=need):
        return lib.fp8_matmul(fp8_w(), x, s, M, tr, out, ws, n, None)

    assert f(tr=2) == qn.QN_ERR_UNSUPPORTED
    assert f(M=-1) == qn.QN_ERR_SHAPE
    assert f(M=BIG) == qn.QN_ERR_SHAPE
    assert f(x=None, s=None, M=0, out=None, ws=None, n=0) == qn.QN_OK
    for k in ("x", "s", "out"):
        assert f(**{k: None}) == qn.QN_ERR_NULL
    for k in ("x", "s", "out", "ws"):
        assert f(**{k: ODD}) == qn.QN_ERR_ALIGN
    assert f(ws=None) == qn.QN_ERR_WORKSPACE
    assert f(n=need - 1) == qn.QN_ERR_WORKSPACE
    assert lib.fp8_dequant(fp8_w(), 2, FAKE, None) == qn.QN_ERR_UNSUPPORTED
    assert lib.fp8_dequant(fp8_w(), qn.QN_F32, None, None) == qn.QN_ERR_NULL
    assert lib.fp8_dequant(fp8_w(), qn.QN_F32, ODD, None) == qn.QN_ERR_ALIGN


@pytest.mark.parametrize("name,op", [("fp8_linear_fwd", qn.QN_OP_FP8_FWD),
                                     ("fp8_linear_bwd_dx", qn.QN_OP_FP8_BWD_DX)])
def test_fp8_linear_argument_errors(lib, name, op):  # noqa: F811
    f = getattr(lib, name)
    need = qn.qn_workspace_bytes(op, 32, 128, 128, 8)

    def call(w=fp8_w(), x=FAKE, M=32, A=FAKE, B=FAKE, r=8, out=FAKE, low=None, ws=FAKE,
             n=need):
        return f(w, x, M, A, B, r, 16.0, out, low, ws, n, None)

    assert call(M=-1) == qn.QN_ERR_SHAPE
    assert call(M=BIG) == qn.QN_ERR_SHAPE
    assert call(r=-1) == qn.QN_ERR_SHAPE
    assert call(r=129) == qn.QN_ERR_UNSUPPORTED
    assert call(M=0, x=None, out=None, ws=None, n=0) == qn.QN_OK
    assert call(A=None) == qn.QN_ERR_NULL
    assert call(B=None) == qn.QN_ERR_NULL
    assert call(x=None) == qn.QN_ERR_NULL
    assert call(out=None) == qn.QN_ERR_NULL
    for k in ("x", "out", "A", "B", "low", "ws"):
        assert call(**{k: ODD}) == qn.QN_ERR_ALIGN
    assert call(ws=None) == qn.QN_ERR_WORKSPACE
    assert call(n=need - 1) == qn.QN_ERR_WORKSPACE
    # the frozen layer still needs room for its input's codes
    assert call(A=None, B=None, n=32 * 128 - 1) == qn.QN_ERR_WORKSPACE
    assert call(A=None, B=None, out=ODD) == qn.QN_ERR_ALIGN


def test_fp8_workspace_sizes(lib):  # noqa: F811
    w = qn.qn_workspace_bytes
    assert w(qn.QN_OP_FP8_FWD, 0, 128, 128, 8) == 0
    assert w(qn.QN_OP_FP8_FWD, -1, 128, 128, 8) == 0
    assert w(qn.QN_OP_FP8_FWD, 100, 4096, 1024, 0) >= 100 * 1024 + 8 * 100 * 4
    assert w(qn.QN_OP_FP8_BWD_DX, 100, 4096, 1024, 0) >= 100 * 4096 + 32 * 100 * 4
    assert w(qn.QN_OP_FP8_FWD, 100, 64, 1024, 16) > w(qn.QN_OP_FP8_FWD, 100, 64, 1024, 0)


def table(tensors, grad=qn.QN_F32, state=qn.QN_STATE_F32, room=None):
    arr = (qn.qn_adamw_tensor * max(1, len(tensors)))(*[qn.qn_adamw_tensor(*t) for t in tensors])
    lib_ = qn.load_library()
    size = lib_.lora_adamw_table_bytes(arr, len(tensors))
    buf = np.zeros(max(8, size) // 8 + 1, np.uint64)
    plan = qn.qn_adamw_plan()
    st = lib_.lora_adamw_table(arr, len(tensors), grad, state, buf.ctypes.data,
                               size if room is None else room, ctypes.byref(plan))
    return st, plan, size


def one(at=0x1000000, n=1000, **kw):
    """A matrix whose operands lie 64 KiB apart from `at` on."""
    t = dict(p=at, g=at + 0x10000, m=at + 0x20000, v=at + 0x30000, ms=at + 0x40000,
             vs=at + 0x50000, b=at + 0x60000, n=n)
    t.update(kw)
    return tuple(t.values())


def test_adamw_table_contents(lib):  # noqa: F811
    st, plan, size = table([one(), one(0x2000000, n=0), one(0x3000000, n=4097)])
    assert st == qn.QN_OK
    assert (plan.chunks, plan.bytes, size) == (4, 4 * 64, 4 * 64)
    st, plan, size = table([])
    assert st == qn.QN_OK and (plan.chunks, size) == (0, 0)
    assert lib.lora_grad_norm_workspace_bytes(ctypes.byref(plan)) == 0


def test_adamw_table_argument_errors(lib):  # noqa: F811
    assert table([one()], grad=2)[0] == qn.QN_ERR_UNSUPPORTED
    assert table([one()], state=2)[0] == qn.QN_ERR_UNSUPPORTED
    assert table([one(n=-1)])[0] == qn.QN_ERR_SHAPE
    assert table([one(n=1 << 43)])[0] == qn.QN_ERR_SHAPE
    assert table([one()], room=8)[0] == qn.QN_ERR_WORKSPACE
    for k in ("p", "g", "m", "v"):
        assert table([one(**{k: None})])[0] == qn.QN_ERR_NULL
        assert table([one(**{k: 0x5000008})])[0] == qn.QN_ERR_ALIGN
    assert table([one(b=0x5000008)])[0] == qn.QN_ERR_ALIGN
    assert table([one(b=None, ms=None, vs=None)])[0] == qn.QN_OK
    for k in ("ms", "vs"):
        assert table([one(**{k: None})], state=qn.QN_STATE_8BIT)[0] == qn.QN_ERR_NULL
        assert table([one(**{k: 0x5000002})], state=qn.QN_STATE_8BIT)[0] == qn.QN_ERR_ALIGN
    # a matrix without elements is not read
    assert table([one(n=0, p=None, g=3, m=None)])[0] == qn.QN_OK


def test_adamw_table_refuses_overlaps(lib):  # noqa: F811
    assert table([one(), one(0x2000000)])[0] == qn.QN_OK
    assert table([one(), one()])[0] == qn.QN_ERR_SHAPE               # the same matrix twice
    assert table([one(), one(0x2000000, m=0x1020000)])[0] == qn.QN_ERR_SHAPE
    assert table([one(g=0x1000000)])[0] == qn.QN_ERR_SHAPE            # gradient inside p
    assert table([one(v=0x1020000)])[0] == qn.QN_ERR_SHAPE            # m and v in one place
    assert table([one(), one(0x2000000, g=0x1010000)])[0] == qn.QN_OK  # a shared gradient
    # neighbours that touch are fine, by one element they are not
    a = one(n=64)
    assert table([a, one(0x1000100, g=0x2010000, m=0x2020000, v=0x2030000, b=0x2060000,
                         n=64)])[0] == qn.QN_OK
    assert table([a, one(0x10000F0, g=0x2010000, m=0x2020000, v=0x2030000, b=0x2060000,
                         n=64)])[0] == qn.QN_ERR_SHAPE
    # the scales count for 8-bit states only
    twice = [one(), one(0x2000000, ms=0x1040000)]
    assert table(twice)[0] == qn.QN_OK
    assert table(twice, state=qn.QN_STATE_8BIT)[0] == qn.QN_ERR_SHAPE


def test_adamw_multi_step_and_norm_argument_errors(lib):  # noqa: F811
    st, plan, _ = table([one()])
    assert st == qn.QN_OK
    hyper = dict(lr=2e-4, b1=0.9, b2=0.999, eps=1e-8, wd=0.0)

    def step(plan=plan, tab=FAKE, c=None, step_=1, **kw):
        h = dict(hyper, **kw)
        return lib.lora_adamw_multi_step(None if plan is None else ctypes.byref(plan), tab, c,
                                         h["lr"], h["b1"], h["b2"], h["eps"], h["wd"], step_,
                                         None)

    assert step(plan=None) == qn.QN_ERR_NULL
    assert step(tab=None) == qn.QN_ERR_NULL
    assert step(tab=ODD) == qn.QN_ERR_ALIGN
    assert step(c=ODD) == qn.QN_ERR_ALIGN
    assert step(step_=0) == qn.QN_ERR_SHAPE
    assert step(lr=-1.0) == qn.QN_ERR_SHAPE
    assert step(b1=1.0) == qn.QN_ERR_SHAPE
    assert step(b2=float("nan")) == qn.QN_ERR_SHAPE
    assert step(eps=0.0) == qn.QN_ERR_SHAPE
    assert step(wd=-1.0) == qn.QN_ERR_SHAPE
    for field, value, status in (("state", 2, qn.QN_ERR_UNSUPPORTED),
                                 ("grad_dtype", 5, qn.QN_ERR_UNSUPPORTED),
                                 ("chunks", 7, qn.QN_ERR_SHAPE), ("chunks", -1, qn.QN_ERR_SHAPE),
                                 ("bytes", 0, qn.QN_ERR_SHAPE)):
        p = qn.qn_adamw_plan.from_buffer_copy(plan)
        setattr(p, field, value)
        assert step(plan=p) == status

    def norm(max_norm=1.0, out=FAKE, ws=FAKE, n=1 << 20, tab=FAKE):
        return lib.lora_grad_norm(ctypes.byref(plan), tab, max_norm, out, ws, n, None)

    assert norm(tab=None) == qn.QN_ERR_NULL
    assert norm(out=None) == qn.QN_ERR_NULL
    assert norm(out=ODD) == qn.QN_ERR_ALIGN
    assert norm(max_norm=0.0) == qn.QN_ERR_SHAPE
    assert norm(max_norm=float("nan")) == qn.QN_ERR_SHAPE
    assert norm(ws=None) == qn.QN_ERR_WORKSPACE
    assert norm(n=7) == qn.QN_ERR_WORKSPACE
    assert norm(ws=ctypes.c_void_p(0x100004)) == qn.QN_ERR_ALIGN
    # a table without elements has nothing to step over
    _, empty, _ = table([])
    assert step(plan=empty, tab=None) == qn.QN_OK


def test_binding_refuses_host_and_mistyped_tensors():
    import torch
    w = torch.zeros(16, 16)
    with pytest.raises(ValueError):
        qn.fp8_quantize_blocks(w)
    with pytest.raises(ValueError):
        qn.Fp8Weight(torch.zeros(16, 16, dtype=torch.uint8), torch.zeros(1))
    with pytest.raises(ValueError):
        qn.lora_adamw_table([], [], [], [])
    with pytest.raises(ValueError):
        qn.lora_adamw_table([w], [w], [w], [w])
    with pytest.raises(ValueError):
        qn.lora_adamw_table([w], [w.half()], [w], [w])


def test_sizes_beyond_a_launch_are_refused(lib):  # noqa: F811
    """A launch has less than 2^32 threads."""
    row = lib.fp8_quantize_rows
    assert row(FAKE, (1 << 26) + 1, 16, FAKE, FAKE, None) == qn.QN_ERR_SHAPE
    assert row(FAKE, (1 << 24) + 1, 1024, FAKE, FAKE, None) == qn.QN_ERR_SHAPE
    assert lib.fp8_quantize_blocks(FAKE, qn.QN_BF16, 1 << 19, 1 << 19, FAKE, FAKE,
                                   None) == qn.QN_ERR_SHAPE
    assert lib.fp8_dequant(fp8_w(N=1 << 18, K=(1 << 17) + 16), qn.QN_BF16, FAKE,
                           None) == qn.QN_ERR_SHAPE
    for f in (lib.fp8_linear_fwd, lib.fp8_linear_bwd_dx):
        for N, K in ((1 << 16, 16), (16, 1 << 16)):
            assert f(fp8_w(N=N, K=K), FAKE, (1 << 18) + 1, None, None, 0, 1.0, FAKE, None, FAKE,
                     BIG, None) == qn.QN_ERR_SHAPE
    n = 2048 * ((1 << 24) - 1)
    big = (qn.qn_adamw_tensor * 1)(qn.qn_adamw_tensor(*one(n=n)))
    assert lib.lora_adamw_table_bytes(big, 1) == 64 * ((1 << 24) - 1)
    big[0].n = n + 1
    assert lib.lora_adamw_table_bytes(big, 1) == 0
    assert table([one(n=n + 1)])[0] == qn.QN_ERR_SHAPE
