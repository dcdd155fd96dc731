"""Host-side checks of the Muon step (CPU: nothing here launches a kernel)."""

import ctypes

import numpy as np
import pytest

import bit_nf4_quantized_22_amd as qn
from tests.test_abi import FAKE, ODD, lib  # noqa: F401

A = 1 << 20


def tensors(*rows):
    """Rows of (rows, cols) or of all six fields; memory far apart."""
    arr = (qn.qn_muon_tensor * max(1, len(rows)))()
    for i, r in enumerate(rows):
        if len(r) == 2:
            base = (4 * i + 1) << 44
            r = tuple(base + (j << 42) for j in range(4)) + tuple(r)
        arr[i] = qn.qn_muon_tensor(*r)
    return arr


def build(arr, count=None, grad=qn.QN_F32, room=None):
    lib = qn.load_library()  # noqa: F811
    n = len(arr) if count is None else count
    size = lib.lora_muon_table_bytes(arr, n)
    host = np.zeros(max(size, 1) + 16, np.uint8)
    plan = qn.qn_muon_plan()
    st = lib.lora_muon_table(arr, n, grad, host.ctypes.data, size if room is None else room,
                             ctypes.byref(plan))
    return st, plan, host, size


def hyper(lr=1e-3, momentum=0.95, weight_decay=0.1, eps=1e-7, ns=(3.4445, -4.775, 2.0315),
          ns_steps=5, nesterov=1, adjust=0):
    return qn.qn_muon_step(lr, momentum, weight_decay, eps, (ctypes.c_double * 3)(*ns), ns_steps,
                           nesterov, adjust)


def parse(plan, host, size):
    """Matrices as (64-bit fields, 32-bit fields), entries as [matrix, index]."""
    n = sum(plan.matrices)
    wide = host[:n * 88].view(np.int64).reshape(n, 11)
    small = host[:n * 88].view(np.int32).reshape(n, 22)[:, 18:]
    return wide, small, host[n * 88:size].view(np.int32).reshape(-1, 2)


LEN, CHUNK, SPAN, PART, FACTOR = range(4, 9)


def test_table_counts_and_order(lib):  # noqa: F811
    shapes = [(128, 300), (16, 16), (5000, 17), (1, 9), (0, 7), (64, 64), (33, 40), (7, 0)]
    st, plan, host, size = build(tensors(*shapes))
    assert st == qn.QN_OK and plan.bytes == size
    assert list(plan.matrices) == [2, 1, 2, 1]
    # few matrices: a chunk and a span for each run of 256 or 128
    assert list(plan.chunks) == list(plan.spans) == [2, 40, 2, 2]
    assert size == 6 * 88 + 2 * 46 * 8
    # doubles: a chunk's sums, and the factor of each matrix
    want = sum(c * t * (t + 1) // 2 * 256 + m * 256 * t * t
               for c, m, t in zip(plan.chunks, plan.matrices, (1, 2, 4, 8)))
    assert lib.lora_muon_workspace_bytes(ctypes.byref(plan)) == plan.ws_bytes == 8 * want
    # the entries lie by class, each with its own room
    wide, small, entries = parse(plan, host, size)
    assert wide[:, LEN].tolist() == [16, 9, 5000, 64, 40, 300]
    assert small[:, 0].tolist() == [16, 1, 17, 64, 33, 128]
    assert small[:, 1].tolist() == [0, 0, 1, 0, 0, 0]
    ends = wide[:, FACTOR] + 256 * np.array([1, 1, 4, 16, 16, 64])
    assert (wide[1:, PART] == ends[:-1]).all() and ends[-1] == want
    at, first = 0, 0
    for m, c, s in zip(plan.matrices, plan.chunks, plan.spans):
        for n, col in ((c, 2), (s, 3)):
            part = entries[at:at + n]
            assert (np.bincount(part[:, 0] - first, minlength=m) == small[first:first + m, col]).all()
            at += n
        first += m
    assert at == len(entries)


def test_long_matrices_and_many(lib):  # noqa: F811
    st, plan, host, size = build(tensors((16, 10_000_000), (2 ** 24 - 1, 1)))
    assert st == qn.QN_OK and sum(plan.chunks) <= 512 and sum(plan.spans) >= 2048
    for shape in ((16, 4096), (64, 4096)):
        st, plan, host, size = build(tensors(*[shape] * 448))
        wide, small, _ = parse(plan, host, size)
        # nearly equal parts of the 16 runs, for either pass
        for length, count in ((CHUNK, 2), (SPAN, 3)):
            assert st == qn.QN_OK and (wide[:, length] % 128 == 0).all()
            assert (small[:, count] * wide[:, length] >= 4096).all()
            assert ((small[:, count] - 1) * wide[:, length] < 4096).all()
    assert sum(plan.chunks) < sum(plan.spans)


def test_table_refusals(lib):  # noqa: F811
    n = 64 * 4
    good = (A, A + 4 * n, A + 8 * n, A + 12 * n, 4, 64)
    assert build(tensors(good))[0] == qn.QN_OK
    for k in range(3):
        bad = list(good)
        bad[k] = None
        assert build(tensors(tuple(bad)))[0] == qn.QN_ERR_NULL
    for k in range(4):
        bad = list(good)
        bad[k] += 8
        assert build(tensors(tuple(bad)))[0] == qn.QN_ERR_ALIGN
    # p over m, the bf16 copy over p, p over g
    for k, v in ((2, A + 4 * n - 16), (3, A + 16), (1, A)):
        bad = list(good)
        bad[k] = v
        assert build(tensors(tuple(bad)))[0] == qn.QN_ERR_SHAPE
    # the same matrix twice; a shared gradient is fine
    assert build(tensors(good, good))[0] == qn.QN_ERR_SHAPE
    other = (2 * A, good[1], 3 * A, None, 4, 64)
    assert build(tensors(good, other))[0] == qn.QN_OK
    for shape in ((-1, 4), (4, -1), (2 ** 24, 1), (1, 2 ** 40)):
        assert build(tensors(shape))[0] == qn.QN_ERR_SHAPE
        assert lib.lora_muon_table_bytes(tensors(shape), 1) == 0
    assert build(tensors((129, 130)))[0] == qn.QN_ERR_UNSUPPORTED
    assert build(tensors(good), grad=2)[0] == qn.QN_ERR_UNSUPPORTED
    assert build(tensors(good), count=-1)[0] == qn.QN_ERR_SHAPE
    assert build(tensors(good), room=8)[0] == qn.QN_ERR_WORKSPACE
    plan = qn.qn_muon_plan()
    f = lib.lora_muon_table
    assert f(None, 1, 0, FAKE, 1 << 20, ctypes.byref(plan)) == qn.QN_ERR_NULL
    assert f(tensors(good), 1, 0, FAKE, 1 << 20, None) == qn.QN_ERR_NULL
    assert f(tensors(good), 1, 0, None, 1 << 20, ctypes.byref(plan)) == qn.QN_ERR_WORKSPACE
    assert f(tensors(good), 1, 0, ODD, 1 << 20, ctypes.byref(plan)) == qn.QN_ERR_ALIGN
    # nothing to do
    assert f(None, 0, 0, None, 0, ctypes.byref(plan)) == qn.QN_OK and plan.bytes == 0
    assert build(tensors((0, 5)))[0] == qn.QN_OK


def test_step_refusals(lib):  # noqa: F811
    _, plan, _, _ = build(tensors((4, 64)))
    need = plan.ws_bytes

    def f(plan=plan, table=FAKE, step=None, ws=FAKE, n=need, **kw):
        s = hyper(**kw) if step is None else step
        return lib.lora_muon_multi_step(ctypes.byref(plan) if plan else None, table,
                                        ctypes.byref(s) if s else None, ws, n, None)

    assert f(plan=None) == qn.QN_ERR_NULL
    assert f(table=None) == qn.QN_ERR_NULL
    assert f(step=False) == qn.QN_ERR_NULL
    assert f(table=ODD) == qn.QN_ERR_ALIGN
    assert f(ws=ODD) == qn.QN_ERR_ALIGN
    assert f(ws=None) == qn.QN_ERR_WORKSPACE
    assert f(n=need - 1) == qn.QN_ERR_WORKSPACE
    nan = float("nan")
    for kw in ({"lr": -1.0}, {"lr": nan}, {"momentum": 1.0}, {"momentum": -0.1}, {"momentum": nan},
               {"weight_decay": -1.0}, {"weight_decay": nan}, {"eps": 0.0}, {"eps": nan},
               {"ns_steps": 0}, {"ns_steps": 33}, {"ns": (nan, 0, 0)},
               {"ns": (1, float("inf"), 0)}, {"nesterov": 2}):
        assert f(**kw) == qn.QN_ERR_SHAPE, kw
    assert f(adjust=2) == qn.QN_ERR_UNSUPPORTED
    for field, value, want in (("bytes", plan.bytes - 8, qn.QN_ERR_SHAPE),
                               ("ws_bytes", -1, qn.QN_ERR_SHAPE),
                               ("grad_dtype", 2, qn.QN_ERR_UNSUPPORTED)):
        bad = qn.qn_muon_plan.from_buffer_copy(plan)
        setattr(bad, field, value)
        assert f(plan=bad) == want
    _, empty, _, _ = build(tensors((0, 5)))
    assert f(plan=empty, table=None, ws=None, n=0) == qn.QN_OK


@pytest.mark.parametrize("shape", [(1, 1), (16, 257), (17, 129), (129, 33), (100, 100)])
def test_chunks_cover_the_long_side(lib, shape):  # noqa: F811
    _, plan, host, size = build(tensors(shape))
    wide, small, _ = parse(plan, host, size)
    assert wide[0, LEN] == max(shape)
    for length, count, total in ((CHUNK, 2, plan.chunks), (SPAN, 3, plan.spans)):
        n, part = small[0, count], wide[0, length]
        assert sum(total) == n and (n - 1) * part < max(shape) <= n * part
