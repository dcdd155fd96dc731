"""Ways to call the microscaled 4-bit layer (GPU): streams, graphs, batches,
values that are not finite, unaligned adapters, offsets past 32 bits, and a
training step on such a weight."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_22_amd as qn
from oracle import mxfp4
from tests.gpu_helpers import bf16_dev, check, f64, synth, to_np
from tests.test_gpu_mxfp4 import (DEV, acts, bf16_of, layer_bound, rel_to_bound, same_codes,
                                  weights)

pytestmark = pytest.mark.gpu


def weight(N, K, seed):
    return qn.mxfp4_quantize_weight(torch.from_numpy(weights(N, K, seed)).to(DEV))


def adapters(N, K, r, seed):
    rng = np.random.default_rng(seed)
    return tuple(bf16_dev(bf16_of(rng.standard_normal(s) * 0.02)) for s in ((r, K), (N, r)))


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("M", [5, 80])
def test_backward_is_the_forwards_derivative(M):
    """With x on the grid of its own codes and dy on its, both roundings are the
    identity, the layer is linear in x, and dx is the exact transpose of the
    forward within the products' bounds: <dy, f(x)> = <dx, x>.  Differences of
    the forward along one element give its column of W."""
    N, K = 272, 416
    rng = np.random.default_rng(M)
    mw = weight(N, K, 9)
    def on_grid(n, grid, top):
        a = rng.choice(grid, (M, n)) * rng.choice([-1, 1], (M, n))
        a[:, ::16] = top
        return bf16_of(a)
    xb = on_grid(K, mxfp4.E2M1, 6.0)
    dyb = on_grid(N, 2.0 ** np.arange(9), 448.0)
    y = to_np(qn.mxfp4_linear_fwd(mw, bf16_dev(xb), None, None, 0, 1.0)).astype(np.float64)
    dx = to_np(qn.mxfp4_linear_bwd_dx(mw, bf16_dev(dyb), None, None, 0, 1.0)).astype(np.float64)
    x, dy = f64(xb), f64(dyb)
    wv = mxfp4.values(*mxfp4.quantize(weights(N, K, 9)))
    mass = np.sum(np.abs(dy) * (np.abs(x) @ np.abs(wv).T))
    bound = 2.0 ** -8 * (np.sum(np.abs(dy * y)) + np.sum(np.abs(dx * x))) * 1.01 \
        + ((K + N + 8) * 2.0 ** -23 + 7 * 2.0 ** -13) * mass
    assert abs(np.sum(dy * y) - np.sum(dx * x)) <= bound
    # x with one element moved by a code: the difference of y is that column of W
    # times the step, both outputs rounded to bf16
    x2 = x.copy()
    x2[:, 37] = np.where(x[:, 37] >= 4, 3.0, 6.0)
    y2 = to_np(qn.mxfp4_linear_fwd(mw, bf16_dev(bf16_of(x2)), None, None, 0, 1.0)).astype(float)
    step = (x2 - x)[:, 37:38]
    tol = 2.0 ** -8 * 1.01 * (np.abs(y) + np.abs(y2)) + (K + 4) * 2.0 ** -22 * (
        np.abs(x) + np.abs(x2)) @ np.abs(wv).T
    assert (np.abs(y2 - y - step * wv[:, 37]) <= tol).all()
    # and dy with a single row of W: dx is that row
    one = np.zeros((M, N))
    one[:, 11] = 1.0
    got = to_np(qn.mxfp4_linear_bwd_dx(mw, bf16_dev(bf16_of(one)), None, None, 0, 1.0))
    assert np.array_equal(got, np.tile(wv[11].astype(np.float32), (M, 1)))


def test_a_row_does_not_depend_on_its_batch():
    """A padded batch gives its first rows the same bits as a longer one, on
    one path (the decode path and the tiles sum in their own orders)."""
    N, K, r = 272, 1056, 16
    mw = weight(N, K, 1)
    A, B = adapters(N, K, r, 3)
    x = bf16_dev(acts(200, K, 8))
    for few, many in ((2, 16), (3, 16), (48, 64)):
        a = qn.mxfp4_linear_fwd(mw, x[:few], A, B, r, 16.0)
        b = qn.mxfp4_linear_fwd(mw, x[:many], A, B, r, 16.0)
        assert same(a, b[:few])


def test_repeated_calls_and_other_streams_give_the_same_bits():
    M, N, K, r = 200, 528, 800, 24
    mw = weight(N, K, 2)
    A, B = adapters(N, K, r, 11)
    for f, L in ((qn.mxfp4_linear_fwd, K), (qn.mxfp4_linear_bwd_dx, N)):
        x = bf16_dev(acts(M, L, 9))
        first = f(mw, x, A, B, r, 16.0)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = f(mw, x, A, B, r, 16.0)
        torch.cuda.synchronize()
        assert same(first, other)
        # on a given stream with nothing passed in: workspace and output are not
        # memory that the current stream's work still uses or gets next
        for _ in range(10):
            got = f(mw, x, A, B, r, 16.0, stream=side)
            torch.full((first.numel() * 4,), 255, dtype=torch.uint8, device=DEV)
            torch.full(first.shape, 3.0, dtype=torch.bfloat16, device=DEV)
            torch.cuda.synchronize()
            assert same(first, got)


@pytest.mark.parametrize("M", [1, 12, 100])
def test_captured_graph_replays(M):
    N, K, r = 272, 1056, 16
    mw = weight(N, K, 1)
    A, B = adapters(N, K, r, 4)
    x, dy = bf16_dev(acts(M, K, 1)), bf16_dev(acts(M, N, 2))
    y, dx = torch.empty((M, N), dtype=torch.bfloat16, device=DEV), torch.empty_like(x)
    ws = [qn.workspace(qn.qn_workspace_bytes(op, M, N, K, r), DEV)
          for op in (qn.QN_OP_MXFP4_FWD, qn.QN_OP_MXFP4_BWD_DX)]

    def both():
        qn.mxfp4_linear_fwd(mw, x, A, B, r, 16.0, y=y, ws=ws[0])
        qn.mxfp4_linear_bwd_dx(mw, dy, A, B, r, 16.0, dx=dx, ws=ws[1])

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for i in range(4):
        x.copy_(bf16_dev(acts(M, K, 20 + i)))
        dy.copy_(bf16_dev(acts(M, N, 30 + i)))
        both()
        torch.cuda.synchronize()
        want = y.clone(), dx.clone()
        y.zero_(), dx.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(y, want[0]) and same(dx, want[1])


def test_empty_batch_writes_nothing():
    mw = weight(32, 32, 1)
    x = torch.empty((0, 32), dtype=torch.bfloat16, device=DEV)
    assert qn.mxfp4_linear_fwd(mw, x, None, None, 0, 1.0).shape == (0, 32)
    assert qn.mxfp4_linear_bwd_dx(mw, x, None, None, 0, 1.0).shape == (0, 32)
    c, s = qn.mxfp4_quantize(x)
    assert c.shape == (0, 16) and s.numel() == 0
    assert qn.mxfp4_matmul(mw, c, s).shape == (0, 32)
    assert qn.mxfp4_unpack_scales(s, 0, 32).shape == (0, 1)
    torch.cuda.synchronize()


@pytest.mark.parametrize("M", [1, 40, 100])
def test_missing_adapter_is_the_frozen_layer(M):
    mw = weight(144, 288, 3)
    x, dy = bf16_dev(acts(M, 288, 1)), bf16_dev(acts(M, 144, 2))
    for f, v in ((qn.mxfp4_linear_fwd, x), (qn.mxfp4_linear_bwd_dx, dy)):
        assert same(f(mw, v, None, None, 0, 1.0), f(mw, v, None, None, 8, 16.0))
    A = bf16_dev(bf16_of(np.zeros((8, 288))))
    with pytest.raises(qn.QnError):
        qn.mxfp4_linear_fwd(mw, x, A, None, 8, 16.0)


def test_binding_refusals_on_the_device():
    mw = weight(32, 64, 3)
    x = bf16_dev(acts(4, 64, 1))
    c, s = qn.mxfp4_quantize(x)
    bad = [lambda: qn.mxfp4_linear_fwd(mw, x.float(), None, None, 0, 1.0),
           lambda: qn.mxfp4_linear_fwd(mw, x[:, :32], None, None, 0, 1.0),
           lambda: qn.mxfp4_linear_fwd(mw, bf16_dev(acts(64, 4, 1)).t(), None, None, 0, 1.0),
           lambda: qn.mxfp4_linear_fwd(mw, x.cpu(), None, None, 0, 1.0),
           lambda: qn.mxfp4_linear_bwd_dx(mw, x, None, None, 0, 1.0),
           lambda: qn.mxfp4_matmul(mw, x, s),
           lambda: qn.mxfp4_matmul(mw, c[:, :16], s),
           lambda: qn.mxfp4_matmul(mw, c, s[:128]),
           lambda: qn.Mxfp4Weight(mw.codes, mw.scale[:0]),
           lambda: qn.Mxfp4Weight(mw.codes.flatten(), mw.scale),
           lambda: qn.mxfp4_quantize(x.half()),
           lambda: qn.mxfp4_quantize(x.t()),
           lambda: qn.mxfp4_pack_scales(s),
           lambda: qn.mxfp4_unpack_scales(s[:100], 4, 64)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(qn.QnError) as e:      # 48 columns: not a multiple of 32
        qn.mxfp4_quantize(bf16_dev(acts(2, 48, 1)))
    assert e.value.status == qn.QN_ERR_SHAPE
    for f in (qn.mxfp4_linear_fwd, ):
        with pytest.raises(qn.QnError) as e:
            f(mw, x, None, None, 0, 1.0, ws=torch.empty(64, dtype=torch.uint8, device=DEV))
        assert e.value.status == qn.QN_ERR_WORKSPACE
    rows = qn.Mxfp4Weight(c, s)               # 4 rows: no weight
    with pytest.raises(qn.QnError) as e:
        qn.mxfp4_linear_fwd(rows, x, None, None, 0, 1.0)
    assert e.value.status == qn.QN_ERR_SHAPE


# every path: one token, few, some, small tiles (split and not), large tiles
@pytest.mark.parametrize("M,N,K", [(1, 144, 288), (5, 144, 288), (40, 144, 1056), (100, 144, 288),
                                   (80, 1040, 2080), (1100, 4096, 416)])
@pytest.mark.parametrize("r", [0, 16])
def test_a_row_that_is_not_finite_spoils_itself_alone(M, N, K, r):
    mw = weight(N, K, 1)
    A, B = adapters(N, K, r, M) if r else (None, None)
    for f, L in ((qn.mxfp4_linear_fwd, K), (qn.mxfp4_linear_bwd_dx, N)):
        x = bf16_dev(acts(M, L, 8))
        good = f(mw, x, A, B, r, 16.0)
        for row, col, v in ((0, 3, np.nan), (M // 2, L - 1, np.inf), (M - 1, 130, -np.inf)):
            y = x.clone()
            y[row, col] = v
            got = f(mw, y, A, B, r, 16.0)
            assert torch.isnan(got[row]).all()
            got[row] = good[row]
            assert same(got, good)


@pytest.mark.parametrize("M", [1, 5, 100, 1100])
def test_a_group_of_the_weight_that_is_not_finite(M):
    """Its row of W is NaN in y; its 32 columns are in dx."""
    N, K = (4096 if M > 1000 else 144), 416
    w = weights(N, K, 1)
    bad = w.copy()
    bad[100, 70] = np.inf
    rc, rb = mxfp4.quantize(bad)
    assert (rb == 255).sum() == 1 and rb[100, 2] == 255
    good = qn.mxfp4_quantize_weight(torch.from_numpy(w).to(DEV))
    mw = qn.mxfp4_quantize_weight(torch.from_numpy(bad).to(DEV))
    assert same_codes(rc, rb, mw.codes)
    x, dy = bf16_dev(acts(M, K, 5)), bf16_dev(acts(M, N, 6))
    y, want = (qn.mxfp4_linear_fwd(m, x, None, None, 0, 1.0) for m in (mw, good))
    assert torch.isnan(y[:, 100]).all()
    y[:, 100] = want[:, 100]
    assert same(y, want)
    dx, want = (qn.mxfp4_linear_bwd_dx(m, dy, None, None, 0, 1.0) for m in (mw, good))
    assert torch.isnan(dx[:, 64:96]).all()
    dx[:, 64:96] = want[:, 64:96]
    assert same(dx, want)
    val = qn.mxfp4_dequant(mw)
    assert torch.isnan(val[100, 64:96]).all() and torch.isnan(val).sum() == 32


def test_backward_of_rows_with_scales_far_apart():
    """Scales over the whole range within a block of 32 rows: exact up to 2^26
    below the largest, nothing beyond (the documented reading)."""
    N, K, M = 80, 96, 40
    rng = np.random.default_rng(5)
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    byte = rng.integers(100, 130, (N, K // 32)).astype(np.uint8)
    byte[3, 0], byte[40, 1], byte[7, 2] = 140, 90, 60
    byte[32:64, 2] = rng.integers(0, 12, 32)
    mw = qn.Mxfp4Weight(torch.from_numpy(mxfp4.pack(codes)).to(DEV),
                        torch.from_numpy(mxfp4.tiles(byte, N, K)).to(DEV))
    wv = mxfp4.turned_values(mxfp4.values(codes, byte), byte)
    assert (wv == 0).sum() > (codes % 8 == 0).sum()
    dyb = acts(M, N, 3)
    dv = mxfp4.row_values8(f64(dyb))
    dx = qn.mxfp4_linear_bwd_dx(mw, bf16_dev(dyb), None, None, 0, 1.0)
    ref = dv @ wv
    bound = layer_bound(ref, dv, wv, None, None, None, 0.0, N, True)
    assert rel_to_bound(to_np(dx), ref, bound) <= 1
    # one row of W at a time: nothing else hides it, and every product is exact
    one = np.zeros((N, N))
    np.fill_diagonal(one, 1.0)
    dx = qn.mxfp4_linear_bwd_dx(mw, bf16_dev(bf16_of(one)), None, None, 0, 1.0)
    assert np.array_equal(to_np(dx), wv.astype(np.float32))


def test_scales_at_the_ends_of_the_range():
    """The largest and least scales on either side, and their padding: x over
    W's scales must cancel exactly."""
    N, K, M = 16, 352, 20                     # ends inside a run of 256, past 128
    codes = np.full((N, K), 2, np.uint8)      # ones
    xc = np.full((M, K), 2, np.uint8)
    for wb, xb in ((0, 254), (254, 0), (127, 127), (250, 10), (1, 253)):
        if wb + xb < 240:
            continue
        mw = qn.Mxfp4Weight(torch.from_numpy(mxfp4.pack(codes)).to(DEV), torch.from_numpy(
            mxfp4.tiles(np.full((N, K // 32), wb, np.uint8), N, K)).to(DEV))
        s = mxfp4.tiles(np.full((M, K // 32), xb, np.uint8), M, K)
        for m in (M, 100):
            c = torch.from_numpy(mxfp4.pack(np.full((m, K), 2, np.uint8))).to(DEV)
            s = mxfp4.tiles(np.full((m, K // 32), xb, np.uint8), m, K)
            got = to_np(qn.mxfp4_matmul(mw, c, torch.from_numpy(s).to(DEV)))
            assert np.array_equal(got, np.full((m, N), K * 2.0 ** (wb + xb - 254), np.float32))


@pytest.mark.parametrize("M", [1, 5, 40, 100])
@pytest.mark.parametrize("r", [8, 16, 40])
def test_adapters_at_any_element(M, r):
    """A and B need no alignment beyond their elements'."""
    N, K = 272, 544
    mw = weight(N, K, 1)
    A, B = adapters(N, K, r, r)

    def moved(t):
        out = torch.empty(t.numel() + 3, dtype=t.dtype, device=DEV)[3:].view(t.shape)
        out.copy_(t)
        assert out.data_ptr() % 4 == 2
        return out

    for f, L in ((qn.mxfp4_linear_fwd, K), (qn.mxfp4_linear_bwd_dx, N)):
        x = bf16_dev(acts(M, L, 8))
        low, low2 = (torch.empty(M * r + 1, dtype=torch.bfloat16, device=DEV)[1:].view(M, r)
                     for _ in range(2))
        a = f(mw, x, A, B, r, 16.0, None, low)
        b = f(mw, x, moved(A), moved(B), r, 16.0, None, low2)
        assert same(a, b) and same(low, low2)


def random_weight(N, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    b = torch.randint(120, 130, (N, K // 32), generator=g, device=DEV, dtype=torch.uint8)
    return qn.Mxfp4Weight(c, qn.mxfp4_pack_scales(b)), c, b


def near(got, want):
    """Equal products, summed in fp32 in other orders and rounded to bf16: 2^-7
    of the largest, and L / 32 steps of 2^-23 of the terms' magnitude, which is
    below 100 times the largest sum here: less than 2^-8.  2^-6 holds both; a
    wrong address is off by the size of the values."""
    assert torch.isfinite(got.float()).all()
    d = (got.float() - want.float()).abs().max()
    assert d <= 2.0 ** -6 * want.float().abs().max()


def test_offsets_past_32_bits_in_the_weight():
    """A weight of more than 2^32 code bytes: its last columns (rows for the
    backward) are those of a small weight of the same codes."""
    N, K, n0 = 524320, 16416, 524160
    mw, c, b = random_weight(N, K, 1)
    assert mw.codes.numel() > 2 ** 32
    end = qn.Mxfp4Weight(c[n0:], qn.mxfp4_pack_scales(b[n0:].contiguous()))
    for M in (1, 3, 40, 100):
        x = bf16_dev(acts(M, K, M))
        near(qn.mxfp4_linear_fwd(mw, x, None, None, 0, 1.0)[:, n0:],
             qn.mxfp4_linear_fwd(end, x, None, None, 0, 1.0))
    for M in (3, 300):
        dy = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
        dy[:, n0:] = bf16_dev(acts(M, N - n0, M))
        near(qn.mxfp4_linear_bwd_dx(mw, dy, None, None, 0, 1.0),
             qn.mxfp4_linear_bwd_dx(end, dy[:, n0:].contiguous(), None, None, 0, 1.0))
    assert torch.equal(qn.mxfp4_unpack_scales(mw.scale, N, K), b)
    val = qn.mxfp4_dequant(mw)
    assert same(val[n0:], qn.mxfp4_dequant(end))
    c1, s1 = qn.mxfp4_quantize(val)
    c2, s2 = qn.mxfp4_quantize(val[n0:].contiguous())
    assert torch.equal(c1[n0:], c2)
    assert torch.equal(qn.mxfp4_unpack_scales(s1, N, K)[n0:],
                       qn.mxfp4_unpack_scales(s2, N - n0, K))


def test_offsets_past_32_bits_in_the_batch():
    """More than 2^32 bytes of x's codes, and 2^32 values of y."""
    M, L, m0 = 524320, 16416, 524200
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randint(-200, 200, (M, L), generator=g, device=DEV, dtype=torch.int16).bfloat16()
    assert x.numel() > 2 ** 33
    last = x[m0:].contiguous()
    mw = random_weight(144, L, 3)[0]
    A, B = adapters(144, L, 16, 1)
    near(qn.mxfp4_linear_fwd(mw, x, A, B, 16, 16.0)[m0:],
         qn.mxfp4_linear_fwd(mw, last, A, B, 16, 16.0))
    wide = random_weight(L, 160, 4)[0]
    dy = x[:, :160].contiguous()
    near(qn.mxfp4_linear_fwd(wide, dy, None, None, 0, 1.0)[m0:],
         qn.mxfp4_linear_fwd(wide, dy[m0:].contiguous(), None, None, 0, 1.0))
    near(qn.mxfp4_linear_bwd_dx(wide, x, None, None, 0, 1.0)[m0:],
         qn.mxfp4_linear_bwd_dx(wide, last, None, None, 0, 1.0))


@pytest.mark.parametrize("M,N,K", [(64, 4096, 4096), (64, 4112, 8192), (64, 4096, 8160),
                                   (33, 5600, 4000), (17, 8192, 4128), (64, 256, 4096),
                                   (17, 144, 8192), (32, 272, 8160), (17, 16384, 4096)])
def test_batches_at_the_border_between_few_and_tiles(M, N, K):
    """Sizes on both sides of the rule that picks the kernel of 17 to 64
    tokens, with a workspace of the asked size and a guard behind it."""
    r = 16
    w = weights(N, K, M)
    xb = acts(M, K, 3)
    A, B = adapters(N, K, r, N)
    mw = qn.mxfp4_quantize_weight(torch.from_numpy(w).to(DEV))
    xf, Af, Bf = f64(xb), to_np(A).astype(float), to_np(B).astype(float)
    need = qn.qn_workspace_bytes(qn.QN_OP_MXFP4_FWD, M, N, K, r)
    buf = torch.full((need + 4096,), 85, dtype=torch.uint8, device=DEV)
    y = qn.mxfp4_linear_fwd(mw, bf16_dev(xb), A, B, r, 16.0, ws=buf[:need])
    torch.cuda.synchronize()
    assert (buf[need:] == 85).all()
    xv = mxfp4.values(*mxfp4.quantize(xf.astype(np.float32)))
    c = np.unique(np.concatenate([np.arange(0, N, 61), np.arange(N - 16, N)]))
    wc = mxfp4.values(*mxfp4.quantize(w[c]))
    ref = xv @ wc.T + (xf @ Af.T) @ Bf[c].T
    bound = layer_bound(ref, xv, wc.T, xf, Af, Bf[c], 1.0, K, False)
    assert rel_to_bound(to_np(y)[:, c], ref, bound) <= 1


# few tokens, two tiles of 16 rows a workgroup: the last one half empty or not;
# one token in its forms
@pytest.mark.parametrize("M,N,K,r", [(5, 4112, 2080, 16), (16, 4128, 2112, 64), (2, 8192, 2080, 0),
                                     (16, 8176, 2080, 24), (31, 4112, 2080, 16),
                                     (32, 5008, 2112, 128), (17, 8192, 2080, 0),
                                     (1, 4112, 4128, 16), (1, 8192, 1056, 128),
                                     (1, 4112, 544, 17), (1, 4096, 1056, 33), (1, 144, 4096, 16),
                                     (1, 144, 4128, 16), (1, 144, 8192, 8), (1, 5008, 416, 0),
                                     # more pairs of row tiles than CUs
                                     (16, 8208, 2080, 64), (2, 8224, 416, 0), (9, 11008, 544, 128),
                                     (3, 8208, 1312, 7), (32, 8208, 2080, 24), (17, 11008, 32, 0),
                                     (31, 8224, 288, 128)])
def test_few_tokens_with_many_columns(M, N, K, r):
    w = weights(N, K, M)
    xb = acts(M, K, 3)
    A, B = adapters(N, K, r, N) if r else (None, None)
    mw = qn.mxfp4_quantize_weight(torch.from_numpy(w).to(DEV))
    xf = f64(xb)
    y = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    u = torch.empty((M, r), dtype=torch.bfloat16, device=DEV) if r else None
    s = 16.0 / r if r else 0.0
    qn.mxfp4_linear_fwd(mw, bf16_dev(xb), A, B, r, 16.0, y=y[:M * N].view(M, N), u_out=u)
    torch.cuda.synchronize()
    assert torch.all(y[M * N:] == 7.0)
    got = to_np(y[:M * N].view(M, N))
    xv = mxfp4.values(*mxfp4.quantize(xf.astype(np.float32)))
    c = np.unique(np.concatenate([np.arange(0, N, 37), np.arange(N - 48, N)]))
    wc = mxfp4.values(*mxfp4.quantize(w[c]))
    ref = xv @ wc.T
    Af = Bf = None
    if r:
        Af, Bf = to_np(A).astype(float), to_np(B).astype(float)[c]
        ref = ref + s * (xf @ Af.T) @ Bf.T
        bu = 2.0 ** -8 * 1.01 * np.abs(xf @ Af.T) + (K + 4) * 2.0 ** -23 * (np.abs(xf) @ np.abs(Af.T))
        assert rel_to_bound(to_np(u), xf @ Af.T, bu + 1e-30) <= 1
    bound = layer_bound(ref, xv, wc.T, xf, Af, Bf, s, K, False)
    assert rel_to_bound(got[:, c], ref, bound) <= 1


def test_a_row_does_not_depend_on_its_batch_with_many_columns():
    """As above for 16 tokens and fewer, where a workgroup has two row tiles and 4
    waves."""
    N, K, r = 8208, 1312, 24
    mw = qn.mxfp4_quantize_weight(torch.from_numpy(weights(N, K, 2)).to(DEV))
    A, B = adapters(N, K, r, 2)
    x = bf16_dev(acts(16, K, 2))
    y = qn.mxfp4_linear_fwd(mw, x, A, B, r, 16.0)
    for M in (2, 7, 15):
        assert torch.equal(qn.mxfp4_linear_fwd(mw, x[:M].contiguous(), A, B, r, 16.0), y[:M])


def test_long_contraction_of_a_few_tokens():
    """More runs than any layer has: the decode projection's slices grow with K
    and have to fit the workspace."""
    M, N, K, r = 2, 16, 2 ** 18 + 8224, 4
    rng = np.random.default_rng(1)
    w = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    xb = acts(M, K, 5)
    A, B = adapters(N, K, r, 1)
    mw = qn.mxfp4_quantize_weight(torch.from_numpy(w).to(DEV))
    wv = mxfp4.values(*mxfp4.quantize(w))
    xf, Af, Bf = f64(xb), to_np(A).astype(float), to_np(B).astype(float)
    xv = mxfp4.values(*mxfp4.quantize(xf.astype(np.float32)))
    for m in (1, 2):
        y = qn.mxfp4_linear_fwd(mw, bf16_dev(xb[:m]), A, B, r, 8.0)
        torch.cuda.synchronize()
        check(f"mxfp4 y {m}x{N}x{K}", to_np(y), xv[:m] @ wv.T + 2.0 * (xf[:m] @ Af.T) @ Bf.T)
