"""The microscaled layer's workspace (GPU): of exactly the asked size, with a
guard behind it, and full of bytes that are NaN as a scale, as an 8-bit code and
as fp32, on every path of the layer and of the product of given codes."""

import pytest
import torch

import bit_nf4_quantized_22_amd as qn
from tests.gpu_helpers import bf16_dev
from tests.test_gpu_mxfp4 import DEV, acts
from tests.test_gpu_mxfp4_calls import adapters, same, weight

pytestmark = pytest.mark.gpu


def filled(need, byte):
    return torch.full((need + 4096,), byte, dtype=torch.uint8, device=DEV)


def outputs(call, need, byte):
    buf = filled(need, byte)
    out = call(buf[:need])
    torch.cuda.synchronize()
    assert (buf[need:] == byte).all()
    return out


# one token; the decode kernel; few; small tiles whole and split; large tiles.
# K and N end in either half of a tile of 256 columns, or with it
@pytest.mark.parametrize("M,N,K", [(1, 144, 288), (1, 272, 416), (2, 272, 608), (5, 144, 288),
                                   (16, 272, 1120), (17, 144, 288), (40, 272, 1056), (64, 400, 512),
                                   (65, 144, 32), (100, 272, 288), (100, 144, 4384),
                                   (80, 1040, 2080), (1100, 4096, 416), (1100, 4112, 288)])
@pytest.mark.parametrize("r", [0, 1, 16, 40])
def test_workspace_need_not_be_clean(M, N, K, r):
    mw = weight(N, K, 1)
    A, B = adapters(N, K, r, M) if r else (None, None)
    for f, L, op in ((qn.mxfp4_linear_fwd, K, qn.QN_OP_MXFP4_FWD),
                     (qn.mxfp4_linear_bwd_dx, N, qn.QN_OP_MXFP4_BWD_DX)):
        x = bf16_dev(acts(M, L, 8))
        low = torch.empty((M, r), dtype=torch.bfloat16, device=DEV) if r else None
        need = qn.qn_workspace_bytes(op, M, N, K, r)

        def call(ws):
            return f(mw, x, A, B, r, 16.0, None, low, ws=ws)

        want = outputs(call, need, 0)
        want_low = low.clone() if r else None
        assert torch.isfinite(want).all()
        got = outputs(call, need, 255)
        assert same(want, got)
        assert not r or same(want_low, low)


@pytest.mark.parametrize("M,N,K", [(1, 144, 288), (5, 272, 416), (40, 144, 1056), (100, 144, 288),
                                   (100, 144, 4384), (1100, 4096, 416)])
def test_product_of_given_codes(M, N, K):
    mw = weight(N, K, 2)
    c, s = qn.mxfp4_quantize(bf16_dev(acts(M, K, 3)))
    need = qn.qn_workspace_bytes(qn.QN_OP_MXFP4_FWD, M, N, K, 0)
    want, got = (outputs(lambda ws: qn.mxfp4_matmul(mw, c, s, ws=ws), need, b) for b in (0, 255))
    assert torch.isfinite(want).all() and same(want, got)
    # the layer's own product of the same codes
    assert M == 1 or same(want, qn.mxfp4_linear_fwd(mw, bf16_dev(acts(M, K, 3)), None, None, 0, 1.0))


@pytest.mark.parametrize("M", [1, 5, 40, 100])
def test_a_smaller_workspace_is_refused(M):
    N, K, r = 144, 288, 16
    mw = weight(N, K, 1)
    A, B = adapters(N, K, r, M)
    for f, L, op in ((qn.mxfp4_linear_fwd, K, qn.QN_OP_MXFP4_FWD),
                     (qn.mxfp4_linear_bwd_dx, N, qn.QN_OP_MXFP4_BWD_DX)):
        x = bf16_dev(acts(M, L, 8))
        for rank in (0, r):
            need = qn.qn_workspace_bytes(op, M, N, K, rank)
            with pytest.raises(qn.QnError) as e:
                f(mw, x, *((A, B) if rank else (None, None)), rank, 16.0,
                  ws=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
            assert e.value.status == qn.QN_ERR_WORKSPACE
