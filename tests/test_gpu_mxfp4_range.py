"""Products of microscaled codes whose scales reach far below 1 (GPU): exact
down to fp32's subnormal numbers, rounded once to bf16's."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_22_amd as qn
from oracle import mxfp4
from tests.gpu_helpers import to_bits16
from tests.test_gpu_mxfp4 import DEV

pytestmark = pytest.mark.gpu


def ones(R, K, byte):
    """A matrix of ones over the power of `byte`: packed codes and scales."""
    return (torch.from_numpy(mxfp4.pack(np.full((R, K), 2, np.uint8))).to(DEV),
            torch.from_numpy(mxfp4.tiles(np.full((R, K // 32), byte, np.uint8), R, K)).to(DEV))


# the power of a product: 2^(wb + xb - 254), at least fp32's least, 2^-149
@pytest.mark.parametrize("wb,xb", [(0, 254), (254, 0), (120, 119), (0, 200), (67, 67), (128, 0),
                                   (0, 127), (60, 59), (118, 0), (0, 112), (56, 50), (0, 105)])
@pytest.mark.parametrize("M", [2, 20, 100])
def test_sums_of_small_products(wb, xb, M):
    N, K = 16, 352
    got = qn.mxfp4_matmul(qn.Mxfp4Weight(*ones(N, K, wb)), *ones(M, K, xb))
    want = torch.full((M, N), K * 2.0 ** (wb + xb - 254), dtype=torch.float32).bfloat16()
    assert np.array_equal(to_bits16(got), to_bits16(want))


@pytest.mark.parametrize("wb", [254, 127, 60, 13, 8, 1, 0])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -10, 2.0 ** -16])
def test_backward_of_small_weights(wb, size):
    M, N, K = 20, 64, 96
    dy = torch.full((M, N), size, dtype=torch.bfloat16, device=DEV)
    got = qn.mxfp4_linear_bwd_dx(qn.Mxfp4Weight(*ones(N, K, wb)), dy, None, None, 0, 1.0)
    # past fp32's largest number infinity
    want = torch.tensor(N * size * 2.0 ** (wb - 127), dtype=torch.float64).float().bfloat16()
    assert np.array_equal(to_bits16(got), to_bits16(want.expand(M, K)))
