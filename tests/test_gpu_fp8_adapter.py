"""The LoRA term of the block-scaled FP8 layer by itself (GPU).

The weight is zero, so that the result is the LoRA term alone, and x, A and B
are positive, so that no sum cancels.  Bounds, per element:
  * u = x A^T sums L products in fp32 and s u B^T the r ranks' products, each
    in two parts: within one ulp (2^-23) of the magnitude summed so far, and
    4 more operations: (L + 2 r + 4) 2^-23;
  * s u enters the product as two bf16 numbers, hi = bf16(s u) and lo = bf16(s
    u - hi): |s u - hi| <= 2^-8 |s u|, and lo's rounding is 2^-8 of that: 2^-16;
  * the result is rounded to bf16 once: half of bf16's spacing at the result.
"""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_22_amd as qn
from tests.gpu_helpers import bf16_dev, f64, synth, to_np
from tests.test_gpu_fp8 import test_few_tokens_with_two_row_tiles as layer_against_the_oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def positive(shape, seed):
    rng = np.random.default_rng(seed)
    return synth.bf16_bits(np.exp(0.5 * rng.standard_normal(shape)).astype(np.float32))


def zero_weight(N, K):
    codes = torch.zeros((N, K), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    return qn.Fp8Weight(codes, torch.ones((-(-N // 128), -(-K // 128)), device=DEV))


def half_spacing(v):
    """Half of bf16's spacing at fp64 v: 8 significant bits."""
    return np.exp2(np.floor(np.log2(np.abs(v))) - 8)


# every kernel that adds the term: one token with u of its own and given, up
# to 16 and up to 64 tokens, small tiles, large tiles; one to four groups of 32
# ranks, whole and not
@pytest.mark.parametrize("M,N,K,r", [(1, 272, 272, 1), (1, 272, 272, 16), (1, 272, 272, 33),
                                     (1, 272, 272, 128), (5, 272, 272, 1), (16, 272, 272, 32),
                                     (16, 144, 272, 72), (3, 4112, 1168, 24), (40, 272, 272, 1),
                                     (33, 144, 272, 64), (64, 144, 272, 97), (100, 272, 272, 1),
                                     (100, 272, 272, 32), (130, 272, 400, 64), (130, 272, 400, 65),
                                     (100, 144, 272, 128), (1100, 4096, 128, 2),
                                     (1100, 4096, 144, 40), (2100, 8000, 48, 100)])
def test_lora_term_is_rounded_once(M, N, K, r):
    xb, dyb, A, B = positive((M, K), 1), positive((M, N), 2), positive((r, K), 3), positive((N, r), 4)
    s, fw = 16.0 / r, zero_weight(N, K)
    y = qn.fp8_linear_fwd(fw, bf16_dev(xb), bf16_dev(A), bf16_dev(B), r, 16.0)
    dx = qn.fp8_linear_bwd_dx(fw, bf16_dev(dyb), bf16_dev(A), bf16_dev(B), r, 16.0)
    torch.cuda.synchronize()
    rows = np.unique(np.concatenate([np.arange(0, M, 41), [M - 1]]))
    Af, Bf = f64(A), f64(B)
    for got, ref, L in ((y, s * (f64(xb[rows]) @ Af.T) @ Bf.T, K),
                        (dx, s * (f64(dyb[rows]) @ Bf) @ Af, N)):
        sums = (2.0 ** -16 + (L + 2 * r + 4) * 2.0 ** -23) * 1.01 * ref
        bound = half_spacing(ref + sums) + sums
        assert np.all(np.abs(to_np(got)[rows].astype(np.float64) - ref) <= bound)


@pytest.mark.parametrize("M", [1, 5, 40, 100])
def test_a_lora_operand_past_bf16s_range_is_an_infinity(M):
    """s u of 3.4e38, which bf16 rounds to an infinity, beside a row that stays
    in range: no NaN comes from splitting it."""
    N, K, r = 144, 272, 3
    x = np.zeros((M, K), np.float32)
    x[0, 5] = 2.0 ** 127
    if M > 1:
        x[1:, 5] = 1.0
    A = np.zeros((r, K), np.float32)
    A[:, 5] = 1.0
    B = np.ones((N, r), np.float32)
    bits = [bf16_dev(synth.bf16_bits(a)) for a in (x, A, B)]
    fw = zero_weight(N, K)
    # alpha / r: 2^127 times this is below fp32's largest number
    y = qn.fp8_linear_fwd(fw, *bits, r, 3 * float(np.float32(1.9999)))
    torch.cuda.synchronize()
    y = to_np(y)
    assert np.all(y[0] == np.inf)
    assert np.all(np.isfinite(y[1:])) and np.all(y[1:] > 5)


# one, two and more groups of slices of u; one and several threads per value of
# u; the forms of 4 waves, of 8, and of two row tiles; contractions of other
# lengths than whole slices
@pytest.mark.parametrize("N,K,r", [(144, 272, 16), (272, 1040, 5), (144, 4096, 16),
                                   (272, 11008, 16), (144, 11008, 128), (4112, 4112, 24),
                                   (16, 2 ** 16 + 528, 8)])
@pytest.mark.parametrize("seed", [1, 2])
def test_up_to_16_tokens_the_batch_does_not_change_a_row(N, K, r, seed):
    """The bits of y and of u: the slices of u are added in an order that
    depends on K alone."""
    rng = np.random.default_rng(seed)
    bits = lambda *shape: bf16_dev(synth.bf16_bits(rng.standard_normal(shape).astype(np.float32)))
    fw = qn.fp8_quantize_weight(bits(N, K))
    A, B, x = bits(r, K), bits(N, r), bits(16, K)

    def both(M):
        u = torch.empty((M, r), dtype=torch.bfloat16, device=DEV)
        y = qn.fp8_linear_fwd(fw, x[:M], A, B, r, 16.0, u_out=u)
        torch.cuda.synchronize()
        return y.view(torch.int16), u.view(torch.int16)

    all_y, all_u = both(16)
    for M in (2, 3, 4, 7, 8, 15):
        y, u = both(M)
        assert torch.equal(u, all_u[:M]) and torch.equal(y, all_y[:M]), M


@pytest.mark.parametrize("N,K,r", [(4096, 4096, 16), (4112, 4096, 16), (8208, 2048, 16),
                                   (8192, 2048, 16)])
def test_one_token_at_the_border_of_an_own_u(N, K, r):
    """A read by all workgroups together: 32 MiB, and just past it."""
    layer_against_the_oracle(1, N, K, r)
