"""Up to 128 tokens on weights of many columns: the large tiles' upper halves
alone (GPU).  Bounds as in tests/test_gpu_fp8.py."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_22_amd as qn
from oracle import fp8
from tests.gpu_helpers import bf16_dev, f64, to_np
from tests.test_gpu_fp8 import DEV, acts, bf16_of, layer_bound, rel_to_bound, weights

pytestmark = pytest.mark.gpu


# both sides of 128 tokens and of one round of the 256 CUs; a last column tile
# that is not whole; a contraction with a partial block; ranks in one and two
# groups of 64
@pytest.mark.parametrize("M,n,L,r", [(32, 65536, 272, 0), (32, 65552, 272, 16), (100, 66064, 400, 16),
                                     (127, 40016, 144, 40), (128, 33024, 272, 72),
                                     (129, 33024, 272, 16), (70, 70000, 128, 8)])
@pytest.mark.parametrize("bwd", [False, True])
def test_few_tokens_into_many_columns(M, n, L, r, bwd):
    N, K = (L, n) if bwd else (n, L)
    w = weights(N, K, M)
    rng = np.random.default_rng(n)
    xb = acts(M, L, 3, 1e-3 if bwd else 1.0)
    A, B = (bf16_of(rng.standard_normal(sh) * 0.02) for sh in ((r, K), (N, r)))
    fw = qn.fp8_quantize_weight(torch.from_numpy(w).to(DEV))
    out = torch.full((M + 1, n), 7.0, dtype=torch.bfloat16, device=DEV)
    low = torch.empty((M, r), dtype=torch.bfloat16, device=DEV) if r else None
    f = qn.fp8_linear_bwd_dx if bwd else qn.fp8_linear_fwd
    f(fw, bf16_dev(xb), bf16_dev(A) if r else None, bf16_dev(B) if r else None, r, 16.0, out[:M], low)
    torch.cuda.synchronize()
    assert torch.all(out[M] == 7.0)
    c = np.unique(np.concatenate([np.arange(0, n, 251), np.arange(n - 300, n)]))
    x, Af, Bf = f64(xb), f64(A), f64(B)
    P, Q = (Bf.T, Af[:, c]) if bwd else (Af, Bf[c].T)
    wv = fp8.weight_values(*fp8.quantize_blocks(w))
    ww = wv[:, c] if bwd else wv[c].T
    qv = fp8.row_values(*fp8.quantize_rows(x.astype(np.float32)))
    s = 16.0 / r if r else 0.0
    ref = qv @ ww + (s * (x @ P.T) @ Q if r else 0.0)
    bound = layer_bound(ref, qv, ww, x, P if r else None, Q.T, s, L)
    assert rel_to_bound(to_np(out[:M])[:, c], ref, bound) <= 1
    assert torch.isfinite(out.float()).all()
