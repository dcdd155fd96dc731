"""33 to 64 tokens on wide microscaled weights, on both sides of the number of
columns past which they run as tiles (GPU)."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_22_amd as qn
from oracle import mxfp4
from tests.gpu_helpers import bf16_dev, f64, to_np
from tests.test_gpu_mxfp4 import DEV, acts, layer_bound, rel_to_bound, weights
from tests.test_gpu_mxfp4_calls import adapters

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,r", [(32, 8208, 1056, 16), (33, 8192, 1056, 16), (33, 8208, 1056, 16),
                                     (64, 8192, 1024, 128), (64, 8208, 1024, 0), (48, 16400, 288, 7),
                                     (64, 28672, 64, 24), (33, 28672, 1024, 16)])
def test_wide_weights(M, N, K, r):
    w, xb = weights(N, K, M), acts(M, K, 3)
    A, B = adapters(N, K, r, N) if r else (None, None)
    mw = qn.mxfp4_quantize_weight(torch.from_numpy(w).to(DEV))
    need = qn.qn_workspace_bytes(qn.QN_OP_MXFP4_FWD, M, N, K, r)
    buf = torch.full((need + 4096,), 255, dtype=torch.uint8, device=DEV)
    y = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    qn.mxfp4_linear_fwd(mw, bf16_dev(xb), A, B, r, 16.0, y=y[:M * N].view(M, N), ws=buf[:need])
    torch.cuda.synchronize()
    assert (buf[need:] == 255).all() and (y[M * N:] == 7.0).all()
    xf, s = f64(xb), 16.0 / r if r else 0.0
    xv = mxfp4.values(*mxfp4.quantize(xf.astype(np.float32)))
    c = np.unique(np.concatenate([np.arange(0, N, 37), np.arange(N - 48, N)]))
    wc = mxfp4.values(*mxfp4.quantize(w[c]))
    ref, Af, Bf = xv @ wc.T, None, None
    if r:
        Af, Bf = to_np(A).astype(float), to_np(B).astype(float)[c]
        ref = ref + s * (xf @ Af.T) @ Bf.T
    bound = layer_bound(ref, xv, wc.T, xf, Af, Bf, s, K, False)
    assert rel_to_bound(to_np(y[:M * N].view(M, N))[:, c], ref, bound) <= 1
