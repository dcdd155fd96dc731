"""Choices that the FP8 layer makes on the host, as its workspace shows them
(CPU: nothing here launches a kernel)."""

import pytest

import bit_nf4_quantized_22_amd as qn


def up(n, b):
    return -(-n // b) * b


def parts(M, N, K, bwd=False):
    """How many fp32 parts of the output the workspace has room for."""
    L, n = (N, K) if bwd else (K, N)
    op = qn.QN_OP_FP8_BWD_DX if bwd else qn.QN_OP_FP8_FWD
    rest = qn.qn_workspace_bytes(op, M, N, K, 0) - up(M * L, 256) - up(M * up(L, 128) // 32, 256)
    assert rest >= 0 and rest % (M * n * 4) == 0
    return rest // (M * n * 4)


# whether the product was measured faster in parts (True), or whole (False)
@pytest.mark.parametrize("M,N,K,split", [
    (128, 4096, 11008, True), (1000, 1024, 8192, True), (65, 4096, 4096, True),
    (128, 11008, 4096, True), (512, 2048, 4096, True), (70, 2000, 5008, True),
    (200, 1040, 1552, False), (333, 2112, 1088, False), (1000, 1024, 2048, False),
    (256, 2048, 1024, False), (500, 1504, 1024, False), (700, 2048, 2048, False)])
def test_a_contraction_is_split_where_that_is_faster(M, N, K, split):
    assert (parts(M, N, K) > 1) == split
    assert (parts(M, K, N, bwd=True) > 1) == split


def test_short_products_are_not_split_beyond_their_gain():
    """Measured least times: 4 to 6 parts and 6 to 8."""
    assert 4 <= parts(100, 1088, 2112) <= 6
    assert 6 <= parts(66, 400, 2064) <= 8


def test_a_table_with_a_missing_matrix_is_refused():
    import torch

    t = torch.zeros(4)
    for k, name in enumerate("pgmv"):
        cols = [[t, t] for _ in range(4)]
        cols[k] = [None, t] if k % 2 else [t, None]
        with pytest.raises(ValueError, match=f"^{name}: missing"):
            qn.lora_adamw_table(*cols)
    with pytest.raises(ValueError, match="device tensor"):   # host memory
        qn.lora_adamw_table([t], [t], [t], [t])
