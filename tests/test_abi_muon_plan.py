"""Plans of the Muon step that no table gave are refused before a launch (CPU)."""

import ctypes

import pytest

import bit_nf4_quantized_22_amd as qn
from tests.test_abi import FAKE, lib  # noqa: F401
from tests.test_abi_muon import build, hyper, tensors


def status(lib, plan, ws=FAKE, room=1 << 62):  # noqa: F811
    return lib.lora_muon_multi_step(ctypes.byref(plan), FAKE, ctypes.byref(hyper()), ws, room, None)


@pytest.mark.parametrize("shapes", [[(4, 64)], [(128, 300), (16, 16), (5000, 17), (33, 40)]])
def test_a_plans_workspace_is_what_its_chunks_need(lib, shapes):  # noqa: F811
    _, plan, _, _ = build(tensors(*shapes))
    for bytes_ in (0, 8, plan.ws_bytes - 8, plan.ws_bytes + 8):
        bad = qn.qn_muon_plan.from_buffer_copy(plan)
        bad.ws_bytes = bytes_
        # without a workspace, and with room for anything
        assert status(lib, bad, ws=None, room=0) == qn.QN_ERR_SHAPE
        assert status(lib, bad) == qn.QN_ERR_SHAPE
    # a chunk more than the workspace was made for, with the table's size to match
    for k in range(4):
        bad = qn.qn_muon_plan.from_buffer_copy(plan)
        if plan.matrices[k]:
            bad.chunks[k] += 1
            bad.bytes += 8
            assert status(lib, bad) == qn.QN_ERR_SHAPE


@pytest.mark.parametrize("k,tiles", enumerate((1, 2, 4, 8)))
def test_a_plans_launches_have_less_than_2_to_the_32_threads(lib, k, tiles):  # noqa: F811
    """Chunks and spans are less than 2^23 in all, and a matrix has one of each,
    of 256 and up to 512 threads; its steps take up to 768."""
    def plan_of(matrices, chunks, spans):
        p = qn.qn_muon_plan()
        p.matrices[k], p.chunks[k], p.spans[k] = matrices, chunks, spans
        p.bytes = 88 * matrices + 8 * (chunks + spans)
        p.ws_bytes = 8 * 256 * (chunks * tiles * (tiles + 1) // 2 + matrices * tiles * tiles)
        return p

    top = 1 << 23
    for sizes in ((top // 2, top // 2, top // 2), (top - 1, top - 1, top - 1), (1, top - 1, 1),
                  (1, 1, top - 1), (1, top // 2, top // 2)):
        assert status(lib, plan_of(*sizes)) == qn.QN_ERR_SHAPE, sizes
    # within the limit, and refused for the workspace alone
    most = top // 2 - 1
    assert 768 * most < 2 ** 32
    assert status(lib, plan_of(most, most, most), room=0) == qn.QN_ERR_WORKSPACE
