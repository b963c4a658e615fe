"""Calls of the training step that are refused before anything is launched (no GPU needed)."""
import ctypes
import os

import pytest

import grouped_gemm_expert_router_amd as moe

F = 1 << 20   # a non-null, 256-aligned address that is never dereferenced on error paths


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        pytest.skip("libmoe.so not built")
    return moe.load_library()


def test_norm_backward_of_neither_part_is_refused(lib):
    """Neither the norm before a block (w_pre) nor the part behind it (y): there is nothing to go back
    through, whatever comes in and is asked for.  The forward call refuses it with the same code."""
    names = ("y", "h_out", "w_post", "gate", "w_pre", "dh_out", "dx", "dh", "dy", "dw_post", "dgate", "dw_pre")
    for T in (1, 4, 4096):
        nd = moe.norm_desc(T, 64)
        for given in ((), ("dh_out",), ("dh_out", "dh"), ("dh",)):
            a = [F if n in given else None for n in names]
            for ws, nb in ((F, 1 << 40), (None, 0)):
                assert lib.moe_norm_backward(ctypes.byref(nd), *a, ws, nb, None) == moe.MOE_ERR_NULL, given
        assert lib.moe_norm_forward(ctypes.byref(nd), None, F, None, None, None, None, None, None) == moe.MOE_ERR_NULL
