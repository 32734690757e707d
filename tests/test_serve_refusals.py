"""Calls of the serving step that are refused before any CUDA work, beside those
of test_serve_abi.py (without a GPU)."""
import pytest

from block_sparse_long_blockmean_b200 import fp2
from tests.test_serve_abi import (INVALID, MB, UNSUPPORTED, append_io, call_append, call_decode, lib,  # noqa: F401
                                  params)


def test_append_refuses_e4m3_of_head_dimension_64(lib):  # noqa: F811
    """No call reads such a cache."""
    scales = dict(q_scale=MB, k_scale=MB, v_scale=MB)
    io = append_io(rotary_dim=64)
    assert call_append(lib, io, params(head_dim=64, **scales), fp2.FP2_FP8_E4M3) == UNSUPPORTED
    # (what is asked for first is the shape: without scales it is the same)
    assert call_append(lib, io, params(head_dim=64), fp2.FP2_FP8_E4M3) == UNSUPPORTED
    assert call_append(lib, io, params(head_dim=64, workspace=None), fp2.FP2_BF16) != UNSUPPORTED


@pytest.mark.parametrize("item", [-1, -2 ** 31])
def test_decode_refuses_a_negative_item(lib, item):  # noqa: F811
    P = params(debug_withhold_k_item=item)
    assert call_decode(lib, P) == INVALID
    assert fp2.decode_workspace_size(P) == 0
