"""The largest int8 batches: their kernels take four rows a workgroup of 256 lanes, and a grid has fewer than 2^32."""
import pytest

from biased_top_routing_amd import _lib as L
from workloads import MID


@pytest.mark.parametrize("rows,status", [((1 << 26) - 4, L.MOE_ERR_NULL), ((1 << 26) - 3, L.MOE_ERR_SHAPE),
                                         ((1 << 26) - 1, L.MOE_ERR_SHAPE)])
def test_rows_to_quantise(rows, status):
    """(sizes are checked before pointers, so a NULL tells that a size is in range)"""
    assert L.lib().moe_quantize_int8(None, 1, rows, 16, 1, 16, 16, None) == status


@pytest.mark.parametrize("T,k,ok", [((1 << 25) - 4, 1, True), ((1 << 25) - 3, 1, False), ((1 << 25) - 1, 1, False),
                                    (((1 << 26) - 4) // 7, 6, True), (((1 << 26) - 4) // 7 + 1, 6, False)])
def test_tokens_of_a_layer(T, k, ok):
    cfg = L.cfg_from(MID, wgt="int8", T=T, k=k, E=8, G=1, M=1, S=0, H=128, I=128)
    assert (L.moe_workspace_bytes(cfg, L.MOE_WS_FFN) > 0) == ok
