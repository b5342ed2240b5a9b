"""The experts of a share have int32 ids: the kernels tell a present id by the unsigned difference to the first one,
which for a share that reaches past 2^31 some negative ids pass too."""
import ctypes

import pytest

from biased_top_routing_amd import _lib as L
from workloads import MID

A = 16   # an aligned address that is never dereferenced


@pytest.mark.parametrize("T", [0, 512])
@pytest.mark.parametrize("E", [6, 8, 512])
def test_first_expert_range(T, E):
    cfg = L.cfg_from(MID, T=T, E=E, G=1, M=1)
    need = L.moe_workspace_bytes(cfg, L.MOE_WS_DISPATCH)

    def call(first):   # (a workspace too small: the check that follows the range's, and nothing is launched)
        return L.lib().moe_dispatch_local(ctypes.byref(cfg), first, *[A] * 8, None, A, need - 1, None)

    present = lambda idx, first: (idx - first) % 2 ** 32 < E     # the kernels' test
    top = 2 ** 31 - E
    assert not any(present(-i, top) for i in (1, 2, 2 ** 31 - 1, 2 ** 31))
    assert call(top) == L.MOE_ERR_WORKSPACE
    for first in (top + 1, 2 ** 31 - 1):
        assert present(-2 ** 31, first)
        assert call(first) == L.MOE_ERR_SHAPE
