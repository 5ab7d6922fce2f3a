"""Sizes of the MXFP8 entry points that no launch holds are refused on the host (fake addresses, refusals only)."""

import pytest
from test_abi_mx_host import P, P2, SHAPE


@pytest.mark.parametrize("T,N", [(64 * 2732, 256 * 6141), (64 * 2732 - 63, 256 * 6141 - 255)])
@pytest.mark.parametrize("dt", [0, 1])
def test_linear_of_more_work_items_than_a_launch_has(T, N, dt):
    """16777212 tiles of 256 x 64 in a grid of whole eights are 2^32 work-items; of 256 x 256 they are under 2^22."""
    from nvfp4_w4a4_mixture_amd import _lib

    L = _lib.lib()
    assert -(-T // 256) * -(-N // 256) < 1 << 22
    assert L.mxfp8_linear(P, P, T, 32, P, P, N, None, 0, None, 0, 0, dt, P2, N, None) == SHAPE
    assert b"too large" in L.moe_last_error()
