"""Host-side checks of the calls around a linear that need no GPU: overlaps, counts and
devices that are refused before anything is launched, and the binding's objects."""
import ctypes

import pytest

from w4a4_rank_assisted_b200 import hsq

A, FAR = 1 << 20, 1 << 30   # fake device addresses: every call below has to be refused before they are touched
INVALID = hsq.HSQ_ERR_INVALID_ARG


@pytest.mark.parametrize("M,r,group", [(1, 4, 64), (2, 0, 128), (4, 1, 64)])
@pytest.mark.parametrize("shift", [0, 64, -64], ids=["same", "above", "below"])
def test_the_stream_form_refuses_y_over_x(M, r, group, shift):
    """With an epilogue, without one, and through one that asks for nothing: its blocks read X while others write Y."""
    lib = hsq.load()
    assert hsq.hsq_fused_form(M, 128, 128, r, group) == 1
    low = None if r == 0 else FAR
    args = (A, FAR, low, FAR, FAR, low, None, M, 128, 128, r, group, A + shift, 0)
    assert lib.hsq_linear_forward_fused(*args, None) == INVALID
    assert lib.hsq_linear_forward_fused_ep(*args, None, None) == INVALID
    assert lib.hsq_linear_forward_fused_ep(*args, ctypes.byref(hsq._CEpilogue()), None) == INVALID
    assert lib.hsq_linear_forward_fused_ep(*args, ctypes.byref(hsq._CEpilogue(act=4)), None) == INVALID
