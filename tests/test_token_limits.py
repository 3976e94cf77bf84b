"""Sizes that a launch of the token operators does not hold, refused before anything is enqueued.  CPU
only: no call here passes its checks."""
import ctypes

import pytest

from aware_conv_amd import _lib as L

WORKSPACE, UNSUPPORTED = -7, -8


def far(i):
    """Distinct fake buffers 1 TiB apart, never dereferenced."""
    return (i + 1) << 40


def conv_backward(C, K, bias=True, T=1):
    """With a workspace that is too short: nothing may run."""
    s = L.CconvShape(1, T, C, K, 0, 1)
    view = lambda i: ctypes.byref(L.GscanView(far(i), T * C, C))  # noqa: E731
    return L.lib.cconv_bwd(ctypes.byref(s), view(0), far(1), far(2) if bias else None, None, None, view(3), None,
                           view(4), far(5), far(6) if bias else None, None, far(7), 0, None)


@pytest.mark.parametrize("C,K,bias,code", [
    ((1 << 27) - 16, 1, True, WORKSPACE), ((1 << 27) - 15, 1, True, UNSUPPORTED), (1 << 27, 1, True, UNSUPPORTED),
    (1 << 27, 1, False, WORKSPACE), (1 << 26, 2, True, WORKSPACE), (1 << 24, 8, True, WORKSPACE)])
def test_launch_that_closes_the_convolutions_sums(C, K, bias, code):
    """A workgroup of 256 threads per 16 values of dw and of dbias: fewer than 2^24 of them."""
    assert (code == UNSUPPORTED) == (-(-C * K // 16) + (-(-C // 16) if bias else 0) >= 1 << 24)
    assert conv_backward(C, K, bias) == code
