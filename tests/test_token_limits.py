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


# segments of a scan ------------------------------------------------------------

def scan_segments(workgroups, N, backward, T=4096):
    """Into how many segments a sequence is cut, from the workspace that they take."""
    waves = -(-(-(-N // 4)) // (1 if N <= 4 else 2 if N <= 32 else 4))
    width, states = (64 if waves <= 2 else 32), 4 * waves * (1 if N <= 4 else 2 if N <= 32 else 4)
    D = width * workgroups
    s = L.SscanShape(1, T, D, N, 1, 2)
    n = ctypes.c_size_t(0)
    assert L.lib.sscan_workspace_size(ctypes.byref(s), backward, ctypes.byref(n)) == 0
    carried = 4 * (D * N + D)  # a segment's state and sum of delta
    if not backward:
        assert n.value % carried == 0
        return max(1, n.value // carried)
    rest = n.value - 4 * workgroups * T * 2 * states
    sums = 4 * (D * N + 2 * D)  # of the parameters' gradients
    return 1 if rest == sums else rest // (carried + sums)


@pytest.mark.parametrize("N", [4, 8, 16, 24, 32, 64])
@pytest.mark.parametrize("workgroups,forward,backward", [(1, 32, 32), (32, 16, 16), (128, 4, 4), (129, 3, 3),
                                                         (170, 3, 3), (171, 1, 1), (191, 1, 1), (192, 1, 1)])
def test_scans_are_cut_where_that_pays(workgroups, forward, backward, N):
    """Two segments cost more than they give, but backwards with up to 8 states."""
    if N <= 8 and 171 <= workgroups < 192:
        backward = 2
    assert scan_segments(workgroups, N, 0) == forward
    assert scan_segments(workgroups, N, 1) == backward
