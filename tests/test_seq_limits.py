"""The sizes at which the recurrence's entry points begin to refuse, as include/gscan.h states
them.  CPU only: the sizes of states and workspace are asked for, and nothing is launched."""
import ctypes

import pytest

from aware_conv_amd import _lib as L
from test_seq_checks import NULL, SHAPE, step

UNSUPPORTED = -8
BCT, BTC = 0, 1


def sizes(B, C, T, layout):
    """(status, states in bytes, workspace in bytes)."""
    s = L.GscanShape(B, C, T, layout, 2, 0, 8.0)
    out = [ctypes.c_size_t(0), ctypes.c_size_t(0)]
    codes = {L.lib.gscan_states_size(ctypes.byref(s), ctypes.byref(out[0])),
             L.lib.gscan_workspace_size(ctypes.byref(s), ctypes.byref(out[1]))}
    assert len(codes) == 1
    return codes.pop(), out[0].value, out[1].value


@pytest.mark.parametrize("B,C,T,fits", [
    # ceil(C / 64) * B * ceil(T / 256) below 2^23
    (1, 1, 1 << 30, True), (1, 64, 1 << 30, True), (1, 65, 1 << 30, False), (2, 1, 1 << 30, False),
    (1, 128, 1 << 29, True), (2, 64, 1 << 29, True), (1, 128, (1 << 30) - 512, True),
    (1, 128, (1 << 30) - 256, True), (1, 128, (1 << 30) - 255, False), (3, 64, 1 << 29, True),
    ((1 << 23) - 1, 1, 1, True), (1 << 23, 1, 1, False), ((1 << 23) - 1, 4, 256, True),
])
def test_tokens(B, C, T, fits):
    code, states, workspace = sizes(B, C, T, BTC)
    assert code == (0 if fits else UNSUPPORTED)
    if fits:
        tiles = -(-T // 128)
        assert states == 4 * tiles * B * C and workspace >= 4 * tiles * B * C


@pytest.mark.parametrize("B,C,T,fits", [
    # B * C * ceil(T / 4096) below 2^23, up to 1024 rows
    (1, 31, 1 << 30, True), (31, 1, 1 << 30, True), (1, 32, 1 << 30, False), (1, 32, (1 << 30) - 4096, True),
    (1, 32, (1 << 30) - 4095, False), (1, 1024, 1 << 25, False), (1, 1024, (1 << 25) - 4096, True),
    # more rows are walked, whatever their length
    (1, 1025, 1 << 25, True), (1 << 25, 1, 1 << 30, True),
])
def test_planes(B, C, T, fits):
    assert sizes(B, C, T, BCT)[0] == (0 if fits else UNSUPPORTED)


def test_rows():
    for layout in (BCT, BTC):
        assert sizes((1 << 25) + 1, 1, 1, layout)[0] == SHAPE
        assert sizes(1, 1, (1 << 30) + 1, layout)[0] == SHAPE
    assert sizes(1, 1 << 25, 1, BTC)[0] == sizes(1, 1 << 25, 1, BCT)[0] == 0


def test_single_positions_are_bound_by_the_rows_alone():
    for B, C in ((1 << 24, 1), (1 << 25, 1), (1 << 24, 2)):
        assert step(B=B, C=C, S=B, x=None) == NULL
    assert step(B=(1 << 25) + 1, C=1, S=1 << 26, x=None) == SHAPE
