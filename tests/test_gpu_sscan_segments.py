"""Scans whose sequences are cut into segments, in the forms that other tests reach whole only: terms
that are absent, groups of channels, a length of its own for each sequence."""
import pytest
import torch

from test_gpu_sscan import check, make

pytestmark = pytest.mark.gpu


def segments(s, backward):
    """From the workspace's size: whether the call is cut at all."""
    import aware_conv_amd.sscan as S
    B, _, D = s["x"].shape
    need = S.sscan_workspace_size(s["x"], s["a_log"], s["b"], backward)
    whole = S.sscan_workspace_size(s["x"][:, :16], s["a_log"], s["b"][:, :16], backward)
    if backward:  # part of it is there for each position
        one = S.sscan_workspace_size(s["x"][:, :32], s["a_log"], s["b"][:, :32], backward) - whole
        need -= one * (s["x"].shape[1] - 16) // 16
    return need > whole


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("without", [(), ("z",), ("d",), ("dt_bias",), ("h0",), ("dh_last",),
                                     ("z", "d", "dt_bias", "h0", "dh_last")])
def test_absent_terms(without, dtype):
    s = make(3, 1104, 70, 16, dtype=dtype, seed=3, without=without)
    if s["dt_bias"] is None:
        s["dt"] -= 4
    assert segments(s, False) and segments(s, True)
    check(s, what=("segments", without, dtype))
    check(s, [1104, 0, 370], what=("segments, lengths", without, dtype))


@pytest.mark.parametrize("N", [3, 8, 16, 21, 40, 64])
@pytest.mark.parametrize("without", [(), ("z",)])
def test_groups(N, without):
    """Channels of a group that do not fill a workgroup; lengths that end in, before and at segments."""
    s = make(4, 656, 54, N, G=3, dtype="f16", seed=N, without=without)
    assert segments(s, False) and segments(s, True)
    check(s, [656, 1, 129, 400], what=("segments, groups", N, without))
    check(s, [128, 640, 127, 0], what=("segments, groups, ends", N, without))


@pytest.mark.parametrize("N,forward,backward", [(6, False, True), (16, False, False)])
def test_a_pass_cut_one_way(N, forward, backward):
    """171 workgroups: with up to 8 states the backward is cut, the forward is not."""
    s = make(1, 272, 171 * 64, N, dtype="f32", seed=N, without=("z",))
    assert segments(s, False) is forward and segments(s, True) is backward
    check(s, what=("171 workgroups", N))
    check(s, [200], what=("171 workgroups, a length", N))


def test_two_runs_agree_bit_for_bit():
    s = make(2, 1500, 50, 16, dtype="bf16", seed=8, without=("z",))
    a, b = check(s, [1500, 900], what="first"), check(s, [1500, 900], what="second")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for k in a[2]:
        assert a[2][k] is None and b[2][k] is None or torch.equal(a[2][k], b[2][k]), k
