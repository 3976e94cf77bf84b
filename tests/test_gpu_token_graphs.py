"""A training pass over the norm, the convolution and the scan, captured into a graph: every replay
gives, bit for bit, what the same calls give eagerly on the same inputs (all sums have a fixed order)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def inputs(B, T, C, N, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    wide = {"x": r(B, T, C), "residual": r(B, T, C), "dt": r(B, T, C) - 1, "b": r(B, T, N), "c": r(B, T, N),
            "z": r(B, T, C), "dy": r(B, T, C)}
    flat = {"norm": 1 + 0.2 * r(C), "w": r(C, 4) / 2, "bias": r(C), "a_log": r(C, N) / 2, "d": r(C)}
    s = {k: v.to(dtype) for k, v in wide.items()}
    s.update(flat)
    s["lengths"] = torch.randint(0, T + 1, (B,), generator=g).int()
    return {k: v.cuda() for k, v in s.items()}


LEAVES = ("x", "residual", "dt", "b", "c", "z", "norm", "w", "bias", "a_log", "d")


def passes(s):
    import aware_conv_amd as A
    p = {k: s[k].detach().requires_grad_() for k in LEAVES}
    y, total = A.rms_norm(p["x"], p["norm"], p["residual"])
    u, _ = A.causal_conv(y, p["w"], p["bias"], lengths=s["lengths"])
    v, last = A.selective_scan(u, p["dt"], p["a_log"], p["b"], p["c"], p["d"], p["z"], lengths=s["lengths"])
    grads = torch.autograd.grad([v, total], [p[k] for k in LEAVES], [s["dy"], s["dy"]])
    return [v.detach(), total.detach(), last.detach(), *grads]


@pytest.mark.parametrize("dtype,B,T,C,N", [(torch.float32, 2, 37, 24, 5), (torch.bfloat16, 1, 1200, 70, 16),
                                           (torch.float16, 3, 300, 130, 16)])
def test_training_pass(dtype, B, T, C, N):
    """(1, 1200, 70): few enough workgroups that a sequence is cut into segments."""
    print("\ncase token graph %s" % ((dtype, B, T, C, N),), flush=True)
    s = inputs(B, T, C, N, dtype, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        passes(s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = passes(s)
    for seed in range(1, 5):
        new = inputs(B, T, C, N, dtype, seed)
        want = passes(new)
        for k in s:
            s[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (seed, k)
