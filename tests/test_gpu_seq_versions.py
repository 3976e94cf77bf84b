"""What the sequence and training operators write in place, as autograd sees it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,dtype", [(32, torch.float32), (8, torch.float16)])
def test_a_backward_pass_over_stepped_weights_is_refused(bits, dtype):
    """A graph from before AdamW.step() saved the weights, and must not go on with new ones."""
    import aware_conv_amd as A
    torch.manual_seed(0)
    layer = A.WTConv2d(4, kernel_size=3, levels=1, device="cuda", dtype=dtype)
    opt = A.AdamW(layer.parameters(), bits=bits)
    x = torch.randn(2, 4, 8, 8, device="cuda", dtype=dtype, requires_grad=True)
    loss = layer(x).float().square().mean()
    loss.backward(retain_graph=True)
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    layer(x).float().square().mean().backward()  # a new graph is in order


def versions(*ts):
    return [t._version for t in ts]


def test_versions_of_what_is_written():
    import aware_conv_amd as A
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    for bits in (32, 8):
        dt = torch.float32 if bits == 32 else torch.float8_e4m3fn
        p, g, w, norm = z(300), z(300), z(300), z(1)
        m, v = z(300, dtype=torch.uint8).view(dt) if bits == 8 else z(300), z(300).to(dt)
        sc = (z(2), z(2))
        step = z(1, dtype=torch.int32)
        out = [p, m, v, w, step] + list(sc if bits == 8 else ())
        before = versions(*out, norm, g)
        A.adamw_grad_norm([g], norm=norm)
        A.adamw_step([p], [g], [m], [v], step, masters=[w], grad_norm=norm, max_norm=1.0,
                     scales=([sc[0]], [sc[1]]) if bits == 8 else None)
        after = versions(*out, norm, g)
        assert all(b > a for a, b in zip(before[:-1], after[:-1])) and before[-1] == after[-1]
    x, lam, h = z(2, 3, 8), z(3), z(2, 3, 8)
    grads = {n: z(2, 3, 8) for n in ("dx", "dr", "di")}
    before = versions(x, lam, h, *grads.values())
    _, _, st = A.gscan_fwd(x, x, x, lam, h=h, save_states=True)
    A.gscan_bwd(x, x, x, lam, st, h, grads=grads)
    after = versions(x, lam, h, *grads.values())
    assert before[:2] == after[:2] and all(b > a for a, b in zip(before[2:], after[2:]))
    x1, state, h1 = z(2, 3), z(4, 3), z(2, 3)
    before = versions(x1, state, h1)
    A.gscan_step(x1, x1, x1, lam, state, h=h1)
    after = versions(x1, state, h1)
    assert before[0] == after[0] and before[1] < after[1] and before[2] < after[2]
    with torch.inference_mode():
        state = z(4, 3)
    A.gscan_step(x1, x1, x1, lam, state)  # has no counter, and needs none
