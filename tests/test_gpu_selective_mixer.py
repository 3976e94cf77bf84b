"""The block of norm, causal convolution and selective scan on the GPU: the operators together, as
a model has them, against the same in plain torch operations in fp64."""
import copy

import pytest
import torch

import token_reference as ref

pytestmark = pytest.mark.gpu


def block(dtype=torch.float32, channels=24, **kw):
    import aware_conv_amd as A
    torch.manual_seed(0)
    m = A.SelectiveMixer(channels, states=5, taps=4, rank=3, device="cuda", dtype=dtype, **kw)
    with torch.no_grad():
        m.norm.normal_(1, 0.2)
        m.conv_b.normal_()
        m.d.normal_()
    return m


def plain(m, x, residual, lengths=None):
    """The block in fp64, on the CPU, differentiable."""
    p = {n: t.detach().double().cpu().requires_grad_() for n, t in m.named_parameters()}
    total = x if residual is None else x + residual
    y = total / torch.sqrt((total ** 2).mean(-1, keepdim=True) + m.eps) * p["norm"]
    u, z = (y @ p["inner.weight"].t()).chunk(2, dim=-1)
    B, T, D = u.shape
    K, N = p["conv_w"].shape[1], p["a_log"].shape[1]
    out = torch.zeros_like(total)
    rows = []
    for i, n in enumerate(ref.counts(B, T, lengths)):
        line = torch.cat([torch.zeros(K - 1, D, dtype=torch.float64), u[i, :n]])
        v = sum(line[k:k + n] * p["conv_w"][:, k] for k in range(K)) + p["conv_b"]
        v = ref.silu(v)
        dt, b, c = (v @ p["low.weight"].t()).split(m.split, dim=-1)
        pre = dt @ p["dt.weight"].t() + p["dt_bias"]
        delta = ref.softplus(pre)
        h, ys = torch.zeros(D, N, dtype=torch.float64), []
        for t in range(n):
            h = torch.exp(-delta[t][:, None] * torch.exp(p["a_log"])) * h + (delta[t] * v[t])[:, None] * b[t]
            ys.append((c[t] * h).sum(1) + p["d"] * v[t])
        s = torch.stack(ys) * ref.silu(z[i, :n]) if n else torch.zeros(0, D, dtype=torch.float64)
        rows.append(torch.cat([s @ p["outer.weight"].t(), torch.zeros(T - n, x.shape[-1], dtype=torch.float64)]))
    return torch.stack(rows), total, p


@pytest.mark.parametrize("lengths", [None, [30, 0, 17]])
@pytest.mark.parametrize("stream", [False, True])
def test_block_against_plain_operations(lengths, stream):
    """Three fp32 products of up to 48 terms, and the operators' own 1e-5: 5e-5 of the largest value,
    for gradients, which pass back through all of it, 2e-4."""
    print("\ncase block %s %s" % (lengths, stream), flush=True)
    m = block()
    g = torch.Generator().manual_seed(1)
    x, res, dy, dt = (torch.randn(3, 30, 24, generator=g) for _ in range(4))
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    xg, rg = x.cuda().requires_grad_(), res.cuda().requires_grad_()
    out, total = m(xg, rg if stream else None, lengths=n)
    if lengths is not None:
        for i, k in enumerate(lengths):  # rows behind a sequence count for nothing
            dt[i, k:] = 0
    ((out * dy.cuda()).sum() + (total * dt.cuda()).sum()).backward()
    x64, r64 = x.double().requires_grad_(), res.double().requires_grad_()
    want, wtotal, p = plain(m, x64, r64 if stream else None, lengths)
    ((want * dy.double()).sum() + (wtotal * dt.double()).sum()).backward()
    near = lambda a, b, tol: bool(((a.detach().double().cpu() - b).abs() <= tol * b.abs().max()).all())  # noqa: E731
    assert near(out, want.detach(), 5e-5) and near(total, wtotal.detach(), 1e-6)
    assert near(xg.grad, x64.grad, 2e-4)
    if stream:
        assert near(rg.grad, r64.grad, 2e-4)
    for k, t in m.named_parameters():
        assert near(t.grad, p[k].grad, 2e-4), k


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 0.05)])
@pytest.mark.parametrize("wide", [False, True])
def test_served_position_by_position(dtype, tol, wide):
    """Two blocks: a padded prompt into rows of a cache, then single positions, against one pass
    over each whole sequence (bf16: its intermediate results round by 2^-8 in other groupings)."""
    print("\ncase served %s %s" % (dtype, wide), flush=True)
    blocks = [block(dtype, residual_fp32=wide), block(dtype, residual_fp32=wide)]
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 40, 24, generator=g).to(dtype).cuda()

    def forward(call):
        y, res = x_, None
        for k, m in enumerate(blocks):
            y, res = call(k, m, y, res)
        return y.float() + res.float()

    with torch.no_grad():
        x_ = x
        want = forward(lambda k, m, y, r: m(y, r))
    caches = [m.new_cache(5) for m in blocks]
    rows, lengths = [4, 0, 2], [20, 3, 9]
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    x_ = x[:, :20]
    got = forward(lambda k, m, y, r: m.prompt(y, caches[k], r, lengths=n, rows=rows))
    for i, k in enumerate(lengths):
        assert (got[i, :k] - want[i, :k]).abs().max() <= tol * want.abs().max()
    untouched = [[t[[1, 3]].clone() for t in c] for c in caches]
    slots = torch.tensor(rows, dtype=torch.int32, device="cuda")
    for step in range(20):
        x_ = torch.stack([x[i, k + step] for i, k in enumerate(lengths)])
        got = forward(lambda k, m, y, r: m.step(y, caches[k], r, slots=slots))
        for i, k in enumerate(lengths):
            assert (got[i] - want[i, k + step]).abs().max() <= tol * want.abs().max(), (step, i)
    for c, u in zip(caches, untouched):
        assert all(torch.equal(t[[1, 3]], v) for t, v in zip(c, u))


def test_captured_step():
    """A serving step in a graph, replayed with other work between, goes on like eager steps."""
    m = block(torch.bfloat16)
    cache = m.new_cache(4)
    other = tuple(t.clone() for t in cache)
    slots = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    x = torch.randn(3, 24, device="cuda").bfloat16()
    res = torch.randn(3, 24, device="cuda").bfloat16()
    m.step(x, tuple(t.clone() for t in cache), res, slots=slots)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.step(x, cache, res, slots=slots)
    for t in cache:
        t.zero_()
    for _ in range(4):
        x.normal_()
        res.normal_()
        want = m.step(x, other, res, slots=slots)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        assert all(torch.equal(a, b) for a, b in zip(cache, other))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_trained_by_adamw(dtype):
    import aware_conv_amd as A
    m = block(dtype)
    opt = A.AdamW(m.parameters(), lr=1e-3, bits=8, max_norm=1.0)
    before = {n: t.detach().clone() for n, t in m.named_parameters()}
    g = torch.Generator(device="cuda").manual_seed(0)
    for _ in range(3):
        x = torch.randn(2, 50, 24, generator=g, device="cuda").to(dtype)
        out, total = m(x)
        opt.zero_grad(set_to_none=True)
        (out.float() + total.float()).square().mean().backward()
        for n, t in m.named_parameters():
            assert t.grad.dtype == t.dtype and torch.isfinite(t.grad).all(), n
        opt.step()
    for n, t in m.named_parameters():
        assert torch.isfinite(t).all() and not torch.equal(t, before[n]), n


def test_a_converted_block_runs_as_one_made_so():
    m = block()
    made = block(torch.bfloat16)
    made.load_state_dict(m.state_dict())
    x = torch.randn(2, 30, 24, device="cuda").bfloat16()
    a, b = copy.deepcopy(m).bfloat16()(x)[0], made(x)[0]
    assert torch.equal(a, b)


def versions(*ts):
    return [t._version for t in ts]


def test_versions_of_what_is_written():
    """Autograd sees what the calls write."""
    import aware_conv_amd as A
    z = lambda *n, **k: torch.zeros(*n, device="cuda", **k)  # noqa: E731
    y, wide = z(2, 5, 6), z(2, 5, 6)
    args = [z(2, 5, 6), z(2, 5, 6), z(6, 4), z(2, 5, 4), z(2, 5, 4)]
    cases = [
        (y,), lambda: A.sscan_fwd(*args, y=y),
        (wide,), lambda: A.sscan_bwd(*args, A.sscan_fwd(*args, save_states=True)[2], y, grads={"dx": wide}),
        (cache := z(3, 6, 4),), lambda: A.sscan_step(*[t[:, 0] if t.dim() == 3 else t for t in args], cache),
        (y,), lambda: A.cconv_fwd(args[0], z(6, 3), y=y),
        (wide,), lambda: A.cconv_bwd(args[0], z(6, 3), y, grads={"dx": wide}),
        (kept := z(2, 2, 6),), lambda: A.cconv_step(args[0][:, 0], z(6, 3), kept),
        (y, wide), lambda: A.rmsnorm_fwd(args[0], z(6), residual=wide, total=wide, y=y),
        (wide,), lambda: A.rmsnorm_bwd(y, z(6), z(2, 5), args[0], grads={"dx": wide}),
        (scale := z(2, 5),), lambda: A.rmsnorm_fwd_e4m3(args[0], z(6), scale=scale),
    ]
    for written, call in zip(cases[::2], cases[1::2]):
        before, kept_ = versions(*written), versions(*args)
        call()
        assert all(a > b for a, b in zip(versions(*written), before)) and versions(*args) == kept_


def test_tensors_on_another_stream():
    """Calls given a stream allocate on it; the current stream is left as it was."""
    import aware_conv_amd as A
    x = torch.randn(2, 300, 20, device="cuda")
    w, taps = torch.ones(20, device="cuda"), torch.randn(20, 4, device="cuda")
    want = A.cconv_fwd(A.rmsnorm_fwd(x, w)[0], taps)[0]
    torch.cuda.synchronize()
    side, current = torch.cuda.Stream(), torch.cuda.current_stream()
    for _ in range(5):
        got = A.cconv_fwd(A.rmsnorm_fwd(x, w, stream=side)[0], taps, stream=side)[0]
        torch.empty_like(x).fill_(3)
    side.synchronize()
    assert torch.equal(got, want) and torch.cuda.current_stream() == current
