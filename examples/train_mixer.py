"""Trains a small block of this package's layers and serves it position by position.

    python examples/train_mixer.py [--steps N] [--bits 8] [--half]

The block mixes planes locally with a WTConv layer and globally with a gated
recurrence over the whole plane (GatedScan2d: its gates are WTConv layers too),
both ways; it learns to reproduce, at each position, the running mean of the
plane up to there, which no local layer can.  It is trained by AdamW with
clipped gradients.  Then the recurrence it learned is run over a sequence as it
would be served, a prompt at once and single positions after it, and compared
with one pass over the whole.  Needs an MI355X."""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import aware_conv_amd as A  # noqa: E402


class Block(torch.nn.Module):
    def __init__(self, channels, **f):
        super().__init__()
        self.local = A.WTConv2d(channels, kernel_size=3, levels=2, **f)
        self.whole = A.GatedScan2d(channels, kernel_size=3, levels=2, both=True, **f)
        self.gain = torch.nn.Parameter(torch.ones(channels, 1, 1, **f))

    def forward(self, x):
        return self.local(x) + self.gain * self.whole(x)


def batch(B, C, side, g, dtype):
    x = torch.randn(B, C, side, side, generator=g, device="cuda") + 1
    n = torch.arange(1, side * side + 1, device="cuda")
    y = (x.flatten(2).cumsum(2) / n).view_as(x)
    return x.to(dtype), y.to(dtype)


def train(steps=200, channels=16, side=16, bits=32, dtype=torch.float32, seed=0, say=None):
    """Losses of each step, and the block."""
    torch.manual_seed(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    block = Block(channels, device="cuda", dtype=dtype)
    opt = A.AdamW(block.parameters(), lr=2e-2, weight_decay=0.0, bits=bits, max_norm=1.0)
    scale = 1024.0 if dtype == torch.float16 else 1.0  # keeps fp16 gradients in their range
    opt.grad_scale = 1 / scale
    losses = []
    for step in range(steps):
        x, y = batch(16, channels, side, g, dtype)
        loss = (block(x).float() - y.float()).square().mean()
        opt.zero_grad(set_to_none=True)
        (loss * scale).backward()
        opt.step()
        losses.append(loss.detach())
        if say and (step % 20 == 0 or step == steps - 1):
            say("step %d: loss %.4f" % (step, float(losses[-1])))
    return torch.stack(losses).cpu(), block


def serve(block, length=300, prompt=200, seed=1):
    """Largest difference between one pass over a sequence and a prompt followed by single
    positions, for the block's first recurrence over [1, length, channels]."""
    lam = block.whole.lam[0].detach().contiguous()
    C = lam.numel()
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, r, i = torch.randn(1, length, 3 * C, generator=g, device="cuda").chunk(3, dim=2)
    whole, _, _ = A.gscan_fwd(x, r, i, lam, layout="btc")
    head = [t[:, :prompt] for t in (x, r, i)]
    h, cache, _ = A.gscan_fwd(*head, lam, layout="btc")
    parts = [h]
    for t in range(prompt, length):
        parts.append(A.gscan_step(x[:, t], r[:, t], i[:, t], lam, cache).unsqueeze(1))
    return float((torch.cat(parts, 1) - whole).abs().max())


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--bits", type=int, default=32, choices=(8, 32))
    ap.add_argument("--half", action="store_true")
    a = ap.parse_args()
    losses, block = train(a.steps, bits=a.bits, dtype=torch.float16 if a.half else torch.float32, say=print)
    print("loss %.4f -> %.4f; served position by position within %.1e of one pass"
          % (losses[0], losses[-1], serve(block)))


if __name__ == "__main__":
    main()
