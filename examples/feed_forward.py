"""A transformer's feed-forward block trained by 1-bit Adam, with its activations kept in 8 bits.

    y = layer_norm(W2 gelu(W1 x + b1) + b2 + x)

Each of the n workers runs the block over its own tokens with the layer operators and leaves its gradients
in the optimizer's gradient type; the optimizer warms up, freezes the variance and goes on with compressed
momentum.  The targets come from a second block of the same shape, so that the loss can fall to zero.  After
training the block answers for single tokens with the same operators.

    python examples/feed_forward.py [--hidden 1024 --inner 4096 --tokens 4096 --workers 4]
                                    [--warmup-steps 20 --steps 40] [--dtype bf16] [--grad f32]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import communication_compressed_optimizer_compress_gb300 as ob  # noqa: E402
from communication_compressed_optimizer_compress_gb300 import layers  # noqa: E402

EPS = 1e-12


class FeedForward:
    """The block: fp32 master parameters, which the optimizer updates, and 16-bit weights for the products."""

    NAMES = ("w1", "b1", "w2", "b2", "gamma", "beta")

    def __init__(self, hidden, inner, dtype=torch.bfloat16, seed=0, scale=0.02):
        gen = torch.Generator("cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=gen, device="cuda") * scale

        self.w1, self.b1 = normal(inner, hidden), normal(inner)
        self.w2, self.b2 = normal(hidden, inner), normal(hidden)
        self.gamma, self.beta = 1 + normal(hidden), normal(hidden)
        self.low1, self.low2 = self.w1.to(dtype), self.w2.to(dtype)

    def parameters(self):
        return [getattr(self, name) for name in self.NAMES]

    def weights_changed(self):
        self.low1.copy_(self.w1)
        self.low2.copy_(self.w2)

    def __call__(self, x):
        """y alone: nothing is kept."""
        h = layers.linear(x, self.low1, self.b1, layers.ACT_GELU)
        s = layers.linear(h, self.low2, self.b2, residual=x)
        return layers.layer_norm(s, self.gamma, self.beta, EPS)[0]

    def forward(self, x):
        """y, and what backward() needs: 8-bit checkpoints of x, of the value before the activation and of the
        value before the norm, and the norm's statistics."""
        h, z8 = layers.linear(x, self.low1, self.b1, layers.ACT_GELU, checkpoint=True)
        s = layers.linear(h, self.low2, self.b2, residual=x)
        y, mean, rstd, s8 = layers.layer_norm(s, self.gamma, self.beta, EPS, checkpoint=True)
        return y, (layers.compress(x), z8, s8, mean, rstd)

    def backward(self, dy, kept, grads, grad_dtype):
        """dx.  ``grads`` (one tensor per parameter) takes the parameters' gradients."""
        x8, z8, s8, mean, rstd = kept
        dw1, db1, dw2, db2, dgamma, dbeta = grads
        ds, dg, db = layers.layer_norm_backward(dy, s8, self.gamma, mean, rstd, grad_dtype=grad_dtype)
        dgamma.copy_(dg)
        dbeta.copy_(db)
        dz, _, _ = layers.linear_backward(ds, z8, self.low2, layers.ACT_GELU, grad_dtype=grad_dtype, dw=dw2, db=db2)
        dx, _, _ = layers.linear_backward(dz, x8, self.low1, add=ds, grad_dtype=grad_dtype, dw=dw1, db=db1)
        return dx


def train(block, teacher, xs, steps, warmup_steps, lr=2e-4, grad_dtype=torch.float32, every=0):
    """The loss before each step and after the last, averaged over the workers: mean over tokens of
    |y - target|^2 / hidden."""
    params, losses = block.parameters(), []
    grads = [[torch.empty_like(p, dtype=grad_dtype) for p in params] for _ in xs]
    targets = [teacher(x) for x in xs]
    with ob.OneBitAdam(params, n_workers=len(xs), warmup_steps=warmup_steps, lr=lr, grad_dtype=grad_dtype) as opt:
        flat = [g for worker in grads for g in worker]
        for step in range(steps):
            loss = 0.0
            for x, target, worker in zip(xs, targets, grads):
                y, kept = block.forward(x)
                err = y.float() - target.float()
                loss = loss + err.square().mean()
                # the loss times hidden / 2, a factor that Adam's update does not depend on, keeps f16 gradients normal
                block.backward((err / x.shape[0]).to(y.dtype), kept, worker, grad_dtype)
            losses.append(loss / len(xs))
            if step == warmup_steps:
                opt.freeze_variance()
            (opt.warmup_step if step < warmup_steps else opt.compress_step)(flat)
            block.weights_changed()
            if every and step % every == 0:
                print(f"step {step:4d}  {'warm-up' if step < warmup_steps else 'compressed'}  loss {float(losses[-1]):.6f}")
        if opt.get_status() or layers.get_status():
            raise RuntimeError(f"status {opt.get_status()}, {layers.get_status()}")
    losses.append(sum((block(x).float() - t.float()).square().mean() for x, t in zip(xs, targets)) / len(xs))
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("hidden", 1024), ("inner", 4096), ("tokens", 4096), ("workers", 4), ("warmup-steps", 20), ("steps", 40)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--dtype", choices=("bf16", "f16"), default="bf16")
    ap.add_argument("--grad", choices=("f32", "f16", "bf16"), default="f32")
    a = ap.parse_args()
    types = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
    dtype = types[a.dtype]
    block, teacher = FeedForward(a.hidden, a.inner, dtype, seed=1), FeedForward(a.hidden, a.inner, dtype, seed=2)
    gen = torch.Generator("cuda").manual_seed(3)
    xs = [torch.randn(a.tokens, a.hidden, generator=gen, device="cuda").to(dtype) for _ in range(a.workers)]

    kept = block.forward(xs[0])[1]
    held = sum(t.numel() * t.element_size() for ck in kept[:3] for t in ck[:2]) + sum(t.numel() * t.element_size() for t in kept[3:])
    print(f"kept for the backward pass: {held / a.tokens:.0f} bytes a token; in 16 bits {2 * (2 * a.hidden + a.inner) + 8}")
    del kept

    torch.cuda.synchronize()
    t = time.perf_counter()
    losses = train(block, teacher, xs, a.steps, a.warmup_steps, grad_dtype=types[a.grad], every=5)
    t = time.perf_counter() - t
    print(f"loss {losses[0]:.6f} -> {losses[-1]:.6f}; {a.steps * a.workers * a.tokens / t:,.0f} tokens/s with the first step's set-up")

    token = xs[0][:1].contiguous()
    for _ in range(10):
        block(token)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(100):
        block(token)
    torch.cuda.synchronize()
    print(f"one token: {(time.perf_counter() - t) * 1e4:.1f} us")


if __name__ == "__main__":
    main()
