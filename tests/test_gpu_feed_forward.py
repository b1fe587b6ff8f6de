"""The feed-forward block of examples/feed_forward.py: its gradients against the formula's in 64 bits and
against differences, its training through both stages of the optimizer, its answer for single tokens.

Tolerance of the gradients, relative in the 2-norm: each of at most 8 roundings to bf16 on the way adds
2^-8; each of the three 8-bit checkpoints is off by at most half of 1/127 of its block's largest value,
taken as 4 times the block's root mean square, 1.6%.  Together 8%: 1/12."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ff():
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _formula(p, x):
    w1, b1, w2, b2, gamma, beta = p
    z = x @ w1.t() + b1
    s = (z * 0.5 * (1 + torch.erf(z / 2 ** 0.5))) @ w2.t() + b2 + x
    c = s - s.mean(1, keepdim=True)
    return c / (c.square().mean(1, keepdim=True) + 1e-12).sqrt() * gamma + beta


def _block(ff, hidden, inner, rows, dtype, seed):
    block = ff.FeedForward(hidden, inner, dtype, seed, scale=0.1)
    gen = torch.Generator("cuda").manual_seed(seed + 10)
    x, dy = (torch.randn(rows, hidden, generator=gen, device="cuda").to(dtype) for _ in range(2))
    exact = [t.double().requires_grad_() for t in (block.low1, block.b1, block.low2, block.b2, block.gamma, block.beta)]
    return block, x, dy, exact, x.double().requires_grad_()


def _rel(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("hidden,inner,rows", [(128, 512, 300), (72, 200, 33), (1024, 4096, 640), (100, 250, 1)])
@pytest.mark.parametrize("grad", [torch.float32, torch.float16])
def test_gradients(ff, hidden, inner, rows, grad):
    block, x, dy, exact, x64 = _block(ff, hidden, inner, rows, torch.bfloat16, 5)
    y, kept = block.forward(x)
    grads = [torch.full_like(p, 7.0, dtype=grad) for p in block.parameters()]
    dx = block.backward(dy, kept, grads, grad)
    y64 = _formula(exact, x64)
    y64.backward(dy.double())
    assert _rel(y, y64.detach()) < 1 / 12
    assert torch.equal(y, block(x)) or rows <= 32  # few rows have their own kernel where nothing is kept
    assert _rel(block(x), y64.detach()) < 1 / 12
    for name, got, want in zip(("dx",) + block.NAMES, [dx] + grads, [x64] + exact):
        assert _rel(got, want.grad) < 1 / 12, name


def test_gradient_along_differences(ff):
    # the loss <y, dy> in 64 bits, a step h either way along a direction; the formula's own error is h^2
    block, x, dy, exact, x64 = _block(ff, 128, 384, 200, torch.bfloat16, 9)
    y, kept = block.forward(x)
    grads = [torch.empty_like(p) for p in block.parameters()]
    dx = block.backward(dy, kept, grads, torch.float32)
    with torch.no_grad():
        for i, got in enumerate([dx] + grads):
            v = got.double() / got.double().norm()  # along the gradient itself the slope is its norm
            at = lambda h: float((_formula([p + h * v if i == k + 1 else p for k, p in enumerate(exact)],  # noqa: E731
                                           x64 + h * v if i == 0 else x64) * dy.double()).sum())
            slope = (at(1e-5) - at(-1e-5)) / 2e-5
            assert abs(slope / float(got.double().norm()) - 1) < 1 / 12, i


@pytest.mark.parametrize("grad", [torch.float32, torch.float16])
def test_training(ff, grad):
    block, teacher = (ff.FeedForward(256, 1024, seed=s) for s in (1, 2))
    gen = torch.Generator("cuda").manual_seed(3)
    xs = [torch.randn(512, 256, generator=gen, device="cuda").bfloat16() for _ in range(4)]
    losses = ff.train(block, teacher, xs, steps=60, warmup_steps=30, grad_dtype=grad)
    assert all(v == v for v in losses)
    assert losses[30] < losses[0] and losses[-1] < losses[30], losses


@pytest.mark.parametrize("rows", [1, 3, 32])
def test_single_tokens(ff, rows):
    # one rounding of h and of s and y each, and the products' operands are exact: 3 of the bound's 8
    block, x, _, exact, x64 = _block(ff, 256, 1024, rows, torch.bfloat16, 11)
    with torch.no_grad():
        assert _rel(block(x), _formula(exact, x64)) < 3 * 2.0 ** -8


def _steps(ff, hidden, inner, rows, n):
    """n steps that each read what the one before wrote, in the same buffers."""
    block, x, dy, _, _ = _block(ff, hidden, inner, rows, torch.bfloat16, 21)
    grads = [torch.empty_like(p) for p in block.parameters()]
    for _ in range(n):
        y, kept = block.forward(x)
        dx = block.backward(dy, kept, grads, torch.float32)
        x.sub_(dx, alpha=0.5)
        dy.copy_(y)
        for p, g in zip(block.parameters(), grads):
            p.sub_(g, alpha=1e-4)
        block.weights_changed()
    return [x, dy] + grads


@pytest.mark.parametrize("hidden,inner,rows", [(1024, 4096, 2048), (72, 200, 33), (100, 250, 700), (256, 1024, 16)])
def test_kernels_that_follow_each_other(ff, monkeypatch, hidden, inner, rows):
    # a kernel comes up beside the last blocks of the one before: the results are those of kernels one at a time
    got = _steps(ff, hidden, inner, rows, 8)
    torch.cuda.synchronize()
    for name in ("compress", "layer_norm", "layer_norm_backward", "linear", "linear_backward"):
        def alone(*a, f=getattr(ff.layers, name), **k):
            torch.cuda.synchronize()
            r = f(*a, **k)
            torch.cuda.synchronize()
            return r
        monkeypatch.setattr(ff.layers, name, alone)
    assert all(torch.equal(a, b) for a, b in zip(got, _steps(ff, hidden, inner, rows, 8)))


def test_graph_with_a_second_stream(ff):
    # a captured call behind two streams' work, and one behind a copy
    block, x, dy, _, _ = _block(ff, 256, 1024, 512, torch.bfloat16, 31)
    other, kept = x.flip(0), torch.empty_like(x)

    def run(side):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            a = ff.layers.linear(other, block.low1, block.b1)
        b = ff.layers.linear(x, block.low1, block.b1, ff.layers.ACT_RELU)
        torch.cuda.current_stream().wait_stream(side)
        s = ff.layers.linear(b, block.low2, residual=x)
        kept.copy_(s)
        return ff.layers.layer_norm(kept, block.gamma, block.beta)[0], ff.layers.linear(a, block.low2)

    want = run(torch.cuda.Stream())
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        got = run(side)
    for _ in range(3):
        for t in got:
            t.zero_()
        kept.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
