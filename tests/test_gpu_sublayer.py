"""A gated feed-forward sublayer of the gated linear layer, the linear layer, dropout and residual norms, run together as a
training step and a step of generation use them: gradients against the formula's in 64 bits and against differences, kernels that
follow each other, captured graphs, streams, two calls at once."""
import pytest
import torch

import communication_compressed_optimizer_compress_gb300 as ob
import sublayer_ref as ref
import test_gpu_layers as base
from communication_compressed_optimizer_compress_gb300 import layers as L

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
P, SCALE, SITE = 0.2, 0.5, 11


class Sublayer:
    """r0 = norm(x); f = W2 (silu(g) u), [g | u] = W1 r0; s = x + scale gate dropout(norm(f)); y = norm(s), all RMS norms."""

    def __init__(self, hidden, inner, dtype, seed, keep="checkpoint"):
        gen = base._gen(seed)
        self.dtype, self.keep = dtype, keep
        self.w1 = base._randn(gen, 2 * inner, hidden, dtype=dtype, scale=1.5 * hidden ** -0.5)
        self.w2 = base._randn(gen, hidden, inner, dtype=dtype, scale=inner ** -0.5)
        self.g0, self.gb, self.g1 = (base._randn(gen, hidden, scale=0.1, shift=1.0) for _ in range(3))
        self.gate = base._randn(gen, hidden, scale=0.1, shift=0.7)
        self.key = torch.tensor([77 + seed, 3], dtype=torch.int64, device="cuda")

    def parameters(self):
        return [self.w1, self.w2, self.g0, self.gb, self.g1, self.gate]

    def _options(self, p):
        return dict(norm=L.NORM_RMS, block_gamma=self.gb, gate=self.gate, scale=SCALE, p=p, key=self.key, site=SITE)

    def forward(self, x, p=P):
        a = L.residual_norm(x, gamma=self.g0, norm=L.NORM_RMS)
        h, z = L.gated_linear(a.y, self.w1, keep=self.keep)
        f = L.linear(h, self.w2)
        r = L.residual_norm(x, f, self.g1, **self._options(p))
        return r.y, (x, a, z, f, r)

    def answer(self, x):
        """y of single tokens: nothing is kept or dropped."""
        a = L.residual_norm(x, gamma=self.g0, norm=L.NORM_RMS)
        f = L.linear(L.gated_linear(a.y, self.w1), self.w2)
        return L.residual_norm(x, f, self.g1, **self._options(0.0)).y

    def backward(self, dy, kept, grad_dtype=F32, p=P):
        x, a, z, f, r = kept
        n = L.residual_norm_backward(dy, None, r.s, f, self.g1, None, r.rstd, block_rstd=r.block_rstd, grad_dtype=grad_dtype, **self._options(p))
        dz, dw2, _ = L.gated_linear_backward(n.dblock, z, self.w2, grad_dtype=grad_dtype, need=("dz", "dw"))
        da, dw1, _ = L.linear_backward(dz, a.y, self.w1, grad_dtype=grad_dtype, need=("dx", "dw"))
        b = L.residual_norm_backward(da, n.dx, x, None, self.g0, None, a.rstd, norm=L.NORM_RMS, has_block=False, grad_dtype=grad_dtype)
        return [b.dx, dw1, dw2, b.dgamma, n.dblock_gamma, n.dgamma, n.dgate]


def _formula(params, x, mask):
    w1, w2, g0, gb, g1, gate = params
    norm = lambda v: v / (v.square().mean(1, keepdim=True) + ref.EPS).sqrt()  # noqa: E731
    g, u = (norm(x) * g0 @ w1.t()).split(w1.shape[0] // 2, 1)
    f = (g * torch.sigmoid(g) * u) @ w2.t()
    return norm(x + SCALE * gate * mask * norm(f) * gb) * g1


def _case(hidden, inner, rows, dtype, seed, keep="checkpoint"):
    layer, gen = Sublayer(hidden, inner, dtype, seed, keep), base._gen(seed + 100)
    x, dy = (base._randn(gen, rows, hidden, dtype=dtype) for _ in range(2))
    mask = ref.stays(rows, hidden, P, layer.key, SITE).double() * ref.factor(P)
    return layer, x, dy, mask


def _rel(got, want):
    return float((got.double() - want).norm() / want.norm())


# Relative in the 2-norm: at most 8 roundings to 16 bits (2^-8 bf16) stand one behind the other on the way to any gradient; of the two
# 8-bit checkpoints each value is off by at most half of 1/127 of its block's largest, taken as 4 times the block's root mean
# square, 1.6%, and enters through a slope of at most 1.1 and a product with the other.  Together 8/256 + 2 * 1.8% < 1/12.
@pytest.mark.parametrize("hidden,inner,rows", [(128, 512, 300), (72, 200, 33), (1024, 4096, 640), (100, 250, 1), (264, 1000, 2100)])
@pytest.mark.parametrize("keep", ["values", "checkpoint"])
def test_gradients(hidden, inner, rows, keep):
    for dtype, grad in ((BF16, F32), (F16, F16)):
        layer, x, dy, mask = _case(hidden, inner, rows, dtype, 5, keep)
        y, kept = layer.forward(x)
        got = layer.backward(dy, kept, grad)
        exact, x64 = [p.double().requires_grad_() for p in layer.parameters()], x.double().requires_grad_()
        y64 = _formula(exact, x64, mask)
        y64.backward(dy.double())
        assert _rel(y, y64.detach()) < 1 / 12
        for name, a, b in zip(("dx", "w1", "w2", "g0", "gb", "g1", "gate"), got, [x64] + exact):
            assert _rel(a, b.grad) < 1 / 12, (name, dtype)
    assert L.get_status() == ob.OK


def test_gradient_along_differences():
    # the loss <y, dy> in 64 bits, a step h either way along each gradient itself, whose slope is its norm
    layer, x, dy, mask = _case(128, 384, 200, BF16, 9)
    y, kept = layer.forward(x)
    got = layer.backward(dy, kept)
    exact, x64 = [p.double() for p in layer.parameters()], x.double()
    for i, g in enumerate(got):
        v = g.double() / g.double().norm()
        at = lambda h: float((_formula([q + h * v if i == k + 1 else q for k, q in enumerate(exact)], x64 + h * v if i == 0 else x64, mask) * dy.double()).sum())  # noqa: E731,E501
        slope = (at(1e-5) - at(-1e-5)) / 2e-5
        assert abs(slope / float(g.double().norm()) - 1) < 1 / 12, i


@pytest.mark.parametrize("rows", [1, 2, 8, 9, 17, 32])
def test_single_tokens(rows):
    # at most 4 roundings on the way to y
    layer, x, _, mask = _case(256, 1024, rows, BF16, 11)
    want = _formula([p.double() for p in layer.parameters()], x.double(), torch.ones_like(mask))
    assert _rel(layer.answer(x), want) < 4 * 2.0 ** -8


def _steps(hidden, inner, rows, n):
    """n steps that each read what the one before wrote, in the same buffers, with new masks."""
    layer, x, dy, _ = _case(hidden, inner, rows, BF16, 21)
    for _ in range(n):
        y, kept = layer.forward(x)
        dx, dw1, dw2, *rest = layer.backward(dy, kept)
        x.sub_(dx, alpha=0.1)
        dy.copy_(L.dropout(y, 0.3, layer.key, 4))
        layer.w1.sub_(dw1, alpha=1e-4)
        layer.w2.sub_(dw2, alpha=1e-4)
        for p, g in zip((layer.g0, layer.gb, layer.g1, layer.gate), rest):
            p.sub_(g, alpha=1e-4)
        layer.key[1] += 1
    return [x, dy, *layer.parameters()]


@pytest.mark.parametrize("hidden,inner,rows", [(1024, 4096, 2048), (72, 200, 33), (100, 250, 700), (256, 1024, 16), (1001, 130, 300)])
def test_kernels_that_follow_each_other(monkeypatch, hidden, inner, rows):
    # a kernel comes up beside the last blocks of the one before: the results are those of kernels one at a time
    got = _steps(hidden, inner, rows, 6)
    torch.cuda.synchronize()
    for name in ("gated_linear", "gated_linear_backward", "dropout", "residual_norm", "residual_norm_backward", "linear", "linear_backward"):
        def alone(*a, f=getattr(L, name), **k):
            torch.cuda.synchronize()
            r = f(*a, **k)
            torch.cuda.synchronize()
            return r
        monkeypatch.setattr(L, name, alone)
    assert all(torch.equal(a, b) for a, b in zip(got, _steps(hidden, inner, rows, 6)))


@pytest.mark.parametrize("hidden,inner,rows", [(256, 1024, 512), (100, 250, 40), (256, 512, 3)])
def test_a_captured_step(hidden, inner, rows):
    """A whole step in a graph, replayed with other inputs, weights and keys, equals the eager one; two graphs that share a pool
    run one after the other."""
    layer, x, dy, _ = _case(hidden, inner, rows, BF16, 31)

    def step():
        y, kept = layer.forward(x)
        return [y, *layer.backward(dy, kept)]

    step()
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.cuda.graph(other, pool=graph.pool()):
        again = step()
    gen = base._gen(3)
    for i in range(3):
        x.copy_(base._randn(gen, rows, hidden, dtype=BF16))
        dy.copy_(base._randn(gen, rows, hidden, dtype=BF16))
        layer.w1.mul_(1.01)
        layer.key[1] = i
        want = [t.clone() for t in step()]
        for g, outs in ((graph, got), (other, again)):
            for t in outs:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_streams_and_two_calls_at_once():
    """`stream=` runs a call there; calls on two streams at once give what they give alone."""
    cases = [_case(512, 1024, 1500, BF16, s) for s in (41, 42)]
    alone = []
    for layer, x, dy, _ in cases:
        y, kept = layer.forward(x)
        alone.append([y, *layer.backward(dy, kept)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(4):
        got = []
        for s, (layer, x, dy, _) in zip(streams, cases):
            with torch.cuda.stream(s):
                y, kept = layer.forward(x)
                got.append([y, *layer.backward(dy, kept)])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for p, q in zip(alone, got) for a, b in zip(p, q))
    layer, x, dy, _ = cases[0]
    s = streams[0]
    s.wait_stream(torch.cuda.current_stream())
    h, z = L.gated_linear(x, layer.w1, keep="values", stream=s)
    dz = L.gated_linear_backward(dy, z, layer.w2, stream=s)
    d = L.dropout(x, 0.5, layer.key, 1, stream=s)
    r = L.residual_norm(x, d, layer.g1, norm=L.NORM_RMS, stream=s)
    g = L.residual_norm_backward(dy, x, r.s, None, layer.g1, None, r.rstd, norm=L.NORM_RMS, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(h, L.gated_linear(x, layer.w1, keep="values")[0]) and torch.equal(dz[1], L.gated_linear_backward(dy, z, layer.w2)[1])
    assert torch.equal(d, L.dropout(x, 0.5, layer.key, 1)) and torch.equal(r.y, L.residual_norm(x, d, layer.g1, norm=L.NORM_RMS).y)
    assert torch.equal(g.dx, L.residual_norm_backward(dy, x, r.s, None, layer.g1, None, r.rstd, norm=L.NORM_RMS).dx)


def test_the_same_results_every_time():
    layer, x, dy, _ = _case(264, 520, 3000, F16, 51)
    first = None
    for _ in range(5):
        y, kept = layer.forward(x)
        got = [y, *layer.backward(dy, kept)]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_the_optimizer_takes_the_gradients():
    """Two workers' gradients of a sublayer go through a warm-up step of 1-bit Adam: finite, moved parameters."""
    layer, x, dy, _ = _case(128, 256, 200, BF16, 61)
    master = [p.float().contiguous() for p in layer.parameters()]
    flat = []
    for rows in (x[:100], x[100:]):
        mask_key = layer.key.clone()
        y, kept = layer.forward(rows.contiguous())
        flat += [g.contiguous() for g in layer.backward(dy[:100].contiguous(), kept, F16)[1:]]
        layer.key.copy_(mask_key + 1)
    before = [p.clone() for p in master]
    with ob.OneBitAdam(master, n_workers=2, warmup_steps=2, lr=1e-3, grad_dtype=F16) as opt:
        opt.warmup_step(flat)
        assert opt.get_status() == ob.OK
    torch.cuda.synchronize()
    assert all(bool(p.isfinite().all()) and not torch.equal(p, b) for p, b in zip(master, before))


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
def test_tensors_of_a_device_that_is_not_current():
    layer, x, dy, _ = _case(128, 256, 100, BF16, 71)
    y, kept = layer.forward(x)
    want = [y, *layer.backward(dy, kept)]
    for name in ("w1", "w2", "g0", "gb", "g1", "gate", "key"):
        setattr(layer, name, getattr(layer, name).to("cuda:1"))
    x1, dy1 = x.to("cuda:1"), dy.to("cuda:1")
    torch.cuda.synchronize()
    y, kept = layer.forward(x1)
    got = [y, *layer.backward(dy1, kept)]
    assert torch.cuda.current_device() == 0
    assert all(b.device.index == 1 and torch.equal(a, b.to("cuda:0")) for a, b in zip(want, got))
