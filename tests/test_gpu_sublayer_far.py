"""The gated sublayer's operators over matrices whose rows and elements lie past 32-bit offsets, in a process that has called none of
them before it captures them, and in inference mode."""
import subprocess
import sys

import pytest
import torch

import communication_compressed_optimizer_compress_gb300 as ob
import sublayer_ref as ref
import test_gpu_layers as base
from communication_compressed_optimizer_compress_gb300 import layers as L

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _key():
    return torch.tensor([2 ** 33 + 1, 5], dtype=torch.int64, device="cuda")


def _flat(v):
    return [v] if torch.is_tensor(v) else [t for p in v for t in _flat(p)] if isinstance(v, tuple) else []


@pytest.mark.parametrize("pad", [8, 3])
def test_rows_far_apart(pad):
    """Row strides of 2^29 elements and a few: the last of nine rows starts past 2^32 elements (9.7 GB a buffer)."""
    rows, cols, far = 9, 264, 2 ** 29 + pad
    gen = base._gen(pad)
    near = [base._randn(gen, rows, cols + pad, dtype=BF16)[:, :cols] for _ in range(4)]
    wide = [torch.empty(rows * far, dtype=BF16, device="cuda").view(rows, far)[:, :cols] for _ in near]
    for a, b in zip(wide, near):
        a.copy_(b)
    v, key = base._randn(gen, cols, shift=1.0), _key()
    w1, w2 = base._randn(gen, 2 * 136, cols, dtype=BF16, scale=0.1), base._randn(gen, cols, 132, dtype=BF16, scale=0.1)

    def run(x, block, dy, ds):
        o = dict(norm=L.NORM_RMS, block_gamma=v, gate=v, p=0.3, key=key)
        r = L.residual_norm(x, block, v, **o)
        return [L.dropout(x, 0.3, key), *_flat(r), *_flat(L.residual_norm_backward(dy, ds, x, block, v, None, r.rstd, block_rstd=r.block_rstd, **o)),
                L.gated_linear(x, w1), *_flat(L.gated_linear(x, w1, keep="checkpoint")), *_flat(L.gated_linear_backward(dy, ds, w2))]

    for a, b in zip(run(*wide), run(*near)):
        assert torch.equal(a, b)
    assert L.get_status() == ob.OK


def test_residual_norm_past_31_bits_of_elements():
    """2.2e9 elements: a call gives each row what two calls on its halves give it, with the masks of its place; the parameters' gradients are the
    halves' sums, within the roundings of sums of a million rows in parts (2^-12 of the terms' sizes)."""
    rows, cols = 2_200_000, 1000
    gen, key = base._gen(1), _key()
    x, block = (torch.empty(rows, cols, dtype=BF16, device="cuda").normal_(generator=gen) for _ in range(2))
    v, w = base._randn(gen, cols, shift=1.0), base._randn(gen, cols)
    half = rows // 2
    o = dict(block_gamma=v, block_beta=w, gate=v)
    r = L.residual_norm(x, block, v, w, **o)
    g = L.residual_norm_backward(x, block, r.s, block, v, r.mean, r.rstd, block_mean=r.block_mean, block_rstd=r.block_rstd, **o)
    sums = None
    for at in (slice(0, half), slice(half, rows)):
        q = L.residual_norm(x[at], block[at], v, w, **o)
        for a, b in zip(r, q):
            assert torch.equal(a[at], b)
        h = L.residual_norm_backward(x[at], block[at], q.s, block[at], v, q.mean, q.rstd, block_mean=q.block_mean, block_rstd=q.block_rstd, **o)
        assert torch.equal(g.dx[at], h.dx) and torch.equal(g.dblock[at], h.dblock)
        sums = [t.double() for t in h[2:]] if sums is None else [a + t.double() for a, t in zip(sums, h[2:])]
        del q, h
    for a, b in zip(g[2:], sums):
        # terms of about 1, 1.5 and 2 in size, at most 5 on average
        assert float((a.double() - b).abs().max()) <= 2.0 ** -12 * 5 * rows
    del r, g
    s = L.residual_norm(x, block, p=0.5, key=key, site=3).s
    for at in (0, 2 ** 31 // cols - 100, rows - 300):
        stays = ref.stays(300, cols, 0.5, key, 3, first_row=at)
        want = x[at: at + 300].float() + torch.where(stays, 2 * block[at: at + 300].float(), 0.0)
        assert torch.equal(s[at: at + 300], want.to(BF16))
    torch.cuda.empty_cache()


def test_gated_linear_past_31_bits_of_elements():
    """2.4e9 elements of z: a call gives each row what two calls on its halves give it."""
    rows, k, n = 300_032, 64, 4096
    gen = base._gen(2)
    x, w, w2 = base._randn(gen, rows, k, dtype=BF16), base._randn(gen, 2 * n, k, dtype=BF16, scale=0.2), base._randn(gen, k, n, dtype=BF16, scale=0.1)
    half = rows // 2
    for keep in ("values", "checkpoint"):
        h, z = L.gated_linear(x, w, keep=keep)
        dz = L.gated_linear_backward(x, z, w2, need=("dz",))[0]
        for at in (slice(0, half), slice(half, rows)):
            p, q = L.gated_linear(x[at], w, keep=keep)
            assert torch.equal(h[at], p) and all(torch.equal(a[at], b) for a, b in zip(_flat(z), _flat(q)))
            assert torch.equal(dz[at], L.gated_linear_backward(x[at], q, w2, need=("dz",))[0])
        del h, z, dz, p, q
        torch.cuda.empty_cache()
    assert L.get_status() == ob.OK


FIRST = """
import torch
from communication_compressed_optimizer_compress_gb300 import layers as L
torch.manual_seed(0)
for rows, cols, n, pad in ((5, 64, 40, 0), (300, 264, 136, 0), (300, 250, 131, 1), (400, 5000, 72, 0)):
    x, b, dy, ds = (torch.randn(rows, cols + pad, device="cuda").bfloat16()[:, :cols] for _ in range(4))
    w, w2, v = torch.randn(2 * n, cols, device="cuda").bfloat16(), torch.randn(cols, n, device="cuda").bfloat16(), torch.randn(cols, device="cuda")
    key = torch.tensor([3, 4], device="cuda")
    o = dict(block_gamma=v, block_beta=v, gate=v, p=0.2, key=key)
    def step():
        h, z = L.gated_linear(x, w, keep="checkpoint")
        r = L.residual_norm(x, b, v, v, **o)
        g = L.residual_norm_backward(dy, ds, r.s, b, v, r.mean, r.rstd, block_mean=r.block_mean, block_rstd=r.block_rstd, **o)
        return [L.gated_linear(x, w), h, L.dropout(x, 0.2, key), *r, *g, *L.gated_linear_backward(dy, z, w2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, step())), (rows, cols)
    with torch.inference_mode():
        inner = step()
    assert all(torch.equal(p, q) and q.is_inference() for p, q in zip(got, inner)), (rows, cols)
assert L.get_status() == 0
print("done")
"""


def test_captured_before_any_other_call():
    """The first call of each kernel in its process is a captured one; the replay gives what an eager call gives, and one in inference mode."""
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stderr[-2000:]
