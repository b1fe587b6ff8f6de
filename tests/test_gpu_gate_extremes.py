"""The gated layer's activations and their derivatives at arguments of every magnitude, infinities and NaN, in every form of
the forward and backward pass.

An argument far from 0 leaves the activation within 2^-20 (1 + |g|) and its derivative, which is flat there, within 2^-20 (1 + 40): nothing
grows beyond the magnitudes to which arguments are held.  At infinities the limits count (0, an infinity, a derivative of 0 or 1), within 2^-20."""
import pytest
import torch

import communication_compressed_optimizer_compress_gb300 as ob
import sublayer_ref as ref
import test_gpu_layers as base
from communication_compressed_optimizer_compress_gb300 import layers as L

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ACTS = [L.ACT_NONE, L.ACT_RELU, L.ACT_GELU, L.ACT_GELU_TANH, L.ACT_SILU]
INF, NAN = float("inf"), float("nan")
FINITE = [0.0, -0.0, 1e-6, -1e-6, 0.3, -3.0, 5.9, -5.9, 6.1, -6.1, 9.0, -9.0, 39.0, -39.0, 41.0, -41.0, 86.0, -86.0, 88.0, -88.0, 89.0, -89.0, 130.0, -130.0, 200.0,
          -200.0, 3e4, -3e4]


def _limits(act, g):
    """(activation, derivative) in 64 bits, with their limits at infinities."""
    a, s = ref.act64(act, g), ref.slope64(act, g)
    if act != L.ACT_NONE:
        a, s = torch.where(g == -INF, 0.0, a), torch.where(g == -INF, 0.0, s)
    a, s = torch.where(g == INF, INF, a), torch.where(g == INF, 1.0, s)
    if act == L.ACT_NONE:
        s = torch.where(g.isnan(), 1.0, s)
    elif act == L.ACT_RELU:
        s = torch.where(g.isnan(), NAN, s)
    return a, s


def _same(got, want, tol, what):
    """Within tol where the value is finite, the same infinity or NaN elsewhere."""
    fine = want.isfinite()
    assert torch.equal(got.double()[~fine].nan_to_num(7.0, 1e30, -1e30), want[~fine].nan_to_num(7.0, 1e30, -1e30)), what
    zero = torch.zeros_like(want)
    base._within(torch.where(fine, got.double(), zero), torch.where(fine, want, zero), torch.where(fine, tol, zero), what)


def _bounded(g, most):
    return 2.0 ** -20 * (1 + torch.where(g.isfinite(), g.abs(), 0.0).clamp(max=most))


# few rows, single blocks, a cut contraction, pairs; on 16 bytes and off
@pytest.mark.parametrize("rows,k,n", [(5, 64, 136), (20, 64, 136), (70, 64, 136), (70, 64, 131), (512, 4096, 256), (2500, 264, 520), (2500, 264, 523)], ids=str)
@pytest.mark.parametrize("dtype", [F16, BF16], ids=base.ids)
def test_forward(rows, k, n, dtype):
    """x is 0, so that the bias alone is g and u."""
    vals = torch.tensor(FINITE + [INF, -INF, NAN], device="cuda")
    x, w = torch.zeros(rows, k, dtype=dtype, device="cuda"), base._randn(base._gen(n), 2 * n, k, dtype=dtype)
    at = torch.arange(n, device="cuda")
    g, u = vals[at % len(vals)], torch.where(at // len(vals) % 2 == 0, 1.5, -0.75)
    b = torch.cat([g, u])
    for act in ACTS:
        a, _ = _limits(act, g.double())
        want = (a * u.double()).expand(rows, n)
        want = torch.where(want.abs() > torch.finfo(dtype).max, want * INF, want)
        tol = base._rounding(want, dtype) + 2 * _bounded(g.double(), 4e4)
        for keep in (None, "values", "checkpoint"):
            h = L.gated_linear(x, w, b, act, keep=keep)
            if keep:
                h, z = h
                if keep == "values":
                    assert torch.equal(z.nan_to_num(7.0, 6e4, -6e4), b.to(dtype).nan_to_num(7.0, 6e4, -6e4).expand(rows, 2 * n))
            _same(h, want, tol, (act, keep))
    assert L.get_status() == ob.OK


@pytest.mark.parametrize("rows,n,out", [(70, 136, 64), (70, 131, 64), (512, 256, 4096), (2500, 520, 264), (2500, 523, 264)], ids=str)
@pytest.mark.parametrize("dtype", [F16, BF16], ids=base.ids)
def test_backward(rows, n, out, dtype):
    gen = base._gen(rows + n)
    w, dy = base._randn(gen, out, n, dtype=dtype, scale=out ** -0.5), base._randn(gen, rows, out, dtype=dtype, scale=0.1)
    at = torch.arange(n, device="cuda")
    u = torch.where(at % 3 == 0, 0.5, -0.75).to(dtype).expand(rows, n)
    dh, ed = dy.double() @ w.double(), (out + 2) * 2.0 ** -23 * (dy.double().abs() @ w.double().abs())
    for keep, vals in (("values", FINITE + [INF, -INF, NAN]), ("checkpoint", FINITE)):
        # (a checkpoint's blocks of 64 columns hold one magnitude each, so that none is rounded to 0)
        order = at % len(vals) if keep == "values" else at // 64 % (len(vals) // 2) * 2 + at % 2
        g = torch.tensor(vals, device="cuda")[order].to(dtype).expand(rows, n)
        if keep == "values":
            kept, g64, u64 = torch.cat([g, u], 1), g.double(), u.double()
        else:
            kept = L.Gated(L.compress(g.contiguous()), L.compress(u.contiguous()))
            g64, u64 = base.values64(kept.gate), base.values64(kept.up)
        for act in ACTS:
            a, s = _limits(act, g64)
            dg, du = dh * u64 * s, dh * a
            tg = 1.01 * (ed * (u64 * s).abs() + (dh * u64).abs() * _bounded(g64, 40.0)) + 2.0 ** -22 * dg.abs() + base._rounding(dg, dtype)
            tu = 1.01 * (ed * a.abs() + dh.abs() * _bounded(g64, 4e4)) + 2.0 ** -22 * du.abs() + base._rounding(du, dtype)
            dz = L.gated_linear_backward(dy, kept, w, act, need=("dz",))[0]
            over = torch.finfo(dtype).max
            _same(dz[:, :n], dg, tg, (keep, act, "dg"))
            _same(dz[:, n:], torch.where(du.abs() > over, du * INF, du), tu, (keep, act, "du"))
    assert L.get_status() == ob.OK
