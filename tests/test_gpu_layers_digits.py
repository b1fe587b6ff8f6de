"""How many digits the layer operators keep where another order of the same operations would lose some.

Each tolerance is that of the operations as the formulas name them, every one rounded to fp32 (2^-24)."""
import math

import pytest
import torch

import test_gpu_layers as base
from communication_compressed_optimizer_compress_gb300 import layers as L

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("kept", ["x", "checkpoint"])
@pytest.mark.parametrize("layout", ["dense", "odd"])
@pytest.mark.parametrize("shape", [(5, 31), (300, 256), (40, 520), (200, 1024), (60, 1155), (20, 2048), (9, 4096), (5, 8192), (3, 9000)], ids=str)
@pytest.mark.parametrize("shift", [0.0, 10.0, 100.0, 1000.0])
def test_normalised_values_of_rows_far_from_zero(shift, shape, layout, kept):
    """x - mean is exact or off by 2^-24 of itself however large the mean is, so that dx and dgamma lose nothing to it.
    (A row of more than 8192 columns reads values of a checkpoint, code times scale, which are rounded themselves.)"""
    rows, cols = shape
    gen = base._gen(rows + cols)
    x = base._lay(base._randn(gen, rows, cols, shift=shift), layout)
    gamma, dy = base._randn(gen, cols, shift=1.0), base._lay(base._randn(gen, rows, cols, scale=0.1), layout)
    _, mean, rstd = L.layer_norm(x, gamma, torch.zeros_like(gamma), base.EPS)
    src, x64 = x, x.double()
    if kept == "checkpoint":
        src = L.compress(x)
        x64 = base.values64(src)
    dx, dg, db = L.layer_norm_backward(dy, src, gamma, mean, rstd)
    d64, r64 = dy.double(), rstd.double()[:, None]
    want, wg, _, xh, g = base._ln_grads64(d64, x64, gamma.double(), mean.double(), rstd.double(), None)
    xe = 2.0 ** -22 * xh.abs()  # of a normalised value
    if kept == "checkpoint" and cols > 8192:
        xe = xe + 2.0 ** -23 * x64.abs() * r64
    base._within(dg, wg, ((min(rows, 512) + 32) * 2.0 ** -24 * (d64 * xh).abs() + d64.abs() * xe).sum(0), "dgamma")
    n = min(cols, 64) + 16  # additions one after another, and of the trees over them
    mean_gx = (g * xh).mean(1, keepdim=True)
    e2 = n * 2.0 ** -23 * (g * xh).abs().mean(1, keepdim=True) + (g.abs() * xe).mean(1, keepdim=True)
    tol = r64 * (2.0 ** -21 * (g.abs() + (xh * mean_gx).abs()) + n * 2.0 ** -23 * g.abs().mean(1, keepdim=True) + xh.abs() * e2 + xe * mean_gx.abs())
    base._within(dx, want, tol + base._rounding(want, F32), "dx")


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=base.ids)
@pytest.mark.parametrize("cols", [64, 1024, 1001, 9000])
def test_constant_rows_are_normalised_to_zero(cols, dtype):
    """x - mean is 0, so dgamma is 0 and dx is what is left of the mean's own term; eps alone decides rstd."""
    x = torch.full((40, cols), 1000.0, device="cuda").to(dtype)
    mean, rstd = x[:, 0].float().contiguous(), torch.full((40,), base.EPS ** -0.5, device="cuda")
    gamma, dy = base._randn(base._gen(1), cols, shift=1.0), base._randn(base._gen(2), 40, cols, dtype=dtype)
    for src in (x, L.compress(x)):
        dx, dg, db = L.layer_norm_backward(dy, src, gamma, mean, rstd)
        if torch.is_tensor(src):
            assert torch.equal(dg, torch.zeros_like(dg))
        else:  # the checkpoint's value of 1000 is off by at most 2^-23 of it
            assert float(dg.abs().max()) <= 40 * 1000 * 2.0 ** -23 * float(rstd[0]) * float(dy.abs().max())


def test_checkpoint_of_the_largest_values_in_fp32():
    """A code times its scale would round past the largest value: 127 (a / 127) with a just below it."""
    top = torch.finfo(F32).max
    x = torch.full((6, 128), top, device="cuda")
    x[:, 1::2] *= 0.5
    ck = L.compress(x)
    mean, rstd = torch.full((6,), top / 2, device="cuda"), torch.full((6,), 2.0 ** -127, device="cuda")
    dy, gamma = base._randn(base._gen(3), 6, 128), torch.ones(128, device="cuda")
    dx, dg, db = L.layer_norm_backward(dy, ck, gamma, mean, rstd)
    _, wg, _, xh, _ = base._ln_grads64(dy.double(), base.values64(ck), gamma.double(), mean.double(), rstd.double(), None)
    base._within(dg, wg, 2.0 ** -20 * (dy.double() * xh).abs().sum(0) + 1e-30, "dgamma")


def _checkpoint_by_definition(x):
    """Codes and scales of an fp32 matrix of whole blocks, operation by operation in fp32: a / 127 and 127 / a rounded,
    x times the latter rounded, and that to the nearest integer, ties to even."""
    v = x.view(x.shape[0], -1, 64)
    a = v.abs().amax(2)
    full = torch.full_like(a, 127.0)  # a tensor: a quotient by a number may be a product with its reciprocal
    zero = a < 2.0 ** -120
    scales = torch.where(zero, 0.0, a / full)
    codes = torch.where(zero[:, :, None], 0.0, torch.round(v * (full / a)[:, :, None]))
    return codes.to(torch.int8).view_as(x), scales


@pytest.mark.parametrize("exponent", [-120, -60, 0, 126])
def test_block_scales_of_every_mantissa(exponent):
    """Both quotients are the rounded ones for every a of a binade: the scale is seen as it is, the factor of the
    codes in values that lie on both sides of a rounding boundary."""
    n, step = 1 << 23, 1 << 18
    k = torch.arange(63, device="cuda") + 0.5 + 64.0 * (torch.arange(63, device="cuda") % 2)
    for first in range(0, n, step):
        m = torch.arange(first, first + step, device="cuda")
        a = ((m + n).double() * 2.0 ** (exponent - 23)).float()[:, None]
        edge = (k[None] * a.double() / 127).float().clamp(max=torch.finfo(F32).max)
        edge = torch.minimum(edge, a)
        side = (m % 3 - 1)[:, None]  # the boundary itself, or a value beside it
        edge = torch.where(side < 0, torch.nextafter(edge, torch.zeros_like(edge)), edge)
        x = torch.cat([a, edge], 1).contiguous()
        ck = L.compress(x)
        codes, scales = _checkpoint_by_definition(x)
        assert torch.equal(ck.scales, scales) and torch.equal(ck.codes, codes), first


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=base.ids)
@pytest.mark.parametrize("shape", [(20000, 256), (3000, 1024), (700, 4096), (90, 20032), (5, 64)], ids=str)
def test_codes_are_the_definitions_in_every_layout(shape, dtype):
    """Products that the rounding to fp32 puts on a tie among them (about one of a thousand codes of random bf16)."""
    rows, cols = shape
    x = base._randn(base._gen(rows), rows, cols, dtype=dtype)
    codes, scales = _checkpoint_by_definition(x.float())
    g = torch.ones(cols, device="cuda")
    for layout in ("dense", "wide", "odd"):
        t = base._lay(x, layout)
        for ck in (L.compress(t), L.layer_norm(t, g, g, checkpoint=True)[3]):
            assert torch.equal(ck.scales, scales)
            assert torch.equal(ck.codes, codes), (layout, int((ck.codes != codes).sum()))


@pytest.mark.parametrize("shape", [(65536, 256), (4096, 1024), (8192, 192), (300, 2048), (40, 4096), (33000, 136), (20000, 203)], ids=str)
@pytest.mark.parametrize("dtype", [F16, BF16], ids=base.ids)
def test_codes_of_a_product_are_those_of_its_values(dtype, shape):
    """With the identity as the weight z is x + bias, rounded once, whatever the product's form: its checkpoint is that of
    the same fp32 matrix by compress(), code by code."""
    rows, cols = shape
    gen = base._gen(cols)
    x, w = base._randn(gen, rows, cols, dtype=dtype), torch.eye(cols, device="cuda", dtype=dtype)
    for bias in (None, base._randn(gen, cols)):
        z = x.float() if bias is None else x.float() + bias
        want = L.compress(z)
        if cols % 64 == 0:
            codes, scales = _checkpoint_by_definition(z)
            assert torch.equal(want.codes, codes) and torch.equal(want.scales, scales)
        for act, residual in ((L.ACT_NONE, None), (L.ACT_GELU, None), (L.ACT_GELU_TANH, x)):
            _, ck = L.linear(x, w, bias, act, residual, checkpoint=True)
            assert torch.equal(ck.scales, want.scales)
            assert torch.equal(ck.codes, want.codes), int((ck.codes != want.codes).sum())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=base.ids)
@pytest.mark.parametrize("cols", [64, 256, 1024, 4096, 16384, 32768])
def test_reciprocal_deviations_are_rounded(cols, dtype):
    """Rows of +-c with whole c have the variance c^2 without any rounding, so that rstd is 1/sqrt(c^2 + eps) rounded:
    within half a unit in the last place, and a thousandth of one for the steps that lead there."""
    c = torch.arange(128, 256, device="cuda", dtype=dtype)
    sign = 1 - 2 * (torch.arange(cols, device="cuda") % 2)
    g = torch.ones(cols, device="cuda")
    for eps in range(40):
        _, mean, rstd = L.layer_norm(c[:, None] * sign.to(dtype), g, g, float(eps))
        assert not mean.any()
        want = (c.double().square() + eps) ** -0.5
        unit = 2.0 ** (torch.floor(torch.log2(want)) - 23)
        base._within(rstd, want, 0.501 * unit, f"rstd, eps {eps}")


def test_reciprocal_deviations_at_the_ends():
    """No variance and no eps, a variance past fp32, one below the normal range."""
    g = torch.ones(64, device="cuda")
    sign = (1 - 2 * (torch.arange(64, device="cuda") % 2)).float()
    x = torch.stack([3.0 * torch.ones_like(sign), 2.0 ** 100 * sign, 2.0 ** -65 * sign])
    assert L.layer_norm(x, g, g, 0.0)[2].tolist() == [math.inf, 0.0, 2.0 ** 65]


@pytest.mark.parametrize("kept", ["x", "checkpoint"])
@pytest.mark.parametrize("act", list(L.ACTIVATIONS.values()), ids=list(L.ACTIVATIONS))
@pytest.mark.parametrize("dtype", [F16, BF16], ids=base.ids)
@pytest.mark.parametrize("shape,need", [((300, 264, 136), ("dx", "dw", "db")), ((333, 520, 1030), ("dw", "db")), ((4096, 512, 256), ("dx", "dw", "db")),
                                        ((9000, 200, 203), ("dx", "dw", "db"))], ids=str)
def test_fp32_gradients_through_an_activation(shape, need, dtype, act, kept):
    """dw in fp32 is dy^T h in fp32 for the h that the forward pass multiplied the weight with: act(v), rounded once to 16
    bits.  Elements of h that lie closer to the middle of two 16-bit values than act(v) is computed may be either of them."""
    rows, cols, out = shape
    gen = base._gen(rows + cols)
    v = base._randn(gen, rows, cols, dtype=dtype, shift=0.1)
    w, dy = base._randn(gen, out, cols, dtype=dtype, scale=0.1), base._randn(gen, rows, out, dtype=dtype, scale=0.1)
    src, v64 = v, v.double()
    if kept == "checkpoint":
        src = L.compress(v)
        v64 = base.values64(src)
    dx, dw, db = L.linear_backward(dy, src, w, act, grad_dtype=F32, need=need)
    assert dw.dtype == F32 and db.dtype == F32 and (dx is None) == ("dx" not in need)
    h = base.act64(act, v64)
    err = 2.0 ** -20 * (1 + v64.abs()) * (act > 1) + 2.0 ** -22 * v64.abs() * (kept == "checkpoint")
    low, high = ((h + s * err).float().to(dtype).double() for s in (-1, 1))
    size = dy.double().abs()
    want = dy.double().t() @ ((low + high) / 2)
    tol = size.t() @ ((high - low).abs() / 2) + (rows + 2) * 2.0 ** -23 * (size.t() @ h.abs())
    base._within(dw, want, tol + base._rounding(want, F32), "dw")
    base._within(db, dy.double().sum(0), (min(rows, 512) + 32) * 2.0 ** -24 * size.sum(0), "db")
