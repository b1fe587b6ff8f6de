"""The layer operators (layer norm, linear, 8-bit activation checkpoints) against their definitions in
64 bits, at the sizes, strides and values where they can go wrong.

Tolerances, with u the unit roundoff of the output's type (2^-8 bf16, 2^-11 f16, 2^-24 f32):
* a result is rounded once: u|y|, plus half the smallest subnormal of f16 (2^-25);
* a product of K terms summed in fp32 in any grouping, each step rounded or truncated, is within
  K 2^-23 sum_k |a_k b_k|;
* a layer norm's fp32 statistics over C columns are within C 2^-23 of the row's largest magnitude
  (relative to the standard deviation for the normalised value); 16 such steps bound the rest;
* an operand rounded to 16 bits before a product adds u sum_k |a_k b_k|;
* the activations are within 2^-20 (1 + |z|) and have slope at most 1.13; their derivatives are within
  2^-20 (1 + |z|) and have slope at most 1 (their inputs are given, so only the first term counts).
"""
import math

import pytest
import torch

import communication_compressed_optimizer_compress_gb300 as ob
from communication_compressed_optimizer_compress_gb300 import layers as L

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
ids = {F32: "f32", F16: "f16", BF16: "bf16"}.get


def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _randn(gen, *shape, dtype=F32, scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale + shift).to(dtype)


def _lay(t, layout):
    """The same values in another layout: contiguous, rows in a wider buffer, or that from an odd element."""
    if layout == "dense":
        return t
    pad, off = (16, 8) if layout == "wide" else (5, 1)
    buf = torch.full((t.shape[0], t.shape[1] + pad), 77.0, device="cuda").to(t.dtype)
    buf[:, off: off + t.shape[1]] = t
    return buf[:, off: off + t.shape[1]]


def _within(got, want, tol, what):
    got, bad = got.double(), None
    assert got.shape == want.shape, (what, got.shape, want.shape)
    excess = (got - want).abs() - tol
    bad = ~(excess <= 0)
    if bad.any():
        k = int(torch.argmax(torch.where(bad, torch.nan_to_num(excess, nan=math.inf), torch.full_like(excess, -math.inf)).reshape(-1)))
        t = torch.as_tensor(tol, device=got.device).expand_as(want)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst at {k}: got {got.reshape(-1)[k]}, "
                             f"want {want.reshape(-1)[k]}, tolerance {t.reshape(-1)[k]}")


def _rounding(want, dtype):
    return U[dtype] * want.abs() * (1 + 2.0 ** -10) + 2.0 ** -25 * (dtype == F16)


# ---------------------------------------------------------------- the definitions in 64 bits


def act64(name, z):
    if name == L.ACT_RELU:
        return z.clamp(min=0)
    if name == L.ACT_GELU:
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == L.ACT_GELU_TANH:
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def slope64(name, z):
    if name == L.ACT_RELU:
        return (z > 0).double()
    if name == L.ACT_GELU:
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == L.ACT_GELU_TANH:
        c = math.sqrt(2 / math.pi)
        p = torch.sigmoid(2 * c * (z + 0.044715 * z ** 3))
        return p + 2 * z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def quant64(x):
    """(codes, steps, values) of the 8-bit checkpoint of x, one step per block of 64 columns."""
    codes, steps = [], []
    for piece in x.double().split(64, 1):
        a = piece.abs().amax(1, keepdim=True)
        step = torch.where(a < 2.0 ** -120, torch.zeros_like(a), a / 127)
        codes.append(torch.where(step > 0, torch.round(piece / step.clamp(min=1e-300)), torch.zeros_like(piece)))
        steps.append(step)
    codes, steps = torch.cat(codes, 1), torch.cat(steps, 1)
    return codes, steps, codes * _spread(steps, x.shape[1])


def _spread(scales, cols):
    return scales.double().repeat_interleave(64, 1)[:, :cols]


def values64(ck):
    cols = ck.codes.shape[-1]
    return ck.codes.reshape(-1, cols).double() * _spread(ck.scales.reshape(-1, ck.scales.shape[-1]), cols)


def _check_checkpoint(ck, x64, noise=0.0):
    """Codes and scales of a checkpoint of x64, known to +-noise: scales within the fp32 rounding, each
    value within half a step, and a code off by one only where the rounding is a tie to that noise."""
    codes, steps, _ = quant64(x64)
    nz = torch.as_tensor(noise, dtype=torch.float64, device="cuda").expand_as(x64)
    block_noise = torch.cat([p.amax(1, keepdim=True) for p in nz.split(64, 1)], 1)
    _within(ck.scales, steps, steps * 2.0 ** -23 + block_noise / 127 + (steps == 0) * 1e-38, "scales")
    step = _spread(steps, x64.shape[1])
    off = (ck.codes.double() - codes).abs()
    assert off.max() <= 1 if off.numel() else True
    frac = torch.where(step > 0, (x64 / step.clamp(min=1e-300)).abs().frac(), torch.zeros_like(step))
    tie = (frac - 0.5).abs() <= 127 * 2.0 ** -22 + 3 * nz / step.clamp(min=1e-300)
    assert not ((off > 0) & ~tie).any(), "a code differs away from a tie"
    assert ck.codes.min() >= -127 if off.numel() else True


# ---------------------------------------------------------------- 8-bit checkpoints

CK_SHAPES = [(1, 1), (3, 63), (5, 64), (7, 65), (2, 128), (33, 130), (9, 1024), (300, 4096), (2, 5003), (4099, 72)]


@pytest.mark.parametrize("layout", ["dense", "wide", "odd"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("shape", CK_SHAPES, ids=str)
def test_checkpoint(shape, dtype, layout):
    gen = _gen(shape[0] * 31 + shape[1])
    x = _lay(_randn(gen, *shape, dtype=dtype, shift=0.3), layout)
    ck = L.compress(x)
    _check_checkpoint(ck, x.double())
    v = values64(ck)
    for act in L.ACTIVATIONS.values():
        want = act64(act, v)
        _within(L.restore(ck, act), want, _rounding(want, dtype) + 2.0 ** -20 * (1 + v.abs()) * (act > 1) + v.abs() * 2.0 ** -24, f"restore {act}")


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
def test_checkpoint_special_values(dtype):
    """Zero blocks, blocks below 2^-120, the type's largest and lowest values, infinities and NaN."""
    top = torch.finfo(dtype).max
    x = torch.zeros(8, 200, device="cuda", dtype=dtype)
    x[1, 0], x[1, 64] = top, -top
    x[2, :] = torch.finfo(dtype).tiny
    x[3, 70] = math.inf
    x[3, 0] = 1.0
    x[4, 130] = math.nan
    x[5, 199] = -math.inf
    x[6, 3], x[6, 4] = 2.0 ** -14, -0.0
    ck = L.compress(x)
    back = L.restore(ck)
    assert torch.equal(back[0], x[0])
    assert back[1, 0] == top and back[1, 64] == -top and back[1, 1:64].abs().max() == 0
    assert back[3, :64][0] == 1 and back[3, 64:128].isnan().all() and back[3, 128:].abs().max() == 0
    assert back[4, 128:192].isnan().all() and not back[4, :128].isnan().any() and not back[4, 192:].isnan().any()
    assert back[5, 192:].isnan().all() and not back[5, :192].isnan().any()
    assert back[6, 3] == 2.0 ** -14
    if dtype != F16:  # 2^-126: below what the format holds
        assert back[2].abs().max() == 0 and ck.scales[2].abs().max() == 0
    assert ck.codes[3, 64:128].abs().max() == 0


def test_checkpoint_past_32_bit_offsets():
    rows, cols = 33000, 65600
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    x[-1] = _randn(_gen(5), cols, dtype=BF16)
    ck = L.compress(x)
    _check_checkpoint(L.Checkpoint(ck.codes[-2:], ck.scales[-2:], BF16), x[-2:].double())
    v = values64(L.Checkpoint(ck.codes[-2:], ck.scales[-2:], BF16))
    _within(L.restore(ck)[-2:], v, _rounding(v, BF16) + v.abs() * 2.0 ** -24, "restore")


# ---------------------------------------------------------------- layer norm

LN_SHAPES = [(1, 1), (2, 2), (5, 31), (1, 64), (3, 65), (33, 768), (300, 1024), (1000, 1155), (17, 4096), (3, 8192),
             (5, 20000), (2, 70001), (2500, 40)]
EPS = 1e-5


def ln64(x, gamma, beta, eps=EPS):
    mean = x.mean(1, keepdim=True)
    rstd = (x.var(1, correction=0, keepdim=True) + eps) ** -0.5
    return (x - mean) * rstd * gamma + beta, mean[:, 0], rstd[:, 0]


@pytest.mark.parametrize("layout", ["dense", "wide", "odd"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("shape", LN_SHAPES, ids=str)
def test_layer_norm(shape, dtype, layout):
    rows, cols = shape
    gen = _gen(rows * 7 + cols)
    x = _lay(_randn(gen, rows, cols, dtype=dtype, shift=0.5), layout)
    gamma, beta = _randn(gen, cols, shift=1.0), _randn(gen, cols)
    y, mean, rstd, ck = L.layer_norm(x, gamma, beta, EPS, checkpoint=True)
    y1, mean1, rstd1 = L.layer_norm(x, gamma, beta, EPS)
    assert torch.equal(y, y1) and torch.equal(mean, mean1) and torch.equal(rstd, rstd1)
    x64 = x.double()
    want, wmean, wrstd = ln64(x64, gamma.double(), beta.double())
    top = x64.abs().amax(1)
    n = min(cols, 64) + 16  # steps of the longest serial sum and of the trees over it
    _within(mean, wmean, n * 2.0 ** -24 * top, "mean")
    _within(rstd, wrstd, wrstd * (n * 2.0 ** -22 + (n * 2.0 ** -24 * top * wrstd) ** 2 + 2.0 ** -20), "rstd")
    norm = (n * 2.0 ** -22 * (1 + top * wrstd))[:, None] * (1 + (x64 - wmean[:, None]).abs() * wrstd[:, None])
    _within(y, want, _rounding(want, dtype) + norm * gamma.double().abs() + 2.0 ** -22 * beta.double().abs(), "y")
    _check_checkpoint(ck, x64)


def _ln_grads64(dy, x, gamma, mean, rstd, add):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return (dx if add is None else dx + add), (dy * xh).sum(0), dy.sum(0), xh, g


@pytest.mark.parametrize("kept", ["x", "checkpoint"])
@pytest.mark.parametrize("layout", ["dense", "odd"])
@pytest.mark.parametrize("dtype,grad,add", [(F32, F32, True), (F16, F16, False), (BF16, F32, True), (BF16, BF16, False)],
                         ids=lambda v: ids(v) if isinstance(v, torch.dtype) else str(v))
@pytest.mark.parametrize("shape", LN_SHAPES, ids=str)
def test_layer_norm_backward(shape, dtype, grad, add, layout, kept):
    rows, cols = shape
    gen = _gen(rows * 11 + cols)
    x = _lay(_randn(gen, rows, cols, dtype=dtype, shift=0.5), layout)
    gamma = _randn(gen, cols, shift=1.0)
    dy = _lay(_randn(gen, rows, cols, dtype=dtype, scale=0.1), layout)
    ad = _lay(_randn(gen, rows, cols, dtype=dtype, scale=0.1), layout) if add else None
    _, mean, rstd = L.layer_norm(x, gamma, torch.zeros_like(gamma), EPS)
    src, x64 = x, x.double()
    if kept == "checkpoint":
        src = L.compress(x)
        x64 = values64(src)
    dx, dg, db = L.layer_norm_backward(dy, src, gamma, mean, rstd, add=ad, grad_dtype=grad)
    assert dg.dtype == grad and db.dtype == grad
    d64, m64, r64 = dy.double(), mean.double(), rstd.double()
    want, wg, wb, xh, g = _ln_grads64(d64, x64, gamma.double(), m64, r64, None if ad is None else ad.double())
    n = min(cols, 64) + 16
    top = x64.abs().amax(1, keepdim=True) * r64[:, None]  # the normalised value's own error is 2^-23 of this
    e1, e2 = n * 2.0 ** -23 * g.abs().mean(1, keepdim=True), (n + top) * 2.0 ** -23 * (g * xh).abs().mean(1, keepdim=True)
    e2 = e2 + 2.0 ** -22 * top * g.abs().mean(1, keepdim=True)
    xe = 2.0 ** -22 * (xh.abs() + top)
    tol = r64[:, None] * (2.0 ** -21 * (g.abs() + (xh * (g * xh).mean(1, keepdim=True)).abs()) + e1 + xh.abs() * e2
                          + xe * ((g * xh).mean(1, keepdim=True)).abs())
    if ad is not None:
        tol = tol + 2.0 ** -22 * ad.double().abs()
    _within(dx, want, tol + _rounding(want, dtype), "dx")
    m = min(rows, 512) + 32
    _within(dg, wg, _rounding(wg, grad) + (m * 2.0 ** -24 * (d64 * xh).abs() + d64.abs() * xe).sum(0), "dgamma")
    _within(db, wb, _rounding(wb, grad) + m * 2.0 ** -24 * d64.abs().sum(0), "dbeta")


def test_layer_norm_backward_against_differences():
    """Directional central differences of the 64-bit definition (step 1e-5: truncation ~1e-10 relative)."""
    gen = _gen(3)
    rows, cols = 37, 200
    x, gamma, beta = _randn(gen, rows, cols), _randn(gen, cols, shift=1.0), _randn(gen, cols)
    dy = _randn(gen, rows, cols)
    _, mean, rstd = L.layer_norm(x, gamma, beta, EPS)
    dx, dg, db = L.layer_norm_backward(dy, x, gamma, mean, rstd)
    args = [x.double(), gamma.double(), beta.double()]
    for k, grad in enumerate((dx, dg, db)):
        u = torch.randn(args[k].shape, generator=gen, device="cuda", dtype=torch.float64)
        f = [(ln64(*[a + s * 1e-5 * u if i == k else a for i, a in enumerate(args)])[0] * dy.double()).sum() for s in (1, -1)]
        want = (f[0] - f[1]) / 2e-5
        tol = 1e-5 * (grad.double() * u).abs().sum() / math.sqrt(u.numel()) + 1e-6
        assert abs(float((grad.double() * u).sum() - want)) <= float(tol), k


def test_layer_norm_special_rows():
    """A constant row (variance 0), a row of the type's largest values, a row with NaN and one with inf."""
    x = _randn(_gen(1), 5, 300)
    x[1] = 3.0
    x[2, 7] = math.nan
    x[3, 9] = math.inf
    y, mean, rstd = L.layer_norm(x, torch.ones(300, device="cuda"), torch.zeros(300, device="cuda"), EPS)
    assert torch.equal(y[1], torch.zeros_like(y[1])) and mean[1] == 3 and abs(float(rstd[1]) - EPS ** -0.5) < 1e-3
    assert y[2].isnan().all() and y[3].isnan().all()
    assert y[0].isfinite().all() and y[4].isfinite().all()


def test_layer_norm_many_rows():
    """More rows than any grid, element offsets past 2^31."""
    rows, cols = 2_200_000, 1024
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    x[-3:] = _randn(_gen(2), 3, cols, dtype=BF16)
    gamma, beta = _randn(_gen(3), cols, shift=1.0), _randn(_gen(4), cols)
    y, mean, rstd = L.layer_norm(x, gamma, beta, EPS)
    want, *_ = ln64(x[-3:].double(), gamma.double(), beta.double())
    _within(y[-3:], want, _rounding(want, BF16) + 2.0 ** -14 * (1 + want.abs()), "y")
    dy = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    dy[-3:] = _randn(_gen(6), 3, cols, dtype=BF16)
    dx, dg, db = L.layer_norm_backward(dy, x, gamma, mean, rstd)
    w, wg, wb, *_ = _ln_grads64(dy[-3:].double(), x[-3:].double(), gamma.double(), mean[-3:].double(), rstd[-3:].double(), None)
    _within(dx[-3:], w, _rounding(w, BF16) + 2.0 ** -14 * (1 + w.abs()), "dx")
    _within(dg, wg, 2.0 ** -14 * (1 + wg.abs()), "dgamma")
    _within(db, wb, 2.0 ** -14 * (1 + wb.abs()), "dbeta")


# ---------------------------------------------------------------- the linear layer

LIN_SHAPES = [(1, 1, 1), (1, 64, 128), (3, 7, 5), (1, 1024, 4096), (16, 1024, 4096), (17, 520, 130), (33, 65, 129), (64, 1024, 512),
              (128, 256, 256), (200, 72, 1000), (257, 520, 1030), (300, 1001, 777), (129, 4096, 64), (512, 64, 520),
              (700, 2048, 256), (1500, 136, 264)]


def _forward64(x, w, bias, act, residual):
    z = x.double() @ w.double().t()
    size = x.double().abs() @ w.double().abs().t()
    if bias is not None:
        z, size = z + bias.double(), size + bias.double().abs()
    y = act64(act, z)
    if residual is not None:
        y = y + residual.double()
    return z, y, size


@pytest.mark.parametrize("dtype", [F16, BF16], ids=ids)
@pytest.mark.parametrize("case", [("dense", L.ACT_GELU, True, False, True), ("odd", L.ACT_GELU_TANH, True, True, True),
                                  ("wide", L.ACT_NONE, False, True, False), ("dense", L.ACT_RELU, True, True, False),
                                  ("dense", L.ACT_NONE, False, False, False), ("wide", L.ACT_GELU, False, True, True)],
                         ids=["gelu_bias_ck", "tanh_bias_res_ck_odd", "res_wide", "relu_bias_res", "plain", "gelu_res_ck_wide"])
@pytest.mark.parametrize("shape", LIN_SHAPES, ids=str)
def test_linear(shape, case, dtype):
    rows, cols, out = shape
    layout, act, with_bias, with_res, with_ck = case
    gen = _gen(rows + 3 * cols + 5 * out)
    x = _lay(_randn(gen, rows, cols, dtype=dtype, shift=0.1), layout)
    w = _lay(_randn(gen, out, cols, dtype=dtype, scale=1.5 / math.sqrt(cols)), layout)
    bias = _randn(gen, out, scale=0.1) if with_bias else None
    res = _lay(_randn(gen, rows, out, dtype=dtype), layout) if with_res else None
    got = L.linear(x, w, bias, act, res, checkpoint=with_ck)
    y, ck = got if with_ck else (got, None)
    z, want, size = _forward64(x, w, bias, act, res)
    zerr = (cols + 2) * 2.0 ** -23 * size
    fn = 2.0 ** -20 * (1 + z.abs()) * (act > 1)
    extra = 2.0 ** -23 * res.double().abs() if with_res else 0.0
    _within(y, want, _rounding(want, dtype) + 1.13 * zerr + fn + extra, "y")
    # the error as a whole: one rounding, and the sums' errors far below their bound
    assert float((y.double() - want).norm()) <= float(want.norm()) * (U[dtype] + 2e-5) + 1e-12
    if with_ck:
        _check_checkpoint(ck, z, zerr)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=ids)
@pytest.mark.parametrize("case", [("dense", L.ACT_GELU, "checkpoint", False, None), ("dense", L.ACT_NONE, "x", True, F32),
                                  ("odd", L.ACT_GELU_TANH, "checkpoint", True, None), ("wide", L.ACT_RELU, "x", False, None),
                                  ("odd", L.ACT_NONE, "x", False, F32), ("dense", L.ACT_NONE, "checkpoint", True, None),
                                  ("wide", L.ACT_GELU, "x", True, None)],
                         ids=["gelu_ck", "none_x_add_f32", "tanh_ck_add_odd", "relu_x_wide", "none_x_odd_f32", "none_ck_add", "gelu_x_add_wide"])
@pytest.mark.parametrize("shape", LIN_SHAPES, ids=str)
def test_linear_backward(shape, case, dtype):
    rows, cols, out = shape
    layout, act, kept, with_add, grad = case
    grad = grad or dtype
    gen = _gen(7 * rows + 3 * cols + 5 * out)
    x = _lay(_randn(gen, rows, cols, dtype=dtype, shift=0.1), layout)
    w = _lay(_randn(gen, out, cols, dtype=dtype, scale=1.5 / math.sqrt(cols)), layout)
    dy = _lay(_randn(gen, rows, out, dtype=dtype, scale=0.1), layout)
    add = _lay(_randn(gen, rows, cols, dtype=dtype, scale=0.1), layout) if with_add else None
    src, v = x, x.double()
    if kept == "checkpoint":
        src = L.compress(x)
        v = values64(src)
    dx, dw, db = L.linear_backward(dy, src, w, act, add=add, grad_dtype=grad)
    assert dw.dtype == grad and db.dtype == grad
    d64, w64 = dy.double(), w.double()
    slope = slope64(act, v)
    if act == L.ACT_RELU and kept == "x":
        assert not (v == 0).any()
    prod, size = d64 @ w64, d64.abs() @ w64.abs()
    want = prod * slope + (0 if add is None else add.double())
    tol = slope.abs() * (out + 2) * 2.0 ** -23 * size + prod.abs() * 2.0 ** -20 * (1 + v.abs()) * (act != 0)
    if kept == "checkpoint":  # the value is one fp32 rounding off
        tol = tol + prod.abs() * 2.0 ** -23 * v.abs()
    _within(dx, want, _rounding(want, dtype) * 1.001 + tol + 2.0 ** -22 * (want.abs() + (0 if add is None else add.double().abs())), "dx")
    h = act64(act, v)
    wdw, sdw = d64.t() @ h, d64.abs().t() @ (h.abs() + 2.0 ** -19 * (act > 1))
    rounded = U[dtype] if (kept == "checkpoint" or act != L.ACT_NONE) else 0.0
    sub = (d64.abs().sum(0)[:, None] * 2.0 ** -25 if rounded and dtype == F16 else 0.0)
    _within(dw, wdw, _rounding(wdw, grad) + ((rows + 2) * 2.0 ** -23 + 1.01 * rounded) * sdw + sub
            + (2.0 ** -20 * d64.abs().t() @ (1 + v.abs()) if act > 1 else 0.0), "dw")
    _within(db, d64.sum(0), _rounding(d64.sum(0), grad) + (min(rows, 512) + 32) * 2.0 ** -24 * d64.abs().sum(0), "db")
    only = L.linear_backward(dy, None if act == L.ACT_NONE else src, w, act, add=add, need=("dx",))
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    mine = torch.empty(out * cols, dtype=grad, device="cuda"), torch.empty(out, dtype=grad, device="cuda")
    none, dw2, db2 = L.linear_backward(dy, src, w, act, grad_dtype=grad, dw=mine[0], db=mine[1], need=("dw", "db"))
    assert none is None and dw2 is mine[0] and torch.equal(mine[0].view_as(dw), dw) and torch.equal(mine[1], db)


def test_linear_backward_against_differences():
    """Directional central differences of the 64-bit definition of y = gelu(v) w^T + b."""
    gen = _gen(9)
    rows, cols, out = 40, 96, 72
    v, w = _randn(gen, rows, cols, dtype=F16), _randn(gen, out, cols, dtype=F16, scale=0.1)
    dy, b = _randn(gen, rows, out, dtype=F16, scale=0.5), _randn(gen, out)
    dx, dw, db = L.linear_backward(dy, v, w, L.ACT_GELU, grad_dtype=F32)
    args = [v.double(), w.double(), b.double()]
    for k, (grad, rel) in enumerate(((dx, 2.0 ** -11), (dw, 2.0 ** -11), (db, 2.0 ** -20))):
        u = torch.randn(args[k].shape, generator=gen, device="cuda", dtype=torch.float64)
        f = []
        for s in (1, -1):
            p = [a + s * 1e-5 * u if i == k else a for i, a in enumerate(args)]
            f.append(((act64(L.ACT_GELU, p[0]) @ p[1].t() + p[2]) * dy.double()).sum())
        want = float((f[0] - f[1]) / 2e-5)
        # each gradient element is off by at most rel of what it sums
        size = {0: (dy.double().abs() @ args[1].abs()) * 1.13, 1: dy.double().abs().t() @ act64(L.ACT_GELU, args[0]).abs(),
                2: dy.double().abs().sum(0)}[k]
        tol = 2 * rel * float((size * u.abs()).square().sum().sqrt()) + 1e-6
        assert abs(float((grad.double() * u).sum()) - want) <= tol, k


def test_rows_of_no_tokens():
    for dtype in (F16, BF16):
        x, w = torch.empty(0, 72, dtype=dtype, device="cuda"), torch.ones(40, 72, dtype=dtype, device="cuda")
        y, ck = L.linear(x, w, None, L.ACT_GELU, checkpoint=True)
        assert y.shape == (0, 40) and ck.codes.shape == (0, 40) and ck.scales.shape == (0, 1)
        dx, dw, db = L.linear_backward(torch.empty(0, 40, dtype=dtype, device="cuda"), ck._replace(codes=ck.codes.new_empty(0, 72), scales=ck.scales.new_empty(0, 2)), w, L.ACT_GELU, grad_dtype=F32)
        assert dx.shape == (0, 72) and torch.equal(dw, torch.zeros_like(dw)) and torch.equal(db, torch.zeros_like(db))
        g = torch.ones(72, device="cuda")
        y, mean, rstd = L.layer_norm(x, g, g)
        dx, dg, db = L.layer_norm_backward(x, x, g, mean, rstd)
        assert dx.shape == (0, 72) and torch.equal(dg, torch.zeros_like(dg)) and torch.equal(db, torch.zeros_like(db))
        assert L.restore(L.compress(x)).shape == (0, 72)


def test_leading_dimensions():
    gen = _gen(12)
    x, w = _randn(gen, 2, 5, 3, 64, dtype=BF16), _randn(gen, 48, 64, dtype=BF16, scale=0.1)
    y, ck = L.linear(x, w, checkpoint=True)
    assert y.shape == (2, 5, 3, 48) and ck.codes.shape == y.shape and ck.scales.shape == (2, 5, 3, 1)
    assert torch.equal(y.view(30, 48), L.linear(x.view(30, 64), w))
    g = torch.ones(48, device="cuda")
    n, mean, rstd = L.layer_norm(y, g, g)
    assert mean.shape == (2, 5, 3) and n.shape == y.shape
    dx, dg, db = L.layer_norm_backward(n, ck, g, mean, rstd)
    dv, dw, db = L.linear_backward(dx, x, w)
    assert dx.shape == y.shape and dv.shape == x.shape and dw.shape == w.shape


def test_non_finite_values_stay_in_their_rows_and_columns():
    """A NaN token spoils its own row of y and dx, and every row of dw; the others are untouched."""
    gen = _gen(13)
    x, w = _randn(gen, 300, 136, dtype=BF16), _randn(gen, 264, 136, dtype=BF16, scale=0.1)
    clean = L.linear(x, w, None, L.ACT_GELU)
    x2 = x.clone()
    x2[77, 5] = math.nan
    x2[78, 6] = math.inf
    y, ck = L.linear(x2, w, None, L.ACT_NONE, checkpoint=True)
    assert y[77].isnan().all() and not y[78].isfinite().any()
    assert L.restore(ck)[77].isnan().all() and L.restore(ck)[78].isnan().all() and L.restore(ck)[79].isfinite().all()
    y = L.linear(x2, w, None, L.ACT_GELU)
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[77:79] = False
    assert torch.equal(y[keep], clean[keep])


def test_results_repeat_bit_for_bit():
    gen = _gen(14)
    x, w = _randn(gen, 5000, 264, dtype=BF16), _randn(gen, 520, 264, dtype=BF16, scale=0.1)
    dy = _randn(gen, 5000, 520, dtype=BF16)
    one = L.linear_backward(dy, x, w, L.ACT_GELU, grad_dtype=F32)
    g = _randn(gen, 264, shift=1.0)
    n1 = L.layer_norm(x, g, g)
    b1 = L.layer_norm_backward(x, x, g, n1[1], n1[2])
    for _ in range(3):
        two = L.linear_backward(dy, x, w, L.ACT_GELU, grad_dtype=F32)
        assert all(torch.equal(a, b) for a, b in zip(one, two))
        b2 = L.layer_norm_backward(x, x, g, n1[1], n1[2])
        assert all(torch.equal(a, b) for a, b in zip(b1, b2))


def test_another_stream_and_a_graph():
    gen = _gen(15)
    x, w = _randn(gen, 700, 264, dtype=F16), _randn(gen, 520, 264, dtype=F16, scale=0.1)
    dy = _randn(gen, 700, 520, dtype=F16)
    want = L.linear_backward(dy, x, w, L.ACT_GELU)
    g = _randn(gen, 264, shift=1.0)
    ln = L.layer_norm(x, g, g, checkpoint=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = L.linear_backward(dy, x, w, L.ACT_GELU, stream=side)
    ln2 = L.layer_norm(x, g, g, checkpoint=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(ln[:3], ln2[:3])) and torch.equal(ln[3].codes, ln2[3].codes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = L.linear_backward(dy, x, w, L.ACT_GELU)
        ln2 = L.layer_norm(x, g, g)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(ln[:3], ln2))


def test_linear_past_32_bit_offsets():
    rows, cols, out = 600_000, 64, 4096
    gen = _gen(16)
    x, w = _randn(gen, rows, cols, dtype=BF16), _randn(gen, out, cols, dtype=BF16, scale=0.2)
    y, ck = L.linear(x, w, None, L.ACT_GELU, checkpoint=True)
    for part in (slice(0, 2), slice(524287, 524290), slice(rows - 2, rows)):
        z, want, size = _forward64(x[part], w, None, L.ACT_GELU, None)
        _within(y[part], want, _rounding(want, BF16) + 80 * 2.0 ** -23 * size + 2.0 ** -20 * (1 + z.abs()), "y")
        _check_checkpoint(L.Checkpoint(ck.codes[part], ck.scales[part], BF16), z, 70 * 2.0 ** -23 * size)
    back = L.linear_backward(y, x, w, need=("dw", "db"), grad_dtype=F32)
    want = torch.zeros(out, cols, dtype=torch.float64, device="cuda")
    size, sums = torch.zeros_like(want), torch.zeros(out, dtype=torch.float64, device="cuda")
    for p in range(0, rows, 100_000):
        d, v = y[p:p + 100_000].double(), x[p:p + 100_000].double()
        want += d.t() @ v
        size += d.abs().t() @ v.abs()
        sums += d.sum(0)
    # 600000 terms: in blocks, the bound of a serial sum would say nothing
    _within(back[1], want, 2e-5 * size, "dw")
    _within(back[2], sums, 2e-5 * y.double().abs().sum(0), "db")


def test_a_wait_that_runs_out_is_reported():
    """With the stall hook every product waits for bytes that no copy brings: its waits end after about a
    second, the status says so, and the next product, with the hook off, is right again."""
    gen = _gen(17)
    x, w = _randn(gen, 600, 520, dtype=BF16), _randn(gen, 600, 520, dtype=BF16, scale=0.1)
    big = _randn(gen, 4096, 256, dtype=BF16), _randn(gen, 4096, 256, dtype=BF16, scale=0.1)
    want = L.linear(x, w), L.linear(*big)
    assert L.get_status() == ob.OK
    L.set_fault_injection(ob.FAULT_STALL_COPIES, 16)
    try:
        for a in ((x, w), big):  # both forms: one block a tile, and pairs
            L.linear(*a)
            assert L.get_status() == ob.ERR_CUDA
            L.clear_status()
            assert L.get_status() == ob.OK
    finally:
        L.set_fault_injection(ob.FAULT_NONE)
    assert torch.equal(L.linear(x, w), want[0]) and torch.equal(L.linear(*big), want[1])
    assert L.get_status() == ob.OK
    for kind, value in ((ob.FAULT_STALL_COPIES, 0), (ob.FAULT_STALL_COPIES, 1 << 20), (ob.FAULT_FAIL_ALLOC, 1)):
        with pytest.raises(ob.OneBitError):
            L.set_fault_injection(kind, value)


# ---------------------------------------------------------------- refusals


def test_refusals():
    x, w = torch.zeros(4, 64, dtype=BF16, device="cuda"), torch.zeros(8, 64, dtype=BF16, device="cuda")
    v = torch.zeros(64, device="cuda")
    for bad in (lambda: L.linear(x, w.t()), lambda: L.linear(x, w[:, :32]), lambda: L.linear(x, w.half()),
                lambda: L.linear(x.cpu(), w), lambda: L.linear(x, w, bias=v), lambda: L.linear(x, w, residual=x),
                lambda: L.linear(x[:1].expand(4, 64), w), lambda: L.linear(x.double(), w.double()),
                lambda: L.layer_norm(x, v[:8], v), lambda: L.layer_norm(x, v.half(), v), lambda: L.layer_norm(x.t(), v, v),
                lambda: L.layer_norm_backward(x, w, v, v[:4], v[:4]), lambda: L.layer_norm_backward(x, x, v, v, v[:4]),
                lambda: L.linear_backward(x, x, w), lambda: L.compress(x.int()),
                lambda: L.restore(L.compress(x)._replace(scales=v)), lambda: L.compress(x[:, :0]),
                lambda: L.linear_backward(w[:4, :8].contiguous(), x, w, dw=v)):
        with pytest.raises(ValueError):
            bad()
    for bad, status in ((lambda: L.linear(x.float(), w.float()), ob.ERR_UNSUPPORTED),
                        (lambda: L.linear(x, w, activation=9), ob.ERR_INVALID_ARG),
                        (lambda: L.layer_norm(x, v, v, -1.0), ob.ERR_INVALID_ARG),
                        (lambda: L.layer_norm(x, v, v, math.nan), ob.ERR_INVALID_ARG),
                        (lambda: L.restore(L.compress(x), 7), ob.ERR_INVALID_ARG),
                        (lambda: L.linear_backward(torch.zeros(4, 8, dtype=BF16, device="cuda"), None, w), ob.ERR_INVALID_ARG)):
        with pytest.raises(ob.OneBitError) as e:
            bad()
        assert e.value.status == status and str(e.value).count(":") >= 2, str(e.value)
