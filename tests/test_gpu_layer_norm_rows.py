"""Layer norm and checkpoints: the widest and narrowest rows of each form that serves a range of widths, and every row
of matrices with more than 2^31 elements.  Checks and tolerances are those of test_gpu_layers."""
import pytest
import torch

import test_gpu_layers as base
from communication_compressed_optimizer_compress_gb300 import layers as L

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("layout", ["dense", "wide", "odd"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=base.ids)
@pytest.mark.parametrize("shape", [(1, 264), (7000, 264), (6001, 400), (5000, 512), (3, 512), (800, 4104), (700, 6000), (650, 8192), (1, 8192),
                                   (330, 8200), (160, 16384), (40, 16392)], ids=str)
def test_forward(shape, dtype, layout):
    base.test_layer_norm(shape, dtype, layout)


def _mostly_one_row(gen, rows, cols, dtype):
    """A matrix whose rows are all the same but for some of their own: at both ends, on both sides of the element 2^31,
    and spread over the whole; which ones they are."""
    at = (1 << 31) // cols
    own = torch.cat([torch.arange(0, 3, device="cuda"), torch.arange(at - 2, at + 3, device="cuda"), torch.arange(rows - 3, rows, device="cuda"),
                     torch.randint(0, rows, (500,), generator=gen, device="cuda")]).unique()
    x = base._randn(gen, 1, cols, dtype=dtype, shift=0.3).expand(rows, cols).contiguous()
    x[own] = base._randn(gen, len(own), cols, dtype=dtype, shift=0.3)
    return x, own


def _others_equal(t, own, what):
    """All rows but `own` hold the same bits; returns one of them."""
    one = torch.ones(len(t), dtype=torch.bool, device="cuda")
    one[own] = False
    first = int(one.nonzero()[0])
    for p in range(0, len(t), 50_000):
        part, keep = t[p:p + 50_000], one[p:p + 50_000]
        same = (part == t[first]).reshape(len(part), -1).all(1)
        assert bool((same | ~keep).all()), (what, p + int((~same & keep).nonzero()[0]))
    return first


def test_every_row_past_2_31_elements():
    """y, its statistics and checkpoint, dx, dgamma and dbeta of 2.2 million rows.  dy is a row of zeros and ones, so that
    dbeta counts the rows without rounding."""
    rows, cols = 2_200_000, 1024
    gen = base._gen(21)
    x, own = _mostly_one_row(gen, rows, cols, BF16)
    gamma, beta = base._randn(gen, cols, shift=1.0), base._randn(gen, cols)
    y, mean, rstd, ck = L.layer_norm(x, gamma, beta, base.EPS, checkpoint=True)
    for t, what in ((y, "y"), (mean, "mean"), (rstd, "rstd"), (ck.codes, "codes"), (ck.scales, "scales")):
        first = _others_equal(t, own, what)
    pick = torch.cat([own, torch.tensor([first], device="cuda")])
    x64 = x[pick].double()
    want, wmean, wrstd = base.ln64(x64, gamma.double(), beta.double())
    n, top = 64 + 16, x64.abs().amax(1)
    base._within(mean[pick], wmean, n * 2.0 ** -24 * top, "mean")
    base._within(rstd[pick], wrstd, wrstd * (n * 2.0 ** -22 + (n * 2.0 ** -24 * top * wrstd) ** 2 + 2.0 ** -20), "rstd")
    norm = (n * 2.0 ** -22 * (1 + top * wrstd))[:, None] * (1 + (x64 - wmean[:, None]).abs() * wrstd[:, None])
    base._within(y[pick], want, base._rounding(want, BF16) + norm * gamma.double().abs() + 2.0 ** -22 * beta.double().abs(), "y")
    base._check_checkpoint(L.Checkpoint(ck.codes[pick], ck.scales[pick], BF16), x64)
    back = L.restore(ck)
    _others_equal(back, own, "restored")
    v = base.values64(L.Checkpoint(ck.codes[pick], ck.scales[pick], BF16))
    base._within(back[pick], v, base._rounding(v, BF16) + v.abs() * 2.0 ** -24, "restored")
    del y, back
    ones = (torch.rand(cols, generator=gen, device="cuda") < 0.5).to(BF16)
    dy = ones.expand(rows, cols).contiguous()
    count = torch.ones(len(pick), dtype=torch.float64, device="cuda")
    count[-1] = rows - len(own)
    m64, r64 = mean[pick].double(), rstd[pick].double()
    for src, s64 in ((x, x64), (ck, v)):
        dx, dg, db = L.layer_norm_backward(dy, src, gamma, mean, rstd)
        _others_equal(dx, own, "dx")
        w, _, _, xh, g = base._ln_grads64(ones.double().expand(len(pick), cols), s64, gamma.double(), m64, r64, None)
        size = r64[:, None] * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
        base._within(dx[pick], w, base._rounding(w, BF16) + n * 2.0 ** -22 * size, "dx")
        assert torch.equal(db, rows * ones.float())
        each = ones.double() * xh
        # a thread adds up the same columns of at most rows / 152 rows, one after another
        base._within(dg, (count[:, None] * each).sum(0), (rows / 152 + 64) * 2.0 ** -24 * (count[:, None] * each.abs()).sum(0), "dgamma")
        del dx


@pytest.mark.parametrize("layout", ["dense", "odd"])
def test_every_checkpoint_past_2_31_elements(layout):
    rows, cols = 33000, 65600
    x, own = _mostly_one_row(base._gen(22), rows, cols, BF16)
    ck = L.compress(base._lay(x, layout))
    for t, what in ((ck.codes, "codes"), (ck.scales, "scales")):
        first = _others_equal(t, own, what)
    pick = torch.cat([own, torch.tensor([first], device="cuda")])
    for part in pick.split(64):
        base._check_checkpoint(L.Checkpoint(ck.codes[part], ck.scales[part], BF16), x[part].double())
    back = L.restore(ck)
    _others_equal(back, own, "restored")
    for part in pick.split(64):
        v = base.values64(L.Checkpoint(ck.codes[part], ck.scales[part], BF16))
        base._within(back[part], v, base._rounding(v, BF16) + v.abs() * 2.0 ** -24, "restored")
