"""The layer operators through the C ABI: outputs of any row stride and alignment, with what lies between and around
their rows left as it was.  Values are compared with the same operators' dense outputs, bit for bit where the layout of
an output does not change the order of any sum, else within the tolerances of test_gpu_layers."""
import ctypes

import pytest
import torch

import communication_compressed_optimizer_compress_gb300 as ob
import test_gpu_layers as base
from communication_compressed_optimizer_compress_gb300 import layers as L

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
CODE = {F32: ob.F32, F16: ob.F16, BF16: ob.BF16}
MARGIN = 1 << 15  # bytes before and behind
LAYOUTS = [(0, 0), (0, 8), (0, 16), (1, 0), (0, 1), (8, 40), (16, 16), (3, 5)]  # offset of the first element, elements between rows


class Out:
    """A matrix of rows x cols somewhere in a buffer of one repeated byte."""

    def __init__(self, rows, cols, dtype, offset=0, gap=0):
        self.size = torch.empty(0, dtype=dtype).element_size()
        self.rows, self.cols, self.ld = rows, cols, cols + gap
        self.start = MARGIN + offset * self.size
        self.bytes = torch.full((self.start + rows * self.ld * self.size + MARGIN,), 0xA5, dtype=torch.uint8, device="cuda")
        self.p = self.bytes.data_ptr() + self.start
        assert self.bytes.data_ptr() % 256 == 0
        self.dtype = dtype

    def values(self):
        inside = self.bytes[self.start: self.start + self.rows * self.ld * self.size].clone()  # a view has to start on its type
        return inside.view(self.dtype).view(self.rows, self.ld)[:, : self.cols]

    def check_surroundings(self, what):
        b, row = self.bytes, self.ld * self.size
        end = self.start + self.rows * row
        assert bool((b[: self.start] == 0xA5).all()) and bool((b[end:] == 0xA5).all()), f"{what}: written outside"
        gaps = b[self.start:end].view(self.rows, row)[:, self.cols * self.size:]
        assert bool((gaps == 0xA5).all()), f"{what}: written between its rows"


def _ok(status):
    assert status == ob.OK, L._functions().onebit_layers_last_error()


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _space(size, *args):
    need = ctypes.c_size_t()
    _ok(size(*args, need))
    return Out(1, max(int(need.value), 1), torch.uint8), need.value


def _done(**outs):
    torch.cuda.synchronize()
    for what, o in outs.items():
        if o is not None:
            o.check_surroundings(what)


SHAPES = [(1, 24, 40), (16, 264, 136), (33, 65, 129), (130, 72, 257), (300, 1001, 777), (512, 4096, 256), (2600, 264, 520), (5000, 256, 1024)]


@pytest.mark.parametrize("offset,gap", LAYOUTS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("case", [(F16, L.ACT_GELU, True, False), (BF16, L.ACT_NONE, False, True), (BF16, L.ACT_GELU_TANH, True, True), (F16, L.ACT_RELU, False, False)],
                         ids=["gelu_ck", "res", "tanh_ck_res", "relu"])
def test_linear(shape, offset, gap, case):
    rows, cols, out = shape
    dtype, act, keep, add = case
    gen = base._gen(rows + out)
    x, w, b = base._randn(gen, rows, cols, dtype=dtype), base._randn(gen, out, cols, dtype=dtype, scale=0.1), base._randn(gen, out)
    res = base._randn(gen, rows, out, dtype=dtype) if add else None
    want = L.linear(x, w, b, act, res, checkpoint=keep)
    y = Out(rows, out, dtype, offset, gap)
    codes, scales = (Out(rows, out, torch.int8, offset), Out(rows, -(-out // 64), F32, offset)) if keep else (None, None)
    a = L.LinearArgs(x.data_ptr(), cols, w.data_ptr(), cols, b.data_ptr(), res.data_ptr() if add else None, out, y.p, y.ld,
                     codes.p if keep else None, scales.p if keep else None, rows, cols, out, CODE[dtype], act)
    f = L._functions()
    ws, need = _space(f.onebit_linear_forward_workspace, a)
    _ok(f.onebit_linear_forward(a, ws.p, need, _stream()))
    _done(y=y, codes=codes, scales=scales, workspace=ws)
    assert torch.equal(y.values(), want[0] if keep else want)
    if keep:
        assert torch.equal(codes.values(), want[1].codes) and torch.equal(scales.values(), want[1].scales)


@pytest.mark.parametrize("offset,gap", LAYOUTS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("case", [(F16, F16, L.ACT_GELU, True, False), (BF16, F32, L.ACT_NONE, False, True), (BF16, BF16, L.ACT_GELU_TANH, False, True), (F16, F32, L.ACT_RELU, True, True)],
                         ids=["gelu_ck", "add_f32", "tanh_add", "relu_ck_add_f32"])
def test_linear_backward(shape, offset, gap, case):
    rows, cols, out = shape
    dtype, grad, act, keep, add = case
    gen = base._gen(rows + out + 1)
    x, w, dy = base._randn(gen, rows, cols, dtype=dtype), base._randn(gen, out, cols, dtype=dtype, scale=0.1), base._randn(gen, rows, out, dtype=dtype)
    ad = base._randn(gen, rows, cols, dtype=dtype) if add else None
    ck = L.compress(x) if keep else None
    want = L.linear_backward(dy, ck if keep else x, w, act, add=ad, grad_dtype=grad)
    dx, dw, db = Out(rows, cols, dtype, offset, gap), Out(out, cols, grad, offset), Out(1, out, grad, offset)
    a = L.LinearGradArgs(dy.data_ptr(), out, None if keep else x.data_ptr(), cols, ck.codes.data_ptr() if keep else None, ck.scales.data_ptr() if keep else None,
                         w.data_ptr(), cols, ad.data_ptr() if add else None, cols, dx.p, dx.ld, dw.p, db.p, rows, cols, out, CODE[dtype], act, CODE[grad])
    f = L._functions()
    ws, need = _space(f.onebit_linear_backward_workspace, a)
    _ok(f.onebit_linear_backward(a, ws.p, need, _stream()))
    _done(dx=dx, dw=dw, db=db, workspace=ws)
    for got, w_, what in zip((dx.values(), dw.values(), db.values()[0]), want, ("dx", "dw", "db")):
        assert torch.equal(got, w_), what


@pytest.mark.parametrize("offset,gap", LAYOUTS)
@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=base.ids)
@pytest.mark.parametrize("shape", [(1, 8), (300, 40), (700, 264), (33, 512), (300, 1024), (200, 1155), (20, 4096), (9, 8192), (5, 20000)], ids=str)
def test_layer_norm_and_checkpoints(shape, dtype, offset, gap):
    rows, cols = shape
    gen, f = base._gen(rows + cols + 2), L._functions()
    x, dy, ad = (base._randn(gen, rows, cols, dtype=dtype, scale=s) for s in (1.0, 0.1, 0.1))
    gamma, beta = base._randn(gen, cols, shift=1.0), base._randn(gen, cols)
    y, mean, rstd = Out(rows, cols, dtype, offset, gap), Out(1, rows, F32, offset), Out(1, rows, F32, offset)
    codes, scales = Out(rows, cols, torch.int8, offset), Out(rows, -(-cols // 64), F32, offset)
    _ok(f.onebit_layer_norm_forward(x.data_ptr(), cols, CODE[dtype], rows, cols, gamma.data_ptr(), beta.data_ptr(), base.EPS, y.p, y.ld, mean.p, rstd.p,
                                    codes.p, scales.p, _stream()))
    _done(y=y, mean=mean, rstd=rstd, codes=codes, scales=scales)
    want, wmean, wrstd = base.ln64(x.double(), gamma.double(), beta.double())
    n, top = min(cols, 64) + 16, x.double().abs().amax(1)
    norm = (n * 2.0 ** -22 * (1 + top * wrstd))[:, None] * (1 + (x.double() - wmean[:, None]).abs() * wrstd[:, None])
    base._within(y.values(), want, base._rounding(want, dtype) + norm * gamma.double().abs() + 2.0 ** -22 * beta.double().abs(), "y")
    base._within(mean.values()[0], wmean, n * 2.0 ** -24 * top, "mean")
    ck = L.compress(x)
    assert torch.equal(codes.values(), ck.codes) and torch.equal(scales.values(), ck.scales)

    codes, scales = Out(rows, cols, torch.int8, offset), Out(rows, -(-cols // 64), F32, offset)
    _ok(f.onebit_checkpoint_compress(x.data_ptr(), cols, CODE[dtype], rows, cols, codes.p, scales.p, _stream()))
    back = Out(rows, cols, dtype, offset, gap)
    _ok(f.onebit_checkpoint_restore(codes.p, scales.p, rows, cols, L.ACT_NONE, back.p, back.ld, CODE[dtype], _stream()))
    _done(codes=codes, scales=scales, restored=back)
    assert torch.equal(codes.values(), ck.codes) and torch.equal(scales.values(), ck.scales) and torch.equal(back.values(), L.restore(ck))

    m, r = mean.values()[0].clone(), rstd.values()[0].clone()
    for kept in (False, True):
        dx, dg, db = Out(rows, cols, dtype, offset, gap), Out(1, cols, F32, offset), Out(1, cols, F32, offset)
        ws, need = _space(f.onebit_layer_norm_backward_workspace, rows, cols)
        _ok(f.onebit_layer_norm_backward(dy.data_ptr(), cols, None if kept else x.data_ptr(), cols, codes.p if kept else None, scales.p if kept else None, CODE[dtype],
                                         rows, cols, gamma.data_ptr(), m.data_ptr(), r.data_ptr(), ad.data_ptr(), cols, dx.p, dx.ld, dg.p, db.p, ob.F32, ws.p, need, _stream()))
        _done(dx=dx, dgamma=dg, dbeta=db, workspace=ws)
        x64 = base.values64(ck) if kept else x.double()
        w, wg, _, xh, g = base._ln_grads64(dy.double(), x64, gamma.double(), m.double(), r.double(), ad.double())
        size = r.double()[:, None] * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
        spread = 1 + (x64.abs().amax(1) * r.double())[:, None]
        base._within(dx.values(), w, base._rounding(w, dtype) + n * 2.0 ** -21 * spread * size + 2.0 ** -22 * ad.double().abs(), "dx")
        k = min(rows, 512) + 32
        base._within(dg.values()[0], wg, (k * 2.0 ** -24 * (dy.double() * xh).abs() + 2.0 ** -21 * spread * dy.double().abs()).sum(0), "dgamma")
        base._within(db.values()[0], dy.double().sum(0), k * 2.0 ** -24 * dy.double().abs().sum(0), "dbeta")


def _among_nan(t, offset, gap):
    """The same matrix with NaN around it and between its rows."""
    rows, cols = t.shape
    flat = torch.full((offset + rows * (cols + gap) + 64,), float("nan"), device="cuda").to(t.dtype)
    m = flat[offset: offset + rows * (cols + gap)].view(rows, cols + gap)[:, :cols]
    m.copy_(t)
    return m


@pytest.mark.parametrize("offset,gap", LAYOUTS)
@pytest.mark.parametrize("shape", [(1, 8, 24), (16, 264, 136), (33, 65, 129), (300, 1001, 777), (257, 136, 200), (512, 4096, 256), (2600, 264, 520)], ids=str)
def test_nothing_around_an_input_enters_a_result(shape, offset, gap):
    rows, cols, out = shape
    gen = base._gen(rows + cols)
    for dtype in (BF16, F16, F32):
        make = lambda *s, scale=1.0: base._randn(gen, *s, dtype=dtype, scale=scale)  # noqa: E731
        x, w, dy, res, ad = make(rows, cols), make(out, cols, scale=0.1), make(rows, out, scale=0.1), make(rows, out), make(rows, cols)
        v = base._randn(gen, cols, shift=1.0)
        inside = [_among_nan(t, offset, gap) for t in (x, w, dy, res, ad)]

        def run(x, w, dy, res, ad):
            _, mean, rstd, ck = n = L.layer_norm(x, v, v, checkpoint=True)
            got = [*n[:3], *ck[:2], *L.compress(x)[:2], *L.layer_norm_backward(ad, x, v, mean, rstd, add=x), *L.layer_norm_backward(ad, ck, v, mean, rstd)]
            if dtype is not F32:
                got += [L.linear(x, w, None, L.ACT_GELU, res), L.linear(x, w, checkpoint=True)[0], *L.linear_backward(dy, x, w, L.ACT_GELU, add=ad),
                        *L.linear_backward(dy, ck, w, grad_dtype=F32), *L.linear_backward(dy, x, w, need=("db",))[2:]]
            return got

        for a, b in zip(run(x, w, dy, res, ad), run(*inside)):
            assert bool(b.isfinite().all())
            # sums over a row or over rows have another order in another layout
            assert float((a.double() - b.double()).norm()) <= 2.0 ** -7 * float(a.double().norm()) + 1e-6
