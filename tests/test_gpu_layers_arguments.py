"""What the layer operators meet around their values: parameters that lie anywhere in a flat fp32 buffer, as an
optimizer's often do, tensors of a device that is not current, errors of earlier calls."""
import ctypes

import pytest
import torch

import communication_compressed_optimizer_compress_gb300 as ob
import test_gpu_layers as base
from communication_compressed_optimizer_compress_gb300 import layers as L
from test_gpu_layers_binding import both  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _in_flat(t, offset):
    """The same values as a view that starts `offset` elements into a flat buffer."""
    flat = torch.full((t.numel() + 8,), 77.0, device="cuda")
    flat[offset: offset + t.numel()] = t
    view = flat[offset: offset + t.numel()]
    assert view.data_ptr() % 16 == 4 * offset % 16
    return view


@pytest.mark.parametrize("offset", [1, 2, 3, 4])
@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=base.ids)
@pytest.mark.parametrize("shape", [(3, 8), (33, 768), (300, 1024), (5, 4096), (2, 20000)], ids=str)
def test_layer_norm_parameters_inside_a_flat_buffer(shape, dtype, offset):
    """gamma and beta need no more than their own type's alignment: the results are within the tolerances of
    test_gpu_layers, whatever their offset, with and without checkpoints and a second gradient."""
    rows, cols = shape
    gen = base._gen(rows + cols + offset)
    x, dy, add = (base._randn(gen, rows, cols, dtype=dtype, scale=s, shift=m) for s, m in ((1.0, 0.5), (0.1, 0.0), (0.1, 0.0)))
    gamma, beta = base._randn(gen, cols, shift=1.0), base._randn(gen, cols)
    want, wmean, wrstd = base.ln64(x.double(), gamma.double(), beta.double())
    n, top = min(cols, 64) + 16, x.double().abs().amax(1)
    norm = (n * 2.0 ** -22 * (1 + top * wrstd))[:, None] * (1 + (x.double() - wmean[:, None]).abs() * wrstd[:, None])
    tol = base._rounding(want, dtype) + norm * gamma.double().abs() + 2.0 ** -22 * beta.double().abs()
    for g, b in ((_in_flat(gamma, offset), beta), (gamma, _in_flat(beta, offset)), (_in_flat(gamma, offset), _in_flat(beta, offset))):
        for ck in (False, True):
            y, mean, rstd, *kept = L.layer_norm(x, g, b, base.EPS, checkpoint=ck)
            base._within(y, want, tol, "y")
            if ck:
                base._check_checkpoint(kept[0], x.double())
    g = _in_flat(gamma, offset)
    for src, x64 in ((x, x.double()), (kept[0], base.values64(kept[0]))):
        for ad in (None, add):
            dx, dg, db = L.layer_norm_backward(dy, src, g, mean, rstd, add=ad)
            w, wg, wb, xh, gg = base._ln_grads64(dy.double(), x64, gamma.double(), mean.double(), rstd.double(), None if ad is None else ad.double())
            # the sums of one row over its columns, of one column over the rows, and a few roundings of each term
            size = rstd.double()[:, None] * (gg.abs() + gg.abs().mean(1, keepdim=True) + xh.abs() * (gg * xh).abs().mean(1, keepdim=True))
            spread = 1 + (x64.abs().amax(1) * rstd.double())[:, None]
            base._within(dx, w, base._rounding(w, dtype) + n * 2.0 ** -21 * spread * size + 2.0 ** -22 * add.double().abs(), "dx")
            m = min(rows, 512) + 32
            base._within(dg, wg, (m * 2.0 ** -24 * (dy.double() * xh).abs() + 2.0 ** -21 * spread * dy.double().abs()).sum(0), "dgamma")
            base._within(db, wb, m * 2.0 ** -24 * dy.double().abs().sum(0), "dbeta")


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
def test_tensors_of_a_device_that_is_not_current():
    """The same results, bit for bit, as with the tensors' device current, and the current device stays."""
    gen = base._gen(4)
    x, w, dy = (base._randn(gen, *s, dtype=BF16, scale=0.3) for s in ((300, 264), (136, 264), (300, 136)))
    g = base._randn(gen, 264, shift=1.0)

    def run(x, w, dy, g):
        y, z = L.linear(x, w, activation=L.ACT_GELU, checkpoint=True)
        n, mean, rstd, ck = L.layer_norm(x, g, g, checkpoint=True)
        got = [y, *z[:2], n, mean, rstd, L.restore(ck), *L.layer_norm_backward(x, ck, g, mean, rstd), *L.linear_backward(dy, ck, w, L.ACT_GELU)]
        got += list(L.linear_backward(dy[None], x[None], w))  # not the binding's case
        return got

    want = run(x, w, dy, g)
    with torch.cuda.device(1):
        other = [t.to("cuda:1") for t in (x, w, dy, g)]
        torch.cuda.synchronize()
    assert torch.cuda.current_device() == 0
    got = run(*other)
    assert torch.cuda.current_device() == 0 and L.get_status(torch.cuda.default_stream(1)) == 0
    for a, b in zip(want, got):
        assert b.device.index == 1 and torch.equal(a, b.to("cuda:0"))


def test_errors_of_earlier_code_are_not_reported_again():
    """A call of the optimizer that fails on a capturing stream leaves its error pending in the runtime.  The layer
    operators, through the binding, which would hand a failed call on, and layers.py, do their work all the same."""
    cuda = ctypes.CDLL("libcuda.so.1")
    opt = ob.OneBitAdam([torch.zeros(64, device="cuda")], n_workers=1, warmup_steps=1)
    side = torch.cuda.Stream()

    def fail():
        torch.cuda.synchronize()
        assert cuda.cuStreamBeginCapture_v2(ctypes.c_void_p(side.cuda_stream), 2) == 0
        with pytest.raises(ob.OneBitError):
            ob._check(ob.lib().onebit_adam_get_status(opt.h, ctypes.c_void_p(side.cuda_stream)), "onebit_adam_get_status")
        graph = ctypes.c_void_p()
        assert cuda.cuStreamEndCapture(ctypes.c_void_p(side.cuda_stream), ctypes.byref(graph)) != 0 and not graph

    L._functions()
    b = L._layers_binding
    gen = base._gen(8)
    x, w, dy = (base._randn(gen, *s, dtype=BF16, scale=0.3) for s in ((300, 264), (136, 264), (300, 136)))
    few, v = x[:16], base._randn(gen, 264, shift=1.0)
    ck, (_, mean, rstd) = L.compress(x), L.layer_norm(x, v, v)
    need = ("dx", "dw", "db")
    for call in (lambda: b.compress(x), lambda: b.compress(x[:, :9]), lambda: b.restore(ck, 0), lambda: b.layer_norm(x, v, v, 1e-5, True),
                 lambda: b.layer_norm_backward(x, ck, v, mean, rstd, None, F32), lambda: b.linear(x, w, None, L.ACT_GELU, None, True),
                 lambda: b.linear(few, w, None, 0, None, False), lambda: b.linear_backward(dy, ck, w, L.ACT_GELU, None, None, None, None, need)):
        want = call()
        fail()
        got = call()
        assert got is not None
        flat = _tensors(got)
        assert flat and all(torch.equal(p, q) for p, q in zip(flat, _tensors(want)))
    fail()
    assert L.compress(x[None]).codes.shape == (1, 300, 264)  # layers.py's own path
    opt.free()
    assert L.get_status() == ob.OK


def _tensors(v):
    return [v] if torch.is_tensor(v) else [t for p in v for t in _tensors(p)] if isinstance(v, (tuple, list)) else []


def test_tensors_that_require_a_gradient():
    """Refused with gradient mode on, where the result would silently have no history; taken with it off."""
    gen = base._gen(9)
    make = lambda: {"x": base._randn(gen, 40, 64, dtype=BF16), "w": base._randn(gen, 32, 64, dtype=BF16),  # noqa: E731
                    "dy": base._randn(gen, 40, 32, dtype=BF16), "res": base._randn(gen, 40, 32, dtype=BF16),
                    "v": base._randn(gen, 64), "b": base._randn(gen, 32), "dw": torch.zeros(32, 64, device="cuda"),
                    "mean": base._randn(gen, 40), "codes": torch.zeros(40, 1, device="cuda")}
    ck8 = torch.zeros(40, 64, dtype=torch.int8, device="cuda")
    calls = {
        "x": [lambda t: L.compress(t["x"]), lambda t: L.layer_norm(t["x"], t["v"], t["v"]), lambda t: L.linear(t["x"], t["w"]),
              lambda t: L.linear_backward(t["dy"], t["x"], t["w"]), lambda t: L.layer_norm_backward(t["x"], t["x"], t["v"], t["mean"], t["mean"]),
              lambda t: L.compress(t["x"][None])],
        "w": [lambda t: L.linear(t["x"], t["w"]), lambda t: L.linear_backward(t["dy"], t["x"], t["w"])],
        "dy": [lambda t: L.linear_backward(t["dy"], t["x"], t["w"])], "res": [lambda t: L.linear(t["x"], t["w"], residual=t["res"])],
        "v": [lambda t: L.layer_norm(t["x"], t["v"], t["v"]), lambda t: L.layer_norm_backward(t["x"], t["x"], t["v"], t["mean"], t["mean"])],
        "b": [lambda t: L.linear(t["x"], t["w"], t["b"])], "dw": [lambda t: L.linear_backward(t["dy"], t["x"], t["w"], dw=t["dw"], grad_dtype=F32)],
        "codes": [lambda t: L.restore(L.Checkpoint(ck8, t["codes"], BF16))],
    }
    for name, fs in calls.items():
        for f in fs:
            t = make()
            f(t)
            t[name].requires_grad_()
            with pytest.raises(ValueError, match="requires a gradient"):
                f(t)
            with torch.no_grad():
                f(t)
            f({k: v.detach() for k, v in t.items()})


@pytest.mark.parametrize("rows", [1, 16, 17, 32])
@pytest.mark.parametrize("cols", [8, 136, 376, 384, 632, 640])
@pytest.mark.parametrize("groups", [151, 152, 303, 304, 3647, 3648])
def test_few_rows_on_both_sides_of_the_block_widths(groups, cols, rows):
    """Outputs of 8 columns a group, less three, where the columns of a block change on 152 SMs."""
    out = 8 * groups - 3
    gen = base._gen(groups + rows)
    x, w, b = base._randn(gen, rows, cols, dtype=BF16), base._randn(gen, out, cols, dtype=BF16, scale=0.1), base._randn(gen, out)
    res = base._randn(gen, rows, out, dtype=BF16)
    z, want, size = base._forward64(x, w, b, L.ACT_GELU, res)
    tol = base._rounding(want, BF16) + 1.13 * (cols + 2) * 2.0 ** -23 * size + 2.0 ** -20 * (1 + z.abs()) + 2.0 ** -23 * res.double().abs()
    base._within(L.linear(x, w, b, L.ACT_GELU, res), want, tol, "y")


@pytest.mark.parametrize("rows,cols,out", [(1, 8, 8), (16, 1024, 136), (33, 72, 200), (700, 264, 520), (257, 63, 1), (2500, 520, 264)])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_both_ways_from_python_agree(both, rows, cols, out, pad):
    """The binding and layers.py, bit for bit, where the kernels behind a call differ: few rows, single and paired blocks, cut
    contractions, aligned and odd rows."""
    gen = base._gen(rows + cols + out)
    lay = lambda r, c: base._randn(gen, r, c + pad, dtype=BF16, scale=0.3)[:, :c]  # noqa: E731
    x, w, dy, res = lay(rows, cols), lay(out, cols), lay(rows, out), lay(rows, out)
    b, v = base._randn(gen, out), base._randn(gen, cols)
    both(lambda: L.linear(x, w, b, L.ACT_GELU, res))
    both(lambda: L.linear(x, w, None, L.ACT_RELU, checkpoint=True))
    kept = both(lambda: L.compress(x))
    both(lambda: L.restore(kept, L.ACT_GELU_TANH))
    _, mean, rstd, ck = both(lambda: L.layer_norm(x, v, v, 1e-5, checkpoint=True))
    both(lambda: L.layer_norm_backward(x, ck, v, mean, rstd, add=x, grad_dtype=BF16))
    for src, act in ((x, L.ACT_NONE), (kept, L.ACT_GELU)):
        both(lambda: L.linear_backward(dy, src, w, act, add=x, grad_dtype=F32))
