"""The gated linear layer, dropout and the residual norm through the C ABI: outputs of any row stride and alignment with what lies
between and around their rows left as it was, inputs among NaN, and the limits of a wait.  Values are compared with the same
operators' dense outputs, within the tolerances of sublayer_ref where a layout changes the order of a sum."""
import ctypes

import pytest
import torch

import communication_compressed_optimizer_compress_gb300 as ob
import sublayer_ref as ref
import test_gpu_layers as base
from communication_compressed_optimizer_compress_gb300 import layers as L
from test_gpu_layers_abi import CODE, LAYOUTS, Out, _among_nan, _done, _ok, _space, _stream

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("offset,gap", LAYOUTS)
@pytest.mark.parametrize("shape", [(1, 24, 40), (16, 264, 136), (33, 65, 129), (130, 72, 257), (300, 1001, 777), (512, 4096, 256), (2600, 264, 520), (5000, 256, 1024)], ids=str)
@pytest.mark.parametrize("keep", [None, "values", "checkpoint"])
def test_gated_linear(shape, offset, gap, keep):
    rows, k, n = shape
    dtype, act = (F16, L.ACT_GELU) if offset % 2 else (BF16, L.ACT_SILU)
    gen, f = base._gen(rows + n), L._functions()
    x, w, b = base._randn(gen, rows, k, dtype=dtype), base._randn(gen, 2 * n, k, dtype=dtype, scale=0.1), base._randn(gen, 2 * n)
    h, z = Out(rows, n, dtype, offset, gap), Out(rows, 2 * n, dtype, offset, gap) if keep == "values" else None
    ck = [Out(rows, n, torch.int8, offset) if i % 2 == 0 else Out(rows, -(-n // 64), F32, offset) for i in range(4)] if keep == "checkpoint" else [None] * 4
    at = lambda o: o.p if o else None  # noqa: E731
    a = L.GatedLinearArgs(x.data_ptr(), k, w.data_ptr(), k, b.data_ptr(), h.p, h.ld, at(z), z.ld if z else 0, *[at(o) for o in ck], rows, k, n, CODE[dtype], act)
    ws, need = _space(f.onebit_gated_linear_forward_workspace, a)
    _ok(f.onebit_gated_linear_forward(a, ws.p, need, _stream()))
    _done(h=h, z=z, workspace=ws, **{f"ck{i}": o for i, o in enumerate(ck)})
    want, kept = L.gated_linear(x, w, b, act, keep=keep) if keep else (L.gated_linear(x, w, b, act), None)
    assert torch.equal(h.values(), want)
    if keep == "values":
        assert torch.equal(z.values(), kept)
    elif keep:
        for o, t in zip(ck, (*kept.gate[:2], *kept.up[:2])):
            assert torch.equal(o.values(), t)


@pytest.mark.parametrize("offset,gap", LAYOUTS)
@pytest.mark.parametrize("shape", [(1, 40, 24), (16, 136, 264), (33, 129, 65), (130, 257, 72), (300, 777, 1001), (512, 256, 4096), (2600, 520, 264), (5000, 1024, 256)], ids=str)
@pytest.mark.parametrize("keep", ["values", "checkpoint"])
def test_gated_linear_backward(shape, offset, gap, keep):
    rows, n, out = shape
    dtype, act, grad = (F16, L.ACT_GELU, F16) if offset % 2 else (BF16, L.ACT_SILU, F32)
    gen, f = base._gen(rows + n + 1), L._functions()
    z, w, dy = base._randn(gen, rows, 2 * n, dtype=dtype), base._randn(gen, out, n, dtype=dtype, scale=0.1), base._randn(gen, rows, out, dtype=dtype)
    kept = z if keep == "values" else L.Gated(L.compress(z[:, :n]), L.compress(z[:, n:]))
    dz, dw, db = Out(rows, 2 * n, dtype, offset, gap), Out(out, n, grad, offset), Out(1, out, grad, offset)
    halves = [None] * 4 if keep == "values" else [t.data_ptr() for c in kept for t in c[:2]]
    a = L.GatedLinearGradArgs(dy.data_ptr(), out, z.data_ptr() if keep == "values" else None, 2 * n, *halves, w.data_ptr(), n, dz.p, dz.ld, dw.p, db.p, rows, n,
                              out, CODE[dtype], act, CODE[grad])
    ws, need = _space(f.onebit_gated_linear_backward_workspace, a)
    _ok(f.onebit_gated_linear_backward(a, ws.p, need, _stream()))
    _done(dz=dz, dw=dw, db=db, workspace=ws)
    g, u = (z[:, :n].double(), z[:, n:].double()) if keep == "values" else (base.values64(kept.gate), base.values64(kept.up))
    # (another layout of dz may sum dh in the epilogue or before it)
    for got, v, t, what in zip((dz.values(), dw.values(), db.values()[0]), ref.gated_grads(dy, g, u, w, act, dtype), (dtype, grad, grad), ("dz", "dw", "db")):
        ref.check(got, v, t, what)


@pytest.mark.parametrize("offset,gap", LAYOUTS)
@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=base.ids)
@pytest.mark.parametrize("shape", [(1, 8), (300, 40), (700, 264), (33, 512), (300, 1024), (200, 1155), (20, 4096), (9, 8192), (5, 20000)], ids=str)
def test_dropout_and_residual_norm(shape, dtype, offset, gap):
    rows, cols = shape
    gen, f = base._gen(rows + cols + 2), L._functions()
    x, b, dy, ds = (base._randn(gen, rows, cols, dtype=dtype) for _ in range(4))
    gamma, beta, bg, bb, gate = (base._randn(gen, cols, shift=s) for s in (1.0, 0.0, 1.0, 0.0, 1.0))
    key = torch.tensor([5, 6], dtype=torch.int64, device="cuda")
    y = Out(rows, cols, dtype, offset, gap)
    _ok(f.onebit_dropout(x.data_ptr(), cols, CODE[dtype], rows, cols, 0.25, key.data_ptr(), 9, y.p, y.ld, _stream()))
    _done(y=y)
    assert torch.equal(y.values(), L.dropout(x, 0.25, key, 9))

    through = torch.where(ref.stays(rows, cols, 0.25, key, 9), 0.5 * ref.factor(0.25), 0.0).double()
    p = dict(gamma=gamma, beta=beta, block_gamma=bg, block_beta=bb, gate=gate)
    s, y = Out(rows, cols, dtype, offset, gap), Out(rows, cols, dtype, offset, gap)
    st = [Out(1, rows, F32, offset) for _ in range(4)]
    a = L.ResidualNormArgs(x.data_ptr(), cols, b.data_ptr(), cols, *[t.data_ptr() for t in (gamma, beta, bg, bb, gate, key)], s.p, s.ld, y.p, y.ld,
                           *[o.p for o in st], rows, cols, CODE[dtype], L.NORM_LAYER, ref.EPS, 0.5, 0.25, 9)
    _ok(f.onebit_residual_norm_forward(a, _stream()))
    names = ("mean", "rstd", "block_mean", "block_rstd")
    _done(s=s, y=y, **dict(zip(names, st)))
    want = ref.residual_norm(x, b, p, True, through)
    ref.check(s.values(), want["s"], dtype, "s")
    ref.check(y.values(), want["y"], dtype, "y")
    for name, o in zip(names, st):
        ref.check(o.values()[0], want[name], F32, name)

    sv, stats = s.values().contiguous(), {name: o.values()[0].clone() for name, o in zip(names, st)}
    dx, db = Out(rows, cols, dtype, offset, gap), Out(rows, cols, dtype, offset, gap)
    gr = [Out(1, cols, F32, offset) for _ in range(5)]
    a = L.ResidualNormGradArgs(dy.data_ptr(), cols, ds.data_ptr(), cols, sv.data_ptr(), cols, b.data_ptr(), cols, *[t.data_ptr() for t in (gamma, bg, bb, gate, key)],
                               *[stats[name].data_ptr() for name in names], dx.p, dx.ld, db.p, db.ld, *[o.p for o in gr], rows, cols, CODE[dtype], L.NORM_LAYER,
                               ob.F32, 0.5, 0.25, 9)
    ws, need = _space(f.onebit_residual_norm_backward_workspace, a)
    _ok(f.onebit_residual_norm_backward(a, ws.p, need, _stream()))
    grads = ("dgamma", "dbeta", "dblock_gamma", "dblock_beta", "dgate")
    _done(dx=dx, dblock=db, workspace=ws, **dict(zip(grads, gr)))
    want = ref.residual_norm_grads(dy, ds, sv, b, p, stats, True, through)
    ref.check(dx.values(), want["dx"], dtype, "dx")
    ref.check(db.values(), want["dblock"], dtype, "dblock")
    for name, o in zip(grads, gr):
        ref.check(o.values()[0], want[name], F32, name)


@pytest.mark.parametrize("offset,gap", LAYOUTS)
@pytest.mark.parametrize("shape", [(1, 8, 24), (16, 264, 136), (33, 65, 129), (300, 1001, 777), (257, 136, 200), (2600, 264, 520)], ids=str)
def test_nothing_around_an_input_enters_a_result(shape, offset, gap):
    rows, k, n = shape
    gen, key = base._gen(rows + k), torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    for dtype in (BF16, F16, F32):
        make = lambda *s, scale=1.0: base._randn(gen, *s, dtype=dtype, scale=scale)  # noqa: E731
        x, w1, w2, dy, z, ds = make(rows, k), make(2 * n, k, scale=0.1), make(k, n, scale=0.1), make(rows, k, scale=0.1), make(rows, 2 * n), make(rows, k)
        v = base._randn(gen, k, shift=1.0)
        inside = [_among_nan(t, offset, gap) for t in (x, w1, w2, dy, z, ds)]

        def run(x, w1, w2, dy, z, ds):
            o = dict(block_gamma=v, block_beta=v, gate=v, p=0.3, key=key)
            r = L.residual_norm(x, ds, v, v, **o)
            got = [L.dropout(x, 0.3, key), *r, *L.residual_norm_backward(dy, ds, x, ds, v, r.mean, r.rstd, block_mean=r.block_mean, block_rstd=r.block_rstd, **o)]
            if dtype is not F32:
                got += [L.gated_linear(x, w1), *L.gated_linear(x, w1, keep="values"), *L.gated_linear_backward(dy, z, w2)]
            return got

        for a, b in zip(run(x, w1, w2, dy, z, ds), run(*inside)):
            assert bool(b.isfinite().all())
            # sums over a row or over rows have another order in another layout
            assert float((a.double() - b.double()).norm()) <= 2.0 ** -7 * float(a.double().norm()) + 1e-6


def test_a_copy_that_never_comes_is_reported():
    """Every wait of the gated products ends: with stages that wait for bytes no copy brings the status says so, and once the hook
    is off the same calls are right again."""
    gen = base._gen(2)
    x, w1 = base._randn(gen, 700, 264, dtype=BF16), base._randn(gen, 1040, 264, dtype=BF16, scale=0.1)
    w2, dy = base._randn(gen, 264, 520, dtype=BF16, scale=0.1), base._randn(gen, 700, 264, dtype=BF16)
    h, z = L.gated_linear(x, w1, keep="values")
    ck = L.gated_linear(x, w1, keep="checkpoint")[1]
    want = [L.gated_linear_backward(dy, k, w2)[0] for k in (z, ck)]
    assert L.get_status() == ob.OK
    for call in (lambda: L.gated_linear(x, w1, keep="values"), lambda: L.gated_linear(x, w1, keep="checkpoint"),
                 lambda: L.gated_linear_backward(dy, z, w2, need=("dz",)), lambda: L.gated_linear_backward(dy, ck, w2, need=("dz",))):
        L.set_fault_injection(ob.FAULT_STALL_COPIES, 16)
        try:
            call()
            assert L.get_status() == ob.ERR_CUDA
        finally:
            L.set_fault_injection(ob.FAULT_NONE)
            L.clear_status()
    assert torch.equal(L.gated_linear(x, w1, keep="values")[0], h)
    assert all(torch.equal(L.gated_linear_backward(dy, k, w2)[0], t) for k, t in zip((z, ck), want))
    assert L.get_status() == ob.OK
