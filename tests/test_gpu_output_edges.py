"""Outputs of the products whose rows start on 16 bytes but do not end there: nothing behind a row's end is written, neither the caller's
memory between rows nor the other half of a matrix of two."""
import pytest
import torch

import communication_compressed_optimizer_compress_gb300 as ob
import sublayer_ref as ref
import test_gpu_layers as base
from communication_compressed_optimizer_compress_gb300 import layers as L
from test_gpu_layers_abi import CODE, Out, _done, _ok, _space, _stream

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


# the halves of z and dz meet in the middle of 16 bytes: single blocks, a cut contraction, pairs
@pytest.mark.parametrize("rows,k,n", [(22, 591, 108), (264, 8, 92), (504, 40, 252), (512, 4096, 260), (3653, 24, 1508), (3000, 264, 1404), (4775, 64, 1860)], ids=str)
def test_halves_that_meet_inside_16_bytes(rows, k, n):
    gen = base._gen(n)
    dtype = (F16, BF16)[n // 4 % 2]
    x, w, b = base._randn(gen, rows, k, dtype=dtype, shift=0.1), base._randn(gen, 2 * n, k, dtype=dtype, scale=k ** -0.5), base._randn(gen, 2 * n)
    w2, dy = base._randn(gen, k, n, dtype=dtype, scale=n ** -0.5), base._randn(gen, rows, k, dtype=dtype, scale=0.1)
    for act in (L.ACT_SILU, L.ACT_NONE):
        h, g, u = ref.gated(x, w, b, act)
        z64 = torch.cat([g[0], u[0]], 1), torch.cat([g[1], u[1]], 1)
        kept = torch.cat([base._randn(gen, rows, n, dtype=dtype), base._randn(gen, rows, n, dtype=dtype, shift=2.0)], 1)
        checkpoints = L.Gated(L.compress(kept[:, :n]), L.compress(kept[:, n:]))
        for _ in range(4):  # (what is written too far races with what belongs there)
            got, z = L.gated_linear(x, w, b, act, keep="values")
            ref.check(got, h, dtype, "h")
            ref.check(z, z64, dtype, "z")
            for form, g64, u64 in ((kept, kept[:, :n].double(), kept[:, n:].double()), (checkpoints, base.values64(checkpoints.gate), base.values64(checkpoints.up))):
                dz, dw, _ = L.gated_linear_backward(dy, form, w2, act, grad_dtype=F32)
                want = ref.gated_grads(dy, g64, u64, w2, act, dtype)
                ref.check(dz, want[0], dtype, "dz")
                ref.check(dw, want[1], F32, "dw")
    assert L.get_status() == ob.OK


# rows, in, out: single blocks, a cut contraction, pairs; widths of every remainder
SHAPES = [(130, 72, 257), (33, 65, 130), (300, 264, 139), (300, 1001, 780), (512, 4096, 261), (2600, 264, 526), (5000, 256, 1031)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_strided_outputs(shape):
    rows, k, n = shape
    dtype = (F16, BF16)[n % 2]
    gen, f = base._gen(rows + n), L._functions()
    whole = lambda c: -c % 8 + 8  # noqa: E731  (a row stride of whole 16 bytes, with a gap)
    x, w, b = base._randn(gen, rows, k, dtype=dtype), base._randn(gen, n, k, dtype=dtype, scale=0.1), base._randn(gen, n)
    for act, residual in ((L.ACT_GELU, None), (L.ACT_NONE, base._randn(gen, rows, n, dtype=dtype))):
        y = Out(rows, n, dtype, 0, whole(n))
        a = L.LinearArgs(x.data_ptr(), k, w.data_ptr(), k, b.data_ptr(), None if residual is None else residual.data_ptr(), n, y.p, y.ld, None, None, rows, k, n, CODE[dtype], act)
        ws, need = _space(f.onebit_linear_forward_workspace, a)
        _ok(f.onebit_linear_forward(a, ws.p, need, _stream()))
        _done(y=y, workspace=ws)
        assert torch.equal(y.values(), L.linear(x, w, b, act, residual))
    dy, x2 = base._randn(gen, rows, k, dtype=dtype), base._randn(gen, rows, n, dtype=dtype)
    w2 = base._randn(gen, k, n, dtype=dtype, scale=0.1)
    dx = Out(rows, n, dtype, 0, whole(n))
    dw, db = torch.empty(k, n, device="cuda"), torch.empty(k, device="cuda")
    a = L.LinearGradArgs(dy.data_ptr(), k, x2.data_ptr(), n, None, None, w2.data_ptr(), n, None, 0, dx.p, dx.ld, dw.data_ptr(), db.data_ptr(), rows, n, k, CODE[dtype],
                         L.ACT_GELU, ob.F32)
    ws, need = _space(f.onebit_linear_backward_workspace, a)
    _ok(f.onebit_linear_backward(a, ws.p, need, _stream()))
    _done(dx=dx, workspace=ws)
    want = L.linear_backward(dy, x2, w2, L.ACT_GELU, grad_dtype=F32)
    assert torch.equal(dx.values(), want[0]) and torch.equal(dw, want[1]) and torch.equal(db, want[2])

    wg, bg = base._randn(gen, 2 * n, k, dtype=dtype, scale=0.1), base._randn(gen, 2 * n)
    h, z = Out(rows, n, dtype, 0, whole(n)), Out(rows, 2 * n, dtype, 0, whole(2 * n))
    a = L.GatedLinearArgs(x.data_ptr(), k, wg.data_ptr(), k, bg.data_ptr(), h.p, h.ld, z.p, z.ld, None, None, None, None, rows, k, n, CODE[dtype], L.ACT_SILU)
    ws, need = _space(f.onebit_gated_linear_forward_workspace, a)
    _ok(f.onebit_gated_linear_forward(a, ws.p, need, _stream()))
    _done(h=h, z=z, workspace=ws)
    want = L.gated_linear(x, wg, bg, L.ACT_SILU, keep="values")
    assert torch.equal(h.values(), want[0]) and torch.equal(z.values(), want[1])
    dz = Out(rows, 2 * n, dtype, 0, whole(2 * n))
    kept = want[1]
    a = L.GatedLinearGradArgs(dy.data_ptr(), k, kept.data_ptr(), 2 * n, None, None, None, None, w2.data_ptr(), n, dz.p, dz.ld, dw.data_ptr(), db.data_ptr(), rows, n, k,
                              CODE[dtype], L.ACT_SILU, ob.F32)
    ws, need = _space(f.onebit_gated_linear_backward_workspace, a)
    _ok(f.onebit_gated_linear_backward(a, ws.p, need, _stream()))
    _done(dz=dz, workspace=ws)
    grads = ref.gated_grads(dy, kept[:, :n].double(), kept[:, n:].double(), w2, L.ACT_SILU, dtype)
    for got, v, t, what in zip((dz.values(), dw, db), grads, (dtype, F32, F32), ("dz", "dw", "db")):
        ref.check(got, v, t, what)
    assert L.get_status() == ob.OK
