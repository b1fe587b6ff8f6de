"""The gated linear layer against its formulas in 64 bits, at the sizes, strides and values where it can go wrong.
The tolerances are derived in sublayer_ref."""
import pytest
import torch

import communication_compressed_optimizer_compress_gb300 as ob
import sublayer_ref as ref
import test_gpu_layers as base
from communication_compressed_optimizer_compress_gb300 import layers as L
from test_gpu_layers_binding import both  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ACTS = [L.ACT_NONE, L.ACT_RELU, L.ACT_GELU, L.ACT_GELU_TANH, L.ACT_SILU]
KEEP = [None, "values", "checkpoint"]


def _check_checkpoints(z, g, u, eg, eu):
    base._check_checkpoint(z.gate, g, eg)
    base._check_checkpoint(z.up, u, eu)


# rows, in, inner: single tokens, both sides of the few-rows limit, single and paired blocks, tiles that end inside, cut contractions
SHAPES = [(1, 8, 8), (1, 1024, 4096), (3, 40, 1), (16, 264, 136), (17, 72, 200), (32, 1000, 333), (33, 64, 64), (130, 65, 127), (257, 520, 129),
          (300, 1001, 777), (512, 4096, 256), (2500, 264, 520), (5000, 256, 1024)]


@pytest.mark.parametrize("layout", ["dense", "wide", "odd"])
@pytest.mark.parametrize("keep", KEEP)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, keep, layout):
    rows, k, n = shape
    for i, act in enumerate(ACTS):
        dtype = (F16, BF16)[(i + rows) % 2]
        gen = base._gen(rows + k + n + act)
        x, w = base._lay(base._randn(gen, rows, k, dtype=dtype, shift=0.1), layout), base._lay(base._randn(gen, 2 * n, k, dtype=dtype, scale=1.5 / k ** 0.5), layout)
        b = base._randn(gen, 2 * n) if i % 2 else None
        h, g, u = ref.gated(x, w, b, act)
        got = L.gated_linear(x, w, b, act, keep=keep)
        if keep is None:
            got = (got, None)
        ref.check(got[0], h, dtype, "h")
        if keep == "values":
            ref.check(got[1], (torch.cat([g[0], u[0]], 1), torch.cat([g[1], u[1]], 1)), dtype, "z")
        elif keep:
            _check_checkpoints(got[1], g[0], u[0], g[1], u[1])
    assert L.get_status() == ob.OK


# rows, inner, out
BACK = [(1, 8, 8), (3, 1, 40), (16, 136, 264), (33, 64, 64), (130, 127, 65), (257, 130, 520), (300, 777, 1001), (512, 256, 4096), (700, 1030, 520),
        (2500, 520, 264), (5000, 1024, 256)]


@pytest.mark.parametrize("layout", ["dense", "wide", "odd"])
@pytest.mark.parametrize("keep", KEEP[1:])
@pytest.mark.parametrize("shape", BACK, ids=str)
def test_backward(shape, keep, layout):
    rows, n, out = shape
    for i, act in enumerate(ACTS):
        dtype, grad = ((F16, F16), (BF16, F32), (F16, F32), (BF16, BF16), (BF16, F16))[(i + rows) % 5]
        gen = base._gen(rows + n + out + act)
        z = base._lay(base._randn(gen, rows, 2 * n, dtype=dtype, scale=1.5, shift=0.1), layout)
        w, dy = base._lay(base._randn(gen, out, n, dtype=dtype, scale=n ** -0.5), layout), base._lay(base._randn(gen, rows, out, dtype=dtype, scale=0.1), layout)
        g, u, kept = z[:, :n].double(), z[:, n:].double(), z
        if keep == "checkpoint":
            kept = L.Gated(L.compress(z[:, :n]), L.compress(z[:, n:]))
            g, u = base.values64(kept.gate), base.values64(kept.up)
        want = ref.gated_grads(dy, g, u, w, act, dtype)
        got = L.gated_linear_backward(dy, kept, w, act, grad_dtype=grad)
        for t, v, type_, what in zip(got, want, (dtype, grad, grad), ("dz", "dw", "db")):
            ref.check(t, v, type_, what)
        dw, db = torch.full((out, n), 7.0, dtype=grad, device="cuda"), torch.full((out,), 7.0, dtype=grad, device="cuda")
        again = L.gated_linear_backward(dy, kept, w, act, grad_dtype=grad, dw=dw, db=db)
        assert again[1] is dw and again[2] is db and all(torch.equal(a, b) for a, b in zip(got, again))
        for need in (("dz",), ("dw",), ("db",), ("dz", "db"), ()):
            part = L.gated_linear_backward(dy, kept, w, act, grad_dtype=grad, need=need)
            for t, v, full, name in zip(part, want, got, ("dz", "dw", "db")):
                assert (t is not None) == (name in need)
                if t is not None:
                    ref.check(t, v, full.dtype, name)
    assert L.get_status() == ob.OK


@pytest.mark.parametrize("dtype", [F16, BF16], ids=base.ids)
def test_large_arguments_of_the_activations(dtype):
    """Gates of every magnitude, infinities and NaN: each as the formula has it (silu of -inf: its limit 0, within 2e-36)."""
    vals = torch.tensor([0.0, -0.0, 1e-6, -1e-6, 0.3, -3.0, 9.0, -9.0, 40.0, -40.0, 88.0, -88.0, 200.0, -200.0, 3e4, -3e4, float("inf"), float("-inf"), float("nan")])
    g = vals.to(dtype).cuda()
    k = 64
    x = torch.zeros(len(vals), k, dtype=dtype, device="cuda")
    x[:, 0], x[:, 1] = g, 1.0
    w = torch.zeros(2 * 8, k, dtype=dtype, device="cuda")
    w[:8, 0], w[8:, 1] = 1.0, 1.0
    for act in ACTS:
        for rows in (x, x.repeat(5, 1)):  # few rows and a tile
            h, z = L.gated_linear(rows, w, None, act, keep="values")
            alone = L.gated_linear(rows, w, None, act)
            g64 = z[:, :8].double()
            finite = rows[:, :1].isfinite().expand_as(h)
            assert torch.equal(z[:, :8][finite], rows[:, :1].expand_as(h)[finite])
            want = torch.where(g64 == float("-inf"), torch.zeros_like(g64) if act != L.ACT_NONE else g64, ref.act64(act, g64))
            for got in (h, alone):
                bad = z[:, 8:].double().isnan() | want.isnan()  # x of inf times the up rows' zeros
                assert bool((got.isnan() | ~bad).all())
                ok = finite
                base._within(torch.where(ok, got, torch.zeros_like(got)), torch.where(ok, want, torch.zeros_like(want)),
                             torch.where(ok, base._rounding(want, dtype) + 2.0 ** -20 * (1 + g64.abs()), torch.ones_like(want)), "h")


@pytest.mark.parametrize("keep", KEEP)
def test_nan_stays_in_its_row(keep):
    rows, k, n = 300, 200, 130
    gen = base._gen(3)
    x, w = base._randn(gen, rows, k, dtype=BF16), base._randn(gen, 2 * n, k, dtype=BF16, scale=0.1)
    clean = L.gated_linear(x, w, keep=keep)
    x[77, 3], x[200, 5] = float("nan"), float("inf")
    dirty = L.gated_linear(x, w, keep=keep)
    others = [r for r in range(rows) if r not in (77, 200)]
    for a, b in zip(_flat(clean), _flat(dirty)):
        assert torch.equal(a[others], b[others])
    assert bool((dirty if keep is None else dirty[0])[77].isnan().all())
    if keep == "checkpoint":
        assert bool(L.restore(dirty[1].gate)[77].isnan().all()) and bool(L.restore(dirty[1].up)[200].isnan().all())


def _flat(v):
    return [v] if torch.is_tensor(v) else [t for p in v for t in _flat(p)] if isinstance(v, tuple) else []


def test_no_rows():
    x, w, w2 = torch.zeros(0, 64, dtype=BF16, device="cuda"), torch.zeros(32, 64, dtype=BF16, device="cuda"), torch.zeros(40, 16, dtype=BF16, device="cuda")
    h, z = L.gated_linear(x, w, keep="values")
    assert h.shape == (0, 16) and z.shape == (0, 32)
    dz, dw, db = L.gated_linear_backward(torch.zeros(0, 40, dtype=BF16, device="cuda"), z, w2)
    assert dz.shape == (0, 32) and not dw.any() and not db.any()


@pytest.mark.parametrize("rows,k,n", [(1, 8, 8), (16, 1024, 136), (33, 72, 200), (257, 63, 1), (2500, 520, 264)])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_both_ways_from_python_agree(both, rows, k, n, pad):  # noqa: F811
    gen = base._gen(rows + k + n)
    lay = lambda r, c: base._randn(gen, r, c + pad, dtype=BF16, scale=0.3)[:, :c]  # noqa: E731
    x, w, w2, dy, b = lay(rows, k), lay(2 * n, k), lay(k, n), lay(rows, k), base._randn(gen, 2 * n)
    both(lambda: L.gated_linear(x, w, b, L.ACT_GELU))
    z = both(lambda: L.gated_linear(x, w, keep="values"))[1]
    ck = both(lambda: L.gated_linear(x, w, keep="checkpoint"))[1]
    assert isinstance(ck, L.Gated) and isinstance(ck.gate, L.Checkpoint)
    dw, db = torch.empty(k, n, dtype=F32, device="cuda"), torch.empty(k, dtype=F32, device="cuda")
    for kept in (z, ck):
        both(lambda: L.gated_linear_backward(dy, kept, w2, L.ACT_SILU))
        out = both(lambda: L.gated_linear_backward(dy, kept, w2, L.ACT_RELU, F32, dw, db))
        assert out[1] is dw and out[2] is db
        for need in (("dz",), ("dw",), ("db",)):
            both(lambda: L.gated_linear_backward(dy, kept, w2, need=need))


def test_more_dimensions():
    gen = base._gen(6)
    x, w, w2 = base._randn(gen, 4, 50, 64, dtype=F16), base._randn(gen, 72, 64, dtype=F16, scale=0.1), base._randn(gen, 24, 36, dtype=F16)
    h, z = L.gated_linear(x, w, keep="values")
    h2, z2 = L.gated_linear(x.reshape(200, 64), w, keep="values")
    assert h.shape == (4, 50, 36) and torch.equal(h.reshape(200, 36), h2) and torch.equal(z.reshape(200, 72), z2)
    _, ck = L.gated_linear(x, w, keep="checkpoint")
    dy = base._randn(gen, 4, 50, 24, dtype=F16)
    for kept, flat in ((z, z2), (ck, L.gated_linear(x.reshape(200, 64), w, keep="checkpoint")[1])):
        dz, dw, db = L.gated_linear_backward(dy, kept, w2)
        dz2, dw2, db2 = L.gated_linear_backward(dy.reshape(200, 24), flat, w2)
        assert dz.shape == (4, 50, 72) and torch.equal(dz.reshape(200, 72), dz2) and torch.equal(dw, dw2) and torch.equal(db, db2)


def test_tensors_that_require_a_gradient():
    gen = base._gen(9)
    x, w, b = base._randn(gen, 40, 64, dtype=BF16), base._randn(gen, 32, 64, dtype=BF16), base._randn(gen, 32)
    w2, dy = base._randn(gen, 24, 16, dtype=BF16), base._randn(gen, 40, 24, dtype=BF16)
    z = L.gated_linear(x, w, b, keep="values")[1]
    for t, call in ((x, lambda: L.gated_linear(x, w, b)), (w, lambda: L.gated_linear(x, w, b)), (b, lambda: L.gated_linear(x, w, b)),
                    (z, lambda: L.gated_linear_backward(dy, z, w2)), (w2, lambda: L.gated_linear_backward(dy, z, w2)), (dy, lambda: L.gated_linear_backward(dy, z, w2))):
        call()
        t.requires_grad_()
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        with torch.no_grad():
            call()
        t.requires_grad_(False)


@pytest.mark.parametrize("offset", [1, 2, 3, 4])
@pytest.mark.parametrize("shape", [(8, 64, 40), (300, 264, 136), (300, 264, 130), (2500, 264, 520), (512, 4096, 256)], ids=str)
def test_a_bias_inside_a_flat_buffer(shape, offset):
    """The bias needs no more than its own type's alignment, whatever its offset, and nothing around it enters a result."""
    rows, k, n = shape
    gen = base._gen(rows + n)
    x, w = base._randn(gen, rows, k, dtype=BF16), base._randn(gen, 2 * n, k, dtype=BF16, scale=0.1)
    flat = torch.full((2 * n + 8,), float("nan"), device="cuda")
    b = flat[offset: offset + 2 * n]
    b.copy_(base._randn(gen, 2 * n))
    h, g, u = ref.gated(x, w, b, L.ACT_SILU)
    for keep in KEEP:
        got = L.gated_linear(x, w, b, L.ACT_SILU, keep=keep)
        ref.check(got if keep is None else got[0], h, BF16, "h")
        if keep == "checkpoint":
            _check_checkpoints(got[1], g[0], u[0], g[1], u[1])
