"""The residual sum with the norms around it against its formulas in 64 bits, at the sizes, strides and values where it can
go wrong.  The tolerances are derived in sublayer_ref."""
import itertools

import pytest
import torch

import sublayer_ref as ref
import test_gpu_layers as base
from communication_compressed_optimizer_compress_gb300 import layers as L
from test_gpu_layers_binding import both  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
# a block, a norm before the next block, a norm behind the block, a gate, a dropout rate
OPTIONS = [(b, pre, post, gate, p) for b, pre, post, gate, p in itertools.product((True, False), (True, False), (True, False), (True, False), (0.0, 0.3))
           if (b or pre) and (b or not (post or gate or p))]


def _key():
    return torch.tensor([2 ** 61 + 12345, 678], dtype=torch.int64, device="cuda")


def _call(gen, rows, cols, dtype, layout, layer, option, size=1.0):
    """Inputs and keyword arguments of one call."""
    has_block, pre, post, gate, p = option
    make = lambda **k: base._lay(base._randn(gen, rows, cols, dtype=dtype, **k), layout)  # noqa: E731
    vector = lambda there, **k: base._randn(gen, cols, **k) if there else None  # noqa: E731
    params = dict(gamma=vector(pre, shift=1.0), beta=vector(pre and layer), block_gamma=vector(post, shift=1.0), block_beta=vector(post and layer),
                  gate=vector(gate))
    x, block = make(scale=size, shift=0.3), make(scale=0.7 * size, shift=-0.2) if has_block else None
    opts = dict(norm=L.NORM_LAYER if layer else L.NORM_RMS, scale=0.75, p=p, key=_key() if p else None, site=9)
    through = None
    if has_block:
        through = torch.full((rows, cols), 0.75, dtype=torch.float64, device="cuda")
        if p:
            through = torch.where(ref.stays(rows, cols, p, opts["key"], 9), through * ref.factor(p), 0.0)
    return x, block, params, opts, through


SHAPES = [(1, 1), (1, 8), (50, 3), (41, 7), (3, 40), (33, 72), (5, 200), (16, 256), (300, 264), (17, 512), (9, 768), (40, 1024), (150, 1155), (7, 1600), (1300, 520), (12, 2048), (6, 3001),
          (5, 4096), (4, 5000), (4, 8192), (3, 8200), (2, 20000), (5, 33000), (2, 70001), (1, 65544), (1601, 1000), (3101, 512), (801, 2048), (401, 4096), (25001, 64),
          (12301, 120), (6203, 256)]


@pytest.mark.parametrize("layout", ["dense", "wide", "odd"])
@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward(shape, layer, layout):
    rows, cols = shape
    for i, option in enumerate(OPTIONS):
        dtype = (F32, F16, BF16)[(i + rows + cols) % 3]
        gen = base._gen(rows * 7 + cols + i)
        x, block, params, opts, through = _call(gen, rows, cols, dtype, layout, layer, option)
        what = (option, base.ids(dtype))
        r = L.residual_norm(x, block, params["gamma"], params["beta"], ref.EPS, block_gamma=params["block_gamma"], block_beta=params["block_beta"],
                            gate=params["gate"], **opts)
        want = ref.residual_norm(x, block, params, layer, through)
        assert r.s is x or block is not None
        for name in ("y", "s"):
            assert (getattr(r, name) is not None) == (name in want)
            if name in want and not (name == "s" and block is None):
                ref.check(getattr(r, name), want[name], dtype, (name, *what))
        stats = {}
        for name, there in (("mean", option[1] and layer), ("rstd", option[1]), ("block_mean", option[2] and layer), ("block_rstd", option[2])):
            stats[name] = getattr(r, name)
            assert (stats[name] is not None) == bool(there)
            if there:
                ref.check(stats[name], want[name], F32, (name, *what))
        # backward, with and without the residual path's gradient
        grad = (F32, dtype)[i % 2]
        dy = base._lay(base._randn(gen, rows, cols, dtype=dtype, scale=0.1), layout) if option[1] else None
        for with_ds in ((True, False) if option[1] else (True,)):
            ds = base._lay(base._randn(gen, rows, cols, dtype=dtype, scale=0.1), layout) if with_ds else None
            kept = block if option[2] or option[3] else None
            g = L.residual_norm_backward(dy, ds, r.s, kept, params["gamma"], r.mean, r.rstd, block_gamma=params["block_gamma"],
                                         block_beta=params["block_beta"], block_mean=r.block_mean, block_rstd=r.block_rstd, gate=params["gate"],
                                         has_block=block is not None, grad_dtype=grad, **opts)
            wg = ref.residual_norm_grads(dy, ds, r.s, block, params, stats, layer, through)
            for name, got in g._asdict().items():
                assert (got is not None) == (name in wg), (name, *what)
                if got is not None:
                    ref.check(got, wg[name], dtype if name in ("dx", "dblock") else grad, (name, *what))


@pytest.mark.parametrize("cols", [264, 1155, 9000, 40000])
def test_values_of_all_sizes(cols):
    """Rows a million apart in size, a large mean, zero rows: statistics as good as for ordinary rows."""
    gen = base._gen(cols)
    for layer in (True, False):
        x, block, params, opts, through = _call(gen, 60, cols, F32, "dense", layer, (True, True, True, True, 0.0))
        grow = torch.logspace(-6, 6, 60, device="cuda")[:, None]
        x, block = x * grow, block * grow.flip(0)
        x[5], block[5], block[9] = 0, 0, 0
        x[7] += 1000 * grow[7]
        r = L.residual_norm(x, block, params["gamma"], params["beta"], ref.EPS, block_gamma=params["block_gamma"], block_beta=params["block_beta"],
                            gate=params["gate"], **opts)
        want = ref.residual_norm(x, block, params, layer, through)
        for name in ("y", "s", "rstd", "block_rstd"):
            ref.check(getattr(r, name), want[name], F32, name)


def test_dropped_values_of_any_kind_leave_no_trace():
    """NaN and infinities in dropped places of a block without a norm, and in the gradient there, enter nothing."""
    rows, cols, p = 50, 200, 0.3
    gen, key = base._gen(5), _key()
    gone = ~ref.stays(rows, cols, p, key, 9)
    for width in (cols, cols + 3):
        x, block, dy, ds = (base._randn(gen, rows, width, dtype=BF16)[:, :cols] for _ in range(4))
        gamma, gate = base._randn(gen, cols, shift=1.0), base._randn(gen, cols)
        opts = dict(norm=L.NORM_RMS, gate=gate, p=p, key=key, site=9)
        clean = L.residual_norm(x, torch.where(gone, 0.0, block.float()).to(BF16), gamma, None, **opts)
        for bad in (float("nan"), float("inf"), torch.finfo(BF16).min):
            dirty = torch.where(gone, bad, block.float()).to(BF16)
            r = L.residual_norm(x, dirty, gamma, None, **opts)
            assert torch.equal(r.s, clean.s) and torch.equal(r.y, clean.y) and torch.equal(r.rstd, clean.rstd)
            only = L.residual_norm_backward(None, torch.where(gone, bad, ds.float()).to(BF16), None, None, None, None, None, norm=L.NORM_RMS, p=p, key=key, site=9)
            assert bool(only.dblock.isfinite().all()) and bool((only.dblock[gone] == 0).all())


def test_no_rows():
    x, v = torch.zeros(0, 64, dtype=BF16, device="cuda"), torch.ones(64, device="cuda")
    r = L.residual_norm(x, x, v, v, block_gamma=v, block_beta=v, gate=v, p=0.1, key=_key())
    assert r.y.shape == r.s.shape == (0, 64) and r.rstd.shape == (0,)
    g = L.residual_norm_backward(x, x, r.s, x, v, r.mean, r.rstd, block_gamma=v, block_beta=v, block_mean=r.block_mean, block_rstd=r.block_rstd, gate=v, p=0.1, key=_key())
    assert g.dx.shape == (0, 64) and all(t.shape == (64,) and not t.any() for t in g[2:])


@pytest.mark.parametrize("shape", [(1, 8), (33, 200), (300, 1155), (20, 9000), (3, 66000)], ids=str)
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_both_ways_from_python_agree(both, shape, pad):  # noqa: F811
    for i, (option, layer) in enumerate(itertools.product(OPTIONS, (True, False))):
        gen, dtype = base._gen(i), (F32, F16, BF16)[i % 3]
        lay = lambda: base._randn(gen, shape[0], shape[1] + pad, dtype=dtype)[:, : shape[1]]  # noqa: E731
        x, block, params, opts, _ = _call(gen, *shape, dtype, "dense", layer, option)
        x, dy, ds = lay(), lay() if option[1] else None, lay()
        rest = dict(block_gamma=params["block_gamma"], block_beta=params["block_beta"], gate=params["gate"], **opts)
        r = both(lambda: L.residual_norm(x, block, params["gamma"], params["beta"], **rest))
        both(lambda: L.residual_norm_backward(dy, ds, r.s, block, params["gamma"], r.mean, r.rstd, block_mean=r.block_mean, block_rstd=r.block_rstd,
                                              has_block=option[0], grad_dtype=dtype, **rest))


def test_more_dimensions():
    gen, v = base._gen(6), torch.ones(64, device="cuda")
    x, b, dy = (base._randn(gen, 3, 5, 64, dtype=F16) for _ in range(3))
    opts = dict(norm=L.NORM_RMS, block_gamma=v, gate=v, p=0.2, key=_key())
    r, flat = L.residual_norm(x, b, v, **opts), L.residual_norm(x.reshape(15, 64), b.reshape(15, 64), v, **opts)
    assert r.y.shape == (3, 5, 64) and r.rstd.shape == (3, 5) and torch.equal(r.y.reshape(15, 64), flat.y)
    g = L.residual_norm_backward(dy, None, r.s, b, v, None, r.rstd, block_rstd=r.block_rstd, **opts)
    h = L.residual_norm_backward(dy.reshape(15, 64), None, flat.s, b.reshape(15, 64), v, None, flat.rstd, block_rstd=flat.block_rstd, **opts)
    assert g.dx.shape == (3, 5, 64) and all(torch.equal(p.reshape(q.shape), q) for p, q in zip(g, h) if p is not None)


def test_tensors_that_require_a_gradient():
    gen = base._gen(9)
    x, b, dy = (base._randn(gen, 10, 64, dtype=BF16) for _ in range(3))
    v, gate = base._randn(gen, 64), base._randn(gen, 64)
    r = L.residual_norm(x, b, v, v, gate=gate)
    calls = ((x, lambda: L.residual_norm(x, b, v, v)), (b, lambda: L.residual_norm(x, b, v, v)), (v, lambda: L.residual_norm(x, b, v, v)),
             (gate, lambda: L.residual_norm(x, b, v, v, gate=gate)), (dy, lambda: L.residual_norm_backward(dy, None, r.s, b, v, r.mean, r.rstd, gate=gate)),
             (b, lambda: L.residual_norm_backward(dy, None, r.s, b, v, r.mean, r.rstd, gate=gate)))
    for t, call in calls:
        call()
        t.requires_grad_()
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        with torch.no_grad():
            call()
        t.requires_grad_(False)
