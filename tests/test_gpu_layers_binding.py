"""The layer operators' two ways from Python give the same results bit for bit: the compiled binding, which
takes the common case, and layers.py's own path, which takes what the binding leaves to it."""
import pytest
import torch

from communication_compressed_optimizer_compress_gb300 import layers as L

pytestmark = pytest.mark.gpu

NAMES = ("compress", "restore", "layer_norm", "layer_norm_backward", "linear", "linear_backward")


class _Declines:
    """A binding that leaves everything to layers.py."""

    def __getattr__(self, name):
        return lambda *a: None


class _Insists:
    """The binding, which must not leave anything to layers.py."""

    def __init__(self, binding):
        self.binding = binding

    def __getattr__(self, name):
        f = getattr(self.binding, name)

        def call(*a):
            r = f(*a)
            assert r is not None, name
            return r

        return call


def _flat(v):
    if torch.is_tensor(v):
        return [v]
    if isinstance(v, (tuple, list)):
        return [t for x in v for t in _flat(x)]
    return [v]


@pytest.fixture
def both(monkeypatch):
    L._functions()
    binding = L._layers_binding

    def run(f):
        monkeypatch.setattr(L, "_layers_binding", _Insists(binding))
        a = f()
        monkeypatch.setattr(L, "_layers_binding", _Declines())
        b = f()
        monkeypatch.setattr(L, "_layers_binding", binding)
        assert type(a) is type(b)
        fa, fb = _flat(a), _flat(b)
        assert len(fa) == len(fb)
        for x, y in zip(fa, fb):
            if torch.is_tensor(x):
                assert x.dtype == y.dtype and x.shape == y.shape and x.stride() == y.stride() and torch.equal(x, y)
            else:
                assert x == y or x is y
        return a

    return run


@pytest.mark.parametrize("pad", [0, 5])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_binding_agrees(both, dtype, pad):
    g = torch.Generator("cuda")
    g.manual_seed(3)

    def r(rows, cols):
        return torch.randn(rows, cols + pad, generator=g, device="cuda").to(dtype)[:, :cols]

    x, w, res, dy = r(70, 264), r(136, 264), r(70, 136), r(70, 136)
    bias, gamma = torch.randn(136, generator=g, device="cuda"), torch.randn(264, generator=g, device="cuda")
    y, ck = both(lambda: L.linear(x, w, bias, L.ACT_GELU, res, checkpoint=True))
    assert isinstance(ck, L.Checkpoint) and ck.dtype == dtype
    both(lambda: L.linear(x, w))
    both(lambda: L.restore(ck, L.ACT_RELU))
    kept = both(lambda: L.compress(x))
    for add in (None, x):
        both(lambda: L.linear_backward(dy, kept, w, L.ACT_GELU, add=add))
        both(lambda: L.linear_backward(dy, x, w, L.ACT_NONE, add=add, grad_dtype=torch.float32))
    for need in (("dx",), ("dw",), ("db",), ("dx", "db")):
        both(lambda: L.linear_backward(dy, x, w, need=need))
    dw, db = torch.empty(136 * 264, dtype=dtype, device="cuda"), torch.empty(136, dtype=dtype, device="cuda")
    out = both(lambda: L.linear_backward(dy, x, w, dw=dw, db=db))
    assert out[1] is dw and out[2] is db
    n = both(lambda: L.layer_norm(x, gamma, gamma, 1e-5))
    both(lambda: L.layer_norm(x, gamma, gamma, 1e-5, checkpoint=True))
    for src in (x, kept):
        for add in (None, x):
            both(lambda: L.layer_norm_backward(x, src, gamma, n[1], n[2], add=add))
    both(lambda: L.layer_norm_backward(x, x, gamma, n[1], n[2], grad_dtype=dtype))


def test_binding_leaves_the_rest_alone():
    """What it does not take it answers with None, and says nothing."""
    L._functions()
    b, x = L._layers_binding, torch.zeros(4, 8, device="cuda")
    v = torch.zeros(8, device="cuda")
    assert b.compress(x.cpu()) is None and b.compress(x.t()) is None and b.compress(x[None]) is None
    assert b.compress(x.double()) is None and b.compress(None) is None and b.compress(x[:0]) is None
    assert b.restore(x, 0) is None and b.restore(L.compress(x), 99) is None and b.restore(L.compress(x), 2 ** 80) is None
    assert b.layer_norm(x, v, v[:4], 1e-5, False) is None and b.layer_norm(x, v, v, 1, False) is None
    assert b.layer_norm(x, v, v, -1.0, False) is None
    assert b.linear(x, x, None, 0, None, False) is None  # f32
    h = x.half()
    assert b.linear(h, h, v, 0, None, False) is None and b.linear(h, h.bfloat16(), None, 0, None, False) is None
    assert b.linear_backward(h[:, :4], h, h, 0, None, None, None, None, ["dx"]) is None
    with pytest.raises(TypeError):
        b.compress()
