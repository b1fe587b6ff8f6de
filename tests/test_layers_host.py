"""The layer operators' C ABI without a GPU: what it refuses, and what it says about workspaces.  Every
call here is refused, or asks for a size, before anything could be enqueued."""
import ctypes

import pytest

import communication_compressed_optimizer_compress_gb300 as ob
from communication_compressed_optimizer_compress_gb300 import layers as L

P = 1 << 20  # stands for a device pointer: no refused call reads it
BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def built():
    from communication_compressed_optimizer_compress_gb300 import _build

    _build.build()


def _at(k):
    return P + k * BIG


def _forward(**kw):
    base = dict(x=_at(0), ldx=64, w=_at(1), ldw=64, bias=_at(2), residual=None, ldr=0, y=_at(3), ldy=32, codes=None, scales=None,
                rows=4, in_=64, out=32, dtype=ob.BF16, activation=L.ACT_GELU)
    base.update(kw)
    a = L.LinearArgs()
    for k, v in base.items():
        setattr(a, k, v)
    return a


def _backward(**kw):
    base = dict(dy=_at(0), lddy=32, x=_at(1), ldx=64, codes=None, scales=None, w=_at(2), ldw=64, add=None, ldadd=0, dx=_at(3),
                lddx=64, dw=_at(4), db=_at(5), rows=4, in_=64, out=32, dtype=ob.BF16, activation=L.ACT_GELU, grad_dtype=ob.F32)
    base.update(kw)
    a = L.LinearGradArgs()
    for k, v in base.items():
        setattr(a, k, v)
    return a


INV, UNS, WS = ob.ERR_INVALID_ARG, ob.ERR_UNSUPPORTED, ob.ERR_WORKSPACE


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(in_=0), INV), (dict(out=0), INV), (dict(rows=(1 << 31) + 1), UNS), (dict(in_=(1 << 24) + 1, ldx=1 << 25, ldw=1 << 25), UNS),
    (dict(dtype=3), INV), (dict(dtype=ob.F32), UNS), (dict(activation=4), INV), (dict(activation=-1), INV), (dict(ldx=63), INV),
    (dict(ldw=63), INV), (dict(ldy=31), INV), (dict(residual=_at(4), ldr=31), INV), (dict(x=None), INV), (dict(w=None), INV),
    (dict(y=None), INV), (dict(codes=_at(4)), INV), (dict(scales=_at(4)), INV), (dict(x=P + 1), INV), (dict(bias=P + 2), INV),
    (dict(y=_at(0)), INV), (dict(y=_at(1) + 2), INV), (dict(codes=_at(3), scales=_at(4)), INV), (dict(codes=_at(4), scales=_at(2)), INV),
    (dict(residual=_at(3) + 8, ldr=32), INV),
])
def test_linear_forward_refuses(kw, status):
    f, a, need = L._functions(), _forward(**kw), ctypes.c_size_t()
    assert f.onebit_linear_forward(a, _at(9), 1 << 38, None) == status
    assert f.onebit_layers_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(in_=0), INV), (dict(dtype=ob.F32), UNS), (dict(grad_dtype=5), INV), (dict(activation=4), INV),
    (dict(lddy=31), INV), (dict(ldx=63), INV), (dict(ldw=63), INV), (dict(lddx=63), INV), (dict(add=_at(6), ldadd=3), INV),
    (dict(dy=None), INV), (dict(x=None), INV), (dict(w=None), INV), (dict(codes=_at(6), scales=_at(7)), INV), (dict(codes=_at(6)), INV),
    (dict(x=None, codes=_at(6)), INV), (dict(dx=_at(0)), INV), (dict(dw=_at(2)), INV), (dict(db=_at(4) + 16), INV),
    (dict(dw=_at(4) + 2), INV), (dict(x=None, dw=None), INV), (dict(dx=_at(9)), INV),
])
def test_linear_backward_refuses(kw, status):
    f, a = L._functions(), _backward(**kw)
    need = ctypes.c_size_t()
    if kw.get("dx") == _at(9):  # an output inside the workspace, where one is needed at all
        assert f.onebit_linear_backward_workspace(a, need) == ob.OK
        if need.value == 0:
            pytest.skip("no workspace for this call")
    assert f.onebit_linear_backward(a, _at(9), 1 << 38, None) == status
    assert f.onebit_layers_last_error()


def test_workspaces():
    f, need = L._functions(), ctypes.c_size_t()
    a = _backward()
    assert f.onebit_linear_backward_workspace(a, need) == ob.OK and need.value > 0
    assert f.onebit_linear_backward(a, None, need.value, None) == WS
    assert f.onebit_linear_backward(a, _at(9), need.value - 1, None) == WS
    assert f.onebit_linear_backward(a, _at(9) + 8, need.value, None) == WS
    assert f.onebit_linear_backward_workspace(a, None) == INV
    assert f.onebit_linear_backward_workspace(None, need) == INV
    assert f.onebit_linear_forward_workspace(None, need) == INV
    assert f.onebit_linear_forward_workspace(_forward(), need) == ob.OK
    assert f.onebit_layer_norm_backward_workspace(1000, 1024, need) == ob.OK and need.value > 0
    assert f.onebit_layer_norm_backward_workspace(-1, 1024, need) == INV
    assert f.onebit_layer_norm_backward_workspace(10, 0, need) == INV
    assert f.onebit_layer_norm_backward_workspace(10, 10, None) == INV


def _ln(**kw):
    d = dict(x=_at(0), ldx=64, dtype=ob.BF16, rows=4, cols=64, gamma=_at(1), beta=_at(2), eps=1e-5, y=_at(3), ldy=64, mean=_at(4),
             rstd=_at(5), codes=None, scales=None, stream=None)
    d.update(kw)
    return L._functions().onebit_layer_norm_forward(*d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(cols=0), INV), (dict(dtype=7), INV), (dict(ldx=63), INV), (dict(ldy=63), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(x=None), INV), (dict(gamma=None), INV), (dict(mean=None), INV), (dict(codes=_at(6)), INV),
    (dict(y=_at(0) + 64), INV), (dict(rstd=_at(4)), INV), (dict(rows=(1 << 31) + 1), UNS), (dict(mean=_at(4) + 2), INV), (dict(x=_at(0) + 1), INV),
])
def test_layer_norm_refuses(kw, status):
    assert _ln(**kw) == status
    assert L._functions().onebit_layers_last_error()


def _lnb(**kw):
    d = dict(dy=_at(0), lddy=64, x=_at(1), ldx=64, codes=None, scales=None, dtype=ob.BF16, rows=4, cols=64, gamma=_at(2), mean=_at(3),
             rstd=_at(4), add=None, ldadd=0, dx=_at(5), lddx=64, dgamma=_at(6), dbeta=_at(7), grad=ob.F32, ws=_at(9), bytes=1 << 30, stream=None)
    d.update(kw)
    return L._functions().onebit_layer_norm_backward(*d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(dtype=7), INV), (dict(grad=7), INV), (dict(lddy=63), INV), (dict(lddx=63), INV), (dict(ldx=63), INV),
    (dict(add=_at(8), ldadd=1), INV), (dict(dy=None), INV), (dict(x=None), INV), (dict(codes=_at(8), scales=_at(8) + 4096), INV),
    (dict(x=None, codes=_at(8)), INV), (dict(dgamma=None), INV), (dict(dx=_at(0)), INV), (dict(dgamma=_at(7) + 4), INV),
    (dict(ws=None), WS), (dict(bytes=1), WS), (dict(ws=_at(9) + 4), WS), (dict(dgamma=_at(6) + 2), INV),
])
def test_layer_norm_backward_refuses(kw, status):
    assert _lnb(**kw) == status
    assert L._functions().onebit_layers_last_error()


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(cols=0), dict(dtype=9), dict(x=None), dict(codes=None), dict(scales=None), dict(ldx=3),
                                dict(codes=_at(0)), dict(scales=_at(2) + 2), dict(x=_at(0) + 1)])
def test_checkpoint_refuses(kw):
    d = dict(x=_at(0), ldx=64, dtype=ob.F16, rows=4, cols=64, codes=_at(1), scales=_at(2))
    d.update(kw)
    f = L._functions()
    assert f.onebit_checkpoint_compress(d["x"], d["ldx"], d["dtype"], d["rows"], d["cols"], d["codes"], d["scales"], None) == INV
    assert f.onebit_checkpoint_restore(d["codes"], d["scales"], d["rows"], d["cols"], 0, d["x"], d["ldx"], d["dtype"], None) == INV
    assert f.onebit_layers_last_error()


def test_checkpoint_outputs_are_disjoint():
    f = L._functions()
    assert f.onebit_checkpoint_compress(_at(0), 64, ob.F16, 4, 64, _at(1), _at(1) + 8, None) == INV
    assert f.onebit_checkpoint_restore(_at(1), _at(2), 4, 64, 4, _at(0), 64, ob.F16, None) == INV  # no such activation


def test_constants_match_the_header():
    import os
    import re

    src = open(os.path.join(os.path.dirname(ob.__file__), "..", "include", "onebit_layers.h")).read()
    for name, value in L.ACTIVATIONS.items():
        assert re.search(rf"ONEBIT_ACT_{name.upper()} = {value}\b", src)
    assert f"#define ONEBIT_CHECKPOINT_BLOCK {L.CHECKPOINT_BLOCK}" in src
