"""The gated linear layer, dropout and the residual norm through the C ABI without a GPU: what they refuse, and what they
say about workspaces.  Every call here is refused, or asks for a size, before anything could be enqueued."""
import ctypes
import os
import re
import types

import pytest
import torch

import communication_compressed_optimizer_compress_gb300 as ob
from communication_compressed_optimizer_compress_gb300 import layers as L
from test_layers_device_host import DEVICE, Tensor, machine  # noqa: F401  (a fixture)

P = 1 << 20  # stands for a device pointer: no refused call reads it
BIG = 1 << 40
INV, UNS, WS = ob.ERR_INVALID_ARG, ob.ERR_UNSUPPORTED, ob.ERR_WORKSPACE
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    from communication_compressed_optimizer_compress_gb300 import _build

    _build.build()


def _at(k):
    return P + k * BIG


def _make(kind, base, kw):
    a = kind()
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


def _gated(**kw):
    return _make(L.GatedLinearArgs, dict(x=_at(0), ldx=64, w=_at(1), ldw=64, bias=_at(2), h=_at(3), ldh=32, rows=4, in_=64, inner=32,
                                         dtype=ob.BF16, activation=L.ACT_SILU), kw)


CK = dict(gate_codes=_at(4), gate_scales=_at(5), up_codes=_at(6), up_scales=_at(7))


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(in_=0), INV), (dict(inner=0), INV), (dict(rows=(1 << 31) + 1), UNS), (dict(inner=(1 << 23) + 1, ldh=1 << 24), UNS),
    (dict(in_=(1 << 24) + 1, ldx=1 << 25, ldw=1 << 25), UNS), (dict(dtype=3), INV), (dict(dtype=ob.F32), UNS), (dict(activation=5), INV),
    (dict(activation=-1), INV), (dict(ldx=63), INV), (dict(ldw=63), INV), (dict(ldh=31), INV), (dict(z=_at(4), ldz=63), INV), (dict(x=None), INV),
    (dict(w=None), INV), (dict(h=None), INV), (dict(CK, gate_codes=None), INV), (dict(CK, gate_scales=None), INV), (dict(CK, up_codes=None), INV),
    (dict(CK, up_scales=None), INV), (dict(CK, z=_at(8), ldz=64), INV), (dict(x=P + 1), INV), (dict(bias=P + 2), INV), (dict(CK, up_scales=_at(7) + 2), INV),
    (dict(h=_at(0)), INV), (dict(h=_at(1) + 4096), INV), (dict(z=_at(3) + 64, ldz=64), INV), (dict(CK, up_codes=_at(4) + 16), INV),
    (dict(CK, up_scales=_at(2) + 252), INV), (dict(h=_at(2) + 192), INV), (dict(h=_at(9)), INV),
])
def test_gated_linear_refuses(kw, status):
    f, a, need = L._functions(), _gated(**kw), ctypes.c_size_t()
    if kw.get("h") == _at(9):  # an output inside the workspace, where one is needed at all
        assert f.onebit_gated_linear_forward_workspace(a, need) == ob.OK
        if need.value == 0:
            pytest.skip("no workspace for this call")
    assert f.onebit_gated_linear_forward(a, _at(9), 1 << 38, None) == status
    assert f.onebit_layers_last_error()


def _gated_grad(**kw):
    return _make(L.GatedLinearGradArgs, dict(dy=_at(0), lddy=48, z=_at(1), ldz=64, w=_at(2), ldw=32, dz=_at(3), lddz=64, dw=_at(8), db=_at(10),
                                             rows=4, inner=32, out=48, dtype=ob.F16, activation=L.ACT_GELU, grad_dtype=ob.F32), kw)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(out=0), INV), (dict(inner=0), INV), (dict(dtype=ob.F32), UNS), (dict(grad_dtype=5), INV), (dict(activation=5), INV),
    (dict(inner=(1 << 23) + 1, ldz=1 << 25, ldw=1 << 25, lddz=1 << 25), UNS), (dict(lddy=47), INV), (dict(ldz=63), INV), (dict(ldw=31), INV),
    (dict(lddz=63), INV), (dict(dy=None), INV), (dict(z=None), INV), (dict(w=None), INV), (dict(CK), INV), (dict(CK, z=None, up_scales=None), INV),
    (dict(z=None, dz=None), INV), (dict(dz=_at(0)), INV), (dict(dz=_at(1) + 128), INV), (dict(dw=_at(2)), INV), (dict(db=_at(8) + 16), INV),
    (dict(dw=_at(8) + 2), INV), (dict(dz=_at(3) + 1), INV), (dict(dw=_at(9)), INV), (dict(CK, z=None, dz=_at(6)), INV),
])
def test_gated_linear_backward_refuses(kw, status):
    f, a = L._functions(), _gated_grad(**kw)
    assert f.onebit_gated_linear_backward(a, _at(9), 1 << 38, None) == status
    assert f.onebit_layers_last_error()


def _dropout(**kw):
    d = dict(x=_at(0), ldx=64, dtype=ob.BF16, rows=4, cols=64, p=0.5, key=_at(1), site=0, y=_at(2), ldy=64, stream=None)
    d.update(kw)
    return L._functions().onebit_dropout(*d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(cols=0), INV), (dict(rows=(1 << 31) + 1), UNS), (dict(cols=(1 << 24) + 1, ldx=1 << 25, ldy=1 << 25), UNS),
    (dict(dtype=3), INV), (dict(ldx=63), INV), (dict(ldy=63), INV), (dict(p=-0.1), INV), (dict(p=1.0), INV), (dict(p=NAN), INV), (dict(p=0.999999), INV),
    (dict(p=float("inf")), INV), (dict(key=None), INV), (dict(key=_at(1) + 4), INV), (dict(x=None), INV), (dict(y=None), INV), (dict(x=_at(0) + 1), INV),
    (dict(y=_at(0) + 128), INV), (dict(y=_at(1)), INV), (dict(y=_at(0)), INV),
])
def test_dropout_refuses(kw, status):
    assert _dropout(**kw) == status
    assert L._functions().onebit_layers_last_error()


def _rn(**kw):
    return _make(L.ResidualNormArgs, dict(x=_at(0), ldx=64, block=_at(1), ldblock=64, gamma=_at(2), beta=_at(3), block_gamma=_at(4), block_beta=_at(5),
                                          gate=_at(6), key=_at(7), s=_at(8), lds=64, y=_at(9), ldy=64, mean=_at(10), rstd=_at(11), block_mean=_at(12),
                                          block_rstd=_at(13), rows=4, cols=64, dtype=ob.BF16, norm=L.NORM_LAYER, eps=1e-5, scale=0.5, p=0.1, site=1), kw)


NO_BLOCK = dict(block=None, s=None, block_gamma=None, block_beta=None, block_mean=None, block_rstd=None, gate=None, p=0.0)
NO_NORM = dict(gamma=None, beta=None, y=None, mean=None, rstd=None)
RMS = dict(norm=L.NORM_RMS, beta=None, block_beta=None, mean=None, block_mean=None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(cols=0), INV), (dict(rows=(1 << 31) + 1), UNS), (dict(dtype=4), INV), (dict(norm=2), INV), (dict(eps=-1.0), INV),
    (dict(eps=NAN), INV), (dict(p=1.0), INV), (dict(p=-1.0), INV), (dict(key=None), INV), (dict(key=_at(7) + 4), INV), (dict(ldx=63), INV),
    (dict(ldblock=63), INV), (dict(lds=63), INV), (dict(ldy=63), INV), ({**NO_BLOCK, **NO_NORM}, INV), (dict(NO_BLOCK, gate=_at(6)), INV),
    (dict(NO_BLOCK, p=0.1), INV), (dict(NO_BLOCK, block_gamma=_at(4), block_beta=_at(5), block_mean=_at(12), block_rstd=_at(13)), INV),
    (dict(NO_BLOCK, s=_at(8)), INV), (dict(s=None), INV), (dict(beta=None), INV), (dict(block_beta=None), INV), (dict(RMS, beta=_at(3)), INV),
    (dict(RMS, block_beta=_at(5)), INV), (dict(RMS, mean=_at(10)), INV), (dict(RMS, block_mean=_at(12)), INV), (dict(x=None), INV), (dict(y=None), INV),
    (dict(rstd=None), INV), (dict(mean=None), INV), (dict(block_rstd=None), INV), (dict(block_mean=None), INV), (dict(NO_NORM, y=_at(9)), INV),
    (dict(NO_NORM, rstd=_at(11)), INV), (dict(x=_at(0) + 1), INV), (dict(gamma=_at(2) + 2), INV), (dict(rstd=_at(11) + 2), INV), (dict(s=_at(0)), INV),
    (dict(y=_at(8) + 16), INV), (dict(y=_at(1)), INV), (dict(mean=_at(11)), INV), (dict(s=_at(6)), INV), (dict(block_rstd=_at(7) + 8), INV),
])
def test_residual_norm_refuses(kw, status):
    f = L._functions()
    assert f.onebit_residual_norm_forward(_rn(**kw), None) == status
    assert f.onebit_layers_last_error()
    assert f.onebit_residual_norm_forward(None, None) == INV


def _rnb(**kw):
    return _make(L.ResidualNormGradArgs, dict(dy=_at(0), lddy=64, ds=_at(1), ldds=64, s=_at(2), lds=64, block=_at(3), ldblock=64, gamma=_at(4),
                                              block_gamma=_at(5), block_beta=_at(6), gate=_at(7), key=_at(8), mean=_at(9), rstd=_at(10),
                                              block_mean=_at(11), block_rstd=_at(12), dx=_at(13), lddx=64, dblock=_at(14), lddblock=64, dgamma=_at(15),
                                              dbeta=_at(16), dblock_gamma=_at(17), dblock_beta=_at(18), dgate=_at(19), rows=4, cols=64, dtype=ob.BF16,
                                              norm=L.NORM_LAYER, grad_dtype=ob.F32, scale=0.5, p=0.1, site=1), kw)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(cols=0), INV), (dict(dtype=4), INV), (dict(norm=2), INV), (dict(grad_dtype=3), INV), (dict(p=1.0), INV),
    (dict(key=None), INV), (dict(lddy=63), INV), (dict(ldds=63), INV), (dict(lds=63), INV), (dict(ldblock=63), INV), (dict(lddx=63), INV),
    (dict(lddblock=63), INV), (dict(dgamma=None), INV), (dict(dbeta=None), INV), (dict(dblock_gamma=None), INV), (dict(dblock_beta=None), INV),
    (dict(dgate=None), INV), (dict(gate=None), INV), (dict(gamma=None), INV), (dict(block_gamma=None), INV), (dict(block_beta=None), INV),
    (dict(norm=L.NORM_RMS), INV), (dict(dx=None), INV), (dict(dy=None), INV), (dict(s=None), INV), (dict(block=None), INV), (dict(dblock=None), INV),
    (dict(rstd=None), INV), (dict(mean=None), INV), (dict(block_rstd=None), INV), (dict(block_mean=None), INV), (dict(dy=_at(0) + 1), INV),
    (dict(dgate=_at(19) + 2), INV), (dict(mean=_at(9) + 2), INV), (dict(dx=_at(0)), INV), (dict(dblock=_at(13)), INV), (dict(dgamma=_at(16)), INV),
    (dict(dx=_at(20)), INV), (dict(dgate=_at(8)), INV), (dict(dblock=_at(11)), INV),
    (dict(gamma=None, dgamma=None, dbeta=None, mean=None, rstd=None, dy=None, ds=None), INV),
])
def test_residual_norm_backward_refuses(kw, status):
    f = L._functions()
    assert f.onebit_residual_norm_backward(_rnb(**kw), _at(20), 1 << 38, None) == status
    assert f.onebit_layers_last_error()
    assert f.onebit_residual_norm_backward(None, _at(20), 1 << 38, None) == INV


def test_workspaces():
    f, need = L._functions(), ctypes.c_size_t()
    for a, size, run, align in ((_gated_grad(), f.onebit_gated_linear_backward_workspace, f.onebit_gated_linear_backward, 256),
                                (_rnb(), f.onebit_residual_norm_backward_workspace, f.onebit_residual_norm_backward, 16)):
        assert size(a, need) == ob.OK and need.value > 0
        assert run(a, None, need.value, None) == WS
        assert run(a, _at(20), need.value - 1, None) == WS
        assert run(a, _at(20) + align // 2, need.value, None) == WS
        assert size(a, None) == INV and size(None, need) == INV
    assert f.onebit_gated_linear_forward_workspace(_gated(), need) == ob.OK
    assert f.onebit_gated_linear_forward_workspace(None, need) == INV and f.onebit_gated_linear_forward_workspace(_gated(), None) == INV


def test_no_rows_are_no_work():
    f, need = L._functions(), ctypes.c_size_t()
    assert f.onebit_gated_linear_forward(_gated(rows=0), None, 0, None) == ob.OK
    assert f.onebit_residual_norm_forward(_rn(rows=0), None) == ob.OK
    assert _dropout(rows=0) == ob.OK
    assert f.onebit_gated_linear_backward_workspace(_gated_grad(rows=0), need) == ob.OK and need.value == 0


def test_silu_is_the_gated_layers_alone():
    f = L._functions()
    a = L.LinearArgs(_at(0), 64, _at(1), 64, None, None, 0, _at(2), 32, None, None, 4, 64, 32, ob.BF16, L.ACT_SILU)
    assert f.onebit_linear_forward(a, _at(9), 1 << 38, None) == INV


def test_structures_match_the_header():
    """Every field of the C structures, in order, with its type."""
    src = open(os.path.join(os.path.dirname(ob.__file__), "..", "include", "onebit_layers.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    kinds = {"int64_t": ctypes.c_int64, "int32_t": ctypes.c_int32, "uint32_t": ctypes.c_uint32, "float": ctypes.c_float}
    for name, kind in (("onebit_gated_linear_t", L.GatedLinearArgs), ("onebit_gated_linear_grad_t", L.GatedLinearGradArgs),
                       ("onebit_residual_norm_t", L.ResidualNormArgs), ("onebit_residual_norm_grad_t", L.ResidualNormGradArgs)):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", src).group(1)
        fields = []
        for line in body.split(";"):
            words = line.replace("const ", "").split(None, 1)
            if words:
                for n in words[1].split(","):
                    pointer = "*" in n or "*" in words[0]
                    fields.append((n.strip(" *").replace("in", "in_") if n.strip() == "in" else n.strip(" *"), ctypes.c_void_p if pointer else kinds[words[0]]))
        assert fields == list(kind._fields_), name
    assert L.GATE_ACTIVATIONS == {**L.ACTIVATIONS, "silu": L.ACT_SILU} and f"ONEBIT_ACT_SILU = {L.ACT_SILU}" in src
    assert re.search(r"ONEBIT_NORM_LAYER = 0, ONEBIT_NORM_RMS = 1", src) and L.NORMS == {"layer": 0, "rms": 1}


def _calls():
    x, w, dy, w2 = Tensor(4, 64), Tensor(32, 64), Tensor(4, 32), Tensor(32, 64)
    v, u, key = Tensor(64, dtype=torch.float32), Tensor(4, dtype=torch.float32), Tensor(2, dtype=torch.int64)
    ck = L.Checkpoint(Tensor(4, 64, dtype=torch.int8), Tensor(4, 1, dtype=torch.float32), torch.bfloat16)
    norm = dict(block_gamma=v, block_beta=v, gate=v, p=0.1, key=key)
    return {
        "gated_linear": lambda **k: L.gated_linear(x, w, keep="checkpoint", **k),
        "gated_linear_backward": lambda **k: L.gated_linear_backward(dy, L.Gated(ck, ck), w2, **k),
        "dropout": lambda **k: L.dropout(x, 0.5, key, **k),
        "residual_norm": lambda **k: L.residual_norm(x, x, v, v, **norm, **k),
        "residual_norm_backward": lambda **k: L.residual_norm_backward(x, x, x, x, v, u, u, block_mean=u, block_rstd=u, **norm, **k),
    }


@pytest.fixture
def two_devices(machine, monkeypatch):  # noqa: F811
    entries = L._fn

    class Entries:
        def __getattr__(self, name):
            f = getattr(entries, name)
            if name.startswith("onebit_gated") and not name.endswith("workspace"):
                return lambda *a: f(*a) if a[1] else ob.ERR_WORKSPACE
            return f

    machine.int64 = torch.int64
    L.torch.int64 = torch.int64
    monkeypatch.setattr(L, "_fn", Entries())
    return machine


@pytest.mark.parametrize("name", sorted(_calls()))
def test_the_tensors_device_is_current(two_devices, name):
    _calls()[name]()
    assert len(two_devices.seen) >= 2 and {d for _, d in two_devices.seen} == {1}, two_devices.seen
    assert two_devices.current == 0
    two_devices.fail = True
    with pytest.raises(ob.OneBitError):
        _calls()[name]()
    assert {d for _, d in two_devices.seen} == {1} and two_devices.current == 0


@pytest.mark.parametrize("name", sorted(_calls()))
def test_a_stream_is_one_of_the_tensors_device(two_devices, name):
    here, there = (types.SimpleNamespace(device=torch.device("cuda", i), cuda_stream=7) for i in (1, 0))
    assert here.device == DEVICE
    _calls()[name](stream=here)
    assert {d for _, d in two_devices.seen} == {1} and two_devices.streams == [here] and two_devices.current == 0
    two_devices.seen.clear()
    with pytest.raises(ValueError, match="stream"):
        _calls()[name](stream=there)
    assert not two_devices.seen and two_devices.current == 0


@pytest.mark.parametrize("call", [
    lambda: L.gated_linear(Tensor(4, 64), Tensor(33, 64)), lambda: L.gated_linear(Tensor(4, 64), Tensor(32, 63)),
    lambda: L.gated_linear(Tensor(4, 64), Tensor(32, 64), keep="all"), lambda: L.gated_linear(Tensor(4, 64), Tensor(32, 64, dtype=torch.float16)),
    lambda: L.gated_linear_backward(Tensor(4, 32), Tensor(4, 127), Tensor(32, 64)), lambda: L.gated_linear_backward(Tensor(4, 32), Tensor(5, 128), Tensor(32, 64)),
    lambda: L.gated_linear_backward(Tensor(4, 32), L.Gated(Tensor(4, 64), Tensor(4, 64)), Tensor(32, 64)),
    lambda: L.dropout(Tensor(4, 64), 0.5, None), lambda: L.dropout(Tensor(4, 64), 0.5, Tensor(3, dtype=torch.int64)),
    lambda: L.dropout(Tensor(4, 64), 0.5, Tensor(2, dtype=torch.float32)), lambda: L.dropout(Tensor(4, 64), 0.5, Tensor(2, dtype=torch.int64), site=-1),
    lambda: L.dropout(Tensor(4, 64), 0.5, Tensor(2, dtype=torch.int64), site=1 << 32),
    lambda: L.residual_norm(Tensor(4, 64), Tensor(4, 63)), lambda: L.residual_norm(Tensor(4, 64), gamma=Tensor(63, dtype=torch.float32)),
    lambda: L.residual_norm_backward(None, None, None, None, None, None, None),
], ids=range(15))
def test_python_refuses(two_devices, call):
    with pytest.raises(ValueError):
        call()
    assert not two_devices.seen and two_devices.current == 0
