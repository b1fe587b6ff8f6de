"""The gated layer's forward workspace through the C ABI without a GPU, in a call that needs one: rows off 16 bytes are realigned
there.  Every call here is refused before anything could be enqueued."""
import ctypes

import pytest

import communication_compressed_optimizer_compress_gb300 as ob
from communication_compressed_optimizer_compress_gb300 import layers as L
from test_sublayer_host import CK, INV, WS, _at, _gated, built  # noqa: F401  (a fixture)

# few rows off 16 bytes, more rows, a bias off 16 bytes (whether a contraction is cut, for partial sums, depends on the device's SMs, of which
# there are none here)
CALLS = [dict(in_=65, ldx=65, ldw=65), dict(rows=100, ldx=65), dict(rows=100, in_=64, ldw=67, **CK), dict(rows=100, bias=_at(2) + 4)]


def _need(a):
    need = ctypes.c_size_t()
    assert L._functions().onebit_gated_linear_forward_workspace(a, need) == ob.OK
    assert need.value > 0
    return need.value


@pytest.mark.parametrize("kw", CALLS, ids=range(len(CALLS)))
def test_a_workspace_that_does_not_do(kw):
    f, a = L._functions(), _gated(**kw)
    need = _need(a)
    for at, size in ((None, need), (_at(9), need - 1), (_at(9), 0), (_at(9) + 128, need), (_at(9) + 16, need)):
        assert f.onebit_gated_linear_forward(a, at, size, None) == WS
        assert f.onebit_layers_last_error()


@pytest.mark.parametrize("name", ["h", "z", "gate_codes", "gate_scales", "up_codes", "up_scales", "x", "w", "bias"])
def test_a_buffer_inside_the_workspace(name):
    """Outputs, and inputs too: the workspace is written."""
    kept = dict(z=_at(8), ldz=64) if name == "z" else CK
    a = _gated(**{**dict(in_=65, ldx=65, ldw=65, rows=100), **kept, name: _at(9) + 64})
    assert L._functions().onebit_gated_linear_forward(a, _at(9), _need(a), None) == INV
    assert L._functions().onebit_layers_last_error()


def test_few_aligned_rows_need_none():
    need = ctypes.c_size_t(7)
    assert L._functions().onebit_gated_linear_forward_workspace(_gated(), need) == ob.OK and need.value == 0
