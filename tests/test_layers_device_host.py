"""Which device is current while the layer operators allocate and call the C entries, without a GPU: the tensors
are stand-ins on cuda:1 while cuda:0 is current, and the C entries note what they find."""
import contextlib
import types

import pytest
import torch

import communication_compressed_optimizer_compress_gb300 as ob
from communication_compressed_optimizer_compress_gb300 import layers as L

DEVICE = torch.device("cuda", 1)


class Tensor:
    """A contiguous tensor of a second GPU, as far as layers.py looks at it."""

    is_cuda = True
    requires_grad = False
    count = 0

    def __init__(self, *shape, dtype=torch.bfloat16, device=DEVICE):
        self.shape, self.dtype, self.device = shape, dtype, device
        Tensor.count += 1
        self.where = Tensor.count << 40

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def stride(self):
        return self.shape[1], 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.where


@pytest.fixture
def machine(monkeypatch):
    """Two devices, the first current; `seen` is what was met and under which current device."""
    m = types.SimpleNamespace(current=0, seen=[], fail=False, streams=[])

    @contextlib.contextmanager
    def device(d):
        before, m.current = m.current, torch.device(d).index if not isinstance(d, int) else d
        try:
            yield
        finally:
            m.current = before

    @contextlib.contextmanager
    def stream(s):
        with device(s.device):
            m.streams.append(s)
            yield

    def empty(*shape, dtype=None, device=None):
        m.seen.append(("empty", m.current))
        shape = shape[0] if shape and isinstance(shape[0], tuple) else shape
        return Tensor(*shape, dtype=dtype, device=device)

    fake = types.SimpleNamespace(
        empty=empty,
        cuda=types.SimpleNamespace(device=device, stream=stream),
        is_grad_enabled=lambda: False,
        _C=types.SimpleNamespace(_cuda_getCurrentRawStream=lambda index: 1000 + index),
        uint8=torch.uint8, int8=torch.int8, float32=torch.float32, float16=torch.float16, bfloat16=torch.bfloat16)

    class Entries:
        def __getattr__(self, name):
            def entry(*args):
                m.seen.append((name, m.current))
                if name.endswith("workspace"):
                    args[-1].value = 512
                    return ob.OK
                if name.startswith("onebit_linear") and args[1] is None:
                    return ob.ERR_WORKSPACE
                return ob.ERR_CUDA if m.fail else ob.OK

            if name == "onebit_layers_last_error":
                return lambda: b"made to fail"
            return entry

    class Declines:
        def __getattr__(self, name):
            return lambda *a: None

    monkeypatch.setattr(L, "torch", fake)
    monkeypatch.setattr(L, "_fn", Entries())
    monkeypatch.setattr(L, "_layers_binding", Declines())
    return m


def _calls():
    x, w, dy = Tensor(4, 64), Tensor(32, 64), Tensor(4, 32)
    v, u = Tensor(64, dtype=torch.float32), Tensor(4, dtype=torch.float32)
    ck = L.Checkpoint(Tensor(4, 64, dtype=torch.int8), Tensor(4, 1, dtype=torch.float32), torch.bfloat16)
    return {
        "compress": lambda **k: L.compress(x, **k),
        "restore": lambda **k: L.restore(ck, **k),
        "layer_norm": lambda **k: L.layer_norm(x, v, v, checkpoint=True, **k),
        "layer_norm_backward": lambda **k: L.layer_norm_backward(x, ck, v, u, u, **k),
        "linear": lambda **k: L.linear(x, w, checkpoint=True, **k),
        "linear_backward": lambda **k: L.linear_backward(dy, x, w, **k),
    }


@pytest.mark.parametrize("fails", [False, True])
@pytest.mark.parametrize("name", sorted(_calls()))
def test_the_tensors_device_is_current(machine, name, fails):
    machine.fail = fails
    with pytest.raises(ob.OneBitError) if fails else contextlib.nullcontext():
        _calls()[name]()
    assert len(machine.seen) >= 2 and {d for _, d in machine.seen} == {1}, machine.seen
    assert machine.current == 0


@pytest.mark.parametrize("name", sorted(_calls()))
def test_a_stream_is_one_of_the_tensors_device(machine, name):
    here, there = (types.SimpleNamespace(device=torch.device("cuda", i), cuda_stream=7) for i in (1, 0))
    _calls()[name](stream=here)
    assert {d for _, d in machine.seen} == {1} and machine.streams == [here] and machine.current == 0
    machine.seen.clear()
    with pytest.raises(ValueError, match="stream"):
        _calls()[name](stream=there)
    assert not machine.seen and machine.current == 0


def test_the_status_is_that_of_the_streams_device(machine):
    s = types.SimpleNamespace(device=DEVICE, cuda_stream=7)
    assert L.get_status(s) == ob.OK
    L.clear_status(s)
    assert machine.seen == [("onebit_layers_get_status", 1), ("onebit_layers_clear_status", 1)] and machine.current == 0
