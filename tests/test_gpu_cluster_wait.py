"""Residual norms of rows that several blocks share: a block's limited wait for the others' sums runs out, is reported, and
leaves nothing behind."""
import time

import pytest
import torch

import communication_compressed_optimizer_compress_gb300 as ob
import test_gpu_layers as base
from communication_compressed_optimizer_compress_gb300 import layers as L

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _flat(r):
    return [t for t in r if t is not None]


# forward shares rows of more than 8192 columns, backward those of more than 4096; two to eight blocks; rows on 16 bytes and off; both
# numbers of sums
@pytest.mark.parametrize("cols,rows,pad,layer", [(9000, 400, 0, True), (9001, 400, 2, False), (32768, 90, 0, False)], ids=str)
def test_a_sum_that_never_comes_is_reported(cols, rows, pad, layer):
    """Every block has several rows before it.  With sums that wait for bytes no block sends, the first wait runs out after about a second and no
    row behind it waits again: a kernel that waited for each of them would take minutes.  The status says so, and once the hook is off the
    same calls give the same bits."""
    gen = base._gen(cols + layer)
    make = lambda: base._randn(gen, rows, cols + pad, dtype=BF16)[:, :cols]  # noqa: E731
    x, block, dy, ds = make(), make(), make(), make()
    v, w = base._randn(gen, cols, shift=1.0), base._randn(gen, cols) if layer else None
    opts = dict(norm=L.NORM_LAYER if layer else L.NORM_RMS, block_gamma=v, block_beta=w, gate=v, scale=0.5, p=0.2,
                key=torch.tensor([5, 6], device="cuda"), site=1)
    forward = lambda: L.residual_norm(x, block, v, w, **opts)  # noqa: E731
    r = forward()
    backward = lambda: L.residual_norm_backward(dy, ds, r.s, block, v, r.mean, r.rstd, block_mean=r.block_mean, block_rstd=r.block_rstd, **opts)  # noqa: E731
    calls = [forward, backward]
    want = [_flat(c()) for c in calls]
    assert L.get_status() == ob.OK
    for call in calls:
        L.set_fault_injection(ob.FAULT_STALL_COPIES, 16)
        try:
            began = time.monotonic()
            call()
            assert L.get_status() == ob.ERR_CUDA
            assert time.monotonic() - began < 20
        finally:
            L.set_fault_injection(ob.FAULT_NONE)
            L.clear_status()
        assert L.get_status() == ob.OK
        for c, t in zip(calls, want):
            assert all(torch.equal(a, b) for a, b in zip(_flat(c()), t))
    assert L.get_status() == ob.OK


def test_rows_of_one_block_wait_for_nothing():
    gen = base._gen(3)
    x, v = base._randn(gen, 300, 4096, dtype=F16), base._randn(gen, 4096, shift=1.0)
    want = L.residual_norm(x, x, v, None, norm=L.NORM_RMS, block_gamma=v)
    L.set_fault_injection(ob.FAULT_STALL_COPIES, 16)
    try:
        got = L.residual_norm(x, x, v, None, norm=L.NORM_RMS, block_gamma=v)
        assert L.get_status() == ob.OK
    finally:
        L.set_fault_injection(ob.FAULT_NONE)
    assert all(torch.equal(a, b) for a, b in zip(_flat(got), _flat(want)))
