"""What dropout drops of a block without a norm behind it enters no result, whatever it was, forward or backward."""
import pytest
import torch

import sublayer_ref as ref
import test_gpu_layers as base
from communication_compressed_optimizer_compress_gb300 import layers as L

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


# rows of one block on 16 bytes and off, of several blocks, and rows read again for each step (backward above 32768 columns)
@pytest.mark.parametrize("rows,cols,pad", [(50, 200, 0), (50, 203, 3), (300, 1024, 0), (40, 1155, 1), (30, 5000, 0), (30, 5003, 2), (70, 33000, 0), (5, 66001, 1)], ids=str)
@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
def test_dropped_values_enter_no_gradient(rows, cols, pad, layer):
    dtype = (F32, F16, BF16)[(rows + cols) % 3]
    gen, p = base._gen(rows + cols), 0.3
    key = torch.tensor([2 ** 40 + 3, 9], dtype=torch.int64, device="cuda")
    gone = ~ref.stays(rows, cols, p, key, 9)
    x, block, dy, ds = (base._randn(gen, rows, cols + pad, dtype=dtype)[:, :cols] for _ in range(4))
    gamma, beta, gate = base._randn(gen, cols, shift=1.0), base._randn(gen, cols) if layer else None, base._randn(gen, cols)
    opts = dict(norm=L.NORM_LAYER if layer else L.NORM_RMS, gate=gate, scale=0.5, p=p, key=key, site=9)

    def run(fill, pre):
        b = torch.empty(rows, cols + pad, dtype=dtype, device="cuda")[:, :cols]
        b.copy_(torch.where(gone, fill, block.float()))
        r = L.residual_norm(x, b, gamma if pre else None, beta if pre else None, **opts)
        g = L.residual_norm_backward(dy if pre else None, ds, r.s, b, gamma if pre else None, r.mean, r.rstd, **opts)
        return [t for t in (*r, *g) if t is not None]

    for pre in (True, False):
        clean = run(0.0, pre)
        assert all(bool(t.isfinite().all()) for t in clean)
        for fill in (float("nan"), float("inf"), torch.finfo(dtype).min):
            for a, b in zip(run(fill, pre), clean):
                assert torch.equal(a, b)
