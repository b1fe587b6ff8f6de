"""Layer norm at the edges of its forms (how many threads have a row, how many columns each), with more rows than
are in flight at once, so that every form's sums over rows and the join of its row groups are met.  The checks and
tolerances are those of test_gpu_layers."""
import pytest
import torch

import test_gpu_layers as base

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ids = base.ids

SHAPES = [(5000, 256), (4000, 257), (3500, 512), (3300, 520), (2600, 768), (1700, 776), (2600, 1016), (1400, 1025), (1300, 1280), (1290, 1288),
          (1200, 1536), (1100, 1544), (900, 2048), (700, 2056), (500, 3000), (400, 3080), (500, 4096), (330, 4104), (153, 1024), (152, 1155),
          (305, 130), (310, 8191)]


@pytest.mark.parametrize("layout", ["dense", "odd"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype, layout):
    base.test_layer_norm(shape, dtype, layout)


@pytest.mark.parametrize("kept", ["x", "checkpoint"])
@pytest.mark.parametrize("layout", ["dense", "odd"])
@pytest.mark.parametrize("dtype,grad,add", [(F32, F32, True), (F32, F16, False), (F16, F16, False), (BF16, F32, True)],
                         ids=lambda v: ids(v) if isinstance(v, torch.dtype) else str(v))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, dtype, grad, add, layout, kept):
    base.test_layer_norm_backward(shape, dtype, grad, add, layout, kept)


@pytest.mark.parametrize("rows", [1, 2, 3, 151, 152, 153, 303, 305, 600, 1217])
@pytest.mark.parametrize("cols", [40, 500, 1024, 1155, 4096])
def test_backward_of_few_rows(rows, cols):
    # blocks whose row groups have no row at all, or one
    base.test_layer_norm_backward((rows, cols), BF16, F32, True, "dense", "x")
    base.test_layer_norm_backward((rows, cols), F32, F32, False, "odd", "x")
