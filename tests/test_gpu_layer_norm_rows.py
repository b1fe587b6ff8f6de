"""Layer norm and checkpoints: the widest and narrowest rows of each form that serves a range of widths, and every row
of matrices with more than 2^31 elements.  Checks and tolerances are those of test_gpu_layers."""
import pytest
import torch

import test_gpu_layers as base

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("layout", ["dense", "wide", "odd"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=base.ids)
@pytest.mark.parametrize("shape", [(1, 264), (7000, 264), (6001, 400), (5000, 512), (3, 512), (800, 4104), (700, 6000), (650, 8192), (1, 8192),
                                   (330, 8200), (160, 16384), (40, 16392)], ids=str)
def test_forward(shape, dtype, layout):
    base.test_layer_norm(shape, dtype, layout)
