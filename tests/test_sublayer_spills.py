"""Register spills of the gated sublayer's kernels, from the summaries that the build leaves beside its objects (-Xptxas -v).  No GPU
needed."""
import os
import re
import shutil
import subprocess

import pytest

# source, kernel, most bytes of spill stores: a form that is not here spills nothing
ALLOWED = [
    ("gated_forward", r"k_product<2, false, false, .*GatedEpilogue<\w+, [34], [01]>", 4),       # silu and the tanh form, pairs, without checkpoints
    ("residual_norm_(bf16|f16)", r"k_rn_forward<\w+, (8|16|32), 1, 1, true, false, false>", 4),  # narrow rows, one at a time: 72 registers
    ("residual_norm_(bf16|f16)", r"k_rn_forward<\w+, (32|64), 1, 1, false, (true|false), false>", 24),  # the same off 16 bytes (80 with a norm behind the block)
    ("residual_norm_f32", r"k_rn_forward<float, (8|16|32|64), 1, 1, false, (true|false), false>", 120),
]
SOURCES = {"gated_forward": 40, "gated_backward": 30, "dropout": 20, "residual_norm_bf16": 100, "residual_norm_f16": 100, "residual_norm_f32": 100}  # kernels at least


@pytest.mark.skipif(shutil.which("c++filt") is None, reason="needs c++filt")
@pytest.mark.parametrize("source", sorted(SOURCES))
def test_no_new_spills(source):
    from communication_compressed_optimizer_compress_gb300 import _build

    try:
        _build.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    _build.build()
    with open(os.path.join(_build.BUILD_DIR, source + ".ptxas")) as f:
        parts = re.split(r"Compiling entry function '", f.read())[1:]
    names = subprocess.run(["c++filt"], input="\n".join(p.split("'")[0] for p in parts), capture_output=True, text=True).stdout.split("\n")
    assert len(parts) >= SOURCES[source]
    for name, part in zip(names, parts):
        stores = int(re.search(r"(\d+) bytes spill stores", part).group(1))
        most = max((n for s, kernel, n in ALLOWED if re.fullmatch(s, source) and re.search(kernel, name)), default=0)
        assert stores <= most, (name, stores)
