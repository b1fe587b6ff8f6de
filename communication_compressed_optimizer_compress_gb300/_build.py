"""Compile the CUDA library in-tree for sm_103a (nvcc only, no cmake).

build() makes libonebit_adam.so.  build(checked=True) makes libonebit_adam_checked.so, the same
library compiled with -DONEBIT_CHECKS: every kernel of the optimizer's steps checks its units of work
against its buffers before touching them, skips any that fail and reports them through
onebit_adam_get_status() (the layer operators have no such checks and are the same in it).  The
package loads the checked library when the environment variable ONEBIT_LIBRARY is "checked".
"""
from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libonebit_adam.so")
LIB_CHECKED = os.path.join(HERE, "libonebit_adam_checked.so")
BUILD_DIR = os.path.join(HERE, "_build")
BINDING = os.path.join(HERE, "_layers_binding.so")

SOURCES = ["onebit_adam.cu", "onebit_noalloc.cu", "activation_checkpoint.cu", "layer_norm.cu", "tensor_product.cu",
           "linear_forward.cu", "linear_backward.cu"]
HEADERS = ["onebit_kernels.cuh", "layers_common.cuh", "tensor_product.cuh", "linear_common.cuh", "few_rows.cuh",
           os.path.join("..", "..", "include", "onebit_adam.h"),
           os.path.join("..", "..", "include", "onebit_layers.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "--fmad=false",            # no contraction: the fp32 op order must match the method's formulas
    "-prec-div=true", "-prec-sqrt=true",
    "-Xcompiler", "-fPIC,-O2",
    "-I", os.path.join(ROOT, "include"),
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build_binding(force: bool = False) -> str:
    """_layers_binding.so: the layer operators' Python entry points in C++ (host code only, against the
    installed torch)."""
    src = os.path.join(CSRC, "layers_binding.cpp")
    header = os.path.join(ROOT, "include", "onebit_layers.h")
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    # built against another torch than the one at hand: built again
    stamp = os.path.join(BUILD_DIR, "binding_torch")
    version = os.path.join(torch_dir, "version.py")
    made_for = open(stamp).read() if os.path.exists(stamp) else ""
    now = open(version).read() + sys.version
    if not force and not _stale(BINDING, [src, header, __file__]) and made_for == now:
        return BINDING
    os.makedirs(BUILD_DIR, exist_ok=True)
    inc, lib = os.path.join(torch_dir, "include"), os.path.join(torch_dir, "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w", "-D_GLIBCXX_USE_CXX11_ABI=1", "-I", inc,
           "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include"),
           "-I", sysconfig.get_paths()["include"], src, "-o", tmp, "-L", lib, "-ltorch_python", "-ltorch_cuda",
           "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    os.replace(tmp, BINDING)
    with open(stamp, "w") as f:
        f.write(now)
    return BINDING


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    lib = LIB_CHECKED if checked else LIB
    bdir = os.path.join(BUILD_DIR, "checked") if checked else BUILD_DIR
    flags = [*NVCC_FLAGS, "-DONEBIT_CHECKS"] if checked else NVCC_FLAGS
    os.makedirs(bdir, exist_ok=True)
    hdrs = [os.path.normpath(os.path.join(CSRC, h)) for h in HEADERS]
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(bdir, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s, *hdrs, __file__]):
            jobs.append([nvcc(), *flags, "-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        if verbose:
            print(r.stdout + r.stderr)

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        binding = ex.submit(build_binding, force)
        list(ex.map(run, jobs))
        binding.result()
    if force or jobs or _stale(lib, objs):
        tmp = lib + f".tmp{os.getpid()}"
        run([nvcc(), "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-o", tmp, *objs])
        os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force=True, verbose=True))
