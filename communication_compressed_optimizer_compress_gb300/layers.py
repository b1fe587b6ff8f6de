"""Layer operators that produce the gradients the optimizer exchanges: layer norm, the linear layer with
a fused epilogue, and activation checkpoints held in 8 bits, forward and backward.

Thin Python binding over the C ABI in ``include/onebit_layers.h`` (the formulas are stated there); every
operator runs in the library's CUDA kernels on the current torch stream, or on ``stream``.  The common case
of each (2-D tensors that need no further look) is called through ``_layers_binding`` (C++), everything else,
and every complaint, comes from here.

Matrices are CUDA tensors whose last dimension is the features and has unit stride.  A 2-D tensor may
have any row stride (a column slice of a wider buffer); one of more dimensions must be contiguous and
counts as its leading dimensions' rows.  Nothing is recorded for autograd: the backward pass is the
operators' own, and with gradient mode on a tensor that requires a gradient is refused.  Gradients come in ``grad_dtype``, the type ``OneBitAdam`` was
configured with, and may be written into the caller's tensors (``dw=``, ``db=``).

    y = W2 gelu(W1 x + b1) + b2 + x, then layer norm, with 8-bit checkpoints:

    h, z8 = layers.linear(x, w1, b1, layers.ACT_GELU, checkpoint=True)
    s = layers.linear(h, w2, b2, residual=x)
    y, mean, rstd, s8 = layers.layer_norm(s, gamma, beta, 1e-12, checkpoint=True)
    ds, dgamma, dbeta = layers.layer_norm_backward(dy, s8, gamma, mean, rstd)
    dz, dw2, db2 = layers.linear_backward(ds, z8, w2, layers.ACT_GELU)
    dx, dw1, db1 = layers.linear_backward(dz, x, w1, add=ds)
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import os
from typing import NamedTuple

import torch

from . import BF16, ERR_WORKSPACE, F16, F32, OK, OneBitError, _stream_ptr, lib

ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH = range(4)
ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH}
CHECKPOINT_BLOCK = 64  # columns of a row that share one scale

_DTYPE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}


class Checkpoint(NamedTuple):
    """A matrix in 8 bits: int8 ``codes`` of its shape, fp32 ``scales`` with one value per 64 columns of
    a row, and the ``dtype`` of the matrix it stands for."""

    codes: torch.Tensor
    scales: torch.Tensor
    dtype: torch.dtype


class LinearArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("w", ctypes.c_void_p), ("ldw", ctypes.c_int64),
                ("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64), ("in_", ctypes.c_int64),
                ("out", ctypes.c_int64), ("dtype", ctypes.c_int32), ("activation", ctypes.c_int32)]


class LinearGradArgs(ctypes.Structure):
    _fields_ = [("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("ldw", ctypes.c_int64), ("add", ctypes.c_void_p), ("ldadd", ctypes.c_int64),
                ("dx", ctypes.c_void_p), ("lddx", ctypes.c_int64), ("dw", ctypes.c_void_p), ("db", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("in_", ctypes.c_int64), ("out", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("activation", ctypes.c_int32), ("grad_dtype", ctypes.c_int32)]


_fn = None
_layers_binding = None


def _load_binding():
    """The compiled binding.  Raises if it has not been built."""
    global _layers_binding
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_layers_binding.so")
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
    spec = importlib.util.spec_from_file_location("_layers_binding", path)
    _layers_binding = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(_layers_binding)


def _functions():
    """The C entries, with their argument types set on first use."""
    global _fn
    if _fn is None:
        L = lib()
        _load_binding()
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        sig = {
            "onebit_checkpoint_compress": [vp, i64, i32, i64, i64, vp, vp, vp],
            "onebit_checkpoint_restore": [vp, vp, i64, i64, i32, vp, i64, i32, vp],
            "onebit_layer_norm_forward": [vp, i64, i32, i64, i64, vp, vp, ctypes.c_float, vp, i64, vp, vp, vp, vp, vp],
            "onebit_layer_norm_backward_workspace": [i64, i64, ctypes.POINTER(sz)],
            "onebit_layer_norm_backward": [vp, i64, vp, i64, vp, vp, i32, i64, i64, vp, vp, vp, vp, i64, vp, i64, vp, vp,
                                           i32, vp, sz, vp],
            "onebit_linear_forward_workspace": [ctypes.POINTER(LinearArgs), ctypes.POINTER(sz)],
            "onebit_linear_forward": [ctypes.POINTER(LinearArgs), vp, sz, vp],
            "onebit_linear_backward_workspace": [ctypes.POINTER(LinearGradArgs), ctypes.POINTER(sz)],
            "onebit_linear_backward": [ctypes.POINTER(LinearGradArgs), vp, sz, vp],
            "onebit_layers_get_status": [vp],
            "onebit_layers_clear_status": [vp],
            "onebit_layers_set_fault_injection": [i32, i64],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.onebit_layers_last_error.argtypes = []
        L.onebit_layers_last_error.restype = ctypes.c_char_p
        names = ("onebit_checkpoint_compress", "onebit_checkpoint_restore", "onebit_layer_norm_forward",
                 "onebit_layer_norm_backward_workspace", "onebit_layer_norm_backward", "onebit_linear_forward_workspace",
                 "onebit_linear_forward", "onebit_linear_backward_workspace", "onebit_linear_backward")
        _layers_binding.setup(tuple(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in names), Checkpoint)
        _fn = L
    return _fn


def _check(status: int, where: str):
    if status != OK:
        raise OneBitError(status, where, _functions().onebit_layers_last_error().decode())


def _code(dtype, what: str) -> int:
    try:
        return _DTYPE[dtype]
    except KeyError:
        raise ValueError(f"{what}: dtype {dtype} is not float32, float16 or bfloat16") from None


def _no_history(t, name: str):
    """The operators record nothing for autograd: with gradient mode on, an input that requires a gradient would be
    detached without a word, so it is refused."""
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name}: requires a gradient, which these operators do not record: call under torch.no_grad(), or detach it")


def _matrix(t, name: str, cols=None, rows=None, dtype=None, device=None):
    """(rows, columns, row stride) of a tensor whose last dimension is the features."""
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    _no_history(t, name)
    shape = t.shape
    if len(shape) == 2:
        r, c = shape
        ld, unit = t.stride()
        if (unit != 1 and c > 1) or (ld < c and r > 1):
            raise ValueError(f"{name}: the last dimension needs unit stride and rows that do not overlap")
        if r <= 1 or ld < c:
            ld = c
    else:
        if not shape or not t.is_contiguous():
            raise ValueError(f"{name}: a tensor that is not 2-D must be contiguous, of at least one dimension")
        c = ld = shape[-1]
        r = t.numel() // c if c else 0
    if c < 1:
        raise ValueError(f"{name}: no columns")
    if (cols is not None and c != cols) or (rows is not None and r != rows):
        raise ValueError(f"{name}: expected {rows if rows is not None else r} x {cols if cols is not None else c}, got {r} x {c}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: expected a tensor on {device}, got {t.device}")
    return r, c, ld


def _vector(t, name: str, n: int, device, dtype=torch.float32):
    """Pointer of a contiguous vector of n values (None: none)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name}: expected {n} contiguous {dtype} values on {device}")
    _no_history(t, name)
    return t.data_ptr()


def _kept(x, name: str, cols=None, rows=None, dtype=None, device=None):
    """(x pointer, row stride, codes pointer, scales pointer, rows, columns, dtype, device) of a
    layer's kept input: a tensor or its Checkpoint."""
    if not isinstance(x, Checkpoint):
        r, c, ld = _matrix(x, name, cols, rows, dtype, device)
        return x.data_ptr(), ld, None, None, r, c, x.dtype, x.device
    if dtype is not None and x.dtype != dtype:
        raise ValueError(f"{name}: expected a checkpoint of {dtype}, got one of {x.dtype}")
    codes = x.codes
    r, c, ld = _matrix(codes, name + ".codes", cols, rows, torch.int8, device)
    if r > 1 and ld != c:
        raise ValueError(f"{name}.codes: a checkpoint is contiguous")
    blocks = -(-c // CHECKPOINT_BLOCK)
    s = _vector(x.scales, name + ".scales", r * blocks, codes.device)
    return None, 0, codes.data_ptr(), s, r, c, x.dtype, codes.device


def _stream(device) -> int:
    """The handle of the device's current stream (without making a Stream object, most of a small call)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


# Outputs, always of rows without gaps.  An allocation is most of what a small call costs the host, and one from plain
# integers costs half of one from a shape, so the 2-D case is written out.
def _like(t, dtype=None):
    return torch.empty(t.shape, dtype=dtype or t.dtype, device=t.device)


def _rows_of(t, rows, device):
    """One fp32 value per row of t."""
    return torch.empty(rows if t.dim() == 2 else t.shape[:-1], device=device, dtype=torch.float32)


def _rows_by(t, rows, cols, dtype, device):
    """t's rows with `cols` columns."""
    if t.dim() == 2:
        return torch.empty(rows, cols, dtype=dtype, device=device)
    return torch.empty((*t.shape[:-1], cols), dtype=dtype, device=device)


def _new_checkpoint(t, rows, cols, dtype, device):
    return Checkpoint(_rows_by(t, rows, cols, torch.int8, device),
                      _rows_by(t, rows, -(-cols // CHECKPOINT_BLOCK), torch.float32, device), dtype)


def _workspace(nbytes: int, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


# The C entries launch on the current device, so the tensors' (or the stream's) is made current around each call;
# the binding does the same.
def _device_of(stream):
    return contextlib.nullcontext() if stream is None else torch.cuda.device(stream.device)


def _on(stream, t):
    """The context in which an operator that was given `stream` calls itself."""
    if t.device != stream.device:
        raise ValueError(f"stream: expected one of {t.device}, got one of {stream.device}")
    return torch.cuda.stream(stream)


def get_status(stream=None) -> int:
    """Waits for the stream; OK, or ERR_CUDA when a product of its device gave up waiting for its copies."""
    with _device_of(stream):
        return int(_functions().onebit_layers_get_status(_stream_ptr(stream)))


def clear_status(stream=None):
    with _device_of(stream):
        _check(_functions().onebit_layers_clear_status(_stream_ptr(stream)), "onebit_layers_clear_status")


def set_fault_injection(kind: int, value: int = 0):
    """Test hook of the whole process: FAULT_STALL_COPIES makes the following products' waits run out."""
    _check(_functions().onebit_layers_set_fault_injection(int(kind), int(value)), "onebit_layers_set_fault_injection")


# Every operator works on the current stream: with `stream` it calls itself with that one current, so that its
# outputs and workspace belong to the stream that writes them.


def compress(x, stream=None) -> Checkpoint:
    """The 8-bit checkpoint of x."""
    if stream is not None:
        with _on(stream, x):
            return compress(x)
    if _fn is None:
        _functions()
    fast = _layers_binding.compress(x)
    if fast is not None:
        return fast
    rows, cols, ld = _matrix(x, "x")
    code, device = _code(x.dtype, "x"), x.device
    with torch.cuda.device(device):
        ck = _new_checkpoint(x, rows, cols, x.dtype, device)
        st = _functions().onebit_checkpoint_compress(x.data_ptr(), ld, code, rows, cols, ck[0].data_ptr(), ck[1].data_ptr(),
                                                     _stream(device))
    if st:
        _check(st, "onebit_checkpoint_compress")
    return ck


def restore(ck: Checkpoint, activation=ACT_NONE, stream=None):
    """activation(the values a checkpoint stands for), in the checkpoint's dtype."""
    if stream is not None:
        with _on(stream, ck[0]):
            return restore(ck, activation)
    if _fn is None:
        _functions()
    fast = _layers_binding.restore(ck, activation)
    if fast is not None:
        return fast
    _, _, codes, scales, rows, cols, dtype, device = _kept(ck, "ck")
    with torch.cuda.device(device):
        x = _like(ck[0], dtype)
        st = _functions().onebit_checkpoint_restore(codes, scales, rows, cols, activation, x.data_ptr(), cols, _code(dtype, "ck"),
                                                    _stream(device))
    if st:
        _check(st, "onebit_checkpoint_restore")
    return x


def layer_norm(x, gamma, beta, eps=1e-5, checkpoint=False, stream=None):
    """(y, mean, rstd), and the 8-bit checkpoint of x where asked for."""
    if stream is not None:
        with _on(stream, x):
            return layer_norm(x, gamma, beta, eps, checkpoint)
    if _fn is None:
        _functions()
    fast = _layers_binding.layer_norm(x, gamma, beta, eps, checkpoint)
    if fast is not None:
        return fast
    rows, cols, ld = _matrix(x, "x")
    code, device = _code(x.dtype, "x"), x.device
    g, b = _vector(gamma, "gamma", cols, device), _vector(beta, "beta", cols, device)
    with torch.cuda.device(device):
        y = _like(x)
        mean, rstd = _rows_of(x, rows, device), _rows_of(x, rows, device)
        ck = _new_checkpoint(x, rows, cols, x.dtype, device) if checkpoint else None
        st = _functions().onebit_layer_norm_forward(
            x.data_ptr(), ld, code, rows, cols, g, b, eps, y.data_ptr(), cols, mean.data_ptr(), rstd.data_ptr(),
            ck[0].data_ptr() if checkpoint else None, ck[1].data_ptr() if checkpoint else None, _stream(device))
    if st:
        _check(st, "onebit_layer_norm_forward")
    return (y, mean, rstd, ck) if checkpoint else (y, mean, rstd)


def layer_norm_backward(dy, x, gamma, mean, rstd, add=None, grad_dtype=torch.float32, stream=None):
    """(dx, dgamma, dbeta) from the layer's input x, a tensor or its Checkpoint; ``add`` joins dx."""
    if stream is not None:
        with _on(stream, dy):
            return layer_norm_backward(dy, x, gamma, mean, rstd, add, grad_dtype)
    if _fn is None:
        _functions()
    fast = _layers_binding.layer_norm_backward(dy, x, gamma, mean, rstd, add, grad_dtype)
    if fast is not None:
        return fast
    rows, cols, lddy = _matrix(dy, "dy")
    dtype, device = dy.dtype, dy.device
    code, gcode = _code(dtype, "dy"), _code(grad_dtype, "grad_dtype")
    xp, ldx, codes, scales, *_ = _kept(x, "x", cols, rows, dtype, device)
    g = _vector(gamma, "gamma", cols, device)
    mu, rs = _vector(mean, "mean", rows, device), _vector(rstd, "rstd", rows, device)
    ap, lda = (add.data_ptr(), _matrix(add, "add", cols, rows, dtype, device)[2]) if add is not None else (None, 0)
    fn, need = _functions(), ctypes.c_size_t()
    with torch.cuda.device(device):
        dx = _like(dy)
        dgamma, dbeta = torch.empty(cols, dtype=grad_dtype, device=device), torch.empty(cols, dtype=grad_dtype, device=device)
        st = fn.onebit_layer_norm_backward_workspace(rows, cols, need)
        if st:
            _check(st, "onebit_layer_norm_backward_workspace")
        ws = _workspace(need.value, device)
        st = fn.onebit_layer_norm_backward(
            dy.data_ptr(), lddy, xp, ldx, codes, scales, code, rows, cols, g, mu, rs, ap, lda, dx.data_ptr(), cols,
            dgamma.data_ptr(), dbeta.data_ptr(), gcode, ws.data_ptr() if ws is not None else None, need.value, _stream(device))
    if st:
        _check(st, "onebit_layer_norm_backward")
    return dx, dgamma, dbeta


def _with_workspace(run, size, args, device, where):
    """Calls run(args, workspace, bytes, stream): without a workspace, which is enough for most calls, and with
    one where the call says that it needs it (it has enqueued nothing then)."""
    stream = _stream(device)
    st = run(args, None, 0, stream)
    if st == ERR_WORKSPACE:
        need = ctypes.c_size_t()
        st = size(args, need)
        if not st:
            ws = _workspace(need.value, device)
            st = run(args, ws.data_ptr(), need.value, stream)
    if st:
        _check(st, where)


def linear(x, w, bias=None, activation=ACT_NONE, residual=None, checkpoint=False, stream=None):
    """y = activation(x w^T + bias) + residual; with ``checkpoint`` (y, the 8-bit checkpoint of x w^T + bias)."""
    if stream is not None:
        with _on(stream, x):
            return linear(x, w, bias, activation, residual, checkpoint)
    if _fn is None:
        _functions()
    fast = _layers_binding.linear(x, w, bias, activation, residual, checkpoint)
    if fast is not None:
        return fast
    rows, cols, ldx = _matrix(x, "x")
    dtype, device = x.dtype, x.device
    code = _code(dtype, "x")
    if w.dim() != 2:
        raise ValueError("w: expected out x in")
    out, _, ldw = _matrix(w, "w", cols, None, dtype, device)
    bp = _vector(bias, "bias", out, device)
    rp, ldr = (residual.data_ptr(), _matrix(residual, "residual", out, rows, dtype, device)[2]) if residual is not None else (None, 0)
    with torch.cuda.device(device):
        y = _rows_by(x, rows, out, dtype, device)
        ck = _new_checkpoint(x, rows, out, dtype, device) if checkpoint else None
        a = LinearArgs(x.data_ptr(), ldx, w.data_ptr(), ldw, bp, rp, ldr, y.data_ptr(), out,
                       ck[0].data_ptr() if checkpoint else None, ck[1].data_ptr() if checkpoint else None, rows, cols, out, code,
                       activation)
        fn = _functions()
        _with_workspace(fn.onebit_linear_forward, fn.onebit_linear_forward_workspace, a, device, "onebit_linear_forward")
    return (y, ck) if checkpoint else y


def linear_backward(dy, x, w, activation=ACT_NONE, add=None, grad_dtype=None, dw=None, db=None, need=("dx", "dw", "db"),
                    stream=None):
    """(dx, dw, db) of y = activation(x) w^T + bias, given dy: x is the value before the activation that
    precedes the product (with ACT_NONE the product's input), a tensor or its Checkpoint; ``add`` joins
    dx.  grad_dtype (default dy's) is the type of dw (out x in) and db; ``dw`` and ``db`` may be the
    caller's contiguous tensors.  What ``need`` leaves out is None.  Whatever grad_dtype, dw is
    summed in fp32 from dy and activation(x) rounded to 16 bits, as the forward product takes it."""
    if stream is not None:
        with _on(stream, dy):
            return linear_backward(dy, x, w, activation, add, grad_dtype, dw, db, need)
    if _fn is None:
        _functions()
    fast = _layers_binding.linear_backward(dy, x, w, activation, add, grad_dtype, dw, db, need)
    if fast is not None:
        return fast
    rows, out, lddy = _matrix(dy, "dy")
    dtype, device = dy.dtype, dy.device
    code = _code(dtype, "dy")
    grad_dtype = dtype if grad_dtype is None else grad_dtype
    gcode = _code(grad_dtype, "grad_dtype")
    if w.dim() != 2:
        raise ValueError("w: expected out x in")
    _, cols, ldw = _matrix(w, "w", None, out, dtype, device)
    xp, ldx, codes, scales = None, 0, None, None
    if x is not None:
        xp, ldx, codes, scales, *_ = _kept(x, "x", cols, rows, dtype, device)
    ap, lda = (add.data_ptr(), _matrix(add, "add", cols, rows, dtype, device)[2]) if add is not None else (None, 0)
    want_dx, want_dw, want_db = "dx" in need, "dw" in need, "db" in need
    with torch.cuda.device(device):
        dx = _rows_by(dy, rows, cols, dtype, device) if want_dx else None
        if not want_dw:
            dw = None
        elif dw is None:
            dw = torch.empty(out, cols, dtype=grad_dtype, device=device)
        if not want_db:
            db = None
        elif db is None:
            db = torch.empty(out, dtype=grad_dtype, device=device)
        a = LinearGradArgs(dy.data_ptr(), lddy, xp, ldx, codes, scales, w.data_ptr(), ldw, ap, lda,
                           dx.data_ptr() if want_dx else None, cols, _vector(dw, "dw", out * cols, device, grad_dtype),
                           _vector(db, "db", out, device, grad_dtype), rows, cols, out, code, activation, gcode)
        fn = _functions()
        _with_workspace(fn.onebit_linear_backward, fn.onebit_linear_backward_workspace, a, device, "onebit_linear_backward")
    return dx, dw, db
