"""Layer operators that produce the gradients the optimizer exchanges: layer norm, the linear layer with
a fused epilogue, the gated linear layer, dropout, the residual sum with the norms around it, and activation
checkpoints held in 8 bits, forward and backward.

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

    s = x + dropout(W2 (silu(Wg x) * (Wu x))), then an RMS norm, W1 holding Wg's rows and then Wu's:

    key = torch.tensor([seed, step], device="cuda")
    h, z8 = layers.gated_linear(x, w1, keep="checkpoint")
    f = layers.linear(h, w2)
    r = layers.residual_norm(x, f, gamma, norm=layers.NORM_RMS, p=0.1, key=key)
    g = layers.residual_norm_backward(dy, ds, r.s, None, gamma, None, r.rstd, norm=layers.NORM_RMS, p=0.1, key=key)
    dz, dw2, _ = layers.gated_linear_backward(g.dblock, z8, w2, need=("dz", "dw"))
    dx, dw1, _ = layers.linear_backward(dz, x, w1, add=g.dx, need=("dx", "dw"))
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import os
from typing import NamedTuple

import torch

from . import BF16, ERR_WORKSPACE, F16, F32, OK, OneBitError, _stream_ptr, lib

ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = range(5)
ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH}
GATE_ACTIVATIONS = {**ACTIVATIONS, "silu": ACT_SILU}  # those of the gated linear layer
NORM_LAYER, NORM_RMS = range(2)
NORMS = {"layer": NORM_LAYER, "rms": NORM_RMS}
CHECKPOINT_BLOCK = 64  # columns of a row that share one scale

_DTYPE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}


class Checkpoint(NamedTuple):
    """A matrix in 8 bits: int8 ``codes`` of its shape, fp32 ``scales`` with one value per 64 columns of
    a row, and the ``dtype`` of the matrix it stands for."""

    codes: torch.Tensor
    scales: torch.Tensor
    dtype: torch.dtype


class Gated(NamedTuple):
    """The checkpoints of a gated linear layer's two halves before the gating."""

    gate: Checkpoint
    up: Checkpoint


class ResidualNorm(NamedTuple):
    """What residual_norm returns; None for what a call does not have."""

    y: torch.Tensor | None
    s: torch.Tensor
    mean: torch.Tensor | None
    rstd: torch.Tensor | None
    block_mean: torch.Tensor | None
    block_rstd: torch.Tensor | None


class ResidualNormGrads(NamedTuple):
    """What residual_norm_backward returns; None for what a call does not have."""

    dx: torch.Tensor
    dblock: torch.Tensor | None
    dgamma: torch.Tensor | None
    dbeta: torch.Tensor | None
    dblock_gamma: torch.Tensor | None
    dblock_beta: torch.Tensor | None
    dgate: torch.Tensor | None


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


def _fields(spec):
    """ctypes fields from "name name:type ..." (pointers where no type is given; ld* are strides)."""
    types = {"i64": ctypes.c_int64, "i32": ctypes.c_int32, "u32": ctypes.c_uint32, "f32": ctypes.c_float}
    out = []
    for word in spec.split():
        name, _, kind = word.partition(":")
        out.append((name, types[kind] if kind else ctypes.c_int64 if name.startswith("ld") else ctypes.c_void_p))
    return out


class GatedLinearArgs(ctypes.Structure):
    _fields_ = _fields("x ldx w ldw bias h ldh z ldz gate_codes gate_scales up_codes up_scales rows:i64 in_:i64 inner:i64 "
                       "dtype:i32 activation:i32")


class GatedLinearGradArgs(ctypes.Structure):
    _fields_ = _fields("dy lddy z ldz gate_codes gate_scales up_codes up_scales w ldw dz lddz dw db rows:i64 inner:i64 out:i64 "
                       "dtype:i32 activation:i32 grad_dtype:i32")


class ResidualNormArgs(ctypes.Structure):
    _fields_ = _fields("x ldx block ldblock gamma beta block_gamma block_beta gate key s lds y ldy mean rstd block_mean block_rstd "
                       "rows:i64 cols:i64 dtype:i32 norm:i32 eps:f32 scale:f32 p:f32 site:u32")


class ResidualNormGradArgs(ctypes.Structure):
    _fields_ = _fields("dy lddy ds ldds s lds block ldblock gamma block_gamma block_beta gate key mean rstd block_mean block_rstd "
                       "dx lddx dblock lddblock dgamma dbeta dblock_gamma dblock_beta dgate rows:i64 cols:i64 dtype:i32 norm:i32 "
                       "grad_dtype:i32 scale:f32 p:f32 site:u32")


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
            "onebit_gated_linear_forward_workspace": [ctypes.POINTER(GatedLinearArgs), ctypes.POINTER(sz)],
            "onebit_gated_linear_forward": [ctypes.POINTER(GatedLinearArgs), vp, sz, vp],
            "onebit_gated_linear_backward_workspace": [ctypes.POINTER(GatedLinearGradArgs), ctypes.POINTER(sz)],
            "onebit_gated_linear_backward": [ctypes.POINTER(GatedLinearGradArgs), vp, sz, vp],
            "onebit_dropout": [vp, i64, i32, i64, i64, ctypes.c_float, vp, ctypes.c_uint32, vp, i64, vp],
            "onebit_residual_norm_forward": [ctypes.POINTER(ResidualNormArgs), vp],
            "onebit_residual_norm_backward_workspace": [ctypes.POINTER(ResidualNormGradArgs), ctypes.POINTER(sz)],
            "onebit_residual_norm_backward": [ctypes.POINTER(ResidualNormGradArgs), vp, sz, vp],
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
                 "onebit_linear_forward", "onebit_linear_backward_workspace", "onebit_linear_backward",
                 "onebit_gated_linear_forward_workspace", "onebit_gated_linear_forward",
                 "onebit_gated_linear_backward_workspace", "onebit_gated_linear_backward", "onebit_dropout",
                 "onebit_residual_norm_forward", "onebit_residual_norm_backward_workspace", "onebit_residual_norm_backward")
        _layers_binding.setup(tuple(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in names), Checkpoint, Gated,
                              ResidualNorm, ResidualNormGrads)
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
    """Waits for the stream; OK, or ERR_CUDA when a kernel of its device gave up waiting for its copies (a product) or for
    another block's part of a row (a residual norm of rows that several blocks share)."""
    with _device_of(stream):
        return int(_functions().onebit_layers_get_status(_stream_ptr(stream)))


def clear_status(stream=None):
    with _device_of(stream):
        _check(_functions().onebit_layers_clear_status(_stream_ptr(stream)), "onebit_layers_clear_status")


def set_fault_injection(kind: int, value: int = 0):
    """Test hook of the whole process: FAULT_STALL_COPIES makes the waits of the following products, and of residual norms of rows
    that several blocks share, run out."""
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


def gated_linear(x, w, bias=None, activation=ACT_SILU, keep=None, stream=None):
    """h = activation(g) * u with [g | u] = z = x w^T + bias; w holds the gate's rows and then as many of the up
    projection.  ``keep``: "values" returns (h, z), "checkpoint" (h, the 8-bit checkpoints of g and u, a Gated)."""
    if stream is not None:
        with _on(stream, x):
            return gated_linear(x, w, bias, activation, keep)
    if _fn is None:
        _functions()
    fast = _layers_binding.gated_linear(x, w, bias, activation, keep)
    if fast is not None:
        return fast
    rows, cols, ldx = _matrix(x, "x")
    dtype, device = x.dtype, x.device
    code = _code(dtype, "x")
    if w.dim() != 2 or w.shape[0] % 2:
        raise ValueError("w: expected 2 inner x in")
    if keep not in (None, "values", "checkpoint"):
        raise ValueError('keep: expected None, "values" or "checkpoint"')
    out, _, ldw = _matrix(w, "w", cols, None, dtype, device)
    inner = out // 2
    bp = _vector(bias, "bias", out, device)
    with torch.cuda.device(device):
        h = _rows_by(x, rows, inner, dtype, device)
        z = _rows_by(x, rows, out, dtype, device) if keep == "values" else None
        if keep == "checkpoint":
            z = Gated(_new_checkpoint(x, rows, inner, dtype, device), _new_checkpoint(x, rows, inner, dtype, device))
        a = GatedLinearArgs(x.data_ptr(), ldx, w.data_ptr(), ldw, bp, h.data_ptr(), inner, z.data_ptr() if keep == "values" else None, out,
                            *([t.data_ptr() for ck in z for t in ck[:2]] if keep == "checkpoint" else [None] * 4), rows, cols, inner, code,
                            activation)
        fn = _functions()
        _with_workspace(fn.onebit_gated_linear_forward, fn.onebit_gated_linear_forward_workspace, a, device, "onebit_gated_linear_forward")
    return h if keep is None else (h, z)


def gated_linear_backward(dy, z, w, activation=ACT_SILU, grad_dtype=None, dw=None, db=None, need=("dz", "dw", "db"), stream=None):
    """(dz, dw, db) of y = (activation(g) * u) w^T + bias, given dy: z = [g | u] is what gated_linear kept, a tensor or a
    Gated; dz is the dy of linear_backward for the gated layer's own weight.  grad_dtype (default dy's) is the type of dw (out x
    inner) and db; ``dw`` and ``db`` may be the caller's contiguous tensors.  What ``need`` leaves out is None.  dw is summed
    in fp32 from dy and activation(g) * u rounded to 16 bits, as the forward product takes it."""
    if stream is not None:
        with _on(stream, dy):
            return gated_linear_backward(dy, z, w, activation, grad_dtype, dw, db, need)
    if _fn is None:
        _functions()
    fast = _layers_binding.gated_linear_backward(dy, z, w, activation, grad_dtype, dw, db, need)
    if fast is not None:
        return fast
    rows, out, lddy = _matrix(dy, "dy")
    dtype, device = dy.dtype, dy.device
    code = _code(dtype, "dy")
    grad_dtype = dtype if grad_dtype is None else grad_dtype
    gcode = _code(grad_dtype, "grad_dtype")
    if w.dim() != 2:
        raise ValueError("w: expected out x inner")
    _, inner, ldw = _matrix(w, "w", None, out, dtype, device)
    zp, ldz, halves = None, 0, [None] * 4
    if isinstance(z, Gated):
        halves = [p for name, ck in zip(("z.gate", "z.up"), z) for p in _kept(_checkpoint(ck, name), name, inner, rows, dtype, device)[2:4]]
    elif z is not None:
        ldz = _matrix(z, "z", 2 * inner, rows, dtype, device)[2]
        zp = z.data_ptr()
    want_dz, want_dw, want_db = "dz" in need, "dw" in need, "db" in need
    with torch.cuda.device(device):
        dz = _rows_by(dy, rows, 2 * inner, dtype, device) if want_dz else None
        if not want_dw:
            dw = None
        elif dw is None:
            dw = torch.empty(out, inner, dtype=grad_dtype, device=device)
        if not want_db:
            db = None
        elif db is None:
            db = torch.empty(out, dtype=grad_dtype, device=device)
        a = GatedLinearGradArgs(dy.data_ptr(), lddy, zp, ldz, *halves, w.data_ptr(), ldw, dz.data_ptr() if want_dz else None, 2 * inner,
                                _vector(dw, "dw", out * inner, device, grad_dtype), _vector(db, "db", out, device, grad_dtype), rows, inner,
                                out, code, activation, gcode)
        fn = _functions()
        _with_workspace(fn.onebit_gated_linear_backward, fn.onebit_gated_linear_backward_workspace, a, device, "onebit_gated_linear_backward")
    return dz, dw, db


def _checkpoint(ck, name):
    if not isinstance(ck, Checkpoint):
        raise ValueError(f"{name}: expected a Checkpoint")
    return ck


def _dropout_key(p, key, site, device):
    """The key's pointer (None: no dropout)."""
    if not 0 <= site < 1 << 32:
        raise ValueError("site: expected a whole number below 2^32")
    if key is None:
        if p > 0:
            raise ValueError("key: dropout needs two int64 values, seed and step")
        return None
    return _vector(key, "key", 2, device, torch.int64)


def dropout(x, p, key, site=0, stream=None):
    """x with each element set to 0 with probability p (in steps of 1/65536), the others divided by 1 - p.  ``key`` is a CUDA
    tensor of two int64 values, seed and step, read when the kernel runs; ``site`` tells the places of a model apart that use one
    key.  The backward pass is the same call on the gradient."""
    if stream is not None:
        with _on(stream, x):
            return dropout(x, p, key, site)
    if _fn is None:
        _functions()
    fast = _layers_binding.dropout(x, p, key, site)
    if fast is not None:
        return fast
    rows, cols, ld = _matrix(x, "x")
    code, device = _code(x.dtype, "x"), x.device
    kp = _dropout_key(p, key, site, device)
    with torch.cuda.device(device):
        y = _like(x)
        st = _functions().onebit_dropout(x.data_ptr(), ld, code, rows, cols, p, kp, site, y.data_ptr(), cols, _stream(device))
    if st:
        _check(st, "onebit_dropout")
    return y


def residual_norm(x, block=None, gamma=None, beta=None, eps=1e-5, norm=NORM_LAYER, block_gamma=None, block_beta=None, gate=None, scale=1.0,
                  p=0.0, key=None, site=0, stream=None) -> ResidualNorm:
    """s = x + scale * gate * dropout(n) and y = norm(s) * gamma + beta, where n is ``block``, a block's output, or with
    ``block_gamma`` norm(block) * block_gamma + block_beta.  Without a block s is x itself; without gamma there is no y.  ``norm`` is
    that of both places: NORM_LAYER, with beta and block_beta, or NORM_RMS, without.  p, key and site as for dropout().  s, mean,
    rstd, block_mean and block_rstd are what the backward pass needs beside the call's arguments."""
    if stream is not None:
        with _on(stream, x):
            return residual_norm(x, block, gamma, beta, eps, norm, block_gamma, block_beta, gate, scale, p, key, site)
    if _fn is None:
        _functions()
    fast = _layers_binding.residual_norm(x, block, gamma, beta, eps, norm, block_gamma, block_beta, gate, scale, p, key, site)
    if fast is not None:
        return fast
    rows, cols, ldx = _matrix(x, "x")
    dtype, device = x.dtype, x.device
    code = _code(dtype, "x")
    bp, ldb = (block.data_ptr(), _matrix(block, "block", cols, rows, dtype, device)[2]) if block is not None else (None, 0)
    vectors = [_vector(v, name, cols, device) for v, name in ((gamma, "gamma"), (beta, "beta"), (block_gamma, "block_gamma"),
                                                              (block_beta, "block_beta"), (gate, "gate"))]
    kp = _dropout_key(p, key, site, device)
    layer = norm == NORM_LAYER
    with torch.cuda.device(device):
        s = _like(x) if block is not None else None
        y = _like(x) if gamma is not None else None
        stats = [_rows_of(x, rows, device) if there else None for there in
                 (gamma is not None and layer, gamma is not None, block_gamma is not None and layer, block_gamma is not None)]
        at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        a = ResidualNormArgs(x.data_ptr(), ldx, bp, ldb, *vectors, kp, at(s), cols, at(y), cols, *[at(t) for t in stats], rows, cols, code,
                             norm, eps, scale, p, site)
        st = _functions().onebit_residual_norm_forward(a, _stream(device))
    if st:
        _check(st, "onebit_residual_norm_forward")
    return ResidualNorm(y, x if s is None else s, *stats)


def residual_norm_backward(dy, ds, s, block, gamma, mean, rstd, norm=NORM_LAYER, block_gamma=None, block_beta=None, block_mean=None,
                           block_rstd=None, gate=None, scale=1.0, p=0.0, key=None, site=0, has_block=True, grad_dtype=torch.float32,
                           stream=None) -> ResidualNormGrads:
    """The gradients of residual_norm's call with these arguments, given dy (of y; None without gamma) and ds, the gradient of
    s from the residual path (or None).  ``block`` may be None where neither block_gamma nor gate is there; ``has_block=False`` stands
    for a call without a block, whose dblock is None.  The parameters' gradients come in grad_dtype."""
    first = ds if dy is None else dy
    if first is None:
        raise ValueError("dy, ds: one of them is needed")
    if stream is not None:
        with _on(stream, first):
            return residual_norm_backward(dy, ds, s, block, gamma, mean, rstd, norm, block_gamma, block_beta, block_mean, block_rstd, gate,
                                          scale, p, key, site, has_block, grad_dtype)
    if _fn is None:
        _functions()
    fast = _layers_binding.residual_norm_backward(dy, ds, s, block, gamma, mean, rstd, norm, block_gamma, block_beta, block_mean, block_rstd,
                                                  gate, scale, p, key, site, has_block, grad_dtype)
    if fast is not None:
        return fast
    rows, cols, _ = _matrix(first, "ds" if dy is None else "dy")
    dtype, device = first.dtype, first.device
    code, gcode = _code(dtype, "dy"), _code(grad_dtype, "grad_dtype")
    inputs = []
    for t, name in ((dy, "dy"), (ds, "ds"), (s if gamma is not None else None, "s"), (block if has_block else None, "block")):
        inputs += [t.data_ptr(), _matrix(t, name, cols, rows, dtype, device)[2]] if t is not None else [None, 0]
    vectors = [_vector(v, name, cols, device) for v, name in ((gamma, "gamma"), (block_gamma, "block_gamma"), (block_beta, "block_beta"),
                                                              (gate, "gate"))]
    kp = _dropout_key(p, key, site, device)
    stats = [_vector(v, name, rows, device) for v, name in ((mean, "mean"), (rstd, "rstd"), (block_mean, "block_mean"), (block_rstd, "block_rstd"))]
    layer = norm == NORM_LAYER
    need, fn = ctypes.c_size_t(), _functions()
    with torch.cuda.device(device):
        dx, dblock = _like(first), _like(first) if has_block else None
        grads = [torch.empty(cols, dtype=grad_dtype, device=device) if there else None for there in
                 (gamma is not None, gamma is not None and layer, block_gamma is not None, block_gamma is not None and layer, gate is not None)]
        at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        a = ResidualNormGradArgs(*inputs, *vectors, kp, *stats, dx.data_ptr(), cols, at(dblock), cols, *[at(t) for t in grads], rows, cols, code,
                                 norm, gcode, scale, p, site)
        st = fn.onebit_residual_norm_backward_workspace(a, need)
        if st:
            _check(st, "onebit_residual_norm_backward_workspace")
        ws = _workspace(need.value, device)
        st = fn.onebit_residual_norm_backward(a, at(ws), need.value, _stream(device))
    if st:
        _check(st, "onebit_residual_norm_backward")
    return ResidualNormGrads(dx, dblock, *grads)
