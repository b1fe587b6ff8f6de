// layers_binding.cpp -- the layer operators called from Python without ctypes.
//
// A small call (16 tokens) spends 3 us on the GPU; through ctypes and Python's allocation calls the host needed
// 15 us for it.  Here the common case of each operator of layers.py (2-D CUDA tensors, unit column stride,
// matching types, at least one row) is checked, its outputs allocated and the C entry called in one step, with the
// tensors' device made current for that time.
// Whatever else it meets -- another layout, an argument that does not fit, a status that is not OK -- it leaves
// to layers.py by returning None: that path then does the call, or says what is wrong with it.  A call with a
// failed check has enqueued nothing by then; one whose launch failed is enqueued again from its start, into new outputs
// (or the caller's dw and db), and fails again.
#include <Python.h>

#include <string.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/onebit_layers.h"

namespace {

struct Entries {
  decltype(&onebit_checkpoint_compress) compress;
  decltype(&onebit_checkpoint_restore) restore;
  decltype(&onebit_layer_norm_forward) ln_forward;
  decltype(&onebit_layer_norm_backward_workspace) ln_workspace;
  decltype(&onebit_layer_norm_backward) ln_backward;
  decltype(&onebit_linear_forward_workspace) forward_workspace;
  decltype(&onebit_linear_forward) forward;
  decltype(&onebit_linear_backward_workspace) backward_workspace;
  decltype(&onebit_linear_backward) backward;
  decltype(&onebit_gated_linear_forward_workspace) gated_forward_workspace;
  decltype(&onebit_gated_linear_forward) gated_forward;
  decltype(&onebit_gated_linear_backward_workspace) gated_backward_workspace;
  decltype(&onebit_gated_linear_backward) gated_backward;
  decltype(&onebit_dropout) dropout;
  decltype(&onebit_residual_norm_forward) rn_forward;
  decltype(&onebit_residual_norm_backward_workspace) rn_workspace;
  decltype(&onebit_residual_norm_backward) rn_backward;
} g_entry;
constexpr int kEntries = 17;
PyTypeObject* g_checkpoint = nullptr;  // layers.Checkpoint
PyTypeObject *g_gated = nullptr, *g_norm = nullptr, *g_norm_grads = nullptr;  // layers.Gated, ResidualNorm, ResidualNormGrads

struct Decline {};  // to layers.py

void require(bool ok) {
  if (!ok) throw Decline{};
}

int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return ONEBIT_F32;
    case at::kHalf: return ONEBIT_F16;
    case at::kBFloat16: return ONEBIT_BF16;
    default: throw Decline{};
  }
}

const at::Tensor& tensor(PyObject* o) {
  require(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

// would it be detached in silence?  (layers.py says so)
bool has_history(const at::Tensor& t) { return t.requires_grad() && at::GradMode::is_enabled(); }

struct Matrix {
  const void* p;
  int64_t rows, cols, ld;
};
Matrix matrix(const at::Tensor& t) {
  require(t.is_cuda() && t.dim() == 2 && !has_history(t));
  const int64_t r = t.size(0), c = t.size(1), ld = t.stride(0);
  require(r > 0 && c > 0 && t.stride(1) == 1 && (ld >= c || r == 1));
  return {t.data_ptr(), r, c, r == 1 ? c : ld};
}
Matrix matrix(const at::Tensor& t, const at::Tensor& like, int64_t rows, int64_t cols) {
  const Matrix m = matrix(t);
  require(m.rows == rows && m.cols == cols && t.scalar_type() == like.scalar_type() && t.device() == like.device());
  return m;
}
const float* vector(PyObject* o, int64_t n, const at::Tensor& like) {
  const at::Tensor& t = tensor(o);
  require(t.scalar_type() == at::kFloat && t.numel() == n && t.is_contiguous() && t.device() == like.device() && !has_history(t));
  return static_cast<const float*>(t.data_ptr());
}

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, const at::Tensor& like) {
  return at::Tensor(at::detail::empty_cuda(size, type, like.device(), std::nullopt));
}
void* stream(const at::Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

// New references; a NULL anywhere is an error that Python has been told of.
PyObject* pack(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New((Py_ssize_t)items.size());
  bool ok = t != nullptr;
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    ok = ok && o;
    if (t) PyTuple_SET_ITEM(t, i++, o);
    else Py_XDECREF(o);
  }
  if (!ok) Py_CLEAR(t);
  return t;
}
PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* none() { return Py_NewRef(Py_None); }

// Several results out of one allocation, each on 256 bytes: an allocation takes the host as long as a third of a launch.  For
// vectors, for what is needed together, and for matrices so small that nothing is lost when one of them outlives the others.
constexpr int64_t kSmall = 1 << 17;  // bytes
int64_t padded(int64_t count, at::ScalarType type) { return (count * (int64_t)c10::elementSize(type) + 255) / 256 * 256; }
struct Pieces {
  at::Tensor all;
  int64_t used = 0;
  Pieces(int64_t bytes, const at::Tensor& like) {
    if (bytes > 0) all = empty({bytes}, at::kByte, like);
  }
  at::Tensor next(at::IntArrayRef size, at::ScalarType type) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset(used / (int64_t)c10::elementSize(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(size);
    used += padded(t.numel(), type);
    return t;
  }
};
struct NewCheckpoint {
  at::Tensor codes, scales;
  NewCheckpoint(int64_t rows, int64_t cols, const at::Tensor& like)
      : codes(empty({rows, cols}, at::kChar, like)),
        scales(empty({rows, blocks(cols)}, at::kFloat, like)) {}
  NewCheckpoint(int64_t rows, int64_t cols, Pieces& from) : codes(from.next({rows, cols}, at::kChar)), scales(from.next({rows, blocks(cols)}, at::kFloat)) {}
  static int64_t blocks(int64_t cols) { return (cols + ONEBIT_CHECKPOINT_BLOCK - 1) / ONEBIT_CHECKPOINT_BLOCK; }
  int8_t* c() const { return static_cast<int8_t*>(codes.data_ptr()); }
  float* s() const { return static_cast<float*>(scales.data_ptr()); }
  PyObject* object(at::ScalarType type) const {
    PyObject* args = pack({wrap(codes), wrap(scales), Py_NewRef(reinterpret_cast<PyObject*>(torch::getTHPDtype(type)))});
    if (!args) return nullptr;
    PyObject* r = PyObject_CallObject(reinterpret_cast<PyObject*>(g_checkpoint), args);
    Py_DECREF(args);
    return r;
  }
};

// A layer's kept input: a matrix or its checkpoint.
struct Kept {
  const void* x = nullptr;
  int64_t ldx = 0, rows = 0, cols = 0;
  const int8_t* codes = nullptr;
  const float* scales = nullptr;
  at::ScalarType type;
  const at::Tensor* on = nullptr;
};
Kept kept(PyObject* o) {
  Kept k;
  if (Py_TYPE(o) == g_checkpoint) {
    require(PyTuple_GET_SIZE(o) == 3);
    const at::Tensor& codes = tensor(PyTuple_GET_ITEM(o, 0));
    const Matrix m = matrix(codes);
    require(codes.scalar_type() == at::kChar && m.ld == m.cols);
    PyObject* type = PyTuple_GET_ITEM(o, 2);
    require(THPDtype_Check(type));
    k.type = reinterpret_cast<THPDtype*>(type)->scalar_type;
    k.rows = m.rows, k.cols = m.cols;
    k.codes = static_cast<const int8_t*>(m.p);
    k.scales = vector(PyTuple_GET_ITEM(o, 1), m.rows * ((m.cols + ONEBIT_CHECKPOINT_BLOCK - 1) / ONEBIT_CHECKPOINT_BLOCK), codes);
    k.on = &codes;
  } else {
    const at::Tensor& t = tensor(o);
    const Matrix m = matrix(t);
    k.type = t.scalar_type();
    k.x = m.p, k.ldx = m.ld, k.rows = m.rows, k.cols = m.cols;
    k.on = &t;
  }
  return k;
}
Kept kept(PyObject* o, const at::Tensor& like, int64_t rows, int64_t cols) {
  const Kept k = kept(o);
  require(k.rows == rows && k.cols == cols && k.type == like.scalar_type() && k.on->device() == like.device());
  return k;
}
at::ScalarType scalar_type(PyObject* o) {
  require(THPDtype_Check(o));
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}
int integer(PyObject* o) {
  require(PyLong_Check(o));
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Decline{};
  }
  require(v >= -1000 && v <= 1000);
  return (int)v;
}

template <typename Run, typename Size, typename Args>
void with_workspace(Run run, Size size, const Args& a, const at::Tensor& like) {
  void* s = stream(like);
  onebit_status_t st = run(&a, nullptr, 0, s);
  if (st == ONEBIT_ERR_WORKSPACE) {
    size_t need = 0;
    require(size(&a, &need) == ONEBIT_OK);
    const at::Tensor ws = empty({(int64_t)need}, at::kByte, like);
    st = run(&a, ws.data_ptr(), need, s);
  }
  require(st == ONEBIT_OK);
}

// The same for calls that need one most of the time: the size first.
template <typename Run, typename Size, typename Args>
void with_sized_workspace(Run run, Size size, const Args& a, const at::Tensor& like) {
  size_t need = 0;
  require(size(&a, &need) == ONEBIT_OK);
  at::Tensor ws;
  if (need > 0) ws = empty({(int64_t)need}, at::kByte, like);
  require(run(&a, need > 0 ? ws.data_ptr() : nullptr, need, stream(like)) == ONEBIT_OK);
}

// compress(x)
PyObject* compress(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0]);
  const Matrix m = matrix(x);
  const c10::cuda::CUDAGuard guard(x.device());
  const int code = dtype_code(x.scalar_type());
  const NewCheckpoint ck(m.rows, m.cols, x);
  require(g_entry.compress(m.p, m.ld, code, m.rows, m.cols, ck.c(), ck.s(), stream(x)) == ONEBIT_OK);
  return ck.object(x.scalar_type());
}

// restore(checkpoint, activation)
PyObject* restore(PyObject* const* a) {
  require(Py_TYPE(a[0]) == g_checkpoint);
  const Kept k = kept(a[0]);
  const c10::cuda::CUDAGuard guard(k.on->device());
  const int code = dtype_code(k.type), act = integer(a[1]);
  at::Tensor x = empty({k.rows, k.cols}, k.type, *k.on);
  require(g_entry.restore(k.codes, k.scales, k.rows, k.cols, act, x.data_ptr(), k.cols, code, stream(x)) == ONEBIT_OK);
  return wrap(std::move(x));
}

// layer_norm(x, gamma, beta, eps, checkpoint)
PyObject* layer_norm(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0]);
  const Matrix m = matrix(x);
  const c10::cuda::CUDAGuard guard(x.device());
  const int code = dtype_code(x.scalar_type());
  const float *gamma = vector(a[1], m.cols, x), *beta = vector(a[2], m.cols, x);
  require(PyFloat_Check(a[3]));
  const bool keep = a[4] == Py_True;
  require(keep || a[4] == Py_False);
  at::Tensor y = empty({m.rows, m.cols}, x.scalar_type(), x), mean = empty({m.rows}, at::kFloat, x), rstd = empty({m.rows}, at::kFloat, x);
  auto run = [&](int8_t* codes, float* scales) {
    require(g_entry.ln_forward(m.p, m.ld, code, m.rows, m.cols, gamma, beta, (float)PyFloat_AS_DOUBLE(a[3]), y.data_ptr(), m.cols,
                               static_cast<float*>(mean.data_ptr()), static_cast<float*>(rstd.data_ptr()), codes, scales, stream(x)) == ONEBIT_OK);
  };
  if (!keep) {
    run(nullptr, nullptr);
    return pack({wrap(std::move(y)), wrap(std::move(mean)), wrap(std::move(rstd))});
  }
  const NewCheckpoint ck(m.rows, m.cols, x);
  run(ck.c(), ck.s());
  return pack({wrap(std::move(y)), wrap(std::move(mean)), wrap(std::move(rstd)), ck.object(x.scalar_type())});
}

// layer_norm_backward(dy, x, gamma, mean, rstd, add, grad_dtype)
PyObject* layer_norm_backward(PyObject* const* a) {
  const at::Tensor& dy = tensor(a[0]);
  const Matrix m = matrix(dy);
  const c10::cuda::CUDAGuard guard(dy.device());
  const int code = dtype_code(dy.scalar_type());
  const Kept k = kept(a[1], dy, m.rows, m.cols);
  const float *gamma = vector(a[2], m.cols, dy), *mean = vector(a[3], m.rows, dy), *rstd = vector(a[4], m.rows, dy);
  Matrix add{nullptr, 0, 0, 0};
  if (a[5] != Py_None) add = matrix(tensor(a[5]), dy, m.rows, m.cols);
  const at::ScalarType grad = scalar_type(a[6]);
  const int gcode = dtype_code(grad);
  size_t need = 0;
  require(g_entry.ln_workspace(m.rows, m.cols, &need) == ONEBIT_OK);
  at::Tensor dx = empty({m.rows, m.cols}, dy.scalar_type(), dy), dgamma = empty({m.cols}, grad, dy), dbeta = empty({m.cols}, grad, dy);
  const at::Tensor ws = empty({(int64_t)need}, at::kByte, dy);
  require(g_entry.ln_backward(m.p, m.ld, k.x, k.ldx, k.codes, k.scales, code, m.rows, m.cols, gamma, mean, rstd, add.p, add.ld, dx.data_ptr(), m.cols,
                              dgamma.data_ptr(), dbeta.data_ptr(), gcode, ws.data_ptr(), need, stream(dy)) == ONEBIT_OK);
  return pack({wrap(std::move(dx)), wrap(std::move(dgamma)), wrap(std::move(dbeta))});
}

// linear(x, w, bias, activation, residual, checkpoint)
PyObject* linear(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0]);
  const at::Tensor& w = tensor(a[1]);
  const Matrix mx = matrix(x), mw = matrix(w);
  const c10::cuda::CUDAGuard guard(x.device());
  require(mw.cols == mx.cols && w.scalar_type() == x.scalar_type() && w.device() == x.device());
  onebit_linear_t p{};
  p.dtype = dtype_code(x.scalar_type());
  p.x = mx.p, p.ldx = mx.ld, p.w = mw.p, p.ldw = mw.ld;
  p.rows = mx.rows, p.in = mx.cols, p.out = mw.rows;
  if (a[2] != Py_None) p.bias = vector(a[2], p.out, x);
  p.activation = integer(a[3]);
  if (a[4] != Py_None) {
    const Matrix r = matrix(tensor(a[4]), x, p.rows, p.out);
    p.residual = r.p, p.ldr = r.ld;
  }
  const bool keep = a[5] == Py_True;
  require(keep || a[5] == Py_False);
  at::Tensor y = empty({p.rows, p.out}, x.scalar_type(), x);
  p.y = y.data_ptr(), p.ldy = p.out;
  if (!keep) {
    with_workspace(g_entry.forward, g_entry.forward_workspace, p, x);
    return wrap(std::move(y));
  }
  const NewCheckpoint ck(p.rows, p.out, x);
  p.codes = ck.c(), p.scales = ck.s();
  with_workspace(g_entry.forward, g_entry.forward_workspace, p, x);
  return pack({wrap(std::move(y)), ck.object(x.scalar_type())});
}

// linear_backward(dy, x, w, activation, add, grad_dtype, dw, db, need)
PyObject* linear_backward(PyObject* const* a) {
  const at::Tensor& dy = tensor(a[0]);
  const at::Tensor& w = tensor(a[2]);
  const Matrix md = matrix(dy), mw = matrix(w);
  const c10::cuda::CUDAGuard guard(dy.device());
  require(mw.rows == md.cols && w.scalar_type() == dy.scalar_type() && w.device() == dy.device());
  onebit_linear_grad_t p{};
  p.dtype = dtype_code(dy.scalar_type());
  p.dy = md.p, p.lddy = md.ld, p.w = mw.p, p.ldw = mw.ld;
  p.rows = md.rows, p.in = mw.cols, p.out = mw.rows;
  if (a[1] != Py_None) {
    const Kept k = kept(a[1], dy, p.rows, p.in);
    p.x = k.x, p.ldx = k.ldx, p.codes = k.codes, p.scales = k.scales;
  }
  p.activation = integer(a[3]);
  if (a[4] != Py_None) {
    const Matrix m = matrix(tensor(a[4]), dy, p.rows, p.in);
    p.add = m.p, p.ldadd = m.ld;
  }
  const at::ScalarType grad = a[5] == Py_None ? dy.scalar_type() : scalar_type(a[5]);
  p.grad_dtype = dtype_code(grad);
  require(PyTuple_Check(a[8]));
  bool want[3] = {false, false, false};
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(a[8]); ++i) {
    PyObject* o = PyTuple_GET_ITEM(a[8], i);
    require(PyUnicode_Check(o));
    for (int k = 0; k < 3; ++k)
      if (PyUnicode_CompareWithASCIIString(o, k == 0 ? "dx" : k == 1 ? "dw" : "db") == 0) want[k] = true;
  }
  at::Tensor dx, dw, db;
  if (want[0]) {
    dx = empty({p.rows, p.in}, dy.scalar_type(), dy);
    p.dx = dx.data_ptr(), p.lddx = p.in;
  }
  auto given = [&](PyObject* o, int64_t n) {
    const at::Tensor& t = tensor(o);
    require(t.scalar_type() == grad && t.numel() == n && t.is_contiguous() && t.device() == dy.device() && !has_history(t));
    return t.data_ptr();
  };
  if (want[1]) {
    if (a[6] != Py_None) p.dw = given(a[6], p.out * p.in);
    else dw = empty({p.out, p.in}, grad, dy), p.dw = dw.data_ptr();
  }
  if (want[2]) {
    if (a[7] != Py_None) p.db = given(a[7], p.out);
    else db = empty({p.out}, grad, dy), p.db = db.data_ptr();
  }
  with_workspace(g_entry.backward, g_entry.backward_workspace, p, dy);
  return pack({want[0] ? wrap(std::move(dx)) : none(), !want[1] ? none() : a[6] != Py_None ? Py_NewRef(a[6]) : wrap(std::move(dw)),
               !want[2] ? none() : a[7] != Py_None ? Py_NewRef(a[7]) : wrap(std::move(db))});
}

// an instance of one of the named tuples: as tuple makes it of its items (through the class's own __new__, a Python function, it
// takes the host as long as two allocations)
PyObject* named(PyTypeObject* type, std::initializer_list<PyObject*> items) {
  PyObject* args = pack({pack(items)});
  if (!args) return nullptr;
  PyObject* r = PyTuple_Type.tp_new(type, args, nullptr);
  Py_DECREF(args);
  return r;
}
PyObject* wrap_or_none(at::Tensor t) { return t.defined() ? wrap(std::move(t)) : none(); }
bool is(PyObject* o, const char* text) { return PyUnicode_Check(o) && PyUnicode_CompareWithASCIIString(o, text) == 0; }

// The names in the tuple `need`, of three.
void wanted(PyObject* need, const char* const (&names)[3], bool (&want)[3]) {
  require(PyTuple_Check(need));
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(need); ++i)
    for (int k = 0; k < 3; ++k)
      if (is(PyTuple_GET_ITEM(need, i), names[k])) want[k] = true;
}

// gated_linear(x, w, bias, activation, keep)
PyObject* gated_linear(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0]);
  const at::Tensor& w = tensor(a[1]);
  const Matrix mx = matrix(x), mw = matrix(w);
  const c10::cuda::CUDAGuard guard(x.device());
  require(mw.cols == mx.cols && mw.rows % 2 == 0 && w.scalar_type() == x.scalar_type() && w.device() == x.device());
  onebit_gated_linear_t p{};
  p.dtype = dtype_code(x.scalar_type());
  p.x = mx.p, p.ldx = mx.ld, p.w = mw.p, p.ldw = mw.ld;
  p.rows = mx.rows, p.in = mx.cols, p.inner = mw.rows / 2;
  if (a[2] != Py_None) p.bias = vector(a[2], mw.rows, x);
  p.activation = integer(a[3]);
  at::Tensor h = empty({p.rows, p.inner}, x.scalar_type(), x);
  p.h = h.data_ptr(), p.ldh = p.inner;
  if (a[4] == Py_None) {
    with_sized_workspace(g_entry.gated_forward, g_entry.gated_forward_workspace, p, x);
    return wrap(std::move(h));
  }
  if (is(a[4], "values")) {
    at::Tensor z = empty({p.rows, mw.rows}, x.scalar_type(), x);
    p.z = z.data_ptr(), p.ldz = mw.rows;
    with_sized_workspace(g_entry.gated_forward, g_entry.gated_forward_workspace, p, x);
    return pack({wrap(std::move(h)), wrap(std::move(z))});
  }
  require(is(a[4], "checkpoint"));
  // (both halves are kept and needed together)
  Pieces pieces(2 * (padded(p.rows * p.inner, at::kChar) + padded(p.rows * NewCheckpoint::blocks(p.inner), at::kFloat)), x);
  const NewCheckpoint gate(p.rows, p.inner, pieces), up(p.rows, p.inner, pieces);
  p.gate_codes = gate.c(), p.gate_scales = gate.s(), p.up_codes = up.c(), p.up_scales = up.s();
  with_sized_workspace(g_entry.gated_forward, g_entry.gated_forward_workspace, p, x);
  return pack({wrap(std::move(h)), named(g_gated, {gate.object(x.scalar_type()), up.object(x.scalar_type())})});
}

// gated_linear_backward(dy, z, w, activation, grad_dtype, dw, db, need)
PyObject* gated_linear_backward(PyObject* const* a) {
  const at::Tensor& dy = tensor(a[0]);
  const at::Tensor& w = tensor(a[2]);
  const Matrix md = matrix(dy), mw = matrix(w);
  const c10::cuda::CUDAGuard guard(dy.device());
  require(mw.rows == md.cols && w.scalar_type() == dy.scalar_type() && w.device() == dy.device());
  onebit_gated_linear_grad_t p{};
  p.dtype = dtype_code(dy.scalar_type());
  p.dy = md.p, p.lddy = md.ld, p.w = mw.p, p.ldw = mw.ld;
  p.rows = md.rows, p.inner = mw.cols, p.out = mw.rows;
  if (Py_TYPE(a[1]) == g_gated) {
    require(PyTuple_GET_SIZE(a[1]) == 2);
    PyObject *gate = PyTuple_GET_ITEM(a[1], 0), *up = PyTuple_GET_ITEM(a[1], 1);
    require(Py_TYPE(gate) == g_checkpoint && Py_TYPE(up) == g_checkpoint);
    const Kept g = kept(gate, dy, p.rows, p.inner), u = kept(up, dy, p.rows, p.inner);
    p.gate_codes = g.codes, p.gate_scales = g.scales, p.up_codes = u.codes, p.up_scales = u.scales;
  } else if (a[1] != Py_None) {
    const Matrix z = matrix(tensor(a[1]), dy, p.rows, 2 * p.inner);
    p.z = z.p, p.ldz = z.ld;
  }
  p.activation = integer(a[3]);
  const at::ScalarType grad = a[4] == Py_None ? dy.scalar_type() : scalar_type(a[4]);
  p.grad_dtype = dtype_code(grad);
  bool want[3] = {false, false, false};
  wanted(a[7], {"dz", "dw", "db"}, want);
  at::Tensor dz, dw, db;
  if (want[0]) {
    dz = empty({p.rows, 2 * p.inner}, dy.scalar_type(), dy);
    p.dz = dz.data_ptr(), p.lddz = 2 * p.inner;
  }
  auto given = [&](PyObject* o, int64_t n) {
    const at::Tensor& t = tensor(o);
    require(t.scalar_type() == grad && t.numel() == n && t.is_contiguous() && t.device() == dy.device() && !has_history(t));
    return t.data_ptr();
  };
  if (want[1]) {
    if (a[5] != Py_None) p.dw = given(a[5], p.out * p.inner);
    else dw = empty({p.out, p.inner}, grad, dy), p.dw = dw.data_ptr();
  }
  if (want[2]) {
    if (a[6] != Py_None) p.db = given(a[6], p.out);
    else db = empty({p.out}, grad, dy), p.db = db.data_ptr();
  }
  with_sized_workspace(g_entry.gated_backward, g_entry.gated_backward_workspace, p, dy);
  return pack({wrap_or_none(std::move(dz)), want[1] && a[5] != Py_None ? Py_NewRef(a[5]) : wrap_or_none(std::move(dw)),
               want[2] && a[6] != Py_None ? Py_NewRef(a[6]) : wrap_or_none(std::move(db))});
}

// a Python float (whole numbers: layers.py)
float real(PyObject* o) {
  require(PyFloat_Check(o));
  return (float)PyFloat_AS_DOUBLE(o);
}
struct DropoutArgs {
  float p;
  const int64_t* key = nullptr;
  uint32_t site;
  DropoutArgs(PyObject* p_, PyObject* key_, PyObject* site_, const at::Tensor& like) : p(real(p_)) {
    if (key_ != Py_None) {
      const at::Tensor& t = tensor(key_);
      require(t.scalar_type() == at::kLong && t.numel() == 2 && t.is_contiguous() && t.device() == like.device());
      key = static_cast<const int64_t*>(t.data_ptr());
    }
    require(PyLong_Check(site_));
    const unsigned long s = PyLong_AsUnsignedLong(site_);
    if (s == (unsigned long)-1 && PyErr_Occurred()) {
      PyErr_Clear();
      throw Decline{};
    }
    require(s <= 0xffffffffu);
    site = (uint32_t)s;
  }
};

// dropout(x, p, key, site)
PyObject* dropout(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0]);
  const Matrix m = matrix(x);
  const c10::cuda::CUDAGuard guard(x.device());
  const int code = dtype_code(x.scalar_type());
  const DropoutArgs d(a[1], a[2], a[3], x);
  at::Tensor y = empty({m.rows, m.cols}, x.scalar_type(), x);
  require(g_entry.dropout(m.p, m.ld, code, m.rows, m.cols, d.p, d.key, d.site, y.data_ptr(), m.cols, stream(x)) == ONEBIT_OK);
  return wrap(std::move(y));
}

const float* vector_or_null(PyObject* o, int64_t n, const at::Tensor& like) { return o == Py_None ? nullptr : vector(o, n, like); }
float* floats(const at::Tensor& t) { return t.defined() ? static_cast<float*>(t.data_ptr()) : nullptr; }
void* bytes(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// residual_norm(x, block, gamma, beta, eps, norm, block_gamma, block_beta, gate, scale, p, key, site)
PyObject* residual_norm(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0]);
  const Matrix m = matrix(x);
  const c10::cuda::CUDAGuard guard(x.device());
  onebit_residual_norm_t p{};
  p.dtype = dtype_code(x.scalar_type());
  p.rows = m.rows, p.cols = m.cols;
  p.x = m.p, p.ldx = m.ld;
  if (a[1] != Py_None) {
    const Matrix b = matrix(tensor(a[1]), x, m.rows, m.cols);
    p.block = b.p, p.ldblock = b.ld;
  }
  p.gamma = vector_or_null(a[2], m.cols, x), p.beta = vector_or_null(a[3], m.cols, x);
  p.block_gamma = vector_or_null(a[6], m.cols, x), p.block_beta = vector_or_null(a[7], m.cols, x), p.gate = vector_or_null(a[8], m.cols, x);
  p.eps = real(a[4]), p.norm = integer(a[5]), p.scale = real(a[9]);
  const DropoutArgs d(a[10], a[11], a[12], x);
  p.p = d.p, p.key = d.key, p.site = d.site;
  at::Tensor s, y, mean, rstd, block_mean, block_rstd;
  const bool layer = p.norm == ONEBIT_NORM_LAYER;
  const at::ScalarType type = x.scalar_type();
  const int64_t matrices = ((p.block != nullptr) + (p.gamma != nullptr)) * padded(m.rows * m.cols, type);
  const int statistics = (1 + layer) * ((p.gamma != nullptr) + (p.block_gamma != nullptr));
  const bool small = matrices <= kSmall;
  Pieces pieces((small ? matrices : 0) + statistics * padded(m.rows, at::kFloat), x);
  auto matrix_out = [&] { return small ? pieces.next({m.rows, m.cols}, type) : empty({m.rows, m.cols}, type, x); };
  if (p.block) s = matrix_out();
  if (p.gamma) y = matrix_out();
  if (p.gamma && layer) mean = pieces.next({m.rows}, at::kFloat);
  if (p.gamma) rstd = pieces.next({m.rows}, at::kFloat);
  if (p.block_gamma && layer) block_mean = pieces.next({m.rows}, at::kFloat);
  if (p.block_gamma) block_rstd = pieces.next({m.rows}, at::kFloat);
  p.s = bytes(s), p.y = bytes(y), p.lds = p.ldy = m.cols;
  p.mean = floats(mean), p.rstd = floats(rstd), p.block_mean = floats(block_mean), p.block_rstd = floats(block_rstd);
  require(g_entry.rn_forward(&p, stream(x)) == ONEBIT_OK);
  return named(g_norm, {wrap_or_none(std::move(y)), s.defined() ? wrap(std::move(s)) : Py_NewRef(a[0]), wrap_or_none(std::move(mean)),
                        wrap_or_none(std::move(rstd)), wrap_or_none(std::move(block_mean)), wrap_or_none(std::move(block_rstd))});
}

// residual_norm_backward(dy, ds, s, block, gamma, mean, rstd, norm, block_gamma, block_beta, block_mean, block_rstd, gate, scale, p, key, site,
//                        has_block, grad_dtype)
PyObject* residual_norm_backward(PyObject* const* a) {
  const at::Tensor& first = tensor(a[0] != Py_None ? a[0] : a[1]);
  const Matrix m = matrix(first);
  const c10::cuda::CUDAGuard guard(first.device());
  const int64_t rows = m.rows, cols = m.cols;
  onebit_residual_norm_grad_t p{};
  p.dtype = dtype_code(first.scalar_type());
  p.rows = rows, p.cols = cols;
  auto input = [&](PyObject* o, const void*& q, int64_t& ld) {
    if (o == Py_None) return;
    const Matrix t = matrix(tensor(o), first, rows, cols);
    q = t.p, ld = t.ld;
  };
  const bool has_block = a[17] == Py_True;
  require(has_block || a[17] == Py_False);
  input(a[0], p.dy, p.lddy);
  input(a[1], p.ds, p.ldds);
  if (a[4] != Py_None) input(a[2], p.s, p.lds);
  if (has_block) input(a[3], p.block, p.ldblock);
  p.gamma = vector_or_null(a[4], cols, first);
  p.mean = vector_or_null(a[5], rows, first), p.rstd = vector_or_null(a[6], rows, first);
  p.norm = integer(a[7]);
  p.block_gamma = vector_or_null(a[8], cols, first), p.block_beta = vector_or_null(a[9], cols, first);
  p.block_mean = vector_or_null(a[10], rows, first), p.block_rstd = vector_or_null(a[11], rows, first);
  p.gate = vector_or_null(a[12], cols, first);
  p.scale = real(a[13]);
  const DropoutArgs d(a[14], a[15], a[16], first);
  p.p = d.p, p.key = d.key, p.site = d.site;
  const at::ScalarType grad = scalar_type(a[18]);
  p.grad_dtype = dtype_code(grad);
  const bool layer = p.norm == ONEBIT_NORM_LAYER;
  at::Tensor dx = empty({rows, cols}, first.scalar_type(), first), dblock, dgamma, dbeta, dblock_gamma, dblock_beta, dgate;
  if (has_block) dblock = empty({rows, cols}, first.scalar_type(), first);
  Pieces grads(((1 + layer) * ((p.gamma != nullptr) + (p.block_gamma != nullptr)) + (p.gate != nullptr)) * padded(cols, grad), first);
  if (p.gamma) dgamma = grads.next({cols}, grad);
  if (p.gamma && layer) dbeta = grads.next({cols}, grad);
  if (p.block_gamma) dblock_gamma = grads.next({cols}, grad);
  if (p.block_gamma && layer) dblock_beta = grads.next({cols}, grad);
  if (p.gate) dgate = grads.next({cols}, grad);
  p.dx = dx.data_ptr(), p.dblock = bytes(dblock), p.lddx = p.lddblock = cols;
  p.dgamma = bytes(dgamma), p.dbeta = bytes(dbeta), p.dblock_gamma = bytes(dblock_gamma), p.dblock_beta = bytes(dblock_beta), p.dgate = bytes(dgate);
  size_t need = 0;
  require(g_entry.rn_workspace(&p, &need) == ONEBIT_OK);
  const at::Tensor ws = empty({(int64_t)need}, at::kByte, first);
  require(g_entry.rn_backward(&p, ws.data_ptr(), need, stream(first)) == ONEBIT_OK);
  return named(g_norm_grads, {wrap(std::move(dx)), wrap_or_none(std::move(dblock)), wrap_or_none(std::move(dgamma)), wrap_or_none(std::move(dbeta)),
                              wrap_or_none(std::move(dblock_gamma)), wrap_or_none(std::move(dblock_beta)), wrap_or_none(std::move(dgate))});
}

// Runs f on the arguments; None where it declines.  No C++ exception passes into Python.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Decline&) {
    return none();
  } catch (const std::exception&) {  // out of memory: layers.py's own allocation says so
    return none();
  }
}

// setup(addresses of the C entries, Checkpoint, Gated, ResidualNorm, ResidualNormGrads)
PyObject* setup(PyObject*, PyObject* const* args, Py_ssize_t n) {
  bool ok = n == 5 && PyTuple_Check(args[0]) && PyTuple_GET_SIZE(args[0]) == kEntries;
  for (int i = 1; i < 5 && ok; ++i) ok = PyType_Check(args[i]);
  if (!ok) {
    PyErr_SetString(PyExc_TypeError, "setup(seventeen addresses, Checkpoint, Gated, ResidualNorm, ResidualNormGrads)");
    return nullptr;
  }
  static_assert(sizeof(Entries) == kEntries * sizeof(void*), "one address each");
  void* p[kEntries];
  for (int i = 0; i < kEntries; ++i) {
    p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args[0], i));
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a NULL address");
      return nullptr;
    }
  }
  memcpy(&g_entry, p, sizeof p);  // in the order of Entries
  g_checkpoint = reinterpret_cast<PyTypeObject*>(Py_NewRef(args[1]));
  g_gated = reinterpret_cast<PyTypeObject*>(Py_NewRef(args[2]));
  g_norm = reinterpret_cast<PyTypeObject*>(Py_NewRef(args[3]));
  g_norm_grads = reinterpret_cast<PyTypeObject*>(Py_NewRef(args[4]));
  return none();
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction as_method(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef g_methods[] = {
    {"setup", as_method(setup), METH_FASTCALL, nullptr},
    {"compress", as_method(call<compress, 1>), METH_FASTCALL, nullptr},
    {"restore", as_method(call<restore, 2>), METH_FASTCALL, nullptr},
    {"layer_norm", as_method(call<layer_norm, 5>), METH_FASTCALL, nullptr},
    {"layer_norm_backward", as_method(call<layer_norm_backward, 7>), METH_FASTCALL, nullptr},
    {"linear", as_method(call<linear, 6>), METH_FASTCALL, nullptr},
    {"linear_backward", as_method(call<linear_backward, 9>), METH_FASTCALL, nullptr},
    {"gated_linear", as_method(call<gated_linear, 5>), METH_FASTCALL, nullptr},
    {"gated_linear_backward", as_method(call<gated_linear_backward, 8>), METH_FASTCALL, nullptr},
    {"dropout", as_method(call<dropout, 4>), METH_FASTCALL, nullptr},
    {"residual_norm", as_method(call<residual_norm, 13>), METH_FASTCALL, nullptr},
    {"residual_norm_backward", as_method(call<residual_norm_backward, 19>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_layers_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers_binding(void) { return PyModule_Create(&g_module); }
