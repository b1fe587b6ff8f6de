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
} g_entry;
PyTypeObject* g_checkpoint = nullptr;  // layers.Checkpoint

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

struct NewCheckpoint {
  at::Tensor codes, scales;
  NewCheckpoint(int64_t rows, int64_t cols, const at::Tensor& like)
      : codes(empty({rows, cols}, at::kChar, like)),
        scales(empty({rows, (cols + ONEBIT_CHECKPOINT_BLOCK - 1) / ONEBIT_CHECKPOINT_BLOCK}, at::kFloat, like)) {}
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

// setup(addresses of the C entries, Checkpoint)
PyObject* setup(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 2 || !PyTuple_Check(args[0]) || PyTuple_GET_SIZE(args[0]) != 9 || !PyType_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "setup(nine addresses, Checkpoint)");
    return nullptr;
  }
  void* p[9];
  for (int i = 0; i < 9; ++i) {
    p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args[0], i));
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a NULL address");
      return nullptr;
    }
  }
  g_entry.compress = reinterpret_cast<decltype(g_entry.compress)>(p[0]);
  g_entry.restore = reinterpret_cast<decltype(g_entry.restore)>(p[1]);
  g_entry.ln_forward = reinterpret_cast<decltype(g_entry.ln_forward)>(p[2]);
  g_entry.ln_workspace = reinterpret_cast<decltype(g_entry.ln_workspace)>(p[3]);
  g_entry.ln_backward = reinterpret_cast<decltype(g_entry.ln_backward)>(p[4]);
  g_entry.forward_workspace = reinterpret_cast<decltype(g_entry.forward_workspace)>(p[5]);
  g_entry.forward = reinterpret_cast<decltype(g_entry.forward)>(p[6]);
  g_entry.backward_workspace = reinterpret_cast<decltype(g_entry.backward_workspace)>(p[7]);
  g_entry.backward = reinterpret_cast<decltype(g_entry.backward)>(p[8]);
  g_checkpoint = reinterpret_cast<PyTypeObject*>(Py_NewRef(args[1]));
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
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_layers_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers_binding(void) { return PyModule_Create(&g_module); }
