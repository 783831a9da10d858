// The calls of mx4.py without Python's cost for each argument: a small extension module that looks at
// the tensors of a regular call (one device, the current stream, rows that lie as the library reads
// them), allocates its outputs and passes addresses and sizes to the C entry points, whose addresses
// bind() is given. Everything else (copies, other streams and devices, what is refused) it leaves to
// the Python function, by returning None, before anything is allocated or enqueued. A status that the
// C entry point returns comes back as a number.
// A queued call of one row takes 5 to 7 us of host time so, 10 to 15 through ctypes; the launch alone
// is 2.6.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "sparse_ffn_mx4.h"

namespace {

decltype(&sparse_ffn_rms_norm) c_norm;
decltype(&sparse_ffn_quantize_mx4) c_quantize;
decltype(&sparse_ffn_dequantize_mx4) c_dequantize;
decltype(&sparse_ffn_mx4_matmul_work_bytes) c_work_bytes;
decltype(&sparse_ffn_mx4_matmul) c_matmul;

constexpr int64_t MOST = INT32_MAX;  // whole numbers of the C entry points

int type_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return SFFN_F32;
    case at::kHalf: return SFFN_F16;
    case at::kBFloat16: return SFFN_BF16;
    default: return -1;
  }
}
at::ScalarType type_for(int code) {
  return code == SFFN_F32 ? at::kFloat : code == SFFN_F16 ? at::kHalf : at::kBFloat16;
}

// The tensor behind a Python object, on device `dev`; null if it is not that
const at::Tensor* tensor(PyObject* o, int64_t dev) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.layout() == at::kStrided && t.is_cuda() && (int64_t)t.get_device() == dev ? &t : nullptr;
}

// Rows [R, K] of a tensor whose last dimension is K, ld elements apart, without a copy
struct Rows {
  int64_t R, K, ld;
  bool ok;
  explicit Rows(const at::Tensor& t) : R(0), K(0), ld(0), ok(false) {
    const int64_t n = t.dim();
    if (n < 1) return;
    K = t.size(n - 1);
    if (K < 1 || K > MOST) return;
    if (n == 2) {
      R = t.size(0);
      ld = R > 1 ? t.stride(0) : K;
      ok = R == 0 || ((t.stride(1) == 1 || K == 1) && ld >= K);
    } else {
      R = t.numel() / K;
      ld = K;
      ok = t.is_contiguous();
    }
    ok = ok && R <= MOST;
  }
};

// Two-dimensional rows in 4-bit blocks as the products read them
struct Blocks {
  int64_t R, B, ldq, lds;
  bool ok;
  Blocks(const at::Tensor& q, const at::Tensor& s) : R(0), B(0), ldq(0), lds(0), ok(false) {
    if (q.scalar_type() != at::kByte || s.scalar_type() != at::kByte || q.dim() != 2 || s.dim() != 2) return;
    R = q.size(0);
    B = s.size(1);
    if (R < 1 || R > MOST || B < 1 || B > MOST / 32 || s.size(0) != R || q.size(1) != 16 * B) return;
    const int64_t room = (B + 15) / 16 * 16;
    ldq = R > 1 ? q.stride(0) : 16 * B;
    lds = R > 1 ? s.stride(0) : room;
    if (q.stride(1) != 1 || (s.stride(1) != 1 && B > 1) || ldq % 16 || ldq < 16 * B || lds % 16 || lds < B) return;
    if (((uintptr_t)q.data_ptr() | (uintptr_t)s.data_ptr()) % 16) return;
    // the scales are read up to the next multiple of 16
    if (B != room && (size_t)(s.storage_offset() + (R - 1) * lds + room) > s.storage().nbytes()) return;
    ok = true;
  }
};

bool whole(PyObject* o, int64_t& v) {
  v = PyLong_AsLongLong(o);
  return !(v == -1 && PyErr_Occurred());
}
bool address(PyObject* o, void*& p) {
  p = nullptr;
  if (!PyLong_Check(o)) {
    PyErr_SetString(PyExc_TypeError, "a stream is a whole number");
    return false;
  }
  p = PyLong_AsVoidPtr(o);
  return p || !PyErr_Occurred();
}
bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments are needed, not %zd", want, n);
  return n == want;
}

// f's status, without the interpreter's lock: allocating may wait for the device, and so may a launch
// behind many others. (The caller holds the tensors meanwhile.)
template <typename F>
int unlocked(F f) {
  struct Free {
    PyThreadState* held = PyEval_SaveThread();
    ~Free() { PyEval_RestoreThread(held); }  // before an exception reaches the handlers, too
  } free;
  return f();
}

PyObject* answer(int status, std::initializer_list<at::Tensor> out) {
  if (status != SFFN_OK) return PyLong_FromLong(status);
  if (out.size() == 1) return THPVariable_Wrap(*out.begin());
  PyObject* t = PyTuple_New((Py_ssize_t)out.size());
  if (!t) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& o : out) {
    PyObject* p = THPVariable_Wrap(o);
    if (!p) {
      Py_DECREF(t);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, i++, p);
  }
  return t;
}

// codes and scales of [..., K], and the scales' row distance
struct NewBlocks {
  at::Tensor q, s, room;  // room: the scales with what lies behind their rows
  int64_t ldq = 0, lds = 0;
  void make(const at::Tensor& like, int64_t K) {
    const int64_t B = (K + 31) / 32;
    ldq = 16 * B;
    lds = (B + 15) / 16 * 16;
    c10::SmallVector<int64_t, 5> shape(like.sizes().begin(), like.sizes().end());
    const auto bytes = like.options().dtype(at::kByte);
    shape.back() = ldq;
    q = at::empty(shape, bytes);
    shape.back() = lds;
    s = at::empty(shape, bytes);
    room = s;
    if (lds != B) s = room.narrow(-1, 0, B);
  }
};

// norm(x, weight, residual, eps, out, residual_out, device, stream)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t out, dev;
  void* stream;
  if (!count(n, 8) || !whole(a[4], out) || !whole(a[6], dev) || !address(a[7], stream)) return nullptr;
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  const at::Tensor* x = tensor(a[0], dev);
  if (!x) Py_RETURN_NONE;
  const int xt = type_of(*x);
  const Rows r(*x);
  if (xt < 0 || !r.ok) Py_RETURN_NONE;
  if (out < 0) out = xt;
  const void* w = nullptr;
  int wt = 0;
  if (a[1] != Py_None) {
    const at::Tensor* t = tensor(a[1], dev);
    if (!t || t->dim() != 1 || t->size(0) != r.K || !t->is_contiguous() || (wt = type_of(*t)) < 0) Py_RETURN_NONE;
    w = t->data_ptr();
  }
  const at::Tensor *res = nullptr, *into = nullptr;
  int64_t ldr = r.K, ldsum = r.K;
  if (a[2] != Py_None) {
    res = tensor(a[2], dev);
    if (!res || res->scalar_type() != x->scalar_type() || res->sizes() != x->sizes()) Py_RETURN_NONE;
    const Rows q(*res);
    if (!q.ok) Py_RETURN_NONE;
    ldr = q.ld;
  }
  if (a[5] != Py_None) {
    into = tensor(a[5], dev);
    if (!res || !into || into->scalar_type() != x->scalar_type() || into->sizes() != x->sizes()) Py_RETURN_NONE;
    const Rows q(*into);
    if (!q.ok) Py_RETURN_NONE;
    ldsum = q.ld;
  }
  if (out > SFFN_MX4) Py_RETURN_NONE;
  at::Tensor sum, y, s;
  NewBlocks b;
  const int st = unlocked([&]() -> int {
    if (into) sum = *into;
    else if (res) sum = at::empty(x->sizes(), x->options());
    void *yp, *sp = nullptr;
    int64_t ldy = r.K;
    if (out == SFFN_MX4) {
      b.make(*x, r.K);
      yp = b.q.data_ptr();
      sp = b.room.data_ptr();
      ldy = b.ldq;
    } else if (out == SFFN_I8) {
      c10::SmallVector<int64_t, 5> shape(x->sizes().begin(), x->sizes().end());
      ldy = (r.K + 15) / 16 * 16;
      shape.back() = ldy;
      y = at::empty(shape, x->options().dtype(at::kChar));
      shape.pop_back();
      s = at::empty(shape, x->options().dtype(at::kFloat));
      yp = y.data_ptr();
      sp = s.data_ptr();
      if (ldy != r.K) y = y.narrow(-1, 0, r.K);
    } else {
      y = at::empty(x->sizes(), x->options().dtype(type_for((int)out)));
      yp = y.data_ptr();
    }
    return c_norm(x->data_ptr(), xt, r.ld, res ? res->data_ptr() : nullptr, ldr, (int)r.R, (int)r.K, w, wt, eps,
                  res ? sum.data_ptr() : nullptr, ldsum, yp, (int)out, ldy, sp, b.lds, stream);
  });
  if (out == SFFN_MX4) return res ? answer(st, {b.q, b.s, sum}) : answer(st, {b.q, b.s});
  if (out == SFFN_I8) return res ? answer(st, {y, s, sum}) : answer(st, {y, s});
  return res ? answer(st, {y, sum}) : answer(st, {y});
  END_HANDLE_TH_ERRORS
}

// quantize(x, device, stream)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t dev;
  void* stream;
  if (!count(n, 3) || !whole(a[1], dev) || !address(a[2], stream)) return nullptr;
  const at::Tensor* x = tensor(a[0], dev);
  if (!x) Py_RETURN_NONE;
  const int xt = type_of(*x);
  const Rows r(*x);
  if (xt < 0 || !r.ok) Py_RETURN_NONE;
  NewBlocks b;
  const int st = unlocked([&]() -> int {
    b.make(*x, r.K);
    return c_quantize(x->data_ptr(), xt, r.ld, (int)r.R, (int)r.K, static_cast<uint8_t*>(b.q.data_ptr()), b.ldq,
                      static_cast<uint8_t*>(b.room.data_ptr()), b.lds, stream);
  });
  return answer(st, {b.q, b.s});
  END_HANDLE_TH_ERRORS
}

// dequantize(q, scale, cols, out, device, stream): two-dimensional rows; cols None: all
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t cols = 0, out, dev;
  void* stream;
  if (!count(n, 6) || !whole(a[3], out) || !whole(a[4], dev) || !address(a[5], stream)) return nullptr;
  if (a[2] != Py_None && !whole(a[2], cols)) {
    if (!PyErr_ExceptionMatches(PyExc_OverflowError)) return nullptr;
    PyErr_Clear();  // more than any blocks hold
    Py_RETURN_NONE;
  }
  const at::Tensor *q = tensor(a[0], dev), *s = tensor(a[1], dev);
  if (!q || !s || out < 0 || out > SFFN_BF16) Py_RETURN_NONE;
  const Blocks b(*q, *s);
  if (!b.ok) Py_RETURN_NONE;
  if (a[2] == Py_None) cols = 32 * b.B;
  if (cols <= 32 * (b.B - 1) || cols > 32 * b.B) Py_RETURN_NONE;
  at::Tensor y;
  const int st = unlocked([&]() -> int {
    y = at::empty({b.R, cols}, q->options().dtype(type_for((int)out)));
    return c_dequantize(static_cast<const uint8_t*>(q->data_ptr()), b.ldq,
                        static_cast<const uint8_t*>(s->data_ptr()), b.lds, (int)b.R, (int)cols, y.data_ptr(),
                        (int)out, cols, stream);
  });
  return answer(st, {y});
  END_HANDLE_TH_ERRORS
}

// matmul(x, w, w_scale, x_scale, bias, out, device, stream): y and scratch allocated here
PyObject* matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t out, dev;
  void* stream;
  if (!count(n, 8) || !whole(a[5], out) || !whole(a[6], dev) || !address(a[7], stream)) return nullptr;
  const at::Tensor *x = tensor(a[0], dev), *w = tensor(a[1], dev), *ws = tensor(a[2], dev);
  if (!x || !w || !ws || x->dim() != 2) Py_RETURN_NONE;
  const Blocks bw(*w, *ws);
  if (!bw.ok) Py_RETURN_NONE;
  int xt;
  int64_t M, K, ldx, ldxs = 0;
  const uint8_t* xs = nullptr;
  if (a[3] != Py_None) {
    const at::Tensor* s = tensor(a[3], dev);
    if (!s) Py_RETURN_NONE;
    const Blocks b(*x, *s);
    if (!b.ok || b.B != bw.B) Py_RETURN_NONE;
    xt = SFFN_MX4;
    M = b.R;
    K = 32 * b.B;
    ldx = b.ldq;
    ldxs = b.lds;
    xs = static_cast<const uint8_t*>(s->data_ptr());
    if (out < 0) out = SFFN_F32;
  } else {
    xt = type_of(*x);
    const Rows r(*x);
    if (xt < 0 || !r.ok || (r.K + 31) / 32 != bw.B) Py_RETURN_NONE;
    M = r.R;
    K = r.K;
    ldx = r.ld;
    if (out < 0) out = xt;
  }
  if (out > SFFN_BF16) Py_RETURN_NONE;
  const float* bias = nullptr;
  if (a[4] != Py_None) {
    const at::Tensor* t = tensor(a[4], dev);
    if (!t || t->scalar_type() != at::kFloat || t->dim() != 1 || t->size(0) != bw.R || !t->is_contiguous())
      Py_RETURN_NONE;
    bias = static_cast<const float*>(t->data_ptr());
  }
  const size_t need = c_work_bytes(xt, (int)M, (int)bw.R, (int)K);
  if (need > ((size_t)1 << 62)) Py_RETURN_NONE;
  at::Tensor y, work;
  const int st = unlocked([&]() -> int {
    y = at::empty({M, bw.R}, x->options().dtype(type_for((int)out)));
    if (need) work = at::empty({(int64_t)need}, x->options().dtype(at::kByte));
    return c_matmul(x->data_ptr(), xt, xs, ldx, ldxs, (int)M, (int)K, static_cast<const uint8_t*>(w->data_ptr()),
                    bw.ldq, static_cast<const uint8_t*>(ws->data_ptr()), bw.lds, bias, (int)bw.R, y.data_ptr(),
                    (int)out, bw.R, need ? work.data_ptr() : nullptr, need, stream);
  });
  return answer(st, {y});
  END_HANDLE_TH_ERRORS
}

// bind(norm, quantize, dequantize, matmul_work_bytes, matmul): the C entry points' addresses
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 5)) return nullptr;
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) return PyErr_Occurred() ? nullptr : (PyErr_SetString(PyExc_ValueError, "null address"), nullptr);
  }
  c_norm = reinterpret_cast<decltype(c_norm)>(p[0]);
  c_quantize = reinterpret_cast<decltype(c_quantize)>(p[1]);
  c_dequantize = reinterpret_cast<decltype(c_dequantize)>(p[2]);
  c_work_bytes = reinterpret_cast<decltype(c_work_bytes)>(p[3]);
  c_matmul = reinterpret_cast<decltype(c_matmul)>(p[4]);
  Py_RETURN_NONE;
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(bind), CALL(norm), CALL(quantize), CALL(dequantize), CALL(matmul),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&module);
  // mx4.py takes the module with that torch only: at::Tensor is another torch's to lay out
  if (m && PyModule_AddStringConstant(m, "built_for", SFFN_TORCH) != 0) Py_CLEAR(m);
  return m;
}
