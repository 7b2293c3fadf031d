// bind.cpp -- the Python calls of the operators around the layer: argument checks and the
// C call, without ctypes' conversions on the way (a call of moe_route_topk on one token
// spent 7 us of which the launch is 2).
//
// The functions are libmoe.so's, given by address (start), so the debug library works the
// same.  A tensor is checked for its type, element count, contiguity and device; what does
// not pass goes to the checks in _lib.py, which name the tensor and the fault.
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "moe.h"

namespace {

// libmoe.so's entry points, in the order of `names`.
struct Lib {
  decltype(&moe_gate_logits) gate_logits;
  decltype(&moe_route_topk) route_topk;
  decltype(&moe_route_bwd) route_bwd;
  decltype(&moe_gate_bwd) gate_bwd;
  decltype(&moe_block_norm) block_norm;
  decltype(&moe_block_norm_bwd) block_norm_bwd;
  decltype(&moe_grad_norm) grad_norm;
  decltype(&moe_grad_clip) grad_clip;
  decltype(&moe_grad_clip_norm) grad_clip_norm;
} lib;
constexpr int ENTRIES = sizeof(Lib) / sizeof(void*);
PyObject *py_need, *py_kind;  // _lib.py's checks
PyObject* dtypes[5];          // torch's, of the types below
enum { F32, BF16, F16, I32, F64 };
constexpr at::ScalarType TYPES[5] = {at::kFloat, at::kBFloat16, at::kHalf, at::kInt, at::kDouble};

// One call's arguments, taken in order; `ok` falls with the first that does not pass, with
// a Python error set.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, at = 0;
  bool ok = true;
  int dev = 0;

  Args(PyObject* const* args, Py_ssize_t count, Py_ssize_t want) : a(args), n(count) {
    if (count != want) {
      PyErr_Format(PyExc_TypeError, "%zd arguments, %zd needed", count, want);
      ok = false;
    }
  }
  PyObject* next() { return a[at++]; }

  int64_t integer() {
    if (!ok) return 0;
    PyObject* o = PyNumber_Index(next());
    const long long v = o ? PyLong_AsLongLong(o) : -1;
    Py_XDECREF(o);
    if (v == -1 && PyErr_Occurred()) ok = false;
    return v;
  }
  double number() {
    if (!ok) return 0;
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) ok = false;
    return v;
  }
  // A ctypes structure; it outlives the call, as its argument.
  template <typename T>
  const T* structure() {
    if (!ok) return nullptr;
    Py_buffer b;
    if (PyObject_GetBuffer(next(), &b, PyBUF_SIMPLE) != 0) {
      ok = false;
      return nullptr;
    }
    const T* p = static_cast<const T*>(b.buf);
    const Py_ssize_t size = b.len;
    PyBuffer_Release(&b);
    if (size != (Py_ssize_t)sizeof(T)) {
      PyErr_Format(PyExc_TypeError, "a structure of %zd bytes, %zd needed", size,
                   (Py_ssize_t)sizeof(T));
      ok = false;
    }
    return p;
  }
  static void* address(PyObject* o) { return PyLong_AsVoidPtr(o); }

  // MOE_ type of the tensor at position `i`.
  int kind(const char* what, Py_ssize_t i, int last) {
    if (!ok) return 0;
    if (THPVariable_Check(a[i])) {
      const at::ScalarType t = THPVariable_Unpack(a[i]).scalar_type();
      for (int k = MOE_F32; k <= last; ++k)
        if (t == TYPES[k]) return k;
    }
    PyObject* r = PyObject_CallFunction(py_kind, "sO(iii)", what, a[i], MOE_F32, MOE_BF16,
                                        last >= MOE_F16 ? MOE_F16 : MOE_BF16);
    const int k = r ? (int)PyLong_AsLong(r) : -1;
    Py_XDECREF(r);
    if (PyErr_Occurred()) ok = false;
    return k;
  }
  // Device address of a tensor of `numel` elements of a type; None is NULL, an integer an
  // address.  more: a longer tensor will do.
  void* tensor(const char* what, int type, int64_t numel, bool more = false) {
    if (!ok) return nullptr;
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    if (PyLong_CheckExact(o)) {
      void* p = address(o);
      if (!p && PyErr_Occurred()) ok = false;
      return p;
    }
    if (THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      const int64_t has = t.numel();
      if (t.scalar_type() == TYPES[type] && (has == numel || (more && has > numel)) &&
          t.is_contiguous() && t.get_device() == dev)
        return t.data_ptr();
    }
    PyObject* r = PyObject_CallFunction(py_need, "sOOLi", what, o, dtypes[type], (long long)numel,
                                        dev);
    void* p = r && r != Py_None ? address(r) : nullptr;
    Py_XDECREF(r);
    if (PyErr_Occurred()) ok = false;
    return p;
  }
  // A workspace: address and bytes.
  void* workspace(size_t* bytes) {
    *bytes = 0;
    if (!ok) return nullptr;
    PyObject* o = next();
    if (THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (t.get_device() == dev && t.is_contiguous()) {
        *bytes = t.nbytes();
        return t.data_ptr();
      }
    }
    PyErr_Format(PyExc_ValueError, "ws: a contiguous tensor on cuda:%d is needed", dev);
    ok = false;
    return nullptr;
  }
  // The last two arguments of every call: the device, which the checks need first, and the
  // stream.
  void device() {
    if (!ok) return;
    const Py_ssize_t keep = at;
    at = n - 2;
    dev = (int)integer();
    at = keep;
  }
  void* stream() {
    at = n - 1;
    return reinterpret_cast<void*>(integer());
  }
};

// The call itself, with other Python threads let in; torch's exceptions become Python's.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}
template <typename F>
PyObject* run(Args& a, F f) {
  if (!a.ok) return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f();
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(rc);
}

using Fast = PyObject* const*;

// Sequences of L of T tokens.
int64_t sequences(int64_t T, int64_t L) { return T > 0 ? (T - 1) / L + 1 : 0; }

int64_t gate_rows(const moe_dims* d, const moe_norm_cfg* c) {
  const int64_t r = c->seq_len > 0 ? sequences(d->T, c->seq_len) : 1;
  return r > 1 ? r : 1;
}

// dims, x, wg, logits, ws
PyObject* gate_logits(PyObject*, Fast args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 7);
    a.device();
    const moe_dims* d = a.structure<moe_dims>();
    if (!a.ok) return nullptr;
    void* x = a.tensor("x", BF16, d->T * d->d);
    void* wg = a.tensor("wg", F32, (int64_t)d->E * d->d);
    void* logits = a.tensor("logits", F32, d->T * d->E);
    size_t bytes;
    void* ws = a.workspace(&bytes);
    void* st = a.stream();
    return run(a, [&] {
      return lib.gate_logits(d, x, (float*)wg, (float*)logits, ws, bytes, st);
    });
  });
}

// dims, cfg, logits, bias, topk_idx, topk_w, probs
PyObject* route_topk(PyObject*, Fast args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 9);
    a.device();
    const moe_dims* d = a.structure<moe_dims>();
    const moe_route_cfg* c = a.structure<moe_route_cfg>();
    const int kind = a.kind("logits", 2, MOE_BF16);
    if (!a.ok) return nullptr;
    void* logits = a.tensor("logits", kind, d->T * d->E);
    void* bias = a.tensor("bias", F32, d->E);
    void* idx = a.tensor("topk_idx", I32, d->T * d->k);
    void* w = a.tensor("topk_w", F32, d->T * d->k);
    void* probs = a.tensor("probs", F32, d->T * d->E);
    void* st = a.stream();
    return run(a, [&] {
      return lib.route_topk(d, c, kind, logits, (float*)bias, (int32_t*)idx, (float*)w,
                            (float*)probs, st);
    });
  });
}

// dims, cfg, logits, topk_idx, topk_w, dw, seq_grad, seq_len, dlogits
PyObject* route_bwd(PyObject*, Fast args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 11);
    a.device();
    const moe_dims* d = a.structure<moe_dims>();
    const moe_route_cfg* c = a.structure<moe_route_cfg>();
    const int kind = a.kind("logits", 2, MOE_BF16);
    if (!a.ok) return nullptr;
    a.at = 7;
    const int64_t L = a.integer();
    const bool seq = args[6] != Py_None && L > 0;
    const int64_t rows = seq ? sequences(d->T, L) : 0;
    a.at = 2;
    void* logits = a.tensor("logits", kind, d->T * d->E);
    void* idx = a.tensor("topk_idx", I32, d->T * d->k);
    void* w = a.tensor("topk_w", F32, d->T * d->k);
    void* dw = a.tensor("dw", F32, d->T * d->k);
    // MoEBuffers.bal_grad holds rows for the shortest sequences; without any the C call answers
    void* sg = a.tensor("seq_grad", F32, rows * d->E, true);
    a.at = 8;
    void* dl = a.tensor("dlogits", kind, d->T * d->E);
    void* st = a.stream();
    return run(a, [&] {
      return lib.route_bwd(d, c, kind, logits, (int32_t*)idx, (float*)w, (float*)dw, (float*)sg,
                           L, dl, st);
    });
  });
}

// dims, x, wg, dlogits, dx, dwg, accumulate, ws
PyObject* gate_bwd(PyObject*, Fast args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 10);
    a.device();
    const moe_dims* d = a.structure<moe_dims>();
    if (!a.ok) return nullptr;
    void* x = a.tensor("x", BF16, d->T * d->d);
    void* wg = a.tensor("wg", F32, (int64_t)d->E * d->d);
    void* dl = a.tensor("dlogits", F32, d->T * d->E);
    void* dx = a.tensor("dx", BF16, d->T * d->d);
    void* dwg = a.tensor("dwg", F32, (int64_t)d->E * d->d);
    const int acc = (int)a.integer();
    size_t bytes;
    void* ws = a.workspace(&bytes);
    void* st = a.stream();
    return run(a, [&] {
      return lib.gate_bwd(d, x, (float*)wg, (float*)dl, dx, (float*)dwg, acc, ws, bytes, st);
    });
  });
}

// dims, cfg, y, res, w_post, gate, w_pre, res_out, n
PyObject* block_norm(PyObject*, Fast args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 11);
    a.device();
    const moe_dims* d = a.structure<moe_dims>();
    const moe_norm_cfg* c = a.structure<moe_norm_cfg>();
    const int kind = a.kind("res", 3, MOE_BF16);
    if (!a.ok) return nullptr;
    const int64_t m = d->T * d->d;
    void* y = a.tensor("y", BF16, m);
    void* res = a.tensor("res", kind, m);
    void* w_post = a.tensor("w_post", F32, d->d);
    void* gate = a.tensor("gate", F32, gate_rows(d, c) * d->d);
    void* w_pre = a.tensor("w_pre", F32, d->d);
    void* out = a.tensor("res_out", kind, m);
    void* nn = a.tensor("n", BF16, m);
    void* st = a.stream();
    return run(a, [&] {
      return lib.block_norm(d, c, kind, y, res, (float*)w_post, (float*)gate, (float*)w_pre, out,
                            nn, st);
    });
  });
}

// dims, cfg, dn, dres_out, y, u, w_post, gate, w_pre, dy, dres, dw_post, dgate, dw_pre,
// accumulate, ws
PyObject* block_norm_bwd(PyObject*, Fast args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 18);
    a.device();
    const moe_dims* d = a.structure<moe_dims>();
    const moe_norm_cfg* c = a.structure<moe_norm_cfg>();
    const int kind = a.kind("dres", 10, MOE_BF16);
    if (!a.ok) return nullptr;
    const int64_t m = d->T * d->d, g = gate_rows(d, c) * d->d;
    void* dn = a.tensor("dn", BF16, m);
    void* du = a.tensor("dres_out", kind, m);
    void* y = a.tensor("y", BF16, m);
    void* u = a.tensor("u", kind, m);
    void* w_post = a.tensor("w_post", F32, d->d);
    void* gate = a.tensor("gate", F32, g);
    void* w_pre = a.tensor("w_pre", F32, d->d);
    void* dy = a.tensor("dy", BF16, m);
    void* dres = a.tensor("dres", kind, m);
    void* dw_post = a.tensor("dw_post", F32, d->d);
    void* dgate = a.tensor("dgate", F32, g);
    void* dw_pre = a.tensor("dw_pre", F32, d->d);
    const int acc = (int)a.integer();
    size_t bytes;
    void* ws = a.workspace(&bytes);
    void* st = a.stream();
    return run(a, [&] {
      return lib.block_norm_bwd(d, c, kind, dn, du, y, u, (float*)w_post, (float*)gate,
                                (float*)w_pre, dy, dres, (float*)dw_post, (float*)dgate,
                                (float*)dw_pre, acc, ws, bytes, st);
    });
  });
}

// list address, tensors, accumulate, sumsq, norm, ws
PyObject* grad_norm(PyObject*, Fast args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 8);
    a.device();
    const moe_grad* g = reinterpret_cast<const moe_grad*>(a.integer());
    const int64_t count = a.integer();
    const int acc = (int)a.integer();
    void* sumsq = a.tensor("sumsq", F64, 1);
    void* norm = a.tensor("norm", F32, 1);
    size_t bytes;
    void* ws = a.workspace(&bytes);
    void* st = a.stream();
    return run(a, [&] {
      return lib.grad_norm(g, count, acc, (double*)sumsq, (float*)norm, ws, bytes, st);
    });
  });
}

// list address, tensors, sumsq, max_norm, norm, coef
PyObject* grad_clip(PyObject*, Fast args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 8);
    a.device();
    const moe_grad* g = reinterpret_cast<const moe_grad*>(a.integer());
    const int64_t count = a.integer();
    void* sumsq = a.tensor("sumsq", F64, 1);
    const float most = (float)a.number();
    void* norm = a.tensor("norm", F32, 1);
    void* coef = a.tensor("coef", F32, 1);
    void* st = a.stream();
    return run(a, [&] {
      return lib.grad_clip(g, count, (double*)sumsq, most, (float*)norm, (float*)coef, st);
    });
  });
}

// list address, tensors, max_norm, sumsq, norm, coef, ws
PyObject* grad_clip_norm(PyObject*, Fast args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 9);
    a.device();
    const moe_grad* g = reinterpret_cast<const moe_grad*>(a.integer());
    const int64_t count = a.integer();
    const float most = (float)a.number();
    void* sumsq = a.tensor("sumsq", F64, 1);
    void* norm = a.tensor("norm", F32, 1);
    void* coef = a.tensor("coef", F32, 1);
    size_t bytes;
    void* ws = a.workspace(&bytes);
    void* st = a.stream();
    return run(a, [&] {
      return lib.grad_clip_norm(g, count, most, (double*)sumsq, (float*)norm, (float*)coef, ws,
                                bytes, st);
    });
  });
}

// start(addresses, need, kind, dtypes)
PyObject* start(PyObject*, PyObject* args) {
  PyObject *addresses, *need, *kind, *types;
  if (!PyArg_ParseTuple(args, "O!OOO!", &PyTuple_Type, &addresses, &need, &kind, &PyTuple_Type,
                        &types))
    return nullptr;
  if (PyTuple_GET_SIZE(addresses) != ENTRIES || PyTuple_GET_SIZE(types) != 5) {
    PyErr_Format(PyExc_TypeError, "%d addresses and 5 types are needed", ENTRIES);
    return nullptr;
  }
  void** to = reinterpret_cast<void**>(&lib);
  for (int i = 0; i < ENTRIES; ++i) {
    to[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addresses, i));
    if (PyErr_Occurred()) return nullptr;
  }
  for (int i = 0; i < 5; ++i) Py_XSETREF(dtypes[i], Py_NewRef(PyTuple_GET_ITEM(types, i)));
  Py_XSETREF(py_need, Py_NewRef(need));
  Py_XSETREF(py_kind, Py_NewRef(kind));
  Py_RETURN_NONE;
}

#define FAST(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, "" }
PyMethodDef methods[] = {FAST(gate_logits),
                         FAST(route_topk),
                         FAST(route_bwd),
                         FAST(gate_bwd),
                         FAST(block_norm),
                         FAST(block_norm_bwd),
                         FAST(grad_norm),
                         FAST(grad_clip),
                         FAST(grad_clip_norm),
                         {"start", start, METH_VARARGS, ""},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
