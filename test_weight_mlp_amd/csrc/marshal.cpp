// Argument marshalling of the attention half's binding: tensors are checked
// against the problem and handed to the C ABI.  A single token's norm and rotation
// takes the device 3.5 us; looking at its eight tensors from Python took 5 us,
// here it takes a fraction of one.
//
// The library's entry points are given by address (bind), so that this module
// works with whichever build of libipttt.so the package loads.  Every call returns
// the entry's status; a tensor that does not fit raises ValueError.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <c10/util/StringUtil.h>

#include <exception>

#include "../../include/ipttt.h"

namespace {

decltype(&ipttt_qk_norm_rope) g_qk;
decltype(&ipttt_qk_norm_rope_backward) g_qk_bwd;
decltype(&ipttt_attention) g_attn;
decltype(&ipttt_attention_backward) g_attn_bwd;

at::ScalarType type_of(int32_t dtype) { return dtype == IPTTT_BF16 ? at::kBFloat16 : at::kFloat; }

const at::Tensor* tensor(PyObject* o, const char* what) {
  if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
  PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
  return nullptr;
}

// The arguments of one call, read in order; ok() is false, with a Python error
// set, once one of them did not fit.  All tensors of a call are on the device of
// its first.
class Reader {
 public:
  Reader(PyObject* const* args, int32_t dtype) : args_(args), dtype_(dtype) {}
  bool ok() const { return ok_; }

  // [rows, heads, D] of the problem's type, any strides but the last
  void heads(const char* what, int64_t rows, int64_t heads, int64_t dim, ipttt_heads* h) {
    const at::Tensor* t = next(what);
    if (t == nullptr) return;
    if (t->dim() != 3 || t->size(0) != rows || t->size(1) != heads || t->size(2) != dim ||
        t->scalar_type() != type_of(dtype_) || !t->is_cuda() || t->stride(2) != 1) {
      fail(*t, what, " device tensor with a contiguous last dimension", {rows, heads, dim}, type_of(dtype_));
      return;
    }
    if (!here(*t, what)) return;
    *h = ipttt_heads{t->data_ptr(), t->stride(0), t->stride(1)};
  }
  // the same, or None
  const ipttt_heads* maybe_heads(const char* what, int64_t rows, int64_t n, int64_t dim, ipttt_heads* h) {
    if (!ok_ || *args_ == Py_None) {
      ++args_;
      return nullptr;
    }
    heads(what, rows, n, dim, h);
    return h;
  }
  // contiguous [a] (b = 0) or [a, b]
  void* flat(const char* what, int64_t a, int64_t b, at::ScalarType type) {
    const at::Tensor* t = next(what);
    if (t == nullptr) return nullptr;
    if (t->dim() != (b == 0 ? 1 : 2) || t->size(0) != a || (b != 0 && t->size(1) != b) || t->scalar_type() != type ||
        !t->is_cuda() || !t->is_contiguous()) {
      const int64_t shape[2] = {a, b};
      fail(*t, what, " contiguous device tensor", {shape, b == 0 ? 1u : 2u}, type);
      return nullptr;
    }
    return here(*t, what) ? t->data_ptr() : nullptr;
  }
  void* maybe_flat(const char* what, int64_t a, at::ScalarType type) {
    if (!ok_ || *args_ == Py_None) {
      ++args_;
      return nullptr;
    }
    return flat(what, a, 0, type);
  }
  // the plan's copy on the device
  const void* plan_table() {
    const at::Tensor* t = next("the plan's table");
    if (t == nullptr) return nullptr;
    if (!t->is_cuda() || !t->is_contiguous()) {
      PyErr_SetString(PyExc_ValueError,
                      c10::str("the plan's table must be a contiguous device tensor, not on ", t->device(),
                               ": build the plan with the device of the call's tensors")
                          .c_str());
      ok_ = false;
      return nullptr;
    }
    return here(*t, "the plan's table") ? t->data_ptr() : nullptr;
  }
  // a workspace: None or any contiguous device tensor
  void* workspace(size_t* bytes) {
    *bytes = 0;
    if (!ok_ || *args_ == Py_None) {
      ++args_;
      return nullptr;
    }
    const at::Tensor* t = next("ws");
    if (t == nullptr) return nullptr;
    if (!t->is_cuda() || !t->is_contiguous()) {
      PyErr_SetString(PyExc_ValueError, "ws must be a contiguous device tensor");
      ok_ = false;
      return nullptr;
    }
    if (!here(*t, "ws")) return nullptr;
    *bytes = t->nbytes();
    return t->data_ptr();
  }

 private:
  const at::Tensor* next(const char* what) {
    PyObject* o = *args_++;
    if (!ok_) return nullptr;
    const at::Tensor* t = tensor(o, what);
    ok_ = t != nullptr;
    return t;
  }
  bool here(const at::Tensor& t, const char* what) {
    const auto device = t.get_device();
    if (device_ < 0) device_ = device;
    if (device == device_) return true;
    PyErr_SetString(PyExc_ValueError,
                    c10::str(what, " must be on device ", (int)device_, " like the call's first tensor, not on ", t.device())
                        .c_str());
    ok_ = false;
    return false;
  }
  void fail(const at::Tensor& t, const char* what, const char* kind, at::IntArrayRef shape, at::ScalarType type) {
    PyErr_SetString(PyExc_ValueError,
                    c10::str(what, " must be a ", shape, " ", type, kind, ", not ", t.sizes(), " ", t.scalar_type(),
                             " of strides ", t.strides(), " on ", t.device())
                        .c_str());
    ok_ = false;
  }
  PyObject* const* args_;
  int32_t dtype_;
  int64_t device_ = -1;
  bool ok_ = true;
};

template <class T>
T* pointer(PyObject* o) {
  return static_cast<T*>(PyLong_AsVoidPtr(o));
}

bool arity(Py_ssize_t n, Py_ssize_t want, const void* fn) {
  if (fn == nullptr) PyErr_SetString(PyExc_RuntimeError, "bind() first");
  else if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
  return fn != nullptr && n == want;
}

// Runs an entry without the interpreter's lock; no C++ exception leaves.
template <class F>
PyObject* call(F&& f) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// qk(problem address, q, k, w_q, w_k, positions, table, q_out, k_out, v, v_out, rows, stream)
PyObject* qk(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!arity(n, 13, reinterpret_cast<const void*>(g_qk))) return nullptr;
    const ipttt_qk_problem* p = pointer<const ipttt_qk_problem>(a[0]);
    if (p == nullptr) return nullptr;
    const int64_t D = p->head_dim;
    Reader r(a + 1, p->dtype);
    ipttt_heads q, k, qo, ko, v, vo;
    r.heads("q", p->tokens, p->heads, D, &q);
    r.heads("k", p->tokens, p->kv_heads, D, &k);
    const void* wq = r.flat("w_q", D, 0, type_of(p->dtype));
    const void* wk = r.flat("w_k", D, 0, type_of(p->dtype));
    const void* pos = r.flat("positions", p->tokens, 0, at::kInt);
    const void* table = r.flat("table", p->table_rows, D, at::kFloat);
    r.heads("q_out", p->tokens, p->heads, D, &qo);
    r.heads("k_out", p->out_rows, p->kv_heads, D, &ko);
    const ipttt_heads* pv = r.maybe_heads("v", p->tokens, p->kv_heads, D, &v);
    const ipttt_heads* pvo = r.maybe_heads("v_out", p->out_rows, p->kv_heads, D, &vo);
    const void* rows = r.maybe_flat("rows", p->tokens, at::kInt);
    if (!r.ok()) return nullptr;
    void* stream = pointer<void>(a[12]);
    return call([&] {
      return g_qk(p, &q, &k, wq, wk, static_cast<const int32_t*>(pos), static_cast<const float*>(table), &qo, &ko, pv,
                  pvo, static_cast<const int32_t*>(rows), stream);
    });
  });
}

// qk_backward(problem address, q, k, w_q, w_k, positions, table, dq_out, dk_out, dq, dk, dw_q, dw_k, ws, stream)
PyObject* qk_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!arity(n, 15, reinterpret_cast<const void*>(g_qk_bwd))) return nullptr;
    const ipttt_qk_problem* p = pointer<const ipttt_qk_problem>(a[0]);
    if (p == nullptr) return nullptr;
    const int64_t D = p->head_dim;
    Reader r(a + 1, p->dtype);
    ipttt_heads q, k, dqo, dko, dq, dk;
    r.heads("q", p->tokens, p->heads, D, &q);
    r.heads("k", p->tokens, p->kv_heads, D, &k);
    const void* wq = r.flat("w_q", D, 0, type_of(p->dtype));
    const void* wk = r.flat("w_k", D, 0, type_of(p->dtype));
    const void* pos = r.flat("positions", p->tokens, 0, at::kInt);
    const void* table = r.flat("table", p->table_rows, D, at::kFloat);
    r.heads("dq_out", p->tokens, p->heads, D, &dqo);
    r.heads("dk_out", p->tokens, p->kv_heads, D, &dko);
    r.heads("dq", p->tokens, p->heads, D, &dq);
    r.heads("dk", p->tokens, p->kv_heads, D, &dk);
    void* dwq = r.flat("dw_q", D, 0, at::kFloat);
    void* dwk = r.flat("dw_k", D, 0, at::kFloat);
    size_t bytes;
    void* ws = r.workspace(&bytes);
    if (!r.ok()) return nullptr;
    void* stream = pointer<void>(a[14]);
    return call([&] {
      return g_qk_bwd(p, &q, &k, wq, wk, static_cast<const int32_t*>(pos), static_cast<const float*>(table), &dqo,
                      &dko, &dq, &dk, static_cast<float*>(dwq), static_cast<float*>(dwk), ws, bytes, stream);
    });
  });
}

// attention(problem address, plan address, scale, plan table, q, k, v, o, lse, ws, stream)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!arity(n, 11, reinterpret_cast<const void*>(g_attn))) return nullptr;
    const ipttt_attn_problem* p = pointer<const ipttt_attn_problem>(a[0]);
    const void* plan = pointer<void>(a[1]);
    const float scale = (float)PyFloat_AsDouble(a[2]);
    if (p == nullptr || PyErr_Occurred() != nullptr) return nullptr;
    Reader r(a + 3, p->dtype);
    const void* dev = r.plan_table();
    ipttt_heads q, k, v, o;
    r.heads("q", p->q_rows, p->heads, p->head_dim, &q);
    r.heads("k", p->k_rows, p->kv_heads, p->head_dim, &k);
    r.heads("v", p->k_rows, p->kv_heads, p->head_dim, &v);
    r.heads("o", p->q_rows, p->heads, p->head_dim, &o);
    void* lse = r.flat("lse", p->q_rows, p->heads, at::kFloat);
    size_t bytes;
    void* ws = r.workspace(&bytes);
    if (!r.ok()) return nullptr;
    void* stream = pointer<void>(a[10]);
    return call([&] {
      return g_attn(plan, dev, scale, &q, &k, &v, &o, static_cast<float*>(lse), ws, bytes, stream);
    });
  });
}

// attention_backward(problem address, plan address, scale, plan table, q, k, v, o, lse, dO, dq, dk, dv, ws, stream)
PyObject* attention_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!arity(n, 15, reinterpret_cast<const void*>(g_attn_bwd))) return nullptr;
    const ipttt_attn_problem* p = pointer<const ipttt_attn_problem>(a[0]);
    const void* plan = pointer<void>(a[1]);
    const float scale = (float)PyFloat_AsDouble(a[2]);
    if (p == nullptr || PyErr_Occurred() != nullptr) return nullptr;
    Reader r(a + 3, p->dtype);
    const void* dev = r.plan_table();
    ipttt_heads q, k, v, o, dO, dq, dk, dv;
    r.heads("q", p->q_rows, p->heads, p->head_dim, &q);
    r.heads("k", p->k_rows, p->kv_heads, p->head_dim, &k);
    r.heads("v", p->k_rows, p->kv_heads, p->head_dim, &v);
    r.heads("o", p->q_rows, p->heads, p->head_dim, &o);
    const void* lse = r.flat("lse", p->q_rows, p->heads, at::kFloat);
    r.heads("dO", p->q_rows, p->heads, p->head_dim, &dO);
    r.heads("dq", p->q_rows, p->heads, p->head_dim, &dq);
    r.heads("dk", p->k_rows, p->kv_heads, p->head_dim, &dk);
    r.heads("dv", p->k_rows, p->kv_heads, p->head_dim, &dv);
    size_t bytes;
    void* ws = r.workspace(&bytes);
    if (!r.ok()) return nullptr;
    void* stream = pointer<void>(a[14]);
    return call([&] {
      return g_attn_bwd(plan, dev, scale, &q, &k, &v, &o, static_cast<const float*>(lse), &dO, &dq, &dk, &dv, ws,
                        bytes, stream);
    });
  });
}

// bind(qk, qk_backward, attention, attention_backward): the entries' addresses
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "four addresses");
    return nullptr;
  }
  void* f[4];
  for (int i = 0; i < 4; ++i) {
    f[i] = pointer<void>(a[i]);
    if (f[i] == nullptr) {
      if (PyErr_Occurred() == nullptr) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  }
  g_qk = reinterpret_cast<decltype(g_qk)>(f[0]);
  g_qk_bwd = reinterpret_cast<decltype(g_qk_bwd)>(f[1]);
  g_attn = reinterpret_cast<decltype(g_attn)>(f[2]);
  g_attn_bwd = reinterpret_cast<decltype(g_attn_bwd)>(f[3]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F));
}

PyMethodDef g_methods[] = {
    {"bind", fast<bind>(), METH_FASTCALL, "the library's entries, by address"},
    {"qk", fast<qk>(), METH_FASTCALL, "ipttt_qk_norm_rope"},
    {"qk_backward", fast<qk_backward>(), METH_FASTCALL, "ipttt_qk_norm_rope_backward"},
    {"attention", fast<attention>(), METH_FASTCALL, "ipttt_attention"},
    {"attention_backward", fast<attention_backward>(), METH_FASTCALL, "ipttt_attention_backward"},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", "argument marshalling of the attention half", -1,
                        g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&g_module); }
