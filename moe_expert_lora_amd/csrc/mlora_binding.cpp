// CPython binding of the MoE layer's operators (mlora_router_topk and the ones
// behind it in mlora.h): argument marshalling only, as the ctypes binding of
// the folds does it. A decode step makes these calls back to back on small
// tensors, and reading a tensor's type, place and sizes through Python takes
// longer than the call; here they are read from the tensor itself. The package's
// Python functions of the same names, which hold the documentation, call these
// with every argument by position.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "mlora.h"

namespace {

PyObject* g_error = nullptr;  // moe_expert_lora_amd.MloraError

// An argument the binding refuses, as the Python exception it becomes.
struct Refused : std::exception {
  PyObject* type;
  std::string message;
  Refused(PyObject* t, std::string m) : type(t), message(std::move(m)) {}
};

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// The kernels run on the current device's stream: a tensor of another device
// is refused with the host's.
void on_device(const at::Tensor& t, const char* name) {
  if (!t.is_cuda())
    throw Refused(PyExc_ValueError, std::string(name) + " must be a device tensor");
  if (t.device().index() != c10::hip::current_device())
    throw Refused(PyExc_ValueError, std::string(name) + " must be on the current device");
}

int32_t code_of(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MLORA_BF16;
    case at::kFloat: return MLORA_F32;
    default: throw Refused(PyExc_TypeError, std::string(name) + ": unsupported dtype");
  }
}

// A contiguous tensor of one dtype.
struct Vec {
  void* p = nullptr;
  int64_t n = 0;
  Vec() = default;
  Vec(PyObject* o, const char* name, at::ScalarType type, bool may_be_none = false) {
    if (may_be_none && o == Py_None) return;
    const at::Tensor& t = tensor(o, name);
    on_device(t, name);
    if (!t.is_contiguous())
      throw Refused(PyExc_ValueError, std::string(name) + " must be contiguous");
    if (t.scalar_type() != type)
      throw Refused(PyExc_TypeError, std::string(name) + " must be " + at::toString(type));
    p = t.data_ptr();
    n = t.numel();
  }
};

// A 2-D tensor with contiguous rows (a column slice of a wider one is fine).
struct Mat {
  void* p;
  int64_t rows, cols, ld;
  int32_t dtype;
  Mat(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    on_device(t, name);
    if (t.dim() != 2) throw Refused(PyExc_ValueError, std::string(name) + " must be 2-D");
    dtype = code_of(t, name);
    rows = t.size(0);
    cols = t.size(1);
    if (rows > 0 && cols > 1 && t.stride(1) != 1)
      throw Refused(PyExc_ValueError, std::string(name) + " must have contiguous rows");
    ld = rows > 1 ? t.stride(0) : cols;
    p = t.data_ptr();
  }
};

void require(bool ok, const char* what) {
  if (!ok) throw Refused(PyExc_ValueError, what);
}
void same_type(const Mat& a, const Mat& b, const char* what) {
  if (a.dtype != b.dtype) throw Refused(PyExc_TypeError, what);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused(nullptr, "");  // the error is set
  return v;
}
int32_t integer32(PyObject* o) {
  const int64_t v = integer(o);
  if (v != (int32_t)v) throw Refused(PyExc_ValueError, "integer argument out of range");
  return (int32_t)v;
}
// A size of a tensor that the library takes in 32 bits.
int32_t size32(int64_t v, const char* name) {
  if (v != (int32_t)v) throw Refused(PyExc_ValueError, std::string(name) + " is too wide");
  return (int32_t)v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused(nullptr, "");
  return v != 0;
}

// The stream's handle; None: the current one.
void* stream_of(PyObject* o) {
  if (o == Py_None) return c10::hip::getCurrentHIPStream().stream();
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw Refused(nullptr, "");
  void* s = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (PyErr_Occurred()) throw Refused(nullptr, "");
  return s;
}

PyObject* done(int32_t rc) {
  if (rc == MLORA_OK) Py_RETURN_NONE;
  PyObject* e = PyObject_CallFunction(g_error, "is", (int)rc, mlora_last_error());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

// Runs a call's body; no C++ exception passes into Python.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F body) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", got, want);
    return nullptr;
  }
  try {
    return done(body());
  } catch (const Refused& r) {
    if (r.type) PyErr_SetString(r.type, r.message.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

typedef PyObject* const* Args;

// logits, indices, weights, renormalize, stream
PyObject* router_topk(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 5, [&] {
    const Mat lg(a[0], "logits");
    const at::Tensor& it = tensor(a[1], "indices");
    require(it.dim() == 2 && it.size(0) == lg.rows && it.sizes() == tensor(a[2], "weights").sizes(),
            "indices and weights must be [n_tokens, top_k]");
    const Vec idx(a[1], "indices", at::kInt), w(a[2], "weights", at::kFloat);
    return mlora_router_topk(lg.p, lg.ld, lg.dtype, lg.rows, size32(lg.cols, "logits"),
                             size32(it.size(1), "indices"), truth(a[3]), (int32_t*)idx.p, (float*)w.p,
                             stream_of(a[4]));
  });
}

// logits, indices, d_weights, d_logits, renormalize, stream
PyObject* router_topk_backward(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const Mat lg(a[0], "logits"), dl(a[3], "d_logits");
    same_type(lg, dl, "d_logits dtype differs from logits'");
    require(dl.rows == lg.rows && dl.cols == lg.cols, "d_logits must have the shape of logits");
    const at::Tensor& it = tensor(a[1], "indices");
    require(it.dim() == 2 && it.size(0) == lg.rows &&
                it.sizes() == tensor(a[2], "d_weights").sizes(),
            "indices and d_weights must be [n_tokens, top_k]");
    const Vec idx(a[1], "indices", at::kInt), dw(a[2], "d_weights", at::kFloat);
    return mlora_router_topk_backward(lg.p, lg.ld, lg.dtype, lg.rows,
                                      size32(lg.cols, "logits"), size32(it.size(1), "indices"),
                                      truth(a[4]), (const int32_t*)idx.p,
                                      (const float*)dw.p, dl.p, dl.ld, stream_of(a[5]));
  });
}

// ids, n_experts, expert_offsets, sorted_ids, slot_rows, workspace, stream
PyObject* moe_sort(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const Vec ids(a[0], "ids", at::kInt), off(a[2], "expert_offsets", at::kInt);
    const Vec order(a[3], "sorted_ids", at::kInt), rows(a[4], "slot_rows", at::kInt);
    const int32_t experts = integer32(a[1]);
    require(off.n == (int64_t)experts + 1, "expert_offsets must have n_experts + 1 entries");
    require(order.n == ids.n && rows.n == ids.n,
            "sorted_ids and slot_rows must have one entry per id");
    void* ws = nullptr;
    uint64_t bytes = 0;
    if (a[5] != Py_None) {
      const at::Tensor& t = tensor(a[5], "workspace");
      bytes = (uint64_t)t.numel() * t.element_size();
      if (bytes) {
        on_device(t, "workspace");
        require(t.is_contiguous(), "workspace must be contiguous");
        ws = t.data_ptr();
      }
    }
    return mlora_moe_sort((const int32_t*)ids.p, ids.n, experts, (int32_t*)off.p,
                          (int32_t*)order.p, (int32_t*)rows.p, ws, bytes, stream_of(a[6]));
  });
}

// x, rows, sorted_ids, slot_rows, top_k, stream
PyObject* moe_dispatch(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const Mat x(a[0], "x"), rows(a[1], "rows");
    const int32_t k = integer32(a[4]);
    same_type(x, rows, "rows dtype differs from x's");
    require(rows.cols == x.cols && rows.rows == x.rows * k, "rows must be [n_tokens * top_k, dim]");
    const Vec order(a[2], "sorted_ids", at::kInt), slots(a[3], "slot_rows", at::kInt);
    require(order.n == rows.rows && slots.n == rows.rows,
            "sorted_ids and slot_rows must have one entry per row");
    return mlora_moe_dispatch(x.p, x.ld, x.dtype, x.rows, x.cols, k, (const int32_t*)order.p,
                              (const int32_t*)slots.p, rows.p, rows.ld, stream_of(a[5]));
  });
}

// rows, out, top_k, weights, slot_rows, stream
PyObject* moe_combine(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const Mat rows(a[0], "rows"), out(a[1], "out");
    const int32_t k = integer32(a[2]);
    same_type(rows, out, "out dtype differs from rows'");
    require(rows.cols == out.cols, "rows and out differ in width");
    const Vec w(a[3], "weights", at::kFloat, true), slots(a[4], "slot_rows", at::kInt, true);
    require((a[3] == Py_None || w.n == out.rows * k) && (a[4] == Py_None || slots.n == out.rows * k),
            "weights and slot_rows must have n_tokens * top_k entries");
    return mlora_moe_combine(rows.p, rows.ld, rows.rows, rows.dtype, out.rows, out.cols, k,
                             (const float*)w.p, (const int32_t*)slots.p, out.p, out.ld,
                             stream_of(a[5]));
  });
}

// d_out, rows, weights, d_rows, d_weights, top_k, slot_rows, sorted_ids, stream
PyObject* moe_combine_backward(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    const Mat dout(a[0], "d_out"), drows(a[3], "d_rows");
    const int32_t k = integer32(a[5]);
    same_type(dout, drows, "d_rows dtype differs from d_out's");
    require(drows.cols == dout.cols && drows.rows == dout.rows * k,
            "d_rows must be [n_tokens * top_k, dim]");
    const Vec w(a[2], "weights", at::kFloat, true), dw(a[4], "d_weights", at::kFloat, true);
    const Vec slots(a[6], "slot_rows", at::kInt, true), order(a[7], "sorted_ids", at::kInt, true);
    const char* per_row = "weights, d_weights and the maps must have one entry per row";
    require(a[2] == Py_None || w.n == drows.rows, per_row);
    require(a[4] == Py_None || dw.n == drows.rows, per_row);
    require(a[6] == Py_None || slots.n == drows.rows, per_row);
    require(a[7] == Py_None || order.n == drows.rows, per_row);
    const void* rp = nullptr;
    int64_t r_ld = 0;
    if (a[4] != Py_None) {
      const Mat rows(a[1], "rows");
      same_type(dout, rows, "rows dtype differs from d_out's");
      require(rows.cols == dout.cols && rows.rows == drows.rows,
              "rows must have the shape of d_rows");
      rp = rows.p;
      r_ld = rows.ld;
    }
    return mlora_moe_combine_backward(dout.p, dout.ld, rp, r_ld, dout.dtype, dout.rows, dout.cols,
                                      k, (const float*)w.p, (const int32_t*)slots.p,
                                      (const int32_t*)order.p, drows.p, drows.ld, (float*)dw.p,
                                      stream_of(a[8]));
  });
}

// route's address, x, out, ids, top_k, x_by_row, stream
PyObject* w4_gather_gemv(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const mlora_w4_route* route = (const mlora_w4_route*)PyLong_AsVoidPtr(a[0]);
    if (PyErr_Occurred()) throw Refused(nullptr, "");
    const Mat x(a[1], "x"), out(a[2], "out");
    if (x.dtype != route->dtype || out.dtype != route->dtype)
      throw Refused(PyExc_TypeError, "x / out dtype differs from the route's");
    require(x.cols == route->k_in && out.cols == route->n_out,
            "x / out widths differ from the route's k_in / n_out");
    const Vec ids(a[3], "ids", at::kInt, true);
    require(a[3] == Py_None || ids.n == out.rows, "ids must have one entry per out row");
    // an ids tensor without entries still says that the rows have experts
    static const int32_t kNone = 0;
    const int32_t* ip = a[3] == Py_None ? nullptr : ids.p ? (const int32_t*)ids.p : &kNone;
    return mlora_w4_gather_gemv(route, x.p, x.rows, x.ld, truth(a[5]), out.p, out.ld, ip, out.rows,
                                integer32(a[4]), stream_of(a[6]));
  });
}

// The class of the exceptions that failing calls raise.
PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

#define MLORA_FAST(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {MLORA_FAST(router_topk),
                          MLORA_FAST(router_topk_backward),
                          MLORA_FAST(moe_sort),
                          MLORA_FAST(moe_dispatch),
                          MLORA_FAST(moe_combine),
                          MLORA_FAST(moe_combine_backward),
                          MLORA_FAST(w4_gather_gemv),
                          {"set_error", set_error, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&kModule); }
