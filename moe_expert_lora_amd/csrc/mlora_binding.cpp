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

// A workspace's memory and size; None: nothing.
struct Space {
  void* p = nullptr;
  uint64_t bytes = 0;
  explicit Space(PyObject* o) {
    if (o == Py_None) return;
    const at::Tensor& t = tensor(o, "workspace");
    bytes = (uint64_t)t.numel() * t.element_size();
    if (!bytes) return;
    on_device(t, "workspace");
    require(t.is_contiguous(), "workspace must be contiguous");
    p = t.data_ptr();
  }
};

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
    const Space ws(a[5]);
    return mlora_moe_sort((const int32_t*)ids.p, ids.n, experts, (int32_t*)off.p,
                          (int32_t*)order.p, (int32_t*)rows.p, ws.p, ws.bytes, stream_of(a[6]));
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

// Bytes of E4M3 codes, 2-D with contiguous rows.
struct Codes {
  uint8_t* p;
  int64_t rows, cols, ld;
  Codes(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    on_device(t, name);
    if (t.scalar_type() != at::kFloat8_e4m3fn && t.scalar_type() != at::kByte)
      throw Refused(PyExc_TypeError, std::string(name) + " must be float8_e4m3fn (or its bytes)");
    if (t.dim() != 2) throw Refused(PyExc_ValueError, std::string(name) + " must be 2-D");
    rows = t.size(0);
    cols = t.size(1);
    if (rows > 0 && cols > 1 && t.stride(1) != 1)
      throw Refused(PyExc_ValueError, std::string(name) + " must have contiguous rows");
    ld = rows > 1 ? t.stride(0) : cols;
    p = static_cast<uint8_t*>(t.data_ptr());
  }
};

// A group's scales of every row: [groups, rows].
float* group_scales(PyObject* o, int64_t k, int64_t rows) {
  const at::Tensor& t = tensor(o, "q_scales");
  const Vec v(o, "q_scales", at::kFloat);
  require(t.dim() == 2 && t.size(0) == (k + 127) / 128 && t.size(1) == rows,
          "q_scales must be [ceil(k / 128), rows of q]");
  return static_cast<float*>(v.p);
}

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused(nullptr, "");
  return (float)v;
}

const mlora_fp8_route* fp8_route(PyObject* o) {
  const void* p = PyLong_AsVoidPtr(o);
  if (PyErr_Occurred()) throw Refused(nullptr, "");
  return static_cast<const mlora_fp8_route*>(p);
}

// x, q, q_scales, up, stream
PyObject* fp8_quant(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 5, [&] {
    const Mat x(a[0], "x");
    const Codes q(a[1], "q");
    const int32_t k = size32(x.cols, "x");
    require(q.rows == x.rows && q.cols == mlora_fp8_row_width(k),
            "q must be [n_rows, mlora_fp8_row_width(k)]");
    float* scales = group_scales(a[2], k, x.rows);
    const void* up = nullptr;
    int64_t up_ld = 0;
    if (a[3] != Py_None) {
      const Mat u(a[3], "up");
      same_type(x, u, "up dtype differs from x's");
      require(u.rows == x.rows && u.cols == x.cols, "up must have the shape of x");
      up = u.p;
      up_ld = u.ld;
    }
    return mlora_fp8_quant(x.p, x.ld, up, up_ld, x.dtype, x.rows, k, q.p, q.ld, scales,
                           stream_of(a[4]));
  });
}

// route's address, q, q_scales, out, expert_offsets, sorted_ids, top_k, stream
PyObject* fp8_gemm(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const mlora_fp8_route* route = fp8_route(a[0]);
    const Codes q(a[1], "q");
    const Mat out(a[3], "out");
    require(q.cols == mlora_fp8_row_width(route->k_in) && out.cols == route->n_out,
            "q / out widths differ from the route's k_in / n_out");
    const float* scales = group_scales(a[2], route->k_in, q.rows);
    const Vec off(a[4], "expert_offsets", at::kInt, true), ids(a[5], "sorted_ids", at::kInt, true);
    require(a[4] == Py_None || off.n == (int64_t)route->n_experts + 1,
            "expert_offsets must have n_experts + 1 entries");
    require(a[5] == Py_None || ids.n == out.rows, "sorted_ids must have one entry per out row");
    // a tensor without entries still says that rows go by it
    static const int32_t kNothing = 0;
    const int32_t* ip = a[5] == Py_None ? nullptr : ids.p ? (const int32_t*)ids.p : &kNothing;
    return mlora_fp8_gemm(route, q.p, q.rows, q.ld, scales, out.p, out.ld, out.dtype, out.rows,
                          (const int32_t*)off.p, ip, integer32(a[6]), stream_of(a[7]));
  });
}

// gate, up, down (addresses), x, logits, out, top_k, workspace, renormalize, indices, weights,
// stream
PyObject* moe_layer(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const mlora_fp8_route *gate = fp8_route(a[0]), *up = fp8_route(a[1]), *down = fp8_route(a[2]);
    const Mat x(a[3], "x"), lg(a[4], "logits"), out(a[5], "out");
    same_type(x, lg, "logits dtype differs from x's");
    same_type(x, out, "out dtype differs from x's");
    require(x.cols == gate->k_in && lg.cols == gate->n_experts && lg.rows == x.rows,
            "x must be [n_tokens, dim] and logits [n_tokens, n_experts]");
    require(out.rows == x.rows && out.cols == x.cols, "out must have the shape of x");
    const int32_t k = integer32(a[6]);
    const Space ws(a[7]);
    const Vec idx(a[9], "indices", at::kInt, true), w(a[10], "weights", at::kFloat, true);
    require((a[9] == Py_None || idx.n == x.rows * k) && (a[10] == Py_None || w.n == x.rows * k),
            "indices and weights must be [n_tokens, top_k]");
    return mlora_moe_layer(gate, up, down, x.p, x.ld, x.dtype, x.rows, lg.p, lg.ld, k, truth(a[8]),
                           out.p, out.ld, (int32_t*)idx.p, (float*)w.p, ws.p, ws.bytes,
                           stream_of(a[11]));
  });
}

// An optional matrix of the residual's type and shape.
struct LikeRows {
  void* p = nullptr;
  int64_t ld = 0;
  LikeRows(PyObject* o, const char* name, const Mat& like) : ld(like.cols) {
    if (o == Py_None) return;
    const Mat m(o, name);
    same_type(m, like, (std::string(name) + " dtype differs from residual's").c_str());
    require(m.rows == like.rows && m.cols == like.cols,
            (std::string(name) + " must have the shape of residual").c_str());
    p = m.p;
    ld = m.ld;
  }
};

const void* norm_weight(PyObject* o, const char* name, int64_t dim, int32_t* code) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  const int32_t c = code_of(t, name);
  if (*code >= 0 && c != *code)
    throw Refused(PyExc_TypeError, "x_weight and y_weight differ in dtype");
  *code = c;
  const Vec v(o, name, t.scalar_type());
  require(v.n == dim, (std::string(name) + " must have dim entries").c_str());
  return v.p;
}

enum { kNoGate, kChannelGate, kTokenGate, kFullGate };

// y, x_weight, y_weight, gate, residual_scale, y_scale, weight_offset, eps from a[at] on
mlora_norm_block norm_block(const Mat& res, Args a) {
  mlora_norm_block b{};
  b.residual = res.p;
  b.residual_ld = res.ld;
  b.dtype = res.dtype;
  b.dim = size32(res.cols, "residual");
  b.n_tokens = res.rows;
  const LikeRows y(a[0], "y", res);
  b.y = y.p;
  b.y_ld = y.ld;
  // rows without entries have no memory; the block still has a y then
  static const char kNothing = 0;
  if (a[0] != Py_None && !b.y) b.y = &kNothing;
  int32_t code = -1;
  b.x_weight = norm_weight(a[1], "x_weight", res.cols, &code);
  b.y_weight = norm_weight(a[2], "y_weight", res.cols, &code);
  b.w_dtype = code < 0 ? MLORA_F32 : code;
  if (a[3] != Py_None) {
    const at::Tensor& t = tensor(a[3], "gate");
    on_device(t, "gate");
    if (code_of(t, "gate") != res.dtype)
      throw Refused(PyExc_TypeError, "gate dtype differs from residual's");
    if (t.dim() == 1) {
      require(t.size(0) == res.cols && t.is_contiguous(), "a gate per channel must be [dim]");
      b.gate_form = kChannelGate;
    } else {
      require(t.dim() == 2 && t.size(0) == res.rows && (t.size(1) == 1 || t.size(1) == res.cols),
              "gate must be [dim], [n_tokens, 1] or [n_tokens, dim]");
      b.gate_form = t.size(1) == 1 ? kTokenGate : kFullGate;
      require(t.size(1) == 1 || res.rows == 0 || t.stride(1) == 1, "gate must have contiguous rows");
      b.gate_ld = res.rows > 1 ? t.stride(0) : t.size(1);
    }
    b.gate = t.data_ptr();
  }
  b.residual_scale = real(a[4]);
  b.y_scale = real(a[5]);
  b.weight_offset = real(a[6]);
  b.eps = real(a[7]);
  return b;
}

// residual, r, x, y, x_weight, y_weight, gate, residual_scale, y_scale, weight_offset, eps, stream
PyObject* block_norm(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const Mat res(a[0], "residual");
    const mlora_norm_block b = norm_block(res, a + 3);
    const LikeRows r(a[1], "r", res), x(a[2], "x", res);
    return mlora_block_norm(&b, r.p, r.ld, x.p, x.ld, stream_of(a[11]));
  });
}

// A [dim] vector of sums, or None.
float* sums_of(PyObject* o, const char* name, int64_t dim) {
  const Vec v(o, name, at::kFloat, true);
  require(o == Py_None || v.n == dim, (std::string(name) + " must have dim entries").c_str());
  return static_cast<float*>(v.p);
}

// residual, d_r, d_x, d_residual, d_y, d_x_weight, d_y_weight, d_gate, y, x_weight, y_weight, gate,
// residual_scale, y_scale, weight_offset, eps, workspace, stream
PyObject* block_norm_backward(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 18, [&] {
    const Mat res(a[0], "residual");
    const mlora_norm_block b = norm_block(res, a + 8);
    const LikeRows dr(a[1], "d_r", res), dx(a[2], "d_x", res), dres(a[3], "d_residual", res),
        dy(a[4], "d_y", res);
    float *dwx = sums_of(a[5], "d_x_weight", res.cols), *dwy = sums_of(a[6], "d_y_weight", res.cols);
    void* dg = nullptr;
    int64_t dg_ld = 0;
    if (a[7] != Py_None) {
      require(b.gate_form != kNoGate, "d_gate without a gate");
      if (b.gate_form == kFullGate) {
        const LikeRows g(a[7], "d_gate", res);
        dg = g.p;
        dg_ld = g.ld;
      } else {
        const Vec g(a[7], "d_gate", at::kFloat);
        require(tensor(a[7], "d_gate").sizes() == tensor(a[11], "gate").sizes(),
                "d_gate must have the gate's shape");
        dg = g.p;
        dg_ld = 1;
      }
    }
    const Space ws(a[16]);
    return mlora_block_norm_backward(&b, dr.p, dr.ld, dx.p, dx.ld, dres.p, dres.ld, dy.p, dy.ld,
                                     dwx, dwy, dg, dg_ld, ws.p, ws.bytes, stream_of(a[17]));
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
                          MLORA_FAST(fp8_quant),
                          MLORA_FAST(fp8_gemm),
                          MLORA_FAST(moe_layer),
                          MLORA_FAST(block_norm),
                          MLORA_FAST(block_norm_backward),
                          {"set_error", set_error, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&kModule); }
