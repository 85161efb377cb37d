// decode_binding.cpp -- the Python module _decode behind the package's single-token entry points
// (decode.py) and those for runs of tokens (runs.py): checks every tensor against the sizes a call implies, takes its address, and calls the C ABI
// of include/qv_decode.h and include/qv_runs.h on the current stream.
//
// The calls below take a few microseconds on the device, and the same checks written in Python and
// passed on by ctypes took 9 to 15, so a serving loop would wait for its own binding.  Host code only.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <sstream>
#include <string>

#include "qv_decode.h"
#include "qv_decode_internal.h"
#include "qv_runs.h"

namespace {

struct Bad {  // becomes a ValueError
  std::string text;
};
struct Raised {};  // a Python error is set

using Shape = std::initializer_list<int64_t>;

std::string shape_text(Shape s) {
  std::ostringstream o;
  o << "(";
  const char* comma = "";
  for (int64_t n : s) o << comma << n, comma = ", ";
  o << (s.size() == 1 ? ",)" : ")");
  return o.str();
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "float32";
    case at::kBFloat16: return "bfloat16";
    case at::kByte: return "uint8";
    case at::kChar: return "int8";
    case at::kInt: return "int32";
    case at::kLong: return "int64";
    case at::kHalf: return "float16";
    case at::kDouble: return "float64";
    case at::kFloat8_e4m3fn: return "float8_e4m3fn";
    case at::kFloat8_e5m2: return "float8_e5m2";
    default: return c10::toString(t);
  }
}

// One call: its name for messages, and the GPU that every operand has to be on.
struct Call {
  const char* what;
  int device = -1;

  [[noreturn]] void bad(const std::string& text) const { throw Bad{std::string(what) + ": " + text}; }

  [[noreturn]] void bad(const char* name, const at::Tensor& t, const std::string& wanted) const {
    std::ostringstream o;
    o << name << " is " << type_name(t.scalar_type()) << " " << t.sizes() << " with strides " << t.strides()
      << ", expected " << wanted;
    bad(o.str());
  }

  const at::Tensor& tensor(const char* name, PyObject* o) const {
    if (o == Py_None) bad(std::string(name) + " is required");
    if (!THPVariable_Check(o)) bad(std::string(name) + " must be a torch tensor");
    return THPVariable_Unpack(o);
  }

  void dense(const char* name, const at::Tensor& t, at::ScalarType type, Shape shape) const {
    if (t.scalar_type() != type || !t.sizes().equals(c10::IntArrayRef(shape)) || !t.is_contiguous())
      bad(name, t, std::string("dense ") + type_name(type) + " " + shape_text(shape));
  }

  // Row stride of a float operand [M, N] with unit column stride.
  int64_t rows(const char* name, const at::Tensor& t, int64_t M, int64_t N, qv_dtype* type) const {
    *type = float_type(name, t);
    if (t.dim() != 2 || t.size(0) != M || t.size(1) != N) bad(name, t, "shape " + shape_text({M, N}));
    if ((t.stride(1) != 1 && N > 1) || (t.stride(0) < N && M > 1))
      bad(name, t, "unit column stride and a row stride of at least " + std::to_string(N));
    return M > 1 ? t.stride(0) : N;  // a single row has no stride of its own
  }

  qv_dtype float_type(const char* name, const at::Tensor& t) const {
    if (t.scalar_type() == at::kFloat) return QV_F32;
    if (t.scalar_type() == at::kBFloat16) return QV_BF16;
    bad(name, t, "float32 or bfloat16");
  }

  // Rows [T, heads, D] of `type` with unit channel stride.
  qv_heads heads(const char* name, const at::Tensor& t, int64_t T, int64_t H, int64_t D, qv_dtype type) const {
    if (float_type(name, t) != type) bad(name, t, type == QV_F32 ? "float32" : "bfloat16");
    if (t.dim() != 3 || t.size(0) != T || t.size(1) != H || t.size(2) != D)
      bad(name, t, "shape " + shape_text({T, H, D}));
    if (t.stride(2) != 1 || (t.stride(1) < D && H > 1)) bad(name, t, "unit channel stride and heads that do not overlap");
    return {t.data_ptr(), T > 1 ? t.stride(0) : 0, H > 1 ? t.stride(1) : D};
  }

  // The same for rows that are written.
  qv_heads output(const char* name, const at::Tensor& t, int64_t T, int64_t H, int64_t D, qv_dtype type) const {
    const qv_heads h = heads(name, t, T, H, D, type);
    if (qv::rows_overlap(T, h.token_stride, H, h.head_stride, D)) bad(name, t, "tokens and heads that do not overlap");
    return h;
  }

  // Row stride of a page table [rows, pages].
  int64_t table(const at::Tensor& t) const {
    if (t.scalar_type() != at::kInt || t.dim() != 2 || (t.stride(1) != 1 && t.size(1) > 1) ||
        (t.stride(0) < t.size(1) && t.size(0) > 1))
      bad("page_table", t, "int32 [sequences, pages] with unit column stride");
    return t.size(0) > 1 ? t.stride(0) : t.size(1);
  }

  void* workspace(const at::Tensor& t, size_t need) const {
    if (t.scalar_type() != at::kByte || !t.is_contiguous())
      bad("workspace", t, "dense uint8 of at least " + std::to_string(need) + " bytes");
    if ((size_t)t.numel() < need)
      bad("workspace holds " + std::to_string(t.numel()) + " bytes, needs " + std::to_string(need));
    return t.data_ptr();
  }

  // Every operand on one GPU (checked after the shapes, so that shape errors are reported first).
  void on_gpu(const at::Tensor& t) {
    if (!t.is_cuda()) bad("every operand must be a GPU tensor (got one on " + t.device().str() + ")");
    on_device(t.get_device());
  }
  void on_device(int d) {
    if (device >= 0 && d != device) bad("operands are on different devices");
    device = d;
  }

  // The given torch stream, or the current one of the operands' GPU.
  void* stream(PyObject* o) const {
    if (o == Py_None) return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
    PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
    if (!raw) throw Raised{};
    void* s = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    if (PyErr_Occurred()) throw Raised{};
    return s;
  }
};

int64_t whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

// Any other number stands for one that the library refuses.
qv_epilogue epilogue(PyObject* o) {
  const int64_t v = whole(o);
  return v == QV_EPI_NONE ? QV_EPI_NONE : (v == QV_EPI_GELU ? QV_EPI_GELU : (qv_epilogue)-1);
}

void* address(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

// Of a table, whose address says that there is one: a tensor without elements has none of its own.
const float* table_address(const at::Tensor* t) {
  alignas(16) static const float none[4] = {};
  return t && t->numel() == 0 ? none : (const float*)address(t);
}

PyObject* qv_error = nullptr;  // the package's QVError

PyObject* done(const Call& c, qv_status st) {
  if (st == QV_OK) Py_RETURN_NONE;
  PyObject* e = PyObject_CallFunction(qv_error, "is", (int)st, c.what);
  if (e) {
    PyErr_SetObject(qv_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

template <typename F>
PyObject* guarded(const char* what, Py_ssize_t given, Py_ssize_t wanted, F&& body) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", what, wanted, given);
    return nullptr;
  }
  try {
    Call c{what};
    return body(c);
  } catch (const Bad& b) {
    PyErr_SetString(PyExc_ValueError, b.text.c_str());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// ------------------------------------------------------------------------------------ few-row linears

struct Linear {
  const at::Tensor *X, *Wq, *ws, *bias, *Y;
  int64_t M, K, N, group, ldx, ldy;
  qv_dtype xt, yt;
};

Linear linear_operands(const Call& c, PyObject* X, PyObject* Wq, PyObject* ws, PyObject* group, PyObject* bias,
                       PyObject* Y) {
  Linear l;
  l.X = &c.tensor("X", X);
  l.Wq = &c.tensor("Wq", Wq);
  if (l.X->dim() != 2) c.bad("X", *l.X, "a 2-D tensor");
  if (l.Wq->dim() != 2) c.bad("Wq", *l.Wq, "a 2-D tensor");
  l.M = l.X->size(0);
  l.K = l.X->size(1);
  l.N = l.Wq->size(0);
  c.dense("Wq", *l.Wq, at::kByte, {l.N, l.K / 2});
  l.group = whole(group);
  if (l.group <= 0 || l.K % l.group != 0)
    c.bad("group " + std::to_string(l.group) + " must be positive and divide K = " + std::to_string(l.K));
  l.ws = &c.tensor("w_scale", ws);
  const int64_t G = l.K / l.group;
  if (G == 1 && l.ws->dim() == 1)
    c.dense("w_scale", *l.ws, at::kFloat, {l.N});
  else
    c.dense("w_scale", *l.ws, at::kFloat, {l.N, G});
  l.bias = bias == Py_None ? nullptr : &c.tensor("bias", bias);
  if (l.bias) c.dense("bias", *l.bias, at::kFloat, {l.N});
  l.Y = &c.tensor("Y", Y);
  l.ldx = c.rows("X", *l.X, l.M, l.K, &l.xt);
  l.ldy = c.rows("Y", *l.Y, l.M, l.N, &l.yt);
  return l;
}

void linear_device(Call& c, const Linear& l) {
  c.on_gpu(*l.X);
  c.on_gpu(*l.Wq);
  c.on_gpu(*l.ws);
  if (l.bias) c.on_gpu(*l.bias);
  c.on_gpu(*l.Y);
}

// X, Wq, w_scale, group, bias, Y, epi, stream
PyObject* w4a16_gemv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("qv_w4a16_gemv", n, 8, [&](Call& c) {
    const Linear l = linear_operands(c, a[0], a[1], a[2], a[3], a[4], a[5]);
    const qv_epilogue epi = epilogue(a[6]);
    linear_device(c, l);
    const c10::hip::HIPGuard on((c10::DeviceIndex)c.device);
    return done(c, qv_w4a16_gemv(l.X->data_ptr(), l.xt, l.M, l.K, l.ldx, (const uint8_t*)l.Wq->data_ptr(),
                                 (const float*)l.ws->data_ptr(), l.group, (const float*)address(l.bias), l.N, epi,
                                 l.Y->data_ptr(), l.yt, l.ldy, c.stream(a[7])));
  });
}

// X, inv_smooth, Wq, w_scale, group, bias, Y, workspace, epi, stream
PyObject* w4a16_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("qv_w4a16_linear", n, 10, [&](Call& c) {
    const Linear l = linear_operands(c, a[0], a[2], a[3], a[4], a[5], a[6]);
    const at::Tensor* inv = a[1] == Py_None ? nullptr : &c.tensor("inv_smooth", a[1]);
    if (inv) c.dense("inv_smooth", *inv, at::kFloat, {l.K});
    const at::Tensor& work = c.tensor("workspace", a[7]);
    void* w = c.workspace(work, qv_w4a16_linear_workspace_size(l.M, l.K));
    const qv_epilogue epi = epilogue(a[8]);
    linear_device(c, l);
    if (inv) c.on_gpu(*inv);
    c.on_gpu(work);
    const c10::hip::HIPGuard on((c10::DeviceIndex)c.device);
    return done(c, qv_w4a16_linear(l.X->data_ptr(), l.xt, l.M, l.K, l.ldx, (const float*)address(inv),
                                   (const uint8_t*)l.Wq->data_ptr(), (const float*)l.ws->data_ptr(), l.group,
                                   (const float*)address(l.bias), l.N, epi, l.Y->data_ptr(), l.yt, l.ldy, w,
                                   (size_t)work.numel(), c.stream(a[9])));
  });
}

// ---------------------------------------------------------------------------------------- paged cache

struct Cache {
  qv_kv_cache c;
  int device;
};

// k_pages, v_pages, k_scale, v_scale -> (bytes of a Cache, pages, heads, page_size, head_dim)
PyObject* kv_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("QVKVCache", n, 4, [&](Call& c) -> PyObject* {
    const at::Tensor &k = c.tensor("k_pages", a[0]), &v = c.tensor("v_pages", a[1]);
    const bool fp8 = k.scalar_type() == at::kFloat8_e4m3fn, q8 = fp8 || k.scalar_type() == at::kChar;
    if ((!q8 && k.scalar_type() != at::kBFloat16) || k.dim() != 4)
      c.bad("k_pages", k, "bfloat16, int8 or float8_e4m3fn [pages, heads, page_size, D]");
    if (v.scalar_type() != k.scalar_type() || !v.sizes().equals(k.sizes()) || !v.strides().equals(k.strides()))
      c.bad("v_pages", v, "type, shape and strides of k_pages");
    const int64_t D = k.size(3);
    if (k.size(1) == 0 || k.size(2) == 0 || D == 0) c.bad("k_pages", k, "at least one head, token and channel");
    if (k.stride(3) != 1 && D > 1) c.bad("k_pages", k, "unit channel stride");
    int64_t stride[3];
    for (int i = 0; i < 3; ++i) {
      stride[i] = k.size(i) > 1 ? k.stride(i) : D;  // an extent of one has no stride of its own
      if (stride[i] < D) c.bad("k_pages", k, "tokens that do not overlap");
    }
    const at::Tensor* s[2] = {nullptr, nullptr};
    if (q8) {
      for (int i = 0; i < 2; ++i) {
        const char* name = i ? "v_scale" : "k_scale";
        s[i] = &c.tensor(name, a[2 + i]);
        int64_t scales = k.size(2);  // of a page and head
        if (fp8) {
          scales = s[i]->dim() == 3 ? s[0]->size(2) : 0;
          if (scales <= 0 || k.size(2) % scales != 0 || k.size(2) / scales % 16 != 0)
            c.bad(name, *s[i], "[pages, heads, blocks] with blocks of a multiple of 16 tokens that divides the page size " +
                                   std::to_string(k.size(2)));
        }
        c.dense(name, *s[i], at::kFloat, {k.size(0), k.size(1), scales});
      }
    } else if (a[2] != Py_None || a[3] != Py_None) {
      c.bad("a bfloat16 cache has no scales");
    }
    c.on_gpu(k);
    c.on_gpu(v);
    if (q8) c.on_gpu(*s[0]), c.on_gpu(*s[1]);
    Cache out;
    std::memset(&out, 0, sizeof out);
    out.c.k_pages = k.data_ptr();
    out.c.v_pages = v.data_ptr();
    out.c.k_scale = (float*)address(s[0]);
    out.c.v_scale = (float*)address(s[1]);
    out.c.num_pages = k.size(0);
    out.c.heads = k.size(1);
    out.c.page_size = k.size(2);
    out.c.head_dim = D;
    out.c.page_stride = stride[0];
    out.c.head_stride = stride[1];
    out.c.token_stride = stride[2];
    out.c.dtype = fp8 ? QV_KV_FP8 : (q8 ? QV_KV_INT8 : QV_KV_BF16);
    out.c.scale_tokens = fp8 ? (int32_t)(k.size(2) / s[0]->size(2)) : 0;
    out.device = c.device;
    return Py_BuildValue("y#LLLL", (const char*)&out, (Py_ssize_t)sizeof out, (long long)k.size(0),
                         (long long)k.size(1), (long long)k.size(2), (long long)D);
  });
}

const Cache& cache_of(const Call& c, PyObject* handle) {
  if (!PyBytes_CheckExact(handle) || PyBytes_GET_SIZE(handle) != (Py_ssize_t)sizeof(Cache))
    c.bad("cache must be a QVKVCache");
  return *reinterpret_cast<const Cache*>(PyBytes_AS_STRING(handle));
}

// cache, page_table, token_seq, token_index, K, V, cos, sin, position, Q, Q_out, stream
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("qv_kv_append", n, 12, [&](Call& c) {
    const Cache& kv = cache_of(c, a[0]);
    const int64_t H = kv.c.heads, D = kv.c.head_dim;
    c.on_device(kv.device);
    const at::Tensor &table = c.tensor("page_table", a[1]), &index = c.tensor("token_index", a[3]),
                     &K = c.tensor("K", a[4]), &V = c.tensor("V", a[5]);
    const int64_t ld = c.table(table);
    const qv_dtype type = c.float_type("K", K);
    const int64_t T = K.dim() > 0 ? K.size(0) : 0;
    const qv_heads k = c.heads("K", K, T, H, D, type), v = c.heads("V", V, T, H, D, type);
    c.dense("token_index", index, at::kInt, {T});
    const at::Tensor* opt[4] = {nullptr, nullptr, nullptr, nullptr};  // token_seq, cos, sin, position
    if (a[2] != Py_None) {
      opt[0] = &c.tensor("token_seq", a[2]);
      c.dense("token_seq", *opt[0], at::kInt, {T});
    } else if (T > table.size(0)) {
      c.bad(std::to_string(T) + " tokens of " + std::to_string(table.size(0)) + " sequences need token_seq");
    }
    int64_t axes = 1, places = 0;
    if (a[8] != Py_None) {
      opt[3] = &c.tensor("position", a[8]);
      if (opt[3]->dim() == 2) axes = opt[3]->size(1);
      if (axes != 1 && axes != 2) c.bad("position", *opt[3], "1 or 2 axes");
      c.dense("position", *opt[3], at::kInt, {T, axes});
    }
    if ((a[6] == Py_None) != (a[7] == Py_None)) c.bad("cos and sin come together");
    if (a[6] != Py_None) {
      opt[1] = &c.tensor("cos", a[6]);
      opt[2] = &c.tensor("sin", a[7]);
      places = opt[1]->dim() == 2 ? opt[1]->size(0) : 0;
      c.dense("cos", *opt[1], at::kFloat, {places, D / 2 / axes});
      c.dense("sin", *opt[2], at::kFloat, {places, D / 2 / axes});
    }
    if ((a[9] == Py_None) != (a[10] == Py_None)) c.bad("Q and Q_out come together");
    qv_heads q, qo;
    int64_t Hq = 0;
    const at::Tensor *Q = nullptr, *Qo = nullptr;
    if (a[9] != Py_None) {
      Q = &c.tensor("Q", a[9]);
      Qo = &c.tensor("Q_out", a[10]);
      Hq = Q->dim() == 3 ? Q->size(1) : 0;
      if (Hq == 0) c.bad("Q", *Q, "[T, q_heads, D]");
      q = c.heads("Q", *Q, T, Hq, D, type);
      qo = c.output("Q_out", *Qo, T, Hq, D, type);
    }
    for (const at::Tensor* t : {&table, &index, &K, &V, opt[0], opt[1], opt[2], opt[3], Q, Qo})
      if (t) c.on_gpu(*t);
    const c10::hip::HIPGuard on((c10::DeviceIndex)c.device);
    return done(c, qv_kv_append(&kv.c, (const int32_t*)table.data_ptr(), table.size(0), table.size(1), ld,
                                (const int32_t*)address(opt[0]), (const int32_t*)index.data_ptr(), T, &k, &v, type,
                                table_address(opt[1]), table_address(opt[2]), places, axes,
                                (const int32_t*)address(opt[3]), Q ? &q : nullptr, Q ? &qo : nullptr, Hq,
                                c.stream(a[11])));
  });
}

// Q, cache, page_table, lens, O, workspace, scale, window, stream
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("qv_paged_attention", n, 9, [&](Call& c) {
    const Cache& kv = cache_of(c, a[1]);
    c.on_device(kv.device);
    const at::Tensor &Q = c.tensor("Q", a[0]), &table = c.tensor("page_table", a[2]), &lens = c.tensor("lens", a[3]),
                     &O = c.tensor("O", a[4]), &work = c.tensor("workspace", a[5]);
    const int64_t D = kv.c.head_dim;
    if (kv.c.heads <= 0) c.bad("the cache has no heads");
    if (Q.dim() != 3 || Q.size(1) == 0 || Q.size(1) % kv.c.heads != 0 || Q.size(2) != D)
      c.bad("Q", Q, "[B, a multiple of " + std::to_string(kv.c.heads) + " heads, " + std::to_string(D) + "]");
    const int64_t B = Q.size(0), Hq = Q.size(1);
    const qv_dtype type = c.float_type("Q", Q);
    const qv_heads q = c.heads("Q", Q, B, Hq, D, type), o = c.output("O", O, B, Hq, D, type);
    const int64_t ld = c.table(table);
    if (table.size(0) != B) c.bad("page_table", table, std::to_string(B) + " rows");
    c.dense("lens", lens, at::kInt, {B});
    const double scale = a[6] == Py_None ? 1.0 / std::sqrt((double)D) : PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    const int64_t window = whole(a[7]);
    if (window < 0) c.bad("window " + std::to_string(window) + " must not be negative");
    void* w = c.workspace(
        work, qv_paged_attention_workspace_size(B, Hq, kv.c.heads, D, table.size(1) * kv.c.page_size));
    for (const at::Tensor* t : {&Q, &table, &lens, &O, &work}) c.on_gpu(*t);
    const c10::hip::HIPGuard on((c10::DeviceIndex)c.device);
    return done(c, qv_paged_attention(&q, type, B, Hq, &kv.c, (const int32_t*)table.data_ptr(), table.size(1), ld,
                                      (const int32_t*)lens.data_ptr(), (float)scale, window, &o, w,
                                      (size_t)work.numel(), c.stream(a[8])));
  });
}

// Q, starts, max_run, cache, page_table, lens, O, workspace, scale, window, sinks, causal, stream
PyObject* run_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("qv_run_attention", n, 13, [&](Call& c) {
    const Cache& kv = cache_of(c, a[3]);
    c.on_device(kv.device);
    const at::Tensor &Q = c.tensor("Q", a[0]), &table = c.tensor("page_table", a[4]), &lens = c.tensor("lens", a[5]),
                     &O = c.tensor("O", a[6]), &work = c.tensor("workspace", a[7]);
    const int64_t D = kv.c.head_dim;
    if (kv.c.heads <= 0) c.bad("the cache has no heads");
    if (Q.dim() != 3 || Q.size(1) == 0 || Q.size(1) % kv.c.heads != 0 || Q.size(2) != D)
      c.bad("Q", Q, "[T, a multiple of " + std::to_string(kv.c.heads) + " heads, " + std::to_string(D) + "]");
    const int64_t T = Q.size(0), Hq = Q.size(1), max_run = whole(a[2]);
    const qv_dtype type = c.float_type("Q", Q);
    const qv_heads q = c.heads("Q", Q, T, Hq, D, type), o = c.output("O", O, T, Hq, D, type);
    const int64_t ld = c.table(table), B = table.size(0);
    c.dense("lens", lens, at::kInt, {B});
    const at::Tensor* starts = a[1] == Py_None ? nullptr : &c.tensor("starts", a[1]);
    if (starts) c.dense("starts", *starts, at::kInt, {B + 1});
    if (max_run < 0 || max_run > T) c.bad("max_run " + std::to_string(max_run) + " of " + std::to_string(T) + " rows");
    if (!starts && (T != B || max_run > 1))
      c.bad(std::to_string(T) + " rows of " + std::to_string(B) + " sequences in runs of up to " + std::to_string(max_run) +
            " need starts");
    const double scale = a[8] == Py_None ? 1.0 / std::sqrt((double)D) : PyFloat_AsDouble(a[8]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    const int64_t window = whole(a[9]), sinks = whole(a[10]);
    if (window < 0) c.bad("window " + std::to_string(window) + " must not be negative");
    if (sinks < 0) c.bad("sinks " + std::to_string(sinks) + " must not be negative");
    if (!std::isfinite((float)scale)) c.bad("scale " + std::to_string(scale) + " must be finite");
    const int causal = PyObject_IsTrue(a[11]);
    if (causal < 0) throw Raised{};
    void* w = c.workspace(
        work, qv_run_attention_workspace_size(T, B, max_run, Hq, kv.c.heads, D, table.size(1) * kv.c.page_size));
    for (const at::Tensor* t : {&Q, starts, &table, &lens, &O, &work})
      if (t) c.on_gpu(*t);
    const c10::hip::HIPGuard on((c10::DeviceIndex)c.device);
    return done(c, qv_run_attention(&q, type, T, Hq, (const int32_t*)address(starts), B, max_run, &kv.c,
                                    (const int32_t*)table.data_ptr(), table.size(1), ld, (const int32_t*)lens.data_ptr(),
                                    (float)scale, window, sinks, causal, &o, w, (size_t)work.numel(), c.stream(a[12])));
  });
}

// runs, lens, free_pages, free_count, page_size, page_table, starts, lens_out, free_left, token_seq, token_index, slots,
// status, stream
PyObject* page_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("qv_page_tables", n, 14, [&](Call& c) {
    static const char* const names[] = {"runs", "lens", "free_pages", "free_count", nullptr, "page_table", "starts",
                                        "lens_out", "free_left", "token_seq", "token_index", "slots", "status"};
    const at::Tensor* t[13] = {};
    for (int i = 0; i < 13; ++i)
      if (i != 4) t[i] = &c.tensor(names[i], a[i]);
    const int64_t page_size = whole(a[4]);
    if (page_size <= 0) c.bad("page_size " + std::to_string(page_size) + " must be positive");
    const int64_t ld = c.table(*t[5]), B = t[5]->size(0);
    const int64_t F = t[2]->dim() == 1 ? t[2]->size(0) : 0, T = t[9]->dim() == 1 ? t[9]->size(0) : 0;
    const int64_t sizes[13] = {B, B, F, 1, 0, 0, B + 1, B, 1, T, T, T, B};
    for (int i = 0; i < 13; ++i)
      if (i != 4 && i != 5) c.dense(names[i], *t[i], i == 11 ? at::kLong : at::kInt, {sizes[i]});
    for (int i = 0; i < 13; ++i)
      if (t[i]) c.on_gpu(*t[i]);
    const c10::hip::HIPGuard on((c10::DeviceIndex)c.device);
    auto p = [&](int i) { return (int32_t*)t[i]->data_ptr(); };
    return done(c, qv_page_tables(p(0), p(1), B, page_size, p(2), F, p(3), p(5), t[5]->size(1), ld, p(6), p(7), p(8), p(9),
                                  p(10), (int64_t*)t[11]->data_ptr(), T, p(12), c.stream(a[13])));
  });
}

PyMethodDef methods[] = {
    {"w4a16_gemv", (PyCFunction)(void (*)(void))w4a16_gemv, METH_FASTCALL, nullptr},
    {"w4a16_linear", (PyCFunction)(void (*)(void))w4a16_linear, METH_FASTCALL, nullptr},
    {"kv_cache", (PyCFunction)(void (*)(void))kv_cache, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void (*)(void))paged_attention, METH_FASTCALL, nullptr},
    {"run_attention", (PyCFunction)(void (*)(void))run_attention, METH_FASTCALL, nullptr},
    {"page_tables", (PyCFunction)(void (*)(void))page_tables, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decode", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode(void) {
  PyObject* package = PyImport_ImportModule("bit_ptq_reconstruction_amd");
  if (!package) return nullptr;
  qv_error = PyObject_GetAttrString(package, "QVError");
  Py_DECREF(package);
  if (!qv_error) return nullptr;
  return PyModule_Create(&module);
}
