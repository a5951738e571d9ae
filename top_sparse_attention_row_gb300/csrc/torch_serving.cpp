// Native binding of the serving-step operators (module _serving): argument checks, output tensors and
// streams in C++, for calls whose kernels take a few microseconds.  Same checks and errors as the rest of
// the binding: TypeError for a wrong type, ValueError for a wrong shape, device or layout, RuntimeError for
// a status of the library.  No computation happens here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <string>

#include "qsa.h"

namespace {

struct PythonError {};   // a Python exception is set

[[noreturn]] void fail(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw PythonError();
}

std::string shape_text(c10::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}
std::string type_text(at::ScalarType t) {
  switch (t) {
    case at::kInt: return "torch.int32";
    case at::kFloat: return "torch.float32";
    case at::kByte: return "torch.uint8";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    default: return std::string("torch.") + c10::toString(t);
  }
}

const at::Tensor& tensor_of(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
bool given(PyObject* o) { return o != nullptr && o != Py_None; }

void check_type(const at::Tensor& t, const char* name, at::ScalarType type, c10::Device device) {
  if (t.scalar_type() != type)
    fail(PyExc_TypeError, std::string(name) + " must be " + type_text(type) + ", got " + type_text(t.scalar_type()));
  if (t.device() != device)
    fail(PyExc_ValueError, std::string(name) + " must be on " + device.str() + ", got " + t.device().str());
}
void check_shape(const at::Tensor& t, const char* name, c10::IntArrayRef shape) {
  if (t.sizes() != shape)
    fail(PyExc_ValueError, std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
}
// A contiguous tensor of this type, place and shape.
const at::Tensor& checked(PyObject* o, const char* name, at::ScalarType type, c10::Device device,
                          std::initializer_list<int64_t> shape) {
  const at::Tensor& t = tensor_of(o, name);
  check_type(t, name, type, device);
  check_shape(t, name, c10::IntArrayRef(shape.begin(), shape.size()));
  if (!t.is_contiguous()) fail(PyExc_ValueError, std::string(name) + " must be contiguous");
  return t;
}
// Rows [n, heads, dim] with contiguous heads; returns the row stride in elements.
int64_t checked_rows(const at::Tensor& t, const char* name, at::ScalarType type, c10::Device device, int64_t n,
                     int64_t heads, int64_t dim) {
  check_type(t, name, type, device);
  const int64_t shape[3] = {n, heads, dim};
  check_shape(t, name, c10::IntArrayRef(shape, 3));
  if ((dim > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != dim))
    fail(PyExc_ValueError, std::string(name) + " must have contiguous heads (strides (any, " + std::to_string(dim) +
                               ", 1)), got " + shape_text(t.strides()));
  return n > 1 ? t.stride(0) : heads * dim;
}
const at::Tensor& ranked(PyObject* o, const char* name, int64_t dims) {
  const at::Tensor& t = tensor_of(o, name);
  if (t.dim() != dims)
    fail(PyExc_ValueError, std::string(name) + " must have " + std::to_string(dims) + " dims, got " +
                               std::to_string(t.dim()));
  return t;
}
int32_t dtype_code(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return QSA_BF16;
  if (t.scalar_type() == at::kHalf) return QSA_FP16;
  fail(PyExc_TypeError, std::string(name) + " must be bfloat16 or float16, got " + type_text(t.scalar_type()));
}
int32_t int32_of(long long v, const char* name) {
  if (v > INT32_MAX || v < INT32_MIN) fail(PyExc_ValueError, std::string(name) + " is out of range");
  return static_cast<int32_t>(v);
}

// Makes the tensors' device current for the call and finds the stream to launch on; tensors made here for
// another stream than the current one are recorded on it.
class Launch {
 public:
  Launch(c10::Device device, PyObject* stream) : device_(device) {
    if (!device.is_cuda()) fail(PyExc_ValueError, "tensors must be CUDA tensors");
    if (c10::cuda::current_device() != device.index()) guard_.emplace(device);
    if (!given(stream)) {
      raw_ = c10::cuda::getCurrentCUDAStream(device.index()).stream();
      return;
    }
    PyObject* const n = PyLong_Check(stream) ? Py_NewRef(stream) : PyObject_GetAttrString(stream, "cuda_stream");
    if (!n) throw PythonError();
    raw_ = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(n));
    Py_DECREF(n);
    if (PyErr_Occurred()) throw PythonError();
    other_ = raw_ != c10::cuda::getCurrentCUDAStream(device.index()).stream();
  }
  at::Tensor empty(c10::IntArrayRef shape, at::ScalarType type) {
    at::Tensor t = at::empty(shape, at::TensorOptions().dtype(type).device(device_));
    if (other_) t.record_stream(c10::cuda::getStreamFromExternal(raw_, device_.index()));
    return t;
  }
  void* stream() const { return raw_; }

 private:
  c10::Device device_;
  std::optional<c10::cuda::CUDAGuard> guard_;
  cudaStream_t raw_ = nullptr;
  bool other_ = false;
};

void check_status(qsa_status st, const char* what) {
  if (st == QSA_OK) return;
  static const char* const names[] = {"QSA_OK", "QSA_ERR_INVALID_ARG", "QSA_ERR_UNSUPPORTED", "QSA_ERR_WORKSPACE",
                                      "QSA_ERR_CUDA", "QSA_ERR_TIMEOUT"};
  const int n = static_cast<int>(st);
  fail(PyExc_RuntimeError, std::string(what) + " failed: " + (n >= 0 && n < 6 ? names[n] : std::to_string(n)) + " (" +
                               qsa_status_string(st) + ")");
}

template <typename F>
PyObject* guarded(F&& body) {
  try {
    return body();
  } catch (const PythonError&) {
    return nullptr;
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// A tensor over `n` elements of `block`'s storage from element `at` on.
at::Tensor piece(const at::Tensor& block, int64_t at, int64_t n) {
  auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(block.storage()), block.key_set(), block.dtype());
  impl->set_sizes_contiguous(n);
  impl->set_storage_offset(at);
  return at::Tensor(std::move(impl));
}

PyObject* g_plan_type = nullptr;   // the PagePlan named tuple

PyObject* page_plan(PyObject*, PyObject* args, PyObject* kw) {
  static const char* names[] = {"past_lens", "new_lens", "page_table", "free_pages", "free_head", "page_size",
                                "max_rows", "n_pages", "free_head_out", "cu_seqlens_q", "kv_lens", "positions",
                                "slots", "shortfall", "stream", nullptr};
  PyObject *past_o, *new_o, *table_o, *free_o, *head_o;
  PyObject *out[6] = {nullptr, nullptr, nullptr, nullptr, nullptr, nullptr}, *stream = nullptr;
  long long page_size, max_rows, n_pages = 0;
  if (!PyArg_ParseTupleAndKeywords(args, kw, "OOOOOLL|$LOOOOOOO:page_plan", const_cast<char**>(names), &past_o, &new_o,
                                   &table_o, &free_o, &head_o, &page_size, &max_rows, &n_pages, &out[0], &out[1],
                                   &out[2], &out[3], &out[4], &out[5], &stream))
    return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& past = ranked(past_o, "past_lens", 1);
    const c10::Device dev = past.device();
    const int64_t n = past.size(0);
    const int64_t ppr = ranked(table_o, "page_table", 2).size(1), n_free = ranked(free_o, "free_pages", 1).size(0);
    if (max_rows < 0) fail(PyExc_ValueError, "max_rows must not be negative");
    checked(past_o, "past_lens", at::kInt, dev, {n});
    const at::Tensor& fresh = checked(new_o, "new_lens", at::kInt, dev, {n});
    const at::Tensor& table = checked(table_o, "page_table", at::kInt, dev, {n, ppr});
    const at::Tensor& pages = checked(free_o, "free_pages", at::kInt, dev, {n_free});
    const at::Tensor& head = checked(head_o, "free_head", at::kInt, dev, {1});
    Launch on(dev, stream);
    // outputs that the caller did not bring share one allocation, each on a 16-byte boundary
    static const char* const out_names[6] = {"free_head_out", "cu_seqlens_q", "kv_lens", "positions", "slots",
                                             "shortfall"};
    const int64_t sizes[6] = {1, n + 1, n, max_rows, max_rows, 1};
    at::Tensor t[6], block;
    int64_t room = 0;
    for (int i = 0; i < 6; ++i) {
      if (given(out[i])) t[i] = checked(out[i], out_names[i], at::kInt, dev, {sizes[i]});
      else room += (sizes[i] + 3) / 4 * 4;
    }
    if (room > 0) {
      block = on.empty({room}, at::kInt);
      int64_t at = 0;
      for (int i = 0; i < 6; ++i) {
        if (t[i].defined()) continue;
        t[i] = piece(block, at, sizes[i]);
        at += (sizes[i] + 3) / 4 * 4;
      }
    }
    auto p = [](const at::Tensor& x) { return static_cast<int32_t*>(x.data_ptr()); };
    check_status(qsa_page_plan(p(past), p(fresh), p(table), p(pages), n_free, p(head), p(t[0]), p(t[1]), p(t[2]), p(t[3]),
                               p(t[4]), p(t[5]), int32_of(n, "n_requests"), int32_of(ppr, "pages_per_req"),
                               int32_of(page_size, "page_size"), n_pages, max_rows, on.stream()),
                 "qsa_page_plan");
    static const int order[6] = {1, 2, 3, 4, 0, 5};
    PyObject* const values = PyTuple_New(6);
    if (!values) throw PythonError();
    for (int i = 0; i < 6; ++i) PyTuple_SET_ITEM(values, i, THPVariable_Wrap(t[order[i]]));
    if (!g_plan_type) return values;
    PyObject* const one = PyTuple_Pack(1, values);
    PyObject* const plan = one ? PyTuple_Type.tp_new(reinterpret_cast<PyTypeObject*>(g_plan_type), one, nullptr) : nullptr;
    Py_XDECREF(one);
    Py_DECREF(values);
    if (!plan) throw PythonError();
    return plan;
  });
}

PyObject* set_plan_type(PyObject*, PyObject* type) {
  Py_XSETREF(g_plan_type, Py_NewRef(type));
  Py_RETURN_NONE;
}

// The rotation of a RopeTable: its _raw is (address of the steps, rot_dim, magnitude).
const qsa_rope_spec* spec_of(PyObject* table, PyObject* layout, long long offset, int transpose, qsa_rope_spec* s) {
  if (!given(table)) return nullptr;
  static PyObject* const name = PyUnicode_InternFromString("_raw");
  PyObject* const raw = PyObject_GetAttr(table, name);
  if (!raw) throw PythonError();
  unsigned long long steps = 0;
  int rot = 0;
  float magnitude = 1.0f;
  const int ok = PyArg_ParseTuple(raw, "Kif", &steps, &rot, &magnitude);
  Py_DECREF(raw);
  if (!ok) throw PythonError();
  int32_t code = QSA_ROPE_HALF;
  if (given(layout)) {
    if (PyUnicode_Check(layout) && PyUnicode_CompareWithASCIIString(layout, "interleaved") == 0) code = QSA_ROPE_INTERLEAVED;
    else if (!PyUnicode_Check(layout) || PyUnicode_CompareWithASCIIString(layout, "half") != 0)
      fail(PyExc_ValueError, "layout must be one of ['half', 'interleaved']");
  }
  *s = qsa_rope_spec{reinterpret_cast<const uint64_t*>(steps), rot, int32_of(offset, "rot_offset"), code,
                     transpose ? 1 : 0, magnitude};
  return s;
}

PyObject* rope(PyObject*, PyObject* args, PyObject* kw) {
  static const char* names[] = {"x", "positions", "table", "layout", "rot_offset", "transpose", "out", "stream", nullptr};
  PyObject *x_o, *pos_o, *table, *layout = nullptr, *out_o = nullptr, *stream = nullptr;
  long long offset = 0;
  int transpose = 0;
  if (!PyArg_ParseTupleAndKeywords(args, kw, "OOO|$OLpOO:rope", const_cast<char**>(names), &x_o, &pos_o, &table, &layout,
                                   &offset, &transpose, &out_o, &stream))
    return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& x = ranked(x_o, "x", 3);
    const c10::Device dev = x.device();
    const int64_t R = x.size(0), H = x.size(1), D = x.size(2);
    const int32_t code = dtype_code(x, "x");
    const int64_t xs = checked_rows(x, "x", x.scalar_type(), dev, R, H, D);
    const at::Tensor& pos = checked(pos_o, "positions", at::kInt, dev, {R});
    qsa_rope_spec s;
    if (!given(table)) fail(PyExc_TypeError, "table must be a RopeTable");
    spec_of(table, layout, offset, transpose, &s);
    Launch on(dev, stream);
    const at::Tensor out = given(out_o) ? tensor_of(out_o, "out") : on.empty({R, H, D}, x.scalar_type());
    const int64_t os = checked_rows(out, "out", x.scalar_type(), dev, R, H, D);
    if (R > 0)
      check_status(qsa_rope(x.data_ptr(), out.data_ptr(), static_cast<const int32_t*>(pos.data_ptr()), &s, R,
                            int32_of(H, "heads"), int32_of(D, "head dim"), xs, os, code, on.stream()),
                   "qsa_rope");
    return given(out_o) ? Py_NewRef(out_o) : THPVariable_Wrap(out);
  });
}

// rope_append and rope_append_fp4 (fp4: with scales, global scales and the values seen).
PyObject* append(PyObject* args, PyObject* kw, bool fp4) {
  static const char* names[] = {"q", "k", "v", "k_cache", "v_cache", "positions", "slots", "table", "layout",
                                "rot_offset", "q_out", "stream", nullptr};
  static const char* names4[] = {"q", "k", "v", "k_cache", "k_scale", "v_cache", "v_scale", "positions", "slots",
                                 "table", "k_global", "v_global", "layout", "rot_offset", "q_out", "k_seen", "v_seen",
                                 "stream", nullptr};
  PyObject *q_o, *k_o, *v_o, *kc_o, *vc_o, *ks_o = nullptr, *vs_o = nullptr, *pos_o, *slots_o, *table;
  PyObject *layout = nullptr, *q_out_o = nullptr, *k_seen_o = nullptr, *v_seen_o = nullptr, *stream = nullptr;
  long long offset = 0;
  float kg = 1.0f, vg = 1.0f;
  const int ok = fp4 ? PyArg_ParseTupleAndKeywords(args, kw, "OOOOOOOOOO|$ffOLOOOO:rope_append_fp4",
                                                   const_cast<char**>(names4), &q_o, &k_o, &v_o, &kc_o, &ks_o, &vc_o,
                                                   &vs_o, &pos_o, &slots_o, &table, &kg, &vg, &layout, &offset, &q_out_o,
                                                   &k_seen_o, &v_seen_o, &stream)
                     : PyArg_ParseTupleAndKeywords(args, kw, "OOOOOOOO|$OLOO:rope_append", const_cast<char**>(names), &q_o,
                                                   &k_o, &v_o, &kc_o, &vc_o, &pos_o, &slots_o, &table, &layout, &offset,
                                                   &q_out_o, &stream);
  if (!ok) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& k = ranked(k_o, "k", 3);
    const c10::Device dev = k.device();
    const at::ScalarType type = k.scalar_type();
    const int32_t code = dtype_code(k, "k");
    const int64_t R = k.size(0), Hkv = k.size(1), D = k.size(2);
    if (given(v_o) != given(vc_o)) fail(PyExc_ValueError, "v and v_cache come together");
    if (fp4 && !given(v_o)) fail(PyExc_ValueError, "a 4-bit cache has v rows");
    const int64_t k_stride = checked_rows(k, "k", type, dev, R, Hkv, D);
    const at::Tensor* const v = given(v_o) ? &tensor_of(v_o, "v") : nullptr;
    const int64_t v_stride = v ? checked_rows(*v, "v", type, dev, R, Hkv, D) : 0;
    const at::Tensor& slots = checked(slots_o, "slots", at::kInt, dev, {R});
    const int32_t* pos = nullptr;
    if (given(pos_o)) pos = static_cast<const int32_t*>(checked(pos_o, "positions", at::kInt, dev, {R}).data_ptr());
    else if (given(table)) fail(PyExc_ValueError, "positions are needed with a rope table");
    qsa_rope_spec spec;
    const qsa_rope_spec* const s = spec_of(table, layout, offset, 0, &spec);
    Launch on(dev, stream);
    const int64_t S = ranked(kc_o, "k_cache", 3).size(0);
    const at::ScalarType cache_type = fp4 ? at::kByte : type;
    const int64_t width = fp4 ? D / 2 : D;
    const at::Tensor& kc = checked(kc_o, "k_cache", cache_type, dev, {S, Hkv, width});
    const at::Tensor* const vc = v ? &checked(vc_o, "v_cache", cache_type, dev, {S, Hkv, width}) : nullptr;
    int64_t Hq = 0, q_stride = 0, q_out_stride = 0;
    const at::Tensor* q = nullptr;
    at::Tensor q_out;
    if (given(q_o)) {
      q = &ranked(q_o, "q", 3);
      Hq = q->size(1);
      q_stride = checked_rows(*q, "q", type, dev, R, Hq, D);
      q_out = given(q_out_o) ? tensor_of(q_out_o, "q_out") : on.empty({R, Hq, D}, type);
      q_out_stride = checked_rows(q_out, "q_out", type, dev, R, Hq, D);
    }
    const int32_t hq = int32_of(Hq, "query heads"), hkv = int32_of(Hkv, "KV heads"), dim = int32_of(D, "head dim");
    if (fp4) {
      auto bytes = [](const at::Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); };
      uint8_t* const ks = bytes(checked(ks_o, "k_scale", at::kByte, dev, {S, Hkv, D / 16}));
      uint8_t* const vs = bytes(checked(vs_o, "v_scale", at::kByte, dev, {S, Hkv, D / 16}));
      void* const k_seen = given(k_seen_o) ? checked(k_seen_o, "k_seen", type, dev, {R, Hkv, D}).data_ptr() : nullptr;
      void* const v_seen = given(v_seen_o) ? checked(v_seen_o, "v_seen", type, dev, {R, Hkv, D}).data_ptr() : nullptr;
      if (R > 0)
        check_status(qsa_rope_append_fp4(q ? q->data_ptr() : nullptr, q ? q_out.data_ptr() : nullptr, k.data_ptr(),
                                         v->data_ptr(), kc.data_ptr(), ks, vc->data_ptr(), vs, kg, vg, k_seen, v_seen, pos,
                                         static_cast<const int32_t*>(slots.data_ptr()), s, R, S, hq, hkv, dim, q_stride,
                                         q_out_stride, k_stride, v_stride, code, on.stream()),
                     "qsa_rope_append_fp4");
    } else if (R > 0) {
      check_status(qsa_rope_append(q ? q->data_ptr() : nullptr, q ? q_out.data_ptr() : nullptr, k.data_ptr(),
                                   v ? v->data_ptr() : nullptr, kc.data_ptr(), v ? vc->data_ptr() : nullptr, pos,
                                   static_cast<const int32_t*>(slots.data_ptr()), s, R, S, hq, hkv, dim, q_stride,
                                   q_out_stride, k_stride, v_stride, code, on.stream()),
                   "qsa_rope_append");
    }
    if (!q) Py_RETURN_NONE;
    return given(q_out_o) ? Py_NewRef(q_out_o) : THPVariable_Wrap(q_out);
  });
}
PyObject* rope_append(PyObject*, PyObject* args, PyObject* kw) { return append(args, kw, false); }
PyObject* rope_append_fp4(PyObject*, PyObject* args, PyObject* kw) { return append(args, kw, true); }

PyObject* out_and_lse(PyObject* out_o, const at::Tensor& out, PyObject* lse_o, const at::Tensor& lse) {
  PyObject* const pair = PyTuple_New(2);
  if (!pair) throw PythonError();
  PyTuple_SET_ITEM(pair, 0, given(out_o) ? Py_NewRef(out_o) : THPVariable_Wrap(out));
  PyTuple_SET_ITEM(pair, 1, given(lse_o) ? Py_NewRef(lse_o) : lse.defined() ? THPVariable_Wrap(lse) : Py_NewRef(Py_None));
  return pair;
}

PyObject* window(PyObject* args, PyObject* kw, bool fp4) {
  static const char* names[] = {"q", "k_cache", "v_cache", "cu_seqlens_q", "kv_lens", "page_table", "page_size",
                                "scale", "window", "n_sink", "out", "lse", "want_lse", "workspace", "stream", nullptr};
  static const char* names4[] = {"q", "k_cache", "k_scale", "v_cache", "v_scale", "cu_seqlens_q", "kv_lens",
                                 "page_table", "page_size", "scale", "k_global", "v_global", "window", "n_sink", "out",
                                 "lse", "want_lse", "workspace", "stream", nullptr};
  PyObject *q_o, *kc_o, *vc_o, *ks_o = nullptr, *vs_o = nullptr, *cu_o, *kv_o, *table_o;
  PyObject *out_o = nullptr, *lse_o = nullptr, *ws_o = nullptr, *stream = nullptr;
  long long page_size, win = 0, sink = 0;
  float scale, kg = 1.0f, vg = 1.0f;
  int want_lse = 1;
  const int ok =
      fp4 ? PyArg_ParseTupleAndKeywords(args, kw, "OOOOOOOOLf|$ffLLOOpOO:window_attention_fp4_paged",
                                        const_cast<char**>(names4), &q_o, &kc_o, &ks_o, &vc_o, &vs_o, &cu_o, &kv_o,
                                        &table_o, &page_size, &scale, &kg, &vg, &win, &sink, &out_o, &lse_o, &want_lse,
                                        &ws_o, &stream)
          : PyArg_ParseTupleAndKeywords(args, kw, "OOOOOOLf|$LLOOpOO:window_attention_paged", const_cast<char**>(names),
                                        &q_o, &kc_o, &vc_o, &cu_o, &kv_o, &table_o, &page_size, &scale, &win, &sink,
                                        &out_o, &lse_o, &want_lse, &ws_o, &stream);
  if (!ok) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& q = ranked(q_o, "q", 3);
    const c10::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    const int32_t code = dtype_code(q, "q");
    const int64_t R = q.size(0), Hq = q.size(1), D = q.size(2);
    const int64_t S = ranked(kc_o, "k_cache", 3).size(0), Hkv = ranked(kc_o, "k_cache", 3).size(1);
    const int64_t n = ranked(table_o, "page_table", 2).size(0), ppr = ranked(table_o, "page_table", 2).size(1);
    checked(q_o, "q", type, dev, {R, Hq, D});
    const at::ScalarType cache_type = fp4 ? at::kByte : type;
    const int64_t width = fp4 ? D / 2 : D;
    const at::Tensor& kc = checked(kc_o, "k_cache", cache_type, dev, {S, Hkv, width});
    const at::Tensor& vc = checked(vc_o, "v_cache", cache_type, dev, {S, Hkv, width});
    const at::Tensor& table = checked(table_o, "page_table", at::kInt, dev, {n, ppr});
    const at::Tensor& cu = checked(cu_o, "cu_seqlens_q", at::kInt, dev, {n + 1});
    const at::Tensor& kv = checked(kv_o, "kv_lens", at::kInt, dev, {n});
    if (page_size < 1 || S % page_size != 0)
      fail(PyExc_ValueError, "the caches' " + std::to_string(S) + " slots are not whole pages of " + std::to_string(page_size));
    Launch on(dev, stream);
    const at::Tensor out = given(out_o) ? checked(out_o, "out", type, dev, {R, Hq, D}) : on.empty({R, Hq, D}, type);
    at::Tensor lse;
    if (given(lse_o)) lse = checked(lse_o, "lse", at::kFloat, dev, {R, Hq});
    else if (want_lse) lse = on.empty({R, Hq}, at::kFloat);
    const int32_t nr = int32_of(n, "n_requests"), pr = int32_of(ppr, "pages_per_req"), ps = int32_of(page_size, "page_size");
    const int32_t hq = int32_of(Hq, "query heads"), hkv = int32_of(Hkv, "KV heads"), dim = int32_of(D, "head dim");
    const int32_t w = int32_of(win, "window"), k = int32_of(sink, "n_sink");
    at::Tensor ws;
    size_t ws_bytes = 0;
    if (given(ws_o)) {
      ws = tensor_of(ws_o, "workspace");
      if (ws.device() != dev || !ws.is_contiguous())
        fail(PyExc_ValueError, "workspace must be contiguous and on " + dev.str());
      ws_bytes = ws.nbytes();
    } else if (R > 0) {
      ws_bytes = qsa_window_workspace_bytes(R, nr, pr, ps, hq, hkv, dim, w, k, fp4 ? 1 : 0, 0);
      if (ws_bytes > 0) ws = on.empty({static_cast<int64_t>(ws_bytes)}, at::kByte);
    }
    if (R > 0) {
      auto ints = [](const at::Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); };
      float* const lp = lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr;
      void* const wp = ws.defined() ? ws.data_ptr() : nullptr;
      if (fp4) {
        auto bytes = [](const at::Tensor& t) { return static_cast<const uint8_t*>(t.data_ptr()); };
        const uint8_t* const ks = bytes(checked(ks_o, "k_scale", at::kByte, dev, {S, Hkv, D / 16}));
        const uint8_t* const vs = bytes(checked(vs_o, "v_scale", at::kByte, dev, {S, Hkv, D / 16}));
        check_status(qsa_window_attention_fp4_paged(q.data_ptr(), kc.data_ptr(), ks, vc.data_ptr(), vs, kg, vg, ints(cu),
                                                    ints(kv), ints(table), out.data_ptr(), lp, R, nr, pr, ps, S / page_size,
                                                    hq, hkv, dim, scale, w, k, code, wp, ws_bytes, on.stream()),
                     "qsa_window_attention_fp4_paged");
      } else {
        check_status(qsa_window_attention_paged(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), ints(cu), ints(kv), ints(table),
                                                out.data_ptr(), lp, R, nr, pr, ps, S / page_size, hq, hkv, dim, scale, w, k,
                                                code, wp, ws_bytes, on.stream()),
                     "qsa_window_attention_paged");
      }
    }
    return out_and_lse(out_o, out, lse_o, lse);
  });
}
PyObject* window_attention_paged(PyObject*, PyObject* args, PyObject* kw) { return window(args, kw, false); }
PyObject* window_attention_fp4_paged(PyObject*, PyObject* args, PyObject* kw) { return window(args, kw, true); }

// The ragged batch over a paged cache that these calls share.
struct Paged {
  const at::Tensor *table, *cu, *kv;
  int32_t n, ppr, ps;
  Paged(PyObject* cu_o, PyObject* kv_o, PyObject* table_o, long long page_size, c10::Device dev) {
    const int64_t rows = ranked(table_o, "page_table", 2).size(0), width = ranked(table_o, "page_table", 2).size(1);
    table = &checked(table_o, "page_table", at::kInt, dev, {rows, width});
    cu = &checked(cu_o, "cu_seqlens_q", at::kInt, dev, {rows + 1});
    kv = &checked(kv_o, "kv_lens", at::kInt, dev, {rows});
    n = int32_of(rows, "n_requests");
    ppr = int32_of(width, "pages_per_req");
    ps = int32_of(page_size, "page_size");
  }
  // Pages of a cache of so many slots.
  int64_t pages_of(int64_t slots) const {
    if (ps < 1 || slots % ps != 0)
      fail(PyExc_ValueError, "the caches' " + std::to_string(slots) + " slots are not whole pages of " + std::to_string(ps));
    return slots / ps;
  }
};
const int32_t* ints(const at::Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); }

// The workspace that was given, or one of `need` bytes.
struct Workspace {
  at::Tensor t;
  Workspace(PyObject* o, size_t need, Launch& on, c10::Device dev) {
    if (given(o)) {
      t = tensor_of(o, "workspace");
      if (t.device() != dev || !t.is_contiguous())
        fail(PyExc_ValueError, "workspace must be contiguous and on " + dev.str());
    } else if (need > 0) {
      t = on.empty({static_cast<int64_t>(need)}, at::kByte);
    }
  }
  void* data() const { return t.defined() ? t.data_ptr() : nullptr; }
  size_t bytes() const { return t.defined() ? t.nbytes() : 0; }
};

PyObject* page_bounds(PyObject*, PyObject* args, PyObject* kw) {
  static const char* names[] = {"k_cache", "cu_seqlens_q", "kv_lens", "page_table", "page_size", "bounds", "stream", nullptr};
  PyObject *kc_o, *cu_o, *kv_o, *table_o, *bounds_o, *stream = nullptr;
  long long page_size;
  if (!PyArg_ParseTupleAndKeywords(args, kw, "OOOOLO|$O:page_bounds", const_cast<char**>(names), &kc_o, &cu_o, &kv_o,
                                   &table_o, &page_size, &bounds_o, &stream))
    return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& kc = ranked(kc_o, "k_cache", 3);
    const c10::Device dev = kc.device();
    const int32_t code = dtype_code(kc, "k_cache");
    const int64_t S = kc.size(0), H = kc.size(1), D = kc.size(2);
    checked(kc_o, "k_cache", kc.scalar_type(), dev, {S, H, D});
    const Paged b(cu_o, kv_o, table_o, page_size, dev);
    const int64_t pages = b.pages_of(S);
    const at::Tensor& bounds = checked(bounds_o, "bounds", kc.scalar_type(), dev, {pages, H, 2, D});
    Launch on(dev, stream);
    if (b.n > 0)
      check_status(qsa_page_bounds(kc.data_ptr(), ints(*b.cu), ints(*b.kv), ints(*b.table), bounds.data_ptr(), b.n, b.ppr,
                                   b.ps, pages, int32_of(H, "KV heads"), int32_of(D, "head dim"), code, on.stream()),
                   "qsa_page_bounds");
    return Py_NewRef(bounds_o);
  });
}

PyObject* page_select(PyObject*, PyObject* args, PyObject* kw) {
  static const char* names[] = {"q", "bounds", "cu_seqlens_q", "kv_lens", "page_table", "page_size", "n_select", "n_first",
                                "n_last", "out", "workspace", "stream", nullptr};
  PyObject *q_o, *bounds_o, *cu_o, *kv_o, *table_o, *out_o = nullptr, *ws_o = nullptr, *stream = nullptr;
  long long page_size, n_select, n_first = 1, n_last = 1;
  if (!PyArg_ParseTupleAndKeywords(args, kw, "OOOOOLL|$LLOOO:page_select", const_cast<char**>(names), &q_o, &bounds_o,
                                   &cu_o, &kv_o, &table_o, &page_size, &n_select, &n_first, &n_last, &out_o, &ws_o, &stream))
    return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& q = ranked(q_o, "q", 3);
    const c10::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    const int32_t code = dtype_code(q, "q");
    const int64_t R = q.size(0), Hq = q.size(1), D = q.size(2);
    checked(q_o, "q", type, dev, {R, Hq, D});
    const int64_t pages = ranked(bounds_o, "bounds", 4).size(0), H = ranked(bounds_o, "bounds", 4).size(1);
    const at::Tensor& bounds = checked(bounds_o, "bounds", type, dev, {pages, H, 2, D});
    const Paged b(cu_o, kv_o, table_o, page_size, dev);
    const int32_t k = int32_of(n_select, "n_select"), first = int32_of(n_first, "n_first"), last = int32_of(n_last, "n_last");
    if (k < 1) fail(PyExc_ValueError, "n_select must be at least 1");
    const int32_t hq = int32_of(Hq, "query heads"), hkv = int32_of(H, "KV heads"), dim = int32_of(D, "head dim");
    Launch on(dev, stream);
    const at::Tensor out = given(out_o) ? checked(out_o, "out", at::kInt, dev, {R, H, n_select}) : on.empty({R, H, n_select}, at::kInt);
    if (R > 0) {
      const Workspace ws(ws_o, given(ws_o) ? 0 : qsa_page_select_workspace_bytes(R, b.n, b.ppr, hq, hkv, dim), on, dev);
      check_status(qsa_page_select(q.data_ptr(), bounds.data_ptr(), ints(*b.cu), ints(*b.kv), ints(*b.table),
                                   static_cast<int32_t*>(out.data_ptr()), R, b.n, b.ppr, b.ps, pages, hq, hkv, dim, k, first,
                                   last, code, ws.data(), ws.bytes(), on.stream()),
                   "qsa_page_select");
    }
    return given(out_o) ? Py_NewRef(out_o) : THPVariable_Wrap(out);
  });
}

// selected_attention_paged (with the pages of each row) and prefix_attention_paged (with groups of requests).
PyObject* context_attention(PyObject* args, PyObject* kw, bool prefix) {
  static const char* names_s[] = {"q", "k_cache", "v_cache", "pages", "cu_seqlens_q", "kv_lens", "page_table", "page_size",
                                  "scale", "out", "lse", "want_lse", "workspace", "stream", nullptr};
  static const char* names_p[] = {"q", "k_cache", "v_cache", "cu_seqlens_q", "kv_lens", "page_table", "page_size", "scale",
                                  "cu_groups", "prefix_lens", "out", "lse", "want_lse", "workspace", "stream", nullptr};
  PyObject *q_o, *kc_o, *vc_o, *pages_o = nullptr, *cu_o, *kv_o, *table_o, *groups_o = nullptr, *prefix_o = nullptr;
  PyObject *out_o = nullptr, *lse_o = nullptr, *ws_o = nullptr, *stream = nullptr;
  long long page_size;
  float scale;
  int want_lse = 1;
  const int ok =
      prefix ? PyArg_ParseTupleAndKeywords(args, kw, "OOOOOOLfOO|$OOpOO:prefix_attention_paged", const_cast<char**>(names_p),
                                           &q_o, &kc_o, &vc_o, &cu_o, &kv_o, &table_o, &page_size, &scale, &groups_o,
                                           &prefix_o, &out_o, &lse_o, &want_lse, &ws_o, &stream)
             : PyArg_ParseTupleAndKeywords(args, kw, "OOOOOOOLf|$OOpOO:selected_attention_paged", const_cast<char**>(names_s),
                                           &q_o, &kc_o, &vc_o, &pages_o, &cu_o, &kv_o, &table_o, &page_size, &scale, &out_o,
                                           &lse_o, &want_lse, &ws_o, &stream);
  if (!ok) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& q = ranked(q_o, "q", 3);
    const c10::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    const int32_t code = dtype_code(q, "q");
    const int64_t R = q.size(0), Hq = q.size(1), D = q.size(2);
    const int64_t S = ranked(kc_o, "k_cache", 3).size(0), H = ranked(kc_o, "k_cache", 3).size(1);
    checked(q_o, "q", type, dev, {R, Hq, D});
    const at::Tensor& kc = checked(kc_o, "k_cache", type, dev, {S, H, D});
    const at::Tensor& vc = checked(vc_o, "v_cache", type, dev, {S, H, D});
    const Paged b(cu_o, kv_o, table_o, page_size, dev);
    const int64_t n_pages = b.pages_of(S);
    const int32_t hq = int32_of(Hq, "query heads"), hkv = int32_of(H, "KV heads"), dim = int32_of(D, "head dim");
    const at::Tensor *pages = nullptr, *groups = nullptr, *lens = nullptr;
    int32_t k = 0, n_groups = 0;
    if (prefix) {
      const int64_t G = ranked(prefix_o, "prefix_lens", 1).size(0);
      lens = &checked(prefix_o, "prefix_lens", at::kInt, dev, {G});
      groups = &checked(groups_o, "cu_groups", at::kInt, dev, {G + 1});
      n_groups = int32_of(G, "n_groups");
    } else {
      const int64_t K = ranked(pages_o, "pages", 3).size(2);
      pages = &checked(pages_o, "pages", at::kInt, dev, {R, H, K});
      k = int32_of(K, "n_select");
    }
    Launch on(dev, stream);
    const at::Tensor out = given(out_o) ? checked(out_o, "out", type, dev, {R, Hq, D}) : on.empty({R, Hq, D}, type);
    at::Tensor lse;
    if (given(lse_o)) lse = checked(lse_o, "lse", at::kFloat, dev, {R, Hq});
    else if (want_lse) lse = on.empty({R, Hq}, at::kFloat);
    if (R > 0) {
      size_t need = 0;
      if (!given(ws_o))
        need = prefix ? qsa_prefix_workspace_bytes(R, b.n, n_groups, b.ppr, b.ps, hq, hkv, dim, 0)
                      : qsa_selected_workspace_bytes(R, b.n, b.ppr, b.ps, k, hq, hkv, dim, 0);
      const Workspace ws(ws_o, need, on, dev);
      float* const lp = lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr;
      if (prefix)
        check_status(qsa_prefix_attention_paged(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), ints(*b.cu), ints(*b.kv),
                                                ints(*b.table), ints(*groups), ints(*lens), out.data_ptr(), lp, R, b.n,
                                                n_groups, b.ppr, b.ps, n_pages, hq, hkv, dim, scale, code, ws.data(),
                                                ws.bytes(), on.stream()),
                     "qsa_prefix_attention_paged");
      else
        check_status(qsa_selected_attention_paged(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), ints(*pages), ints(*b.cu),
                                                  ints(*b.kv), ints(*b.table), out.data_ptr(), lp, R, b.n, b.ppr, b.ps,
                                                  n_pages, k, hq, hkv, dim, scale, code, ws.data(), ws.bytes(), on.stream()),
                     "qsa_selected_attention_paged");
    }
    return out_and_lse(out_o, out, lse_o, lse);
  });
}
PyObject* selected_attention_paged(PyObject*, PyObject* args, PyObject* kw) { return context_attention(args, kw, false); }
PyObject* prefix_attention_paged(PyObject*, PyObject* args, PyObject* kw) { return context_attention(args, kw, true); }

// Signatures and documentation, as help() shows them.
constexpr char k_doc_page_plan[] = R"doc(page_plan(past_lens, new_lens, page_table, free_pages, free_head, page_size, max_rows, *, n_pages=0, free_head_out=None, cu_seqlens_q=None, kv_lens=None, positions=None, slots=None, shortfall=None, stream=None)
--

Page tables and slot maps of a step from its requests' lengths (qsa_page_plan).

past_lens, new_lens [n_requests] int32; page_table [n_requests, pages_per_req] int32 is
updated in place with pages taken from free_pages [n_free] int32, of which free_head [1] int32
are taken already; free_head_out = free_head updates it in place (None = a new tensor), and so does
kv_lens = past_lens with the lengths.
Returns cu_seqlens_q [n_requests + 1], kv_lens [n_requests], positions and slots [max_rows] (-1 on
rows past the last request), free_head [1] and shortfall [1], all int32.)doc";
constexpr char k_doc_rope[] = R"doc(rope(x, positions, table, *, layout="half", rot_offset=0, transpose=False, out=None, stream=None)
--

Rotates x [R, H, D] (bf16 or fp16, contiguous heads) to positions [R] int32 (qsa_rope).

transpose=True applies the transposed rotation, which takes the output's gradient to the
input's.  Rows with a negative position are not written.  out may be x.)doc";
constexpr char k_doc_rope_append[] = R"doc(rope_append(q, k, v, k_cache, v_cache, positions, slots, table, *, layout="half", rot_offset=0, q_out=None, stream=None)
--

Rotates q into q_out and k into the cache, and copies v into the cache (qsa_rope_append).

q [R, Hq, D] or None, k, v [R, Hkv, D] (bf16 or fp16, contiguous heads, any row stride); k_cache,
v_cache [n_slots, Hkv, D]; v and v_cache None for a cache of latent rows.  positions, slots [R]
int32: rows with a negative position are left out, rows with a slot outside the cache write no
cache row.  table None: nothing turns.  Returns q_out (a new tensor unless given; may be q).)doc";
constexpr char k_doc_rope_append_fp4[] = R"doc(rope_append_fp4(q, k, v, k_cache, k_scale, v_cache, v_scale, positions, slots, table, *, k_global=1.0, v_global=1.0, layout="half", rot_offset=0, q_out=None, k_seen=None, v_seen=None, stream=None)
--

rope_append into a cache held in 4 bits (qsa_rope_append_fp4): k_cache, v_cache [n_slots, Hkv,
D / 2] uint8 e2m1 pairs, k_scale, v_scale [n_slots, Hkv, D / 16] uint8 e4m3 block scales, k_global,
v_global the caches' fp32 scales.  k_seen, v_seen [R, Hkv, D] (optional) receive the values that the
cache now holds.  Returns q_out.)doc";
constexpr char k_doc_window_attention_paged[] = R"doc(window_attention_paged(q, k_cache, v_cache, cu_seqlens_q, kv_lens, page_table, page_size, scale, *, window=0, n_sink=0, out=None, lse=None, want_lse=True, workspace=None, stream=None)
--

Sliding-window attention with sink tokens over a paged cache (qsa_window_attention_paged).

q [R, Hq, D] bf16 or fp16 (D 64, 128 or 256); k_cache, v_cache [n_pages * page_size, Hkv, D] of the
same type; cu_seqlens_q [n_requests + 1], kv_lens [n_requests], page_table [n_requests,
pages_per_req] int32.  A row at position p sees the positions up to p that are among the last
`window` (0 = all) or the first n_sink.  Rows behind the last request are left as they were (in an
`out` that is not given: uninitialised).  Returns out [R, Hq, D] and lse [R, Hq] fp32 (None unless
wanted).)doc";
constexpr char k_doc_window_attention_fp4_paged[] = R"doc(window_attention_fp4_paged(q, k_cache, k_scale, v_cache, v_scale, cu_seqlens_q, kv_lens, page_table, page_size, scale, *, k_global=1.0, v_global=1.0, window=0, n_sink=0, out=None, lse=None, want_lse=True, workspace=None, stream=None)
--

window_attention_paged over a cache held in 4 bits, as rope_append_fp4 writes it
(qsa_window_attention_fp4_paged): k_cache, v_cache [n_pages * page_size, Hkv, D / 2] uint8, k_scale,
v_scale [n_pages * page_size, Hkv, D / 16] uint8, k_global, v_global the caches' fp32 scales.)doc";

constexpr char k_doc_page_bounds[] = R"doc(page_bounds(k_cache, cu_seqlens_q, kv_lens, page_table, page_size, bounds, *, stream=None)
--

Bounds of the pages that the step's rows reach, for page_select (qsa_page_bounds).

k_cache [n_pages * page_size, Hkv, D] bf16 or fp16 (D 64, 128 or 256), with the step's rows written;
cu_seqlens_q [n_requests + 1], kv_lens [n_requests], page_table [n_requests, pages_per_req] int32;
bounds [n_pages, Hkv, 2, D] of the cache's type: the smallest and the largest value of each key dim
over the page's filled positions.  Other pages are left as they were.  Returns bounds.)doc";
constexpr char k_doc_page_select[] = R"doc(page_select(q, bounds, cu_seqlens_q, kv_lens, page_table, page_size, n_select, *, n_first=1, n_last=1, out=None, workspace=None, stream=None)
--

Chooses up to n_select pages for every row and KV head by page_bounds' bounds (qsa_page_select).

q [R, Hq, D], bounds [n_pages, Hkv, 2, D] of one type; the batch as in window_attention_paged.  A row
takes the first n_first pages of its request, the last n_last up to its own, and of the others those
with the highest score, the most that q.k can be for a key of the page and a query head of the group;
ties go to the lower page.  Returns pages [R, Hkv, n_select] int32, places in the request's page
table in increasing order, then -1.  Rows behind the last request are left as they were.)doc";
constexpr char k_doc_selected_attention_paged[] = R"doc(selected_attention_paged(q, k_cache, v_cache, pages, cu_seqlens_q, kv_lens, page_table, page_size, scale, *, out=None, lse=None, want_lse=True, workspace=None, stream=None)
--

Attention of each row over the positions of its listed pages, up to its own
(qsa_selected_attention_paged).

pages [R, Hkv, n_select] int32 as page_select returns them, or in any order, with entries < 0 left
out; page_size a multiple of 8; the rest as in window_attention_paged.  Returns out [R, Hq, D] and
lse [R, Hq] fp32 (None unless wanted).)doc";
constexpr char k_doc_prefix_attention_paged[] = R"doc(prefix_attention_paged(q, k_cache, v_cache, cu_seqlens_q, kv_lens, page_table, page_size, scale, cu_groups, prefix_lens, *, out=None, lse=None, want_lse=True, workspace=None, stream=None)
--

Attention of a batch whose requests begin alike: window_attention_paged without a window, with the
shared keys read once for all requests of a group (qsa_prefix_attention_paged).

cu_groups [n_groups + 1] int32: group g is the requests cu_groups[g] .. cu_groups[g + 1] - 1;
prefix_lens [n_groups] int32: the positions below it hold the same keys for all of them that have rows
in the step.  The rest as in window_attention_paged.  Returns out [R, Hq, D] and lse [R, Hq] fp32 (None unless wanted).)doc";

#define QSA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_VARARGS | METH_KEYWORDS, k_doc_##f}
PyMethodDef methods[] = {QSA_METHOD(page_plan), QSA_METHOD(rope), QSA_METHOD(rope_append), QSA_METHOD(rope_append_fp4),
                         QSA_METHOD(window_attention_paged), QSA_METHOD(window_attention_fp4_paged),
                         QSA_METHOD(page_bounds), QSA_METHOD(page_select), QSA_METHOD(selected_attention_paged),
                         QSA_METHOD(prefix_attention_paged),
                         {"set_plan_type", set_plan_type, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&module); }
