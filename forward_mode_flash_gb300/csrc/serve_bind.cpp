// serve_bind.cpp -- the Python binding of the serving entry points (packed
// prompts, paged cache, chunks and single tokens over it) and of the norms and
// rotation of queries and keys as a native module.
//
// These calls are short: through ctypes one took 10 to 19 us of host time for
// 3 to 5 us on the GPU, from here 4 to 7.  This module reads the tensors' layouts,
// allocates the outputs and calls the C ABI in one step.  It checks nothing
// itself: a call is made only for layouts (types, devices, sizes, strides) that
// were `remember`ed after Python has checked them; for any other it returns None.
// So these times are of layouts that recur.  A call with another number of rows
// or another width of the block table than before is checked in full: 12 us
// (packed prompts), 14 (rows written), 27 (single tokens).  At 512 layouts all are
// forgotten.  Chunks take 12 to 15 us (two launches), rows appended 6 to 7.
//
// Entry points are passed as addresses, since a process may have two builds of
// the library loaded.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <unordered_map>
#include <vector>

#include "jvp_attn.h"

namespace {

// ------------------------------------------------------------------ layouts
struct Key {
  std::vector<int64_t> x;
  bool operator==(const Key& o) const { return x == o.x; }
};
struct KeyHash {
  size_t operator()(const Key& k) const {
    uint64_t h = 0x9E3779B97F4A7C15ull;
    for (int64_t v : k.x) h = (h ^ static_cast<uint64_t>(v)) * 0xD6E8FEB86659FD93ull, h ^= h >> 32;
    return static_cast<size_t>(h);
  }
};
struct Plan {
  int64_t workspace;  // bytes (single-token attention)
};
constexpr size_t kMaxPlans = 512;
// (Used with the GIL held.)
std::unordered_map<Key, Plan, KeyHash>& plans() {
  static auto* m = new std::unordered_map<Key, Plan, KeyHash>();
  return *m;
}

// Everything a call description depends on: all of a tensor but its address
// and values.
void add_layout(Key* key, const at::Tensor* t) {
  if (!t) {
    key->x.push_back(-1);
    return;
  }
  const auto sizes = t->sizes();
  const auto strides = t->strides();
  key->x.push_back(static_cast<int64_t>(t->scalar_type()) |
                   static_cast<int64_t>(t->device().type()) << 8 |
                   static_cast<int64_t>(t->device().index() & 0xFF) << 16 |
                   static_cast<int64_t>(sizes.size()) << 24);
  key->x.insert(key->x.end(), sizes.begin(), sizes.end());
  key->x.insert(key->x.end(), strides.begin(), strides.end());
}

struct BadArgument {};  // a Python error is set

const at::Tensor* tensor(PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "expected a tensor, got %s", Py_TYPE(o)->tp_name);
    throw BadArgument();
  }
  return &THPVariable_Unpack(o);
}
// The tensors of a call, in the order of its arguments, and their key.
template <int N>
struct Tensors {
  const at::Tensor* t[N];
  Key key;
  Tensors(int64_t op, PyObject* const* args) {
    key.x.reserve(10 * N + 1);
    key.x.push_back(op);
    for (int i = 0; i < N; ++i) {
      t[i] = tensor(args[i]);
      add_layout(&key, t[i]);
    }
  }
  const Plan* plan() const {
    const auto it = plans().find(key);
    return it == plans().end() ? nullptr : &it->second;
  }
  const at::Tensor& operator[](int i) const { return *t[i]; }
};

// ------------------------------------------------------------------ descriptions
template <typename T = void>
T* data(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
int dtype_code(at::ScalarType t) {
  return t == at::kFloat     ? JVP_F32
         : t == at::kHalf    ? JVP_F16
         : t == at::kBFloat16 ? JVP_BF16
                              : JVP_E4M3;
}
jvp_strides_t row_strides(const at::Tensor& t) { return {0, t.stride(1), t.stride(0), 1}; }
jvp_strides_t token_strides(const at::Tensor& t) { return {t.stride(0), t.stride(1), 0, 1}; }
jvp_cache_t cache(const at::Tensor& k, const at::Tensor& v, const at::Tensor& table) {
  jvp_cache_t c{};
  c.pages = k.size(0), c.Hkv = k.size(1), c.page_size = k.size(2), c.D = k.size(3);
  c.B = table.size(0), c.max_pages = table.size(1), c.table_stride = table.stride(0);
  c.dtype = dtype_code(k.scalar_type());
  c.k_strides = {k.stride(0), k.stride(1), k.stride(2), 1};
  c.v_strides = {v.stride(0), v.stride(1), v.stride(2), 1};
  return c;
}
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType dtype, c10::Device device) {
  return at::empty(sizes, at::TensorOptions().dtype(dtype).device(device));
}

// ------------------------------------------------------------------ calls
template <typename F>
F* entry(PyObject* address) {
  void* p = PyLong_AsVoidPtr(address);
  if (!p) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no entry point");
    throw BadArgument();
  }
  return reinterpret_cast<F*>(p);
}
bool truth(PyObject* o) {
  const int b = PyObject_IsTrue(o);
  if (b < 0) throw BadArgument();
  return b != 0;
}
float scale_of(PyObject* o, int64_t D) {
  if (o == Py_None) return static_cast<float>(D > 0 ? 1.0 / std::sqrt(static_cast<double>(D)) : 1.0);
  const double s = PyFloat_AsDouble(o);
  if (s == -1.0 && PyErr_Occurred()) throw BadArgument();
  return static_cast<float>(s);
}
// Calls with the device current, on its current stream, without the GIL.
template <typename F>
int call(c10::Device device, F&& f) {
  const c10::cuda::CUDAGuard guard(device);
  void* stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = f(stream);
  Py_END_ALLOW_THREADS
  return st;
}
PyObject* none() { Py_RETURN_NONE; }
PyObject* result(int status, const at::Tensor& o, const at::Tensor& second, bool pair) {
  if (status != JVP_OK) return PyLong_FromLong(status);
  PyObject* a = THPVariable_Wrap(o);
  if (!pair || !a) return a;
  PyObject* b = THPVariable_Wrap(second);
  PyObject* t = b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_DECREF(a);
  Py_XDECREF(b);
  return t;
}
// Runs a method's body; C++ exceptions become Python ones.
template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F&& f) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", wanted, given);
    return nullptr;
  }
  try {
    return f();
  } catch (const BadArgument&) {
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

enum Op : int64_t { kPacked, kWrite, kRead, kDecode, kRope, kRopeBwd, kAppend, kChunk };

// remember(op, workspace bytes, tensors ...): the layouts of these arguments
// have been checked.
PyObject* remember(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, n < 2 ? 2 : n, [&]() -> PyObject* {
    Key key;
    key.x.push_back(PyLong_AsLongLong(a[0]));
    if (PyErr_Occurred()) throw BadArgument();
    const int64_t bytes = PyLong_AsLongLong(a[1]);
    if (PyErr_Occurred()) throw BadArgument();
    for (Py_ssize_t i = 2; i < n; ++i) add_layout(&key, tensor(a[i]));
    if (plans().size() >= kMaxPlans) plans().clear();
    plans()[std::move(key)] = Plan{bytes};
    return none();
  });
}

// packed(entry, q, k, v, cu_seqlens, out, is_causal, scale, return_lse)
PyObject* packed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const Tensors<5> t(kPacked, a + 1);
    if (!t.plan()) return none();
    auto* f = entry<decltype(jvp_attn_fwd_packed)>(a[0]);
    const bool causal = truth(a[6]), want_lse = truth(a[8]);
    const at::Tensor &q = t[0], &k = t[1], &v = t[2], &cu = t[3];
    const jvp_packed_shape_t shape{q.size(0), cu.size(0) - 1, q.size(1), k.size(1), q.size(2)};
    const float scale = scale_of(a[7], shape.D);
    const at::Tensor o = t.t[4] ? t[4] : empty(q.sizes(), q.scalar_type(), q.device());
    at::Tensor lse;
    if (want_lse) lse = empty({shape.H, shape.T}, at::kFloat, q.device());
    const jvp_strides_t in[3] = {row_strides(q), row_strides(k), row_strides(v)};
    const jvp_strides_t out = row_strides(o);
    const int st = call(q.device(), [&](void* stream) {
      return f(&shape, static_cast<jvp_dtype_t>(dtype_code(q.scalar_type())), data(&q), data(&k),
               data(&v), in, data<int32_t>(&cu), causal ? 1 : 0, scale, data(&o), &out,
               want_lse ? data<float>(&lse) : nullptr, stream);
    });
    return result(st, o, lse, want_lse);
  });
}

// write(entry, k, v, k_cache, v_cache, block_table, start_pos, cu_seqlens,
//       k_scale, v_scale): the status
PyObject* write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Tensors<9> t(kWrite, a + 1);
    if (!t.plan()) return none();
    auto* f = entry<decltype(jvp_attn_cache_write)>(a[0]);
    const at::Tensor &k = t[0], &v = t[1];
    const jvp_cache_t c = cache(t[2], t[3], t[4]);
    const jvp_strides_t in[2] = {row_strides(k), row_strides(v)};
    return PyLong_FromLong(call(k.device(), [&](void* stream) {
      return f(&c, static_cast<jvp_dtype_t>(dtype_code(k.scalar_type())), k.size(0), data(&k),
               data(&v), in, data<int32_t>(&t[4]), data<int32_t>(t.t[5]), data<int32_t>(t.t[6]),
               data(&t[2]), data(&t[3]), data<uint8_t>(t.t[7]), data<uint8_t>(t.t[8]), stream);
    }));
  });
}

// read(entry, k, v, k_cache, ... as write): the status
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Tensors<9> t(kRead, a + 1);
    if (!t.plan()) return none();
    auto* f = entry<decltype(jvp_attn_cache_read)>(a[0]);
    const at::Tensor &k = t[0], &v = t[1];
    const jvp_cache_t c = cache(t[2], t[3], t[4]);
    const jvp_strides_t out[2] = {row_strides(k), row_strides(v)};
    return PyLong_FromLong(call(k.device(), [&](void* stream) {
      return f(&c, static_cast<jvp_dtype_t>(dtype_code(k.scalar_type())), k.size(0), data(&t[2]),
               data(&t[3]), data<uint8_t>(t.t[7]), data<uint8_t>(t.t[8]), data<int32_t>(&t[4]),
               data<int32_t>(t.t[5]), data<int32_t>(t.t[6]), data(&k), data(&v), out, stream);
    }));
  });
}

// empty_rows(k_cache, rows, dtype): new k, v [rows, Hkv, D] for read, of the
// cache's type (bfloat16 for an e4m3 one) if dtype is None
PyObject* empty_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    const at::Tensor* c = tensor(a[0]);
    const int64_t rows = PyLong_AsLongLong(a[1]);
    if (rows == -1 && PyErr_Occurred()) throw BadArgument();
    if (!c || c->dim() != 4 || (a[2] != Py_None && !THPDtype_Check(a[2]))) {
      PyErr_SetString(PyExc_TypeError, "expected a cache [pages, Hkv, page_size, D] and a dtype");
      throw BadArgument();
    }
    const at::ScalarType t = a[2] != Py_None ? reinterpret_cast<THPDtype*>(a[2])->scalar_type
                             : c->scalar_type() == at::kFloat8_e4m3fn ? at::kBFloat16
                                                                      : c->scalar_type();
    const at::Tensor k = empty({rows, c->size(1), c->size(3)}, t, c->device());
    return result(JVP_OK, k, empty(k.sizes(), t, c->device()), true);
  });
}

// A single-token call through an entry point of type F; more: its window and sinks.
template <typename F, typename... More>
PyObject* decode_call(PyObject* const* a, PyObject* workspace, PyObject* scale_arg, PyObject* lse_arg,
                      More... more) {
  const Tensors<8> t(kDecode, a + 1);
  const Plan* plan = t.plan();
  if (!plan) return none();
  // (by value: an allocation may run Python code, which may remember layouts)
  const int64_t need = plan->workspace;
  auto* f = entry<F>(a[0]);
  const at::Tensor* given = tensor(workspace);
  const bool want_lse = truth(lse_arg);
  const at::Tensor &q = t[0], &kc = t[1], &vc = t[2], &table = t[3], &lens = t[4];
  const jvp_cache_t c = cache(kc, vc, table);
  const float scale = scale_of(scale_arg, c.D);
  const at::Tensor o = t.t[7] ? t[7] : empty(q.sizes(), q.scalar_type(), q.device());
  at::Tensor lse, ws;
  if (want_lse) lse = empty({q.size(0), q.size(1)}, at::kFloat, q.device());
  if (given) ws = *given;
  else if (need > 0) ws = empty({need}, at::kByte, q.device());
  const size_t bytes = ws.defined() ? ws.nbytes() : 0;
  const jvp_strides_t qs = token_strides(q), os = token_strides(o);
  const int st = call(q.device(), [&](void* stream) {
    return f(&c, q.size(1), static_cast<jvp_dtype_t>(dtype_code(q.scalar_type())), data(&q), &qs,
             data(&kc), data(&vc), data<uint8_t>(t.t[5]), data<uint8_t>(t.t[6]),
             data<int32_t>(&table), data<int32_t>(&lens), more..., scale, data(&o), &os,
             want_lse ? data<float>(&lse) : nullptr, ws.defined() ? data(&ws) : nullptr, bytes,
             stream);
  });
  return result(st, o, lse, want_lse);
}

// decode(entry, q, k_cache, v_cache, block_table, seq_lens, k_scale, v_scale,
//        out, workspace, scale, return_lse)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    return decode_call<decltype(jvp_attn_decode)>(a, a[9], a[10], a[11]);
  });
}

int64_t integer(PyObject* o) {
  const int64_t x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw BadArgument();
  return x;
}

// decode_window(entry, q, ... out, workspace as decode, window, sinks, scale, return_lse)
PyObject* decode_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    return decode_call<decltype(jvp_attn_decode_window)>(a, a[9], a[12], a[13], integer(a[10]),
                                                         integer(a[11]));
  });
}

// chunk(entry, q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, k_scale,
//       v_scale, out, workspace, window, sinks, scale, return_lse)
PyObject* chunk(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    const Tensors<9> t(kChunk, a + 1);
    const Plan* plan = t.plan();
    if (!plan) return none();
    const int64_t need = plan->workspace;  // (by value, as in decode)
    auto* f = entry<decltype(jvp_attn_chunk)>(a[0]);
    const at::Tensor* given = tensor(a[10]);
    const int64_t window = integer(a[11]), sinks = integer(a[12]);
    const bool want_lse = truth(a[14]);
    const at::Tensor &q = t[0], &kc = t[1], &vc = t[2], &table = t[3];
    const jvp_cache_t c = cache(kc, vc, table);
    const float scale = scale_of(a[13], c.D);
    const at::Tensor o = t.t[8] ? t[8] : empty(q.sizes(), q.scalar_type(), q.device());
    at::Tensor lse, ws;
    if (want_lse) lse = empty({q.size(1), q.size(0)}, at::kFloat, q.device());
    if (given) ws = *given;
    else if (need > 0) ws = empty({need}, at::kByte, q.device());
    const size_t bytes = ws.defined() ? ws.nbytes() : 0;
    const jvp_strides_t qs = row_strides(q), os = row_strides(o);
    const int st = call(q.device(), [&](void* stream) {
      return f(&c, q.size(1), static_cast<jvp_dtype_t>(dtype_code(q.scalar_type())), q.size(0),
               data(&q), &qs, data(&kc), data(&vc), data<uint8_t>(t.t[6]), data<uint8_t>(t.t[7]),
               data<int32_t>(&table), data<int32_t>(t.t[4]), data<int32_t>(t.t[5]), window, sinks,
               scale, data(&o), &os, want_lse ? data<float>(&lse) : nullptr,
               ws.defined() ? data(&ws) : nullptr, bytes, stream);
    });
    return result(st, o, lse, want_lse);
  });
}

// The angles and norm weights of a call: tensors (or none) and numbers.
jvp_rope_t rope_of(const at::Tensor* table, const at::Tensor* qw, const at::Tensor* kw, PyObject* eps,
                   PyObject* interleaved) {
  jvp_rope_t r{};
  if (table) r.table = data<float>(table), r.rows = table->size(0), r.dim = table->size(1);
  r.interleaved = truth(interleaved) ? 1 : 0;
  r.q_weight = data(qw), r.k_weight = data(kw);
  if (qw) r.weight_dtype = dtype_code(qw->scalar_type());
  const double e = PyFloat_AsDouble(eps);
  if (e == -1.0 && PyErr_Occurred()) throw BadArgument();
  r.eps = static_cast<float>(e);
  return r;
}
jvp_strides_t strides_of(const at::Tensor* t) {
  if (!t) return {0, 0, 0, 1};
  return {t->stride(0), t->stride(1), t->stride(2), 1};
}
jvp_shape_t dense_shape(const at::Tensor& q, const at::Tensor& k) {
  return {q.size(0), q.size(1), q.size(2), q.size(2), q.size(3), k.size(1)};
}
PyObject* results(int status, const std::vector<at::Tensor>& out) {
  if (status != JVP_OK) return PyLong_FromLong(status);
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(out.size()));
  for (size_t i = 0; t && i < out.size(); ++i) {
    PyObject* x = out[i].defined() ? THPVariable_Wrap(out[i]) : none();
    if (!x) {
      Py_DECREF(t);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, static_cast<Py_ssize_t>(i), x);
  }
  return t;
}

// rope(entry, q, k, dq, dk, table, positions, q_weight, k_weight, eps, interleaved):
// the outputs for q and k (and, given dq and dk, for these)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const Tensors<8> t(kRope, a + 1);
    if (!t.plan()) return none();
    auto* f = entry<decltype(jvp_attn_norm_rope)>(a[0]);
    const at::Tensor &q = t[0], &k = t[1];
    const jvp_rope_t r = rope_of(t.t[4], t.t[6], t.t[7], a[9], a[10]);
    const jvp_shape_t shape = dense_shape(q, k);
    std::vector<at::Tensor> out;
    jvp_strides_t in[4], os[4];
    void* y[4] = {};
    for (int i = 0; i < (t.t[2] ? 4 : 2); ++i)
      out.push_back(empty(t[i].sizes(), q.scalar_type(), q.device()));
    for (size_t i = 0; i < 4; ++i) {
      const bool on = i < out.size();
      os[i] = strides_of(on ? &out[i] : nullptr), y[i] = on ? data(&out[i]) : nullptr;
      in[i] = strides_of(t.t[i]);
    }
    const at::Tensor* at = t.t[5];
    return results(call(q.device(), [&](void* stream) {
      return f(&shape, static_cast<jvp_dtype_t>(dtype_code(q.scalar_type())), &r, data<int32_t>(at),
               at ? at->stride(0) : 0, data(&q), data(&k), data(t.t[2]), data(t.t[3]), in, y[0],
               y[1], y[2], y[3], os, stream);
    }), out);
  });
}

// rope_bwd(entry, q, k, dq, dk, g_q, g_k, g_dq, g_dk, table, positions, q_weight,
//          k_weight, eps, interleaved): gradients of q, k (, dq, dk), the weights
PyObject* rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    const Tensors<12> t(kRopeBwd, a + 1);
    const Plan* plan = t.plan();
    if (!plan) return none();
    const int64_t need = plan->workspace;  // (by value, as in decode)
    auto* f = entry<decltype(jvp_attn_norm_rope_bwd)>(a[0]);
    const at::Tensor &q = t[0], &k = t[1];
    const jvp_rope_t r = rope_of(t.t[8], t.t[10], t.t[11], a[13], a[14]);
    const jvp_shape_t shape = dense_shape(q, k);
    const size_t rows = t.t[2] ? 4 : 2;
    std::vector<at::Tensor> out;
    for (size_t i = 0; i < rows; ++i)
      out.push_back(empty(t[static_cast<int>(i)].sizes(), q.scalar_type(), q.device()));
    at::Tensor ws;
    for (int i = 0; i < 2; ++i)
      out.push_back(t.t[10] ? empty({shape.D}, at::kFloat, q.device()) : at::Tensor());
    if (t.t[10]) ws = empty({need}, at::kByte, q.device());
    jvp_strides_t in[8], os[4];
    void* y[4] = {};
    for (int i = 0; i < 8; ++i) in[i] = strides_of(t.t[i]);
    for (size_t i = 0; i < 4; ++i)
      os[i] = strides_of(i < rows ? &out[i] : nullptr), y[i] = i < rows ? data(&out[i]) : nullptr;
    float* gw[2] = {};
    for (int i = 0; i < 2; ++i) gw[i] = out[rows + i].defined() ? data<float>(&out[rows + i]) : nullptr;
    const at::Tensor* at = t.t[9];
    return results(call(q.device(), [&](void* stream) {
      return f(&shape, static_cast<jvp_dtype_t>(dtype_code(q.scalar_type())), &r, data<int32_t>(at),
               at ? at->stride(0) : 0, data(&q), data(&k), data(t.t[2]), data(t.t[3]), data(t.t[4]),
               data(t.t[5]), data(t.t[6]), data(t.t[7]), in, y[0], y[1], y[2], y[3], os, gw[0],
               gw[1], ws.defined() ? data(&ws) : nullptr, ws.defined() ? ws.nbytes() : 0, stream);
    }), out);
  });
}

// append(entry, q, k, v, k_cache, v_cache, block_table, table, start_pos, cu_seqlens,
//        q_weight, k_weight, k_scale, v_scale, out, eps, interleaved): the queries
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    const Tensors<14> t(kAppend, a + 1);
    if (!t.plan()) return none();
    auto* f = entry<decltype(jvp_attn_cache_append)>(a[0]);
    const at::Tensor &q = t[0], &k = t[1], &v = t[2];
    const jvp_cache_t c = cache(t[3], t[4], t[5]);
    const jvp_rope_t r = rope_of(t.t[6], t.t[9], t.t[10], a[15], a[16]);
    const at::Tensor o = t.t[13] ? t[13] : empty(q.sizes(), q.scalar_type(), q.device());
    const jvp_strides_t in[3] = {row_strides(q), row_strides(k), row_strides(v)};
    const jvp_strides_t os = row_strides(o);
    const int st = call(q.device(), [&](void* stream) {
      return f(&c, q.size(1), static_cast<jvp_dtype_t>(dtype_code(q.scalar_type())), q.size(0),
               data(&q), data(&k), data(&v), in, &r, data<int32_t>(&t[5]), data<int32_t>(t.t[7]),
               data<int32_t>(t.t[8]), data(&o), &os, data(&t[3]), data(&t[4]),
               data<uint8_t>(t.t[11]), data<uint8_t>(t.t[12]), stream);
    });
    return result(st, o, o, false);
  });
}

#define JVP_METHOD(f) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {JVP_METHOD(remember),   JVP_METHOD(packed), JVP_METHOD(write),
                         JVP_METHOD(read),       JVP_METHOD(decode), JVP_METHOD(empty_rows),
                         JVP_METHOD(rope),       JVP_METHOD(rope_bwd), JVP_METHOD(append),
                         JVP_METHOD(decode_window), JVP_METHOD(chunk),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve_bind", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve_bind() {
  PyObject* m = PyModule_Create(&module);
  const struct { const char* name; Op op; } ops[] = {
      {"PACKED", kPacked}, {"WRITE", kWrite}, {"READ", kRead}, {"DECODE", kDecode},
      {"ROPE", kRope}, {"ROPE_BWD", kRopeBwd}, {"APPEND", kAppend}, {"CHUNK", kChunk}};
  for (const auto& o : ops)
    if (m && PyModule_AddIntConstant(m, o.name, o.op))
      Py_CLEAR(m);
  return m;
}
