// Argument marshalling of the bounded-memory operators for Python: checks that the tensors are what the
// configuration says and passes their pointers and the CUDA stream to the C entry points.  A call of these
// operators can be a few microseconds of device work, which the same checks in Python would double.
//
// Each function takes the arguments of the Python function of its name (see the package), raises ValueError
// for tensors that do not fit, and returns the C entry point's status.
#include <Python.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/mka.h"

namespace {

struct Refused : std::runtime_error {  // becomes a ValueError
  using std::runtime_error::runtime_error;
};
struct Raised {};  // a Python exception is set
// Lets other Python threads run during the call: a launch can wait for room in the stream's queue.  (The caller
// holds the arguments.)
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// The C structure inside a ctypes structure.
template <typename T>
const T* structure(PyObject* o, const char* what) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Raised();
  const bool fits = b.len == (Py_ssize_t)sizeof(T);
  const T* p = (const T*)b.buf;  // (a ctypes structure does not move while it lives)
  PyBuffer_Release(&b);
  if (!fits) throw Refused(std::string(what) + " is not the structure that this call takes");
  return p;
}
// A tensor; nullptr for None where that is allowed.
const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
int32_t to_i32(long long v, const char* name) {
  if (v != (int32_t)v) throw Refused(std::string(name) + " is out of range");
  return (int32_t)v;
}
[[noreturn]] void refuse(const at::Tensor& t, const char* name, const std::string& want) {
  std::ostringstream s;
  s << name << " must be " << want << ", not " << t.scalar_type() << " " << t.sizes() << " of strides " << t.strides();
  throw Refused(s.str());
}
std::string shape(std::initializer_list<long long> v) {
  std::string s = "[";
  for (long long x : v) s += (s.size() > 1 ? ", " : "") + std::to_string(x);
  return s + "]";
}

// Pointer of a contiguous tensor of that type and number of elements (null passes).
template <typename P = void>
P* dense(const at::Tensor* t, const char* name, at::ScalarType type, long long numel) {
  if (!t) return nullptr;
  if (t->scalar_type() != type || t->numel() != numel || !t->is_contiguous())
    refuse(*t, name, std::string("contiguous ") + c10::toString(type) + ", " + std::to_string(numel) + " elements");
  return (P*)t->data_ptr();
}
const int32_t* positions(const at::Tensor* t, const char* name, int32_t B) {
  return dense<const int32_t>(t, name, at::kInt, B);
}
size_t bytes(const at::Tensor& t) {
  if (!t.is_contiguous()) throw Refused("ws must be contiguous");
  return t.nbytes();
}

// The stream of a call on `ts` (null ones pass): they must live on the current device, and a stream other than
// the current one is recorded on them.
template <size_t N>
void* call_stream(PyObject* stream, const at::Tensor* const (&ts)[N]) {
  const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream();
  for (const at::Tensor* t : ts)
    if (t && (!t->is_cuda() || t->get_device() != current.device_index()))
      throw Refused("every tensor of the call must live on the current CUDA device (" +
                    std::to_string((int)current.device_index()) + ")");
  if (stream == Py_None) return (void*)current.stream();
  long long v[3];
  const char* names[3] = {"stream_id", "device_index", "device_type"};
  for (int i = 0; i < 3; ++i) {
    PyObject* a = PyObject_GetAttrString(stream, names[i]);
    if (!a) throw Raised();
    v[i] = PyLong_AsLongLong(a);
    Py_DECREF(a);
    if (v[i] == -1 && PyErr_Occurred()) throw Raised();
  }
  const c10::cuda::CUDAStream s =
      c10::cuda::CUDAStream(c10::Stream::unpack3(v[0], (c10::DeviceIndex)v[1], (c10::DeviceType)v[2]));
  if (s.device_index() != current.device_index()) throw Refused("the stream must be one of the current CUDA device");
  if (s != current)
    for (const at::Tensor* t : ts)
      if (t) t->record_stream(s);
  return (void*)s.stream();
}

// The tensors of an 8-bit cache, checked against its configuration.
struct Cache {
  const at::Tensor* t[4];
  const mka_kv8_cache* c;
};
Cache cache_of(PyObject* o, const mka_kv8_config& c) {
  Cache x;
  x.c = structure<mka_kv8_cache>(o, "cache");
  PyObject* tensors = PyObject_GetAttrString(o, "tensors");
  if (!tensors) throw Raised();
  const bool four = PyTuple_Check(tensors) && PyTuple_GET_SIZE(tensors) == 4;
  for (int i = 0; four && i < 4; ++i) x.t[i] = tensor(PyTuple_GET_ITEM(tensors, i), "a cache tensor");
  Py_DECREF(tensors);  // (the cache object keeps them)
  if (!four) throw Refused("cache must come from kv8_cache()");
  const long long nb = c.block > 0 ? ((long long)c.max_positions + c.block - 1) / c.block : 0;
  const int64_t codes[4] = {c.batch, c.n_kv_heads, c.max_positions, c.d_head}, scales[3] = {c.batch, c.n_kv_heads, nb};
  if (x.t[0]->sizes() != at::IntArrayRef(codes, 4))
    refuse(*x.t[0], "the cache's codes", shape({c.batch, c.n_kv_heads, c.max_positions, c.d_head}));
  if (c.block > 0 && x.t[2]->sizes() != at::IntArrayRef(scales, 3))
    refuse(*x.t[2], "the cache's scales", shape({c.batch, c.n_kv_heads, nb}));
  return x;
}

// K/V rows [B, n, Hkv, dh] or [B, n, Hkv * dh], both alike.
struct Rows {
  int32_t n;
  int64_t row, batch;
};
Rows kv_rows(const mka_kv8_config& c, const at::Tensor& k, const at::Tensor& v, const char* name) {
  const at::ScalarType type = c.dtype == MKA_BF16 ? at::kBFloat16 : at::kFloat;
  const int64_t width = (int64_t)c.n_kv_heads * c.d_head;
  auto rows = [&](const at::Tensor& t) -> Rows {  // (the stride of a dimension of size 1 does not count)
    const auto s = t.sizes(), st = t.strides();
    bool ok = t.scalar_type() == type && s.size() >= 3 && s[0] == c.batch;
    if (ok && s.size() == 4) ok = s[2] == c.n_kv_heads && s[3] == c.d_head && st[3] == 1 && (c.n_kv_heads == 1 || st[2] == c.d_head);
    else if (ok) ok = s.size() == 3 && s[2] == width && st[2] == 1;
    if (!ok)
      refuse(t, name, std::string(c10::toString(type)) + " [" + std::to_string(c.batch) + ", n, " + std::to_string(c.n_kv_heads) +
                          ", " + std::to_string(c.d_head) + "] with contiguous rows, two tensors of the same type, shape and strides");
    return {to_i32(s[1], "n"), s[1] > 1 ? st[1] : width, c.batch > 1 ? st[0] : 0};
  };
  const Rows a = rows(k), b = rows(v);
  if (a.n != b.n || a.row != b.row || a.batch != b.batch) refuse(v, name, "two tensors of the same type, shape and strides");
  return a;
}

// Row stride of t [B, S, heads, dh] or [B, S, heads * dh] (see mka_attn_strides).
int32_t row_stride(const at::Tensor& t, const char* name, const mka_attn_config& c, int32_t heads) {
  const int64_t B = c.batch, S = c.seq, d = c.d_head, width = heads * d;
  const auto s = t.sizes(), st = t.strides();
  bool ok = t.scalar_type() == at::kBFloat16 && s.size() >= 3 && s[0] == B && s[1] == S;
  if (ok && s.size() == 4) ok = s[2] == heads && s[3] == d && st[3] == 1 && (heads == 1 || st[2] == d);
  else if (ok) ok = s.size() == 3 && s[2] == width && st[2] == 1;
  const int64_t ld = !ok ? 0 : S > 1 ? st[1] : B > 1 ? st[0] : width;
  if (!ok || (B > 1 && st[0] != S * ld))
    refuse(t, name, "BFloat16 " + shape({B, S, heads, d}) + " with contiguous rows, evenly spaced over the whole batch");
  return to_i32(ld, name);
}

// ---------------------------------------------------------------- the operators
int window_attention(PyObject* const* a) {  // c, q, k, v, lens, out, lse, stream
  const auto& c = *structure<mka_attn_config>(a[0], "c");
  const at::Tensor *q = tensor(a[1], "q"), *k = tensor(a[2], "k"), *v = tensor(a[3], "v"), *lens = tensor(a[4], "lens", true),
                   *out = tensor(a[5], "out"), *lse = tensor(a[6], "lse", true);
  const mka_attn_strides st = {row_stride(*q, "q", c, c.n_q_heads), row_stride(*k, "k", c, c.n_kv_heads),
                               row_stride(*v, "v", c, c.n_kv_heads), row_stride(*out, "out", c, c.n_q_heads), 0};
  const long long pad = ((long long)c.seq + 127) / 128 * 128;
  const int32_t* pl = positions(lens, "lens", c.batch);
  float* ps = dense<float>(lse, "lse", at::kFloat, (long long)c.batch * c.n_q_heads * pad);
  void* s = call_stream(a[7], {q, k, v, lens, out, lse});
  Unlocked unlocked;
  return mka_window_attention(&c, &st, q->data_ptr(), k->data_ptr(), v->data_ptr(), pl, out->data_ptr(), ps, s);
}

int window_attention_backward(PyObject* const* a) {  // c, q, k, v, out, lse, dout, lens, dq, dk, dv, ws, stream
  const auto& c = *structure<mka_attn_config>(a[0], "c");
  const at::Tensor *q = tensor(a[1], "q"), *k = tensor(a[2], "k"), *v = tensor(a[3], "v"), *out = tensor(a[4], "out"),
                   *lse = tensor(a[5], "lse"), *dout = tensor(a[6], "dout"), *lens = tensor(a[7], "lens", true),
                   *dq = tensor(a[8], "dq"), *dk = tensor(a[9], "dk"), *dv = tensor(a[10], "dv"), *ws = tensor(a[11], "ws");
  const mka_attn_strides st = {row_stride(*q, "q", c, c.n_q_heads), row_stride(*k, "k", c, c.n_kv_heads),
                               row_stride(*v, "v", c, c.n_kv_heads), row_stride(*out, "out", c, c.n_q_heads),
                               row_stride(*dout, "dout", c, c.n_q_heads)};
  const long long rows = (long long)c.batch * c.seq, pad = ((long long)c.seq + 127) / 128 * 128;
  const int32_t* pl = positions(lens, "lens", c.batch);
  const float* ps = dense<float>(lse, "lse", at::kFloat, (long long)c.batch * c.n_q_heads * pad);
  void* pq = dense(dq, "dq", at::kBFloat16, rows * c.n_q_heads * c.d_head);
  void* pk = dense(dk, "dk", at::kBFloat16, rows * c.n_kv_heads * c.d_head);
  void* pv = dense(dv, "dv", at::kBFloat16, rows * c.n_kv_heads * c.d_head);
  const size_t n = bytes(*ws);
  void* s = call_stream(a[12], {q, k, v, out, lse, dout, lens, dq, dk, dv, ws});
  Unlocked unlocked;
  return mka_window_attention_backward(&c, &st, q->data_ptr(), k->data_ptr(), v->data_ptr(), out->data_ptr(), ps,
                                       dout->data_ptr(), pl, pq, pk, pv, ws->data_ptr(), n, s);
}

int kv8_append(PyObject* const* a) {  // c, cache, k_new, v_new, pos, count, stream
  const auto& c = *structure<mka_kv8_config>(a[0], "c");
  const Cache x = cache_of(a[1], c);
  const at::Tensor *k = tensor(a[2], "k_new"), *v = tensor(a[3], "v_new"), *pos = tensor(a[4], "pos"),
                   *count = tensor(a[5], "count", true);
  const Rows r = kv_rows(c, *k, *v, "k_new, v_new");
  const int32_t *pp = positions(pos, "pos", c.batch), *pc = positions(count, "count", c.batch);
  void* s = call_stream(a[6], {k, v, pos, count, x.t[0], x.t[1], x.t[2], x.t[3]});
  Unlocked unlocked;
  return mka_kv8_append(&c, x.c, k->data_ptr(), v->data_ptr(), r.row, r.batch, r.n, pp, pc, s);
}

int kv8_read(PyObject* const* a) {  // c, cache, first, rows, k_out, v_out, stream
  const auto& c = *structure<mka_kv8_config>(a[0], "c");
  const Cache x = cache_of(a[1], c);
  const at::Tensor *first = tensor(a[2], "first", true), *rows = tensor(a[3], "rows", true), *k = tensor(a[4], "k_out"),
                   *v = tensor(a[5], "v_out");
  const Rows r = kv_rows(c, *k, *v, "k_out, v_out");
  const int32_t *pf = positions(first, "first", c.batch), *pr = positions(rows, "rows", c.batch);
  void* s = call_stream(a[6], {first, rows, k, v, x.t[0], x.t[1], x.t[2], x.t[3]});
  Unlocked unlocked;
  return mka_kv8_read(&c, x.c, pf, pr, r.n, k->data_ptr(), v->data_ptr(), r.row, r.batch, s);
}

int kv8_attention(PyObject* const* a) {  // c, cache, q, lens, out, weights, ws, stream
  const auto& c = *structure<mka_kv8_config>(a[0], "c");
  const Cache x = cache_of(a[1], c);
  const at::Tensor *q = tensor(a[2], "q"), *lens = tensor(a[3], "lens"), *out = tensor(a[4], "out"),
                   *weights = tensor(a[5], "weights", true), *ws = tensor(a[6], "ws");
  const at::ScalarType type = c.dtype == MKA_BF16 ? at::kBFloat16 : at::kFloat;
  const int32_t n = q->dim() >= 2 ? to_i32(q->size(1), "n") : 0;
  const long long numel = (long long)c.batch * n * c.n_q_heads * c.d_head;
  void *pq = dense(q, "q", type, numel), *po = dense(out, "out", type, numel);
  const int32_t* pl = positions(lens, "lens", c.batch);
  float* pw = dense<float>(weights, "weights", at::kFloat, (long long)c.batch * c.n_kv_heads * c.max_positions);
  const size_t nb = bytes(*ws);
  void* s = call_stream(a[7], {q, lens, out, weights, ws, x.t[0], x.t[1], x.t[2], x.t[3]});
  Unlocked unlocked;
  return mka_kv8_attention(&c, x.c, pq, n, pl, po, pw, ws->data_ptr(), nb, s);
}

int kv8_evict(PyObject* const* a) {  // c, cache, lens, weights, keep, first, recent, dst_c, dst, dst_lens, dst_weights, kept, ws, stream
  const auto &c = *structure<mka_kv8_config>(a[0], "c"), &d = *structure<mka_kv8_config>(a[7], "dst_c");
  const Cache x = cache_of(a[1], c), y = cache_of(a[8], d);
  const at::Tensor *lens = tensor(a[2], "lens"), *w = tensor(a[3], "weights"), *lens2 = tensor(a[9], "dst_lens"),
                   *w2 = tensor(a[10], "dst_weights", true), *kept = tensor(a[11], "kept"), *ws = tensor(a[12], "ws");
  const int32_t keep = to_i32(integer(a[4]), "keep"), first = to_i32(integer(a[5]), "first"),
                recent = to_i32(integer(a[6]), "recent");
  const long long heads = (long long)c.batch * c.n_kv_heads;
  const int32_t* pl = positions(lens, "lens", c.batch);
  const float* pw = dense<float>(w, "weights", at::kFloat, heads * c.max_positions);
  int32_t* pl2 = dense<int32_t>(lens2, "dst_lens", at::kInt, c.batch);
  float* pw2 = dense<float>(w2, "dst_weights", at::kFloat, heads * d.max_positions);
  int32_t* pk = dense<int32_t>(kept, "kept", at::kInt, heads * keep);
  const size_t nb = bytes(*ws);
  void* s = call_stream(a[13], {lens, w, lens2, w2, kept, ws, x.t[0], x.t[1], x.t[2], x.t[3], y.t[0], y.t[1], y.t[2], y.t[3]});
  Unlocked unlocked;
  return mka_kv8_evict(&c, x.c, pl, pw, keep, first, recent, &d, y.c, pl2, pw2, pk, ws->data_ptr(), nb, s);
}

template <int (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(F(args));
  } catch (const Raised&) {
    return nullptr;
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyMethodDef methods[] = {
    {"window_attention", (PyCFunction)(void*)entry<window_attention, 8>, METH_FASTCALL, nullptr},
    {"window_attention_backward", (PyCFunction)(void*)entry<window_attention_backward, 13>, METH_FASTCALL, nullptr},
    {"kv8_append", (PyCFunction)(void*)entry<kv8_append, 7>, METH_FASTCALL, nullptr},
    {"kv8_read", (PyCFunction)(void*)entry<kv8_read, 7>, METH_FASTCALL, nullptr},
    {"kv8_attention", (PyCFunction)(void*)entry<kv8_attention, 8>, METH_FASTCALL, nullptr},
    {"kv8_evict", (PyCFunction)(void*)entry<kv8_evict, 14>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  // the torch that this was built against: the package refuses another one's
  if (m && PyModule_AddStringConstant(m, "torch_version", MKA_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
