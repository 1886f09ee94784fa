// q4_serve_py.cpp -- the native half of the Python bindings of q4serve.h and
// (q4_experts_py.h) q4experts.h: it
// checks tensors against the sizes the kernels will use, allocates outputs and
// workspaces, and calls the C ABI.  serve.py and mixture.py hold the public functions and
// their documentation; each passes its arguments on by position.
//
// In C++ because of latency: a decode step makes several calls whose kernels
// take 5 to 10 us, and the same checks in Python with a ctypes call of 34
// arguments took 13 us of host time for the cache append, these take 2.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <exception>
#include <optional>
#include <string>

#include "q4experts.h"
#include "q4serve.h"

namespace {

PyObject* g_error = nullptr;  // q4linear.Q4Error

// A refusal: becomes a Python ValueError.
struct Refused {
  std::string what;
};

[[noreturn]] void refuse(const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  throw Refused{buf};
}

std::string shape(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

struct PyFailed {};  // a Python error is set

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyFailed{};
  return v;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyFailed{};
  return v;
}

bool given(PyObject* o) { return o != Py_None; }

const char* type_name(at::ScalarType t) { return c10::toString(t); }

int32_t dtype_of(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kFloat: return Q4_DTYPE_F32;
    case at::kHalf: return Q4_DTYPE_F16;
    case at::kBFloat16: return Q4_DTYPE_BF16;
    default: refuse("%s must be float32, float16 or bfloat16, got %s", name, type_name(t.scalar_type()));
  }
}

void same_device(const at::Tensor& t, const char* name, const at::Device& dev) {
  if (t.device() != dev)
    refuse("%s must be on %s, got %s", name, dev.str().c_str(), t.device().str().c_str());
}

void on_gpu(const at::Device& dev, const char* name) {
  if (!dev.is_cuda()) refuse("%s must be a device tensor", name);
}

// [T, heads, dim] of a type, unit stride along dim.
void check_rows(const at::Tensor& t, const char* name, at::ScalarType type, const at::Device& dev) {
  if (t.dim() != 3 || t.scalar_type() != type)
    refuse("%s must be a 3-D %s tensor, got %s %s", name, type_name(type), shape(t).c_str(),
           type_name(t.scalar_type()));
  same_device(t, name, dev);
  if (t.stride(2) != 1) refuse("%s must have unit stride along head_dim", name);
}

const void* vector(const at::Tensor& t, const char* name, int64_t n, at::ScalarType type,
                   const at::Device& dev) {
  if (t.dim() != 1 || t.scalar_type() != type || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    refuse("%s must be a contiguous %s vector of %lld, got %s %s", name, type_name(type),
           (long long)n, shape(t).c_str(), type_name(t.scalar_type()));
  same_device(t, name, dev);
  return t.data_ptr();
}

struct Cache {
  int8_t *k, *v;
  float *ks, *vs;
  int64_t pages, heads, page, dim;
};

Cache cache_of(PyObject* const* a, const at::Device& dev) {
  const at::Tensor &k = tensor(a[0], "k_cache"), &v = tensor(a[1], "v_cache"),
                   &ks = tensor(a[2], "k_scale"), &vs = tensor(a[3], "v_scale");
  if (k.dim() != 4 || v.dim() != 4 || k.scalar_type() != at::kChar || v.scalar_type() != at::kChar)
    refuse("k_cache must be int8 [pages, kv_heads, page, head_dim], v_cache int8 [pages, kv_heads, "
           "head_dim, page], got %s and %s", shape(k).c_str(), shape(v).c_str());
  Cache c{nullptr, nullptr, nullptr, nullptr, k.size(0), k.size(1), k.size(2), k.size(3)};
  if (v.size(0) != c.pages || v.size(1) != c.heads || v.size(2) != c.dim || v.size(3) != c.page ||
      !k.is_contiguous() || !v.is_contiguous())
    refuse("k_cache [pages, kv_heads, page, head_dim] and v_cache [pages, kv_heads, head_dim, page] "
           "must be contiguous, got %s and %s", shape(k).c_str(), shape(v).c_str());
  for (const at::Tensor* s : {&ks, &vs})
    if (s->scalar_type() != at::kFloat || s->dim() != 2 || s->size(0) != c.pages ||
        s->size(1) != c.heads || !s->is_contiguous())
      refuse("k_scale and v_scale must be contiguous float32 [%lld, %lld], got %s %s",
             (long long)c.pages, (long long)c.heads, shape(*s).c_str(), type_name(s->scalar_type()));
  if ((c.page != 16 && c.page != 32 && c.page != 64 && c.page != 128) || c.dim % 16 || c.dim < 16 ||
      c.dim > 256)
    refuse("a page has 16, 32, 64 or 128 tokens and head_dim is a multiple of 16 up to 256, got "
           "%lld and %lld", (long long)c.page, (long long)c.dim);
  same_device(k, "k_cache", dev);
  same_device(v, "v_cache", dev);
  same_device(ks, "k_scale", dev);
  same_device(vs, "v_scale", dev);
  c.k = (int8_t*)k.data_ptr();
  c.v = (int8_t*)v.data_ptr();
  c.ks = (float*)ks.data_ptr();
  c.vs = (float*)vs.data_ptr();
  return c;
}

struct Tables {
  int64_t batch, ld, cols;
  const int32_t *table, *cu, *lengths;
};

Tables tables_of(PyObject* const* a, int64_t T, const at::Device& dev) {
  const at::Tensor& t = tensor(a[0], "page_table");
  if (t.scalar_type() != at::kInt || t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
    refuse("page_table must be int32 [batch, max_pages] with unit stride along its rows, got %s %s",
           shape(t).c_str(), type_name(t.scalar_type()));
  same_device(t, "page_table", dev);
  Tables r;
  r.batch = t.size(0);
  r.cols = t.size(1);
  r.ld = r.batch > 1 ? t.stride(0) : r.cols;
  if (T > 0 && r.batch == 0) refuse("%lld new tokens of no sequence", (long long)T);
  r.table = (const int32_t*)t.data_ptr();
  r.cu = (const int32_t*)vector(tensor(a[1], "cu_new"), "cu_new", r.batch + 1, at::kInt, dev);
  r.lengths = (const int32_t*)vector(tensor(a[2], "lengths"), "lengths", r.batch, at::kInt, dev);
  return r;
}

// What the caller gave, or a new one of what is needed.
struct Workspace {
  at::Tensor own;
  void* p = nullptr;
  size_t n = 0;
  Workspace(PyObject* o, size_t need, const at::TensorOptions& like) {
    if (given(o)) {
      const at::Tensor& t = tensor(o, "workspace");
      if (!t.is_contiguous()) refuse("workspace must be contiguous");
      same_device(t, "workspace", like.device());
      p = t.data_ptr();
      n = t.numel() * t.element_size();
    } else if (need) {
      own = at::empty({(int64_t)need}, like.dtype(at::kByte));
      p = own.data_ptr();
      n = need;
    }
  }
};

void check(q4_status st, const char* what) {
  if (st == Q4_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, what);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw PyFailed{};
}

void* stream_of(PyObject* o) { return (void*)(uintptr_t)integer(o); }

// k, v, cache (4), tables (3), q, q_out, inv_freq, interleaved, max_new, stream
PyObject* kv_append(PyObject* const* a) {
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
  const at::Device dev = k.device();
  const int32_t dtype = dtype_of(k, "k");
  check_rows(k, "k", k.scalar_type(), dev);
  check_rows(v, "v", k.scalar_type(), dev);
  const Cache c = cache_of(a + 2, dev);
  const int64_t T = k.size(0);
  if (k.size(1) != c.heads || k.size(2) != c.dim || v.sizes() != k.sizes())
    refuse("k and v must be [T, %lld, %lld], got %s and %s", (long long)c.heads, (long long)c.dim,
           shape(k).c_str(), shape(v).c_str());
  const Tables t = tables_of(a + 6, T, dev);
  at::Tensor q, q_out;
  int64_t heads = c.heads;
  if (given(a[9])) {
    q = tensor(a[9], "q");
    check_rows(q, "q", k.scalar_type(), dev);
    heads = q.size(1);
    if (q.size(0) != T || q.size(2) != c.dim || heads == 0 || heads % c.heads)
      refuse("q must be [%lld, a multiple of %lld, %lld], got %s", (long long)T, (long long)c.heads,
             (long long)c.dim, shape(q).c_str());
    if (given(a[10])) {
      q_out = tensor(a[10], "q_out");
      check_rows(q_out, "q_out", k.scalar_type(), dev);
      if (q_out.sizes() != q.sizes())
        refuse("q_out must be %s, got %s", shape(q).c_str(), shape(q_out).c_str());
    }
  } else if (given(a[10])) {
    refuse("q_out without q");
  }
  int64_t rot = 0;
  const float* freq = nullptr;
  if (given(a[11])) {
    const at::Tensor& f = tensor(a[11], "inv_freq");
    rot = 2 * f.numel();
    freq = (const float*)vector(f, "inv_freq", rot / 2, at::kFloat, dev);
    if (rot > c.dim)
      refuse("inv_freq has %lld entries, more than head_dim / 2 = %lld", (long long)(rot / 2),
             (long long)(c.dim / 2));
  }
  const int interleaved = PyObject_IsTrue(a[12]);
  if (interleaved < 0) throw PyFailed{};
  const int64_t max_new = given(a[13]) ? integer(a[13]) : T;
  on_gpu(dev, "k");
  const c10::DeviceGuard guard(dev);
  if (q.defined() && !q_out.defined()) q_out = at::empty(q.sizes(), q.options());
  const bool has_q = q.defined();
  check(q4_kv_append(k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1),
                     has_q ? q.data_ptr() : nullptr, has_q ? q.stride(0) : 0,
                     has_q ? q.stride(1) : 0, has_q ? q_out.data_ptr() : nullptr,
                     has_q ? q_out.stride(0) : 0, has_q ? q_out.stride(1) : 0, dtype, T, t.batch,
                     heads, c.heads, c.dim, c.k, c.v, c.ks, c.vs, c.pages, c.page, t.table, t.ld,
                     t.cols, t.cu, t.lengths, max_new, freq, rot, interleaved, stream_of(a[14])),
        "q4_kv_append");
  if (!has_q) Py_RETURN_NONE;
  return THPVariable_Wrap(q_out);
}

// cache (4), type code, stream
PyObject* kv_dequant(PyObject* const* a) {
  const at::Tensor& first = tensor(a[0], "k_cache");
  const at::Device dev = first.device();
  const Cache c = cache_of(a, dev);
  const int64_t code = integer(a[4]);
  const at::ScalarType type = code == Q4_DTYPE_F32 ? at::kFloat : code == Q4_DTYPE_F16 ? at::kHalf : at::kBFloat16;
  on_gpu(dev, "k_cache");
  const c10::DeviceGuard guard(dev);
  const at::Tensor k = at::empty({c.pages, c.heads, c.page, c.dim}, first.options().dtype(type));
  const at::Tensor v = at::empty(k.sizes(), k.options());
  check(q4_kv_dequant(c.k, c.v, c.ks, c.vs, c.pages, c.heads, c.page, c.dim, (int32_t)code,
                      k.data_ptr(), v.data_ptr(), stream_of(a[5])),
        "q4_kv_dequant");
  PyObject* r = PyTuple_New(2);
  if (!r) throw PyFailed{};
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(k));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(v));
  return r;
}

// q, cache (4), tables (3), softmax_scale, window, max_new, max_len, out, workspace, stream
PyObject* attention(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  const at::Device dev = q.device();
  const int32_t dtype = dtype_of(q, "q");
  check_rows(q, "q", q.scalar_type(), dev);
  const Cache c = cache_of(a + 1, dev);
  const int64_t T = q.size(0), heads = q.size(1);
  if (q.size(2) != c.dim || heads == 0 || heads % c.heads)
    refuse("q must be [T, a multiple of %lld, %lld], got %s", (long long)c.heads, (long long)c.dim,
           shape(q).c_str());
  const Tables t = tables_of(a + 5, T, dev);
  const double scale = given(a[8]) ? number(a[8]) : 1.0 / std::sqrt((double)c.dim);
  const int64_t window = integer(a[9]);
  const int64_t max_new = given(a[10]) ? integer(a[10]) : T;
  // the table's reach, as far as int32 lengths go
  const int64_t reach = std::min<int64_t>(t.cols * c.page, INT32_MAX);
  const int64_t max_len = given(a[11]) ? integer(a[11]) : reach;
  at::Tensor out;
  if (given(a[12])) {
    out = tensor(a[12], "out");
    check_rows(out, "out", q.scalar_type(), dev);
    if (out.sizes() != q.sizes())
      refuse("out must be %s, got %s", shape(q).c_str(), shape(out).c_str());
  } else if (max_new >= 0 && max_new < T && max_new * t.batch < T) {
    // queries past max_new are left alone: a new tensor has nothing there
    refuse("max_new = %lld leaves out some of %lld new tokens of %lld sequences; give a bound, or out",
           (long long)max_new, (long long)T, (long long)t.batch);
  }
  on_gpu(dev, "q");
  const c10::DeviceGuard guard(dev);
  if (!out.defined()) out = at::empty(q.sizes(), q.options());
  const size_t need =
      given(a[13]) ? 0 : q4_attention_workspace_bytes(dtype, T, t.batch, heads, c.heads, c.dim, c.page,
                                                      max_new, max_len, window);
  const Workspace ws(a[13], need, q.options());
  check(q4_attention(q.data_ptr(), q.stride(0), q.stride(1), out.data_ptr(), out.stride(0),
                     out.stride(1), dtype, T, t.batch, heads, c.heads, c.dim, c.k, c.v, c.ks, c.vs,
                     c.pages, c.page, t.table, t.ld, t.cols, t.cu, t.lengths, max_new, max_len,
                     (float)scale, window, ws.p, ws.n, stream_of(a[14])),
        "q4_attention");
  return THPVariable_Wrap(out);
}

int64_t check_logits(const at::Tensor& t, const char* name) {
  if (t.dim() != 2 || t.size(1) < 1 || (t.size(1) > 1 && t.stride(1) != 1))
    refuse("%s must be 2-D [M, vocab] with unit stride along its rows, got %s", name, shape(t).c_str());
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

const int64_t* targets_of(PyObject* o, int64_t M, const at::Device& dev) {
  if (!given(o)) return nullptr;
  return (const int64_t*)vector(tensor(o, "targets"), "targets", M, at::kLong, dev);
}

// logits, targets, top_k, workspace, stream -> logprob, entropy, lse, ids, top
PyObject* token_logprobs(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "logits");
  const at::Device dev = x.device();
  const int64_t ld = check_logits(x, "logits");
  const int32_t dtype = dtype_of(x, "logits");
  const int64_t M = x.size(0), V = x.size(1), k = integer(a[2]);
  const int64_t most = V < 32 ? V : 32;
  if (k < 0 || k > most) refuse("top_k must be 0 .. %lld, got %lld", (long long)most, (long long)k);
  const int64_t* targets = targets_of(a[1], M, dev);
  on_gpu(dev, "logits");
  const c10::DeviceGuard guard(dev);
  // tensors of their own: views of one would share its version counter, and an
  // in-place change of one would spoil what autograd saved of another
  const at::TensorOptions f32 = x.options().dtype(at::kFloat);
  const at::Tensor logprob = targets ? at::empty({M}, f32) : at::Tensor();
  const at::Tensor entropy = at::empty({M}, f32), lse = at::empty({M}, f32), top = at::empty({M, k}, f32);
  const at::Tensor ids = at::empty({M, k}, x.options().dtype(at::kLong));
  const Workspace ws(a[3], given(a[3]) ? 0 : q4_token_logprobs_workspace_bytes(M, V, k, dtype), x.options());
  check(q4_token_logprobs(x.data_ptr(), ld, dtype, M, V, targets, k,
                          targets ? (float*)logprob.data_ptr() : nullptr, (float*)entropy.data_ptr(),
                          (float*)lse.data_ptr(), (int64_t*)ids.data_ptr(), (float*)top.data_ptr(),
                          ws.p, ws.n, stream_of(a[4])),
        "q4_token_logprobs");
  PyObject* r = PyTuple_New(5);
  if (!r) throw PyFailed{};
  if (targets) {
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(logprob));
  } else {
    Py_INCREF(Py_None);
    PyTuple_SET_ITEM(r, 0, Py_None);
  }
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(entropy));
  PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(lse));
  PyTuple_SET_ITEM(r, 3, THPVariable_Wrap(ids));
  PyTuple_SET_ITEM(r, 4, THPVariable_Wrap(top));
  return r;
}

// logits, targets, lse, entropy, g_logprob, g_entropy, dlogits, stream
PyObject* token_logprobs_backward(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "logits");
  const at::Device dev = x.device();
  const int64_t ld = check_logits(x, "logits");
  const int32_t dtype = dtype_of(x, "logits");
  const int64_t M = x.size(0), V = x.size(1);
  const int64_t* targets = targets_of(a[1], M, dev);
  auto row = [&](PyObject* o, const char* name) -> const float* {
    return given(o) ? (const float*)vector(tensor(o, name), name, M, at::kFloat, dev) : nullptr;
  };
  const float *lse = row(a[2], "lse"), *entropy = row(a[3], "entropy");
  const float *gl = row(a[4], "g_logprob"), *ge = row(a[5], "g_entropy");
  at::Tensor dx;
  if (given(a[6])) {
    dx = tensor(a[6], "dlogits");
    if (dx.sizes() != x.sizes() || dx.scalar_type() != x.scalar_type())
      refuse("dlogits must be %s %s, got %s %s", type_name(x.scalar_type()), shape(x).c_str(),
             type_name(dx.scalar_type()), shape(dx).c_str());
    same_device(dx, "dlogits", dev);
  }
  on_gpu(dev, "logits");
  const c10::DeviceGuard guard(dev);
  if (!dx.defined()) dx = at::empty({M, V}, x.options());
  const int64_t ldd = check_logits(dx, "dlogits");
  check(q4_token_logprobs_backward(x.data_ptr(), ld, dtype, M, V, targets, lse, entropy, gl, ge,
                                   dx.data_ptr(), ldd, stream_of(a[7])),
        "q4_token_logprobs_backward");
  return THPVariable_Wrap(dx);
}

}  // namespace

#include "q4_experts_py.h"

namespace {

// No C++ exception leaves: each becomes a Python error.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n != N) {
      PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
      return nullptr;
    }
    return F(args);
  } catch (const PyFailed&) {
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

#define Q4_METHOD(name, n) \
  {#name, (PyCFunction)(void (*)(void))entry<name, n>, METH_FASTCALL, nullptr}

PyMethodDef methods[] = {Q4_METHOD(kv_append, 15),
                         Q4_METHOD(kv_dequant, 6),
                         Q4_METHOD(attention, 15),
                         Q4_METHOD(token_logprobs, 5),
                         Q4_METHOD(token_logprobs_backward, 8),
                         Q4_METHOD(route, 9),
                         Q4_METHOD(route_backward, 8),
                         Q4_METHOD(experts, 13),
                         Q4_METHOD(experts_backward, 13),
                         Q4_METHOD(head_cross_entropy, 8),
                         Q4_METHOD(head_cross_entropy_backward, 11),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve_native", nullptr, -1, methods,
                      nullptr,               nullptr,          nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve_native() { return PyModule_Create(&module); }
