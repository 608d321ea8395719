// The Python side of the calls that a decode step makes once per layer around the
// attention: tensors in, the C ABI call out.  Their kernels take two to ten
// microseconds, and reading a tensor's properties through Python attributes and
// converting twenty arguments through ctypes took 6 to 9 on the host (norm and
// rotation of one token: 18.8 us a call at first, 8.9 with every property read once).
// Here a call checks its tensors directly.  No step of any operator runs here.
//
// Every function takes positional arguments from its wrapper in __init__.py (which
// documents them) and returns the C call's status; a tensor of the wrong shape, type,
// layout or device raises ValueError before the call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <string>

#include "../../include/k8v4.h"

namespace {

struct Api {
  decltype(&qk_norm_rope_k8v4) norm_rope = nullptr;
  decltype(&kv_append_k8v4_rope) append_rope = nullptr;
  decltype(&spec_accept_k8v4) accept = nullptr;
  decltype(&attn_k8v4_decode_shared) decode_shared = nullptr;
} g_api;

struct Bad {                       // a refused argument: what to say
  std::string what;
};
[[noreturn]] void bad(const std::string& what) { throw Bad{what}; }
struct Raised {};                  // a Python error is set

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad(std::string(name) + ": a tensor expected");
  return THPVariable_Unpack(o);
}
int device_of(const at::Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }

int dtype_of(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return K8V4_BF16;
  if (t.scalar_type() == at::kFloat) return K8V4_F32;
  bad(std::string(name) + ": bfloat16 or float32 expected");
}
int32_t fits(int64_t n, const char* name) {
  if (n < 0 || n > INT32_MAX) bad(std::string(name) + ": too large");
  return static_cast<int32_t>(n);
}

// a contiguous tensor of n elements of a type on a device; its address
void* flat(const at::Tensor& t, int64_t n, at::ScalarType type, int dev, const char* name) {
  if (t.numel() != n || t.scalar_type() != type || !t.is_contiguous() || device_of(t) != dev)
    bad(std::string(name) + ": " + std::to_string(n) + " contiguous " + c10::toString(type) +
        " on the other tensors' device expected");
  return t.data_ptr();
}
void* flat(PyObject* o, int64_t n, at::ScalarType type, int dev, const char* name) {
  return flat(tensor(o, name), n, type, dev, name);
}
void* flat_or_null(PyObject* o, int64_t n, at::ScalarType type, int dev, const char* name) {
  return o == Py_None ? nullptr : flat(o, n, type, dev, name);
}

// tokens [n_seqs, n_tok, heads, 256]: heads contiguous, tokens evenly spaced over
// the sequences (a slice of a packed projection qualifies); the spacing in elements
int64_t token_stride(const at::Tensor& t, int64_t heads, const char* name) {
  if (t.dim() != 4 || t.size(2) != heads || t.size(3) != 256)
    bad(std::string(name) + ": [n_seqs, n_tok, " + std::to_string(heads) + ", 256] expected");
  if (heads > 0 && t.numel() > 0 && (t.stride(3) != 1 || (heads > 1 && t.stride(2) != 256)))
    bad(std::string(name) + ": heads must be contiguous");
  if (t.size(1) <= 1) return t.size(0) > 1 ? t.stride(0) : heads * 256;
  if (t.size(0) > 1 && t.stride(0) != t.size(1) * t.stride(1)) bad(std::string(name) + ": tokens must be evenly spaced");
  return t.stride(1);
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v == 1;
}

k8v4_rope rope_of(PyObject* table, PyObject* interleaved, int dev) {
  const at::Tensor& t = tensor(table, "rope_table");
  if (t.dim() != 2) bad("rope_table: [n_pos, rot_dim] expected");
  k8v4_rope r;
  r.table = static_cast<const float*>(flat(t, t.numel(), at::kFloat, dev, "rope_table"));
  r.n_pos = t.size(0);
  r.rot_dim = fits(t.size(1), "rope_table");
  r.interleaved = truth(interleaved);
  return r;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
template <typename T>
T* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Raised{};
  return static_cast<T*>(p);
}

// Run a C call with the tensors' device current, on `stream` (an address) or, for
// None, on that device's current stream.
template <typename F>
PyObject* call(int dev, PyObject* stream, F&& f) {
  if (dev < 0) bad("CUDA tensors expected");
  void* s = stream == Py_None ? nullptr : address<void>(stream);
  int rc;
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  if (stream == Py_None) s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  Py_BEGIN_ALLOW_THREADS
  rc = f(s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

// nothing thrown leaves a function that Python calls
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Bad& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// q, k, pos, rope_table, q_out, k_out, q_weight, k_weight, eps, interleaved, stream
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    if (q.dim() != 4) bad("q: [n_seqs, n_tok, heads, 256] expected");
    const int dev = device_of(q), dtype = dtype_of(q, "q");
    const int32_t n_seqs = fits(q.size(0), "q"), n_tok = fits(q.size(1), "q"), n_q = fits(q.size(2), "q");
    const int64_t q_stride = token_stride(q, n_q, "q");
    const at::Tensor& q_out = tensor(a[4], "q_out");
    if (q_out.sizes() != q.sizes()) bad("q_out: the shape of q expected");
    void* qo = flat(q_out, q.numel(), q.scalar_type(), dev, "q_out");
    const void* kp = nullptr;
    void* ko = nullptr;
    int32_t n_k = 0;
    int64_t k_stride = 0;
    if (a[1] != Py_None) {
      const at::Tensor& k = tensor(a[1], "k");
      if (k.dim() != 4 || k.size(0) != n_seqs || k.size(1) != n_tok || k.scalar_type() != q.scalar_type() ||
          device_of(k) != dev)
        bad("k: the dtype, device and tokens of q expected");
      n_k = fits(k.size(2), "k");
      k_stride = token_stride(k, n_k, "k");
      const at::Tensor& k_out = tensor(a[5], "k_out");
      if (k_out.sizes() != k.sizes()) bad("k_out: the shape of k expected");
      ko = flat(k_out, k.numel(), k.scalar_type(), dev, "k_out");
      kp = k.data_ptr();
    }
    const auto* pos = static_cast<const int64_t*>(flat(a[2], n_seqs, at::kLong, dev, "pos"));
    const k8v4_rope rope = rope_of(a[3], a[9], dev);
    const auto* qw = static_cast<const float*>(flat_or_null(a[6], 256, at::kFloat, dev, "q_weight"));
    const auto* kw = static_cast<const float*>(flat_or_null(a[7], 256, at::kFloat, dev, "k_weight"));
    const float eps = static_cast<float>(number(a[8]));
    const void* qp = q.data_ptr();
    return call(dev, a[10], [&](void* s) {
      return g_api.norm_rope(qp, q_stride, n_q, kp, k_stride, n_k, dtype, qw, kw, eps, pos, n_seqs, n_tok, &rope, qo, ko, s);
    });
  });
}

// cache (address of its descriptor), pages, page_table, pos, k, v, rope_table, k_weight, eps, interleaved, stream
PyObject* append_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const auto* cache = address<const k8v4_cache>(a[0]);
    const at::Tensor& k = tensor(a[4], "k");
    const at::Tensor& v = tensor(a[5], "v");
    const int dev = device_of(k), dtype = dtype_of(k, "k");
    if (k.sizes() != v.sizes() || v.scalar_type() != k.scalar_type() || device_of(v) != dev ||
        device_of(tensor(a[1], "pages")) != dev)
      bad("k and v: one shape, dtype and device, the cache's");
    const int64_t k_stride = token_stride(k, cache->n_kv_heads, "k"), v_stride = token_stride(v, cache->n_kv_heads, "v");
    const int32_t n_seqs = fits(k.size(0), "k"), n_tok = fits(k.size(1), "k");
    const at::Tensor& table = tensor(a[2], "page_table");
    if (table.dim() != 2 || table.size(0) != n_seqs) bad("page_table: [n_seqs, max_pages] expected");
    const int64_t max_pages = table.size(1);
    const auto* pt = static_cast<const int32_t*>(flat(table, n_seqs * max_pages, at::kInt, dev, "page_table"));
    const auto* pos = static_cast<const int64_t*>(flat(a[3], n_seqs, at::kLong, dev, "pos"));
    const k8v4_rope rope = rope_of(a[6], a[9], dev);
    const auto* kw = static_cast<const float*>(flat_or_null(a[7], 256, at::kFloat, dev, "k_weight"));
    const float eps = static_cast<float>(number(a[8]));
    const void *kp = k.data_ptr(), *vp = v.data_ptr();
    return call(dev, a[10], [&](void* s) {
      return g_api.append_rope(cache, pt, max_pages, n_seqs, pos, n_tok, kp, k_stride, vp, v_stride, dtype, kw, eps, &rope, s);
    });
  });
}

// target_probs, draft_probs, draft_tokens, u_accept, u_sample, tokens, n_accepted, n_drafts, stream
PyObject* accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor& p = tensor(a[0], "target_probs");
    if (p.dim() != 3 || p.size(1) < 1) bad("target_probs: [n_seqs, n + 1, vocab] expected");
    const int dev = device_of(p), dtype = dtype_of(p, "target_probs");
    const int32_t b = fits(p.size(0), "target_probs"), drafts = fits(p.size(1) - 1, "target_probs"),
                  vocab = fits(p.size(2), "target_probs");
    const int64_t bn = static_cast<int64_t>(b) * drafts;
    const void* pp = flat(p, p.numel(), p.scalar_type(), dev, "target_probs");
    const void* qp = nullptr;
    if (a[1] != Py_None) {
      const at::Tensor& q = tensor(a[1], "draft_probs");
      if (q.dim() != 3 || q.size(0) != b || q.size(1) != drafts || q.size(2) != vocab) bad("draft_probs: [n_seqs, n, vocab] expected");
      qp = flat(q, q.numel(), p.scalar_type(), dev, "draft_probs");
    }
    const auto* tok = static_cast<const int32_t*>(flat(a[2], bn, at::kInt, dev, "draft_tokens"));
    const auto* u = static_cast<const float*>(flat(a[3], bn, at::kFloat, dev, "u_accept"));
    const auto* us = static_cast<const float*>(flat(a[4], b, at::kFloat, dev, "u_sample"));
    auto* out = static_cast<int32_t*>(flat(a[5], bn + b, at::kInt, dev, "tokens"));
    auto* acc = static_cast<int32_t*>(flat(a[6], b, at::kInt, dev, "n_accepted"));
    const auto* count = static_cast<const int32_t*>(flat_or_null(a[7], b, at::kInt, dev, "n_drafts"));
    return call(dev, a[8], [&](void* s) {
      return g_api.accept(pp, qp, dtype, tok, count, u, us, b, drafts, vocab, out, acc, s);
    });
  });
}

// cache (address of its descriptor), pages, q, page_table, seq_lens, max_seq_len, shared_len, out, ws, sm_scale, stream
PyObject* decode_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const auto* cache = address<const k8v4_cache>(a[0]);
    const at::Tensor& q = tensor(a[2], "q");
    const int dev = device_of(q), dtype = dtype_of(q, "q");
    const int64_t rows = 8 * static_cast<int64_t>(cache->n_kv_heads);
    if (q.dim() != 3 || q.size(1) != rows || q.size(2) != 256 || device_of(tensor(a[1], "pages")) != dev)
      bad("q: [n_seqs, 8H, 256] on the cache's device expected");
    const int32_t n_seqs = fits(q.size(0), "q");
    const void* qp = flat(q, q.numel(), q.scalar_type(), dev, "q");
    const at::Tensor& table = tensor(a[3], "page_table");
    if (table.dim() != 2 || table.size(0) != n_seqs) bad("page_table: [n_seqs, max_pages] expected");
    const int64_t max_pages = table.size(1);
    const auto* pt = static_cast<const int32_t*>(flat(table, n_seqs * max_pages, at::kInt, dev, "page_table"));
    const auto* lens = static_cast<const int32_t*>(flat(a[4], n_seqs, at::kInt, dev, "seq_lens"));
    const int32_t max_len = fits(integer(a[5]), "max_seq_len");
    const int64_t shared = integer(a[6]);
    if (shared < INT32_MIN || shared > INT32_MAX) bad("shared_len: too large");
    auto* out = static_cast<float*>(flat(a[7], q.numel(), at::kFloat, dev, "out"));
    const at::Tensor& ws = tensor(a[8], "ws");
    void* wp = flat(ws, ws.numel(), at::kByte, dev, "ws");
    const float scale = static_cast<float>(number(a[9]));
    return call(dev, a[10], [&](void* s) {
      return g_api.decode_shared(cache, qp, dtype, pt, max_pages, lens, n_seqs, max_len, static_cast<int32_t>(shared),
                                 scale, out, wp, static_cast<size_t>(ws.numel()), s);
    });
  });
}

// the addresses of the four C entry points, in the order of Api
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    g_api.norm_rope = reinterpret_cast<decltype(g_api.norm_rope)>(address<void>(a[0]));
    g_api.append_rope = reinterpret_cast<decltype(g_api.append_rope)>(address<void>(a[1]));
    g_api.accept = reinterpret_cast<decltype(g_api.accept)>(address<void>(a[2]));
    g_api.decode_shared = reinterpret_cast<decltype(g_api.decode_shared)>(address<void>(a[3]));
    Py_RETURN_NONE;
  });
}

#define K8V4_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {K8V4_METHOD(norm_rope), K8V4_METHOD(append_rope), K8V4_METHOD(accept),
                           K8V4_METHOD(decode_shared), K8V4_METHOD(bind), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_k8v4_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__k8v4_binding(void) { return PyModule_Create(&g_module); }
