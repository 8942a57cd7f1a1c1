// The plain form of paged.py's calls, without Python between their arguments and the C entry points: a
// layer's step makes several of them on a few kilobytes each, and there the wrappers cost more than the
// kernels (a call's wall time on 64 tokens: 20 us from Python, 5 us from here).  What is handled here: outputs and workspace allocated by the call, on the current stream of
// the tensors' device, which is the current one.  Anything else, and any argument that is not as it
// should be, returns None: the Python form then does the call, or says what is wrong with it.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/fa_paged.h"

namespace {

struct Entry {
  decltype(&fa_qk_norm_rope) norm;
  decltype(&fa_qk_norm_rope_backward) norm_back;
  decltype(&fa_qk_norm_rope_backward_workspace_size) norm_back_ws;
  decltype(&fa_cache_append) append;
  decltype(&fa_cache_read) read;
  decltype(&fa_paged_decode) decode;
  decltype(&fa_paged_decode_workspace_size) decode_ws;
} fn;

PyObject *s_q, *s_k, *s_v, *s_O, *s_lse, *s_dq, *s_dk, *s_dwq, *s_dwk;

int act_of(at::ScalarType t) {
  return t == at::kFloat ? FA_ACT_F32 : t == at::kHalf ? FA_ACT_F16 : t == at::kBFloat16 ? FA_ACT_BF16 : -1;
}

// The arguments of one call; ok turns false at the first that is not as expected.
struct Args {
  PyObject* const* a;
  int device = -1;
  bool ok = true;

  const at::Tensor* tensor(int i) {  // on the call's device, which the first tensor sets
    if (!THPVariable_Check(a[i])) return ok = false, nullptr;
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (!t.is_cuda()) return ok = false, nullptr;
    if (device < 0) device = t.get_device();
    if (t.get_device() != device) return ok = false, nullptr;
    return &t;
  }
  // [n][heads][D] of type t with contiguous components
  const at::Tensor* heads(int i, at::ScalarType t, int64_t n, int64_t D) {
    const at::Tensor* x = tensor(i);
    if (!ok) return nullptr;
    if (x->dim() != 3 || x->scalar_type() != t || x->size(0) != n || n > INT32_MAX || x->size(2) != D || x->stride(2) != 1 || x->numel() == 0)
      ok = false;
    return x;
  }
  template <typename T>
  T* flat(int i, at::ScalarType t, int64_t n, bool optional) {  // [n], contiguous
    if (optional && a[i] == Py_None) return nullptr;
    const at::Tensor* x = tensor(i);
    if (!ok) return nullptr;
    if (x->dim() != 1 || x->scalar_type() != t || x->size(0) != n || !x->is_contiguous()) return ok = false, nullptr;
    return static_cast<T*>(x->data_ptr());
  }
  bool rope(int i, int style, fa_rope* r, const fa_rope** p) {  // int64 [pairs] or None
    *p = nullptr;
    if (a[i] == Py_None) return false;
    const at::Tensor* x = tensor(i);
    if (!ok) return false;
    if (x->dim() != 1 || x->scalar_type() != at::kLong || !x->is_contiguous()) return ok = false, false;
    *r = fa_rope{static_cast<const uint64_t*>(x->data_ptr()), (int32_t)(2 * x->size(0)), style};
    *p = r;
    return true;
  }
  long long integer(int i) {
    const long long v = PyLong_AsLongLong(a[i]);
    if (v == -1 && PyErr_Occurred()) PyErr_Clear(), ok = false;
    return v;
  }
  double number(int i) {
    const double v = PyFloat_AsDouble(a[i]);
    if (v == -1.0 && PyErr_Occurred()) PyErr_Clear(), ok = false;
    return v;
  }
  bool here() { return ok && c10::cuda::current_device() == device; }
};

// (straight from the allocator: at::empty's dispatch is most of what it costs)
at::Tensor make(at::IntArrayRef shape, at::ScalarType t, int device) {
  return at::Tensor(at::detail::empty_cuda(shape, t, at::Device(at::kCUDA, device), std::nullopt));
}
void put(PyObject* d, PyObject* key, const at::Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  PyDict_SetItem(d, key, o);
  Py_DECREF(o);
}
void* at_of(const at::Tensor* t) { return t->data_ptr(); }

// C++ exceptions (an allocation that fails) become the Python path's to meet again
template <typename F>
PyObject* guarded(F f) {
  try {
    PyObject* r = f();
    if (r) return r;
  } catch (const std::exception&) {
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

// (q, k, pos, wq, wk, eps, rope, style, dtype)
PyObject* norm(PyObject*, PyObject* const* argv, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    Args a{argv};
    const at::Tensor* q = a.tensor(0);
    if (!a.ok || q->dim() != 3) return nullptr;
    const at::ScalarType xt = q->scalar_type();
    const int64_t N = q->size(0), H = q->size(1), D = q->size(2);
    a.heads(0, xt, N, D);
    const at::Tensor* k = a.ok && argv[1] != Py_None ? a.heads(1, xt, N, D) : nullptr;
    const int64_t Hkv = a.ok && k ? k->size(1) : 0;
    const float* wq = a.ok ? a.flat<float>(3, at::kFloat, D, true) : nullptr;
    const float* wk = a.ok ? a.flat<float>(4, at::kFloat, D, true) : nullptr;
    if (!a.ok) return nullptr;
    fa_rope r;
    const fa_rope* rp;
    const int32_t* pos = a.rope(6, (int)a.integer(7), &r, &rp) ? a.flat<int32_t>(2, at::kInt, N, false) : nullptr;
    const double eps = a.number(5);
    if (argv[8] != Py_None && !THPDtype_Check(argv[8])) return nullptr;
    const at::ScalarType yt = argv[8] == Py_None ? xt : reinterpret_cast<THPDtype*>(argv[8])->scalar_type;
    if (!a.here() || act_of(xt) < 0 || act_of(yt) < 0) return nullptr;
    const at::Tensor oq = make({N, H, D}, yt, a.device), ok = k ? make({N, Hkv, D}, yt, a.device) : at::Tensor();
    const fa_qk_views views = {q->stride(0), q->stride(1), k ? k->stride(0) : 0, k ? k->stride(1) : 0};
    if (fn.norm(at_of(q), k ? at_of(k) : nullptr, act_of(xt), &views, wq, wk, (float)eps, pos, rp, N, H, Hkv, D, oq.data_ptr(),
                k ? ok.data_ptr() : nullptr, act_of(yt), c10::cuda::getCurrentCUDAStream(a.device).stream()) != FA_OK)
      return nullptr;
    PyObject* d = PyDict_New();
    put(d, s_q, oq);
    if (k) put(d, s_k, ok);
    else PyDict_SetItem(d, s_k, Py_None);
    return d;
  });
}

// (gq, gk, q, k, pos, wq, wk, eps, rope, style)
PyObject* norm_back(PyObject*, PyObject* const* argv, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    Args a{argv};
    const at::Tensor* q = a.tensor(2);
    if (!a.ok || q->dim() != 3 || (argv[1] == Py_None) != (argv[3] == Py_None)) return nullptr;
    const at::ScalarType xt = q->scalar_type();
    const int64_t N = q->size(0), H = q->size(1), D = q->size(2);
    a.heads(2, xt, N, D);
    const at::Tensor* k = a.ok && argv[3] != Py_None ? a.heads(3, xt, N, D) : nullptr;
    const int64_t Hkv = a.ok && k ? k->size(1) : 0;
    const at::Tensor* gq = a.ok ? a.tensor(0) : nullptr;
    if (!a.ok) return nullptr;
    const at::ScalarType yt = gq->scalar_type();
    a.heads(0, yt, N, D);
    const at::Tensor* gk = a.ok && k ? a.heads(1, yt, N, D) : nullptr;
    if (!a.ok || gq->size(1) != H || !gq->is_contiguous() || (gk && (gk->size(1) != Hkv || !gk->is_contiguous()))) return nullptr;
    const float* wq = a.flat<float>(5, at::kFloat, D, true);
    const float* wk = a.ok ? a.flat<float>(6, at::kFloat, D, true) : nullptr;
    if (!a.ok) return nullptr;
    fa_rope r;
    const fa_rope* rp;
    const int32_t* pos = a.rope(8, (int)a.integer(9), &r, &rp) ? a.flat<int32_t>(4, at::kInt, N, false) : nullptr;
    const double eps = a.number(7);
    if (!a.here() || act_of(xt) < 0 || act_of(yt) < 0) return nullptr;
    const size_t need = fn.norm_back_ws(N, H, Hkv, D);
    const at::Tensor dq = make({N, H, D}, xt, a.device), dk = k ? make({N, Hkv, D}, xt, a.device) : at::Tensor();
    const at::Tensor dwq = wq ? make({D}, at::kFloat, a.device) : at::Tensor();
    const at::Tensor dwk = wk && k ? make({D}, at::kFloat, a.device) : at::Tensor();
    const at::Tensor ws = make({(int64_t)need}, at::kByte, a.device);
    const fa_qk_views views = {q->stride(0), q->stride(1), k ? k->stride(0) : 0, k ? k->stride(1) : 0};
    auto at_or_null = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    if (fn.norm_back(at_of(gq), gk ? at_of(gk) : nullptr, act_of(yt), at_of(q), k ? at_of(k) : nullptr, act_of(xt), &views, wq, wk,
                     (float)eps, pos, rp, N, H, Hkv, D, dq.data_ptr(), at_or_null(dk), static_cast<float*>(at_or_null(dwq)),
                     static_cast<float*>(at_or_null(dwk)), ws.data_ptr(), need,
                     c10::cuda::getCurrentCUDAStream(a.device).stream()) != FA_OK)
      return nullptr;
    PyObject* d = PyDict_New();
    put(d, s_dq, dq);
    if (k) put(d, s_dk, dk);
    if (dwq.defined()) put(d, s_dwq, dwq);
    if (dwk.defined()) put(d, s_dwk, dwk);
    return d;
  });
}

// The cache: the address of its fa_paged_cache and its device, as PagedCache keeps them
const fa_paged_cache* cache_of(Args& a, int i) {
  const fa_paged_cache* c = reinterpret_cast<const fa_paged_cache*>(a.integer(i));
  a.device = (int)a.integer(i + 1);
  return a.ok && c ? c : (a.ok = false, nullptr);
}

// (k, v, cache, device, seq, pos, k_norm, eps, rope, style)
PyObject* append(PyObject*, PyObject* const* argv, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    Args a{argv};
    const fa_paged_cache* c = cache_of(a, 2);
    if (!a.ok) return nullptr;
    const at::Tensor* k = a.tensor(0);
    if (!a.ok || k->dim() != 3) return nullptr;
    const at::ScalarType xt = k->scalar_type();
    const int64_t T = k->size(0);
    a.heads(0, xt, T, c->D);
    const at::Tensor* v = a.ok ? a.heads(1, xt, T, c->Dv) : nullptr;
    if (!a.ok || k->size(1) != c->Hkv || v->size(1) != c->Hkv) return nullptr;
    const int32_t* seq = a.flat<int32_t>(4, at::kInt, T, false);
    const int32_t* pos = a.ok ? a.flat<int32_t>(5, at::kInt, T, false) : nullptr;
    const float* w = a.ok ? a.flat<float>(6, at::kFloat, c->D, true) : nullptr;
    const double eps = a.number(7);
    if (!a.ok) return nullptr;
    fa_rope r;
    const fa_rope* rp;
    a.rope(8, (int)a.integer(9), &r, &rp);
    if (!a.here() || act_of(xt) < 0) return nullptr;
    const fa_kv_views views = {k->stride(0), k->stride(1), v->stride(0), v->stride(1)};
    if (fn.append(at_of(k), at_of(v), act_of(xt), &views, c, seq, pos, T, w, (float)eps, rp,
                  c10::cuda::getCurrentCUDAStream(a.device).stream()) != FA_OK)
      return nullptr;
    Py_RETURN_TRUE;
  });
}

// (cache, device, seq, pos, dtype)
PyObject* read(PyObject*, PyObject* const* argv, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    Args a{argv};
    const fa_paged_cache* c = cache_of(a, 0);
    if (!a.ok) return nullptr;
    const at::Tensor* s = a.tensor(2);
    if (!a.ok || s->dim() != 1 || !THPDtype_Check(argv[4])) return nullptr;
    const int64_t T = s->size(0);
    const int32_t* seq = a.flat<int32_t>(2, at::kInt, T, false);
    const int32_t* pos = a.ok ? a.flat<int32_t>(3, at::kInt, T, false) : nullptr;
    const at::ScalarType yt = reinterpret_cast<THPDtype*>(argv[4])->scalar_type;
    if (!a.here() || act_of(yt) < 0) return nullptr;
    const at::Tensor k = make({T, c->Hkv, c->D}, yt, a.device), v = make({T, c->Hkv, c->Dv}, yt, a.device);
    if (fn.read(c, seq, pos, T, act_of(yt), k.data_ptr(), v.data_ptr(), c10::cuda::getCurrentCUDAStream(a.device).stream()) != FA_OK)
      return nullptr;
    PyObject* d = PyDict_New();
    put(d, s_k, k), put(d, s_v, v);
    return d;
  });
}

// (q, cache, device, seq_lens, scale, alibi_slopes, softcap, sinks)
PyObject* decode(PyObject*, PyObject* const* argv, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    Args a{argv};
    const fa_paged_cache* c = cache_of(a, 1);
    if (!a.ok) return nullptr;
    const at::Tensor* q = a.tensor(0);
    if (!a.ok || q->dim() != 3) return nullptr;
    const at::ScalarType xt = q->scalar_type();
    const int64_t B = c->B, H = q->size(1);
    a.heads(0, xt, B, c->D);
    const int32_t* lens = a.ok ? a.flat<int32_t>(3, at::kInt, B, false) : nullptr;
    const float* alibi = a.ok ? a.flat<float>(5, at::kFloat, H, true) : nullptr;
    const float* sinks = a.ok ? a.flat<float>(7, at::kFloat, H, true) : nullptr;
    const double scale = a.number(4), softcap = a.number(6);
    if (!a.here() || act_of(xt) < 0) return nullptr;
    const size_t need = fn.decode_ws(c, H);
    const at::Tensor O = make({B, H, c->Dv}, xt, a.device), lse = make({B, H}, at::kFloat, a.device);
    const at::Tensor ws = make({(int64_t)need}, at::kByte, a.device);
    if (fn.decode(at_of(q), act_of(xt), q->stride(0), q->stride(1), c, lens, H, (float)scale, alibi, (float)softcap, sinks,
                  O.data_ptr(), static_cast<float*>(lse.data_ptr()), ws.data_ptr(), need,
                  c10::cuda::getCurrentCUDAStream(a.device).stream()) != FA_OK)
      return nullptr;
    PyObject* d = PyDict_New();
    put(d, s_O, O), put(d, s_lse, lse);
    return d;
  });
}

// The addresses of libfa_back.so's entry points, in Entry's order
PyObject* bind(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  if (n != 7) return PyErr_Format(PyExc_TypeError, "seven addresses expected");
  void* p[7];
  for (int i = 0; i < 7; ++i)
    if (!(p[i] = PyLong_AsVoidPtr(argv[i]))) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "address 0");
  fn.norm = reinterpret_cast<decltype(fn.norm)>(p[0]);
  fn.norm_back = reinterpret_cast<decltype(fn.norm_back)>(p[1]);
  fn.norm_back_ws = reinterpret_cast<decltype(fn.norm_back_ws)>(p[2]);
  fn.append = reinterpret_cast<decltype(fn.append)>(p[3]);
  fn.read = reinterpret_cast<decltype(fn.read)>(p[4]);
  fn.decode = reinterpret_cast<decltype(fn.decode)>(p[5]);
  fn.decode_ws = reinterpret_cast<decltype(fn.decode_ws)>(p[6]);
  Py_RETURN_NONE;
}

#define FAST(name, n)                                                                                      \
  PyObject* py_##name(PyObject* self, PyObject* const* argv, Py_ssize_t argc) {                            \
    if (argc != n || !fn.norm) return PyErr_Format(PyExc_TypeError, #name ": %d arguments, after bind()", n); \
    return name(self, argv, argc);                                                                         \
  }
FAST(norm, 9)
FAST(norm_back, 10)
FAST(append, 10)
FAST(read, 5)
FAST(decode, 8)

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_norm)), METH_FASTCALL, nullptr},
    {"norm_back", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_norm_back)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_append)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_read)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_decode)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", "plain calls of paged.py", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast(void) {
  PyObject** names[] = {&s_q, &s_k, &s_v, &s_O, &s_lse, &s_dq, &s_dk, &s_dwq, &s_dwk};
  const char* text[] = {"q", "k", "v", "O", "lse", "dq", "dk", "dwq", "dwk"};
  for (int i = 0; i < 9; ++i) *names[i] = PyUnicode_InternFromString(text[i]);
  return PyModule_Create(&module);
}
