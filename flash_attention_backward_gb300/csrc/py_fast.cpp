// The plain form of paged.py's and pages.py's calls, without Python between their arguments and the C entry points: a
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

#include "../../include/fa_paged_ext.h"

namespace {

struct Entry {
  decltype(&fa_qk_norm_rope) norm;
  decltype(&fa_qk_norm_rope_backward) norm_back;
  decltype(&fa_qk_norm_rope_backward_workspace_size) norm_back_ws;
  decltype(&fa_cache_append) append;
  decltype(&fa_cache_read) read;
  decltype(&fa_paged_decode) decode;
  decltype(&fa_paged_decode_workspace_size) decode_ws;
  decltype(&fa_qk_norm_rope_axes) norm_axes;
  decltype(&fa_qk_norm_rope_axes_backward) norm_axes_back;
  decltype(&fa_cache_append_axes) append_axes;
  decltype(&fa_paged_decode_pages) decode_pages;
  decltype(&fa_pages_extend) extend;
  decltype(&fa_pages_trim) trim;
  decltype(&fa_page_bounds) bounds;
  decltype(&fa_page_select) select;
  decltype(&fa_page_select_workspace_size) select_ws;
} fn;
constexpr int kEntries = sizeof(Entry) / sizeof(void*);

PyObject *s_q, *s_k, *s_v, *s_O, *s_lse, *s_dq, *s_dk, *s_dwq, *s_dwk, *s_seq, *s_pos, *s_row, *s_starts, *s_first;

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
  // axes i (uint8 [pairs]) of the rotation r, and positions j (int32 [axes][n], rows of neighbouring elements) or None
  const int32_t* axes(int i, int j, const fa_rope& r, int64_t n, fa_rope_axes* out) {
    const uint8_t* axis = flat<uint8_t>(i, at::kByte, r.n_rot / 2, false);
    const at::Tensor* x = ok ? tensor(j) : nullptr;
    if (!ok) return nullptr;
    if (x->dim() != 2 || x->scalar_type() != at::kInt || x->size(0) > INT32_MAX || x->size(1) != n || (n > 1 && x->stride(1) != 1)) return ok = false, nullptr;
    *out = fa_rope_axes{r.freqs, axis, x->stride(0), r.n_rot, r.style, (int32_t)x->size(0)};
    return static_cast<const int32_t*>(x->data_ptr());
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
// n elements of a one-dimensional tensor from `at` on, as a tensor of the same storage (a view's dispatch costs more than
// an allocation)
at::Tensor part(const at::Tensor& whole, int64_t at, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(), whole.dtype());
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  return t;
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

// (q, k, pos, wq, wk, eps, rope, style, dtype, rope_axes)
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
    fa_rope_axes ra;
    const bool turns = a.rope(6, (int)a.integer(7), &r, &rp), several = argv[9] != Py_None;
    if (several && !turns) return nullptr;
    const int32_t* pos = several ? a.axes(9, 2, r, N, &ra) : turns ? a.flat<int32_t>(2, at::kInt, N, false) : nullptr;
    const double eps = a.number(5);
    if (argv[8] != Py_None && !THPDtype_Check(argv[8])) return nullptr;
    const at::ScalarType yt = argv[8] == Py_None ? xt : reinterpret_cast<THPDtype*>(argv[8])->scalar_type;
    if (!a.here() || act_of(xt) < 0 || act_of(yt) < 0) return nullptr;
    const at::Tensor oq = make({N, H, D}, yt, a.device), ok = k ? make({N, Hkv, D}, yt, a.device) : at::Tensor();
    const fa_qk_views views = {q->stride(0), q->stride(1), k ? k->stride(0) : 0, k ? k->stride(1) : 0};
    auto call = [&](auto entry, auto* turn) {
      return entry(at_of(q), k ? at_of(k) : nullptr, act_of(xt), &views, wq, wk, (float)eps, pos, turn, N, H, Hkv, D, oq.data_ptr(),
                   k ? ok.data_ptr() : nullptr, act_of(yt), c10::cuda::getCurrentCUDAStream(a.device).stream());
    };
    if ((several ? call(fn.norm_axes, &ra) : call(fn.norm, rp)) != FA_OK) return nullptr;
    PyObject* d = PyDict_New();
    put(d, s_q, oq);
    if (k) put(d, s_k, ok);
    else PyDict_SetItem(d, s_k, Py_None);
    return d;
  });
}

// (gq, gk, q, k, pos, wq, wk, eps, rope, style, rope_axes)
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
    fa_rope_axes ra;
    const bool turns = a.rope(8, (int)a.integer(9), &r, &rp), several = argv[10] != Py_None;
    if (several && !turns) return nullptr;
    const int32_t* pos = several ? a.axes(10, 4, r, N, &ra) : turns ? a.flat<int32_t>(4, at::kInt, N, false) : nullptr;
    const double eps = a.number(7);
    if (!a.here() || act_of(xt) < 0 || act_of(yt) < 0) return nullptr;
    const size_t need = fn.norm_back_ws(N, H, Hkv, D);
    const at::Tensor dq = make({N, H, D}, xt, a.device), dk = k ? make({N, Hkv, D}, xt, a.device) : at::Tensor();
    const at::Tensor dwq = wq ? make({D}, at::kFloat, a.device) : at::Tensor();
    const at::Tensor dwk = wk && k ? make({D}, at::kFloat, a.device) : at::Tensor();
    const at::Tensor ws = make({(int64_t)need}, at::kByte, a.device);
    const fa_qk_views views = {q->stride(0), q->stride(1), k ? k->stride(0) : 0, k ? k->stride(1) : 0};
    auto at_or_null = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    auto call = [&](auto entry, auto* turn) {
      return entry(at_of(gq), gk ? at_of(gk) : nullptr, act_of(yt), at_of(q), k ? at_of(k) : nullptr, act_of(xt), &views, wq, wk,
                   (float)eps, pos, turn, N, H, Hkv, D, dq.data_ptr(), at_or_null(dk), static_cast<float*>(at_or_null(dwq)),
                   static_cast<float*>(at_or_null(dwk)), ws.data_ptr(), need, c10::cuda::getCurrentCUDAStream(a.device).stream());
    };
    if ((several ? call(fn.norm_axes_back, &ra) : call(fn.norm_back, rp)) != FA_OK)
      return nullptr;
    PyObject* d = PyDict_New();
    put(d, s_dq, dq);
    if (k) put(d, s_dk, dk);
    if (dwq.defined()) put(d, s_dwq, dwq);
    if (dwk.defined()) put(d, s_dwk, dwk);
    return d;
  });
}

// A structure whose address and device a Python object keeps (PagedCache, PageLists)
template <typename T>
const T* held(Args& a, int i) {
  const T* c = reinterpret_cast<const T*>(a.integer(i));
  a.device = (int)a.integer(i + 1);
  return a.ok && c ? c : (a.ok = false, nullptr);
}
const fa_paged_cache* cache_of(Args& a, int i) { return held<fa_paged_cache>(a, i); }

// (k, v, cache, device, seq, pos, k_norm, eps, rope, style, rope_axes, rope_pos)
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
    fa_rope_axes ra;
    const bool turns = a.rope(8, (int)a.integer(9), &r, &rp), several = argv[10] != Py_None;
    if (several != (argv[11] != Py_None) || (several && !turns)) return nullptr;
    const int32_t* rope_pos = several ? a.axes(10, 11, r, T, &ra) : nullptr;
    if (!a.here() || act_of(xt) < 0) return nullptr;
    const fa_kv_views views = {k->stride(0), k->stride(1), v->stride(0), v->stride(1)};
    cudaStream_t st = c10::cuda::getCurrentCUDAStream(a.device).stream();
    if ((several ? fn.append_axes(at_of(k), at_of(v), act_of(xt), &views, c, seq, pos, T, w, (float)eps, rope_pos, &ra, st)
                 : fn.append(at_of(k), at_of(v), act_of(xt), &views, c, seq, pos, T, w, (float)eps, rp, st)) != FA_OK)
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

// (q, cache, device, seq_lens, scale, alibi_slopes, softcap, sinks, pages)
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
    const at::Tensor* pages = a.ok && argv[8] != Py_None ? a.tensor(8) : nullptr;
    if (pages && (pages->dim() != 3 || pages->scalar_type() != at::kInt || pages->size(0) != B || pages->size(1) != c->Hkv ||
                  pages->size(2) > INT32_MAX || !pages->is_contiguous()))
      return nullptr;
    if (!a.here() || act_of(xt) < 0) return nullptr;
    const size_t need = fn.decode_ws(c, H);
    const at::Tensor O = make({B, H, c->Dv}, xt, a.device), lse = make({B, H}, at::kFloat, a.device);
    const at::Tensor ws = make({(int64_t)need}, at::kByte, a.device);
    cudaStream_t st = c10::cuda::getCurrentCUDAStream(a.device).stream();
    float* out_lse = static_cast<float*>(lse.data_ptr());
    if ((pages ? fn.decode_pages(at_of(q), act_of(xt), q->stride(0), q->stride(1), c, lens, static_cast<const int32_t*>(at_of(pages)),
                                 pages->size(2), H, (float)scale, alibi, (float)softcap, sinks, O.data_ptr(), out_lse, ws.data_ptr(), need, st)
               : fn.decode(at_of(q), act_of(xt), q->stride(0), q->stride(1), c, lens, H, (float)scale, alibi, (float)softcap, sinks,
                           O.data_ptr(), out_lse, ws.data_ptr(), need, st)) != FA_OK)
      return nullptr;
    PyObject* d = PyDict_New();
    put(d, s_O, O), put(d, s_lse, lse);
    return d;
  });
}

// (lists, device, new_tokens, T)
PyObject* extend(PyObject*, PyObject* const* argv, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    Args a{argv};
    const fa_page_lists* l = held<fa_page_lists>(a, 0);
    if (!a.ok) return nullptr;
    const int32_t* news = a.flat<int32_t>(2, at::kInt, l->B, false);
    const long long T = a.integer(3);
    if (!a.here() || T < 0 || T > INT32_MAX) return nullptr;
    // one allocation: each part on 16 bytes
    const int64_t B = l->B, t4 = (T + 3) / 4 * 4, b4 = (B + 4) / 4 * 4;
    const at::Tensor whole = make({3 * t4 + 2 * b4}, at::kInt, a.device);
    const at::Tensor seq = part(whole, 0, T), pos = part(whole, t4, T), row = part(whole, 2 * t4, T);
    const at::Tensor starts = part(whole, 3 * t4, B + 1), first = part(whole, 3 * t4 + b4, B);
    auto p = [](const at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); };
    if (fn.extend(l, news, (int)T, p(starts), p(first), p(seq), p(pos), p(row), c10::cuda::getCurrentCUDAStream(a.device).stream()) != FA_OK)
      return nullptr;
    PyObject* d = PyDict_New();
    put(d, s_seq, seq), put(d, s_pos, pos), put(d, s_row, row), put(d, s_starts, starts), put(d, s_first, first);
    return d;
  });
}

// (lists, device, keep)
PyObject* trim(PyObject*, PyObject* const* argv, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    Args a{argv};
    const fa_page_lists* l = held<fa_page_lists>(a, 0);
    if (!a.ok) return nullptr;
    const int32_t* keep = a.flat<int32_t>(2, at::kInt, l->B, false);
    if (!a.here() || fn.trim(l, keep, c10::cuda::getCurrentCUDAStream(a.device).stream()) != FA_OK) return nullptr;
    Py_RETURN_TRUE;
  });
}

// (cache, device, bounds, seq_lens, first)
PyObject* bounds(PyObject*, PyObject* const* argv, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    Args a{argv};
    const fa_paged_cache* c = cache_of(a, 0);
    const fa_page_bounds_pool* pool = reinterpret_cast<const fa_page_bounds_pool*>(a.integer(2));
    if (!a.ok) return nullptr;
    const int32_t* lens = a.flat<int32_t>(3, at::kInt, c->B, false);
    const int32_t* first = a.ok ? a.flat<int32_t>(4, at::kInt, c->B, true) : nullptr;
    if (!a.here() || fn.bounds(c, pool, first, lens, c10::cuda::getCurrentCUDAStream(a.device).stream()) != FA_OK) return nullptr;
    Py_RETURN_TRUE;
  });
}

// (q, cache, device, bounds, seq_lens, K, scale, first, last, alibi_slopes)
PyObject* select_pages(PyObject*, PyObject* const* argv, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    Args a{argv};
    const fa_paged_cache* c = cache_of(a, 1);
    const fa_page_bounds_pool* pool = reinterpret_cast<const fa_page_bounds_pool*>(a.integer(3));
    if (!a.ok) return nullptr;
    const at::Tensor* q = a.tensor(0);
    if (!a.ok || q->dim() != 3) return nullptr;
    const at::ScalarType xt = q->scalar_type();
    const int64_t B = c->B, H = q->size(1);
    a.heads(0, xt, B, c->D);
    const int32_t* lens = a.ok ? a.flat<int32_t>(4, at::kInt, B, false) : nullptr;
    const float* alibi = a.ok ? a.flat<float>(9, at::kFloat, H, true) : nullptr;
    const long long K = a.integer(5), first = a.integer(7), last = a.integer(8);
    const double scale = a.number(6);
    if (!a.here() || act_of(xt) < 0 || K < 1 || K > INT32_MAX || first < 0 || first > K || last < 0 || last > K) return nullptr;
    const size_t need = fn.select_ws(c, H, (int)K);
    if (!need) return nullptr;
    const at::Tensor pages = make({B, c->Hkv, (int64_t)K}, at::kInt, a.device), ws = make({(int64_t)need}, at::kByte, a.device);
    if (fn.select(at_of(q), act_of(xt), q->stride(0), q->stride(1), c, pool, lens, H, (float)scale, alibi, (int)K, (int)first, (int)last,
                  static_cast<int32_t*>(pages.data_ptr()), ws.data_ptr(), need, c10::cuda::getCurrentCUDAStream(a.device).stream()) != FA_OK)
      return nullptr;
    return THPVariable_Wrap(pages);
  });
}

// The addresses of libfa_back.so's entry points, in Entry's order
PyObject* bind(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  if (n != kEntries) return PyErr_Format(PyExc_TypeError, "%d addresses expected", kEntries);
  void* p[kEntries];
  for (int i = 0; i < kEntries; ++i)
    if (!(p[i] = PyLong_AsVoidPtr(argv[i]))) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "address 0");
  int i = 0;
  auto take = [&](auto& entry) { entry = reinterpret_cast<std::decay_t<decltype(entry)>>(p[i++]); };
  take(fn.norm), take(fn.norm_back), take(fn.norm_back_ws), take(fn.append), take(fn.read), take(fn.decode), take(fn.decode_ws);
  take(fn.norm_axes), take(fn.norm_axes_back), take(fn.append_axes), take(fn.decode_pages), take(fn.extend), take(fn.trim);
  take(fn.bounds), take(fn.select), take(fn.select_ws);
  Py_RETURN_NONE;
}

// n arguments, of which the last `more` may be left out (None then)
#define FAST(name, n, more)                                                                                \
  PyObject* py_##name(PyObject* self, PyObject* const* argv, Py_ssize_t argc) {                            \
    if (argc > n || argc < n - more || !fn.norm)                                                           \
      return PyErr_Format(PyExc_TypeError, #name ": %d arguments, after bind()", n);                       \
    PyObject* all[n];                                                                                      \
    for (Py_ssize_t i = 0; i < n; ++i) all[i] = i < argc ? argv[i] : Py_None;                              \
    return name(self, all, n);                                                                             \
  }
FAST(norm, 10, 1)
FAST(norm_back, 11, 1)
FAST(append, 12, 2)
FAST(read, 5, 0)
FAST(decode, 9, 1)
FAST(extend, 4, 0)
FAST(trim, 3, 0)
FAST(bounds, 5, 0)
FAST(select_pages, 10, 0)

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_norm)), METH_FASTCALL, nullptr},
    {"norm_back", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_norm_back)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_append)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_read)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_decode)), METH_FASTCALL, nullptr},
    {"extend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_extend)), METH_FASTCALL, nullptr},
    {"trim", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_trim)), METH_FASTCALL, nullptr},
    {"bounds", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_bounds)), METH_FASTCALL, nullptr},
    {"select", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_select_pages)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", "plain calls of paged.py and pages.py", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast(void) {
  PyObject** names[] = {&s_q, &s_k, &s_v, &s_O, &s_lse, &s_dq, &s_dk, &s_dwq, &s_dwk, &s_seq, &s_pos, &s_row, &s_starts, &s_first};
  const char* text[] = {"q", "k", "v", "O", "lse", "dq", "dk", "dwq", "dwk", "seq", "pos", "row", "starts", "first"};
  for (int i = 0; i < 14; ++i) *names[i] = PyUnicode_InternFromString(text[i]);
  return PyModule_Create(&module);
}

// Linked without the compiler's start files: their exit routine is all that the module would run when the process ends,
// and it would run from this file.  A process whose file was written anew in place after its last call ends in order so;
// nothing else about such a process is safe, a call into the module least of all (build.py writes beside the old file
// and renames, which leaves a process the file that it has loaded).  The one symbol of the start files that the headers name (a
// place that is registered with destructors of function-local objects):
asm(".pushsection .data\n.hidden __dso_handle\n.globl __dso_handle\n.balign 8\n__dso_handle: .quad __dso_handle\n.popsection");
