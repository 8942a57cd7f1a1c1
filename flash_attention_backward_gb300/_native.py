"""ctypes binding of libfa_back.so: the C ABI under the same names, argument marshalling only."""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa_back.so")

FA_F32, FA_F16, FA_Q8_0, FA_Q4_0 = 0, 1, 2, 3
STATUS = {0: "FA_OK", 1: "FA_ERR_NULL", 2: "FA_ERR_TYPE", 3: "FA_ERR_SHAPE", 4: "FA_ERR_ALIGN",
          5: "FA_ERR_UNSUPPORTED", 6: "FA_ERR_DEVICE", 7: "FA_ERR_CUDA", 8: "FA_ERR_TIMEOUT",
          9: "FA_ERR_WORKSPACE", 10: "FA_ERR_PAGE"}

FA_MASK_F16, FA_MASK_BITS = 0, 1

# fa_paged.h
FA_ACT_F32, FA_ACT_F16, FA_ACT_BF16, FA_ACT_RAW = 0, 1, 2, 3
FA_ROPE_PAIRS, FA_ROPE_HALVES = 0, 1

_lib = None


class fa_strides(ctypes.Structure):
    """struct fa_strides of the header: element strides of Q and dO, byte strides of the K and V
    rows, word strides of the mask."""
    _fields_ = [(n, ctypes.c_int64) for n in ("q_row", "q_head", "q_comp", "do_row", "do_head", "do_comp",
                                             "k_cell", "k_head", "v_cell", "v_head", "mask_head", "mask_row")]


class fa_rope(ctypes.Structure):
    """struct fa_rope of fa_paged.h."""
    _fields_ = [("freqs", ctypes.c_void_p), ("n_rot", ctypes.c_int32), ("style", ctypes.c_int32)]


class fa_qk_views(ctypes.Structure):
    """struct fa_qk_views of fa_paged.h (element strides)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("q_row", "q_head", "k_row", "k_head")]


class fa_kv_views(ctypes.Structure):
    """struct fa_kv_views of fa_paged.h (element strides)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("k_row", "k_head", "v_row", "v_head")]


class fa_paged_cache(ctypes.Structure):
    """struct fa_paged_cache of fa_paged.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "page_table")] + [
        (n, ctypes.c_int32) for n in ("k_type", "v_type", "num_pages", "page_size", "B", "max_pages", "Hkv", "D", "Dv")]


class fa_rope_axes(ctypes.Structure):
    """struct fa_rope_axes of fa_paged_ext.h."""
    _fields_ = [("freqs", ctypes.c_void_p), ("axis", ctypes.c_void_p), ("pos_stride", ctypes.c_int64), ("n_rot", ctypes.c_int32),
                ("style", ctypes.c_int32), ("n_axes", ctypes.c_int32)]


class fa_page_lists(ctypes.Structure):
    """struct fa_page_lists of fa_paged_ext.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("page_table", "seq_lens", "free_pages", "num_free")] + [
        (n, ctypes.c_int32) for n in ("num_pages", "page_size", "B", "max_pages")]


class fa_page_bounds_pool(ctypes.Structure):
    """struct fa_page_bounds_pool of fa_paged_ext.h."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class NativeLibraryMissing(RuntimeError):
    """libfa_back.so is not built or cannot be loaded; there is no fallback path."""


def lib():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise NativeLibraryMissing(
            f"{LIB_PATH} is missing: build it with `python -m flash_attention_backward_gb300.build`")
    try:
        L = ctypes.CDLL(LIB_PATH)
    except OSError as e:  # pragma: no cover - depends on the machine
        raise NativeLibraryMissing(f"cannot load {LIB_PATH}: {e}") from e
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.fa_row_bytes.restype = ctypes.c_long
    L.fa_row_bytes.argtypes = [i, i]
    L.fa_back_workspace_size.restype = sz
    L.fa_back_workspace_size.argtypes = [i] * 6
    L.fa_back_workspace_size_min.restype = sz
    L.fa_back_workspace_size_min.argtypes = [i] * 6
    L.fa_back_plan_info.restype = i
    L.fa_back_plan_info.argtypes = [i] * 6 + [sz, vp, vp, vp]
    L.fa_back.restype = i
    L.fa_back.argtypes = [vp, vp, i, vp, i, vp, i, vp, f, i, i, i, i, i, i, i, vp, vp, vp, vp, vp, vp, sz, vp]
    L.fa_back_nocopy.restype = i
    L.fa_back_nocopy.argtypes = [vp, vp, i, vp, i, vp, i, vp, f, i, i, i, i, i, i, i, vp, vp, vp, vp, vp, vp, sz, vp]
    L.fa_back_workspace_size_nocopy.restype = sz
    L.fa_back_workspace_size_nocopy.argtypes = [i] * 6
    L.fa_back_ext.restype = i
    L.fa_back_ext.argtypes = [vp, vp, i, vp, i, vp, i, vp, f, i, i, i, i, i, i, i, vp, f, vp, vp, vp, vp, vp, vp, vp,
                              vp, sz, vp]
    L.fa_back_with_stats.restype = i
    L.fa_back_with_stats.argtypes = [vp, vp, i, vp, i, vp, i, vp, vp, vp, f, i, i, i, i, i, i, i, vp, vp, vp, vp, sz,
                                     vp]
    L.fa_back_batched.restype = i
    L.fa_back_batched.argtypes = [i, vp, vp, i, vp, i, vp, i, i, vp, f, i, i, i, i, i, i, i, vp, vp, vp, vp, vp, vp,
                                  sz, vp]
    L.fa_back_strided_workspace_size.restype = sz
    L.fa_back_strided_workspace_size.argtypes = [i] * 9
    L.fa_back_strided.restype = i
    L.fa_back_strided.argtypes = [vp, vp, i, vp, i, vp, i, i, vp, ctypes.POINTER(fa_strides), f, i, i, i, i, i, i, i,
                                  vp, vp, vp, vp, vp, vp, sz, vp]
    L.fa_forward_workspace_size.restype = sz
    L.fa_forward_workspace_size.argtypes = [i] * 6
    L.fa_forward.restype = i
    L.fa_forward.argtypes = [vp, vp, i, vp, i, vp, i, f, i, i, i, i, i, i, i, vp, vp, vp, sz, vp]
    L.fa_back_get_error.restype = i
    L.fa_back_get_error.argtypes = []
    L.fa_back_status_string.restype = ctypes.c_char_p
    L.fa_back_status_string.argtypes = [i]
    L.fa_back_noalloc.restype = i
    L.fa_back_noalloc.argtypes = [vp, vp, i, vp, i, vp, i, vp, f, i, i, i, i, i, i, i, vp, vp, vp, vp, vp, vp]
    L.fa_back_test_wait_limit.restype = i
    L.fa_back_test_wait_limit.argtypes = [ctypes.c_ulonglong]
    L.fa_back_selftest_timeout.restype = i
    L.fa_back_selftest_timeout.argtypes = [ctypes.c_ulonglong, vp]
    L.fa_back_profile.restype = i
    L.fa_back_profile.argtypes = [i]
    L.fa_back_profile_read.restype = i
    L.fa_back_profile_read.argtypes = [vp, vp, vp, i]
    P, i64 = ctypes.POINTER, ctypes.c_int64
    L.fa_rope_frequencies.restype = i
    L.fa_rope_frequencies.argtypes = [i, ctypes.c_double, ctypes.c_double, vp, vp]
    L.fa_qk_norm_rope.restype = i
    L.fa_qk_norm_rope.argtypes = [vp, vp, i, P(fa_qk_views), vp, vp, f, vp, P(fa_rope), i, i, i, i, vp, vp, i, vp]
    L.fa_qk_norm_rope_backward_workspace_size.restype = sz
    L.fa_qk_norm_rope_backward_workspace_size.argtypes = [i] * 4
    L.fa_qk_norm_rope_backward.restype = i
    L.fa_qk_norm_rope_backward.argtypes = [vp, vp, i, vp, vp, i, P(fa_qk_views), vp, vp, f, vp, P(fa_rope), i, i, i, i,
                                           vp, vp, vp, vp, vp, sz, vp]
    L.fa_cache_append.restype = i
    L.fa_cache_append.argtypes = [vp, vp, i, P(fa_kv_views), P(fa_paged_cache), vp, vp, i, vp, f, P(fa_rope), vp]
    L.fa_cache_read.restype = i
    L.fa_cache_read.argtypes = [P(fa_paged_cache), vp, vp, i, i, vp, vp, vp]
    L.fa_paged_decode_workspace_size.restype = sz
    L.fa_paged_decode_workspace_size.argtypes = [P(fa_paged_cache), i]
    L.fa_paged_decode.restype = i
    L.fa_paged_decode.argtypes = [vp, i, i64, i64, P(fa_paged_cache), vp, i, f, vp, f, vp, vp, vp, vp, sz, vp]
    L.fa_qk_norm_rope_axes.restype = i
    L.fa_qk_norm_rope_axes.argtypes = [vp, vp, i, P(fa_qk_views), vp, vp, f, vp, P(fa_rope_axes), i, i, i, i, vp, vp, i, vp]
    L.fa_qk_norm_rope_axes_backward.restype = i
    L.fa_qk_norm_rope_axes_backward.argtypes = [vp, vp, i, vp, vp, i, P(fa_qk_views), vp, vp, f, vp, P(fa_rope_axes), i, i, i,
                                                i, vp, vp, vp, vp, vp, sz, vp]
    L.fa_cache_append_axes.restype = i
    L.fa_cache_append_axes.argtypes = [vp, vp, i, P(fa_kv_views), P(fa_paged_cache), vp, vp, i, vp, f, vp, P(fa_rope_axes), vp]
    L.fa_pages_extend.restype = i
    L.fa_pages_extend.argtypes = [P(fa_page_lists), vp, i, vp, vp, vp, vp, vp, vp]
    L.fa_pages_trim.restype = i
    L.fa_pages_trim.argtypes = [P(fa_page_lists), vp, vp]
    L.fa_page_bounds.restype = i
    L.fa_page_bounds.argtypes = [P(fa_paged_cache), P(fa_page_bounds_pool), vp, vp, vp]
    L.fa_page_select_workspace_size.restype = sz
    L.fa_page_select_workspace_size.argtypes = [P(fa_paged_cache), i, i]
    L.fa_page_select.restype = i
    L.fa_page_select.argtypes = [vp, i, i64, i64, P(fa_paged_cache), P(fa_page_bounds_pool), vp, i, f, vp, i, i, i, vp, vp, sz, vp]
    L.fa_paged_decode_pages.restype = i
    L.fa_paged_decode_pages.argtypes = [vp, i, i64, i64, P(fa_paged_cache), vp, vp, i, i, f, vp, f, vp, vp, vp, vp, sz, vp]
    _lib = L
    return L


def fa_row_bytes(type_: int, D: int) -> int:
    return int(lib().fa_row_bytes(type_, D))


def fa_back_workspace_size(N: int, M: int, H: int, Hkv: int, D: int, Dv: int) -> int:
    return int(lib().fa_back_workspace_size(N, M, H, Hkv, D, Dv))


def fa_back_workspace_size_min(N: int, M: int, H: int, Hkv: int, D: int, Dv: int) -> int:
    return int(lib().fa_back_workspace_size_min(N, M, H, Hkv, D, Dv))


def fa_back_plan_info(N: int, M: int, H: int, Hkv: int, D: int, Dv: int, workspace_bytes: int):
    """(status, level, key_splits, plan_bytes) of the plan fa_back runs with this workspace."""
    level, splits, nbytes = ctypes.c_int(-1), ctypes.c_int(0), ctypes.c_size_t(0)
    rc = int(lib().fa_back_plan_info(N, M, H, Hkv, D, Dv, workspace_bytes, ctypes.byref(level), ctypes.byref(splits),
                                     ctypes.byref(nbytes)))
    return rc, level.value, splits.value, nbytes.value


def fa_back(q, k, k_type, v, v_type, mask, mask_heads, dO, scale, N, M, H, Hkv, D, Dv, causal,
            dQ, dK, dV, lse, delta, workspace, workspace_bytes, stream) -> int:
    """Direct call of the C entry point; pointers are integers (device addresses) or None."""
    return int(lib().fa_back(q, k, k_type, v, v_type, mask, mask_heads, dO, float(scale), N, M, H, Hkv, D, Dv,
                             int(causal), dQ, dK, dV, lse, delta, workspace, workspace_bytes, stream))


def fa_back_nocopy(q, k, k_type, v, v_type, mask, mask_heads, dO, scale, N, M, H, Hkv, D, Dv, causal,
                   dQ, dK, dV, lse, delta, workspace, workspace_bytes, stream) -> int:
    """fa_back restricted to the plans without a decoded copy of the cache (levels 3 and 0)."""
    return int(lib().fa_back_nocopy(q, k, k_type, v, v_type, mask, mask_heads, dO, float(scale), N, M, H, Hkv, D,
                                    Dv, int(causal), dQ, dK, dV, lse, delta, workspace, workspace_bytes, stream))


def fa_back_workspace_size_nocopy(N: int, M: int, H: int, Hkv: int, D: int, Dv: int) -> int:
    return int(lib().fa_back_workspace_size_nocopy(N, M, H, Hkv, D, Dv))


def fa_back_ext(q, k, k_type, v, v_type, mask, mask_heads, dO, scale, N, M, H, Hkv, D, Dv, causal,
                alibi_slopes, softcap, sinks, dsinks, dQ, dK, dV, lse, delta, workspace, workspace_bytes,
                stream) -> int:
    """fa_back with the score extensions (ALiBi slopes, soft cap, sink logits); see the header."""
    return int(lib().fa_back_ext(q, k, k_type, v, v_type, mask, mask_heads, dO, float(scale), N, M, H, Hkv, D, Dv,
                                 int(causal), alibi_slopes, float(softcap), sinks, dsinks, dQ, dK, dV, lse, delta,
                                 workspace, workspace_bytes, stream))


def fa_back_with_stats(q, k, k_type, v, v_type, mask, mask_heads, dO, lse, delta, scale, N, M, H, Hkv, D, Dv,
                       causal, dQ, dK, dV, workspace, workspace_bytes, stream) -> int:
    return int(lib().fa_back_with_stats(q, k, k_type, v, v_type, mask, mask_heads, dO, lse, delta, float(scale), N,
                                        M, H, Hkv, D, Dv, int(causal), dQ, dK, dV, workspace, workspace_bytes,
                                        stream))


def fa_back_batched(B, q, k, k_type, v, v_type, mask, mask_heads, mask_per_batch, dO, scale, N, M, H, Hkv, D, Dv,
                    causal, dQ, dK, dV, lse, delta, workspace, workspace_bytes, stream) -> int:
    return int(lib().fa_back_batched(B, q, k, k_type, v, v_type, mask, mask_heads, int(mask_per_batch), dO,
                                     float(scale), N, M, H, Hkv, D, Dv, int(causal), dQ, dK, dV, lse, delta,
                                     workspace, workspace_bytes, stream))


def fa_back_strided_workspace_size(N: int, M: int, H: int, Hkv: int, D: int, Dv: int, k_type: int, v_type: int,
                                   mask_heads: int) -> int:
    return int(lib().fa_back_strided_workspace_size(N, M, H, Hkv, D, Dv, k_type, v_type, mask_heads))


def fa_back_strided(q, k, k_type, v, v_type, mask, mask_format, mask_heads, dO, strides, scale, N, M, H, Hkv, D, Dv,
                    causal, dQ, dK, dV, lse, delta, workspace, workspace_bytes, stream) -> int:
    """strides: an fa_strides, or None for a NULL pointer."""
    st = None if strides is None else ctypes.byref(strides)
    return int(lib().fa_back_strided(q, k, k_type, v, v_type, mask, mask_format, mask_heads, dO, st, float(scale), N,
                                     M, H, Hkv, D, Dv, int(causal), dQ, dK, dV, lse, delta, workspace,
                                     workspace_bytes, stream))


def fa_forward_workspace_size(N: int, M: int, H: int, Hkv: int, D: int, Dv: int) -> int:
    return int(lib().fa_forward_workspace_size(N, M, H, Hkv, D, Dv))


def fa_forward(q, k, k_type, v, v_type, mask, mask_heads, scale, N, M, H, Hkv, D, Dv, causal, O, lse,
               workspace, workspace_bytes, stream) -> int:
    return int(lib().fa_forward(q, k, k_type, v, v_type, mask, mask_heads, float(scale), N, M, H, Hkv, D, Dv,
                                int(causal), O, lse, workspace, workspace_bytes, stream))


def fa_back_get_error() -> int:
    return int(lib().fa_back_get_error())


def fa_back_status_string(status: int) -> str:
    return lib().fa_back_status_string(status).decode()


def fa_back_profile(enable: bool) -> int:
    return int(lib().fa_back_profile(1 if enable else 0))


def fa_back_profile_read(max_kernels: int = 32) -> dict:
    """{kernel name: (summed ms, launches)} of the recorded fa_back calls; clears the record."""
    ms = (ctypes.c_float * max_kernels)()
    cnt = (ctypes.c_int * max_kernels)()
    names = (ctypes.c_char_p * max_kernels)()
    n = int(lib().fa_back_profile_read(ms, cnt, names, max_kernels))
    return {names[k].decode(): (float(ms[k]), int(cnt[k])) for k in range(n) if cnt[k] > 0}


NOALLOC_SCRATCH_BYTES = 64 << 20


def fa_back_noalloc(q, k, k_type, v, v_type, mask, mask_heads, dO, scale, N, M, H, Hkv, D, Dv, causal,
                    dQ, dK, dV, lse, delta, stream) -> int:
    """fa_back with the library's static scratch instead of a caller workspace (see the header)."""
    return int(lib().fa_back_noalloc(q, k, k_type, v, v_type, mask, mask_heads, dO, float(scale), N, M, H, Hkv,
                                     D, Dv, int(causal), dQ, dK, dV, lse, delta, stream))


def fa_back_selftest_timeout(limit_ns: int, stream=None) -> int:
    return int(lib().fa_back_selftest_timeout(limit_ns, stream))


def fa_back_test_wait_limit(limit_ns: int) -> int:
    """Failure-detection hook: the next call's kernels give up on waits longer than limit_ns."""
    return int(lib().fa_back_test_wait_limit(limit_ns))


# ---- fa_paged.h.  Structures (or None for a NULL pointer) go where the header takes pointers to them:
# ctypes passes their address.

def fa_rope_frequencies(n_rot: int, base: float, scale: float, factors, out) -> int:
    """factors, out: host addresses (float32 and uint64 arrays of n_rot / 2) or None."""
    return lib().fa_rope_frequencies(n_rot, base, scale, factors, out)


def fa_qk_norm_rope(q, k, x_type, views, wq, wk, eps, pos, rope, N, H, Hkv, D, q_out, k_out, y_type, stream) -> int:
    return (_lib or lib()).fa_qk_norm_rope(q, k, x_type, views, wq, wk, eps, pos, rope, N, H, Hkv, D, q_out, k_out,
                                           y_type, stream)


def fa_qk_norm_rope_backward_workspace_size(N: int, H: int, Hkv: int, D: int) -> int:
    return (_lib or lib()).fa_qk_norm_rope_backward_workspace_size(N, H, Hkv, D)


def fa_qk_norm_rope_backward(gq, gk, y_type, q, k, x_type, views, wq, wk, eps, pos, rope, N, H, Hkv, D, dq, dk, dwq,
                             dwk, workspace, workspace_bytes, stream) -> int:
    return (_lib or lib()).fa_qk_norm_rope_backward(gq, gk, y_type, q, k, x_type, views, wq, wk, eps, pos, rope, N, H,
                                                    Hkv, D, dq, dk, dwq, dwk, workspace, workspace_bytes, stream)


def fa_cache_append(k, v, x_type, views, cache, seq, pos, T, k_norm, eps, rope, stream) -> int:
    return (_lib or lib()).fa_cache_append(k, v, x_type, views, cache, seq, pos, T, k_norm, eps, rope, stream)


def fa_cache_read(cache, seq, pos, T, y_type, k_out, v_out, stream) -> int:
    return (_lib or lib()).fa_cache_read(cache, seq, pos, T, y_type, k_out, v_out, stream)


def fa_paged_decode_workspace_size(cache, H: int) -> int:
    return (_lib or lib()).fa_paged_decode_workspace_size(cache, H)


def fa_paged_decode(q, act, q_row, q_head, cache, seq_lens, H, scale, alibi_slopes, softcap, sinks, O, lse, workspace,
                    workspace_bytes, stream) -> int:
    return (_lib or lib()).fa_paged_decode(q, act, q_row, q_head, cache, seq_lens, H, scale, alibi_slopes, softcap,
                                           sinks, O, lse, workspace, workspace_bytes, stream)


# ---- fa_paged_ext.h

def fa_qk_norm_rope_axes(q, k, x_type, views, wq, wk, eps, pos, rope, N, H, Hkv, D, q_out, k_out, y_type, stream) -> int:
    return (_lib or lib()).fa_qk_norm_rope_axes(q, k, x_type, views, wq, wk, eps, pos, rope, N, H, Hkv, D, q_out, k_out,
                                                y_type, stream)


def fa_qk_norm_rope_axes_backward(gq, gk, y_type, q, k, x_type, views, wq, wk, eps, pos, rope, N, H, Hkv, D, dq, dk, dwq,
                                  dwk, workspace, workspace_bytes, stream) -> int:
    return (_lib or lib()).fa_qk_norm_rope_axes_backward(gq, gk, y_type, q, k, x_type, views, wq, wk, eps, pos, rope, N, H,
                                                         Hkv, D, dq, dk, dwq, dwk, workspace, workspace_bytes, stream)


def fa_cache_append_axes(k, v, x_type, views, cache, seq, pos, T, k_norm, eps, rope_pos, rope, stream) -> int:
    return (_lib or lib()).fa_cache_append_axes(k, v, x_type, views, cache, seq, pos, T, k_norm, eps, rope_pos, rope, stream)


def fa_pages_extend(lists, new_tokens, T, starts, first, seq, pos, row, stream) -> int:
    return (_lib or lib()).fa_pages_extend(lists, new_tokens, T, starts, first, seq, pos, row, stream)


def fa_pages_trim(lists, keep, stream) -> int:
    return (_lib or lib()).fa_pages_trim(lists, keep, stream)


def fa_page_bounds(cache, bounds, first, seq_lens, stream) -> int:
    return (_lib or lib()).fa_page_bounds(cache, bounds, first, seq_lens, stream)


def fa_page_select_workspace_size(cache, H: int, K: int) -> int:
    return (_lib or lib()).fa_page_select_workspace_size(cache, H, K)


def fa_page_select(q, act, q_row, q_head, cache, bounds, seq_lens, H, scale, alibi_slopes, K, first, last, pages, workspace,
                   workspace_bytes, stream) -> int:
    return (_lib or lib()).fa_page_select(q, act, q_row, q_head, cache, bounds, seq_lens, H, scale, alibi_slopes, K, first,
                                          last, pages, workspace, workspace_bytes, stream)


def fa_paged_decode_pages(q, act, q_row, q_head, cache, seq_lens, pages, K, H, scale, alibi_slopes, softcap, sinks, O, lse,
                          workspace, workspace_bytes, stream) -> int:
    return (_lib or lib()).fa_paged_decode_pages(q, act, q_row, q_head, cache, seq_lens, pages, K, H, scale, alibi_slopes,
                                                 softcap, sinks, O, lse, workspace, workspace_bytes, stream)
