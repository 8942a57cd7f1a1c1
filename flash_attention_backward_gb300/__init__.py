"""GB300 (sm_103a) flash-attention backward over a raw F32/F16/q8_0/q4_0 K/V cache.

The computation lives in libfa_back.so (hand-written CUDA, C ABI in include/fa_back.h).
This package only marshals arguments: ``_native`` mirrors the C entry points under the same
names, and ``backward`` allocates outputs and workspace with PyTorch and calls ``fa_back``
on the current stream.  ``paged`` does the same for include/fa_paged.h: the paged cache (append,
read, single-token attention) and the per-head norm and rotation with its gradient, and ``pages`` for
include/fa_paged_ext.h: page lists, page bounds and the selection of pages.
"""
from ._native import (  # noqa: F401
    FA_F16, FA_F32, FA_MASK_BITS, FA_MASK_F16, FA_Q4_0, FA_Q8_0, STATUS, NativeLibraryMissing, LIB_PATH,
    fa_back, fa_back_batched, fa_back_ext, fa_back_get_error, fa_back_noalloc, fa_back_nocopy, fa_back_plan_info,
    fa_back_profile, fa_back_workspace_size_nocopy,
    fa_back_profile_read, fa_back_selftest_timeout, fa_back_status_string, fa_back_strided,
    fa_back_strided_workspace_size, fa_back_test_wait_limit, fa_strides,
    fa_back_with_stats, fa_back_workspace_size, fa_back_workspace_size_min, fa_forward, fa_forward_workspace_size,
    fa_row_bytes, lib,
    FA_ACT_BF16, FA_ACT_F16, FA_ACT_F32, FA_ACT_RAW, FA_ROPE_HALVES, FA_ROPE_PAIRS, fa_cache_append, fa_cache_read,
    fa_kv_views, fa_paged_cache, fa_paged_decode, fa_paged_decode_workspace_size, fa_qk_norm_rope,
    fa_qk_norm_rope_backward, fa_qk_norm_rope_backward_workspace_size, fa_qk_views, fa_rope, fa_rope_frequencies,
    fa_cache_append_axes, fa_page_bounds, fa_page_bounds_pool, fa_page_lists, fa_page_select, fa_page_select_workspace_size,
    fa_paged_decode_pages, fa_pages_extend, fa_pages_trim, fa_qk_norm_rope_axes, fa_qk_norm_rope_axes_backward, fa_rope_axes,
)
from .api import FaBackError, Workspace, backward, backward_strided, forward  # noqa: F401
from .paged import (  # noqa: F401
    PagedCache, cache_append, cache_read, paged_decode, qk_norm_rope, qk_norm_rope_backward, rope_frequencies,
)
from .pages import (  # noqa: F401
    PageBounds, PageLists, page_bounds, page_select, pages_extend, pages_trim, rope_sections,
)
