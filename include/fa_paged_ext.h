/*
 * fa_paged_ext.h -- C ABI of what serves around the paged cache of fa_paged.h (same library, same types,
 * status codes and conventions):
 *
 *   fa_qk_norm_rope_axes, fa_qk_norm_rope_axes_backward, fa_cache_append_axes
 *                       norm, rotation and append with positions of several axes (time, height and
 *                       width of images and video)
 *   fa_pages_extend     page tables, lengths and the slots of new tokens, from the requests' lengths
 *   fa_pages_trim       pages behind a length go back
 *   fa_page_bounds      the largest and smallest component of each page's keys, in 8 bits
 *   fa_page_select      the pages whose bounds promise each query the largest scores
 *   fa_paged_decode_pages
 *                       attention of one new token per sequence over selected pages
 *
 * A decode step of long contexts is, in this order: fa_pages_extend, the norm and rotation of the queries,
 * fa_cache_append, fa_page_bounds, fa_page_select and fa_paged_decode_pages.
 */
#ifndef FA_PAGED_EXT_H
#define FA_PAGED_EXT_H

#include "fa_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The rotation by positions of several axes: pair i of token n's heads turns by
 * pos[axis[i] * pos_stride + n] * freqs[i]; everything else is as in fa_rope.  axis [n_rot / 2] (device)
 * holds an axis 0 .. n_axes-1 for each pair (one of n_axes or more counts as the last); n_axes is 1 .. 8 and
 * pos_stride >= 0 (in elements; N where the axes' positions [n_axes][N] lie one after another).  A NULL
 * pointer to this structure, freqs NULL or n_rot 0: no rotation.
 */
typedef struct fa_rope_axes {
  const uint64_t* freqs;
  const uint8_t* axis;
  int64_t pos_stride;
  int32_t n_rot, style, n_axes;
} fa_rope_axes;

/* fa_qk_norm_rope() and its gradient with positions pos [n_axes][N] of several axes.  Workspace:
 * fa_qk_norm_rope_backward_workspace_size(). */
fa_status fa_qk_norm_rope_axes(const void* q, const void* k, int x_type, const fa_qk_views* views, const float* wq,
                               const float* wk, float eps, const int32_t* pos, const fa_rope_axes* rope, int N, int H,
                               int Hkv, int D, void* q_out, void* k_out, int y_type, void* stream);
fa_status fa_qk_norm_rope_axes_backward(const void* gq, const void* gk, int y_type, const void* q, const void* k,
                                        int x_type, const fa_qk_views* views, const float* wq, const float* wk,
                                        float eps, const int32_t* pos, const fa_rope_axes* rope, int N, int H, int Hkv,
                                        int D, void* dq, void* dk, float* dwq, float* dwk, void* workspace,
                                        size_t workspace_bytes, void* stream);

/* fa_cache_append() with keys rotated by positions rope_pos [n_axes][T] of several axes; pos[t] only says
 * where token t is stored. */
fa_status fa_cache_append_axes(const void* k, const void* v, int x_type, const fa_kv_views* views,
                               const fa_paged_cache* cache, const int32_t* seq, const int32_t* pos, int T,
                               const float* k_norm, float eps, const int32_t* rope_pos, const fa_rope_axes* rope,
                               void* stream);

/*
 * Who holds which page: the page table and lengths of B requests, and the pages that nobody holds, as a
 * stack free_pages[0 .. num_free[0]) of which the last one is taken first.  All in device memory and edited in
 * place.  A request holds the first ceil(seq_lens[b] / page_size) entries of its row; a negative length marks
 * a slot without a request.  A new request is a length of 0; one that has ended is trimmed to 0.  A page is on the
 * stack or held by one request, once.
 * num_pages * page_size < 2^31, max_pages * page_size <= 2^30, B <= 2^20 (else FA_ERR_UNSUPPORTED).
 * Alignment: 4 bytes.
 */
typedef struct fa_page_lists {
  int32_t* page_table; /* [B][max_pages]                                */
  int32_t* seq_lens;   /* [B]                                           */
  int32_t* free_pages; /* [num_pages]                                   */
  int32_t* num_free;   /* [1]                                           */
  int32_t num_pages, page_size, B, max_pages;
} fa_page_lists;

/*
 * Makes room for new_tokens[b] further tokens of each request b and says where they go.  The call's tokens are
 * numbered request by request: those of b are starts[b] .. starts[b+1]-1, and token t of a request of length L
 * is its position pos[t] = L + t - starts[b], stored in row row[t] = page * page_size + offset of the pools;
 * seq[t] = b.  These seq and pos are what fa_cache_append() takes.  Then seq_lens[b] grows by new_tokens[b].
 * Tokens behind the last one, up to T, get seq = pos = row = -1.
 *   A request gets room for all its tokens or for none.  Pages are handed out in the order of the requests; a
 * request that needs some is refused when those that it and the requests before it ask for are more than there
 * are, or when its tokens would not fit its table row (it then asks for none) or end behind T (likewise).
 * A refused request keeps its length, and its tokens get seq = pos = row = -1: padding for fa_cache_append().
 *   first[b] is the length before the call, where the request's new tokens begin, or -1 for a request that gets
 * none (refused, new_tokens[b] <= 0 or no request): what fa_page_bounds() takes.
 * starts [B+1] (clamped at T), first [B], seq, pos, row [T]; T <= 2^30 (else FA_ERR_UNSUPPORTED).  A num_free
 * outside [0, num_pages] counts as the nearest of them.  Page numbers are handed on as they are; where one is
 * outside [0, num_pages), row is -1 and fa_back_get_error() reports FA_ERR_PAGE.
 */
fa_status fa_pages_extend(const fa_page_lists* lists, const int32_t* new_tokens, int T, int32_t* starts, int32_t* first,
                          int32_t* seq, int32_t* pos, int32_t* row, void* stream);

/*
 * Shortens each request b to keep[b] positions (tokens that were rejected; 0 for a request that has ended) and
 * gives the pages behind them back, the one that would have been taken last first: trimming to the lengths
 * before a fa_pages_extend() call undoes it.  Their table entries become -1.  A negative keep[b], or one that is
 * not below the length, leaves the request as it is.  Pages for which the stack has no place (more than
 * num_pages in all: one was given back twice) are dropped, and fa_back_get_error() reports FA_ERR_PAGE.
 */
fa_status fa_pages_trim(const fa_page_lists* lists, const int32_t* keep, void* stream);

/*
 * Bounds of a page's keys, for each KV head: codes [num_pages][Hkv][2][D] (int8; [0] of the largest, [1] of the
 * smallest components) and scales [num_pages][Hkv][D / 32] (f32).  With hi and lo the largest and smallest value of
 * a component over the page's rows below seq_lens[b], and fl() a rounding to f32, in blocks of 32 components:
 *   m = max(|hi|, |lo|);  d = fl(m / 127);  codes ceil(fl(hi / d)) and floor(fl(lo / d)), within -127 .. 127
 * (d and codes 0 where m <= 1e-30): code * d bounds the keys, but for a rounding.  A NaN does not enter hi and lo
 * (a component of NaNs only has hi = -inf and lo = inf); with m infinite the scale is, and the codes are 127 and -127.
 * (A q8_0 or q4_0 block whose stored scale is infinite counts as infinite, whatever its codes.)
 *   Computed for the pages of positions first[b] .. seq_lens[b]-1 of each sequence b, from all their rows
 * (first NULL: from 0; a negative first[b], or one that is not below the length: none; a length beyond the table counts
 * as the table's).  Other pages' bounds are left as they were; those of a page that fa_pages_trim() has cut go on covering
 * what it held until they are computed again.  Sequences of a call that hold the same page hold as many of its rows each (a
 * common prefix of whole pages); otherwise its bounds are not defined.  D of the cache.  Alignment: codes and scales 16 bytes.
 */
typedef struct fa_page_bounds_pool {
  int8_t* codes;
  float* scales;
} fa_page_bounds_pool;

fa_status fa_page_bounds(const fa_paged_cache* cache, const fa_page_bounds_pool* bounds, const int32_t* first,
                         const int32_t* seq_lens, void* stream);

/*
 * For query b and each KV head, the min(K, n) pages of the n = ceil(seq_lens[b] / page_size) of sequence b whose
 * bounds promise the largest scores, in ascending order: pages [B][Hkv][K], -1 behind the last.  The first
 * `first` and the last `last` pages are always among them (first + last <= K), then the largest scores, of equal ones
 * the lowest page.  The score of a page for
 * query head h, every step rounded to f32 (fl) so that it is the same everywhere: q in blocks of 32 components,
 *   m = max |q|;  c = q fl(127 / m) rounded twice, to f32 and to the nearest whole number (ties to even), within
 *   -127 .. 127;  e = fl(m / 127)  (zeros where m <= 1e-30)
 *   I = sum over the block of c * hi code (c > 0) or c * lo code;  term = fl(fl(I d) e)
 *   the terms summed as a tree, neighbours first;  s = fl(scale * sum)
 *   s = fl(s + fl(alibi_slopes[h] * (position of the page's last key - (L - 1)))) where slopes are given
 * A KV head's score is the largest of its query heads'; a NaN counts as infinity (q that is not finite: whatever
 * is chosen is K pages of the sequence).  A negative scale counts as -scale with -q; one that is not finite is refused
 * (FA_ERR_SHAPE).  A soft cap does not change the order without slopes, and is left out with them.
 * seq_lens[b] = 0 gives -1 everywhere; a negative one marks a padding slot, whose row is left as it was; pages on an
 * invalid page number count as the least (FA_ERR_PAGE).
 * The bounds of all n pages have been computed by fa_page_bounds(); a length beyond the table counts as the table's.  q as in fa_paged_decode().  K >= 1.
 * max_pages <= 2^22, H <= 65535, B * Hkv < 2^22 (else FA_ERR_UNSUPPORTED).  Alignment: q to its element, pages,
 * seq_lens, alibi_slopes 4 bytes, codes and scales 16, workspace 256 bytes.
 */
size_t fa_page_select_workspace_size(const fa_paged_cache* cache, int H, int K);
fa_status fa_page_select(const void* q, int act, int64_t q_row, int64_t q_head, const fa_paged_cache* cache,
                         const fa_page_bounds_pool* bounds, const int32_t* seq_lens, int H, float scale,
                         const float* alibi_slopes, int K, int first, int last, int32_t* pages, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * fa_paged_decode() over selected pages: query heads of KV head hk of sequence b attend over the positions below
 * seq_lens[b] of the pages pages[b][hk][0 .. K-1], distinct page indices of the sequence (not page numbers) in any
 * order; entries outside 0 .. ceil(seq_lens[b] / page_size)-1 are skipped.  At most the first
 * min(K, ceil(seq_lens[b] / page_size)) entries are read.  Positions, ALiBi distances among them, are those of the
 * whole sequence; a score is rounded to 32 bits with its bias, so that pages far from the end, attended alone, have
 * weights off by about 2^-24 of the bias's magnitude.  Workspace: fa_paged_decode_workspace_size().
 */
fa_status fa_paged_decode_pages(const void* q, int act, int64_t q_row, int64_t q_head, const fa_paged_cache* cache,
                                const int32_t* seq_lens, const int32_t* pages, int K, int H, float scale,
                                const float* alibi_slopes, float softcap, const float* sinks, void* O, float* lse,
                                void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_PAGED_EXT_H */
