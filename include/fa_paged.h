/*
 * fa_paged.h -- C ABI of the paged raw K/V cache and of the per-head norm and rotation, beside the
 * attention of fa_back.h (same library, same fa_type formats and fa_status codes).
 *
 *   fa_qk_norm_rope            queries and keys: RMS norm of every head, position rotation
 *   fa_qk_norm_rope_backward   its gradient with respect to q, k and both norm weights
 *   fa_cache_append            keys (normalised, rotated) and values into a paged cache, quantised
 *   fa_cache_read              rows of a paged cache, decoded or raw
 *   fa_paged_decode            attention of one new token per sequence over a paged cache
 *
 * Conventions are those of fa_back.h: every pointer is caller-owned DEVICE memory on the current
 * device unless it is said to be host memory; the library allocates nothing and keeps no
 * reference; arguments are checked on the host before anything is enqueued (the outputs are then
 * untouched); the work is enqueued on `stream` without synchronising and may be captured into a
 * CUDA graph (lengths, positions, page tables and data are read when the work runs, so a replay
 * takes their current values); every output element has one writer and every sum a fixed order, so
 * equal calls give bit-identical outputs.  Calls whose work may overlap on the GPU need
 * workspaces of their own.
 */
#ifndef FA_PAGED_H
#define FA_PAGED_H

#include "fa_back.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations.  Arithmetic is f32 whatever the type; a result is rounded once,
 * to nearest, when it is stored.  FA_ACT_RAW (fa_cache_read only): the cache rows' own bytes. */
typedef enum { FA_ACT_F32 = 0, FA_ACT_F16 = 1, FA_ACT_BF16 = 2, FA_ACT_RAW = 3 } fa_act;

/* How the rotation pairs the components of a head. */
typedef enum {
  FA_ROPE_PAIRS = 0, /* pair i is components 2i and 2i + 1             */
  FA_ROPE_HALVES = 1 /* pair i is components i and i + n_rot / 2       */
} fa_rope_style;

/*
 * The rotation.  Pair i (0 <= i < n_rot / 2) of a head at position p turns by p * freqs[i]:
 *   (a, b) -> (a cos - b sin, a sin + b cos);  components n_rot .. D-1 are not rotated.
 * freqs [n_rot / 2] (device) holds each frequency in turns per position as a 64-bit fixed-point
 * fraction, freq / (2 pi) * 2^64: p * freqs[i] modulo 2^64 is then the exact angle modulo one
 * turn, at any 32-bit position (negative ones turn backwards).  fa_rope_frequencies() fills such
 * an array.  n_rot is even, at most D, and a multiple of 16 for FA_ROPE_HALVES.  freqs NULL or
 * n_rot 0: no rotation.
 */
typedef struct fa_rope {
  const uint64_t* freqs;
  int32_t n_rot;
  int32_t style;
} fa_rope;

/* Fills out [n_rot / 2] (HOST memory) with scale * base^(-2 i / n_rot) / factors[i] radians per
 * position (factors: host memory, or NULL for ones), in the form that fa_rope takes.  FA_ERR_SHAPE
 * for an odd or negative n_rot, a base or scale that is not positive and finite, or a factor that
 * is not. */
fa_status fa_rope_frequencies(int n_rot, double base, double scale, const float* factors, uint64_t* out);

/*
 * Queries and keys of N tokens, head by head:
 *   y = R(pos[n]) (w o x rsqrt(mean(x^2) + eps))       (wq for query heads, wk for key heads)
 * With a NULL weight that tensor's heads are rotated only.  q [N][H][D] and k [N][Hkv][D] may be
 * views: token n, head h starts at element n*row + h*head of its tensor (components contiguous),
 * so both may lie in one fused projection.  Outputs are contiguous, [N][H][D] and [N][Hkv][D], of
 * y_type; q_out may be q itself (and k_out k) when q is contiguous and y_type is x_type.  Hkv may
 * be 0 (k and k_out unused).  wq, wk f32 [D]; eps >= 0; pos [N] (unused without rotation).  The sum
 * of squares is f32: it overflows for components beyond about 1e18, and below 1e-19 it vanishes
 * beside any eps that is not 0.
 * D in {64, 128, 256}.  Alignment: q and k to their element; the outputs 16 bytes.
 */
typedef struct fa_qk_views {
  int64_t q_row, q_head, k_row, k_head; /* in elements, >= 0 */
} fa_qk_views;

fa_status fa_qk_norm_rope(const void* q, const void* k, int x_type, const fa_qk_views* views, const float* wq,
                          const float* wk, float eps, const int32_t* pos, const fa_rope* rope, int N, int H, int Hkv,
                          int D, void* q_out, void* k_out, int y_type, void* stream);

/*
 * The gradient of fa_qk_norm_rope().  gq [N][H][D] and gk [N][Hkv][D] (contiguous, y_type) are the
 * gradients of q_out and k_out; q, k, views, weights, eps, pos and rope are the forward's.  With
 * r = rsqrt(mean(x^2) + eps), g = R(pos)^T gy and h = w o g:
 *   dx = r (h - x r^2 mean(h o x)),   dw = sum over tokens and heads of g o x r
 * (without a weight dx = g, and x is not read: q, k may then be NULL).  dq, dk: contiguous, of
 * x_type, not overlapping the inputs.  dwq, dwk: f32 [D], written where wq / wk is given (NULL: not
 * wanted).  N = 0 writes zeros to dwq and dwk.  Alignment: as for the forward; gq, gk, dq, dk 16
 * bytes, workspace 256 bytes.  The kernel's waits for its own copies are bounded: one that runs out
 * is reported as FA_ERR_TIMEOUT by fa_back_get_error() and leaves the outputs undefined.
 * fa_back_test_wait_limit() applies to the next call here too; a limit of 0 counts every wait as run
 * out (heads of x that do not start on 16 bytes are loaded without copies to wait for).
 */
size_t fa_qk_norm_rope_backward_workspace_size(int N, int H, int Hkv, int D);
fa_status fa_qk_norm_rope_backward(const void* gq, const void* gk, int y_type, const void* q, const void* k, int x_type,
                                   const fa_qk_views* views, const float* wq, const float* wk, float eps,
                                   const int32_t* pos, const fa_rope* rope, int N, int H, int Hkv, int D, void* dq,
                                   void* dk, float* dwq, float* dwk, void* workspace, size_t workspace_bytes,
                                   void* stream);

/*
 * A paged raw cache.  k and v are pools [num_pages][page_size][Hkv][row] of cache rows (row =
 * fa_row_bytes(type, D or Dv)); position j of sequence b is row j % page_size of page
 * page_table[b * max_pages + j / page_size].  A contiguous cache [M][Hkv][row] of fa_back.h is a
 * pool of M / page_size pages in order.  page_size >= 1 is any for which a page's bytes
 * (page_size * Hkv * row, of k and of v) are a multiple of 16; max_pages * page_size <= 2^30.
 * D, Dv in {64, 128, 256}.  Pools 16-byte aligned, page_table 4-byte.
 *
 * Page numbers, sequence numbers and positions live on the device, so the host cannot check them:
 * the kernels do.  A row whose page number is outside [0, num_pages), or whose sequence or
 * position is outside the table, is not touched; fa_back_get_error() then reports FA_ERR_PAGE.
 */
typedef struct fa_paged_cache {
  void* k;
  void* v;
  const int32_t* page_table; /* [B][max_pages] */
  int32_t k_type, v_type, num_pages, page_size, B, max_pages, Hkv, D, Dv;
} fa_paged_cache;

/*
 * Stores token t's keys k[t] and values v[t] as position pos[t] of sequence seq[t], t < T.  Keys
 * are first normalised (k_norm f32 [D], or NULL: not) and rotated by their position pos[t], as in
 * fa_qk_norm_rope().  A token with seq[t] < 0 or pos[t] < 0 is padding and is skipped.  The
 * (sequence, position) pairs of one call must address distinct rows: what a row that two tokens
 * share holds afterwards is not defined.  k [T][Hkv][D] and v [T][Hkv][Dv] (x_type) may be views
 * as above (row, head strides in elements).
 *   FA_F32, FA_F16  the value, rounded to nearest.
 *   FA_Q8_0  d = amax / 127; code = x / d to the nearest, ties away from zero.
 *   FA_Q4_0  d = m / -8 with m the first of the values of largest magnitude; code = min(15,
 *            floor(x / d + 8.5)).
 * The scale is stored as binary16(d), the codes use d itself; a block of no value above 1e-30, whose
 * stored scale is zero, gets zero codes (q4_0: 8).  Blocks with a value above 8.3e6 (q8_0) or 5.2e5
 * (q4_0), or one that is not finite, leave binary16's range: none of their values decodes to a
 * finite one.
 */
typedef struct fa_kv_views {
  int64_t k_row, k_head, v_row, v_head; /* in elements, >= 0 */
} fa_kv_views;

fa_status fa_cache_append(const void* k, const void* v, int x_type, const fa_kv_views* views,
                          const fa_paged_cache* cache, const int32_t* seq, const int32_t* pos, int T,
                          const float* k_norm, float eps, const fa_rope* rope, void* stream);

/*
 * Reads position pos[t] of sequence seq[t], t < T, into k_out[t] and v_out[t]: decoded, [T][Hkv][D]
 * and [T][Hkv][Dv] of y_type, or with FA_ACT_RAW the rows' bytes [T][Hkv][row], which is the
 * contiguous cache that fa_back() and fa_forward() take.  Tokens with seq[t] < 0 or pos[t] < 0 are
 * skipped: their output rows are left as they were.  k_out or v_out may be NULL (not wanted);
 * 16-byte aligned otherwise.
 */
fa_status fa_cache_read(const fa_paged_cache* cache, const int32_t* seq, const int32_t* pos, int T, int y_type,
                        void* k_out, void* v_out, void* stream);

/*
 * Attention of one new token per sequence: query b (head h) attends over positions 0 ..
 * seq_lens[b] - 1 of sequence b, its own among them once fa_cache_append() has stored it.  With
 * L = seq_lens[b], hk = h / (H / Hkv):
 *   x_j = scale * q_bh . k^_j;   s_j = softcap tanh(x_j / softcap) (softcap > 0) or x_j, plus
 *         alibi_slopes[h] (j - (L - 1)) where given
 *   lse = log([exp(sinks[h]) +] sum_j exp(s_j));   O = sum_j exp(s_j - lse) v^_j
 * that is fa_forward() of a single query (N = 1) with the score extensions of fa_back_ext().
 * L = 0 gives O = 0 and lse = -inf (sinks[h] with sinks).  L < 0 marks a padding slot: its O and
 * lse are left as they were.  L above max_pages * page_size counts as that many (FA_ERR_PAGE);
 * keys on an invalid page count as masked (FA_ERR_PAGE).  What rows behind seq_lens[b] hold does
 * not matter.  An infinity or a NaN in q or in a row that counts may turn what it enters into NaN.
 * q [B][H][D] of act type may be a view (q_row, q_head strides in elements); O [B][H][Dv] of the
 * same type and lse [B][H] f32 (NULL: not wanted) are contiguous.  H % Hkv == 0; H at most 65535, B
 * at most 2^20, num_pages * page_size below 2^31 (else FA_ERR_UNSUPPORTED).  Alignment: q to its
 * element, O 16 bytes, lse, seq_lens, alibi_slopes, sinks 4 bytes, workspace 256 bytes.
 * The workspace holds the split partials; its size does not depend on the lengths.
 * The kernel's waits for its own copies are bounded: one that runs out is reported as FA_ERR_TIMEOUT
 * by fa_back_get_error() and leaves the outputs undefined.  fa_back_test_wait_limit() applies to the
 * next call here too; a limit of 0 counts every wait as run out.
 */
size_t fa_paged_decode_workspace_size(const fa_paged_cache* cache, int H);
fa_status fa_paged_decode(const void* q, int act, int64_t q_row, int64_t q_head, const fa_paged_cache* cache,
                          const int32_t* seq_lens, int H, float scale, const float* alibi_slopes, float softcap,
                          const float* sinks, void* O, float* lse, void* workspace, size_t workspace_bytes,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_PAGED_H */
