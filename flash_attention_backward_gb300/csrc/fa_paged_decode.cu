// Host side of fa_paged_decode(): checks, the plan and the launch (kernels: fa_decode.cuh).
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "fa_decode.cuh"

namespace fap {

// The pool as a matrix of cells [rows][Hkv * rb bytes], read in boxes of `box` rows x `pitch` bytes: the row,
// what lies before it back to a 16-byte boundary, and padding that spaces the rows in shared memory.
// Elements are as wide as keeps a box within 256 of them.  by_head: as [rows][Hkv][rb bytes], a box a head's rows and zeros
// behind them.
static bool map_pool(CUtensorMap* m, const void* pool, long long rows, int Hkv, int rb, int pitch, int box_rows, bool by_head) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  if (!fn) return false;
  const int lg = map_es(pitch);
  const auto type = lg == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : lg == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT64;
  const cuuint64_t cell = (cuuint64_t)Hkv * rb;
  const cuuint64_t dims[3] = {by_head ? (cuuint64_t)rb >> lg : cell >> lg, by_head ? (cuuint64_t)Hkv : (cuuint64_t)rows, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {by_head ? (cuuint64_t)rb : cell, cell};
  const cuuint32_t box[3] = {(cuuint32_t)(pitch >> lg), by_head ? 1u : (cuuint32_t)box_rows, (cuuint32_t)box_rows}, es[3] = {1, 1, 1};
  return fn(m, type, by_head ? 3 : 2, const_cast<void*>(pool), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct DecodePlan {
  int R, HG, chunks, nitems, njobs;
  size_t off_jobs, off_items, bytes;
  bool planned;
};

// K: pages of a sequence that count at most
static DecodePlan plan_decode(const Cache& c, int H, int K, bool sel, int nsm) {
  DecodePlan p;
  const int G = H / c.Hkv;
  p.chunks = (G + 7) / 8;
  p.HG = c.Hkv * p.chunks;
  const int ctas = decode_shape(c.D, c.Dv, c.k_type, c.v_type, sel).ctas;
  p.R = std::max(1, ctas * nsm / p.HG);  // items that run at a time
  // at most R + B (see fa_decode.cuh), and no more than tables of this width can ask for
  const long long cap = ((long long)std::min(K, c.max_pages) * c.page_size + 15) / 16, per = (cap + kMinTiles - 1) / kMinTiles;
  p.nitems = (int)std::max(1LL, std::min<long long>(c.B * std::max(per, 1LL), (long long)p.R + c.B));
  p.njobs = per > 1 ? std::min(c.B, p.R) : 0;  // split sequences: none if no sequence can be
  const size_t slots = p.njobs ? std::min(2 * p.R, p.nitems) : 0;
  p.planned = c.B > kPlanBatch;
  p.off_jobs = slots * p.HG * (8 * c.Dv + 16) * sizeof(float);
  p.off_items = p.off_jobs + (size_t)std::max(p.njobs, 1) * sizeof(int4);
  p.bytes = (p.off_items + (p.planned ? (size_t)p.nitems * sizeof(int4) : 0) + 255) / 256 * 256;
  return p;
}

template <int D, bool SEL>
static DecodeFn pick_decode_k(const Cache& c) {
  switch (c.k_type) {
    case FA_F32: return pick_decode<D, FA_F32, SEL>(c.Dv, c.v_type);
    case FA_F16: return pick_decode<D, FA_F16, SEL>(c.Dv, c.v_type);
    case FA_Q8_0: return pick_decode<D, FA_Q8_0, SEL>(c.Dv, c.v_type);
  }
  return pick_decode<D, FA_Q4_0, SEL>(c.Dv, c.v_type);
}
template <bool SEL>
static DecodeFn pick_decode_d(const Cache& c) {
  return c.D == 64 ? pick_decode_k<64, SEL>(c) : c.D == 128 ? pick_decode_k<128, SEL>(c) : pick_decode_k<256, SEL>(c);
}

}  // namespace fap

using namespace fap;

extern "C" size_t fa_paged_decode_workspace_size(const fa_paged_cache* cache, int H) {
  Cache c;
  if (check_cache(cache, &c) != FA_OK || H < 1 || H % c.Hkv) return 0;
  int nsm = 0;
  if (fab_device(&nsm, nullptr) != FA_OK) nsm = 152;
  // of either call: the kernels over selected pages run more CTAs an SM for some types, fewer for others (a plan grows with K)
  return std::max(plan_decode(c, H, c.max_pages, false, nsm).bytes, plan_decode(c, H, c.max_pages, true, nsm).bytes);
}

// pages [B][Hkv][K], or NULL: all of them (K is max_pages then)
static fa_status decode(const void* q, int act, int64_t q_row, int64_t q_head, const fa_paged_cache* cache, const int32_t* seq_lens,
                        const int32_t* pages, int K, int H, float scale, const float* alibi_slopes, float softcap,
                        const float* sinks, void* O, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  DecodeArgs a = {};
  fa_status rc = check_cache(cache, &a.c);
  if (rc != FA_OK) return rc;
  if (!act_type(act)) return FA_ERR_TYPE;
  if (H < 1 || H % a.c.Hkv != 0 || q_row < 0 || q_head < 0) return FA_ERR_SHAPE;
  if (!(softcap >= 0.f) || !std::isfinite(softcap)) return FA_ERR_SHAPE;
  if (H > 65535 || a.c.B > (1 << 20) || (long long)a.c.num_pages * a.c.page_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  if (a.c.B > 0 && (!q || !O || !seq_lens)) return FA_ERR_NULL;
  if (!aligned(q, act_bytes(act)) || !aligned(O, 16) || !aligned(lse, 4) || !aligned(seq_lens, 4) ||
      !aligned(alibi_slopes, 4) || !aligned(sinks, 4))
    return FA_ERR_ALIGN;
  int nsm = 0;
  if ((rc = fab_device(&nsm, &a.c.err)) != FA_OK) return rc;
  const DecodePlan p = plan_decode(a.c, H, K, pages != nullptr, nsm);
  if ((long long)p.nitems * p.HG > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < p.bytes) return FA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA_ERR_ALIGN;
  if (a.c.B == 0) return FA_OK;
  a.q = q, a.act = act, a.q_row = q_row, a.q_head = q_head, a.lens = seq_lens, a.sel = pages, a.K = K;
  a.H = H, a.G = H / a.c.Hkv, a.HG = p.HG, a.chunks = p.chunks;
  a.scale = scale, a.softcap = softcap, a.alibi = alibi_slopes, a.sinks = sinks, a.O = O, a.lse = lse;
  a.part = static_cast<float*>(workspace);
  a.jobs = reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + p.off_jobs);
  a.items = p.planned ? reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + p.off_items) : nullptr;
  a.R = p.R, a.nitems = p.nitems, a.njobs = p.njobs, a.joins = 4 * nsm;
  a.wait_ns = fab_take_wait_ns();
  // boxes of 16 or 8 rows where these never span pages and cells are spaced by multiples of 16 bytes
  DecodeMaps m = {};
  const long long rows = (long long)a.c.num_pages * a.c.page_size;
  const bool spaced = (a.c.Hkv * a.c.rbk) % 16 == 0 && (a.c.Hkv * a.c.rbv) % 16 == 0 && rows > 0;
  a.box = !spaced ? 0 : a.c.page_size % 16 == 0 ? 16 : a.c.page_size % 8 == 0 ? 8 : 0;
  if (a.box && (!map_pool(&m.k, a.c.k, rows, a.c.Hkv, a.c.rbk, smem_pitch(a.c.rbk), a.box, map_by_head(pages, a.c.rbk)) ||
                !map_pool(&m.v, a.c.v, rows, a.c.Hkv, a.c.rbv, smem_pitch(a.c.rbv), a.box, map_by_head(pages, a.c.rbv))))
    return FA_ERR_CUDA;
  const DecodeFn run = pages ? pick_decode_d<true>(a.c) : pick_decode_d<false>(a.c);
  return run(a, m, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

extern "C" fa_status fa_paged_decode(const void* q, int act, int64_t q_row, int64_t q_head, const fa_paged_cache* cache,
                                     const int32_t* seq_lens, int H, float scale, const float* alibi_slopes,
                                     float softcap, const float* sinks, void* O, float* lse, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  return decode(q, act, q_row, q_head, cache, seq_lens, nullptr, cache ? cache->max_pages : 0, H, scale, alibi_slopes, softcap, sinks, O,
                lse, workspace, workspace_bytes, stream);
}

extern "C" fa_status fa_paged_decode_pages(const void* q, int act, int64_t q_row, int64_t q_head, const fa_paged_cache* cache,
                                           const int32_t* seq_lens, const int32_t* pages, int K, int H, float scale,
                                           const float* alibi_slopes, float softcap, const float* sinks, void* O,
                                           float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (K < 1) return FA_ERR_SHAPE;
  if (!pages && (!cache || cache->B > 0)) return FA_ERR_NULL;
  if (!aligned(pages, 4)) return FA_ERR_ALIGN;
  return decode(q, act, q_row, q_head, cache, seq_lens, pages, K, H, scale, alibi_slopes, softcap, sinks, O, lse, workspace,
                workspace_bytes, stream);
}
