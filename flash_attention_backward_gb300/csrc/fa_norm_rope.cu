// Host side of fa_qk_norm_rope() and its gradient: checks, launch shapes, the sum of dw over CTAs (kernels:
// fa_norm_rope.cuh).
#include <algorithm>
#include <cmath>

#include "fa_norm_rope.cuh"

namespace fap {

fa_status check_rope(const fa_rope* r, int D, const int32_t* pos, int N, Rope* out) {
  *out = Rope{nullptr, 0, FA_ROPE_HALVES};
  if (!r || !r->freqs || r->n_rot == 0) return FA_OK;
  if (r->style != FA_ROPE_PAIRS && r->style != FA_ROPE_HALVES) return FA_ERR_SHAPE;
  if (r->n_rot < 0 || (r->n_rot & 1) || r->n_rot > D) return FA_ERR_SHAPE;
  if (r->style == FA_ROPE_HALVES && r->n_rot % 16) return FA_ERR_UNSUPPORTED;
  if (N > 0 && !pos) return FA_ERR_NULL;
  if (!aligned(r->freqs, 8) || !aligned(pos, 4)) return FA_ERR_ALIGN;
  *out = Rope{r->freqs, r->n_rot, r->style};
  return FA_OK;
}

// dw = the CTAs' sums in a fixed order: 32 columns a CTA, each split over 32 rows of threads.  blockIdx.y 0:
// queries, 1: keys.
__global__ void __launch_bounds__(1024) k_dw_reduce(const float* part, int ctas_q, int ctas, int D, float* dwq, float* dwk) {
  __shared__ float red[32][33], lost[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x, b0 = blockIdx.y ? ctas_q : 0, b1 = blockIdx.y ? ctas : ctas_q;
  float* out = blockIdx.y ? dwk : dwq;
  after_last();
  if (!out) return;
  ExactSum s;
  for (int b = b0 + threadIdx.y; b < b1; b += 32) s.add(part[(long long)b * D + c]);
  red[threadIdx.y][threadIdx.x] = s.s, lost[threadIdx.y][threadIdx.x] = s.lost;
  __syncthreads();
  if (threadIdx.y == 0) {
    s = ExactSum();
#pragma unroll
    for (int y = 0; y < 32; ++y) s.add(red[y][threadIdx.x]), s.lost += lost[y][threadIdx.x];
    out[c] = s.value();
  }
}

static bool rows_on_16(const void* p, long long row, long long head, int es) {
  return aligned(p, 16) && (row * es) % 16 == 0 && (head * es) % 16 == 0;
}

// Checks what both directions take; fills everything but the outputs and the gradients.
static fa_status norm_args(const void* q, const void* k, int x_type, const fa_qk_views* vw, const float* wq,
                           const float* wk, float eps, const int32_t* pos, const fa_rope* rope, int N, int H, int Hkv,
                           int D, int y_type, bool back, NormArgs* a) {
  if (!act_type(x_type) || !act_type(y_type)) return FA_ERR_TYPE;
  if (N < 0 || H < 1 || Hkv < 0 || !(eps >= 0.f) || !std::isfinite(eps)) return FA_ERR_SHAPE;
  if (!head_size(D)) return FA_ERR_UNSUPPORTED;
  if ((long long)H + Hkv > (1 << 20) || (long long)N * (H + Hkv) > (1LL << 36)) return FA_ERR_UNSUPPORTED;
  const bool readq = !back || wq, readk = !back || wk;
  const fa_qk_views none = {(int64_t)H * D, D, (int64_t)Hkv * D, D};
  const fa_qk_views v = vw ? *vw : none;
  if (v.q_row < 0 || v.q_head < 0 || v.k_row < 0 || v.k_head < 0) return FA_ERR_SHAPE;
  if (N > 0 && ((readq && !q) || (Hkv > 0 && readk && !k))) return FA_ERR_NULL;
  const int es = act_bytes(x_type);
  if (!aligned(q, es) || !aligned(k, es) || !aligned(wq, 4) || !aligned(wk, 4)) return FA_ERR_ALIGN;
  NormArgs z = {};
  *a = z;
  const fa_status rc = check_rope(rope, D, pos, N, &a->rope);
  if (rc != FA_OK) return rc;
  NormSide& sq = a->side[0];
  NormSide& sk = a->side[1];
  sq.x = q, sq.row = v.q_row, sq.head = v.q_head, sq.w = wq, sq.H = H;
  sk.x = k, sk.row = v.k_row, sk.head = v.k_head, sk.w = wk, sk.H = Hkv;
  a->eps = eps, a->pos = pos, a->N = N;
  a->vec = rows_on_16(q, v.q_row, v.q_head, es) && (Hkv == 0 || rows_on_16(k, v.k_row, v.k_head, es));
  return FA_OK;
}

// Heads of a token that one warp takes out of H: `most` where there are tokens enough to give every SM
// 16 warps of that, else fewer, down to the heads that lie side by side in a warp; equal chunks.
static void chunk_heads(int H, long long rows_a_warp, int side, int most, int* HC, int* nchunk) {
  *HC = 1, *nchunk = 0;
  if (H == 0) return;
  const int hc = (int)std::max(1LL, std::min<long long>(rows_a_warp, most / side)) * side;
  *nchunk = (H + hc - 1) / hc;
  *HC = ((H + *nchunk - 1) / *nchunk + side - 1) / side * side;
  *nchunk = (H + *HC - 1) / *HC;
}
static long long rows_a_warp(const NormArgs& a, int D, int nsm) {
  return (long long)a.N * (a.side[0].H + a.side[1].H) / (16LL * nsm * (256 / D));
}

static int back_ctas(int nsm) { return kBackCtas * nsm; }

}  // namespace fap

using namespace fap;

extern "C" fa_status fa_rope_frequencies(int n_rot, double base, double scale, const float* factors, uint64_t* out) {
  if (n_rot < 0 || (n_rot & 1) || !(base > 0) || !std::isfinite(base) || !(scale > 0) || !std::isfinite(scale))
    return FA_ERR_SHAPE;
  if (n_rot > 0 && !out) return FA_ERR_NULL;
  for (int i = 0; factors && i < n_rot / 2; ++i)
    if (!(factors[i] > 0) || !std::isfinite(factors[i])) return FA_ERR_SHAPE;
  for (int i = 0; i < n_rot / 2; ++i) {
    double f = scale * std::pow(base, -2.0 * i / n_rot);
    if (factors) f /= factors[i];
    double turns = f / (2.0 * 3.14159265358979323846);
    turns -= std::floor(turns);  // whole turns do nothing at whole positions
    out[i] = (uint64_t)std::ldexp(turns, 64);
  }
  return FA_OK;
}

extern "C" fa_status fa_qk_norm_rope(const void* q, const void* k, int x_type, const fa_qk_views* views,
                                     const float* wq, const float* wk, float eps, const int32_t* pos,
                                     const fa_rope* rope, int N, int H, int Hkv, int D, void* q_out, void* k_out,
                                     int y_type, void* stream) {
  NormArgs a;
  fa_status rc = norm_args(q, k, x_type, views, wq, wk, eps, pos, rope, N, H, Hkv, D, y_type, false, &a);
  if (rc != FA_OK) return rc;
  if (N > 0 && (!q_out || (Hkv > 0 && !k_out))) return FA_ERR_NULL;
  if (!aligned(q_out, 16) || !aligned(k_out, 16)) return FA_ERR_ALIGN;
  int nsm = 0;
  if ((rc = fab_device(&nsm, nullptr)) != FA_OK) return rc;
  if (N == 0) return FA_OK;
  a.side[0].y = q_out, a.side[1].y = k_out;
  chunk_heads(H + Hkv, rows_a_warp(a, D, nsm), 256 / D, 32, &a.HC, &a.nchunk);
  const long long items = (long long)N * a.nchunk;  // (that many heads would not fit in memory)
  if (items > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  long long grid = (items + 7) / 8;
  const int ctas = x_type == FA_ACT_F32 ? kForwardCtas<float> : kForwardCtas<__half>;
  if (ctas) grid = std::min<long long>(grid, (long long)ctas * nsm);
  return launch_next(pick_norm_fwd(D, x_type, y_type, a.vec, a.rope.style), dim3((unsigned)grid), dim3(256), 0,
                     static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

extern "C" size_t fa_qk_norm_rope_backward_workspace_size(int N, int H, int Hkv, int D) {
  if (N < 0 || H < 1 || Hkv < 0 || !head_size(D)) return 0;
  int nsm = 0;
  if (fab_device(&nsm, nullptr) != FA_OK) nsm = 152;
  return (size_t)back_ctas(nsm) * D * sizeof(float);
}

extern "C" fa_status fa_qk_norm_rope_backward(const void* gq, const void* gk, int y_type, const void* q, const void* k,
                                              int x_type, const fa_qk_views* views, const float* wq, const float* wk,
                                              float eps, const int32_t* pos, const fa_rope* rope, int N, int H,
                                              int Hkv, int D, void* dq, void* dk, float* dwq, float* dwk,
                                              void* workspace, size_t workspace_bytes, void* stream) {
  NormArgs a;
  fa_status rc = norm_args(q, k, x_type, views, wq, wk, eps, pos, rope, N, H, Hkv, D, y_type, true, &a);
  if (rc != FA_OK) return rc;
  if (N > 0 && (!gq || !dq || (Hkv > 0 && (!gk || !dk)))) return FA_ERR_NULL;
  if (!aligned(gq, 16) || !aligned(gk, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dwq, 4) || !aligned(dwk, 4))
    return FA_ERR_ALIGN;
  int nsm = 0, *err = nullptr;
  if ((rc = fab_device(&nsm, &err)) != FA_OK) return rc;
  if (!workspace || workspace_bytes < (size_t)back_ctas(nsm) * D * sizeof(float)) return FA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA_ERR_ALIGN;
  a.side[0].gy = gq, a.side[1].gy = gk, a.side[0].y = dq, a.side[1].y = dk;
  a.part = static_cast<float*>(workspace);
  a.err = err;
  const BackKernel k_back = pick_norm_back(D, x_type, y_type, a.vec, a.rope.style);
  for (NormSide& sd : a.side) sd.nchunk = (sd.H + k_back.heads - 1) / k_back.heads;
  // CTAs shared out by the heads of either side; every side that has heads gets one
  const long long iq = (long long)N * a.side[0].nchunk, ik = (long long)N * a.side[1].nchunk;
  if (iq > 0x7fffffffLL || ik > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  const int all = back_ctas(nsm);
  int ck = Hkv ? (int)std::min<long long>(std::max(1LL, (long long)all * Hkv / (H + Hkv)), std::max(1LL, (ik + 7) / 8)) : 0;
  const int cq = (int)std::min<long long>(all - ck, std::max(1LL, (iq + 7) / 8));
  a.ctas_q = cq;
  a.wait_ns = fab_take_wait_ns();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (k_back.smem > 48 * 1024 && !allow_smem(reinterpret_cast<const void*>(k_back.fn), k_back.smem, k_back.ready)) return FA_ERR_CUDA;
  if (launch_next(k_back.fn, dim3(cq + ck), dim3(kBackWarps * 32), k_back.smem, s, a) != cudaSuccess) return FA_ERR_CUDA;
  float* oq = wq ? dwq : nullptr;
  float* ok = wk && Hkv ? dwk : nullptr;
  if ((oq || ok) &&
      launch_next(k_dw_reduce, dim3(D / 32, 2), dim3(32, 32), 0, s, a.part, cq, cq + ck, D, oq, ok) != cudaSuccess)
    return FA_ERR_CUDA;
  if (wk && !Hkv && dwk) cudaMemsetAsync(dwk, 0, D * sizeof(float), s);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
