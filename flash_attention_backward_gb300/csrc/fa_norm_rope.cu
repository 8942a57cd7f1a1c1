// Queries and keys of a layer, head by head: RMS norm and position rotation in one pass, and the
// gradient.  Both are bound by memory: a head is read once and written once (backward: x and gy
// read, dx written), everything between stays in registers.
//
//   y = R (w o x r),  r = rsqrt(mean(x^2) + eps)
//   g = R^T gy,  dw = sum g o x r,  h = g o w,  dx = r (h - x r^2 mean(h o x))
#include <algorithm>
#include <cmath>

#include "fa_paged.cuh"

namespace fap {

fa_status check_rope(const fa_rope* r, int D, const int32_t* pos, int N, Rope* out) {
  *out = Rope{nullptr, 0, FA_ROPE_PAIRS};
  if (!r || !r->freqs || r->n_rot == 0) return FA_OK;
  if (r->style != FA_ROPE_PAIRS && r->style != FA_ROPE_HALVES) return FA_ERR_SHAPE;
  if (r->n_rot < 0 || (r->n_rot & 1) || r->n_rot > D) return FA_ERR_SHAPE;
  if (r->style == FA_ROPE_HALVES && r->n_rot % 16) return FA_ERR_UNSUPPORTED;
  if (N > 0 && !pos) return FA_ERR_NULL;
  if (!aligned(r->freqs, 8) || !aligned(pos, 4)) return FA_ERR_ALIGN;
  *out = Rope{r->freqs, r->n_rot, r->style};
  return FA_OK;
}

struct NormArgs {
  const void *q, *k;            // x
  const void *gq, *gk;          // backward: gradients of the outputs
  long long q_row, q_head, k_row, k_head;
  const float *wq, *wk;
  float eps;
  const int32_t* pos;
  Rope rope;
  int N, H, HT;                 // HT = H + Hkv
  void *qo, *ko;                // y, or dx
  int HC, nchunk;               // heads of one token that a lane group takes, chunks of a token
  bool vecq, veck;              // rows of q / k start on 16 bytes
  float* part;                  // backward: [CTA][2][D] sums of dw
};

// One lane group (D / 8 lanes) takes HC heads of one token: the rotation's factors are computed once
// for them.
template <int D, typename TX, typename TY>
__global__ void __launch_bounds__(256) k_norm_rope(const NormArgs a) {
  constexpr int LG = D / 8, GW = 32 / LG;
  const int lane = threadIdx.x & 31, lg = lane & (LG - 1), e0 = lg * 8;
  const long long item = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * GW + lane / LG;
  const bool live = item < (long long)a.N * a.nchunk;
  const int n = live ? (int)(item / a.nchunk) : 0;
  const int h0 = live ? (int)(item - (long long)n * a.nchunk) * a.HC : 0;
  Turn8 t;
  t.set(a.rope, live && a.rope.n_rot ? a.pos[n] : 0, e0);
  for (int i = 0; i < a.HC; ++i) {
    const int h = h0 + i;
    const bool on = live && h < a.HT, isq = h < a.H;
    float x[8] = {};
    if (on) {
      if (isq) load8(static_cast<const TX*>(a.q) + n * a.q_row + h * a.q_head + e0, a.vecq, x);
      else load8(static_cast<const TX*>(a.k) + n * a.k_row + (h - a.H) * a.k_head + e0, a.veck, x);
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
    ss = group_sum<LG>(ss);
    const float* w = isq ? a.wq : a.wk;
    if (on && w) {
      const float r = inv_rms(ss, 1.f / D, a.eps);
      float wv[8];
      load8(w + e0, false, wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] * r * wv[j];
    }
    if (a.rope.n_rot) t.apply(x, a.rope.style, 1.f);
    if (on) {
      TY* y = isq ? static_cast<TY*>(a.qo) + ((long long)n * a.H + h) * D
                  : static_cast<TY*>(a.ko) + ((long long)n * (a.HT - a.H) + (h - a.H)) * D;
      store8(y + e0, x);
    }
  }
}

template <int D, typename TX, typename TY>
__global__ void __launch_bounds__(256) k_norm_rope_back(const NormArgs a) {
  constexpr int LG = D / 8, GW = 32 / LG, GC = 8 * GW;  // lane groups of a CTA
  __shared__ float red[GC][2 * D];
  const int lane = threadIdx.x & 31, lg = lane & (LG - 1), e0 = lg * 8;
  const int grp = (threadIdx.x >> 5) * GW + lane / LG;
  float dw[2][8] = {};
  const long long items = (long long)a.N * a.nchunk, step = (long long)gridDim.x * GC;
  const long long rounds = (items + step - 1) / step;
  for (long long rd = 0; rd < rounds; ++rd) {
    const long long item = rd * step + (long long)blockIdx.x * GC + grp;
    const bool live = item < items;
    const int n = live ? (int)(item / a.nchunk) : 0;
    const int h0 = live ? (int)(item - (long long)n * a.nchunk) * a.HC : 0;
    Turn8 t;
    t.set(a.rope, live && a.rope.n_rot ? a.pos[n] : 0, e0);
    for (int i = 0; i < a.HC; ++i) {
      const int h = h0 + i;
      const bool on = live && h < a.HT, isq = h < a.H;
      const float* w = isq ? a.wq : a.wk;
      float x[8] = {}, g[8] = {}, wv[8] = {};
      const long long at = isq ? ((long long)n * a.H + h) * D : ((long long)n * (a.HT - a.H) + (h - a.H)) * D;
      if (on) {
        load8((isq ? static_cast<const TY*>(a.gq) : static_cast<const TY*>(a.gk)) + at + e0, true, g);
        if (w) {
          if (isq) load8(static_cast<const TX*>(a.q) + n * a.q_row + h * a.q_head + e0, a.vecq, x);
          else load8(static_cast<const TX*>(a.k) + n * a.k_row + (h - a.H) * a.k_head + e0, a.veck, x);
          load8(w + e0, false, wv);
        }
      }
      if (a.rope.n_rot) t.apply(g, a.rope.style, -1.f);
      float ss = 0.f, hx = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss), hx = fmaf(g[j] * wv[j], x[j], hx);
      ss = group_sum<LG>(ss);
      hx = group_sum<LG>(hx);
      if (on && w) {
        const float r = inv_rms(ss, 1.f / D, a.eps);
        const float m = hx * (1.f / D) * r * r;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = g[j] * x[j] * r;
          if (isq) dw[0][j] += d;
          else dw[1][j] += d;
          g[j] = r * fmaf(-x[j], m, g[j] * wv[j]);
        }
      }
      if (on) store8((isq ? static_cast<TX*>(a.qo) : static_cast<TX*>(a.ko)) + at + e0, g);
    }
  }
  // the CTA's groups in order, one column a thread
#pragma unroll
  for (int j = 0; j < 8; ++j) red[grp][e0 + j] = dw[0][j], red[grp][D + e0 + j] = dw[1][j];
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += 256) {
    float s = 0.f;
    for (int g = 0; g < GC; ++g) s += red[g][c];
    a.part[(long long)blockIdx.x * 2 * D + c] = s;
  }
}

// dw[c] = the CTAs' sums in a fixed order: 32 columns a CTA, each split over 32 rows of threads.
__global__ void __launch_bounds__(1024) k_dw_reduce(const float* part, int nblk, int D, float* dwq, float* dwk) {
  __shared__ float red[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  for (int b = threadIdx.y; b < nblk; b += 32) s += part[(long long)b * 2 * D + c];
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0) {
    s = 0.f;
#pragma unroll
    for (int y = 0; y < 32; ++y) s += red[y][threadIdx.x];
    float* out = c < D ? dwq : dwk;
    if (out) out[c < D ? c : c - D] = s;
  }
}

typedef void (*NormKernel)(const NormArgs);

template <int D, typename TX>
static NormKernel pick_y(bool back, int ty) {
  switch (ty) {
    case FA_ACT_F32: return back ? k_norm_rope_back<D, TX, float> : k_norm_rope<D, TX, float>;
    case FA_ACT_F16: return back ? k_norm_rope_back<D, TX, __half> : k_norm_rope<D, TX, __half>;
  }
  return back ? k_norm_rope_back<D, TX, __nv_bfloat16> : k_norm_rope<D, TX, __nv_bfloat16>;
}
template <int D>
static NormKernel pick_x(bool back, int tx, int ty) {
  switch (tx) {
    case FA_ACT_F32: return pick_y<D, float>(back, ty);
    case FA_ACT_F16: return pick_y<D, __half>(back, ty);
  }
  return pick_y<D, __nv_bfloat16>(back, ty);
}
static NormKernel pick_norm(bool back, int D, int tx, int ty) {
  return D == 64 ? pick_x<64>(back, tx, ty) : D == 128 ? pick_x<128>(back, tx, ty) : pick_x<256>(back, tx, ty);
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
  a->q = q, a->k = k, a->q_row = v.q_row, a->q_head = v.q_head, a->k_row = v.k_row, a->k_head = v.k_head;
  a->wq = wq, a->wk = wk, a->eps = eps, a->pos = pos, a->N = N, a->H = H, a->HT = H + Hkv;
  a->vecq = rows_on_16(q, v.q_row, v.q_head, es), a->veck = rows_on_16(k, v.k_row, v.k_head, es);
  return FA_OK;
}

// Heads of a token that one lane group takes: enough to share the rotation's factors, few enough
// that every SM has warps.
static void chunk_heads(NormArgs* a, int D, int nsm) {
  const long long want = 16LL * nsm * (256 / D);  // lane groups: two CTAs' worth of warps an SM
  long long hc = (long long)a->N * a->HT / want;
  hc = std::max(1LL, std::min<long long>(hc, a->HT));
  a->nchunk = (int)((a->HT + hc - 1) / hc);
  a->HC = (a->HT + a->nchunk - 1) / a->nchunk;
  a->nchunk = (a->HT + a->HC - 1) / a->HC;
}

static int back_ctas(int nsm) { return 2 * nsm; }

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
  int nsm = 0, *err = nullptr;
  if ((rc = fab_device(&nsm, &err)) != FA_OK) return rc;
  if (N == 0) return FA_OK;
  a.qo = q_out, a.ko = k_out;
  chunk_heads(&a, D, nsm);
  const long long per = 8 * (256 / D), blocks = ((long long)N * a.nchunk + per - 1) / per;
  if (blocks > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  pick_norm(false, D, x_type, y_type)<<<(unsigned)blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

extern "C" size_t fa_qk_norm_rope_backward_workspace_size(int N, int H, int Hkv, int D) {
  if (N < 0 || H < 1 || Hkv < 0 || !head_size(D)) return 0;
  int nsm = 0, *err = nullptr;
  if (fab_device(&nsm, &err) != FA_OK) nsm = 152;
  return (size_t)back_ctas(nsm) * 2 * D * sizeof(float);
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
  if (!workspace || workspace_bytes < (size_t)back_ctas(nsm) * 2 * D * sizeof(float)) return FA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA_ERR_ALIGN;
  a.gq = gq, a.gk = gk, a.qo = dq, a.ko = dk;
  a.part = static_cast<float*>(workspace);
  chunk_heads(&a, D, nsm);
  const long long per = 8 * (256 / D), want = ((long long)N * a.nchunk + per - 1) / per;
  const int blocks = (int)std::max(1LL, std::min<long long>(want, back_ctas(nsm)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  pick_norm(true, D, x_type, y_type)<<<blocks, 256, 0, s>>>(a);
  float* oq = wq ? dwq : nullptr;
  float* ok = wk ? dwk : nullptr;
  if (oq || ok) k_dw_reduce<<<2 * D / 32, dim3(32, 32), 0, s>>>(a.part, blocks, D, oq, ok);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
