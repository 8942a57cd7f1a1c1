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

// Queries or keys: one of them a CTA.
struct NormSide {
  const void* x;
  const void* gy;      // backward: gradient of the output
  long long row, head; // strides of x
  const float* w;
  void* y;             // y, or dx
  int H;               // heads
  int HC, nchunk;      // heads of one token that a warp takes, chunks of a token
  bool vec;            // x starts every head on 16 bytes
};
struct NormArgs {
  NormSide side[2];
  int ctas_q;          // CTAs 0 .. ctas_q - 1 take queries, the rest keys
  float eps;
  const int32_t* pos;
  Rope rope;
  int N;
  float* part;         // backward: [CTA][D] sums of dw
};

// Rows that a lane group has under way at a time: 32 or 64 bytes a lane of x (and as much of gy).
template <typename T>
constexpr int kRows = sizeof(T) == 2 ? 4 : 2;

// A warp takes HC heads of one token, D / 8 lanes a head: the rotation's factors are computed once for
// them, and the loads of the next kRows heads are issued together.
template <int D, typename TX, typename TY>
__global__ void __launch_bounds__(256) k_norm_rope(const NormArgs a) {
  constexpr int LG = D / 8, GW = 32 / LG, U = kRows<TX>;
  const bool isq = blockIdx.x < a.ctas_q;
  const NormSide& sd = a.side[isq ? 0 : 1];
  const int lane = threadIdx.x & 31, grp = lane / LG, e0 = (lane & (LG - 1)) * 8;
  const long long item = (long long)(blockIdx.x - (isq ? 0 : a.ctas_q)) * 8 + (threadIdx.x >> 5);
  if (item >= (long long)a.N * sd.nchunk) return;
  const int n = (int)(item / sd.nchunk), h0 = (int)(item - (long long)n * sd.nchunk) * sd.HC;
  const int h1 = min(sd.H, h0 + sd.HC);
  const TX* x0 = static_cast<const TX*>(sd.x) + n * sd.row + e0;
  TY* y0 = static_cast<TY*>(sd.y) + (long long)n * sd.H * D + e0;
  float w[8];
  if (sd.w) load8(sd.w + e0, false, w);
  Turn8<D> t;
  for (int h = h0 + grp, first = 1; h - grp < h1; h += U * GW, first = 0) {
    Oct<TX> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u * GW < h1) load8_raw(x0 + (h + u * GW) * sd.head, sd.vec, raw[u]);
    if (first) t.set(a.rope, a.rope.n_rot ? a.pos[n] : 0, e0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h - grp + u * GW >= h1) break;  // (the same in all lanes)
      const bool on = h + u * GW < h1;
      float x[8] = {};
      if (on) unpack8(raw[u], x);
      if (sd.w) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
        const float r = inv_rms(group_sum<LG>(ss), 1.f / D, a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
      }
      if (a.rope.n_rot) t.apply(x, a.rope.style, 1.f);
      if (on) store8(y0 + (h + u * GW) * D, x);
    }
  }
}

// The same shape, in a loop over the items; dw is summed by lane over all of them, then over the CTA's
// lane groups in order.
template <int D, typename TX, typename TY>
__global__ void __launch_bounds__(256, 2) k_norm_rope_back(const NormArgs a) {
  constexpr int LG = D / 8, GW = 32 / LG, U = kRows<TX> < kRows<TY> ? kRows<TX> : kRows<TY>;
  __shared__ float red[8 * GW][D];
  const bool isq = blockIdx.x < a.ctas_q;
  const NormSide& sd = a.side[isq ? 0 : 1];
  const int lane = threadIdx.x & 31, grp = lane / LG, e0 = (lane & (LG - 1)) * 8, warp = threadIdx.x >> 5;
  const long long items = (long long)a.N * sd.nchunk;
  const int ctas = isq ? a.ctas_q : gridDim.x - a.ctas_q, cta = blockIdx.x - (isq ? 0 : a.ctas_q);
  float w[8], dw[8] = {};
  if (sd.w) load8(sd.w + e0, false, w);
  for (long long item = (long long)cta * 8 + warp; item < items; item += (long long)ctas * 8) {
    const int n = (int)(item / sd.nchunk), h0 = (int)(item - (long long)n * sd.nchunk) * sd.HC;
    const int h1 = min(sd.H, h0 + sd.HC);
    const TX* x0 = static_cast<const TX*>(sd.x) + n * sd.row + e0;
    const TY* g0 = static_cast<const TY*>(sd.gy) + (long long)n * sd.H * D + e0;
    TX* d0 = static_cast<TX*>(sd.y) + (long long)n * sd.H * D + e0;
    Turn8<D> t;
    for (int h = h0 + grp, first = 1; h - grp < h1; h += U * GW, first = 0) {
      Oct<TX> rx[U];
      Oct<TY> rg[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * GW < h1) {
          load8_raw(g0 + (h + u * GW) * D, true, rg[u]);
          if (sd.w) load8_raw(x0 + (h + u * GW) * sd.head, sd.vec, rx[u]);
        }
      if (first) t.set(a.rope, a.rope.n_rot ? a.pos[n] : 0, e0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h - grp + u * GW >= h1) break;  // (the same in all lanes)
        const bool on = h + u * GW < h1;
        float x[8] = {}, g[8] = {};
        if (on) unpack8(rg[u], g);
        if (a.rope.n_rot) t.apply(g, a.rope.style, -1.f);
        if (sd.w) {
          if (on) unpack8(rx[u], x);
          float ss = 0.f, hx = 0.f, gx[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            gx[j] = g[j] * x[j];
            ss = fmaf(x[j], x[j], ss), hx = fmaf(gx[j], w[j], hx);
          }
          ss = group_sum<LG>(ss);
          hx = group_sum<LG>(hx);
          const float r = inv_rms(ss, 1.f / D, a.eps), m = -hx * (1.f / D) * r * r * r;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (on) dw[j] = fmaf(gx[j], r, dw[j]);
            g[j] = fmaf(g[j] * w[j], r, x[j] * m);
          }
        }
        if (on) store8(d0 + (h + u * GW) * D, g);
      }
    }
  }
  if (!sd.w) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) red[warp * GW + grp][e0 + j] = dw[j];
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += 256) {
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < 8 * GW; ++g) s += red[g][c];
    a.part[(long long)blockIdx.x * D + c] = s;
  }
}

// dw = the CTAs' sums in a fixed order: 32 columns a CTA, each split over 32 rows of threads.  blockIdx.y 0:
// queries, 1: keys.
__global__ void __launch_bounds__(1024) k_dw_reduce(const float* part, int ctas_q, int ctas, int D, float* dwq, float* dwk) {
  __shared__ float red[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x, b0 = blockIdx.y ? ctas_q : 0, b1 = blockIdx.y ? ctas : ctas_q;
  float* out = blockIdx.y ? dwk : dwq;
  if (!out) return;
  float s = 0.f;
  for (int b = b0 + threadIdx.y; b < b1; b += 32) s += part[(long long)b * D + c];
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0) {
    s = 0.f;
#pragma unroll
    for (int y = 0; y < 32; ++y) s += red[y][threadIdx.x];
    out[c] = s;
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
  NormSide& sq = a->side[0];
  NormSide& sk = a->side[1];
  sq.x = q, sq.row = v.q_row, sq.head = v.q_head, sq.w = wq, sq.H = H, sq.vec = rows_on_16(q, v.q_row, v.q_head, es);
  sk.x = k, sk.row = v.k_row, sk.head = v.k_head, sk.w = wk, sk.H = Hkv, sk.vec = rows_on_16(k, v.k_row, v.k_head, es);
  a->eps = eps, a->pos = pos, a->N = N;
  return FA_OK;
}

// Heads of a token that one warp takes: `most` where there are tokens enough to fill the card with warps
// of that, else fewer, down to the heads that lie side by side in a warp.
static void chunk_heads(NormArgs* a, int D, int nsm, int most) {
  const int side = 256 / D;  // heads side by side
  const long long rows = (long long)a->N * (a->side[0].H + a->side[1].H) / (16LL * nsm * side);
  for (NormSide& s : a->side) {
    if (s.H == 0) {
      s.HC = 1, s.nchunk = 0;
      continue;
    }
    const int hc = (int)std::max(1LL, std::min<long long>(rows, most / side)) * side;
    s.nchunk = (s.H + hc - 1) / hc;
    s.HC = ((s.H + s.nchunk - 1) / s.nchunk + side - 1) / side * side;
    s.nchunk = (s.H + s.HC - 1) / s.HC;
  }
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
  a.side[0].y = q_out, a.side[1].y = k_out;
  chunk_heads(&a, D, nsm, 16);
  const long long bq = ((long long)N * a.side[0].nchunk + 7) / 8, bk = ((long long)N * a.side[1].nchunk + 7) / 8;
  if (bq + bk > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  a.ctas_q = (int)bq;
  pick_norm(false, D, x_type, y_type)<<<(unsigned)(bq + bk), 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

extern "C" size_t fa_qk_norm_rope_backward_workspace_size(int N, int H, int Hkv, int D) {
  if (N < 0 || H < 1 || Hkv < 0 || !head_size(D)) return 0;
  int nsm = 0, *err = nullptr;
  if (fab_device(&nsm, &err) != FA_OK) nsm = 152;
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
  chunk_heads(&a, D, nsm, 8);
  // CTAs shared out by the heads of either side; every side that has heads gets one
  const long long iq = (long long)N * a.side[0].nchunk, ik = (long long)N * a.side[1].nchunk;
  const int all = back_ctas(nsm);
  int ck = Hkv ? (int)std::min<long long>(std::max(1LL, (long long)all * Hkv / (H + Hkv)), std::max(1LL, (ik + 7) / 8)) : 0;
  const int cq = (int)std::min<long long>(all - ck, std::max(1LL, (iq + 7) / 8));
  a.ctas_q = cq;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  pick_norm(true, D, x_type, y_type)<<<cq + ck, 256, 0, s>>>(a);
  float* oq = wq ? dwq : nullptr;
  float* ok = wk && Hkv ? dwk : nullptr;
  if (oq || ok) k_dw_reduce<<<dim3(D / 32, 2), dim3(32, 32), 0, s>>>(a.part, cq, cq + ck, D, oq, ok);
  if (wk && !Hkv && dwk) cudaMemsetAsync(dwk, 0, D * sizeof(float), s);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
