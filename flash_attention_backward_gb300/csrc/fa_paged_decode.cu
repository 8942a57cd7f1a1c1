// Attention of one new token per sequence over a paged raw cache (include/fa_paged.h).
#include <algorithm>
#include <cmath>

#include "fa_paged.cuh"

namespace fap {

struct DecodeArgs {
  Cache c;
  const void* q;
  long long q_row, q_head;
  const int32_t* lens;
  int H, G;
  float scale, softcap;
  const float *alibi, *sinks;
  void* O;
  float* lse;
};

__device__ __forceinline__ float cache_value(const uint8_t* row, int type, int e) {
  if (type == FA_F32) return reinterpret_cast<const float*>(row)[e];
  if (type == FA_F16) return __half2float(reinterpret_cast<const __half*>(row)[e]);
  const uint8_t* blk = row + (e >> 5) * (type == FA_Q8_0 ? 34 : 18);
  const float d = __half2float(*reinterpret_cast<const __half*>(blk));
  e &= 31;
  if (type == FA_Q8_0) return d * (float)(int8_t)blk[2 + e];
  return d * (float)((int)((blk[2 + (e & 15)] >> (e < 16 ? 0 : 4)) & 15) - 8);
}

// One CTA per (sequence, query head); its warps take keys in turn, each with its own running
// maximum and sum, joined at the end.
template <typename T>
__global__ void __launch_bounds__(256) k_decode_simple(const DecodeArgs a) {
  const int b = blockIdx.y, h = blockIdx.x, hk = h / a.G, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int L = a.lens[b];
  if (L < 0) return;
  if (L > a.c.max_pages * a.c.page_size) {
    L = a.c.max_pages * a.c.page_size;
    *a.c.err = FA_ERR_PAGE;
  }
  const T* q = static_cast<const T*>(a.q) + b * a.q_row + h * a.q_head;
  float qv[8], o[8] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) qv[i] = lane + 32 * i < a.c.D ? to_f32(q[lane + 32 * i]) : 0.f;
  for (int j = warp; j < L; j += 8) {
    const long long cell = cache_row(a.c, b, j);
    if (cell < 0) continue;
    const uint8_t* kr = a.c.k + (cell * a.c.Hkv + hk) * (long long)a.c.rbk;
    const uint8_t* vr = a.c.v + (cell * a.c.Hkv + hk) * (long long)a.c.rbv;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < a.c.D) s = fmaf(qv[i], cache_value(kr, a.c.k_type, lane + 32 * i), s);
    s = group_sum<32>(s) * a.scale;
    if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
    if (a.alibi) s = fmaf(a.alibi[h], (float)(j - (L - 1)), s);
    const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.f : expf(m - mn), p = mn == -INFINITY ? 0.f : expf(s - mn);
    l = l * f + p, m = mn;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < a.c.Dv) o[i] = fmaf(p, cache_value(vr, a.c.v_type, lane + 32 * i), o[i] * f);
  }
  __shared__ float sm[8], sl[8], so[8][256];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int i = 0; i < 8; ++i) so[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float M = a.sinks ? a.sinks[h] : -INFINITY, S = 0.f, x = 0.f;
  for (int w = 0; w < 8; ++w) M = fmaxf(M, sm[w]);
  const float Mf = M == -INFINITY ? 0.f : M;
  if (a.sinks) S = expf(a.sinks[h] - Mf);
  for (int w = 0; w < 8; ++w) {
    const float f = expf(sm[w] - Mf);
    S += sl[w] * f, x += so[w][threadIdx.x] * f;
  }
  if (threadIdx.x < a.c.Dv)
    static_cast<T*>(a.O)[((long long)b * a.H + h) * a.c.Dv + threadIdx.x] = from_f32<T>(S > 0.f ? x / S : 0.f);
  if (threadIdx.x == 0 && a.lse) a.lse[(long long)b * a.H + h] = Mf + logf(S);
}

}  // namespace fap

using namespace fap;

extern "C" size_t fa_paged_decode_workspace_size(const fa_paged_cache* cache, int H) {
  Cache c;
  if (check_cache(cache, &c) != FA_OK || H < 1 || H % c.Hkv) return 0;
  return 256;
}

extern "C" fa_status fa_paged_decode(const void* q, int act, int64_t q_row, int64_t q_head, const fa_paged_cache* cache,
                                     const int32_t* seq_lens, int H, float scale, const float* alibi_slopes,
                                     float softcap, const float* sinks, void* O, float* lse, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  DecodeArgs a = {};
  fa_status rc = check_cache(cache, &a.c);
  if (rc != FA_OK) return rc;
  if (!act_type(act)) return FA_ERR_TYPE;
  if (H < 1 || H % a.c.Hkv != 0 || q_row < 0 || q_head < 0) return FA_ERR_SHAPE;
  if (!(softcap >= 0.f) || !std::isfinite(softcap)) return FA_ERR_SHAPE;
  if (H > 65535 || a.c.B > 65535) return FA_ERR_UNSUPPORTED;
  if (a.c.B > 0 && (!q || !O || !seq_lens)) return FA_ERR_NULL;
  if (!aligned(q, act_bytes(act)) || !aligned(O, 16) || !aligned(lse, 4) || !aligned(seq_lens, 4) ||
      !aligned(alibi_slopes, 4) || !aligned(sinks, 4))
    return FA_ERR_ALIGN;
  int nsm = 0;
  if ((rc = fab_device(&nsm, &a.c.err)) != FA_OK) return rc;
  if (!workspace || workspace_bytes < fa_paged_decode_workspace_size(cache, H)) return FA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA_ERR_ALIGN;
  if (a.c.B == 0) return FA_OK;
  a.q = q, a.q_row = q_row, a.q_head = q_head, a.lens = seq_lens, a.H = H, a.G = H / a.c.Hkv;
  a.scale = scale, a.softcap = softcap, a.alibi = alibi_slopes, a.sinks = sinks, a.O = O, a.lse = lse;
  const dim3 grid(H, a.c.B);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (act == FA_ACT_F32) k_decode_simple<float><<<grid, 256, 0, s>>>(a);
  else if (act == FA_ACT_F16) k_decode_simple<__half><<<grid, 256, 0, s>>>(a);
  else k_decode_simple<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
