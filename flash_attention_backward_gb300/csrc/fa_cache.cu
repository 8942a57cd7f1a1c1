// Rows into and out of a paged raw K/V cache.  Both directions are bound by memory: a token's
// activations are read once and its cache rows written once (append), or the other way (read).
#include <algorithm>
#include <cmath>

#include "fa_paged.cuh"

namespace fap {

fa_status check_cache(const fa_paged_cache* c, Cache* out) {
  if (!c) return FA_ERR_NULL;
  if (c->k_type < FA_F32 || c->k_type > FA_Q4_0 || c->v_type < FA_F32 || c->v_type > FA_Q4_0) return FA_ERR_TYPE;
  if (c->num_pages < 0 || c->page_size < 1 || c->B < 0 || c->max_pages < 0 || c->Hkv < 1) return FA_ERR_SHAPE;
  if (!head_size(c->D) || !head_size(c->Dv)) return FA_ERR_UNSUPPORTED;
  if (c->Hkv > 256 || c->B > (1 << 24) || (long long)c->max_pages * c->page_size > (1LL << 30)) return FA_ERR_UNSUPPORTED;
  const long rbk = fa_row_bytes(c->k_type, c->D), rbv = fa_row_bytes(c->v_type, c->Dv);
  if (((long long)c->page_size * c->Hkv * rbk) % 16 || ((long long)c->page_size * c->Hkv * rbv) % 16) return FA_ERR_ALIGN;
  if ((c->num_pages > 0 && (!c->k || !c->v)) || (c->B > 0 && c->max_pages > 0 && !c->page_table)) return FA_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4)) return FA_ERR_ALIGN;
  *out = Cache{static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->page_table, c->k_type, c->v_type,
               c->num_pages, c->page_size, c->B, c->max_pages, c->Hkv, c->D, c->Dv, (int)rbk, (int)rbv, nullptr};
  return FA_OK;
}

struct RowArgs {
  Cache c;
  const int32_t *seq, *pos;
  int T;
  const void *xk, *xv;  // append: activations
  long long k_row, k_head, v_row, v_head;
  bool veck, vecv;
  const float* wk;
  float eps;
  Rope rope;
  void *ko, *vo;  // read: outputs
  int HC, nchunk;
};

// ------------------------------------------------------------------------------------------------
// block quantisers: four neighbouring lanes hold a block of 32, eight elements each.
//
// A code is the nearest integer to x / d (q8_0: d = amax / 127, ties away from zero; q4_0: d = m / -8,
// ties up).  x * (1 / d) is off by about 2^-23 of itself, so where it falls within 2^-12 of a border
// between two codes the decision is taken again on exact products: 127 |x| against (n + 1/2) amax,
// or -8 x against (k - 1/2) m, each product as the f32 pair that fma gives.

__device__ __forceinline__ float prod_diff(float a, float b, float c, float d) {  // a b - c d
  const float p = a * b, q = c * d;
  return (p - q) + (fmaf(a, b, -p) - fmaf(c, d, -q));
}

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(kFull, v, 1));
  return fmaxf(v, __shfl_xor_sync(kFull, v, 2));
}

constexpr float kNearBorder = 0x1p-12f;
constexpr float kTiny = 1e-30f;  // below this the binary16 scale is zero, whatever the codes

// Eight codes as bytes in lo, hi; the block's scale in d.
__device__ __forceinline__ void quant_q8(const float (&x)[8], uint32_t& lo, uint32_t& hi, __half& d) {
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(x[i]));
  am = quad_max(am);
  d = __float2half_rn(am / 127.f);
  const float inv = am > kTiny ? 127.f / am : 0.f;
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = fabsf(x[i]) * inv;
    float n = floorf(y);
    const float f = y - n;
    bool up = f >= 0.5f;
    if (fabsf(f - 0.5f) < kNearBorder && inv > 0.f) up = prod_diff(127.f, fabsf(x[i]), n + 0.5f, am) >= 0.f;
    n = fminf(n + (up ? 1.f : 0.f), 127.f);
    const int c = (int)copysignf(n, x[i]);
    w[i >> 2] |= (uint32_t)(c & 255) << (8 * (i & 3));
  }
  lo = w[0], hi = w[1];
}

// Eight codes 0..15 as bytes.
__device__ __forceinline__ void quant_q4(const float (&x)[8], uint32_t& lo, uint32_t& hi, __half& d) {
  float am = 0.f, m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (fabsf(x[i]) > am) am = fabsf(x[i]), m = x[i];
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {  // the first of equal magnitudes: the lower lane's
    const float am2 = __shfl_xor_sync(kFull, am, o), m2 = __shfl_xor_sync(kFull, m, o);
    const bool lower = (threadIdx.x & o) != 0;  // the partner is the lower lane
    if (am2 > am || (am2 == am && lower)) am = am2, m = m2;
  }
  d = __float2half_rn(m * -0.125f);
  const float inv = am > kTiny ? -8.f / m : 0.f;
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = fmaf(x[i], inv, 0.5f);
    float n = floorf(t);
    const float k = rintf(t);
    if (fabsf(t - k) < kNearBorder && inv != 0.f) {
      const float df = prod_diff(-8.f, x[i], k - 0.5f, m);
      n = (m > 0.f ? df >= 0.f : df <= 0.f) ? k : k - 1.f;
    }
    const int c = (int)fminf(fmaxf(n + 8.f, 0.f), 15.f);
    w[i >> 2] |= (uint32_t)c << (8 * (i & 3));
  }
  lo = w[0], hi = w[1];
}

__device__ __forceinline__ void put16(uint8_t* p, uint32_t v) { *reinterpret_cast<uint16_t*>(p) = (uint16_t)v; }

// The lane's eight elements e0 .. e0+7 of a row; every lane of the warp takes part.
__device__ __forceinline__ void store_row8(uint8_t* row, int type, int e0, const float (&x)[8], bool on) {
  const int j = (e0 >> 3) & 3;
  if (type == FA_F32) {
    if (on) store8(reinterpret_cast<float*>(row) + e0, x);
  } else if (type == FA_F16) {
    if (on) store8(reinterpret_cast<__half*>(row) + e0, x);
  } else {
    uint32_t lo, hi;
    __half d;
    if (type == FA_Q8_0) {
      quant_q8(x, lo, hi, d);
      uint8_t* blk = row + (e0 >> 5) * 34;
      if (on) {
        if (j == 0) put16(blk, __half_as_ushort(d));
        uint8_t* p = blk + 2 + 8 * j;
        put16(p, lo), put16(p + 2, lo >> 16), put16(p + 4, hi), put16(p + 6, hi >> 16);
      }
    } else {
      quant_q4(x, lo, hi, d);
      const uint32_t lo2 = __shfl_xor_sync(kFull, lo, 2), hi2 = __shfl_xor_sync(kFull, hi, 2);
      if (on && j < 2) {  // byte b: element b low, element b + 16 high
        lo |= lo2 << 4, hi |= hi2 << 4;
        uint8_t* blk = row + (e0 >> 5) * 18;
        if (j == 0) put16(blk, __half_as_ushort(d));
        uint8_t* p = blk + 2 + 8 * j;
        put16(p, lo), put16(p + 2, lo >> 16), put16(p + 4, hi), put16(p + 6, hi >> 16);
      }
    }
  }
}

// K (IS_K) or V rows: a warp takes HC heads of one token, D / 8 lanes a head.
template <int D, typename TX, bool IS_K>
__device__ __forceinline__ void append_rows(const RowArgs& a) {
  constexpr int LG = D / 8, GW = 32 / LG, U = sizeof(TX) == 2 ? 4 : 2;
  const int lane = threadIdx.x & 31, grp = lane / LG, e0 = (lane & (LG - 1)) * 8;
  const unsigned item = blockIdx.x * 8u + (threadIdx.x >> 5);
  const int t = item / (unsigned)a.nchunk, h0 = (int)(item - (unsigned)t * a.nchunk) * a.HC;
  if (t >= a.T) return;
  const int h1 = min(a.c.Hkv, h0 + a.HC), b = a.seq[t], pos = a.pos[t];
  const bool vec = IS_K ? a.veck : a.vecv;
  const TX* x0 = (IS_K ? static_cast<const TX*>(a.xk) + t * a.k_row : static_cast<const TX*>(a.xv) + t * a.v_row) + e0;
  const long long head = IS_K ? a.k_head : a.v_head;
  float w[8];
  if (IS_K && a.wk) load8(a.wk + e0, false, w);
  if (b < 0 || pos < 0) return;
  const int rb = IS_K ? a.c.rbk : a.c.rbv, type = IS_K ? a.c.k_type : a.c.v_type;
  Turn8<D> turn;
  uint8_t* cell = nullptr;
  for (int h = h0 + grp, first = 1; h - grp < h1; h += U * GW, first = 0) {
    Oct<TX> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u * GW < h1) load8_raw(x0 + (h + u * GW) * head, vec, raw[u]);
    if (first) {
      const long long row = cache_row(a.c, b, pos);
      if (row < 0) return;
      cell = (IS_K ? a.c.k : a.c.v) + row * a.c.Hkv * (long long)rb;
      if (IS_K) turn.set(a.rope, pos, e0, 1.f);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h - grp + u * GW >= h1) break;  // (the same in all lanes)
      const bool on = h + u * GW < h1;
      float x[8] = {};
      if (on) unpack8(raw[u], x);
      if (IS_K) {
        if (a.wk) {
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
          const float r = inv_rms(group_sum<LG>(ss), 1.f / D, a.eps);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
        }
        if (a.rope.n_rot) turn.apply(x, a.rope.style);
      }
      store_row8(cell + (on ? h + u * GW : 0) * (long long)rb, type, e0, x, on);
    }
  }
}

// blockIdx.y 0: keys, 1: values
template <typename TX>
__global__ void __launch_bounds__(256) k_cache_append(const RowArgs a) {
  if (blockIdx.y == 0) {
    if (a.c.D == 64) append_rows<64, TX, true>(a);
    else if (a.c.D == 128) append_rows<128, TX, true>(a);
    else append_rows<256, TX, true>(a);
  } else {
    if (a.c.Dv == 64) append_rows<64, TX, false>(a);
    else if (a.c.Dv == 128) append_rows<128, TX, false>(a);
    else append_rows<256, TX, false>(a);
  }
}

// ------------------------------------------------------------------------------------------------
// read

__device__ __forceinline__ uint32_t get16(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }

__device__ __forceinline__ void load_row8(const uint8_t* row, int type, int e0, float (&x)[8]) {
  const int j = (e0 >> 3) & 3;
  if (type == FA_F32) {
    load8(reinterpret_cast<const float*>(row) + e0, true, x);
  } else if (type == FA_F16) {
    load8(reinterpret_cast<const __half*>(row) + e0, true, x);
  } else if (type == FA_Q8_0) {
    const uint8_t* blk = row + (e0 >> 5) * 34;
    const float d = __half2float(__ushort_as_half((unsigned short)get16(blk)));
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint32_t w = get16(blk + 2 + 8 * j + i);
      x[i] = d * (float)(int8_t)(w & 255), x[i + 1] = d * (float)(int8_t)(w >> 8);
    }
  } else {
    const uint8_t* blk = row + (e0 >> 5) * 18;
    const float d = __half2float(__ushort_as_half((unsigned short)get16(blk)));
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint32_t w = get16(blk + 2 + 8 * (j & 1) + i) >> (j < 2 ? 0 : 4);
      x[i] = d * (float)((int)(w & 15) - 8), x[i + 1] = d * (float)((int)((w >> 8) & 15) - 8);
    }
  }
}

template <int D, typename TY, bool IS_K>
__device__ __forceinline__ void read_rows(const RowArgs& a) {
  constexpr int LG = D / 8, GW = 32 / LG;
  const int lane = threadIdx.x & 31, e0 = (lane & (LG - 1)) * 8;
  const long long item = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * GW + lane / LG;
  const long long t = item / a.c.Hkv;
  const int h = (int)(item - t * a.c.Hkv);
  if (t >= a.T) return;
  const int b = a.seq[t], pos = a.pos[t];
  if (b < 0 || pos < 0) return;
  const long long cell = cache_row(a.c, b, pos);
  if (cell < 0) return;
  const int rb = IS_K ? a.c.rbk : a.c.rbv, type = IS_K ? a.c.k_type : a.c.v_type;
  float x[8];
  load_row8((IS_K ? a.c.k : a.c.v) + (cell * a.c.Hkv + h) * (long long)rb, type, e0, x);
  store8(static_cast<TY*>(IS_K ? a.ko : a.vo) + item * D + e0, x);
}

template <typename TY>
__global__ void __launch_bounds__(256) k_cache_read(const RowArgs a) {
  if (blockIdx.y == 0) {
    if (!a.ko) return;
    if (a.c.D == 64) read_rows<64, TY, true>(a);
    else if (a.c.D == 128) read_rows<128, TY, true>(a);
    else read_rows<256, TY, true>(a);
  } else {
    if (!a.vo) return;
    if (a.c.Dv == 64) read_rows<64, TY, false>(a);
    else if (a.c.Dv == 128) read_rows<128, TY, false>(a);
    else read_rows<256, TY, false>(a);
  }
}

// A token's cell (all KV heads' rows) is contiguous: one warp copies it in 4-byte words.
__global__ void __launch_bounds__(256) k_cache_read_raw(const RowArgs a) {
  const long long t = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const bool is_k = blockIdx.y == 0;
  void* out = is_k ? a.ko : a.vo;
  if (t >= a.T || !out) return;
  const int b = a.seq[t], pos = a.pos[t];
  if (b < 0 || pos < 0) return;
  const long long cell = cache_row(a.c, b, pos);
  if (cell < 0) return;
  const int words = a.c.Hkv * (is_k ? a.c.rbk : a.c.rbv) / 4;
  const uint32_t* src = reinterpret_cast<const uint32_t*>(is_k ? a.c.k : a.c.v) + cell * words;
  uint32_t* dst = static_cast<uint32_t*>(out) + t * words;
  for (int i = threadIdx.x & 31; i < words; i += 32) dst[i] = src[i];
}

}  // namespace fap

using namespace fap;

static fa_status row_args(const fa_paged_cache* cache, const int32_t* seq, const int32_t* pos, int T, RowArgs* a) {
  RowArgs z = {};
  *a = z;
  const fa_status rc = check_cache(cache, &a->c);
  if (rc != FA_OK) return rc;
  if (T < 0) return FA_ERR_SHAPE;
  if (T > 0 && (!seq || !pos)) return FA_ERR_NULL;
  if (!aligned(seq, 4) || !aligned(pos, 4)) return FA_ERR_ALIGN;
  a->seq = seq, a->pos = pos, a->T = T;
  return FA_OK;
}

extern "C" fa_status fa_cache_append(const void* k, const void* v, int x_type, const fa_kv_views* views,
                                     const fa_paged_cache* cache, const int32_t* seq, const int32_t* pos, int T,
                                     const float* k_norm, float eps, const fa_rope* rope, void* stream) {
  RowArgs a;
  fa_status rc = row_args(cache, seq, pos, T, &a);
  if (rc != FA_OK) return rc;
  if (!act_type(x_type)) return FA_ERR_TYPE;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return FA_ERR_SHAPE;
  const fa_kv_views none = {(int64_t)a.c.Hkv * a.c.D, a.c.D, (int64_t)a.c.Hkv * a.c.Dv, a.c.Dv};
  const fa_kv_views w = views ? *views : none;
  if (w.k_row < 0 || w.k_head < 0 || w.v_row < 0 || w.v_head < 0) return FA_ERR_SHAPE;
  if (T > 0 && (!k || !v)) return FA_ERR_NULL;
  const int es = act_bytes(x_type);
  if (!aligned(k, es) || !aligned(v, es) || !aligned(k_norm, 4)) return FA_ERR_ALIGN;
  if ((rc = check_rope(rope, a.c.D, pos, T, &a.rope)) != FA_OK) return rc;
  int nsm = 0;
  if ((rc = fab_device(&nsm, &a.c.err)) != FA_OK) return rc;
  if (T == 0) return FA_OK;
  a.xk = k, a.xv = v, a.k_row = w.k_row, a.k_head = w.k_head, a.v_row = w.v_row, a.v_head = w.v_head;
  a.veck = aligned(k, 16) && (w.k_row * es) % 16 == 0 && (w.k_head * es) % 16 == 0;
  a.vecv = aligned(v, 16) && (w.v_row * es) % 16 == 0 && (w.v_head * es) % 16 == 0;
  a.wk = k_norm, a.eps = eps;
  // heads that a warp takes: at least those that lie side by side, more where there are tokens enough
  const int side = 256 / std::min(a.c.D, a.c.Dv);
  const long long hc = (long long)T * a.c.Hkv / (16LL * nsm * side) * side;
  a.HC = (int)std::max<long long>(side, std::min<long long>(hc, 16));
  a.nchunk = (a.c.Hkv + a.HC - 1) / a.HC;
  const long long blocks = ((long long)T * a.nchunk + 7) / 8;
  if (blocks > 0x0fffffffLL) return FA_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks, 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (x_type == FA_ACT_F32) k_cache_append<float><<<grid, 256, 0, s>>>(a);
  else if (x_type == FA_ACT_F16) k_cache_append<__half><<<grid, 256, 0, s>>>(a);
  else k_cache_append<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

extern "C" fa_status fa_cache_read(const fa_paged_cache* cache, const int32_t* seq, const int32_t* pos, int T,
                                   int y_type, void* k_out, void* v_out, void* stream) {
  RowArgs a;
  fa_status rc = row_args(cache, seq, pos, T, &a);
  if (rc != FA_OK) return rc;
  if (!act_type(y_type) && y_type != FA_ACT_RAW) return FA_ERR_TYPE;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return FA_ERR_ALIGN;
  int nsm = 0;
  if ((rc = fab_device(&nsm, &a.c.err)) != FA_OK) return rc;
  if (T == 0 || (!k_out && !v_out)) return FA_OK;
  a.ko = k_out, a.vo = v_out;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (y_type == FA_ACT_RAW) {
    k_cache_read_raw<<<dim3((unsigned)(((long long)T + 7) / 8), 2), 256, 0, s>>>(a);
  } else {
    const int per = 8 * (256 / std::max(a.c.D, a.c.Dv));
    const long long blocks = ((long long)T * a.c.Hkv + per - 1) / per;
    if (blocks > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks, 2);
    if (y_type == FA_ACT_F32) k_cache_read<float><<<grid, 256, 0, s>>>(a);
    else if (y_type == FA_ACT_F16) k_cache_read<__half><<<grid, 256, 0, s>>>(a);
    else k_cache_read<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
