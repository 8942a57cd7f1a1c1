// Rows into and out of a paged raw K/V cache.  A token's activations are read once and its cache rows
// written once (append), or the other way (read).  On a GB300, of GPU time: 2048 tokens of 4 KV heads of
// 256 (f32 to q8_0, keys normalised and rotated) 8.0 us where their bytes would take 3.1 at the copy rate, 5003 tokens
// of 8 heads of 128 (bf16 to f16 and q4_0) 14.7 for 4.9; reading those back in binary16 4.3 for 1.9 and 6.3 for 4.9,
// raw 3.4 for 1.3 and 7.8 for 3.9; 64 tokens 3.4 and 1.9, a launch and its latencies.  Norm, rotation, largest
// magnitude, codes, border test and packing are 25 to 33 instructions a value and lane (counted), but fewer than half
// of the issue slots are used (1.9 and 2.1 of 4 a cycle and SM): an append's warps, 30 % of an SM's, wait for their
// loads and for the shuffles of one row at a time.  The decoded read waits for loads and, since one kernel
// holds every type of K and V, for instructions.
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
  uint32_t mul;
  int shift;
  page_divisor(c->page_size, &mul, &shift);
  *out = Cache{static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->page_table, c->k_type, c->v_type,
               c->num_pages, c->page_size, c->B, c->max_pages, c->Hkv, c->D, c->Dv, (int)rbk, (int)rbv, nullptr, mul, shift};
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
// A code is the nearest integer to y = x / d (q8_0: d = amax / 127, ties away from zero; q4_0: d = m / -8,
// ties up).  Adding 1.5 * 2^23 to x * (1 / d) rounds it to the nearest integer, which is then in the
// sum's low bits; the remainder x * (1 / d) - n says how near a border it was.  The product is off by
// about 2^-23 of itself, so within 2^-12 of a border between two codes the decision is taken again, out
// of line, on exact products: 127 |x| against (n + 1/2) amax, or -8 x against (k - 1/2) m, each product
// as the f32 pair that fma gives.

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
constexpr float kNearBorder = 0.5f - 0x1p-12f;
constexpr float kTiny = 1e-30f;       // below this the binary16 scale is zero, whatever the codes

__device__ __forceinline__ float prod_diff(float a, float b, float c, float d) {  // a b - c d
  const float p = a * b, q = c * d;
  return (p - q) + (fmaf(a, b, -p) - fmaf(c, d, -q));
}
// The code of x near a border, plus kMagic
static __device__ __noinline__ float q8_border(float x, float inv, float am) {
  const float n = floorf(fabsf(x) * inv);
  return kMagic + copysignf(prod_diff(127.f, fabsf(x), n + 0.5f, am) >= 0.f ? n + 1.f : n, x);
}
static __device__ __noinline__ float q4_border(float x, float inv, float m) {
  const float k = rintf(fmaf(x, inv, 0.5f)), df = prod_diff(-8.f, x, k - 0.5f, m);
  return kMagic + 8.f + ((m > 0.f ? df >= 0.f : df <= 0.f) ? k : k - 1.f);
}
// The largest and the smallest of three; a NaN wins, so that a block that holds one gets a NaN for its scale.
__device__ __forceinline__ float largest(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float smallest(float a, float b, float c) {
  float y;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint32_t low_bytes(const float* t) {  // the low bytes of four sums
  const uint32_t a = __byte_perm(__float_as_uint(t[0]), __float_as_uint(t[1]), 0x0040);
  const uint32_t b = __byte_perm(__float_as_uint(t[2]), __float_as_uint(t[3]), 0x0040);
  return __byte_perm(a, b, 0x5410);
}

// Eight codes as bytes in lo, hi; the block's scale in d.
__device__ __forceinline__ void quant_q8(const float (&x)[8], uint32_t& lo, uint32_t& hi, __half& d) {
  float am = largest(largest(fabsf(x[0]), fabsf(x[1]), fabsf(x[2])), largest(fabsf(x[3]), fabsf(x[4]), fabsf(x[5])),
                     largest(fabsf(x[6]), fabsf(x[7]), 0.f));
  am = largest(am, __shfl_xor_sync(kFull, am, 1), 0.f);
  am = largest(am, __shfl_xor_sync(kFull, am, 2), 0.f);
  d = __float2half_rn(am / 127.f);
  const float inv = am > kTiny ? 127.f * __frcp_rn(am) : 0.f;
  float t[8], near = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = fmaf(x[i], inv, kMagic);
    near = fmaxf(near, fabsf(fmaf(x[i], inv, kMagic - t[i])));
  }
  if (near > kNearBorder) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (fabsf(fmaf(x[i], inv, kMagic - t[i])) > kNearBorder) t[i] = q8_border(x[i], inv, am);
  }
  lo = low_bytes(t), hi = low_bytes(t + 4);
}

// The first of the block's values of largest magnitude, where two signs share it (all lanes of the warp)
static __device__ __noinline__ float first_largest(float4 a, float4 b) {
  const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float m = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i)
    if (fabsf(x[i]) > fabsf(m)) m = x[i];
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {  // of equal ones the lower lane's
    const float m2 = __shfl_xor_sync(kFull, m, o);
    const bool lower = (threadIdx.x & o) != 0;  // the partner is the lower lane
    if (fabsf(m2) > fabsf(m) || (fabsf(m2) == fabsf(m) && lower)) m = m2;
  }
  return m;
}

// Eight codes 0..15 as bytes.
__device__ __forceinline__ void quant_q4(const float (&x)[8], uint32_t& lo, uint32_t& hi, __half& d) {
  float top = largest(largest(x[0], x[1], x[2]), largest(x[3], x[4], x[5]), largest(x[6], x[7], x[7]));
  float low = smallest(smallest(x[0], x[1], x[2]), smallest(x[3], x[4], x[5]), smallest(x[6], x[7], x[7]));
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    const float t2 = __shfl_xor_sync(kFull, top, o), l2 = __shfl_xor_sync(kFull, low, o);
    top = largest(top, t2, t2), low = smallest(low, l2, l2);
  }
  float m = (top > -low ? top : low) + 0.f;  // (+0 for a block of zeros, whatever their signs)
  const bool both = top == -low;
  if (__any_sync(kFull, both && top > 0.f)) {
    const float f = first_largest(make_float4(x[0], x[1], x[2], x[3]), make_float4(x[4], x[5], x[6], x[7]));
    if (both) m = f;
  }
  d = __float2half_rn(m * -0.125f);
  const float inv = fabsf(m) > kTiny ? -8.f * __frcp_rn(m) : 0.f;
  float t[8], near = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = fmaf(x[i], inv, kMagic + 8.f);
    near = fmaxf(near, fabsf(fmaf(x[i], inv, kMagic + 8.f - t[i])));
  }
  if (near > kNearBorder) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (fabsf(fmaf(x[i], inv, kMagic + 8.f - t[i])) > kNearBorder) t[i] = q4_border(x[i], inv, m);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = fminf(t[i], kMagic + 15.f);
  lo = low_bytes(t), hi = low_bytes(t + 4);
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
    uint8_t* p;
    if (type == FA_Q8_0) {
      quant_q8(x, lo, hi, d);
      p = row + (e0 >> 5) * 34;
    } else {
      quant_q4(x, lo, hi, d);
      const uint32_t lo2 = __shfl_xor_sync(kFull, lo, 2), hi2 = __shfl_xor_sync(kFull, hi, 2);
      lo |= lo2 << 4, hi |= hi2 << 4;  // byte b: element b low, element b + 16 high
      p = row + (e0 >> 5) * 18;
      on = on && j < 2;
    }
    if (on) {
      if (j == 0) put16(p, __half_as_ushort(d));
      p += 2 + 8 * j;
      put16(p, lo), put16(p + 2, lo >> 16), put16(p + 4, hi), put16(p + 6, hi >> 16);
    }
  }
}

constexpr int kAppendCtas = 3;  // CTAs an SM (2048 tokens with read-back 12.8 us, 14.2 with two)

// K (IS_K) or V rows: a warp takes HC heads of a token, D / 8 lanes a head, and goes on to another token.
template <int D, typename TX, bool IS_K, bool AXES>
__device__ __forceinline__ void append_rows(const RowArgs& a) {
  constexpr int LG = D / 8, GW = 32 / LG;
  const int lane = threadIdx.x & 31, grp = lane / LG, e0 = (lane & (LG - 1)) * 8;
  const bool vec = IS_K ? a.veck : a.vecv;
  const long long head = IS_K ? a.k_head : a.v_head;
  const int rb = IS_K ? a.c.rbk : a.c.rbv, type = IS_K ? a.c.k_type : a.c.v_type;
  const bool norm = IS_K && a.wk, turns = IS_K && a.rope.n_rot;
  // A key's squares are summed up as fa_qk_norm_rope() does it, so that a key stored through either is the
  // same: with FA_ROPE_HALVES from other components than the lane's eight, which it loads beside them (they are
  // in the cache then).
  const bool apart = norm && a.rope.style == FA_ROPE_HALVES;
  int ea = 0, eb = 0;
  if (apart) place_eight<D>(FA_ROPE_HALVES, a.rope.n_rot, ea, eb);
  float w[8];
  if (norm) load8(a.wk + e0, false, w);
  PairPos<D, AXES> axes;
  if (turns) axes.look_up(a.rope);
  const unsigned items = (unsigned)a.T * a.nchunk, step = gridDim.x * 8;
  for (unsigned item = blockIdx.x * 8u + (threadIdx.x >> 5); item < items; item += step) {
    const int t = item / (unsigned)a.nchunk, h0 = (int)(item - (unsigned)t * a.nchunk) * a.HC;
    const int b = a.seq[t], pos = a.pos[t];
    const TX* x0 = (IS_K ? static_cast<const TX*>(a.xk) + t * a.k_row : static_cast<const TX*>(a.xv) + t * a.v_row) + e0;
    int left = min(a.c.Hkv - h0, a.HC);
    if (b < 0 || pos < 0) continue;
    x0 += h0 * head;
    Oct<TX> raw;
    auto load = [&] {  // (lanes without a head of their own: the last head's elements, unheeded)
      const TX* p = x0 + min(grp, left - 1) * head;
      if (vec) load8_raw(p, true, raw);
      else raw = load8_any(p);
    };
    load();
    const long long cell = cache_row(a.c, b, pos);
    if (cell < 0) continue;
    uint8_t* row = (IS_K ? a.c.k : a.c.v) + (cell * a.c.Hkv + h0 + grp) * rb;
    Turn8<D> turn;
    if (turns) {
      int at[D / 64];
      axes.hand_round(AXES ? axes.load(a.rope, t) : pos, at);
      turn.set(a.rope, at, e0);
    }
#pragma unroll 1
    for (;;) {
      float x[8], r = 1.f;
      unpack8(raw, x);
      if (norm) {
        float2 sq[4];
        if (apart) {
          const TX* p = x0 - e0 + min(grp, left - 1) * head;
          Eight<TX> other;
          if (vec) load_eight<TX, true>(p, ea, eb, other);
          else load_eight<TX, false>(p, ea, eb, other);
          unpack_eight(other, sq);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) sq[j] = make_float2(x[2 * j], x[2 * j + 1]);
        }
        r = inv_rms(square_sum<D>(sq), 1.f / D, a.eps);
      }
      const bool on = grp < left, more = left > GW;
      left -= GW;
      x0 += GW * head;
      if (more) load();  // the next heads, ahead of this one's work
      if (norm) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
      }
      if (turns) turn.apply(x, a.rope.style);
      store_row8(row, type, e0, x, on);
      if (!more) break;
      row += GW * rb;
    }
  }
}

// blockIdx.y 0: keys, 1: values
template <int D, int DV, typename TX, bool AXES>
__global__ void __launch_bounds__(256, kAppendCtas) k_cache_append(const RowArgs a) {
  after_last();
  lets_next();
  if (blockIdx.y == 0) append_rows<D, TX, true, AXES>(a);
  else append_rows<DV, TX, false, AXES>(a);
}

typedef void (*RowKernel)(const RowArgs);
template <int D, typename TX, bool AXES>
static RowKernel pick_append_v(int Dv) {
  return Dv == 64 ? k_cache_append<D, 64, TX, AXES> : Dv == 128 ? k_cache_append<D, 128, TX, AXES> : k_cache_append<D, 256, TX, AXES>;
}
template <typename TX, bool AXES>
static RowKernel pick_append_d(int D, int Dv) {
  return D == 64 ? pick_append_v<64, TX, AXES>(Dv) : D == 128 ? pick_append_v<128, TX, AXES>(Dv) : pick_append_v<256, TX, AXES>(Dv);
}
template <bool AXES>
static RowKernel pick_append(int x_type, int D, int Dv) {
  return x_type == FA_ACT_F32   ? pick_append_d<float, AXES>(D, Dv)
         : x_type == FA_ACT_F16 ? pick_append_d<__half, AXES>(D, Dv)
                                : pick_append_d<__nv_bfloat16, AXES>(D, Dv);
}

// ------------------------------------------------------------------------------------------------
// read

__device__ __forceinline__ uint32_t get16(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }

// byte b (0, 1) of w as a number, less `bias`: as the low byte of 2^23
__device__ __forceinline__ float byte_minus(uint32_t w, int b, float bias) {
  return __uint_as_float(__byte_perm(w, 0x4b000000u, b ? 0x7441 : 0x7440)) - (8388608.f + bias);
}

template <int TYPE>
__device__ __forceinline__ void load_row8(const uint8_t* row, int e0, float (&x)[8]) {
  const int j = (e0 >> 3) & 3;
  if (TYPE == FA_F32) {
    load8(reinterpret_cast<const float*>(row) + e0, true, x);
  } else if (TYPE == FA_F16) {
    load8(reinterpret_cast<const __half*>(row) + e0, true, x);
  } else if (TYPE == FA_Q8_0) {
    const uint8_t* blk = row + (e0 >> 5) * 34;
    const float d = __half2float(__ushort_as_half((unsigned short)get16(blk)));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = get16(blk + 2 + 8 * j + 2 * i) ^ 0x8080u;  // code + 128
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = d * byte_minus(w[i >> 1], i & 1, 128.f);
  } else {
    const uint8_t* blk = row + (e0 >> 5) * 18;
    const float d = __half2float(__ushort_as_half((unsigned short)get16(blk)));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (get16(blk + 2 + 8 * (j & 1) + 2 * i) >> (j < 2 ? 0 : 4)) & 0x0f0fu;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = d * byte_minus(w[i >> 1], i & 1, 8.f);
  }
}

// K (IS_K) or V rows: a warp takes HC heads of a token.
template <int D, typename TY, bool IS_K, int TYPE>
__device__ __forceinline__ void read_rows(const RowArgs& a) {
  constexpr int LG = D / 8, GW = 32 / LG, RB = TYPE == FA_F32 ? 4 * D : TYPE == FA_F16 ? 2 * D : TYPE == FA_Q8_0 ? D / 32 * 34 : D / 32 * 18;
  const int lane = threadIdx.x & 31, e0 = (lane & (LG - 1)) * 8;
  const unsigned item = blockIdx.x * 8u + (threadIdx.x >> 5), t = item / (unsigned)a.nchunk;
  if (t >= (unsigned)a.T) return;
  const int b = a.seq[t], pos = a.pos[t], h0 = (int)(item - t * a.nchunk) * a.HC, h1 = min(a.c.Hkv, h0 + a.HC);
  if (b < 0 || pos < 0) return;
  const long long cell = cache_row(a.c, b, pos);
  if (cell < 0) return;
  int h = h0 + lane / LG;
  const uint8_t* row = (IS_K ? a.c.k : a.c.v) + (cell * a.c.Hkv + h) * RB;
  TY* y = static_cast<TY*>(IS_K ? a.ko : a.vo) + ((long long)t * a.c.Hkv + h) * D + e0;
#pragma unroll 4
  for (; h < h1; h += GW, row += GW * RB, y += GW * D) {
    float x[8];
    load_row8<TYPE>(row, e0, x);
    store8(y, x);
  }
}
template <int D, typename TY, bool IS_K>
__device__ __forceinline__ void read_type(const RowArgs& a) {
  switch (IS_K ? a.c.k_type : a.c.v_type) {
    case FA_F32: return read_rows<D, TY, IS_K, FA_F32>(a);
    case FA_F16: return read_rows<D, TY, IS_K, FA_F16>(a);
    case FA_Q8_0: return read_rows<D, TY, IS_K, FA_Q8_0>(a);
    default: return read_rows<D, TY, IS_K, FA_Q4_0>(a);
  }
}

template <typename TY>
__global__ void __launch_bounds__(256) k_cache_read(const RowArgs a) {
  after_last();
  lets_next();
  if (blockIdx.y == 0) {
    if (!a.ko) return;
    if (a.c.D == 64) read_type<64, TY, true>(a);
    else if (a.c.D == 128) read_type<128, TY, true>(a);
    else read_type<256, TY, true>(a);
  } else {
    if (!a.vo) return;
    if (a.c.Dv == 64) read_type<64, TY, false>(a);
    else if (a.c.Dv == 128) read_type<128, TY, false>(a);
    else read_type<256, TY, false>(a);
  }
}

// A token's cell (all KV heads' rows) is contiguous: one warp copies it in 4-byte words.
__global__ void __launch_bounds__(256) k_cache_read_raw(const RowArgs a) {
  after_last();
  lets_next();
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

// rope: by the rows' positions; axes: by rope_pos
static fa_status append(const void* k, const void* v, int x_type, const fa_kv_views* views, const fa_paged_cache* cache,
                        const int32_t* seq, const int32_t* pos, int T, const float* k_norm, float eps, const fa_rope* rope,
                        const int32_t* rope_pos, const fa_rope_axes* axes, void* stream) {
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
  if ((rc = check_rope(rope, axes, a.c.D, axes ? rope_pos : pos, T, &a.rope)) != FA_OK) return rc;
  int nsm = 0;
  if ((rc = fab_device(&nsm, &a.c.err)) != FA_OK) return rc;
  if (T == 0) return FA_OK;
  a.xk = k, a.xv = v, a.k_row = w.k_row, a.k_head = w.k_head, a.v_row = w.v_row, a.v_head = w.v_head;
  a.veck = aligned(k, 16) && (w.k_row * es) % 16 == 0 && (w.k_head * es) % 16 == 0;
  a.vecv = aligned(v, 16) && (w.v_row * es) % 16 == 0 && (w.v_head * es) % 16 == 0;
  a.wk = k_norm, a.eps = eps;
  // Heads that a warp takes of a token: one row (the heads that lie side by side), two, four, up to all,
  // whichever is done first by the warps that the SMs hold.  A token costs a warp about as much as two
  // rows before its first one (its page and the rotation's factors).
  const int side = 256 / std::min(a.c.D, a.c.Dv), all = (a.c.Hkv + side - 1) / side;
  const long long warps = 8LL * kAppendCtas * nsm;
  long long best = -1;
  for (int rows = 1;; rows = std::min(2 * rows, all)) {
    const long long items = (long long)T * ((all + rows - 1) / rows), cost = (2 * items + warps - 1) / warps * (2 + rows);
    if (best < 0 || cost <= best) best = cost, a.HC = rows * side;
    if (rows == all) break;
  }
  a.nchunk = (a.c.Hkv + a.HC - 1) / a.HC;
  if ((long long)T * a.nchunk > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  const long long blocks = ((long long)T * a.nchunk + 7) / 8;
  const dim3 grid((unsigned)std::min<long long>(blocks, kAppendCtas * nsm), 2);
  const RowKernel k_append = a.rope.axis ? pick_append<true>(x_type, a.c.D, a.c.Dv) : pick_append<false>(x_type, a.c.D, a.c.Dv);
  return launch_next(k_append, grid, dim3(256), 0, static_cast<cudaStream_t>(stream), a) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

extern "C" fa_status fa_cache_append(const void* k, const void* v, int x_type, const fa_kv_views* views,
                                     const fa_paged_cache* cache, const int32_t* seq, const int32_t* pos, int T,
                                     const float* k_norm, float eps, const fa_rope* rope, void* stream) {
  return append(k, v, x_type, views, cache, seq, pos, T, k_norm, eps, rope, nullptr, nullptr, stream);
}
extern "C" fa_status fa_cache_append_axes(const void* k, const void* v, int x_type, const fa_kv_views* views,
                                          const fa_paged_cache* cache, const int32_t* seq, const int32_t* pos, int T,
                                          const float* k_norm, float eps, const int32_t* rope_pos,
                                          const fa_rope_axes* rope, void* stream) {
  return append(k, v, x_type, views, cache, seq, pos, T, k_norm, eps, nullptr, rope_pos, rope, stream);
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
    return launch_next(k_cache_read_raw, dim3((unsigned)(((long long)T + 7) / 8), 2), dim3(256), 0, s, a) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
  } else {
    // heads that a warp takes of a token: one row of them, up to four where the card is full without
    const int side = 256 / std::min(a.c.D, a.c.Dv), all = (a.c.Hkv + side - 1) / side;
    const long long rows = std::max(1LL, std::min({4LL, (long long)all, (long long)T * all / (64LL * nsm)}));
    a.HC = (int)rows * side;
    a.nchunk = (a.c.Hkv + a.HC - 1) / a.HC;
    const long long blocks = ((long long)T * a.nchunk + 7) / 8;
    if ((long long)T * a.nchunk > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks, 2);
    const RowKernel k_read = y_type == FA_ACT_F32 ? k_cache_read<float> : y_type == FA_ACT_F16 ? k_cache_read<__half> : k_cache_read<__nv_bfloat16>;
    return launch_next(k_read, grid, dim3(256), 0, s, a) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
  }
}
