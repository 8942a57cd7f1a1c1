// Which pages of a long cache a query should attend over: bounds of each page's keys in 8 bits, a score from
// them, and the pages with the largest scores.
//
// max over a page's keys of q . k is at most sum max(q_i hi_i, q_i lo_i).  In 8 bits that sum is whole
// numbers, exact in any order, and each block of 32 adds two f32 products and one sum in a fixed tree: the score is
// the same bits wherever and however it is computed, and so are the pages chosen by it.
#include <algorithm>
#include <cmath>

#include "fa_paged.cuh"
#include "sm100.cuh"

namespace fap {

constexpr float kTinyAmax = 1e-30f;

struct BoundArgs {
  Cache c;
  int8_t* codes;
  float* scales;
  const int32_t *first, *lens;
  int Z;  // CTAs that share a sequence's pages (of one KV head)
};

__device__ __forceinline__ int len_of(const Cache& c, const int32_t* lens, int b) {
  return min(lens[b], c.max_pages * c.page_size);
}
__device__ __forceinline__ int page_of(const Cache& c, int j) { return (int)((uint64_t)(uint32_t)j * c.page_mul >> c.page_shift); }
__device__ __forceinline__ int pages_of(const Cache& c, int len) { return len > 0 ? page_of(c, len - 1) + 1 : 0; }

// ------------------------------------------------------------------------------------------------
// bounds: a lane holds eight components, D / 8 lanes a row.  A warp takes a page of its own, or where there are not as
// many pages the CTA's warps share one.

constexpr int kBoundWarps = 4;

__device__ __forceinline__ uint32_t load_u32(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }
// of three; a NaN gives way
__device__ __forceinline__ float most3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float least3(float a, float b, float c) {
  float y;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// 32768 + byte b of w
__device__ __forceinline__ float place_byte(uint32_t w, int b) { return __uint_as_float(__byte_perm(w, 0x47000000u, 0x7404 | b << 4)); }

template <int TYPE>
struct Raw8 {  // a row's eight components e0 .. e0 + 7 as they lie in memory
  uint32_t w[TYPE == FA_F32 ? 8 : TYPE == FA_F16 ? 4 : 3];

  // where in a row the lane's components start
  static __device__ __forceinline__ int place(int e0) {
    const int blk = e0 >> 5, j = (e0 >> 3) & 3;
    if (TYPE == FA_F32) return 4 * e0;
    if (TYPE == FA_F16) return 2 * e0;
    if (TYPE == FA_Q8_0) return (blk >> 1) * 68 + (blk & 1 ? 36 : 0) + 8 * j;  // a word (see load)
    return blk * 18 + 2 + 8 * (j & 1);
  }
  // p: there; e0 tells the lanes apart
  __device__ __forceinline__ void load(const uint8_t* p, int e0) {
    const int blk = e0 >> 5, j = (e0 >> 3) & 3;
    if (TYPE == FA_F32 || TYPE == FA_F16) {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
      if (TYPE == FA_F32) {
        const uint4 b = *reinterpret_cast<const uint4*>(p + 16);
        w[4 % (sizeof(w) / 4)] = b.x, w[5 % (sizeof(w) / 4)] = b.y, w[6 % (sizeof(w) / 4)] = b.z, w[7 % (sizeof(w) / 4)] = b.w;
      }
    } else if (TYPE == FA_Q8_0) {  // pairs of blocks are 17 words: the first one's codes start in the middle of one
      const bool odd = blk & 1;
      const uint32_t a = load_u32(p), b = load_u32(p + 4), c = odd ? 0 : load_u32(p + 8);
      w[0] = __funnelshift_r(a, b, odd ? 0 : 16), w[1] = __funnelshift_r(b, c, odd ? 0 : 16);
      w[2] = *reinterpret_cast<const uint16_t*>(p - 8 * j - (odd ? 2 : 0));
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
      w[0] = h[0] | (uint32_t)h[1] << 16, w[1] = h[2] | (uint32_t)h[3] << 16;
      if (j >= 2) w[0] >>= 4, w[1] >>= 4;
      w[2] = *reinterpret_cast<const uint16_t*>(p - 2 - 8 * (j & 1));
    }
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    if (TYPE == FA_F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i % (sizeof(w) / 4)]);
    } else if (TYPE == FA_F16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i % (sizeof(w) / 4)]));
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
      }
    } else {  // (32768 + code + bias) d - (32768 + bias) d: the second product is exact, and so is the sum
      constexpr uint32_t kMask = TYPE == FA_Q8_0 ? 0xffffffffu : 0x0f0f0f0fu, kFlip = TYPE == FA_Q8_0 ? 0x80808080u : 0;
      const float d = __half2float(__ushort_as_half((unsigned short)w[2]));
      // (an infinite scale makes infinities of its block, whose bounds are infinite then)
      const float off = fabsf(d) < INFINITY ? -(32768.f + (TYPE == FA_Q8_0 ? 128.f : 8.f)) * d : 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t u = (w[k] & kMask) ^ kFlip;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float2 y = __ffma2_rn(make_float2(place_byte(u, i), place_byte(u, i + 1)), make_float2(d, d), make_float2(off, off));
          x[4 * k + i] = y.x, x[4 * k + i + 1] = y.y;
        }
      }
    }
  }
};

// Largest and smallest values of rows r0, r0 + step, ... of a page's `rows` (at least one), the lane's components
template <int TYPE>
__device__ __forceinline__ void row_range(const uint8_t* page, unsigned cell, int e0, int r0, int step, int rows, float (&hi)[8], float (&lo)[8]) {
  constexpr int U = TYPE == FA_F32 ? 4 : 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) hi[i] = -INFINITY, lo[i] = INFINITY;
#pragma unroll 1
  for (int r = r0; r < rows; r += U * step) {
    Raw8<TYPE> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u].load(page + (uint64_t)(unsigned)min(r + u * step, rows - 1) * cell, e0);  // (the last row again does nothing)
#pragma unroll
    for (int u = 0; u < U; u += 2) {
      float x[8], y[8];
      raw[u].values(x), raw[u + 1].values(y);
#pragma unroll
      for (int i = 0; i < 8; ++i) hi[i] = most3(hi[i], x[i], y[i]), lo[i] = least3(lo[i], x[i], y[i]);
    }
  }
}

// Codes and scale of the lane's components: four neighbouring lanes hold a block of 32.
template <int D>
__device__ __forceinline__ void put_bounds(const BoundArgs& a, long long rec, int e0, const float (&hi)[8], const float (&lo)[8], bool on) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = most3(m, fabsf(hi[i]), fabsf(lo[i]));
  m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
  m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
  float d = 0.f;
  uint32_t up[2] = {}, down[2] = {};
  if (!(m < INFINITY)) {
    d = INFINITY, up[0] = up[1] = 0x7f7f7f7fu, down[0] = down[1] = 0x81818181u;
  } else if (m > kTinyAmax) {
    d = __fdiv_rn(m, 127.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int u = max(-127, min(127, __float2int_ru(__fdiv_rn(hi[i], d)))), l = max(-127, min(127, __float2int_rd(__fdiv_rn(lo[i], d))));
      up[i >> 2] |= (uint32_t)(u & 255) << (8 * (i & 3)), down[i >> 2] |= (uint32_t)(l & 255) << (8 * (i & 3));
    }
  }
  if (!on) return;
  *reinterpret_cast<uint2*>(a.codes + rec * 2 * D + e0) = make_uint2(up[0], up[1]);
  *reinterpret_cast<uint2*>(a.codes + rec * 2 * D + D + e0) = make_uint2(down[0], down[1]);
  if ((e0 & 31) == 0) a.scales[rec * (D / 32) + (e0 >> 5)] = d;
}

template <int D, int TYPE>
__global__ void __launch_bounds__(kBoundWarps * 32) k_page_bounds(const BoundArgs a) {
  constexpr int LG = D / 8, GW = 32 / LG;  // lanes of a row, rows side by side in a warp
  constexpr int RB = TYPE == FA_F32 ? 4 * D : TYPE == FA_F16 ? 2 * D : TYPE == FA_Q8_0 ? D / 32 * 34 : D / 32 * 18;
  __shared__ float4 s_part[kBoundWarps - 1][4][32];
  after_last();
  lets_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = (lane & (LG - 1)) * 8, grp = lane / LG;
  const unsigned hk = blockIdx.x % a.c.Hkv, rest = blockIdx.x / a.c.Hkv, z = rest % a.Z;
  const int b = rest / a.Z, L = len_of(a.c, a.lens, b), f = a.first ? a.first[b] : 0;
  if (f < 0 || f >= L) return;
  const int n = pages_of(a.c, L), p0 = page_of(a.c, f);
  const bool apart = n - p0 > a.Z;  // a warp a page
  const unsigned cell = (unsigned)a.c.Hkv * RB;
  const int all = apart ? a.Z * kBoundWarps : a.Z;
  for (int p = p0 + (int)(apart ? z * kBoundWarps + warp : z); p < n; p += all) {
    const int page = a.c.table[(long long)b * a.c.max_pages + p];
    if (page < 0 || page >= a.c.num_pages) {
      if (lane == 0) report_page(a.c.err);
      continue;
    }
    const int rows = min(a.c.page_size, L - p * a.c.page_size);
    const uint8_t* at = a.c.k + (long long)page * a.c.page_size * cell + hk * RB + Raw8<TYPE>::place(e0);
    float hi[8], lo[8];
    row_range<TYPE>(at, cell, e0, apart ? grp : warp * GW + grp, apart ? GW : kBoundWarps * GW, rows, hi, lo);
#pragma unroll
    for (int o = LG; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        hi[i] = fmaxf(hi[i], __shfl_xor_sync(kFull, hi[i], o)), lo[i] = fminf(lo[i], __shfl_xor_sync(kFull, lo[i], o));
    if (!apart) {
      if (warp) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          s_part[warp - 1][i][lane] = make_float4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
          s_part[warp - 1][2 + i][lane] = make_float4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
        }
      }
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int w = 0; w < kBoundWarps - 1; ++w)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4 x = s_part[w][i][lane], y = s_part[w][2 + i][lane];
            hi[4 * i] = fmaxf(hi[4 * i], x.x), hi[4 * i + 1] = fmaxf(hi[4 * i + 1], x.y), hi[4 * i + 2] = fmaxf(hi[4 * i + 2], x.z),
                   hi[4 * i + 3] = fmaxf(hi[4 * i + 3], x.w);
            lo[4 * i] = fminf(lo[4 * i], y.x), lo[4 * i + 1] = fminf(lo[4 * i + 1], y.y), lo[4 * i + 2] = fminf(lo[4 * i + 2], y.z),
                   lo[4 * i + 3] = fminf(lo[4 * i + 3], y.w);
          }
      }
    }
    if (apart || warp == 0) put_bounds<D>(a, (long long)page * a.c.Hkv + hk, e0, hi, lo, grp == 0);
    // (shared by the CTA, a page is its only one: there are no more than Z)
  }
}

typedef void (*BoundKernel)(const BoundArgs);
template <int D>
static BoundKernel pick_bounds(int t) {
  return t == FA_F32 ? k_page_bounds<D, FA_F32> : t == FA_F16 ? k_page_bounds<D, FA_F16> : t == FA_Q8_0 ? k_page_bounds<D, FA_Q8_0> : k_page_bounds<D, FA_Q4_0>;
}

// ------------------------------------------------------------------------------------------------
// scores, as whole numbers in their order

struct SelectArgs {
  Cache c;
  const int8_t* codes;
  const float* scales;
  const void* q;
  int act;
  long long q_row, q_head;
  const int32_t* lens;
  int H, G, K, first, last;
  float scale;
  const float* alibi;
  uint32_t* keys;  // [B][Hkv][max_pages]
  int32_t* pages;
  int chunk, chunks;  // pages that a CTA scores, CTAs of a sequence and KV head
};

constexpr uint32_t kForced = 0xffffffffu, kNoPage = 0;  // above and below every score
__device__ __forceinline__ uint32_t key_of(float s) {
  s = s != s ? INFINITY : s + 0.f;  // (one zero)
  const uint32_t u = __float_as_uint(s);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float act_at(const void* p, int act, long long i) {
  if (act == FA_ACT_F32) return static_cast<const float*>(p)[i];
  if (act == FA_ACT_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// q of `ng` query heads from h0 on in 8 bits: a warp a block, a lane a component (WARPS warps of the CTA).
constexpr int kHeads = 16;  // query heads whose codes lie in shared memory at a time
template <int D>
struct Codes {
  uint32_t q[kHeads][D / 4];
  float e[kHeads][D / 32];
};
template <int D, int WARPS>
__device__ __forceinline__ void quantise_q(const SelectArgs& a, Codes<D>& s, int b, int h0, int ng) {
  constexpr int NB = D / 32;
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int i = threadIdx.x >> 5; i < ng * NB; i += WARPS) {
    const int g = i / NB, k = i % NB;
    const float x = act_at(a.q, a.act, b * a.q_row + (h0 + g) * a.q_head + k * 32 + lane);
    const float m = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(fabsf(x))));
    const bool some = m > kTinyAmax;
    const int c = some ? max(-127, min(127, __float2int_rn(__fmul_rn(x, __fdiv_rn(127.f, m))))) : 0;
    reinterpret_cast<int8_t*>(s.q[g])[k * 32 + lane] = (int8_t)c;
    if (lane == 0) s.e[g][k] = some ? __fdiv_rn(m, 127.f) : 0.f;
  }
}

// A block of 32 components of a page's bounds
struct Block {
  uint4 hi[2], lo[2];
  float d;
};
template <int D>
__device__ __forceinline__ void load_block(const SelectArgs& a, int page, unsigned hk, int blk, Block& x) {
  if (page >= 0) {
    const long long rec = (long long)page * a.c.Hkv + hk;
    const uint4* p = reinterpret_cast<const uint4*>(a.codes + rec * 2 * D) + 2 * blk;
    x.hi[0] = p[0], x.hi[1] = p[1], x.lo[0] = p[D / 16], x.lo[1] = p[D / 16 + 1];
    x.d = a.scales[rec * (D / 32) + blk];
  } else {  // no page: nothing to read, and none may exist
    x.hi[0] = x.hi[1] = x.lo[0] = x.lo[1] = make_uint4(0, 0, 0, 0);
    x.d = 0.f;
  }
}
// The largest score of `ng` query heads for the page whose blocks D / 32 neighbouring lanes hold; far: the
// distance of its last key
template <int D>
__device__ __forceinline__ float best_score(const SelectArgs& a, const Codes<D>& s, const Block& x, int blk, int h0, int ng, float far) {
  const uint32_t hi[8] = {x.hi[0].x, x.hi[0].y, x.hi[0].z, x.hi[0].w, x.hi[1].x, x.hi[1].y, x.hi[1].z, x.hi[1].w};
  const uint32_t lo[8] = {x.lo[0].x, x.lo[0].y, x.lo[0].z, x.lo[0].w, x.lo[1].x, x.lo[1].y, x.lo[1].z, x.lo[1].w};
  float best = -INFINITY;
#pragma unroll 4
  for (int g = 0; g < ng; ++g) {
    const uint4* qv = reinterpret_cast<const uint4*>(s.q[g]) + 2 * blk;
    const uint4 q0 = qv[0], q1 = qv[1];
    const uint32_t qw[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
    int I = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t neg;  // 0xff in the bytes of negative codes
      asm("prmt.b32 %0, %1, %1, 0xba98;" : "=r"(neg) : "r"(qw[i]));
      I = __dp4a((int)((hi[i] & ~neg) | (lo[i] & neg)), (int)qw[i], I);
    }
    float t = __fmul_rn(__fmul_rn((float)I, x.d), s.e[g][blk]);
#pragma unroll
    for (int o = 1; o < D / 32; o <<= 1) t = __fadd_rn(t, __shfl_xor_sync(kFull, t, o));
    t = __fmul_rn(t, a.scale);
    if (a.alibi) t = __fadd_rn(t, __fmul_rn(a.alibi[h0 + g], far));
    best = fmaxf(best, t != t ? INFINITY : t);
  }
  return best;
}

// The scores of pages [c0, c1) of sequence b (length L, n pages) and KV head hk as keys, through put(page, key) and,
// where the query heads do not lie in shared memory at once, get(page).  A lane takes a block of 32 components, D / 32
// lanes a page; a warp looks 32 page numbers up at once and has the next pages' bounds under way while it works.
template <int D, int WARPS, typename Put, typename Get>
__device__ __forceinline__ void score_pages(const SelectArgs& a, Codes<D>& s, int b, unsigned hk, int L, int n, int c0, int c1, Put put, Get get) {
  constexpr int NB = D / 32, PW = 32 / NB, STEP = WARPS * PW;  // blocks; pages that a warp, and the CTA, takes at a time
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blk = lane & (NB - 1), mine = lane / NB;
  for (int g0 = 0; g0 < a.G; g0 += kHeads) {
    const int ng = min(kHeads, a.G - g0), h0 = (int)hk * a.G + g0;
    int found = -1;
    auto look_up = [&](int p0) {  // the warp's next NB turns, from page p0 on
      const int p = p0 + (lane / PW) * STEP + lane % PW;
      found = p < c1 ? a.c.table[(long long)b * a.c.max_pages + p] : -1;
      if (found < 0 || found >= a.c.num_pages) {
        if (p < c1) report_page(a.c.err);
        found = -1;
      }
    };
    const int first = c0 + warp * PW;
    int turn = 0;  // of the look-up
    Block x, y;
    int page = -1;
    look_up(first);
    if (first < c1) page = __shfl_sync(kFull, found, mine), load_block<D>(a, page, hk, blk, x);
    if (g0) __syncthreads();
    quantise_q<D, WARPS>(a, s, b, h0, ng);
    __syncthreads();
    for (int p0 = first; p0 < c1; p0 += STEP) {
      int page2 = -1;
      if (p0 + STEP < c1) {
        if (++turn == NB) turn = 0, look_up(p0 + STEP);
        page2 = __shfl_sync(kFull, found, turn * PW + mine);
        load_block<D>(a, page2, hk, blk, y);
      }
      const int p = p0 + mine;
      const float far = (float)(min((long long)(p + 1) * a.c.page_size, (long long)L) - L);
      const float best = best_score<D>(a, s, x, blk, h0, ng, far);
      if (p < c1 && blk == 0) {
        uint32_t key = page < 0 ? kNoPage : key_of(best);
        if (g0 && page >= 0) key = max(key, get(p));
        if (p < a.first || p >= n - a.last) key = kForced;
        put(p, key);
      }
      x = y, page = page2;
    }
  }
}

// ------------------------------------------------------------------------------------------------
// the K largest of n keys, by a CTA.  Its warps own neighbouring stretches of the pages, so that what they choose is in
// ascending order.  The K-th largest is found by bisection between the smallest and the largest: a count a step, and
// as a rule it ends when exactly K are above, after little more than log2(n) steps.

constexpr int kPickWarps = 8;

struct Count {  // a word from each warp, double-buffered: one barrier a sum
  uint32_t s[2][kPickWarps];
  uint32_t ends[2][kPickWarps];
};
// Sum over the CTA; every thread gets it.
__device__ __forceinline__ uint32_t cta_sum(uint32_t v, Count& c, int& turn) {
  const uint32_t w = __reduce_add_sync(kFull, v);
  if ((threadIdx.x & 31) == 0) c.s[turn][threadIdx.x >> 5] = w;
  __syncthreads();
  const uint4* s = reinterpret_cast<const uint4*>(c.s[turn]);
  turn ^= 1;
  uint32_t sum = 0;
#pragma unroll
  for (int i = 0; i < kPickWarps / 4; ++i) {
    const uint4 x = s[i];
    sum += (x.x + x.y) + (x.z + x.w);
  }
  return sum;
}

__device__ __forceinline__ void pick(const SelectArgs& a, const uint32_t* keys, int32_t* out, int n, Count& cnt) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rounds = (n + kPickWarps * 32 - 1) / (kPickWarps * 32), base = warp * rounds * 32 + lane;
  // the range of the scores that are not forced
  uint32_t least = 0xffffffffu, most = 0;
  for (int i = 0, p = base; i < rounds; ++i, p += 32) {
    const uint32_t k = p < n ? keys[p] : kForced;
    if (k != kForced) least = min(least, k), most = max(most, k);
  }
  least = __reduce_min_sync(kFull, least), most = __reduce_max_sync(kFull, most);
  if (lane == 0) cnt.ends[0][warp] = least, cnt.ends[1][warp] = most;
  __syncthreads();
  uint32_t lo = __reduce_min_sync(kFull, cnt.ends[0][lane & (kPickWarps - 1)]);
  uint32_t hi = __reduce_max_sync(kFull, cnt.ends[1][lane & (kPickWarps - 1)]);
  int turn = 0;
  const uint32_t K = (uint32_t)a.K;
  uint32_t above = (uint32_t)(a.first + a.last);  // keys above hi
  bool ties = false;                              // T is shared by more keys than there is room for
  uint32_t T = kForced;
  if (above < K) {  // at least K keys are at or above lo, and fewer above hi
    while (lo < hi) {
      const uint32_t mid = lo + ((hi - lo) >> 1) + 1;
      uint32_t c = 0;
#pragma unroll 4
      for (int i = 0, p = base; i < rounds; ++i, p += 32) c += p < n && keys[p] >= mid;
      c = cta_sum(c, cnt, turn);
      if (c == K) {
        T = mid;
        break;
      }
      if (c > K) lo = mid;
      else hi = mid - 1, above = c;
    }
    if (lo == hi) T = lo, ties = true;
  }
  // who is chosen, in order: those above T (or at it), and the first K - above of those at T
  const uint32_t room = ties ? K - above : 0;
  uint32_t chosen = 0, equal = 0;  // of this warp's
  for (int i = 0, p = base; i < rounds; ++i, p += 32) {
    const uint32_t k = p < n ? keys[p] : 0;
    const bool same = p < n && ties && k == T;
    chosen += __popc(__ballot_sync(kFull, p < n && k >= T && !same));
    equal += __popc(__ballot_sync(kFull, same));
  }
  __syncthreads();  // (`ends` has been read)
  if (lane == 0) cnt.ends[0][warp] = chosen, cnt.ends[1][warp] = equal;
  __syncthreads();
  uint32_t before = 0, eq_before = 0;
  for (int w = 0; w < warp; ++w) before += cnt.ends[0][w], eq_before += cnt.ends[1][w];
  before += min(eq_before, room);
  const uint32_t below = (1u << lane) - 1;
  for (int i = 0, p = base; i < rounds; ++i, p += 32) {
    const uint32_t k = p < n ? keys[p] : 0;
    const bool same = p < n && ties && k == T;
    const uint32_t eq = __ballot_sync(kFull, same);
    const bool take = same ? eq_before + __popc(eq & below) < room : p < n && k >= T;
    const uint32_t all = __ballot_sync(kFull, take);
    if (take) out[before + __popc(all & below)] = p;
    before += __popc(all), eq_before += __popc(eq);
  }
}

// A sequence of at most K pages: all of them
__device__ __forceinline__ void pick_all(const SelectArgs& a, int32_t* out, int n) {
  for (int i = threadIdx.x; i < a.K; i += kPickWarps * 32) out[i] = i < n ? i : -1;
}

// ---- in one: a cluster a sequence and KV head, whose CTAs score a stretch of the pages each; the keys go to the first
// one's shared memory, and it chooses.
__device__ __forceinline__ uint32_t at_first_cta(const void* p) {
  uint32_t a = fab::smem_u32(p), r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
  return r;
}
template <int D>
__global__ void __launch_bounds__(kPickWarps * 32, 3) k_page_select(const SelectArgs a) {
  extern __shared__ __align__(16) uint32_t s_keys[];
  __shared__ __align__(16) Codes<D> s_codes;
  __shared__ __align__(16) Count s_cnt;
  cluster_arrive();
  after_last();
  lets_next();
  const unsigned C = cluster_ctas(), rank = cluster_rank(), job = blockIdx.x / C, hk = job % a.c.Hkv;
  const int b = job / a.c.Hkv;
  if (a.lens[b] < 0) return;  // (the cluster's CTAs all leave, here and below)
  const int L = len_of(a.c, a.lens, b), n = pages_of(a.c, L);
  int32_t* out = a.pages + (long long)job * a.K;
  if (n <= a.K) {
    if (rank == 0) pick_all(a, out, n);
    return;
  }
  const uint32_t keys = at_first_cta(s_keys);
  auto put = [&](int p, uint32_t k) { asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(keys + 4 * p), "r"(k) : "memory"); };
  auto get = [&](int p) {
    uint32_t k;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(k) : "r"(keys + 4 * p) : "memory");
    return k;
  };
  cluster_wait();  // the first CTA's memory is there
  score_pages<D, kPickWarps>(a, s_codes, b, hk, L, n, (int)((long long)n * rank / C), (int)((long long)n * (rank + 1) / C), put, get);
  cluster_barrier();
  if (rank == 0) pick(a, s_keys, out, n, s_cnt);
}

// ---- in two, where the keys of a sequence may not fit there: scores into the workspace, then the choice
template <int D>
__global__ void __launch_bounds__(kPickWarps * 32, 3) k_page_scores(const SelectArgs a) {
  __shared__ __align__(16) Codes<D> s_codes;
  after_last();
  lets_next();
  const unsigned hk = blockIdx.x % a.c.Hkv, rest = blockIdx.x / a.c.Hkv;
  const int b = rest / a.chunks, c0 = (rest % a.chunks) * a.chunk;
  const int L = len_of(a.c, a.lens, b), n = pages_of(a.c, L);
  if (c0 >= n || n <= a.K) return;
  uint32_t* keys = a.keys + ((long long)b * a.c.Hkv + hk) * a.c.max_pages;
  auto put = [&](int p, uint32_t k) { keys[p] = k; };
  auto get = [&](int p) { return keys[p]; };
  score_pages<D, kPickWarps>(a, s_codes, b, hk, L, n, c0, min(n, c0 + a.chunk), put, get);
}
__global__ void __launch_bounds__(kPickWarps * 32) k_page_pick(const SelectArgs a) {
  __shared__ __align__(16) Count s_cnt;
  after_last();
  lets_next();
  const int b = blockIdx.x / a.c.Hkv;
  if (a.lens[b] < 0) return;
  const int n = pages_of(a.c, len_of(a.c, a.lens, b));
  int32_t* out = a.pages + (long long)blockIdx.x * a.K;
  if (n <= a.K) pick_all(a, out, n);
  else pick(a, a.keys + (long long)blockIdx.x * a.c.max_pages, out, n, s_cnt);
}

static fa_status check_bounds(const Cache& c, const fa_page_bounds_pool* p) {
  if (!p) return FA_ERR_NULL;
  if (c.num_pages > 0 && (!p->codes || !p->scales)) return FA_ERR_NULL;
  return aligned(p->codes, 16) && aligned(p->scales, 16) ? FA_OK : FA_ERR_ALIGN;
}
constexpr int kOnePages = 49152;  // keys that fit shared memory beside the rest (192 KB)
static size_t key_bytes(const Cache& c) {
  if (c.max_pages <= kOnePages) return 256;
  return std::max<size_t>(256, ((size_t)c.B * c.Hkv * c.max_pages * sizeof(uint32_t) + 255) / 256 * 256);
}
template <int D>
static cudaError_t run_select(SelectArgs a, int nsm, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};  // devices that the kernel's shared memory has been allowed on
  const long long rows = (long long)a.c.B * a.c.Hkv;
  if (a.c.max_pages <= kOnePages) {
    // CTAs of a cluster: as many as give each at least a turn of its warps, and all of them two to an SM
    unsigned C = 1;
    const int turn = kPickWarps * 32 / (D / 32);
    while (C < 8 && a.c.max_pages > 2 * (int)C * turn && rows * C * 2 <= 2LL * nsm) C *= 2;
    if (!allow_smem(reinterpret_cast<const void*>(k_page_select<D>), kOnePages * 4, &ready)) return cudaErrorInvalidValue;
    return launch_clusters(k_page_select<D>, (unsigned)(rows * C), C, kPickWarps * 32, (size_t)a.c.max_pages * 4, s, a);
  }
  const long long turn = kPickWarps * 32 / (D / 32), most = (a.c.max_pages + turn - 1) / turn;
  const long long want = std::min(most, std::max(1LL, 8LL * nsm / rows));
  a.chunk = (int)((most + want - 1) / want * turn);
  a.chunks = (a.c.max_pages + a.chunk - 1) / a.chunk;
  if (rows * a.chunks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const cudaError_t e = launch_next(k_page_scores<D>, dim3((unsigned)(rows * a.chunks)), dim3(kPickWarps * 32), 0, s, a);
  if (e != cudaSuccess) return e;
  return launch_next(k_page_pick, dim3((unsigned)rows), dim3(kPickWarps * 32), 0, s, a);
}
static bool select_range(const Cache& c, int H) {
  return c.max_pages <= (1 << 22) && H <= 65535 && (long long)c.B * c.Hkv < (1 << 22);
}

}  // namespace fap

using namespace fap;

extern "C" fa_status fa_page_bounds(const fa_paged_cache* cache, const fa_page_bounds_pool* bounds, const int32_t* first,
                                    const int32_t* seq_lens, void* stream) {
  BoundArgs a = {};
  fa_status rc = check_cache(cache, &a.c);
  if (rc != FA_OK) return rc;
  if ((rc = check_bounds(a.c, bounds)) != FA_OK) return rc;
  if (a.c.B > 0 && !seq_lens) return FA_ERR_NULL;
  if (!aligned(first, 4) || !aligned(seq_lens, 4)) return FA_ERR_ALIGN;
  int nsm = 0;
  if ((rc = fab_device(&nsm, &a.c.err)) != FA_OK) return rc;
  if (a.c.B == 0 || a.c.max_pages == 0) return FA_OK;
  a.codes = bounds->codes, a.scales = bounds->scales, a.first = first, a.lens = seq_lens;
  const long long rows = (long long)a.c.B * a.c.Hkv;
  a.Z = (int)std::max(1LL, std::min<long long>(a.c.max_pages, 8LL * nsm / rows));
  if (rows * a.Z > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  const BoundKernel k = a.c.D == 64 ? pick_bounds<64>(a.c.k_type) : a.c.D == 128 ? pick_bounds<128>(a.c.k_type) : pick_bounds<256>(a.c.k_type);
  return launch_next(k, dim3((unsigned)(rows * a.Z)), dim3(kBoundWarps * 32), 0, static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

extern "C" size_t fa_page_select_workspace_size(const fa_paged_cache* cache, int H, int K) {
  Cache c;
  if (check_cache(cache, &c) != FA_OK || H < 1 || H % c.Hkv || K < 1 || !select_range(c, H)) return 0;
  return key_bytes(c);
}

extern "C" fa_status fa_page_select(const void* q, int act, int64_t q_row, int64_t q_head, const fa_paged_cache* cache,
                                    const fa_page_bounds_pool* bounds, const int32_t* seq_lens, int H, float scale,
                                    const float* alibi_slopes, int K, int first, int last, int32_t* pages,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  SelectArgs a = {};
  fa_status rc = check_cache(cache, &a.c);
  if (rc != FA_OK) return rc;
  if ((rc = check_bounds(a.c, bounds)) != FA_OK) return rc;
  if (!act_type(act)) return FA_ERR_TYPE;
  if (H < 1 || H % a.c.Hkv != 0 || q_row < 0 || q_head < 0) return FA_ERR_SHAPE;
  if (K < 1 || first < 0 || last < 0 || (long long)first + last > K) return FA_ERR_SHAPE;
  if (!select_range(a.c, H) || (long long)a.c.B * a.c.Hkv * K > (1LL << 40)) return FA_ERR_UNSUPPORTED;
  if (a.c.B > 0 && (!q || !seq_lens || !pages)) return FA_ERR_NULL;
  if (!aligned(q, act_bytes(act)) || !aligned(seq_lens, 4) || !aligned(alibi_slopes, 4) || !aligned(pages, 4)) return FA_ERR_ALIGN;
  int nsm = 0;
  if ((rc = fab_device(&nsm, &a.c.err)) != FA_OK) return rc;
  if (!workspace || workspace_bytes < key_bytes(a.c)) return FA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA_ERR_ALIGN;
  if (a.c.B == 0) return FA_OK;
  a.codes = bounds->codes, a.scales = bounds->scales, a.q = q, a.act = act, a.q_row = q_row, a.q_head = q_head, a.lens = seq_lens;
  a.H = H, a.G = H / a.c.Hkv, a.K = K, a.first = first, a.last = last, a.scale = scale, a.alibi = alibi_slopes;
  a.keys = static_cast<uint32_t*>(workspace), a.pages = pages;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.c.D == 64 ? run_select<64>(a, nsm, s) : a.c.D == 128 ? run_select<128>(a, nsm, s) : run_select<256>(a, nsm, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
