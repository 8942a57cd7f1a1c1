// Which pages of a long cache a query should attend over: bounds of each page's keys in 8 bits, a score from
// them, and the pages with the largest scores.
//
// max over a page's keys of q . k is at most sum max(q_i hi_i, q_i lo_i).  In 8 bits that sum is whole
// numbers, exact in any order, and each block of 32 adds two f32 products and one sum in a fixed tree: the score is
// the same bits wherever and however it is computed, and so are the pages chosen by it.
//
// On a GB300 (6754 GB/s measured copy rate), of GPU time.  Bounds of 75520 q8_0 keys of 4 KV heads of 256 in pages of 64 (85 MB)
// 24.6 us, 51 % of that rate: some 45 instructions a row and warp, and loads of a row's 272 bytes in words, each touching
// two or three lines.  Of the last pages of 64 sequences 5.0 us: launch, lengths, page number, rows, one after another.
// Selection among 1180 pages for 4 KV heads of 256 (6 query heads each, 64 chosen) 8.2 us, for 48 ragged sequences of up to
// 512 pages and 8 KV heads of 128 (4 query heads each) 14.3 us, where their bytes would take 0.4 and 3.9: a chain of latencies
// too (lengths, page numbers and queries, bounds, 16 pages a warp at a time, histograms), which the larger batch
// goes through one and a half times, two CTAs an SM.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fa_mma.cuh"
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

// CTAs of four warps, eight an SM, eight rows a warp under way: 24.6 us for the 75520 keys above, of which each of those
// warps takes one page; with four rows 26.0, with sixteen and five CTAs 24.2, with eight and six CTAs (two pages for some) 28.4.
constexpr int kBoundWarps = 4, kBoundCtas = 8;

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
  // top: the largest magnitude of the quantised types' scales so far
  __device__ __forceinline__ void values(float (&x)[8], float& top) const {
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
      const float d = __half2float(__ushort_as_half((unsigned short)w[2])), off = -(32768.f + (TYPE == FA_Q8_0 ? 128.f : 8.f)) * d;
      top = fmaxf(top, fabsf(d));  // (an infinite one makes NaN here, which gives way, and of its block infinities: row_range)
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
  constexpr int U = TYPE == FA_F32 ? 4 : 8;  // rows under way at a time
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) hi[i] = -INFINITY, lo[i] = INFINITY;
  auto take = [&](const Raw8<TYPE> (&raw)[U]) {
#pragma unroll
    for (int u = 0; u < U; u += 2) {
      float x[8], y[8];
      raw[u].values(x, top), raw[u + 1].values(y, top);
#pragma unroll
      for (int i = 0; i < 8; ++i) hi[i] = most3(hi[i], x[i], y[i]), lo[i] = least3(lo[i], x[i], y[i]);
    }
  };
  const uint64_t stride = (uint64_t)(unsigned)step * cell;
  const uint8_t* at = page + (uint64_t)(unsigned)min(r0, rows - 1) * cell;
  int r = r0;
#pragma unroll 1
  for (; r + (U - 1) * step < rows; r += U * step, at += U * stride) {
    Raw8<TYPE> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u].load(at + u * stride, e0);
    take(raw);
  }
  if (r < rows) {
    Raw8<TYPE> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u].load(page + (uint64_t)(unsigned)min(r + u * step, rows - 1) * cell, e0);  // (the last row again does nothing)
    take(raw);
  }
  if (top == INFINITY) {
#pragma unroll
    for (int i = 0; i < 8; ++i) hi[i] = INFINITY;
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
__global__ void __launch_bounds__(kBoundWarps * 32, kBoundCtas) k_page_bounds(const BoundArgs a) {
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
  float scale, top;  // |scale|; the code of a block's largest magnitude, 127 with the sign of scale (q changes it with scale)
  bool vec;        // every head of q starts on 16 bytes
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
// The whole numbers come from the tensor core: 16 pages by 8 query heads a product, the page's codes (largest ones,
// then smallest) against q's positive and negative codes.  A code enters as the binary16 number 1152 + code, which is an
// "and" and an "exclusive or" away from its byte, and 1152 times the sum of q's codes is taken off beforehand: all
// sums stay whole numbers below 2^24, exact in f32.  (With products of four bytes on the plain units instead: 12.8 us for
// 11.9 with the long sequence above, 17.1 for 16.5 with the ragged ones.)
//
// Of a block of 32 components, lane t = lane & 3 holds components 8 t .. 8 t + 7 of pages g and g + 8, g = lane >> 2: a word
// a k16 step, its bytes 0 and 2 the first pair of the operand, 1 and 3 the second.
constexpr int kHeads = 8;  // query heads at a time
constexpr float kCodeBias = 1152.f;
template <int D>
struct Queries {
  float4 start[D / 32][4];   // of heads 2 t and 2 t + 1: what a block's sums start from, and the scales e
  uint4 b[D / 32][2][32];    // a lane's operands of a block's four steps
};
// Query heads h0 .. h0 + ng - 1 in 8 bits: a thread takes the eight components that a lane holds of one head's block.
template <int D, int WARPS>
struct HeadPart {
  static_assert(WARPS * 32 >= D, "a part a thread");
  uint4 raw[2];  // as they lie in memory, not looked at before they are there
  // (D / 32 blocks of 8 heads by 4: whole warps take part or none of their lanes)
  static __device__ __forceinline__ bool mine() { return threadIdx.x < D; }
  static __device__ __forceinline__ int block() { return threadIdx.x >> 5; }
  static __device__ __forceinline__ int head() { return (threadIdx.x >> 2) & 7; }

  __device__ __forceinline__ void ask(const SelectArgs& a, int b, int h0, int ng) {
    if (!mine()) return;
    const long long at = b * a.q_row + (h0 + min(head(), ng - 1)) * a.q_head + block() * 32 + 8 * (threadIdx.x & 3);
    auto load = [&](auto* q) {
      Oct<std::remove_const_t<std::remove_pointer_t<decltype(q)>>> o;
      load8_raw(q + at, a.vec, o);
#pragma unroll
      for (int i = 0; i < (int)sizeof(o) / 16; ++i) raw[i] = reinterpret_cast<const uint4*>(&o)[i];
    };
    if (a.act == FA_ACT_F32) load(static_cast<const float*>(a.q));
    else load(static_cast<const __half*>(a.q));  // (two bytes of either kind)
  }
  __device__ __forceinline__ void put(const SelectArgs& a, Queries<D>& s, int ng) {
    if (!mine()) return;
    const int k = block(), g = head(), lane = threadIdx.x & 31;
    float x[8];
    if (a.act == FA_ACT_F32) unpack8(*reinterpret_cast<const Oct<float>*>(raw), x);
    else if (a.act == FA_ACT_F16) unpack8(*reinterpret_cast<const Oct<__half>*>(raw), x);
    else unpack8(*reinterpret_cast<const Oct<__nv_bfloat16>*>(raw), x);
    uint32_t top = 0;  // largest magnitude, as bits (a NaN is above infinity)
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(fabsf(x[j])));
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
    const float m = __uint_as_float(top);
    const bool some = m > kTinyAmax && g < ng;
    const float r = __fdiv_rn(a.top, m);
    int c[8], sum = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = some ? max(-127, min(127, __float2int_rn(__fmul_rn(x[j], r)))) : 0;
      sum += c[j];
    }
    sum += __shfl_xor_sync(kFull, sum, 1);
    sum += __shfl_xor_sync(kFull, sum, 2);
    uint32_t w[8];
    auto pair = [&](int lo, int hi) { return pack_h2((float)lo, (float)hi); };
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const int c0 = c[4 * st], c1 = c[4 * st + 1], c2 = c[4 * st + 2], c3 = c[4 * st + 3];
      w[2 * st] = pair(max(c0, 0), max(c2, 0)), w[2 * st + 1] = pair(max(c1, 0), max(c3, 0));
      w[4 + 2 * st] = pair(min(c0, 0), min(c2, 0)), w[5 + 2 * st] = pair(min(c1, 0), min(c3, 0));
    }
    s.b[k][0][lane] = make_uint4(w[0], w[1], w[2], w[3]), s.b[k][1][lane] = make_uint4(w[4], w[5], w[6], w[7]);
    if ((lane & 3) == 0) {
      float* st = reinterpret_cast<float*>(&s.start[k][g >> 1]);
      st[g & 1] = -kCodeBias * (float)sum, st[2 + (g & 1)] = some ? __fdiv_rn(m, 127.f) : 0.f;
    }
  }
};

// A warp's slot in shared memory: the codes of 16 pages, brought by asynchronous copies of 16 bytes a lane.  (Loaded
// into registers as the products take them, eight bytes of eight pages at a time: the same times, but a hundred
// registers more and spills.  Two slots a warp: the same.)  Rows start 32 bytes, modulo 128, after one another: the words
// of a fragment load lie in different banks.
template <int D>
struct Slot {
  static constexpr int PITCH = 2 * D + 32, BYTES = 16 * PITCH;
};
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void step(float (&c)[4], uint32_t w0, uint32_t w1, uint32_t b0, uint32_t b1) {
  constexpr uint32_t kMask = 0x00ff00ffu, kBias = 0x64806480u;  // 1152, 1152; the exclusive or flips the code's sign bit
  mma_f16(c, and_xor(w0, kMask, kBias), and_xor(w1, kMask, kBias), and_xor(w0 >> 8, kMask, kBias), and_xor(w1 >> 8, kMask, kBias), b0, b1);
}

// The scores of pages [c0, c1) of sequence b (length L, n pages) and KV head hk as keys, through put(page, key) and,
// where there are more than eight query heads, get(page); ready() is called before the first of them, and range(least,
// most) in the end by every warp, with the range of its keys that are not forced.
template <int D, int WARPS, typename Ready, typename Put, typename Get, typename Range>
__device__ __forceinline__ void score_pages(const SelectArgs& a, Queries<D>& s, uint8_t* slots, int b, unsigned hk, int L, int n, int c0, int c1, Ready ready,
                                            Put put, Get get, Range range) {
  using Sl = Slot<D>;
  constexpr int NB = D / 32, TURN = WARPS * 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint8_t* mine = slots + warp * Sl::BYTES;
  const uint32_t slot = fab::smem_u32(mine);
  // Page number of page p0 + (lane & 15), not looked at before it is used (that would wait for it); and then: -1 for none.
  auto look_up = [&](int p0) {
    const int p = p0 + (lane & 15);
    return p < c1 ? a.c.table[(long long)b * a.c.max_pages + p] : 0;
  };
  auto checked = [&](int page, int p0) {
    if (p0 + (lane & 15) >= c1) return -1;
    if (page >= 0 && page < a.c.num_pages) return page;
    report_page(a.c.err);
    return -1;
  };
  auto fetch = [&](int found) {  // their codes into the slot (where there is no page, whatever lies there)
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const int row = (i * 32 + lane) / (D / 8), off = (i * 32 + lane) % (D / 8) * 16, page = __shfl_sync(kFull, found, row);
      if (page >= 0) copy16(slot + row * Sl::PITCH + off, a.codes + ((long long)page * a.c.Hkv + hk) * 2 * D + off);
    }
    copies_end();
  };
  auto scales = [&](int found, float (&d)[NB]) {  // page lane & 15's
    const float* p = a.scales + ((long long)found * a.c.Hkv + hk) * NB;
#pragma unroll
    for (int k = 0; k < NB; k += 2) {
      const float2 v = found >= 0 ? *reinterpret_cast<const float2*>(p + k) : make_float2(0.f, 0.f);
      d[k] = v.x, d[k + 1] = v.y;
    }
  };
  for (int g0 = 0; g0 < a.G; g0 += kHeads) {
    const int ng = min(kHeads, a.G - g0), h0 = (int)hk * a.G + g0;
    int p0 = c0 + warp * 16, now = look_up(p0);
    float d[NB];
    HeadPart<D, WARPS> q;
    q.ask(a, b, h0, ng);
    now = checked(now, p0);
    fetch(now), scales(now, d);
    if (g0) __syncthreads();
    q.put(a, s, ng);
    __syncthreads();
    ready();
    uint32_t least = 0xffffffffu, most = 0;
    const float slope[2] = {a.alibi && 2 * t < ng ? a.alibi[h0 + 2 * t] : 0.f, a.alibi && 2 * t + 1 < ng ? a.alibi[h0 + 2 * t + 1] : 0.f};
    for (; p0 < c1; p0 += TURN) {
      const int next = look_up(p0 + TURN);
      copies_wait();
      __syncwarp();
      const uint8_t* at = mine + g * Sl::PITCH + 8 * t;
      auto word2 = [&](int off) { return *reinterpret_cast<const uint2*>(at + off); };
      float l0[4], l1[4], l2[4], sum[4];  // the tree over the blocks, a level each
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const float4 st = s.start[k][t];
        const uint4 b0 = s.b[k][0][lane], b1 = s.b[k][1][lane];
        float c[4] = {st.x, st.y, st.x, st.y};
        const uint2 up0 = word2(32 * k), up8 = word2(32 * k + 8 * Sl::PITCH);
        const uint2 low0 = word2(32 * k + D), low8 = word2(32 * k + D + 8 * Sl::PITCH);
        const float dk[2] = {__shfl_sync(kFull, d[k], g), __shfl_sync(kFull, d[k], g + 8)};
        step(c, up0.x, up8.x, b0.x, b0.y);
        step(c, up0.y, up8.y, b0.z, b0.w);
        step(c, low0.x, low8.x, b1.x, b1.y);
        step(c, low0.y, low8.y, b1.z, b1.w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = __fmul_rn(__fmul_rn(c[i], dk[i >> 1]), i & 1 ? st.w : st.z);
          if (!(k & 1)) {
            l0[i] = v;
            continue;
          }
          v = __fadd_rn(l0[i], v);
          if (NB > 2 && !(k & 2)) {
            l1[i] = v;
            continue;
          }
          if (NB > 2) v = __fadd_rn(l1[i], v);
          if (NB > 4 && !(k & 4)) {
            l2[i] = v;
            continue;
          }
          if (NB > 4) v = __fadd_rn(l2[i], v);
          sum[i] = v;
        }
      }
      float best[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int p = p0 + g + 8 * i;
        const float far = (float)(min((long long)(p + 1) * a.c.page_size, (long long)L) - L);
        best[i] = -INFINITY;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v = __fmul_rn(sum[2 * i + j], a.scale);
          if (a.alibi) v = __fadd_rn(v, __fmul_rn(slope[j], far));
          v = v != v ? INFINITY : v;
          if (2 * t + j < ng) best[i] = fmaxf(best[i], v);
        }
        best[i] = fmaxf(best[i], __shfl_xor_sync(kFull, best[i], 1));
        best[i] = fmaxf(best[i], __shfl_xor_sync(kFull, best[i], 2));
      }
      const int p = p0 + g + 8 * (t & 1), page = __shfl_sync(kFull, now, g + 8 * (t & 1));
      if (t < 2 && p < c1) {
        uint32_t key = page < 0 ? kNoPage : key_of(t ? best[1] : best[0]);
        if (g0 && key != kNoPage) key = max(key, get(p));
        if (p < a.first || p >= n - a.last) key = kForced;
        else least = min(least, key), most = max(most, key);
        put(p, key);
      }
      __syncwarp();  // (the slot has been read)
      now = checked(next, p0 + TURN);
      fetch(now), scales(now, d);
    }
    copies_wait();
    if (g0 + kHeads >= a.G) range(__reduce_min_sync(kFull, least), __reduce_max_sync(kFull, most));
  }
}

// ------------------------------------------------------------------------------------------------
// the K largest of n keys, by a CTA.  Its warps own neighbouring stretches of the pages, so that what they choose is in
// ascending order.  The K-th largest is found by counting keys in 256 equal bins between the smallest and the largest,
// then in 256 of the bin that it lies in, and so on: it ends when exactly K are above a bin's start, after two rounds
// as a rule.  (Bisection, a count a step, took 12 steps for 1180 pages: 3 us.)

constexpr int kBins = 256, kHeld = 8;  // kHeld: keys that a thread holds in registers

struct Bins {
  alignas(16) uint32_t n[2][kBins];  // two, so that one is empty again in time
  uint32_t ends[2][16];      // a word a warp
  uint32_t least, most;      // the range of the keys that are not forced
};
// Before the keys' range is gathered and before pick(), with a barrier behind it
__device__ __forceinline__ void clear_bins(Bins& s) {
  for (int i = threadIdx.x; i < 2 * kBins; i += blockDim.x) (&s.n[0][0])[i] = 0;
  if (threadIdx.x == 0) s.least = 0xffffffffu, s.most = 0;
}

template <int WARPS, bool HELD>
__device__ __forceinline__ void pick(const SelectArgs& a, const uint32_t* keys, int32_t* out, int n, Bins& s) {
  static_assert(WARPS * 32 >= kBins && WARPS <= 16, "a thread a bin");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rounds = (n + WARPS * 32 - 1) / (WARPS * 32), base = warp * rounds * 32 + lane;
  const uint32_t K = (uint32_t)a.K;
  uint32_t r[HELD ? kHeld : 1];
  if (HELD) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i < rounds) r[i] = base + i * 32 < n ? keys[base + i * 32] : 0;
  }
  auto each = [&](auto f) {  // f(key, page, there is one) for the thread's keys
    if (HELD) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (i < rounds) f(r[HELD ? i : 0], base + i * 32, base + i * 32 < n);
    } else {
#pragma unroll 4
      for (int i = 0; i < rounds; ++i) f(base + i * 32 < n ? keys[base + i * 32] : 0u, base + i * 32, base + i * 32 < n);
    }
  };
  uint32_t lo = s.least, hi = s.most, T = kForced, above = (uint32_t)(a.first + a.last);
  bool ties = false;  // T is shared by more keys than there is room for
  int use = 0;        // of the two sets of bins
  // `above` keys are above hi, and at least K - above in [lo, hi], which a round makes 256 times smaller: four at most
  for (int round = 0; round < 4 && above < K; ++round) {
    const int shift = max(0, 24 - __clz(hi - lo | 1));  // (hi - lo) >> shift < 256
    uint32_t* bins = s.n[use];
    each([&](uint32_t k, int, bool in) {
      if (in && k >= lo && k <= hi) atomicAdd(&bins[(k - lo) >> shift], 1u);
    });
    __syncthreads();
    // Every warp for itself: a lane eight bins, the highest ones first; keys above each lane's bins, and then each bin's
    const uint4 low = reinterpret_cast<const uint4*>(bins)[62 - 2 * lane], high = reinterpret_cast<const uint4*>(bins)[63 - 2 * lane];
    const uint32_t c[8] = {high.w, high.z, high.y, high.x, low.w, low.z, low.y, low.x};
    const uint32_t sum = ((c[0] + c[1]) + (c[2] + c[3])) + ((c[4] + c[5]) + (c[6] + c[7]));
    uint32_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(kFull, upto, o);
      if (lane >= o) upto += x;
    }
    upto += above - sum;
    uint32_t bin = 0, at = 0, all = 0;  // in the lane that holds the K-th largest: its bin, keys above it and with it
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (upto < K && K <= upto + c[i]) bin = kBins - 1 - 8 * lane - i, at = upto, all = upto + c[i];
      upto += c[i];
    }
    const int who = __ffs(__ballot_sync(kFull, all != 0)) - 1;
    if (who < 0) break;  // (keys that change meanwhile: a workspace that another call uses)
    bin = __shfl_sync(kFull, bin, who), above = __shfl_sync(kFull, at, who), all = __shfl_sync(kFull, all, who);
    lo += bin << shift;
    T = lo;
    if (all == K) break;
    if (shift == 0) {
      ties = true;
      break;
    }
    hi = lo + min(hi - lo, (1u << shift) - 1);
    use ^= 1;
    if (use == 0) {  // a third round (of four at most): the first two's bins have to be empty again
      __syncthreads();
      for (int i = tid; i < 2 * kBins; i += WARPS * 32) (&s.n[0][0])[i] = 0;
      __syncthreads();
    }
  }
  // who is chosen, in order: those above T (or at it), and the first K - above of those at T
  const uint32_t room = ties ? K - above : 0;
  uint32_t chosen = 0, equal = 0;  // of this warp's
  each([&](uint32_t k, int, bool in) {
    const bool same = in && ties && k == T;
    chosen += __popc(__ballot_sync(kFull, in && k >= T && !same));
    equal += __popc(__ballot_sync(kFull, same));
  });
  if (lane == 0) s.ends[0][warp] = chosen, s.ends[1][warp] = equal;
  __syncthreads();
  uint32_t before = __reduce_add_sync(kFull, lane < warp ? s.ends[0][lane & 15] : 0);  // (warp < 16)
  uint32_t eq_before = __reduce_add_sync(kFull, lane < warp ? s.ends[1][lane & 15] : 0);
  before += min(eq_before, room);
  const uint32_t below = (1u << lane) - 1;
  each([&](uint32_t k, int p, bool in) {
    const bool same = in && ties && k == T;
    const uint32_t eq = __ballot_sync(kFull, same);
    const bool take = same ? eq_before + __popc(eq & below) < room : in && k >= T;
    const uint32_t all = __ballot_sync(kFull, take);
    const uint32_t at = before + __popc(all & below);
    if (take && at < K) out[at] = p;
    before += __popc(all), eq_before += __popc(eq);
  });
}
template <int WARPS>
__device__ __forceinline__ void pick(const SelectArgs& a, const uint32_t* keys, int32_t* out, int n, Bins& s) {
  if (n <= kHeld * WARPS * 32) pick<WARPS, true>(a, keys, out, n, s);
  else pick<WARPS, false>(a, keys, out, n, s);
}

// A sequence of at most K pages: all of them
__device__ __forceinline__ void pick_all(const SelectArgs& a, int32_t* out, int n) {
  for (int i = threadIdx.x; i < a.K; i += blockDim.x) out[i] = i < n ? i : -1;
}

// ---- in one: a cluster a sequence and KV head, whose CTAs score a stretch of the pages each; the keys go to the first
// one's shared memory, and it chooses.
__device__ __forceinline__ uint32_t at_first_cta(const void* p) {
  uint32_t a = fab::smem_u32(p), r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
  return r;
}
template <int D, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) k_page_select(const SelectArgs a) {
  extern __shared__ __align__(16) uint8_t s_slots[];  // and the keys behind them
  __shared__ __align__(16) Queries<D> s_q;
  __shared__ Bins s_bins;
  uint32_t* s_keys = reinterpret_cast<uint32_t*>(s_slots + WARPS * Slot<D>::BYTES);
  if (cluster_rank() == 0) clear_bins(s_bins);
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
  const uint32_t keys = at_first_cta(s_keys), bins = at_first_cta(&s_bins.least);
  bool there = false;
  auto ready = [&] {  // the first CTA's memory is there
    if (!there) cluster_wait();
    there = true;
  };
  auto put = [&](int p, uint32_t k) { asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(keys + 4 * p), "r"(k) : "memory"); };
  auto get = [&](int p) {
    uint32_t k;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(k) : "r"(keys + 4 * p) : "memory");
    return k;
  };
  score_pages<D, WARPS>(a, s_q, s_slots, b, hk, L, n, (int)((long long)n * rank / C), (int)((long long)n * (rank + 1) / C), ready, put, get,
                        [&](uint32_t least, uint32_t most) {
                          if ((threadIdx.x & 31) == 0) {
                            asm volatile("red.shared::cluster.min.u32 [%0], %1;" ::"r"(bins), "r"(least) : "memory");
                            asm volatile("red.shared::cluster.max.u32 [%0], %1;" ::"r"(bins + 4), "r"(most) : "memory");
                          }
                        });
  cluster_barrier();
  if (rank == 0) pick<WARPS>(a, s_keys, out, n, s_bins);
}

// ---- in two, where the keys of a sequence may not fit there: scores into the workspace, then the choice
constexpr int kWideWarps = 8;
template <int D>
__global__ void __launch_bounds__(kWideWarps * 32, 2) k_page_scores(const SelectArgs a) {
  extern __shared__ __align__(16) uint8_t s_slots[];
  __shared__ __align__(16) Queries<D> s_q;
  after_last();
  lets_next();
  const unsigned hk = blockIdx.x % a.c.Hkv, rest = blockIdx.x / a.c.Hkv;
  const int b = rest / a.chunks, c0 = (rest % a.chunks) * a.chunk;
  const int L = len_of(a.c, a.lens, b), n = pages_of(a.c, L);
  if (c0 >= n || n <= a.K) return;
  uint32_t* keys = a.keys + ((long long)b * a.c.Hkv + hk) * a.c.max_pages;
  auto put = [&](int p, uint32_t k) { keys[p] = k; };
  auto get = [&](int p) { return keys[p]; };
  score_pages<D, kWideWarps>(a, s_q, s_slots, b, hk, L, n, c0, min(n, c0 + a.chunk), [] {}, put, get, [](uint32_t, uint32_t) {});
}
__global__ void __launch_bounds__(kWideWarps * 32) k_page_pick(const SelectArgs a) {
  __shared__ Bins s_bins;
  after_last();
  lets_next();
  const int b = blockIdx.x / a.c.Hkv;
  if (a.lens[b] < 0) return;
  const int n = pages_of(a.c, len_of(a.c, a.lens, b));
  int32_t* out = a.pages + (long long)blockIdx.x * a.K;
  if (n <= a.K) pick_all(a, out, n);
  if (n <= a.K) return;
  const uint32_t* keys = a.keys + (long long)blockIdx.x * a.c.max_pages;
  clear_bins(s_bins);
  __syncthreads();
  uint32_t least = 0xffffffffu, most = 0;
#pragma unroll 4
  for (int p = threadIdx.x; p < n; p += kWideWarps * 32) {
    const uint32_t k = keys[p];
    if (k != kForced) least = min(least, k), most = max(most, k);
  }
  atomicMin(&s_bins.least, least), atomicMax(&s_bins.most, most);
  __syncthreads();
  pick<kWideWarps>(a, keys, out, n, s_bins);
}

static fa_status check_bounds(const Cache& c, const fa_page_bounds_pool* p) {
  if (!p) return FA_ERR_NULL;
  if (c.num_pages > 0 && (!p->codes || !p->scales)) return FA_ERR_NULL;
  return aligned(p->codes, 16) && aligned(p->scales, 16) ? FA_OK : FA_ERR_ALIGN;
}
// Bytes of the slots of a CTA, and how many keys fit shared memory beside them
template <int D, int WARPS>
constexpr int kSlotBytes = WARPS * Slot<D>::BYTES;
constexpr int kSmemKeys = 208 * 1024;
static int one_pages(int D) {
  return (kSmemKeys - (D == 64 ? kSlotBytes<64, 16> : D == 128 ? kSlotBytes<128, 16> : kSlotBytes<256, 16>)) / 4;
}
static size_t key_bytes(const Cache& c) {
  if (c.max_pages <= one_pages(c.D)) return 256;
  return std::max<size_t>(256, ((size_t)c.B * c.Hkv * c.max_pages * sizeof(uint32_t) + 255) / 256 * 256);
}
template <int D, int WARPS>
static cudaError_t run_clusters(const SelectArgs& a, unsigned C, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};  // devices that the kernel's shared memory has been allowed on
  if (!allow_smem(reinterpret_cast<const void*>(k_page_select<D, WARPS>), kSmemKeys, &ready)) return cudaErrorInvalidValue;
  return launch_clusters(k_page_select<D, WARPS>, (unsigned)a.c.B * a.c.Hkv * C, C, WARPS * 32,
                         kSlotBytes<D, WARPS> + (size_t)a.c.max_pages * 4, s, a);
}
template <int D>
static cudaError_t run_select(SelectArgs a, int nsm, cudaStream_t s) {
  const long long rows = (long long)a.c.B * a.c.Hkv;
  constexpr int turn = 8 * 16;  // pages that eight warps take at a time
  if (a.c.max_pages <= one_pages(D)) {
    // CTAs of a cluster: as many as get a turn each, while all of them run at once, two to an SM; and where even
    // eight leave SMs free and have more than a turn each, CTAs of twice the warps, one to an SM.
    unsigned C = 1;
    while (C < 8 && a.c.max_pages > (int)C * turn && rows * C * 2 <= 2LL * nsm) C *= 2;
    if (C == 8 && a.c.max_pages > (int)C * turn && rows * C <= nsm) return run_clusters<D, 16>(a, C, s);
    return run_clusters<D, 8>(a, C, s);
  }
  const long long most = (a.c.max_pages + turn - 1) / turn, want = std::min(most, std::max(1LL, 8LL * nsm / rows));
  a.chunk = (int)((most + want - 1) / want * turn);
  a.chunks = (a.c.max_pages + a.chunk - 1) / a.chunk;
  if (rows * a.chunks > 0x7fffffffLL) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> ready{0};
  constexpr int bytes = kSlotBytes<D, kWideWarps>;
  if (!allow_smem(reinterpret_cast<const void*>(k_page_scores<D>), bytes, &ready)) return cudaErrorInvalidValue;
  const cudaError_t e = launch_next(k_page_scores<D>, dim3((unsigned)(rows * a.chunks)), dim3(kWideWarps * 32), bytes, s, a);
  if (e != cudaSuccess) return e;
  return launch_next(k_page_pick, dim3((unsigned)rows), dim3(kWideWarps * 32), 0, s, a);
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
  // (the host does not know the lengths: a prompt of 75520 keys among 64 requests has 4 CTAs a KV head, 947 us for 28 alone)
  a.Z = (int)std::max(1LL, std::min<long long>(a.c.max_pages, (long long)kBoundCtas * nsm / rows));
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
  if (K < 1 || first < 0 || last < 0 || (long long)first + last > K || !std::isfinite(scale)) return FA_ERR_SHAPE;
  if (!select_range(a.c, H) || (long long)a.c.B * a.c.Hkv * K > (1LL << 40)) return FA_ERR_UNSUPPORTED;
  if (a.c.B > 0 && (!q || !seq_lens || !pages)) return FA_ERR_NULL;
  if (!aligned(q, act_bytes(act)) || !aligned(seq_lens, 4) || !aligned(alibi_slopes, 4) || !aligned(pages, 4)) return FA_ERR_ALIGN;
  int nsm = 0;
  if ((rc = fab_device(&nsm, &a.c.err)) != FA_OK) return rc;
  if (!workspace || workspace_bytes < key_bytes(a.c)) return FA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA_ERR_ALIGN;
  if (a.c.B == 0) return FA_OK;
  a.codes = bounds->codes, a.scales = bounds->scales, a.q = q, a.act = act, a.q_row = q_row, a.q_head = q_head, a.lens = seq_lens;
  a.H = H, a.G = H / a.c.Hkv, a.K = K, a.first = first, a.last = last, a.scale = std::fabs(scale), a.top = std::copysign(127.f, scale);
  a.alibi = alibi_slopes;
  a.keys = static_cast<uint32_t*>(workspace), a.pages = pages;
  const int es = act_bytes(act);
  a.vec = aligned(q, 16) && (q_row * es) % 16 == 0 && (q_head * es) % 16 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.c.D == 64 ? run_select<64>(a, nsm, s) : a.c.D == 128 ? run_select<128>(a, nsm, s) : run_select<256>(a, nsm, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
