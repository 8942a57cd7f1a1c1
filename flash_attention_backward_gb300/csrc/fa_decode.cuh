// Single-token attention over a paged raw cache: the tile arithmetic.
//
// A warp takes 16 keys of one KV head at a time and up to eight query heads of its group.  Both
// products run on the tensor core with keys (S^T = K Q^T) or value components (O^T += V^T P) as the
// 16 rows and the query heads as the 8 columns, so a group of one to eight heads costs the same and
// a cache row is decoded once for all of them.  One new token means 8 columns at most: a tcgen05
// product has 128 rows of A in shared memory, so its operand would have to be decoded, scaled and
// stored there first, where mma.sync takes the decoded codes from registers.
//
// Precision.  Codes are exact in binary16 (q8_0, q4_0 keys) and in bf16 (values), and block scales
// are applied in f32, to the product (keys) or to the weight (values).  q is split into two binary16
// parts (22 bits of the head's largest magnitude, after an exact power-of-two scale), a weight times
// block scale into three bf16 parts (all 24 bits, with f32's range; two parts, 16 bits, for 16-bit outputs),
// a weight alone into two binary16 parts (22 bits), and for f32 rows all operands into two tf32 parts (three products).
//
// Bounds, on a GB300 (6787 GB/s measured copy rate; the floor is the rows, read once).  binary16 and f32 rows
// wait for DRAM: 48 ragged sequences of up to 8192 keys (32 heads, 8 KV heads of 128) in 109 us, 82 % of that rate,
// f32 rows 240 us, 74 %; one sequence of 75520 f32 keys (24 heads, 4 KV heads of 256) 97 us, 94 %.  Quantised rows
// wait for latencies: the same sequence in q8_0 (164 MB) takes 47 us, 51 %, a ragged batch of q4_0 keys and q8_0
// values with every extension 44 us, 29 %.  A tile of q8_0 keys and values of 256 is about 1365 instructions a warp,
// some 420 of them for the decoding of 8192 codes and 80 products; the 26 million of the sequence would be issued in
// 22 us, but at 1.8 of 4 a cycle and SM, no pipe above 37 %, what is short is work to switch to: three warps a
// scheduler (168 registers: 64 sums a lane), in phases of their own on some 20 KB of straight-line code ("wait" and "no
// instruction" lead the stalls), and a single slot of copies a warp.  Sixteen warps an SM at 128 registers did not
// help (45.4 us for 43.2 before the sums of tiles were kept apart), nor did rolling the key loop up.  A short call is
// a chain of latencies: launch, lengths, first rows, four tiles, the join's launch (512 keys, 2 KV heads of 128: 9 us).
// More than eight query heads to a KV head read and decode its rows once for each eight (24 heads, 2 KV heads,
// f16: 46 us where 12 heads take 36); more than 256 sequences take a launch more (300: 155 us, 83 %).
#pragma once
#include "fa_paged.cuh"
#include "sm100.cuh"

namespace fap {

using fab::lds_u16;
using fab::lds_u32;
using fab::lds_v4;
using fab::smem_u32;

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the first product of a sum: C is zero
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// (x & m) | v and (x & m) ^ v in one instruction (with two constants the compiler was seen to take two)
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t m, uint32_t v) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(x), "r"(m), "r"(v));
  return y;
}
__device__ __forceinline__ uint32_t and_xor(uint32_t x, uint32_t m, uint32_t v) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(y) : "r"(x), "r"(m), "r"(v));
  return y;
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {  // a in the low half
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_b2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lo_h(uint32_t x) { return __half2float(__ushort_as_half((unsigned short)x)); }
__device__ __forceinline__ float hi_h(uint32_t x) { return __half2float(__ushort_as_half((unsigned short)(x >> 16))); }
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bsub2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r =
      __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// ------------------------------------------------------------------------------------------------
// Which component of a head each operand element is.  The order inside a product is free as long as
// both operands agree, so it follows the words that a lane loads.  q8_0 and q4_0 blocks are 34 and
// 18 bytes: only every other block starts on a word, so words are taken from pairs of blocks (17 and 9
// words).  The first block's first and last half-word share one virtual word.

// q8_0: component of byte c of virtual word i (0..7) of block parity odd
__host__ __device__ __forceinline__ int q8_comp(bool odd, int i, int c) {
  return odd ? 4 * i + c : i == 0 ? (c < 2 ? c : 28 + c) : 4 * i - 2 + c;
}
// q4_0: byte (0..15) at byte c of virtual word i (0..3)
__host__ __device__ __forceinline__ int q4_byte(bool odd, int i, int c) {
  return odd ? 4 * i + c : i == 0 ? (c < 2 ? c : 12 + c) : 4 * i - 2 + c;
}

// Component of element e (0, 1) of B register r (0, 1) that lane t = lane & 3 holds at k16 step ks
__device__ __forceinline__ int k_comp16(int type, int ks, int t, int r, int e) {
  if (type == FA_F16) return ks * 16 + 2 * t + 8 * r + e;
  const int blk = ks >> 1, st = ks & 1;
  const bool odd = blk & 1;
  if (type == FA_Q8_0) return blk * 32 + q8_comp(odd, t + 4 * st, r + 2 * e);
  return blk * 32 + q4_byte(odd, t, st + 2 * e) + 16 * r;
}

// Component of the output tile n (16 rows), row g + 8 half
__device__ __forceinline__ int v_comp(int type, int n, int g, int half) {
  if (type == FA_F16 || type == FA_F32) return 16 * n + g + 8 * half;
  const int blk = n >> 1, T = n & 1;
  if (type == FA_Q8_0) return blk * 32 + q8_comp(blk & 1, g, 2 * T + half);
  return blk * 32 + 2 * g + T + 16 * half;
}

// A tile's sum goes to the running one by itself: the tensor core cuts off what it adds to an accumulator, half a
// unit a step on average and always towards zero, which a chain over all of a sequence's tiles would add up (96
// sequences of 20000 keys, 8 KV heads of 128, f32 outputs against 64 bits: f16 rows 1.2e-5 in one chain, 5.3e-7 so).
__device__ __forceinline__ void add_tile(float (&o)[4], const float (&c)[4]) {
  const float2 x = __fadd2_rn(make_float2(o[0], o[1]), make_float2(c[0], c[1]));
  const float2 y = __fadd2_rn(make_float2(o[2], o[3]), make_float2(c[2], c[3]));
  o[0] = x.x, o[1] = x.y, o[2] = y.x, o[3] = y.y;
}

// ------------------------------------------------------------------------------------------------
// scores: s[i] of keys g, g, g + 8, g + 8 and heads 2t, 2t + 1, 2t, 2t + 1 (the C fragment)

template <int D>
__device__ __forceinline__ void scores_f16(float (&s)[4], uint32_t rows, uint32_t qf, int lane) {
  const uint32_t at = lds_u32(rows + 4 * (lane & 15)) + (lane >> 4) * 16;
  float c2[4] = {};
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    uint32_t a0, a1, a2, a3;
    ldsm4(at + ks * 32, a0, a1, a2, a3);
    const uint4 b = lds_v4(qf + ks * 512);
    mma_f16(s, a0, a1, a2, a3, b.x, b.y);
    mma_f16(c2, a0, a1, a2, a3, b.z, b.w);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] += c2[i];
}

// the word's bytes 0, 2 and 1, 3 as binary16 pairs of signed codes: 1024 + (c + 128) - 1152
__device__ __forceinline__ void q8_h2(uint32_t w, uint32_t& x0, uint32_t& x1) {
  constexpr uint32_t kBias = 0x64806480u;  // 1152, 1152; xor with it sets the exponent and flips the sign bit
  x0 = hsub2(and_xor(w, 0x00ff00ffu, kBias), kBias);
  x1 = hsub2(and_xor(w >> 8, 0x00ff00ffu, kBias), kBias);
}

template <int D>
__device__ __forceinline__ void scores_q8(float (&s)[4], uint32_t rows, uint32_t qf, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const uint32_t r0 = lds_u32(rows + 4 * g), r1 = lds_u32(rows + 4 * g + 32);
#pragma unroll
  for (int pr = 0; pr < D / 64; ++pr) {
    const uint32_t p0 = r0 + pr * 68, p1 = r1 + pr * 68;
    const uint32_t h0 = lds_u32(p0), h1 = lds_u32(p1), m0 = lds_u32(p0 + 32), m1 = lds_u32(p1 + 32);
    uint32_t u0 = lds_u32(p0 + 4 * t), u1 = lds_u32(p1 + 4 * t);
    if (t == 0) u0 = __byte_perm(u0, m0, 0x5432), u1 = __byte_perm(u1, m1, 0x5432);
    uint32_t a0, a1, a2, a3;
    float c[4];
    uint4 b = lds_v4(qf + (pr * 4 + 0) * 512);
    q8_h2(u0, a0, a2), q8_h2(u1, a1, a3);
    mma_f16_first(c, a0, a1, a2, a3, b.x, b.y);
    mma_f16(c, a0, a1, a2, a3, b.z, b.w);
    b = lds_v4(qf + (pr * 4 + 1) * 512);
    q8_h2(lds_u32(p0 + 16 + 4 * t), a0, a2), q8_h2(lds_u32(p1 + 16 + 4 * t), a1, a3);
    mma_f16(c, a0, a1, a2, a3, b.x, b.y);
    mma_f16(c, a0, a1, a2, a3, b.z, b.w);
    float d0 = lo_h(h0), d1 = lo_h(h1);
    s[0] = fmaf(d0, c[0], s[0]), s[1] = fmaf(d0, c[1], s[1]), s[2] = fmaf(d1, c[2], s[2]), s[3] = fmaf(d1, c[3], s[3]);
    float e[4];
    b = lds_v4(qf + (pr * 4 + 2) * 512);
    q8_h2(lds_u32(p0 + 36 + 4 * t), a0, a2), q8_h2(lds_u32(p1 + 36 + 4 * t), a1, a3);
    mma_f16_first(e, a0, a1, a2, a3, b.x, b.y);
    mma_f16(e, a0, a1, a2, a3, b.z, b.w);
    b = lds_v4(qf + (pr * 4 + 3) * 512);
    q8_h2(lds_u32(p0 + 52 + 4 * t), a0, a2), q8_h2(lds_u32(p1 + 52 + 4 * t), a1, a3);
    mma_f16(e, a0, a1, a2, a3, b.x, b.y);
    mma_f16(e, a0, a1, a2, a3, b.z, b.w);
    d0 = hi_h(m0), d1 = hi_h(m1);
    s[0] = fmaf(d0, e[0], s[0]), s[1] = fmaf(d0, e[1], s[1]), s[2] = fmaf(d1, e[2], s[2]), s[3] = fmaf(d1, e[3], s[3]);
  }
}

// bytes 0, 2 of the word: low and high nibbles as binary16 pairs, minus 8
__device__ __forceinline__ void q4_h2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  constexpr uint32_t kExp = 0x64006400u, kBias = 0x64086408u;  // 1024, 1032
  lo = hsub2(and_or(w, 0x000f000fu, kExp), kBias);
  hi = hsub2(and_or(w >> 4, 0x000f000fu, kExp), kBias);
}

template <int D>
__device__ __forceinline__ void scores_q4(float (&s)[4], uint32_t rows, uint32_t qf, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const uint32_t r0 = lds_u32(rows + 4 * g), r1 = lds_u32(rows + 4 * g + 32);
#pragma unroll
  for (int pr = 0; pr < D / 64; ++pr) {
    const uint32_t p0 = r0 + pr * 36, p1 = r1 + pr * 36;
    const uint32_t h0 = lds_u32(p0), h1 = lds_u32(p1), m0 = lds_u32(p0 + 16), m1 = lds_u32(p1 + 16);
    uint32_t u0 = lds_u32(p0 + 4 * t), u1 = lds_u32(p1 + 4 * t);
    if (t == 0) u0 = __byte_perm(u0, m0, 0x5432), u1 = __byte_perm(u1, m1, 0x5432);
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      uint32_t a0, a1, a2, a3;
      float c[4];
      uint4 b = lds_v4(qf + (pr * 4 + 2 * o) * 512);
      q4_h2(u0, a0, a2), q4_h2(u1, a1, a3);
      mma_f16_first(c, a0, a1, a2, a3, b.x, b.y);
      mma_f16(c, a0, a1, a2, a3, b.z, b.w);
      b = lds_v4(qf + (pr * 4 + 2 * o + 1) * 512);
      q4_h2(u0 >> 8, a0, a2), q4_h2(u1 >> 8, a1, a3);
      mma_f16(c, a0, a1, a2, a3, b.x, b.y);
      mma_f16(c, a0, a1, a2, a3, b.z, b.w);
      const float d0 = o ? hi_h(m0) : lo_h(h0), d1 = o ? hi_h(m1) : lo_h(h1);
      s[0] = fmaf(d0, c[0], s[0]), s[1] = fmaf(d0, c[1], s[1]), s[2] = fmaf(d1, c[2], s[2]), s[3] = fmaf(d1, c[3], s[3]);
      if (o == 0) u0 = lds_u32(p0 + 20 + 4 * t), u1 = lds_u32(p1 + 20 + 4 * t);
    }
  }
}

// An f32 as two tf32 parts, of 11 bits each; the second one is rounded to them (the tensor core cuts off the
// bits below, which are the last two of 13 here; an infinity or NaN is in the first part already)
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t& hi, uint32_t& lo) {
  hi = x & 0xffffe000u;
  lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi)) + 0x1000u;
}

template <int D>
__device__ __forceinline__ void scores_f32(float (&s)[4], uint32_t rows, uint32_t qf, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const uint32_t r0 = lds_u32(rows + 4 * g) + 4 * t, r1 = lds_u32(rows + 4 * g + 32) + 4 * t;
  float c2[4] = {}, c3[4] = {};
#pragma unroll 1
  for (int k0 = 0; k0 < D / 8; k0 += 8) {
    float c[4] = {};
#pragma unroll
    for (int ks = k0; ks < k0 + 8; ++ks) {
      uint32_t h[4], l[4];
      split_tf32(lds_u32(r0 + ks * 32), h[0], l[0]);
      split_tf32(lds_u32(r1 + ks * 32), h[1], l[1]);
      split_tf32(lds_u32(r0 + ks * 32 + 16), h[2], l[2]);
      split_tf32(lds_u32(r1 + ks * 32 + 16), h[3], l[3]);
      const uint4 b = lds_v4(qf + ks * 512);
      mma_tf32(c, h[0], h[1], h[2], h[3], b.x, b.y);
      mma_tf32(c2, h[0], h[1], h[2], h[3], b.z, b.w);
      mma_tf32(c3, l[0], l[1], l[2], l[3], b.x, b.y);
    }
    add_tile(s, c);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] += c2[i] + c3[i];
}

// C fragment (keys x heads) to weights' ownership: head g, keys 2t, 2t + 1, 2t + 8, 2t + 9.  Each f32 goes
// through the 16-bit transposition as its two halves.
__device__ __forceinline__ void transpose_scores(float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t a = __float_as_uint(s[i]), b = __float_as_uint(s[i + 1]);
    const uint32_t lo = movm_t(__byte_perm(a, b, 0x5410)), hi = movm_t(__byte_perm(a, b, 0x7632));
    s[i] = __uint_as_float(__byte_perm(lo, hi, 0x5410)), s[i + 1] = __uint_as_float(__byte_perm(lo, hi, 0x7632));
  }
}

// ------------------------------------------------------------------------------------------------
// values: o[n] += V^T P for the DV / 16 tiles of 16 components; p: head g, keys 2t, 2t+1, 2t+8, 2t+9

template <int DV>
__device__ __forceinline__ void values_f16(float (&o)[DV / 16][4], const float (&p)[4], uint32_t rows, int lane) {
  const uint32_t at = lds_u32(rows + 4 * ((lane & 7) + (lane >> 4) * 8)) + ((lane >> 3) & 1) * 16;
  const uint32_t h0 = pack_h2(p[0], p[1]), h1 = pack_h2(p[2], p[3]);
  const uint32_t l0 = pack_h2(p[0] - lo_h(h0), p[1] - hi_h(h0)), l1 = pack_h2(p[2] - lo_h(h1), p[3] - hi_h(h1));
#pragma unroll
  for (int n = 0; n < DV / 16; ++n) {
    uint32_t a0, a1, a2, a3;
    ldsm4_t(at + n * 32, a0, a1, a2, a3);
    float c[4];
    mma_f16_first(c, a0, a1, a2, a3, l0, l1);
    mma_f16(c, a0, a1, a2, a3, h0, h1);
    add_tile(o[n], c);
  }
}

template <int DV>
__device__ __forceinline__ void values_f32(float (&o)[DV / 16][4], const float (&p)[4], uint32_t rows, int lane) {
  const int g = lane >> 2, t = lane & 3;
  uint32_t ph[4], pl[4], r[4];  // keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    split_tf32(__float_as_uint(p[i]), ph[i], pl[i]);
    r[i] = lds_u32(rows + 4 * (8 * (i >> 1) + 2 * t + (i & 1))) + 4 * g;
  }
#pragma unroll
  for (int n = 0; n < DV / 16; ++n) {
    uint32_t h[2][4], l[2][4];
    float c[4] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) split_tf32(lds_u32(r[2 * k + (i >> 1)] + n * 64 + 32 * (i & 1)), h[k][i], l[k][i]);
      mma_tf32(c, l[k][0], l[k][1], l[k][2], l[k][3], ph[2 * k], ph[2 * k + 1]);
      mma_tf32(c, h[k][0], h[k][1], h[k][2], h[k][3], pl[2 * k], pl[2 * k + 1]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) mma_tf32(c, h[k][0], h[k][1], h[k][2], h[k][3], ph[2 * k], ph[2 * k + 1]);
    add_tile(o[n], c);
  }
}

// Weights times block scales as three bf16 parts of eight bits each, which hold all 24 of an f32: the parts
// are cut off, so the high halves of two values and of what they leave are pairs already.  Two parts, the second one
// rounded, hold 16 bits, of which a 16-bit output keeps 11 or 8: they do for those (24 ragged sequences of mixed
// types, f16 outputs: 43.7 us, 45.5 with three; f32 outputs, 512 q8_0 keys: 1.6e-6 off 64 bits with two, 2.4e-7).
template <int PARTS>
struct Scaled {
  uint32_t h0, h1, m0, m1, l0, l1;
  static __device__ __forceinline__ uint32_t take(float& x, float& y) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    x -= __uint_as_float(a & 0xffff0000u), y -= __uint_as_float(b & 0xffff0000u);
    return __byte_perm(a, b, 0x7632);
  }
  __device__ __forceinline__ Scaled(const float (&p)[4], float d0, float d1, float d2, float d3) {
    float x0 = p[0] * d0, x1 = p[1] * d1, x2 = p[2] * d2, x3 = p[3] * d3;
    h0 = take(x0, x1), h1 = take(x2, x3);
    if (PARTS == 2) {
      m0 = pack_b2(x0, x1), m1 = pack_b2(x2, x3), l0 = l1 = 0;
    } else {
      m0 = take(x0, x1), m1 = take(x2, x3);
      l0 = take(x0, x1), l1 = take(x2, x3);
    }
  }
};

template <int PARTS>
__device__ __forceinline__ void add_scaled(float (&o)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, const Scaled<PARTS>& b) {
  float c[4];
  if (PARTS == 2) {
    mma_bf16_first(c, a0, a1, a2, a3, b.m0, b.m1);
  } else {
    mma_bf16_first(c, a0, a1, a2, a3, b.l0, b.l1);
    mma_bf16(c, a0, a1, a2, a3, b.m0, b.m1);
  }
  mma_bf16(c, a0, a1, a2, a3, b.h0, b.h1);
  add_tile(o, c);
}

// byte B of two keys' words as a bf16 pair of signed codes: (128 + low seven bits) - (128 or 256)
template <int B>
__device__ __forceinline__ uint32_t q8_b2(uint32_t k0, uint32_t k1) {
  const uint32_t v = __byte_perm(k0, k1, B * 0x11 + (4 + B) * 0x1100);  // to bytes 0 and 2
  return bsub2(and_or(v, 0x007f007fu, 0x43004300u), and_or(v, 0x00800080u, 0x43004300u));
}

template <int DV, int PARTS>
__device__ __forceinline__ void values_q8(float (&o)[DV / 16][4], const float (&p)[4], uint32_t rows, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const uint32_t r[4] = {lds_u32(rows + 8 * t), lds_u32(rows + 8 * t + 4), lds_u32(rows + 8 * t + 32), lds_u32(rows + 8 * t + 36)};
#pragma unroll
  for (int pr = 0; pr < DV / 64; ++pr) {
    uint32_t w[4], x[4];
    float d[4], e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t at = r[i] + pr * 68, h = lds_u32(at), m = lds_u32(at + 32);
      w[i] = lds_u32(at + 4 * g);
      if (g == 0) w[i] = __byte_perm(h, m, 0x5432);
      x[i] = lds_u32(at + 36 + 4 * g);
      d[i] = lo_h(h), e[i] = hi_h(m);
    }
    {
      const Scaled<PARTS> b(p, d[0], d[1], d[2], d[3]);
      const uint32_t a0 = q8_b2<0>(w[0], w[1]), a1 = q8_b2<1>(w[0], w[1]), a2 = q8_b2<0>(w[2], w[3]), a3 = q8_b2<1>(w[2], w[3]);
      add_scaled(o[4 * pr], a0, a1, a2, a3, b);
      const uint32_t c0 = q8_b2<2>(w[0], w[1]), c1 = q8_b2<3>(w[0], w[1]), c2 = q8_b2<2>(w[2], w[3]), c3 = q8_b2<3>(w[2], w[3]);
      add_scaled(o[4 * pr + 1], c0, c1, c2, c3, b);
    }
    {
      const Scaled<PARTS> b(p, e[0], e[1], e[2], e[3]);
      const uint32_t a0 = q8_b2<0>(x[0], x[1]), a1 = q8_b2<1>(x[0], x[1]), a2 = q8_b2<0>(x[2], x[3]), a3 = q8_b2<1>(x[2], x[3]);
      add_scaled(o[4 * pr + 2], a0, a1, a2, a3, b);
      const uint32_t c0 = q8_b2<2>(x[0], x[1]), c1 = q8_b2<3>(x[0], x[1]), c2 = q8_b2<2>(x[2], x[3]), c3 = q8_b2<3>(x[2], x[3]);
      add_scaled(o[4 * pr + 3], c0, c1, c2, c3, b);
    }
  }
}

// nibble at bit SH of bytes 0 and 2 as a bf16 pair, minus 8
template <int SH>
__device__ __forceinline__ uint32_t q4_b2(uint32_t w) {
  return bsub2(and_or(w >> SH, 0x000f000fu, 0x43004300u), 0x43084308u);
}

template <int DV, int PARTS>
__device__ __forceinline__ void values_q4(float (&o)[DV / 16][4], const float (&p)[4], uint32_t rows, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const uint32_t r[4] = {lds_u32(rows + 8 * t), lds_u32(rows + 8 * t + 4), lds_u32(rows + 8 * t + 32), lds_u32(rows + 8 * t + 36)};
#pragma unroll
  for (int blk = 0; blk < DV / 32; ++blk) {
    uint32_t w[4];
    float d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = lds_u16(r[i] + blk * 18 + 2 + 2 * g);  // components 2g, 2g + 1 and 2g + 16, 2g + 17
      d[i] = lo_h(lds_u16(r[i] + blk * 18));
    }
    const Scaled<PARTS> b(p, d[0], d[1], d[2], d[3]);
    const uint32_t u = w[0] | w[1] << 16, v = w[2] | w[3] << 16;
    {
      const uint32_t a0 = q4_b2<0>(u), a1 = q4_b2<4>(u), a2 = q4_b2<0>(v), a3 = q4_b2<4>(v);
      add_scaled(o[2 * blk], a0, a1, a2, a3, b);
    }
    {
      const uint32_t a0 = q4_b2<8>(u), a1 = q4_b2<12>(u), a2 = q4_b2<8>(v), a3 = q4_b2<12>(v);
      add_scaled(o[2 * blk + 1], a0, a1, a2, a3, b);
    }
  }
}

// ------------------------------------------------------------------------------------------------
// the kernel

constexpr int kMinTiles = 4;     // an item has at least this many tiles of 16 keys (where its sequence has)
constexpr int kPlanBatch = 256;  // with more sequences than this, a kernel of its own lays out the items
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.f;  // the running maximum moves when a score exceeds it by this
// Weights are exp2(x - max + lift).  Lifted by 7 (weights <= 2^15) the binary16 parts' small end is out of the way;
// of f32 values, whose weights need no such room, they stay <= 1, so that no product leaves f32's range.
__host__ __device__ constexpr float weight_lift(int vt) { return vt == FA_F32 ? -kRescale : 7.f; }
constexpr uint64_t kDrainNs = 2000000000ull;

struct DecodeArgs {
  Cache c;
  const void* q;
  int act;
  long long q_row, q_head;
  const int32_t* lens;
  int H, G, HG, chunks;  // query heads, heads of a group, (KV head, chunk of 8 heads) pairs, chunks of a group
  float scale, softcap;
  float lift;   // weight_lift() of the value type
  const float *alibi, *sinks;
  void* O;
  float* lse;
  float* part;  // [slots][HG]: partial O [8][DV], then maxima [8] and sums [8] of an item of a split sequence
  int4* jobs;   // [njobs]: the split sequences: {b, first slot, slots, 0}; b = -1 behind the last one
  int4* items;  // [nitems] laid out beforehand: {b, splits, split, slot}, b = -1 behind the last one; or NULL
  int R, nitems, njobs;  // items that the card holds at a time, that can be at most, split sequences at most
  int box;      // rows of the tensor maps' boxes, 16 or 8: a tile is one or two; 0: one bulk copy a row
  uint64_t wait_ns;   // a wait for a copy gives up after this long (0, the failure-detection hook: at once)
};

struct DecodeMaps {
  CUtensorMap k, v;
};

// ---- what a kernel's shape fixes, for the host too
__host__ __device__ constexpr int cache_row_bytes(int type, int D) {
  return type == FA_F32 ? 4 * D : type == FA_F16 ? 2 * D : type == FA_Q8_0 ? D / 32 * 34 : D / 32 * 18;
}
// bytes of a row's bulk copy: it and what pads its ends to 16-byte boundaries (the row starts up to 16 bytes,
// less its own excess over a multiple of 16, behind one)
__host__ __device__ constexpr int copy_bytes(int rb) { return (rb + 15) / 16 * 16; }
// Rows in shared memory start an odd multiple of 16 bytes after one another: the eight rows that a
// fragment load touches then lie in different banks.
__host__ __device__ constexpr int smem_pitch(int rb) { return copy_bytes(rb) % 32 == 16 ? copy_bytes(rb) : copy_bytes(rb) + 16; }
// log2 of the tensor map's element size: a box is at most 256 elements wide
__host__ __device__ constexpr int map_es(int pitch) { return pitch <= 512 ? 1 : pitch <= 1024 ? 2 : 3; }

// CTAs of few warps, several to an SM: a short sequence is a few tiles, and while one CTA starts, joins its
// warps or waits for its first rows, the others work.  Registers (about 168 a thread for Dv = 256, else
// 128) allow 12 or 16 warps an SM; shared memory may allow fewer.  What it has left goes to slots (a
// tile's key rows and value rows) of each warp's ring, which also takes the warp's sums in the end: one for
// q8_0 and f16 rows of 256 (a key row's copy is then asked for as soon as its scores are done, a value row's behind
// the products), two for q8_0 of 128, up to four for smaller rows.
// (Against CTAs that fill an SM with 8, 12 or 16 warps: 9.0 us for 11.8 with 512 keys, 41 for 58 with a
// ragged batch of mixed types.)
constexpr int kWarps = 4;
constexpr int kSmemSm = 227 * 1024;  // of an SM, for dynamic and static arrays and 1 KB a CTA
constexpr int kSlotCtl = 160;        // a slot's row addresses, barriers and mask (struct Slot of the kernel)
struct DecodeShape {
  int ctas, slots, smem, pk, pv, qf, stage, ring;
};
__host__ __device__ constexpr DecodeShape decode_shape(int D, int DV, int kt, int vt) {
  DecodeShape c{};
  c.pk = smem_pitch(cache_row_bytes(kt, D)), c.pv = smem_pitch(cache_row_bytes(vt, DV));
  c.qf = (kt == FA_F32 ? D / 8 : D / 16) * 512;
  c.stage = 16 * (c.pk + c.pv);
  const int sums = DV * 32, slot = c.stage + kSlotCtl, fixed = c.qf + DV * 4 + 3 * 1024;
  c.ctas = (DV == 256 ? 12 : 16) / kWarps;
  while (c.ctas > 1 && fixed + kWarps * (slot > sums ? slot : sums) > kSmemSm / c.ctas) --c.ctas;
  c.slots = (kSmemSm / c.ctas - fixed) / (kWarps * slot);
  if (c.slots > 4) c.slots = 4;
  c.ring = c.slots * c.stage > sums ? c.slots * c.stage : (sums + 127) / 128 * 128;
  c.smem = c.qf + kWarps * c.ring;
  return c;
}

__device__ __forceinline__ float act_load(const void* p, int act, long long i) {
  if (act == FA_ACT_F32) return static_cast<const float*>(p)[i];
  if (act == FA_ACT_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void act_store(void* p, int act, long long i, float x) {
  if (act == FA_ACT_F32) static_cast<float*>(p)[i] = x;
  else if (act == FA_ACT_F16) static_cast<__half*>(p)[i] = __float2half_rn(x);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
}

// Keys of sequence b: its length, 0 for padding, at most the table's capacity
__device__ __forceinline__ int seq_keys(const DecodeArgs& a, int b) {
  const int L = a.lens[b];
  return min(max(L, 0), a.c.max_pages * a.c.page_size);
}
__device__ __forceinline__ int tiles_of(int keys) { return (keys + 15) >> 4; }

// ---- the items of work: a sequence of n tiles is cut into ceil(n / chunk) of nearly equal size.  The chunk
// is what makes the items of all U tiles fit the card at once (R items), but not so small that joining the
// parts costs more than it gains: with w tiles an item a sequence of n takes about w / 4 tile times and
// n / w parts, least near w = 0.37 sqrt(n) as measured.  A chunk of U / (R - B) always fits, U / R never
// unless all divide; chunks between the two are tried where the batch is small (fit_chunk).  Whatever
// chunk is taken is at least U / R, or no sequence's n is above it, so there are at most R + B items, R split
// sequences and 2 R parts.
constexpr long long kMaxTiles = 1 << 26;  // of a sequence (2^30 positions)
__host__ __device__ __forceinline__ int least_chunk(long long U, int R) {
  const long long fits = (U + R - 1) / R, joins = (long long)(0.37f * sqrtf((float)U)), c = fits > joins ? fits : joins;
  return (int)(c < kMinTiles ? kMinTiles : c < kMaxTiles ? c : kMaxTiles);
}
__host__ __device__ __forceinline__ int safe_chunk(long long U, int B, int R) {
  const long long room = R - B > (R + 1) / 2 ? R - B : (R + 1) / 2, c = (U + room - 1) / room;
  const int least = least_chunk(U, R);
  return (int)(c < least ? least : c < kMaxTiles ? c : kMaxTiles);
}
// The least of the block's candidates between the two whose items fit (tiles: the B sequences'), if that
// saves more than joining further parts costs (about six tile times of a warp); all threads get it.  (A
// rounding here costs a wave, not correctness.)
template <int NW>
__device__ __forceinline__ int fit_chunk(const int* tiles, int B, int R, int lo, int hi, int* smem) {
  constexpr int kWorth = 6 * NW;
  if (hi - lo <= kWorth) return hi;
  const int c = lo + (int)((long long)(hi - lo) * threadIdx.x / (NW * 32 - 1));
  const uint32_t inv = (uint32_t)((0x100000000ull + c - 1) / c);
  int items = 0;
  for (int b = 0; b < B; ++b) items += (int)((uint64_t)(uint32_t)(tiles[b] + c - 1) * inv >> 32);
  int best = items <= R ? c : hi;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(kFull, best, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = best;
  __syncthreads();
  for (int w = 0; w < NW; ++w) best = min(best, smem[w]);
  return hi - best > kWorth ? best : hi;
}
// What a sequence adds to the running counts: items, and for one that is split its slots and itself
struct Counts {
  int items, slots, split;
};
__host__ __device__ __forceinline__ uint64_t pack_counts(int n, int chunk) {
  const uint32_t s = (n + chunk - 1) / chunk;
  return (uint64_t)s | (s > 1 ? ((uint64_t)s << 32) + (1ull << 48) : 0ull);
}
__host__ __device__ __forceinline__ Counts unpack_counts(uint64_t x) {
  return Counts{(int)(uint32_t)x, (int)((x >> 32) & 0xffff), (int)(x >> 48)};
}
// Sum of v over the block, and over the threads before this one (the warps' sums in `smem`, a word each)
template <int NW, typename T>
__device__ __forceinline__ T block_scan(T v, T* smem, T* before) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) smem[warp] = x;
  __syncthreads();
  T all = 0;
  *before = x - v;
  for (int w = 0; w < NW; ++w) {
    if (w < warp) *before += smem[w];
    all += smem[w];
  }
  return all;
}

// Lays out the items of a large batch, whose lengths every CTA would otherwise read and scan: one CTA.
static __global__ void __launch_bounds__(1024) k_decode_plan(const DecodeArgs a) {
  __shared__ uint64_t s_scan[32];
  after_last();
  const int B = a.c.B;
  uint64_t U = 0, before;
  for (int c0 = 0; c0 < B; c0 += 1024) {
    const int b = c0 + threadIdx.x;
    U += block_scan<32, uint64_t>(b < B ? tiles_of(seq_keys(a, b)) : 0, s_scan, &before);
  }
  const int chunk = safe_chunk((long long)U, B, a.R);
  uint64_t base = 0;
  for (int c0 = 0; c0 < B; c0 += 1024) {
    const int b = c0 + threadIdx.x;
    const uint64_t v = b < B ? pack_counts(tiles_of(seq_keys(a, b)), chunk) : 0;
    const uint64_t all = block_scan<32, uint64_t>(v, s_scan, &before);
    const Counts at = unpack_counts(base + before), own = unpack_counts(v);
    for (int i = 0; i < own.items; ++i) a.items[at.items + i] = make_int4(b, own.items, i, at.slots + i);
    if (own.split) a.jobs[at.split] = make_int4(b, at.slots, own.items, 0);
    base += all;
  }
  const Counts total = unpack_counts(base);
  for (int i = total.items + threadIdx.x; i < a.nitems; i += 1024) a.items[i] = make_int4(-1, 0, 0, 0);
  for (int i = total.split + threadIdx.x; i < a.njobs; i += 1024) a.jobs[i] = make_int4(-1, 0, 0, 0);
}

__device__ __forceinline__ void sts_u32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// (out of line: it is rarely entered)
static __device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = fab::globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (bar_try(bar, parity)) return true;
    if ((it & 255u) == 0 && fab::globaltimer_ns() - t0 > limit_ns) return false;
  }
}

// A box of rows of one KV head by TMA: x (elements, a multiple of 16 bytes) is where the head's rows start
// in a cell, y the first row of the pool.
__device__ __forceinline__ void tile_rows(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// An untiled bulk copy of a cache row and the bytes up to the 16-byte boundaries around it: those lie
// in the same page, whose size is a multiple of 16 bytes.
__device__ __forceinline__ void bulk_row(uint32_t dst, const uint8_t* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// A tile's rows one by one: key `lane` & 15 is row `row` of the pool (-1: none), `first` the head's row of
// cell 0 (out of line: only caches whose tiles are not boxes of a tensor map come here).
static __device__ __noinline__ void fetch_rows(uint32_t sl, int kv, uint32_t dst, int pitch, const uint8_t* first, int row,
                                               long long cell, int rb, uint32_t zero) {
  const int lane = threadIdx.x & 31;
  const uint32_t bar = sl + 128 + 8 * kv, ok = __ballot_sync(kFull, row >= 0) & 0xffffu, nb = copy_bytes(rb);
  if (lane == 0) {
    if (kv == 0) sts_u32(sl + 144, ok);
    bar_expect(bar, __popc(ok) * nb);
  }
  __syncwarp();
  if (lane < 16) {
    const uint8_t* src = first + max(row, 0) * cell;
    const uint32_t in = (uint32_t)reinterpret_cast<uintptr_t>(src) & 15;
    sts_u32(sl + 64 * kv + 4 * lane, kv && row < 0 ? zero : dst + lane * pitch + in);
    if (row >= 0) bulk_row(dst + lane * pitch, src - in, nb, bar);
  }
}

// Soft cap and distance bias of a lane's four scores (keys at distances d, d + 1, d + 8, d + 9; out of line)
static __device__ __noinline__ float4 cap_and_bias(float4 x, float cap, float slope, int d) {
  if (cap > 0.f) {
    const float inv = fminf(1.f / cap, 3.4028234e38f);  // (a denormal cap: not infinity, which 0 times is NaN)
    x = make_float4(cap * tanhf(x.x * inv), cap * tanhf(x.y * inv), cap * tanhf(x.z * inv), cap * tanhf(x.w * inv));
  }
  return make_float4(fmaf(slope, (float)d, x.x), fmaf(slope, (float)(d + 1), x.y), fmaf(slope, (float)(d + 8), x.z),
                     fmaf(slope, (float)(d + 9), x.w));
}

// One item (blockIdx.x / HG): a sequence, or a part of a long one, for one (KV head, chunk of eight query
// heads) (blockIdx.x % HG).  Consecutive CTAs take the same keys of the different heads, so a page's
// neighbouring rows are read at the same time.  Each warp takes every NW-th tile of 16 keys with a ring, a
// running maximum and sums of its own: no barrier until the item's last tile.
template <int D, int DV, int KT, int VT>
__global__ void __launch_bounds__(kWarps * 32, decode_shape(D, DV, KT, VT).ctas)
    k_decode(const DecodeArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  constexpr DecodeShape C = decode_shape(D, DV, KT, VT);
  constexpr int NW = kWarps, SLOTS = C.slots, PK = C.pk, PV = C.pv;
  constexpr float kLift = weight_lift(VT);
  constexpr int RBK = cache_row_bytes(KT, D), RBV = cache_row_bytes(VT, DV);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_scan[NW];
  __shared__ int4 s_item;
  __shared__ int s_tiles[kPlanBatch];
  __shared__ float s_qs[8], s_ml[NW][16];
  // a slot: where its 16 key rows and its 16 value rows start, the barriers of either, the tile's key mask
  struct Slot {
    uint32_t rows[2][16];
    uint64_t bar[2];
    uint32_t valid, pad[3];
  };
  static_assert(sizeof(Slot) == kSlotCtl && SLOTS >= 1, "shared memory plan");
  __shared__ __align__(16) Slot s_slot[NW][SLOTS];
  __shared__ __align__(16) uint32_t s_zero[DV + 4];  // the value row of a key that is not there
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int hg = blockIdx.x % a.HG, r = blockIdx.x / a.HG, hk = hg / a.chunks;
  const int head0 = hk * a.G + (hg - hk * a.chunks) * 8, nh = min(8, a.G - (hg - hk * a.chunks) * 8);
  const int B = a.c.B;
  const uint32_t qf = smem_u32(smem), ring = qf + C.qf + warp * C.ring, ctl = smem_u32(&s_slot[warp][0]);
  constexpr int kSums = C.ring / 4;  // floats from one warp's sums (in its ring) to the next's
  float* acc = reinterpret_cast<float*>(smem + C.qf);
  const int shift_k = hk * RBK & 15, shift_v = hk * RBV & 15;
  if (lane < 2 * SLOTS) fab::mbar_init(&s_slot[warp][lane >> 1].bar[lane & 1], 1);
  for (int i = threadIdx.x; i < DV + 4; i += NW * 32) s_zero[i] = 0;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {  // the rows of a whole tile
    const int kv = lane >> 4, r16 = lane & 15;
    s_slot[warp][i].rows[kv][r16] = ring + i * C.stage + (kv ? 16 * PK + shift_v + r16 * PV : shift_k + r16 * PK);
    if (lane == 0) s_slot[warp][i].valid = 0xffffu;
  }
  fab::fence_mbar_init();  // ordered before the first copy by the barriers below
  after_last();

  // ---- the item: {sequence, its splits, this split, slot}
  if (a.items) {
    if (threadIdx.x == 0) s_item = a.items[r];
  } else {  // from the lengths
    if (threadIdx.x == 0) s_item = make_int4(-1, 0, 0, 0);
    uint64_t U = 0, base = 0, before;
    int n_own = 0;
    for (int c0 = 0; c0 < B; c0 += NW * 32) {
      const int b = c0 + threadIdx.x;
      n_own = b < B ? tiles_of(seq_keys(a, b)) : 0;
      if (b < B) s_tiles[b] = n_own;
      U += block_scan<NW, uint64_t>(n_own, s_scan, &before);
    }
    const int chunk = fit_chunk<NW>(s_tiles, B, a.R, least_chunk((long long)U, a.R), safe_chunk((long long)U, B, a.R),
                                    reinterpret_cast<int*>(s_scan));
    const bool lists = r == 0 && hg == 0;  // this CTA lists the split sequences
    for (int c0 = 0; c0 < B; c0 += NW * 32) {
      const int b = c0 + threadIdx.x;
      if (B > NW * 32) n_own = b < B ? s_tiles[b] : 0;
      const uint64_t v = pack_counts(n_own, chunk), all = block_scan<NW, uint64_t>(v, s_scan, &before);
      const Counts at = unpack_counts(base + before), own = unpack_counts(v);
      if (at.items <= r && r < at.items + own.items) s_item = make_int4(b, own.items, r - at.items, at.slots + r - at.items);
      if (lists && own.split) a.jobs[at.split] = make_int4(b, at.slots, own.items, 0);
      base += all;
      if (!lists && unpack_counts(base).items > r) break;
    }
    if (lists)
      for (int i = unpack_counts(base).split + threadIdx.x; i < a.njobs; i += NW * 32) a.jobs[i] = make_int4(-1, 0, 0, 0);
  }
  // sequences without keys: their rows, by the CTA whose turn it is
  for (int b = r + a.nitems * threadIdx.x; b < B; b += a.nitems * NW * 32) {
    const int L = a.lens[b];
    if (L > a.c.max_pages * a.c.page_size && hg == 0) report_page(a.c.err);
    if (L < 0 || seq_keys(a, b) > 0) continue;
    for (int h = head0; h < head0 + nh; ++h) {
      const long long at = (long long)b * a.H + h;
      for (int d = 0; d < DV; ++d) act_store(a.O, a.act, at * DV + d, 0.f);
      if (a.lse) a.lse[at] = a.sinks ? a.sinks[h] : -INFINITY;
    }
  }
  __syncthreads();
  const int4 item = s_item;
  if (item.x < 0) return;
  const int b = item.x, keys = seq_keys(a, b);
  const long long n_all = tiles_of(keys);
  const int j0 = 16 * (int)(n_all * item.z / item.y);  // the item's keys [j0, j1) and tiles
  const int j1 = min(keys, 16 * (int)(n_all * (item.z + 1) / item.y)), ntile = tiles_of(j1 - j0);
  const bool whole = item.y == 1;

  // ---- rows of a tile: key `lane` & 15 a lane.  Boxes of rows (16 or 8 in one page) go by the tensor maps,
  // else each row is copied by itself.  The first rows of the warp's next 32 boxes are looked up at once, a
  // box a lane; single rows a tile at a time.
  const int boxes = a.box == 8 ? 2 : 1, per_batch = 32 / boxes;  // boxes of a tile, tiles of a lookup
  auto lookup = [&](int j) {  // row of the pool of key j, -1 where there is none
    if (j >= j1) return -1;
    const int p = (int)((uint64_t)j * a.c.page_mul >> a.c.page_shift);
    const int page = a.c.table[(long long)b * a.c.max_pages + p];
    if (page >= 0 && page < a.c.num_pages) return page * a.c.page_size + (j - p * a.c.page_size);
    report_page(a.c.err);
    return -1;
  };
  int found = -1, found_at = -1000;  // the lookup's rows, and the warp's turn that it starts with
  auto row_of = [&](int turn) {  // of the warp's turn-th tile
    if (!a.box) return lookup(j0 + 16 * (warp + NW * turn) + (lane & 15));
    if (turn - found_at >= per_batch) {
      const int l = a.box == 8 ? lane >> 1 : lane;
      found = lookup(j0 + 16 * (warp + NW * (turn + l)) + (a.box == 8 ? 8 * (lane & 1) : 0));
      found_at = turn;
    }
    return __shfl_sync(kFull, found, (turn - found_at) * boxes + (a.box == 8 ? (lane >> 3) & 1 : 0));
  };
  // by slot (keys: bits 0 .. 3, values: 4 .. 7): parity awaited, copies under way, mask or places not the usual ones
  uint32_t phases = 0, armed = 0, patched = 0;
  auto fetch = [&](int kv, int slot, int row, int tile) {
    const uint32_t sl = ctl + slot * (uint32_t)sizeof(Slot), bar = sl + 128 + 8 * kv;
    const uint32_t dst = ring + slot * C.stage + (kv ? 16 * PK : 0);
    const int pitch = kv ? PV : PK;
    armed |= 1u << (4 * kv + slot);
    const int n = min(16, j1 - (j0 + tile * 16));  // the rows behind them are not used
    const CUtensorMap* map = kv ? &map_v : &map_k;
    const int x = kv ? (hk * RBV & ~15) >> map_es(PV) : (hk * RBK & ~15) >> map_es(PK);
    // A slot's mask and its value rows' places are rewritten for a tile with rows missing, and after one.
    const uint32_t bit = 1u << (4 * kv + slot);
    if (a.box == 16) {
      if (lane == 0) {
        bar_expect(bar, row >= 0 ? 16 * pitch : 0);
        if (row >= 0) tile_rows(dst, map, x, row, bar);
      }
      const bool part = n < 16 || row < 0;
      if (part || (patched & bit)) {
        patched = part ? patched | bit : patched & ~bit;
        if (kv == 0) {
          if (lane == 0) sts_u32(sl + 144, row >= 0 ? (1u << n) - 1 : 0);
        } else if (lane < 16) {
          sts_u32(sl + 64 + 4 * lane, lane < n && row >= 0 ? dst + lane * pitch + shift_v : smem_u32(s_zero));
        }
      }
      return;
    }
    if (a.box) {
      const uint32_t ok = __ballot_sync(kFull, (lane & 15) < n && row >= 0) & 0xffffu;
      if (lane == 0) bar_expect(bar, (((ok & 0xff) ? 1 : 0) + ((ok >> 8) ? 1 : 0)) * 8 * pitch);
      __syncwarp();
      if (lane == 0 ? ok & 0xff : lane == 8 && (ok >> 8)) tile_rows(dst + lane * pitch, map, x, row, bar);
      if (ok != 0xffffu || (patched & bit)) {
        patched = ok != 0xffffu ? patched | bit : patched & ~bit;
        if (kv == 0) {
          if (lane == 0) sts_u32(sl + 144, ok);
        } else if (lane < 16) {
          sts_u32(sl + 64 + 4 * lane, ok >> lane & 1 ? dst + lane * pitch + shift_v : smem_u32(s_zero));
        }
      }
      return;
    }
    const uint8_t* pool = kv ? a.c.v : a.c.k;
    const int rb = kv ? RBV : RBK;
    fetch_rows(sl, kv, dst, pitch, pool + (long long)hk * rb, row, (long long)a.c.Hkv * rb, rb, smem_u32(s_zero));
  };
  // the slot's copies have arrived (all lanes agree)
  auto arrived = [&](int kv, int slot) {
    const uint32_t bit = 1u << (4 * kv + slot), bar = ctl + slot * (uint32_t)sizeof(Slot) + 128 + 8 * kv;
    const uint32_t parity = (phases & bit) != 0;
    bool came = a.wait_ns > 0 && bar_try(bar, parity);
    if (!__all_sync(kFull, came)) {
      came = a.wait_ns > 0 && bar_wait_slow(bar, parity, a.wait_ns);
      if (!__all_sync(kFull, came)) return false;
    }
    phases ^= bit, armed &= ~bit;
    return true;
  };
  int slot = 0;
  auto prefetch = [&] {
    for (int i = 0, sl = slot; i < SLOTS; ++i) {
      const int tile = warp + i * NW;
      if (tile < ntile) {
        const int row = row_of(i);
        fetch(0, sl, row, tile), fetch(1, sl, row, tile);
      }
      if (++sl == SLOTS) sl = 0;
    }
  };
  // q of the chunk's heads, a head a warp: scaled by a power of two into range, split into parts
  auto load_q = [&] {
    for (int h = warp; h < 8; h += NW) {
      const long long at = b * a.q_row + (head0 + h) * a.q_head;
      float m = 0.f;
      if (h < nh)
        for (int d = lane; d < D; d += 32) m = fmaxf(m, fabsf(act_load(a.q, a.act, at + d)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      // the largest magnitude goes to 2^8 (binary16 parts), or with f32 keys into 2^-80 .. 2^60 (whose tf32
      // parts are not denormal, and whose products with keys have room)
      const int e = m > 0.f && m < INFINITY ? ilogbf(m) : 8;
      const int up = KT == FA_F32 ? min(max(e, -80), 60) - e : min(8 - e, 126);
      const float qs = ldexpf(1.f, up);
      if (lane == 0) s_qs[h] = qs;
      constexpr int steps = KT == FA_F32 ? D / 8 : D / 16;
      for (int ks = g; ks < steps; ks += 8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (KT == FA_F32) {
            split_tf32(__float_as_uint(h < nh ? act_load(a.q, a.act, at + ks * 8 + t + 4 * i) * qs : 0.f), w[i], w[2 + i]);
          } else {
            const float x = h < nh ? act_load(a.q, a.act, at + k_comp16(KT, ks, t, i, 0)) * qs : 0.f;
            const float y = h < nh ? act_load(a.q, a.act, at + k_comp16(KT, ks, t, i, 1)) * qs : 0.f;
            w[i] = pack_h2(x, y);
            w[2 + i] = pack_h2(x - lo_h(w[i]), y - hi_h(w[i]));
          }
        }
        fab::sts_v4(qf + ks * 512 + (h * 4 + t) * 16, w[0], w[1], w[2], w[3]);
      }
    }
  };

  prefetch();
  load_q();
  __syncthreads();
  bool dead = false;  // a wait ran out: no more work is issued
  {
    // ---- the warp's tiles
    const float qscale = a.scale / s_qs[g];
    const float slope = a.alibi && g < nh ? a.alibi[head0 + g] : 0.f;
    const bool ext = a.softcap > 0.f || a.alibi;
    float o[DV / 16][4];
#pragma unroll
    for (int n = 0; n < DV / 16; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
    float m = -INFINITY, l = 0.f;  // head g: the maximum that weights refer to (log2), this lane's sum
    int next = warp + SLOTS * NW, turn = SLOTS;
    for (int tile = warp; tile < ntile; tile += NW, next += NW, ++turn) {
      const int row = next < ntile ? row_of(turn) : -1;
      const uint32_t sl = ctl + slot * (uint32_t)sizeof(Slot), qa = qf + lane * 16;
      dead = !arrived(0, slot);
      if (dead) break;
      float s[4] = {};
      if (KT == FA_Q8_0) scores_q8<D>(s, sl, qa, lane);
      else if (KT == FA_F16) scores_f16<D>(s, sl, qa, lane);
      else if (KT == FA_Q4_0) scores_q4<D>(s, sl, qa, lane);
      else scores_f32<D>(s, sl, qa, lane);
      transpose_scores(s);
      const uint32_t ok = lds_u32(sl + 144);
      __syncwarp();
      if (next < ntile) fetch(0, slot, row, next);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] *= qscale;
      if (ext) {
        const float4 x = cap_and_bias(make_float4(s[0], s[1], s[2], s[3]), a.softcap, slope,
                                      j0 + tile * 16 + 2 * t - (keys - 1));
        s[0] = x.x, s[1] = x.y, s[2] = x.z, s[3] = x.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] *= kLog2e;
      if (ok != 0xffffu) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!((ok >> (2 * t + (i & 1) + 8 * (i >> 1))) & 1)) s[i] = -INFINITY;
      }
      float mx = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
      const bool first = m == -INFINITY, move = first ? mx > m : mx > m + kRescale;
      if (__any_sync(kFull, move)) {
        const float f = move && !first ? fab::ex2(m - mx) : 1.f;  // (nothing has been summed up to the first)
        if (move) m = mx;
        if (__any_sync(kFull, f != 1.f)) {
          l *= f;
          const float f0 = __shfl_sync(kFull, f, 8 * t), f1 = __shfl_sync(kFull, f, 8 * t + 4);
#pragma unroll
          for (int n = 0; n < DV / 16; ++n) o[n][0] *= f0, o[n][1] *= f1, o[n][2] *= f0, o[n][3] *= f1;
        }
      }
      const float ref = m == -INFINITY ? 0.f : m - kLift;
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = fab::ex2(s[i] - ref);
      l += (p[0] + p[1]) + (p[2] + p[3]);
      dead = !arrived(1, slot);
      if (dead) break;
      if (VT == FA_Q8_0 && a.act == FA_ACT_F32) values_q8<DV, 3>(o, p, sl + 64, lane);
      else if (VT == FA_Q8_0) values_q8<DV, 2>(o, p, sl + 64, lane);
      else if (VT == FA_F16) values_f16<DV>(o, p, sl + 64, lane);
      else if (VT == FA_Q4_0 && a.act == FA_ACT_F32) values_q4<DV, 3>(o, p, sl + 64, lane);
      else if (VT == FA_Q4_0) values_q4<DV, 2>(o, p, sl + 64, lane);
      else values_f32<DV>(o, p, sl + 64, lane);
      __syncwarp();
      if (next < ntile) fetch(1, slot, row, next);
      if (++slot == SLOTS) slot = 0;
    }
    if (dead) {  // let the copies in flight land: nothing more is issued
      if (lane == 0) {
        atomicExch(a.c.err, FA_ERR_TIMEOUT);
        for (int i = 0; i < 8; ++i)
          if ((armed >> i) & 1) bar_wait_slow(ctl + (i & 3) * (uint32_t)sizeof(Slot) + 128 + 8 * (i >> 2), (phases >> i) & 1, kDrainNs);
      }
      __syncwarp();
    }
    lets_next();  // (the join, whose CTAs are large: not before the tiles are done)
    // ---- the warps' sums (in their rings), joined in the warps' order
    l += __shfl_xor_sync(kFull, l, 1);
    l += __shfl_xor_sync(kFull, l, 2);
    if (t == 0) s_ml[warp][g] = m, s_ml[warp][8 + g] = l;
#pragma unroll
    for (int n = 0; n < DV / 16; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[warp * kSums + (n * 4 + i) * 32 + lane] = o[n][i];
    __syncthreads();
    float M[2] = {-INFINITY, -INFINITY}, S[2] = {0.f, 0.f}, fw[2][NW];  // heads 2t, 2t + 1
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int w = 0; w < NW; ++w) M[i] = fmaxf(M[i], s_ml[w][2 * t + i]);
      const float ref = M[i] == -INFINITY ? 0.f : M[i];
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        fw[i][w] = fab::ex2(s_ml[w][2 * t + i] - ref);
        S[i] = fmaf(s_ml[w][8 + 2 * t + i], fw[i][w], S[i]);
      }
    }
    float* part = a.part + ((long long)item.w * a.HG + hg) * (8 * DV + 16);  // (a split sequence's)
    float fin[2], lse[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float total = S[i], top = M[i], f = 1.f;
      if (whole && a.sinks && 2 * t + i < nh) {  // one more term of the sum, without a value
        const float sk = a.sinks[head0 + 2 * t + i] * kLog2e;
        top = fmaxf(M[i], sk);
        if (top > -INFINITY) {
          f = exp2f(M[i] - top);
          total = S[i] * f + exp2f(sk - top + kLift);
        }
      }
      fin[i] = whole ? (total == 0.f ? 0.f : f / total) : 1.f;
      lse[i] = total == 0.f ? -INFINITY : (top - kLift + log2f(total)) * kLn2;
    }
    for (int n = warp; n < DV / 16; n += NW) {
      float x[4] = {};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float* p = acc + w * kSums + n * 128 + lane;
        x[0] = fmaf(p[0], fw[0][w], x[0]), x[1] = fmaf(p[32], fw[1][w], x[1]);
        x[2] = fmaf(p[64], fw[0][w], x[2]), x[3] = fmaf(p[96], fw[1][w], x[3]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = 2 * t + (i & 1), d = v_comp(VT, n, g, i >> 1);
        if (h < nh) {
          if (whole) act_store(a.O, a.act, ((long long)b * a.H + head0 + h) * DV + d, x[i] * fin[i & 1]);
          else part[h * DV + d] = x[i];
        }
      }
    }
    if (warp == 0 && g == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = 2 * t + i;
        if (h < nh && whole && a.lse) a.lse[(long long)b * a.H + head0 + h] = lse[i];
        if (!whole) part[8 * DV + h] = M[i], part[8 * DV + 8 + h] = S[i];
      }
    }
  }
}

// Joins the parts of a split sequence (blockIdx.x), in their order, for a query head (blockIdx.y).  The grid
// starts while the items' last CTAs run.  Each group of threads takes every GR-th part with a running
// maximum, then the groups are joined: bound by the latency of a launch and two rounds of loads (75520 keys:
// about 114 parts of 24 heads, 2.8 MB, read from L2).
template <int DV>
__global__ void __launch_bounds__(512) k_decode_join(const DecodeArgs a) {
  constexpr int LN = DV / 4, GR = 512 / LN;  // threads of a row (four components each), rows read at a time
  __shared__ float s_m[GR], s_l[GR];
  __shared__ float4 s_x[512];
  const int h = blockIdx.y, hk = h / a.G, hc = (h - hk * a.G) >> 3, hg = hk * a.chunks + hc, c = (h - hk * a.G) & 7;
  const int tid = threadIdx.x, ln = tid % LN, gr = tid / LN;
  after_last();
  const int4 job = a.jobs[blockIdx.x];
  if (job.x < 0) return;
  const int np = job.z;
  float M = -INFINITY, S = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int Q = 4;  // parts under way at a time
  for (int i0 = gr; i0 < np; i0 += Q * GR) {
    float m[Q], l[Q];
    float4 v[Q];
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      const int i = i0 + k * GR;
      m[k] = -INFINITY, l[k] = 0.f, v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < np) {
        const float* p = a.part + ((long long)(job.y + i) * a.HG + hg) * (8 * DV + 16);
        m[k] = p[8 * DV + c], l[k] = p[8 * DV + 8 + c], v[k] = *reinterpret_cast<const float4*>(p + c * DV + 4 * ln);
      }
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < Q; ++k) top = fmaxf(top, m[k]);
    const float ref = top == -INFINITY ? 0.f : top, f0 = fab::ex2(M - ref);
    M = top, S *= f0;
    x.x *= f0, x.y *= f0, x.z *= f0, x.w *= f0;
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      const float f = fab::ex2(m[k] - ref);
      S = fmaf(l[k], f, S);
      x.x = fmaf(v[k].x, f, x.x), x.y = fmaf(v[k].y, f, x.y), x.z = fmaf(v[k].z, f, x.z), x.w = fmaf(v[k].w, f, x.w);
    }
  }
  if (ln == 0) s_m[gr] = M, s_l[gr] = S;
  s_x[tid] = x;
  __syncthreads();
  if (gr > 0) return;
  const float sk = a.sinks ? a.sinks[h] * kLog2e : -INFINITY;
  float top = sk;
#pragma unroll
  for (int i = 0; i < GR; ++i) top = fmaxf(top, s_m[i]);
  const float ref = top == -INFINITY ? 0.f : top;
  S = 0.f, x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < GR; ++i) {
    const float f = fab::ex2(s_m[i] - ref);
    const float4 v = s_x[i * LN + ln];
    S = fmaf(s_l[i], f, S);
    x.x = fmaf(v.x, f, x.x), x.y = fmaf(v.y, f, x.y), x.z = fmaf(v.z, f, x.z), x.w = fmaf(v.w, f, x.w);
  }
  if (a.sinks) S += fab::ex2(sk - ref + a.lift);
  const float inv = S == 0.f ? 0.f : 1.f / S;
  const long long at = ((long long)job.x * a.H + h) * DV + 4 * ln;
  act_store(a.O, a.act, at, x.x * inv), act_store(a.O, a.act, at + 1, x.y * inv);
  act_store(a.O, a.act, at + 2, x.z * inv), act_store(a.O, a.act, at + 3, x.w * inv);
  if (tid == 0 && a.lse) a.lse[(long long)job.x * a.H + h] = S == 0.f ? -INFINITY : (ref - a.lift + log2f(S)) * kLn2;
}

typedef cudaError_t (*DecodeFn)(DecodeArgs a, const DecodeMaps& m, cudaStream_t s);

template <int D, int DV, int KT, int VT>
cudaError_t run_decode(DecodeArgs a, const DecodeMaps& m, cudaStream_t s) {
  constexpr DecodeShape C = decode_shape(D, DV, KT, VT);
  a.lift = weight_lift(VT);
  static std::atomic<uint64_t> ready{0};  // devices that the kernel's shared memory has been allowed on
  cudaError_t e = cudaSuccess;
  if (!allow_smem(reinterpret_cast<const void*>(k_decode<D, DV, KT, VT>), C.smem, &ready)) return cudaErrorInvalidValue;
  if (a.items && (e = launch_next(k_decode_plan, dim3(1), dim3(1024), 0, s, a)) != cudaSuccess) return e;
  e = launch_next(k_decode<D, DV, KT, VT>, dim3((unsigned)(a.nitems * a.HG)), dim3(kWarps * 32), C.smem, s, a, m.k, m.v);
  if (e != cudaSuccess) return e;
  if (a.njobs > 0) return launch_next(k_decode_join<DV>, dim3(a.njobs, a.H), dim3(512), 0, s, a);
  return cudaSuccess;
}
template <int D, int DV, int KT>
DecodeFn pick_decode_v(int vt) {
  switch (vt) {
    case FA_F32: return run_decode<D, DV, KT, FA_F32>;
    case FA_F16: return run_decode<D, DV, KT, FA_F16>;
    case FA_Q8_0: return run_decode<D, DV, KT, FA_Q8_0>;
  }
  return run_decode<D, DV, KT, FA_Q4_0>;
}
// The kernel for D and the key type KT; a translation unit each, so that they compile in parallel.
template <int D, int KT>
DecodeFn pick_decode(int Dv, int vt);
template <> DecodeFn pick_decode<64, FA_F32>(int, int);
template <> DecodeFn pick_decode<64, FA_F16>(int, int);
template <> DecodeFn pick_decode<64, FA_Q8_0>(int, int);
template <> DecodeFn pick_decode<64, FA_Q4_0>(int, int);
template <> DecodeFn pick_decode<128, FA_F32>(int, int);
template <> DecodeFn pick_decode<128, FA_F16>(int, int);
template <> DecodeFn pick_decode<128, FA_Q8_0>(int, int);
template <> DecodeFn pick_decode<128, FA_Q4_0>(int, int);
template <> DecodeFn pick_decode<256, FA_F32>(int, int);
template <> DecodeFn pick_decode<256, FA_F16>(int, int);
template <> DecodeFn pick_decode<256, FA_Q8_0>(int, int);
template <> DecodeFn pick_decode<256, FA_Q4_0>(int, int);
#define FAP_INSTANTIATE_DECODE(D, KT)                              \
  template <>                                                      \
  DecodeFn pick_decode<D, KT>(int Dv, int vt) {                    \
    return Dv == 64    ? pick_decode_v<D, 64, KT>(vt)              \
           : Dv == 128 ? pick_decode_v<D, 128, KT>(vt)             \
                       : pick_decode_v<D, 256, KT>(vt);            \
  }

}  // namespace fap
