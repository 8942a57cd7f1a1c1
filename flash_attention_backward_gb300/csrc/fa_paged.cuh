// Device code shared by the paged-cache and the norm / rotation kernels: activation types, the
// rotation of a head, page lookup and the host-side checks of a paged cache.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/fa_paged_ext.h"
#include "fa_internal.h"

namespace fap {

constexpr unsigned kFull = 0xffffffffu;

// ------------------------------------------------------------------------------------------------
// activations: eight consecutive elements of a row as f32.  One lane owns eight elements (16 bytes
// of a 16-bit type, 32 of f32), so a head of D is held by D / 8 neighbouring lanes.

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename T>
struct alignas(16) Oct {
  T v[8];
};

// vec: p is 16-byte aligned (warp-uniform); otherwise element by element
template <typename T>
__device__ __forceinline__ void load8_raw(const T* p, bool vec, Oct<T>& o) {
  if (vec) {
    constexpr int n = sizeof(Oct<T>) / 16;
#pragma unroll
    for (int i = 0; i < n; ++i) reinterpret_cast<uint4*>(&o)[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = p[i];
  }
}
// (out of line, so that the 16-byte path is not left with eight predicated loads)
template <typename T>
__device__ __noinline__ Oct<T> load8_any(const T* p) {
  Oct<T> o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o.v[i] = p[i];
  return o;
}
template <typename T>
__device__ __forceinline__ void unpack8(const Oct<T>& o, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = to_f32(o.v[i]);
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, bool vec, float (&x)[8]) {
  Oct<T> o;
  load8_raw(p, vec, o);
  unpack8(o, x);
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  Oct<T> o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o.v[i] = from_f32<T>(x[i]);
  constexpr int n = sizeof(Oct<T>) / 16;
#pragma unroll
  for (int i = 0; i < n; ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(&o)[i];
}

// ------------------------------------------------------------------------------------------------
// rotation

struct Rope {
  const uint64_t* freqs;
  int n_rot, style;
  const int32_t* pos;   // [n_axes][tokens], an axis every `stride`
  const uint8_t* axis;  // [n_rot / 2], or NULL: one axis
  long long stride;
  int n_axes;
};

// A warp's lanes share out a token's D / 2 pairs, D / 64 neighbouring ones each: the positions of a lane's pairs.
// With several axes a lane looks its pairs' axes up once, a byte each, and of a token lane a loads axis a's position
// and hands it round.  (In kernels of their own: with both in one the plain rotation of 2048 tokens of 28 heads of 256,
// f32, took 25.7 us for 21.2.)
template <int D, bool AXES>
struct PairPos {
  static constexpr int P = D / 64;
  uint32_t axes = 0;

  __device__ __forceinline__ void look_up(const Rope& r) {
#pragma unroll
    for (int i = 0; AXES && i < P; ++i) {
      const int pair = (int)(threadIdx.x & 31) * P + i;
      if (pair < r.n_rot >> 1) axes |= (uint32_t)min((int)r.axis[pair], r.n_axes - 1) << (8 * i);
    }
  }
  // Of token n: what this lane loads...
  __device__ __forceinline__ int load(const Rope& r, long long n) const {
    if (!AXES) return r.pos[n];
    const int lane = threadIdx.x & 31;
    return lane < r.n_axes ? r.pos[lane * r.stride + n] : 0;
  }
  // ...and what its pairs get (all lanes of the warp take part)
  __device__ __forceinline__ void hand_round(int mine, int (&pos)[P]) const {
#pragma unroll
    for (int i = 0; i < P; ++i) pos[i] = AXES ? __shfl_sync(kFull, mine, axes >> (8 * i) & 255) : mine;
  }
};

// sin and cos of pos * freq, modulo 2^64 in units of 2^-64 turns: the wrap of the integer product is the
// reduction modulo one turn, with no rounding.  Of the 32 bits that are kept (1.5e-9 rad) f32 holds 24: the
// others, below 4e-7 rad, are added to first order, so that what is left is the error of sincospif, of one
// rounding and those 1.5e-9 rad, at every position.  (All 32 at once in f32 would be up to 9.4e-8 rad off.)
__device__ __forceinline__ void sin_cos_turn(uint64_t freq, int pos, float* sn, float* cs) {
  const int a = (int)(((uint64_t)(int64_t)pos * freq) >> 32);
  float s, c;
  sincospif((float)(a & ~0xff) * 0x1p-31f, &s, &c);
  const float rest = (float)(a & 0xff) * (float)(3.14159265358979323846 * 0x1p-31);
  *sn = fmaf(c, rest, s), *cs = fmaf(-s, rest, c);
}

// A warp that holds heads of one token: D / 8 lanes a head, so 256 / D heads side by side.  Factors of a
// lane's eight elements e0 .. e0+7: y[i] = x[i] c[i] + partner[i] s[i], the sign of the pair's first /
// second member in s, for its first n elements; the others are not rotated and not touched (turned by nothing,
// an infinity would become NaN and a NaN would enter its partner).  The token's n_rot / 2 <= D / 2 angles
// are shared out over the lanes, D / 64 neighbouring ones each, and handed round by shuffles.
template <int D>
struct Turn8 {
  float c[8], s[8];
  int src;  // partner lane (FA_ROPE_HALVES)
  int n;    // the lane's elements that are rotated, its first ones (FA_ROPE_HALVES: all or none)

  // All lanes of the warp take part; pos: of the lane's pairs (PairPos).
  __device__ __forceinline__ void set(const Rope& r, const int (&pos)[D / 64], int e0) {
    constexpr int P = D / 64;
    const int lane = threadIdx.x & 31, half = r.n_rot >> 1;
    src = lane;
    n = min(max(r.n_rot - e0, 0), 8);
    if (half == 0) return;
    float cs[P], sn[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      cs[i] = 1.f, sn[i] = 0.f;
      const int p = lane * P + i;
      if (p < half) sin_cos_turn(r.freqs[p], pos[i], &sn[i], &cs[i]);
    }
    const bool in = e0 < r.n_rot;
    if (r.style == FA_ROPE_HALVES) {  // n_rot % 16 == 0: a lane lies in one half
      const bool second = e0 >= half;
      const int p0 = !in ? 0 : second ? e0 - half : e0;
      if (in) src = lane + (second ? -(half >> 3) : half >> 3);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float ci = __shfl_sync(kFull, cs[i % P], (p0 + i) / P), si = __shfl_sync(kFull, sn[i % P], (p0 + i) / P);
        c[i] = ci;
        s[i] = second ? si : -si;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = (e0 >> 1) + i;
        const float ci = __shfl_sync(kFull, cs[i % P], p / P), si = __shfl_sync(kFull, sn[i % P], p / P);
        c[2 * i] = c[2 * i + 1] = ci;
        s[2 * i] = -si, s[2 * i + 1] = si;
      }
    }
  }
  // All lanes of the warp take part.
  __device__ __forceinline__ void apply(float (&x)[8], int style) const {
    float p[8];
    if (style == FA_ROPE_HALVES) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = __shfl_sync(kFull, x[i], src);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = x[i ^ 1];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < n ? fmaf(p[i], s[i], x[i] * c[i]) : x[i];
  }
};

// Sum over the LG lanes (a power of two) that hold one head.
template <int LG>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// A lane's four rotation pairs: components [ea, ea + 4) and [eb, eb + 4) of the head.
//   FA_ROPE_HALVES  pair i is (x[ea + i], x[eb + i]).  The rotated components are pairs 0 .. n_rot / 2 - 1
//                   (i, i + n_rot / 2); the others pair up likewise and are not turned (n_rot % 16 == 0:
//                   a lane's pairs are all of one kind).
//   FA_ROPE_PAIRS   eight neighbouring components, pair i is (x[ea + 2i], x[ea + 2i + 1]).
template <typename T>
struct alignas(4 * sizeof(T)) Four {
  T v[4];
};
template <typename T>
struct Eight {
  Four<T> a, b;
};

template <typename T, bool VEC>
__device__ __forceinline__ void load_eight(const T* p, int ea, int eb, Eight<T>& o) {
  if (VEC) {
    o.a = *reinterpret_cast<const Four<T>*>(p + ea);
    o.b = *reinterpret_cast<const Four<T>*>(p + eb);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) o.a.v[i] = p[ea + i], o.b.v[i] = p[eb + i];
  }
}
template <typename T>
__device__ __forceinline__ void unpack_eight(const Eight<T>& o, float2 (&x)[4]) {
  x[0] = make_float2(to_f32(o.a.v[0]), to_f32(o.a.v[1])), x[1] = make_float2(to_f32(o.a.v[2]), to_f32(o.a.v[3]));
  x[2] = make_float2(to_f32(o.b.v[0]), to_f32(o.b.v[1])), x[3] = make_float2(to_f32(o.b.v[2]), to_f32(o.b.v[3]));
}

// Where the lane's four pairs lie.  (The norm kernels say it again in their own words: with this in their place 16411 tokens
// of 10 heads of 64 took 18.3 us for 17.9.)
template <int D>
__device__ __forceinline__ void place_eight(int style, int n_rot, int& ea, int& eb) {
  const int p = (threadIdx.x & (D / 8 - 1)) * 4, half = n_rot >> 1;
  if (style == FA_ROPE_PAIRS) ea = 2 * p, eb = ea + 4;
  else if (p < half) ea = p, eb = p + half;
  else ea = n_rot + (p - half), eb = ea + (D - n_rot) / 2;
}
// Sum of squares of a head that D / 8 lanes hold so.  The order of the sum is part of the result: whoever
// normalises a head takes it from here, so that equal heads give equal bits.
template <int D>
__device__ __forceinline__ float square_sum(const float2 (&x)[4]) {
  float2 q = __fmul2_rn(x[0], x[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) q = __ffma2_rn(x[i], x[i], q);
  return group_sum<D / 8>(q.x + q.y);
}

// 1 / sqrt(v): the hardware approximation and one Newton step (it alone is off by up to two units,
// and the whole head is scaled by it)
__device__ __forceinline__ float inv_rms(float sum, float inv_n, float eps) {
  const float v = fmaf(sum, inv_n, eps);
  const float r = rsqrtf(v);
  const float h = fmaf(-v * r, r, 1.f);
  return (h == h) ? fmaf(0.5f * r, h, r) : r;  // v = 0 or inf: r is the limit itself
}

// ------------------------------------------------------------------------------------------------
// paged cache

struct Cache {
  uint8_t* k;
  uint8_t* v;
  const int32_t* table;
  int k_type, v_type, num_pages, page_size, B, max_pages, Hkv, D, Dv;
  int rbk, rbv;  // bytes of a row
  int* err;
  uint32_t page_mul;  // j / page_size = j * page_mul >> page_shift for 0 <= j < 2^30
  int page_shift;
};

// FA_ERR_PAGE, unless something is recorded already: outputs are defined after it, and not after a timeout.
__device__ __forceinline__ void report_page(int* err) { atomicCAS(err, FA_OK, FA_ERR_PAGE); }

// Row (page * page_size + offset) of position j of sequence b, or -1 (and FA_ERR_PAGE recorded)
__device__ __forceinline__ long long cache_row(const Cache& c, int b, int j) {
  if (b < c.B && j < c.max_pages * c.page_size) {
    const int p = (int)((uint64_t)j * c.page_mul >> c.page_shift);
    const int page = c.table[(long long)b * c.max_pages + p];
    if (page >= 0 && page < c.num_pages) return (long long)page * c.page_size + (j - p * c.page_size);
  }
  report_page(c.err);
  return -1;
}

// ---- launches that overlap.  A kernel launched by launch_next() may start while the one before it on the
// stream still runs its last CTAs; it begins with after_last(), which waits for all of that one's work.
// lets_next() says that the next one's CTAs may take what is free from here on.  (Without such a launch
// before or behind them both do nothing.)  What that one writes (lengths, positions, page tables) is not
// read-only while this kernel runs: it is read by ordinary loads, which after_last() orders, and not by the
// non-coherent ones of __ldg and const __restrict__.
__device__ __forceinline__ void after_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void lets_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---- clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// (arrive releases and wait acquires at cluster scope)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_barrier() { cluster_arrive(), cluster_wait(); }

// ---- host
template <typename... P, typename... A>
inline cudaError_t launch_next(void (*k)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid, cfg.blockDim = block, cfg.dynamicSmemBytes = smem, cfg.stream = s, cfg.attrs = &early, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, static_cast<P>(args)...);
}
// The same for clusters of `cluster` CTAs
template <typename... P, typename... A>
inline cudaError_t launch_clusters(void (*k)(P...), unsigned grid, unsigned cluster, unsigned block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster, at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid), cfg.blockDim = dim3(block), cfg.dynamicSmemBytes = smem, cfg.stream = s, cfg.attrs = at, cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, static_cast<P>(args)...);
}
// Allows a kernel's dynamic shared memory on the current device, once for each (ready: the devices so far).
inline bool allow_smem(const void* k, int bytes, std::atomic<uint64_t>* ready) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev < 64 && (ready->load() >> dev & 1)) return true;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  if (dev < 64) ready->fetch_or(1ull << dev);
  return true;
}
// j / page_size = j * mul >> shift for 0 <= j < 2^30
inline void page_divisor(int page_size, uint32_t* mul, int* shift) {
  int lg = 0;
  while ((1LL << lg) < page_size) ++lg;
  *mul = (uint32_t)(((1ULL << (30 + lg)) + page_size - 1) / page_size), *shift = 30 + lg;
}
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool head_size(int d) { return d == 64 || d == 128 || d == 256; }
inline int act_bytes(int t) { return t == FA_ACT_F32 ? 4 : 2; }
inline bool act_type(int t) { return t >= FA_ACT_F32 && t <= FA_ACT_BF16; }

// The argument checks of a paged cache, and its device form but for `err`.
fa_status check_cache(const fa_paged_cache* c, Cache* out);
// The checks of a rotation by pos; axes: of several axes (r is not looked at then).
fa_status check_rope(const fa_rope* r, const fa_rope_axes* axes, int D, const int32_t* pos, int N, Rope* out);

}  // namespace fap
