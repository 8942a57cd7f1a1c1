// Device code shared by the paged-cache and the norm / rotation kernels: activation types, the
// rotation of a head, page lookup and the host-side checks of a paged cache.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/fa_paged.h"
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

  // All lanes of the warp take part; pos is the same in all.
  __device__ __forceinline__ void set(const Rope& r, int pos, int e0) {
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
      if (p < half) sin_cos_turn(r.freqs[p], pos, &sn[i], &cs[i]);
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
// Allows a kernel's dynamic shared memory on the current device, once for each (ready: the devices so far).
inline bool allow_smem(const void* k, int bytes, std::atomic<uint64_t>* ready) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev < 64 && (ready->load() >> dev & 1)) return true;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  if (dev < 64) ready->fetch_or(1ull << dev);
  return true;
}
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool head_size(int d) { return d == 64 || d == 128 || d == 256; }
inline int act_bytes(int t) { return t == FA_ACT_F32 ? 4 : 2; }
inline bool act_type(int t) { return t >= FA_ACT_F32 && t <= FA_ACT_BF16; }

// The argument checks of a paged cache, and its device form but for `err`.
fa_status check_cache(const fa_paged_cache* c, Cache* out);
fa_status check_rope(const fa_rope* r, int D, const int32_t* pos, int N, Rope* out);

}  // namespace fap
