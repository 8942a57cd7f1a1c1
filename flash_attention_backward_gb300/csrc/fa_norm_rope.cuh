// Queries and keys of a layer, head by head: RMS norm and position rotation in one pass, and the
// gradient.
//
//   y = R (w o x r),  r = rsqrt(mean(x^2) + eps)
//   g = R^T gy,  dw = sum g o x r,  h = g o w,  dx = r (h - x r^2 mean(h o x))
//
// A head is read once and written once (backward: x and gy read, dx written), everything between stays in
// registers.  The arithmetic has to stay out of the way: a head of 128 bf16 components is 256 bytes, so an SM
// takes one every ten cycles at the card's bandwidth.  Hence the layout: D / 8 lanes a head, and a lane holds both
// members of its four rotation pairs, which makes the rotation free of shuffles; packed pairs of f32
// (fma.rn.f32x2) halve the instructions; the angles of a token are computed once for all heads of it that a warp
// takes.
//
// Measured on a GB300 (6787 GB/s copy rate).  Forward, 2048 tokens of 28 heads of 256, f32, 117 MB: 21.1 us a call
// over changing inputs, 82 % of the copy rate (17.7 us of GPU time over the same inputs, part of which L2 then
// holds).  16411 tokens of 10 heads of 64, bf16 to f32, 63 MB: 16.1 us, 58 %, at 2.4 of 4 instructions a cycle and SM: the
// 16 angles of a token (half of the warp's lanes) are shared by ten heads only, and those are two and a half rounds
// of four.  Gradient, 8191 tokens of 40 heads of 128, bf16, 252
// MB: 52 us, 71 %, at 2.4 instructions a cycle beside 52 % of DRAM; 2048 tokens of 28 heads of 256, f32, 176 MB:
// 34.4 us, 75 %.  Heads off 16 bytes: forward 20.1 us for 17.7, gradient 49.7 for 33.5.  64 tokens: 2.4 us, a launch
// and two latencies.
#pragma once
#include "fa_paged.cuh"
#include "sm100.cuh"

namespace fap {

struct NormSide {  // queries or keys
  const void* x;
  const void* gy;      // backward: gradient of the output
  long long row, head; // strides of x
  const float* w;
  void* y;             // y, or dx
  int H;               // heads
  int nchunk;          // backward: chunks of a token's heads
};
struct NormArgs {
  NormSide side[2];
  int HC, nchunk;      // forward: heads (queries', then keys') of one token that a warp takes, chunks of a token
  int ctas_q;          // backward: CTAs 0 .. ctas_q - 1 take queries, the rest keys
  float eps;
  Rope rope;
  int N;
  bool vec;            // both start every head of x on 16 bytes (or have none)
  float* part;         // backward: [CTA][D] sums of dw
  int* err;
  uint64_t wait_ns;    // backward: a wait for a copy gives up after this long (0, the failure-detection hook: at once)
};

// Rows that a lane group has under way at a time: 32 or 64 bytes a lane of x (and as much of gy).
template <typename T>
constexpr int kRows = sizeof(T) == 2 ? 4 : 2;
constexpr uint64_t kCopyDrainNs = 2000000000ull;  // after a wait that ran out: for the copies in flight to land

template <typename T>
__device__ __forceinline__ void store_eight(T* p, int ea, int eb, const float2 (&x)[4]) {
  Four<T> a, b;
  a.v[0] = from_f32<T>(x[0].x), a.v[1] = from_f32<T>(x[0].y), a.v[2] = from_f32<T>(x[1].x), a.v[3] = from_f32<T>(x[1].y);
  b.v[0] = from_f32<T>(x[2].x), b.v[1] = from_f32<T>(x[2].y), b.v[2] = from_f32<T>(x[3].x), b.v[3] = from_f32<T>(x[3].y);
  *reinterpret_cast<Four<T>*>(p + ea) = a;
  *reinterpret_cast<Four<T>*>(p + eb) = b;
}

// What a lane keeps for a token: its components, the norm's weights, the factors of its pairs.
template <int D, int STYLE>
struct Lane {
  int ea, eb;
  int n;  // the lane's pairs that turn, its first ones.  The others are not touched: turned by nothing, an
          // infinity would become NaN, and a NaN would enter its partner.
  bool norm;
  float2 w[4];
  float2 c[2], s[2], ns[2];  // cos, sin, -sin of pairs (0, 1) and (2, 3)
  static constexpr int P = D / 64;

  __device__ __forceinline__ void place(const Rope& r) {
    const int p = (threadIdx.x & (D / 8 - 1)) * 4, half = r.n_rot >> 1;
    n = min(max(half - p, 0), 4);
    if (STYLE == FA_ROPE_PAIRS) ea = 2 * p, eb = ea + 4;
    else if (p < half) ea = p, eb = p + half;
    else ea = r.n_rot + (p - half), eb = ea + (D - r.n_rot) / 2;
  }
  __device__ __forceinline__ void weights(const float* weight) {
    norm = weight != nullptr;
    if (norm) {
      Eight<float> o;
      load_eight<float, false>(weight, ea, eb, o);
      unpack_eight(o, w);
    }
  }
  // The factors (sin_cos_turn) at the positions of the lane's share of the token's pairs (PairPos); sign -1 turns
  // back (the transpose).
  __device__ __forceinline__ void turn(const Rope& r, const int (&pos)[P], float sign) {
    const int lane = threadIdx.x & 31, half = r.n_rot >> 1;
    float cs[P], sn[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      cs[i] = 1.f, sn[i] = 0.f;
      if (lane * P + i < half) {
        sin_cos_turn(r.freqs[lane * P + i], pos[i], &sn[i], &cs[i]);
        sn[i] *= sign;
      }
    }
    const int p = (lane & (D / 8 - 1)) * 4;
    float cc[4], ss[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cc[i] = P == 4 ? cs[i % P] : __shfl_sync(kFull, cs[i % P], (p + i) / P);  // (D = 256: the lane's own)
      ss[i] = P == 4 ? sn[i % P] : __shfl_sync(kFull, sn[i % P], (p + i) / P);
    }
    c[0] = make_float2(cc[0], cc[1]), c[1] = make_float2(cc[2], cc[3]);
    s[0] = make_float2(ss[0], ss[1]), s[1] = make_float2(ss[2], ss[3]);
    ns[0] = make_float2(-ss[0], -ss[1]), ns[1] = make_float2(-ss[2], -ss[3]);
  }
  // Takes over the factors of another lane's, of the same token.
  __device__ __forceinline__ void turned_as(const Lane& o) {
#pragma unroll
    for (int i = 0; i < 2; ++i) c[i] = o.c[i], s[i] = o.s[i], ns[i] = o.ns[i];
  }
  // An unrotated component: x c + 0 s with c = 1, s = 0 and 0 for the partner, whose value must not enter
  // (16411 tokens of 10 heads of 64, half of each rotated: 17.7 us a call; 18.1 with the result selected, 18.2 with
  // a branch).
  __device__ __forceinline__ void rotate(float2 (&x)[4]) const {
    if (STYLE == FA_ROPE_HALVES) {
      if (n == 0) return;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 a = x[i], b = x[2 + i];
        x[i] = __ffma2_rn(b, ns[i], __fmul2_rn(a, c[i]));
        x[2 + i] = __ffma2_rn(a, s[i], __fmul2_rn(b, c[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ci = i & 1 ? c[i >> 1].y : c[i >> 1].x, si = i & 1 ? s[i >> 1].y : s[i >> 1].x;
        const uint32_t on = i < n ? 0xffffffffu : 0u;
        const float a = x[i].x, b = x[i].y;
        x[i].x = fmaf(__uint_as_float(__float_as_uint(b) & on), -si, a * ci);
        x[i].y = fmaf(__uint_as_float(__float_as_uint(a) & on), si, b * ci);
      }
    }
  }
  __device__ __forceinline__ void forward(float2 (&x)[4], float eps) const {
    if (norm) {
      const float r = inv_rms(square_sum<D>(x), 1.f / D, eps);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __fmul2_rn(__fmul2_rn(x[i], make_float2(r, r)), w[i]);
    }
    rotate(x);
  }
  // g: gradient of the output, becomes dx.  on: the lane's head counts
  __device__ __forceinline__ void backward(const float2 (&x)[4], float2 (&g)[4], float2 (&dw)[4], float eps, bool on) const {
    rotate(g);
    if (!norm) return;
    float2 gx[4], q = make_float2(0.f, 0.f), z = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      gx[i] = __fmul2_rn(g[i], x[i]);
      q = __ffma2_rn(x[i], x[i], q);
      z = __ffma2_rn(gx[i], w[i], z);
    }
    const float ss = group_sum<D / 8>(q.x + q.y), hx = group_sum<D / 8>(z.x + z.y);
    const float r = inv_rms(ss, 1.f / D, eps), m = -hx * (1.f / D) * r * r;
    const float rd = on ? r : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dw[i] = __ffma2_rn(gx[i], make_float2(rd, rd), dw[i]);
      g[i] = __fmul2_rn(make_float2(r, r), __ffma2_rn(x[i], make_float2(m, m), __fmul2_rn(g[i], w[i])));
    }
  }
};

// A warp takes HC heads of one token, 256 / D side by side, and loads the next kRows of each together.
// VEC: every head of x starts on 16 bytes (else it is loaded element by element).  Lanes without a head of
// their own (the last ones of a token) work on the last head and store nothing.
// With 16-bit x, whose time is its instructions, a warp goes on to further tokens with both weights at hand
// (16411 tokens of 10 heads of 64: 18.5 -> 15.5 us); with f32 x, whose time is its bytes, many short warps
// keep more loads in flight (2048 tokens of 28 heads of 256: 17.7 us, and 23.9 the other way).
template <typename TX>
constexpr int kForwardCtas = sizeof(TX) == 2 ? 3 : 0;  // CTAs an SM, or 0: a warp takes one item
template <int D, typename TX, typename TY, bool VEC, int STYLE, bool AXES>
__global__ void __launch_bounds__(256, kForwardCtas<TX>) k_norm_rope(const NormArgs a) {
  constexpr int GW = 256 / D, U = kRows<TX>;
  after_last();
  lets_next();
  const int grp = (threadIdx.x & 31) / (D / 8);
  const unsigned items = (unsigned)a.N * a.nchunk;
  constexpr bool ON = kForwardCtas<TX> > 0;
  Lane<D, STYLE> lanes[1 + ON];  // queries' (and keys'); one for both where each item is another warp's
#pragma unroll
  for (int k = 0; k <= ON; ++k) {
    lanes[k].place(a.rope);
    if (ON) lanes[k].weights(a.side[k].w);
  }
  PairPos<D, AXES> axes;
  axes.look_up(a.rope);
  for (unsigned item = blockIdx.x * 8u + (threadIdx.x >> 5); item < items; item += gridDim.x * 8u) {
    const int n = item / (unsigned)a.nchunk, c0 = (int)(item - (unsigned)n * a.nchunk) * a.HC;
    bool turned = false;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const NormSide& sd = a.side[k];
      const int first = k ? a.side[0].H : 0;  // the side's first head among all
      const int h0 = max(c0 - first, 0);
      int left = min(sd.H, c0 + a.HC - first) - h0;  // heads that the warp still has
      if (left <= 0) continue;
      Lane<D, STYLE>& ln = lanes[ON ? k : 0];
      const long long head = sd.head;
      const TX* x0 = static_cast<const TX*>(sd.x) + n * sd.row + h0 * head;
      TY* y0 = static_cast<TY*>(sd.y) + ((long long)n * sd.H + h0 + grp) * D;
      Eight<TX> raw[U];
      auto fetch = [&] {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u * GW < left) load_eight<TX, VEC>(x0 + min(grp + u * GW, left - 1) * head, ln.ea, ln.eb, raw[u]);
      };
      fetch();
      if (!ON) ln.weights(sd.w);
      if (!turned) {
        int pos[D / 64];
        axes.hand_round(AXES || a.rope.n_rot ? axes.load(a.rope, n) : 0, pos);
        lanes[0].turn(a.rope, pos, 1.f);
      }
      turned = true;
      if (ON && k) ln.turned_as(lanes[0]);
      for (;;) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (u * GW >= left) break;  // (the same in all lanes)
          float2 x[4];
          unpack_eight(raw[u], x);
          ln.forward(x, a.eps);
          if (grp + u * GW < left) store_eight(y0 + u * GW * D, ln.ea, ln.eb, x);
        }
        left -= U * GW;
        if (left <= 0) break;
        x0 += U * GW * head, y0 += U * GW * D;
        fetch();
      }
    }
    if (!ON) break;
  }
}

// The gradient.  Each warp takes a run of items (HC heads of a token), which pass through a ring of its own
// in shared memory: bulk copies bring x and gy of the items to come while one is worked on, which takes
// the loads off the registers and the issue slots.  A token's factors are computed when the run comes to
// it.  dw is summed by lane over the run (put_dw), then over the CTA's lane groups in order.  (Loads into registers
// instead of the ring: 79 us for 8191 tokens of 40 heads of 128, bf16, against 52.)
constexpr int kBackCtas = 2, kBackWarps = 8;
// Slots of a warp's ring and their bytes: a head of f32 takes up to 2 KB, and an item of one or two would
// cost more in its handling than in its work (2048 tokens of 28 heads of 256: 33.8 us with 2 slots of
// 6 KB, 34.9 with 3 of 4).
template <typename TX, typename TY>
constexpr int kBackSlots = sizeof(TX) + sizeof(TY) == 8 ? 2 : 3;
template <typename TX, typename TY>
constexpr int kBackBytes = sizeof(TX) + sizeof(TY) == 8 ? 6144 : 4096;
// Heads of an item: what a slot holds, in multiples of those side by side in a warp
template <int D, typename TX, typename TY>
constexpr int kBackHeads = kBackBytes<TX, TY> / (256 * (int)(sizeof(TX) + sizeof(TY))) * (256 / D);

__device__ __forceinline__ void bulk_run(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// dw: a lane sums its rows' terms in registers, adds them to its lane group's row of `red` after so many items as
// there will be such sums, and starts again: no f32 sum takes more than some sqrt of the lane's rows.  What is
// left is added up with what its roundings lose.  (Doubles there: 58.3 us for 52.6 with 8191 tokens of 40 heads
// of 128, bf16; plain f32 sums: 51.5.)
struct ExactSum {
  float s = 0.f, lost = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float t = s + x, z = t - s;
    lost += (s - (t - z)) + (x - z);
    s = t;
  }
  __device__ __forceinline__ float value() const { return fabsf(s) < INFINITY ? s + lost : s; }
};
__device__ __forceinline__ unsigned dw_run(unsigned items) { return max(16u, (unsigned)sqrtf((float)items)); }
template <int D>
__device__ __forceinline__ void put_dw(float2 (&dw)[4], int ea, int eb, float* red, bool more) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float4* r = reinterpret_cast<float4*>(red + (i ? eb : ea));  // (both are multiples of four)
    float4 x = make_float4(dw[2 * i].x, dw[2 * i].y, dw[2 * i + 1].x, dw[2 * i + 1].y);
    if (more) {
      const float4 y = *r;
      x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    *r = x;
    dw[2 * i] = dw[2 * i + 1] = make_float2(0.f, 0.f);
  }
}
template <int D, int GROUPS>
__device__ __forceinline__ void sum_dw(const NormArgs& a, float (*red)[D]) {
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kBackWarps * 32) {
    ExactSum s;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) s.add(red[g][c]);
    a.part[(long long)blockIdx.x * D + c] = s.value();
  }
}

template <int D, typename TX, typename TY, int STYLE, bool AXES>
__global__ void __launch_bounds__(kBackWarps * 32, kBackCtas) k_norm_rope_back(const NormArgs a) {
  constexpr int GW = 256 / D, HC = kBackHeads<D, TX, TY>, GB = HC * D * sizeof(TY), XB = HC * D * sizeof(TX), S = kBackSlots<TX, TY>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) float red[kBackWarps * GW][D];
  __shared__ uint64_t s_bar[kBackWarps][S];
  after_last();
  const bool isq = blockIdx.x < a.ctas_q;
  const NormSide sd = a.side[isq ? 0 : 1];
  const int lane = threadIdx.x & 31, grp = lane / (D / 8), warp = threadIdx.x >> 5;
  const int ctas = isq ? a.ctas_q : gridDim.x - a.ctas_q, me = (blockIdx.x - (isq ? 0 : a.ctas_q)) * kBackWarps + warp;
  const unsigned items = (unsigned)a.N * sd.nchunk;
  const unsigned first = (unsigned)((unsigned long long)items * me / (ctas * kBackWarps));
  const unsigned last = (unsigned)((unsigned long long)items * (me + 1) / (ctas * kBackWarps));
  const uint32_t slots = fab::smem_u32(ring) + warp * S * (GB + XB);
  if (lane < S) fab::mbar_init(&s_bar[warp][lane], 1);
  fab::fence_mbar_init();
  __syncwarp();

  float2 dw[4] = {};
  Lane<D, STYLE> ln;
  ln.place(a.rope);
  ln.weights(sd.w);
  // token and first head of the next item to fetch, and of the one to work on
  int fn = first / (unsigned)sd.nchunk, fh = (int)(first - (unsigned)fn * sd.nchunk) * HC, n = fn, h = fh;
  unsigned fetched = first;
  auto fetch = [&](int slot) {
    const int cnt = min(HC, sd.H - fh);
    const uint32_t at = slots + slot * (GB + XB), bar = fab::smem_u32(&s_bar[warp][slot]);
    const TX* x = static_cast<const TX*>(sd.x) + fn * sd.row + fh * sd.head;
    if (lane == 0) {
      fab::mbar_arrive_expect_tx(&s_bar[warp][slot], cnt * D * (sizeof(TY) + (ln.norm ? sizeof(TX) : 0)));
      bulk_run(at, static_cast<const TY*>(sd.gy) + ((long long)fn * sd.H + fh) * D, cnt * D * sizeof(TY), bar);
      if (ln.norm && sd.head == D) bulk_run(at + GB, x, cnt * D * sizeof(TX), bar);
    }
    if (ln.norm && sd.head != D) {
      __syncwarp();
      if (lane < cnt) bulk_run(at + GB + lane * D * (int)sizeof(TX), x + lane * sd.head, D * sizeof(TX), bar);
    }
    ++fetched;
    if ((fh += HC) >= sd.H) fh = 0, ++fn;
  };
  for (int i = 0; i < S; ++i)
    if (fetched < last) fetch(i);
  int slot = 0, token = -1;
  uint32_t phase = 0;
  PairPos<D, AXES> axes;
  axes.look_up(a.rope);
  auto pos_of = [&](int t) { return a.rope.n_rot && t < a.N ? axes.load(a.rope, t) : 0; };
  int pos = pos_of(n);
  unsigned run = dw_run(last - first);
  bool put = false;  // sums lie in `red` already
  for (unsigned item = first; item < last; ++item) {
    if (n != token) {
      int at[D / 64];
      axes.hand_round(pos, at);
      ln.turn(a.rope, at, -1.f);
      token = n, pos = pos_of(n + 1);  // the next token's, in time
    }
    const bool came = a.wait_ns > 0 && fab::mbar_wait_bounded(&s_bar[warp][slot], phase, a.wait_ns);
    if (!__all_sync(kFull, came)) {  // let the copies in flight land, then give up
      if (lane == 0) {
        atomicExch(a.err, FA_ERR_TIMEOUT);
        for (unsigned k = item; k < fetched; ++k) {
          fab::mbar_wait_bounded(&s_bar[warp][slot], phase, kCopyDrainNs);
          if (++slot == S) slot = 0, phase ^= 1;
        }
      }
      break;
    }
    const int cnt = min(HC, sd.H - h);
    const TY* gs = reinterpret_cast<const TY*>(ring + warp * S * (GB + XB) + slot * (GB + XB));
    const TX* xs = reinterpret_cast<const TX*>(reinterpret_cast<const uint8_t*>(gs) + GB);
    TX* d0 = static_cast<TX*>(sd.y) + ((long long)n * sd.H + h + grp) * D;
#pragma unroll 2
    for (int k = 0; k < cnt; k += GW) {
      const int hh = min(k + grp, cnt - 1);  // lanes without a head of their own work on the last, unheeded
      Eight<TX> rx;
      Eight<TY> rg;
      float2 x[4], g[4];
      load_eight<TY, true>(gs + hh * D, ln.ea, ln.eb, rg);
      if (ln.norm) load_eight<TX, true>(xs + hh * D, ln.ea, ln.eb, rx);
      unpack_eight(rg, g);
      unpack_eight(rx, x);
      const bool on = k + grp < cnt;
      ln.backward(x, g, dw, a.eps, on);
      if (on) store_eight(d0 + k * D, ln.ea, ln.eb, g);
    }
    __syncwarp();
    if (fetched < last) fetch(slot);
    if (++slot == S) slot = 0, phase ^= 1;
    if ((h += HC) >= sd.H) h = 0, ++n;
    if (ln.norm && --run == 0) {
      put_dw<D>(dw, ln.ea, ln.eb, red[warp * GW + grp], put);
      run = dw_run(last - first), put = true;
    }
  }
  lets_next();
  if (ln.norm) {
    put_dw<D>(dw, ln.ea, ln.eb, red[warp * GW + grp], put);
    sum_dw<D, kBackWarps * GW>(a, red);
  }
}

// The gradient where heads of x do not start on 16 bytes: element by element.
template <int D, typename TX, typename TY, int STYLE, bool AXES>
__global__ void __launch_bounds__(kBackWarps * 32, kBackCtas) k_norm_rope_back_any(const NormArgs a) {
  constexpr int GW = 256 / D, HC = kBackHeads<D, TX, TY>;
  __shared__ __align__(16) float red[kBackWarps * GW][D];
  after_last();
  const bool isq = blockIdx.x < a.ctas_q;
  const NormSide sd = a.side[isq ? 0 : 1];
  const int grp = (threadIdx.x & 31) / (D / 8), warp = threadIdx.x >> 5;
  const unsigned items = (unsigned)a.N * sd.nchunk;
  const int ctas = isq ? a.ctas_q : gridDim.x - a.ctas_q, cta = blockIdx.x - (isq ? 0 : a.ctas_q);
  float2 dw[4] = {};
  Lane<D, STYLE> ln;
  ln.place(a.rope);
  ln.weights(sd.w);
  unsigned run = dw_run(items / (ctas * kBackWarps));
  bool put = false;
  PairPos<D, AXES> axes;
  axes.look_up(a.rope);
  for (unsigned item = cta * kBackWarps + warp; item < items; item += ctas * kBackWarps) {
    const int n = item / (unsigned)sd.nchunk, h0 = (int)(item - (unsigned)n * sd.nchunk) * HC, cnt = min(sd.H - h0, HC);
    const long long at = ((long long)n * sd.H + h0) * D;
    int pos[D / 64];
    axes.hand_round(a.rope.n_rot ? axes.load(a.rope, n) : 0, pos);
    ln.turn(a.rope, pos, -1.f);
#pragma unroll 1
    for (int k = 0; k < cnt; k += GW) {
      const int hh = min(k + grp, cnt - 1);
      Eight<TX> rx;
      Eight<TY> rg;
      float2 x[4], g[4];
      load_eight<TY, true>(static_cast<const TY*>(sd.gy) + at + hh * D, ln.ea, ln.eb, rg);
      if (ln.norm) load_eight<TX, false>(static_cast<const TX*>(sd.x) + n * sd.row + (h0 + hh) * sd.head, ln.ea, ln.eb, rx);
      unpack_eight(rg, g);
      unpack_eight(rx, x);
      const bool on = k + grp < cnt;
      ln.backward(x, g, dw, a.eps, on);
      if (on) store_eight(static_cast<TX*>(sd.y) + at + (k + grp) * D, ln.ea, ln.eb, g);
    }
    if (ln.norm && --run == 0) {
      put_dw<D>(dw, ln.ea, ln.eb, red[warp * GW + grp], put);
      run = dw_run(items / (ctas * kBackWarps)), put = true;
    }
  }
  if (ln.norm) {
    put_dw<D>(dw, ln.ea, ln.eb, red[warp * GW + grp], put);
    sum_dw<D, kBackWarps * GW>(a, red);
  }
}

typedef void (*NormKernel)(const NormArgs);

// The kernels for these types, with positions of one axis or of several; of the gradient's, the heads of an item and
// what there is to know of its dynamic shared memory too.
template <bool AXES>
NormKernel pick_norm_fwd(int D, int tx, int ty, bool vec, int style);
template <> NormKernel pick_norm_fwd<false>(int, int, int, bool, int);  // fa_norm_rope_fwd.cu
template <> NormKernel pick_norm_fwd<true>(int, int, int, bool, int);   // fa_norm_axes_fwd.cu
struct BackKernel {
  NormKernel fn;
  int heads, smem;
  std::atomic<uint64_t>* ready;  // devices that `smem` bytes have been allowed on
};
template <bool AXES>
BackKernel pick_norm_back(int D, int tx, int ty, bool vec, int style);
template <> BackKernel pick_norm_back<false>(int, int, int, bool, int);  // fa_norm_rope_back.cu
template <> BackKernel pick_norm_back<true>(int, int, int, bool, int);   // fa_norm_axes_back.cu

// How these files choose among what they instantiate
template <int D, typename TX, typename TY, bool AXES>
NormKernel norm_fwd_style(bool vec, int style) {
  if (style == FA_ROPE_PAIRS) return vec ? k_norm_rope<D, TX, TY, true, FA_ROPE_PAIRS, AXES> : k_norm_rope<D, TX, TY, false, FA_ROPE_PAIRS, AXES>;
  return vec ? k_norm_rope<D, TX, TY, true, FA_ROPE_HALVES, AXES> : k_norm_rope<D, TX, TY, false, FA_ROPE_HALVES, AXES>;
}
template <int D, typename TX, typename TY, bool AXES>
BackKernel norm_back_style(bool vec, int style) {
  constexpr int heads = kBackHeads<D, TX, TY>, ring = kBackWarps * kBackSlots<TX, TY> * heads * D * (int)(sizeof(TX) + sizeof(TY));
  const bool pairs = style == FA_ROPE_PAIRS;
  static std::atomic<uint64_t> ready[2];
  if (!vec)
    return BackKernel{pairs ? k_norm_rope_back_any<D, TX, TY, FA_ROPE_PAIRS, AXES> : k_norm_rope_back_any<D, TX, TY, FA_ROPE_HALVES, AXES>,
                      heads, 0, nullptr};
  return BackKernel{pairs ? k_norm_rope_back<D, TX, TY, FA_ROPE_PAIRS, AXES> : k_norm_rope_back<D, TX, TY, FA_ROPE_HALVES, AXES>, heads,
                    ring, &ready[pairs]};
}
#define FAP_PICK_NORM(KIND, PICK, STYLE_OF, AXES)                                                   \
  template <int D, typename TX>                                                                     \
  static KIND PICK##_y(int ty, bool vec, int style) {                                               \
    return ty == FA_ACT_F32   ? STYLE_OF<D, TX, float, AXES>(vec, style)                            \
           : ty == FA_ACT_F16 ? STYLE_OF<D, TX, __half, AXES>(vec, style)                           \
                              : STYLE_OF<D, TX, __nv_bfloat16, AXES>(vec, style);                   \
  }                                                                                                 \
  template <int D>                                                                                  \
  static KIND PICK##_x(int tx, int ty, bool vec, int style) {                                       \
    return tx == FA_ACT_F32   ? PICK##_y<D, float>(ty, vec, style)                                  \
           : tx == FA_ACT_F16 ? PICK##_y<D, __half>(ty, vec, style)                                 \
                              : PICK##_y<D, __nv_bfloat16>(ty, vec, style);                         \
  }                                                                                                 \
  template <>                                                                                       \
  KIND PICK<AXES>(int D, int tx, int ty, bool vec, int style) {                                     \
    return D == 64 ? PICK##_x<64>(tx, ty, vec, style) : D == 128 ? PICK##_x<128>(tx, ty, vec, style) : PICK##_x<256>(tx, ty, vec, style); \
  }

}  // namespace fap
