// Page tables, lengths and the slots of new tokens, from the requests' lengths.
//
// Prefix sums over the requests of the tokens and of the pages that they ask for give each request its first token
// and its place on the stack; a token finds its request, and a page its request, by bisection of the sums.  All
// CTAs (a cluster, of one for small calls) take the same sums over 1024 requests at a time, then a share of
// those requests' tokens and pages each.  What is edited in place is written behind a barrier of the cluster, when
// everyone has read it; table entries and stack entries that are written are read by nobody else in the call.
//
// What is read and written is a few kilobytes (a megabyte for 99068 tokens): the calls are launches and chains of latencies,
// on a GB300 one new token for each of 64 requests 3.6 us of GPU time, giving them up again 2.5; 99068 tokens of 509
// requests 8 and 3.
#include <algorithm>

#include "fa_paged.cuh"

namespace fap {

constexpr int kThreads = 1024;
constexpr int kMostCtas = 8;                  // of a cluster
constexpr uint32_t kCap = 0x7fffffffu;        // sums stop here

struct ListArgs {
  int32_t *table, *lens, *free, *num_free;
  int num_pages, page_size, B, max_pages;
  uint32_t page_mul;  // as in Cache
  int page_shift;
  const int32_t* arg;  // new_tokens, or keep
  int T;
  int32_t *starts, *first, *seq, *pos, *row;
  bool slots_apart;  // the tokens' slots are another kernel's
  bool vec;          // seq, pos and row start on 16 bytes
  int* err;

  __device__ __forceinline__ int page_of(int j) const { return (int)((uint64_t)(uint32_t)j * page_mul >> page_shift); }
  __device__ __forceinline__ int pages_of(int len) const { return len > 0 ? page_of(len - 1) + 1 : 0; }
  __device__ __forceinline__ int row_of(int page, int pos, int p) const {  // of position pos, on the request's page p
    if (page >= 0 && page < num_pages) return page * page_size + (pos - p * page_size);
    report_page(err);
    return -1;
  }
  __device__ __forceinline__ int on_stack() const { return min(max(num_free[0], 0), num_pages); }
};

__device__ __forceinline__ uint32_t add_cap(uint32_t a, uint32_t b) { return min(a + b, kCap); }  // a, b <= kCap

// Sums of (x, y) over the threads before this one, and over all of them, stopping at kCap (s: 33 words each).
__device__ __forceinline__ void scan2(uint32_t& x, uint32_t& y, uint32_t& all_x, uint32_t& all_y, uint2* s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t a = x, b = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t c = __shfl_up_sync(kFull, a, o), d = __shfl_up_sync(kFull, b, o);
    if (lane >= o) a = add_cap(a, c), b = add_cap(b, d);
  }
  const uint32_t up_a = __shfl_up_sync(kFull, a, 1), up_b = __shfl_up_sync(kFull, b, 1);
  __syncthreads();  // (the last use of s is over)
  if (lane == 31) s[warp] = make_uint2(a, b);
  __syncthreads();
  if (warp == 0) {
    uint2 v = s[lane];
    uint32_t c = v.x, d = v.y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t e = __shfl_up_sync(kFull, c, o), f = __shfl_up_sync(kFull, d, o);
      if (lane >= o) c = add_cap(c, e), d = add_cap(d, f);
    }
    if (lane == 31) s[32] = make_uint2(c, d);
    const uint32_t e = __shfl_up_sync(kFull, c, 1), f = __shfl_up_sync(kFull, d, 1);
    s[lane] = lane ? make_uint2(e, f) : make_uint2(0, 0);
  }
  __syncthreads();
  const uint2 before = s[warp], all = s[32];
  x = add_cap(before.x, lane ? up_a : 0), y = add_cap(before.y, lane ? up_b : 0);
  all_x = all.x, all_y = all.y;
}
// The last i of the 1024 with v[i] <= x (v ascending, v[0] <= x)
__device__ __forceinline__ int last_at_most(const uint32_t* v, uint32_t x) {
  int i = 0;
#pragma unroll
  for (int step = kThreads / 2; step > 0; step >>= 1)
    if (v[i + step] <= x) i += step;
  return i;
}

__global__ void __launch_bounds__(kThreads) k_pages_extend(const ListArgs a) {
  __shared__ uint2 s_scan[33];
  __shared__ uint32_t s_start[kThreads], s_page[kThreads];  // of the requests: first token, first place on the stack
  __shared__ int s_len[kThreads];                           // length, -1: gets nothing
  const int tid = threadIdx.x;
  after_last();
  lets_next();
  const uint32_t me = cluster_rank() * kThreads + tid, all = cluster_ctas() * kThreads, rank = cluster_rank();
  const uint32_t F = (uint32_t)a.on_stack(), T = (uint32_t)a.T;
  uint32_t tokens = 0, asked = 0, taken = 0;  // before this chunk of requests; taken off the stack
  if (rank == 0 && tid == 0) a.starts[0] = 0;
  for (int c0 = 0; c0 < a.B; c0 += kThreads) {
    const int b = c0 + tid;
    int len = -1, add = 0;
    if (b < a.B) len = a.lens[b], add = len >= 0 ? max(a.arg[b], 0) : 0;
    const bool fits = add > 0 && (long long)len + add <= (long long)a.max_pages * a.page_size;
    const int old = a.pages_of(len);
    const uint32_t need = fits ? (uint32_t)(a.pages_of(len + add) - old) : 0;
    uint32_t start = (uint32_t)add, page = need, chunk_tokens, chunk_asked;
    scan2(start, page, chunk_tokens, chunk_asked, s_scan);
    start = add_cap(start, tokens), page = add_cap(page, asked);
    const uint32_t end = add_cap(start, (uint32_t)add);
    const bool got = fits && end <= T && (need == 0 || add_cap(page, need) <= F);
    s_start[tid] = start, s_page[tid] = page, s_len[tid] = got ? len : -1;
    if (rank == 0 && b < a.B) a.starts[b + 1] = (int)min(end, T), a.first[b] = got ? len : -1;
    // the pages that are handed out reach from `asked` to the end of the last request that gets some
    const uint32_t got_to = got && need ? page + need : 0;
    const uint32_t top = __reduce_max_sync(kFull, got_to);
    __syncthreads();
    if ((tid & 31) == 0) s_scan[tid >> 5].x = top;
    __syncthreads();
    const uint32_t pages_end = max(__reduce_max_sync(kFull, s_scan[tid & 31].x), taken);
    // tokens of these requests (of a large call: k_page_slots)
    const uint32_t t1 = a.slots_apart ? 0 : min(add_cap(tokens, chunk_tokens), T);
    for (uint32_t t = tokens + me; t < t1; t += all) {
      const int i = last_at_most(s_start, t), l = s_len[i];
      int pos = -1, row = -1;
      if (l >= 0) {
        pos = l + (int)(t - s_start[i]);
        const int p = a.page_of(pos), had = a.pages_of(l);
        row = a.row_of(p < had ? a.table[(long long)(c0 + i) * a.max_pages + p] : a.free[F - 1 - (s_page[i] + (uint32_t)(p - had))], pos, p);
      }
      a.seq[t] = l >= 0 ? c0 + i : -1, a.pos[t] = pos, a.row[t] = row;
    }
    // and their pages
    for (uint32_t g = asked + me; g < pages_end; g += all) {
      const int i = last_at_most(s_page, g), l = s_len[i];
      if (l >= 0) a.table[(long long)(c0 + i) * a.max_pages + a.pages_of(l) + (int)(g - s_page[i])] = a.free[F - 1 - g];
    }
    tokens = add_cap(tokens, chunk_tokens), asked = add_cap(asked, chunk_asked), taken = pages_end;
    cluster_barrier();  // everyone has read these lengths (and the count), and this CTA's arrays
    if (rank == 0 && got) a.lens[b] = len + add;
  }
  for (uint32_t t = a.slots_apart ? T : min(tokens, T) + me; t < T; t += all) a.seq[t] = a.pos[t] = a.row[t] = -1;
  if (a.B > 0 && rank == 0 && tid == 0) a.num_free[0] = (int)(F - taken);
}

// The slots of a large call's tokens, from the starts, lengths and tables that k_pages_extend has written: four neighbours
// a thread, of one request and on one page as a rule.  (99068 tokens in the cluster's eight SMs: 6 us of the call's 13.)
constexpr int kSlotThreads = 256, kHeldStarts = 8192;  // requests whose starts lie in shared memory
__global__ void __launch_bounds__(kSlotThreads) k_page_slots(const ListArgs a) {
  extern __shared__ int s_starts[];
  after_last();
  lets_next();
  const bool held = a.B <= kHeldStarts;
  if (held) {
    for (int i = threadIdx.x; i < a.B; i += kSlotThreads) s_starts[i] = a.starts[i];
    __syncthreads();
  }
  auto start = [&](int i) { return held ? s_starts[i] : a.starts[i]; };
  const int t0 = 4 * (blockIdx.x * kSlotThreads + threadIdx.x), end = a.starts[a.B];
  if (t0 >= a.T) return;
  int i = 0;  // the last request that starts at t0 or before
  for (int n = a.B; n > 1;) {
    const int half = n >> 1;
    if (start(i + half) <= t0) i += half, n -= half;
    else n = half;
  }
  int first = a.first[i], at = start(i), next = i + 1 < a.B ? start(i + 1) : end, known = -1, page = -1, seq[4], pos[4], row[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int t = t0 + k;
    seq[k] = pos[k] = row[k] = -1;
    if (t >= end) continue;
    if (t >= next) {
      do {
        ++i, at = next, next = i + 1 < a.B ? start(i + 1) : end;
      } while (t >= next);
      first = a.first[i], known = -1;
    }
    if (first < 0) continue;
    seq[k] = i, pos[k] = first + (t - at);
    const int p = a.page_of(pos[k]);
    if (p != known) known = p, page = a.table[(long long)i * a.max_pages + p];
    row[k] = a.row_of(page, pos[k], p);
  }
  if (a.vec && t0 + 4 <= a.T) {
    *reinterpret_cast<int4*>(a.seq + t0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
    *reinterpret_cast<int4*>(a.pos + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    *reinterpret_cast<int4*>(a.row + t0) = make_int4(row[0], row[1], row[2], row[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (t0 + k < a.T) a.seq[t0 + k] = seq[k], a.pos[t0 + k] = pos[k], a.row[t0 + k] = row[k];
  }
}

__global__ void __launch_bounds__(kThreads) k_pages_trim(const ListArgs a) {
  __shared__ uint2 s_scan[33];
  __shared__ uint32_t s_page[kThreads];
  __shared__ int s_first[kThreads];
  const int tid = threadIdx.x;
  after_last();
  lets_next();
  const uint32_t me = cluster_rank() * kThreads + tid, all = cluster_ctas() * kThreads, rank = cluster_rank();
  const int F = a.on_stack();
  const int most = a.max_pages * a.page_size;
  auto request = [&](int b, int& len, int& keep, int& back) {  // pages that it gives back
    len = keep = -1, back = 0;
    if (b >= a.B) return;
    len = a.lens[b], keep = a.arg[b];
    if (keep < 0 || keep >= len) keep = len;
    else back = a.pages_of(min(len, most)) - a.pages_of(min(keep, most));
  };
  int len, keep, back;
  uint32_t total = 0;
  if (a.B > kThreads) {  // (else the one chunk's sum is the total)
    for (int c0 = 0; c0 < a.B; c0 += kThreads) {
      request(c0 + tid, len, keep, back);
      uint32_t x = (uint32_t)back, y = 0, sum, none;
      scan2(x, y, sum, none, s_scan);
      total = add_cap(total, sum);
    }
  }
  uint32_t before = 0;
  for (int c0 = 0; c0 < a.B; c0 += kThreads) {
    const int b = c0 + tid;
    request(b, len, keep, back);
    uint32_t page = (uint32_t)back, y = 0, sum, none;
    scan2(page, y, sum, none, s_scan);
    if (a.B <= kThreads) total = sum;
    s_page[tid] = add_cap(page, before), s_first[tid] = a.pages_of(min(keep, most));
    __syncthreads();
    const uint32_t end = add_cap(before, sum);
    for (uint32_t g = before + me; g < end; g += all) {
      const int i = last_at_most(s_page, g);
      int32_t* entry = a.table + (long long)(c0 + i) * a.max_pages + s_first[i] + (int)(g - s_page[i]);
      const long long at = F + (long long)(total - 1 - g);
      if (at < a.num_pages) a.free[at] = *entry;
      else report_page(a.err);
      *entry = -1;
    }
    before = end;
    cluster_barrier();
    if (rank == 0 && b < a.B && keep < len) a.lens[b] = keep;
  }
  if (a.B > 0 && rank == 0 && tid == 0) a.num_free[0] = (int)min((long long)F + total, (long long)a.num_pages);
}

static fa_status check_lists(const fa_page_lists* l, const int32_t* arg, ListArgs* a) {
  *a = ListArgs{};
  if (!l) return FA_ERR_NULL;
  if (l->num_pages < 0 || l->page_size < 1 || l->B < 0 || l->max_pages < 0) return FA_ERR_SHAPE;
  if (l->B > (1 << 20) || (long long)l->max_pages * l->page_size > (1LL << 30) || (long long)l->num_pages * l->page_size > 0x7fffffffLL)
    return FA_ERR_UNSUPPORTED;
  if (!l->num_free || (l->num_pages > 0 && !l->free_pages) || (l->B > 0 && (!l->seq_lens || !arg)) ||
      (l->B > 0 && l->max_pages > 0 && !l->page_table))
    return FA_ERR_NULL;
  if (!aligned(l->page_table, 4) || !aligned(l->seq_lens, 4) || !aligned(l->free_pages, 4) || !aligned(l->num_free, 4) || !aligned(arg, 4))
    return FA_ERR_ALIGN;
  a->table = l->page_table, a->lens = l->seq_lens, a->free = l->free_pages, a->num_free = l->num_free;
  a->num_pages = l->num_pages, a->page_size = l->page_size, a->B = l->B, a->max_pages = l->max_pages, a->arg = arg;
  page_divisor(l->page_size, &a->page_mul, &a->page_shift);
  return FA_OK;
}

// One cluster; `work`: tokens or pages that there may be, one for each thread while there are CTAs
static cudaError_t launch_lists(void (*k)(const ListArgs), long long work, const ListArgs& a, cudaStream_t s) {
  int ctas = 1;
  while (ctas < kMostCtas && work > (long long)kThreads * ctas) ctas *= 2;
  return launch_clusters(k, (unsigned)ctas, (unsigned)ctas, kThreads, 0, s, a);
}

}  // namespace fap

using namespace fap;

extern "C" fa_status fa_pages_extend(const fa_page_lists* lists, const int32_t* new_tokens, int T, int32_t* starts,
                                     int32_t* first, int32_t* seq, int32_t* pos, int32_t* row, void* stream) {
  ListArgs a;
  fa_status rc = check_lists(lists, new_tokens, &a);
  if (rc != FA_OK) return rc;
  if (T < 0) return FA_ERR_SHAPE;
  if (T > (1 << 30)) return FA_ERR_UNSUPPORTED;
  if (!starts || (a.B > 0 && !first) || (T > 0 && (!seq || !pos || !row))) return FA_ERR_NULL;
  if (!aligned(starts, 4) || !aligned(first, 4) || !aligned(seq, 4) || !aligned(pos, 4) || !aligned(row, 4)) return FA_ERR_ALIGN;
  int nsm = 0;
  if ((rc = fab_device(&nsm, &a.err)) != FA_OK) return rc;
  a.T = T, a.starts = starts, a.first = first, a.seq = seq, a.pos = pos, a.row = row;
  a.vec = aligned(seq, 16) && aligned(pos, 16) && aligned(row, 16);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // A token a thread of the cluster; more of them are shared out over all SMs, by a launch of their own.  B = 0 has no
  // requests to look for.
  a.slots_apart = T > kThreads * kMostCtas && a.B > 0;
  if (launch_lists(k_pages_extend, T, a, s) != cudaSuccess) return FA_ERR_CUDA;
  if (!a.slots_apart) return FA_OK;
  const unsigned grid = (unsigned)((T + 4LL * kSlotThreads - 1) / (4 * kSlotThreads));
  return launch_next(k_page_slots, dim3(grid), dim3(kSlotThreads), (size_t)std::min(a.B, kHeldStarts) * sizeof(int), s, a) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

extern "C" fa_status fa_pages_trim(const fa_page_lists* lists, const int32_t* keep, void* stream) {
  ListArgs a;
  fa_status rc = check_lists(lists, keep, &a);
  if (rc != FA_OK) return rc;
  int nsm = 0;
  if ((rc = fab_device(&nsm, &a.err)) != FA_OK) return rc;
  if (a.B == 0) return FA_OK;
  const long long work = std::min<long long>(a.num_pages, (long long)a.B * a.max_pages) / 8;  // (few of them come back at a time)
  return launch_lists(k_pages_trim, work, a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
