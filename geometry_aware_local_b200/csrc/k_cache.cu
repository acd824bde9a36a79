// The paged key-value cache's row moves: new rows appended, and the cache cut
// to a budget by accumulated attention weight.
#include "seq.cuh"

namespace pack3d {
namespace seq {
namespace {

// ---- append -----------------------------------------------------------------
// One thread moves one 16-byte chunk of a key row and of its value row: both
// sides of the copy are coalesced, and a row finds its sequence by a binary
// search of cu.  Bound by HBM where there is much to move (65,000 tokens, 2 key
// heads, bf16, 67 MB: 8.9 us, at which most of it is still in L2), else by the
// chain search, length, page, row (64 tokens: 3 us).
__global__ void __launch_bounds__(256) cache_append_kernel(const Cache c, const int32_t* __restrict__ cu, long rows,
                                                           const uint4* __restrict__ k, const uint4* __restrict__ v,
                                                           int chunks) {
  const long total = rows * chunks;
  for (long i = blockIdx.x * (long)blockDim.x + threadIdx.x; i < total; i += (long)gridDim.x * blockDim.x) {
    const long row = i / chunks;
    const int chunk = (int)(i - row * chunks);
    int b = (int)row;
    long in = 0;
    if (cu) {
      int lo = 0, hi = c.B;                 // last b with cu[b] <= row
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid) <= row) lo = mid;
        else hi = mid;
      }
      b = lo;
      const int c0 = __ldg(cu + b), c1 = __ldg(cu + b + 1);
      if (c0 < 0 || c1 < c0 || c1 > rows) {
        set_err(c.err, PACK3D_DEVERR_LENGTHS);
        continue;
      }
      if (row < c0 || row >= c1) continue;  // no sequence's row
      in = row - c0;
    }
    const long at = __ldg(c.lengths + b) + in;
    if (at - in < 0 || at >= c.cap) {
      set_err(c.err, PACK3D_DEVERR_LENGTHS);
      continue;
    }
    const long to = pool_row(c, c.table + (size_t)b * c.max_pages, (int)at);
    if (to < 0) continue;
    ((uint4*)c.k_pages)[to * chunks + chunk] = __ldg(k + i);
    ((uint4*)c.v_pages)[to * chunks + chunk] = __ldg(v + i);
  }
  // Wrong offsets that no row has met.
  if (cu)
    for (long b = blockIdx.x * (long)blockDim.x + threadIdx.x; b < c.B; b += (long)gridDim.x * blockDim.x) {
      const int c0 = __ldg(cu + b), c1 = __ldg(cu + b + 1);
      if (c0 < 0 || c1 < c0 || c1 > rows) set_err(c.err, PACK3D_DEVERR_LENGTHS);
    }
}

// ---- eviction -----------------------------------------------------------------
// Select: one CTA per sequence.  The weights become 32-bit keys whose unsigned
// order is the weights' order (kept in shared memory as far as they fit); the
// key of the last slot that stays is found by a radix search from the top
// digit down (11, 11 and 10 bits: 11 bits of a float's top tell close weights
// apart, so the bins' counters are not all one, and three histograms are
// enough).  Then every warp counts, over its own run of slots, those that stay
// for sure and those that equal that key, one scan over the warps turns the
// counts into places, and a second walk writes the kept slots in order: of the
// equal ones the first few stay.  The slots of one sequence are little to read
// (8,192: 32 KiB); bound by the chain of passes and barriers.  One sequence of
// 1,400 slots cut to 1,024: 8.4 us with the move, 16 of 6,000 to 8,055 cut to
// 4,096: 21.7 us (67 MB moved; four digits of 8 bits: 24.5 and 40 us).
constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32, kBins = 2048;
constexpr int kSelKeys = 40 * 1024;      // keys held in shared memory, at most

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;                                 // NaN: below every number
  const uint32_t u = __float_as_uint(w + 0.f);           // -0 becomes 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum of x over the lanes before this one, and of all lanes.
__device__ __forceinline__ int lanes_before(int x, int* total) {
  int incl = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, d);
    if ((int)(threadIdx.x & 31) >= d) incl += up;
  }
  *total = __shfl_sync(0xffffffffu, incl, 31);
  return incl - x;
}

__global__ void __launch_bounds__(kSelThreads) cache_select_kernel(const Cache c, const float* __restrict__ weights,
                                                                   int budget, int recent, int new_cap, int held,
                                                                   int32_t* __restrict__ kept,
                                                                   float* __restrict__ new_weights,
                                                                   int32_t* __restrict__ new_lengths) {
  extern __shared__ uint32_t keys[];                     // `held` of them
  __shared__ uint32_t hist[kBins];
  __shared__ int s_need;
  __shared__ uint32_t s_prefix;
  __shared__ int2 warp_count[kSelWarps];
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  let_next_begin();
  const int n = cached(c, b);
  const float* w = weights + (size_t)b * c.cap;
  int32_t* kb = kept + (size_t)b * budget;
  float* nw = new_weights + (size_t)b * new_cap;
  const int m = min(n, budget);
  if (tid == 0) new_lengths[b] = m;
  for (int i = m + tid; i < new_cap; i += kSelThreads) nw[i] = 0.f;
  for (int i = m + tid; i < budget; i += kSelThreads) kb[i] = -1;
  if (n <= budget) {
    for (int i = tid; i < n; i += kSelThreads) {
      kb[i] = i;
      nw[i] = w[i];
    }
    return;
  }
  // n > budget >= sinks + recent: the slots [lo, hi) compete for `places`.
  const int lo = c.sinks, hi = n - recent, places = budget - c.sinks - recent;
  for (int i = tid; i < min(n, held); i += kSelThreads) keys[i] = weight_key(__ldg(w + i));
  auto key_of = [&](int i) { return i < held ? keys[i] : weight_key(__ldg(w + i)); };
  if (tid == 0) {
    s_need = places;
    s_prefix = 0;
  }
  if (places > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
      hist[tid] = 0;
      hist[tid + kSelThreads] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix, mask = pass == 0 ? 0u : 0xffffffffu << (shift + bits);
      const int need = s_need;
      for (int i = lo + tid; i < hi; i += kSelThreads) {
        const uint32_t key = key_of(i);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      // From the largest digit down: thread t has the digits top, top - 1.
      const int top = kBins - 1 - 2 * tid, a = hist[top], d = hist[top - 1];
      int all;
      int before = lanes_before(a + d, &all);
      if (lane == 31) warp_count[warp].x = all;
      __syncthreads();
      int others;
      const int mine = lanes_before(warp_count[lane].x, &others);
      before += __shfl_sync(0xffffffffu, mine, warp);
      // The digit at which the places run out.
      if (before < need && before + a + d >= need) {
        const bool second = before + a < need;
        s_need = need - before - (second ? a : 0);
        s_prefix = prefix | ((uint32_t)(second ? top - 1 : top) << shift);
      }
      __syncthreads();
    }
  } else {
    __syncthreads();
  }
  const uint32_t last = s_prefix;
  const int equal_places = places > 0 ? s_need : 0;
  // Warp `warp` walks the slots [begin, end), 32 at a time.
  const int per = ((n + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int begin = min(n, warp * per), end = min(n, begin + per);
  auto look = [&](int i, bool* sure, bool* equal) {
    *sure = *equal = false;
    if (i >= end) return;
    if (i < lo || i >= hi) *sure = true;
    else if (places > 0) {
      const uint32_t key = key_of(i);
      *sure = key > last;
      *equal = key == last;
    }
  };
  int sure_n = 0, equal_n = 0;
  for (int i0 = begin; i0 < end; i0 += 32) {
    bool sure, equal;
    look(i0 + lane, &sure, &equal);
    sure_n += __popc(__ballot_sync(0xffffffffu, sure));
    equal_n += __popc(__ballot_sync(0xffffffffu, equal));
  }
  if (lane == 0) warp_count[warp] = make_int2(sure_n, equal_n);
  __syncthreads();
  int total;
  int sure_at = __shfl_sync(0xffffffffu, lanes_before(warp_count[lane].x, &total), warp);
  int equal_at = __shfl_sync(0xffffffffu, lanes_before(warp_count[lane].y, &total), warp);
  for (int i0 = begin; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    bool sure, equal;
    look(i, &sure, &equal);
    const uint32_t sb = __ballot_sync(0xffffffffu, sure), eb = __ballot_sync(0xffffffffu, equal);
    const uint32_t below = (1u << lane) - 1u;
    const int e = equal_at + __popc(eb & below);         // equal slots before this one
    const int at = sure_at + __popc(sb & below) + min(e, equal_places);
    if (sure || (equal && e < equal_places)) {
      kb[at] = i;
      nw[at] = __ldg(w + i);
    }
    sure_at += __popc(sb);
    equal_at += __popc(eb);
  }
}

// Copies the kept rows to the new pages: one thread per 16-byte chunk of a key
// and a value row.
__global__ void __launch_bounds__(256) cache_move_kernel(const Cache c, const int32_t* kept, int budget,
                                                         const int32_t* __restrict__ new_table, int new_max_pages,
                                                         int chunks) {
  const long total = (long)budget * chunks;
  const int b = blockIdx.y;
  Cache to = c;
  to.max_pages = new_max_pages;
  wait_for_last();
  for (long i = blockIdx.x * (long)blockDim.x + threadIdx.x; i < total; i += (long)gridDim.x * blockDim.x) {
    const int slot = (int)(i / chunks), chunk = (int)(i - (long)slot * chunks);
    const int from = kept[(size_t)b * budget + slot];
    if (from < 0) continue;
    const long src = pool_row(c, c.table + (size_t)b * c.max_pages, from);
    const long dst = pool_row(to, new_table + (size_t)b * new_max_pages, slot);
    if (src < 0 || dst < 0) continue;
    uint4* k = (uint4*)c.k_pages;
    uint4* v = (uint4*)c.v_pages;
    const uint4 a = k[src * chunks + chunk], d = v[src * chunks + chunk];
    k[dst * chunks + chunk] = a;
    v[dst * chunks + chunk] = d;
  }
}

}  // namespace

cudaError_t launch_cache_append(const Cache& c, const int32_t* cu, long rows, const void* k, const void* v,
                                cudaStream_t st) {
  const int chunks = c.Hkv * kDh * c.elem_bytes / 16;
  const long want = (rows * chunks + 255) / 256;
  const unsigned grid = (unsigned)min(want, 148L * 16);
  cache_append_kernel<<<grid, 256, 0, st>>>(c, cu, rows, (const uint4*)k, (const uint4*)v, chunks);
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const Cache& c, const float* weights, int budget, int recent,
                               const int32_t* new_table, int new_max_pages, int32_t* kept, float* new_weights,
                               int32_t* new_lengths, cudaStream_t st) {
  const int held = min(c.cap, kSelKeys);
  cudaError_t e = cudaFuncSetAttribute(cache_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4);
  if (e != cudaSuccess) return e;
  cache_select_kernel<<<c.B, kSelThreads, held * 4, st>>>(c, weights, budget, recent, new_max_pages * c.page, held,
                                                          kept, new_weights, new_lengths);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int chunks = c.Hkv * kDh * c.elem_bytes / 16;
  const long want = ((long)budget * chunks + 255) / 256;
  const dim3 grid((unsigned)min(want, 148L * 16), c.B);
  return launch_behind(cache_move_kernel, grid, 256, 0, st, 1, c, kept, budget, new_table, new_max_pages, chunks);
}

}  // namespace seq
}  // namespace pack3d
