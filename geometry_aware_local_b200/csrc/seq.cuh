// Shared parts of the causal sequence operators (pack3d_seq.h): the resolved
// operator, which keys a query sees, where a CTA's tile lies among the packed
// sequences, and the row-by-row forms of the attention and its gradients.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "pack3d_seq.h"

namespace pack3d {
namespace seq {

// One windowed attention call, resolved on the host.
struct Win {
  const int32_t* cu_q;
  const int32_t* cu_k;
  int B, Tq, Tk;
  int Hq, Hkv, G, gshift;         // G = Hq / Hkv = 1 << gshift
  int window, sinks;
  float scale, scale_log2;        // softmax scale, and times log2(e)
  const void* q;
  const void* k;
  const void* v;
  void* out;                      // backward: the forward's out (read)
  float* lse;                     // nullable in the forward; read by the backward
  const void* dout;
  void* dq;
  void* dk;
  void* dv;
  float* delta;                   // workspace [Tq, Hq]: <dout, out>, the row's sum of P dP
  void* terms;                    // workspace, bf16 [2][Tq, Hq, 8]: -lse / scale, then -delta, in three pieces
  float* part;                    // workspace: partial gradients of the sink rows
  int zero_outside;               // rows of no sequence become 0 instead of staying as they were
  int32_t* err;
  unsigned long long wait_ns;
  int stall;
};

// One sequence and a tile of it.
struct Tile {
  int b;          // sequence
  int t, n;       // tile of the sequence, and its tiles
  int q0, lq;     // its query rows: first packed row, count
  int k0, lk;     // its key rows
};

// Position of the query at row r of its sequence among the sequence's keys.
__device__ __forceinline__ int position(const Tile& s, int r) { return s.lk - s.lq + r; }
// First key the window of position p reaches.
__device__ __forceinline__ int window_low(const Win& w, int p) {
  return w.window > 0 && p >= w.window ? p - w.window + 1 : 0;
}
__device__ __forceinline__ bool sees(const Win& w, int p, int j) {
  return j <= p && (j >= window_low(w, p) || j < w.sinks);
}

// Which CTA takes which piece of which sequence, where every `per` rows (a power
// of two) of a sequence are a piece at most: the pieces of sequence b are the
// CTAs base(b) .. base(b) + n - 1 with base(b) = cu[b] / per + b.  Since
// base(b + 1) - base(b) >= ceil((cu[b + 1] - cu[b]) / per), no two sequences
// share a CTA, some CTAs have no piece, and a piece is found without adding up
// the counts of the sequences before it.
__device__ __forceinline__ int log2_of(int per) { return __ffs(per) - 1; }

// Whether the offsets of sequence b are out of order or out of range.
__device__ __forceinline__ bool off_range(const Win& w, int q0, int q1, int k0, int k1) {
  return q0 < 0 || q1 < q0 || q1 > w.Tq || k0 < 0 || k1 < k0 || k1 > w.Tk;
}
__device__ __forceinline__ bool off_range(const Win& w, int b) {
  return off_range(w, __ldg(w.cu_q + b), __ldg(w.cu_q + b + 1), __ldg(w.cu_k + b), __ldg(w.cu_k + b + 1));
}

// The piece of CTA number x, `per` rows of queries (or of keys with over_keys)
// a piece and count(lq, lk) of them in a sequence of lq queries and lk keys:
// one warp halves the sequences by 32 until 32 are left, one a lane, whose
// offsets it checks.  All 32 lanes call it and get the same answer: whether
// there is such a piece, never with offsets that are wrong; *bad: some of those
// looked at are.
template <typename Count>
__device__ __forceinline__ bool find_piece(const Win& w, int x, int per, bool over_keys, Count count, Tile* out,
                                           bool* bad) {
  const int lane = threadIdx.x & 31, shift = log2_of(per);
  const int32_t* cu = over_keys ? w.cu_k : w.cu_q;
  int lo = 0, hi = w.B;
#pragma unroll 1
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) >> 5, b = lo + lane * step;
    const uint32_t at = __ballot_sync(0xffffffffu, lane == 0 || (b < hi && (__ldg(cu + b) >> shift) + b <= x));
    lo += (at == 0xffffffffu ? 31 : __ffs(~at) - 2) * step;
    hi = min(hi, lo + step);
  }
  const int b = lo + lane;
  const bool in = b < hi;
  const int q0 = in ? __ldg(w.cu_q + b) : 0, q1 = in ? __ldg(w.cu_q + b + 1) : 0;
  const int k0 = in ? __ldg(w.cu_k + b) : 0, k1 = in ? __ldg(w.cu_k + b + 1) : 0;
  const bool off = in && off_range(w, q0, q1, k0, k1);
  *bad = __any_sync(0xffffffffu, off);
  const int n = !in || off ? 0 : count(q1 - q0, k1 - k0);
  const int t = x - (((over_keys ? k0 : q0) >> shift) + b);
  const uint32_t hit = __ballot_sync(0xffffffffu, t >= 0 && t < n);
  if (!hit || *bad) return false;
  const int src = __ffs(hit) - 1;
  out->b = lo + src;
  out->t = __shfl_sync(0xffffffffu, t, src);
  out->n = __shfl_sync(0xffffffffu, n, src);
  out->q0 = __shfl_sync(0xffffffffu, q0, src);
  out->lq = __shfl_sync(0xffffffffu, q1 - q0, src);
  out->k0 = __shfl_sync(0xffffffffu, k0, src);
  out->lk = __shfl_sync(0xffffffffu, k1 - k0, src);
  return true;
}

// The tile of CTA number x: `per` rows of queries, or of keys with over_keys, a
// tile; every sequence starts a new one.  The query tiles' first CTAs look at
// all offsets between them.
__device__ __forceinline__ bool find_tile(const Win& w, int x, int per, bool over_keys, Tile* out, bool* bad) {
  auto count = [=](int lq, int lk) { return ((over_keys ? lk : lq) + per - 1) / per; };
  const bool found = find_piece(w, x, per, over_keys, count, out, bad);
  if (over_keys || w.B <= 32 || x > w.B / 32) return found;
  const int b = 32 * x + (threadIdx.x & 31);
  *bad |= __any_sync(0xffffffffu, b < w.B && off_range(w, b));
  return found && !*bad;
}

// Grid size that covers every tile whatever the offsets are, with a last CTA
// that has none: base(B) <= rows / per + B.
inline long tile_grid(long rows, int per, int batch) { return rows / per + batch + 1; }

// Sets the rows outside [cu[0], cu[B]) of a tensor of T rows of `words` 32-bit
// words to `value`: the work of the CTAs x before base(0) and from base(B) on
// of a tile_grid of `grid`, `warps` a CTA.  Other CTAs return.
__device__ __forceinline__ void fill_outside(const Win& w, const int32_t* cu, int T, int per, int x, int grid,
                                             int warps, void* base, int words, uint32_t value) {
  const int shift = log2_of(per), c0 = __ldg(cu), c1 = __ldg(cu + w.B);
  if (c0 < 0 || c1 < c0 || c1 > T) return;
  const int front = c0 >> shift, back = (c1 >> shift) + w.B;
  if (x >= front && x < back) return;
  const long part = (long)(x < front ? x : front + x - back) * warps + (threadIdx.x >> 5);
  const long parts = (long)(front + grid - back) * warps;
  const long before = (long)c0 * words, total = before + (long)(T - c1) * words;
  uint32_t* p = (uint32_t*)base;
#pragma unroll 1
  for (long i = part * 32 + (threadIdx.x & 31); i < total; i += parts * 32)
    p[i < before ? i : (long)c1 * words + (i - before)] = value;
}

// Launches that follow one another in a call overlap: the second is put in place
// while the first's last CTAs run (they say so as they begin), and each of its
// CTAs waits, before it touches what the first writes or returns, for the first
// to end.  cluster: CTAs of a cluster along x.
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
inline cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, int cluster,
                                 A... args) {
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = cluster;
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attrs;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// SMs of the current device.
inline int sm_count() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 148;
}

// ---- row by row -----------------------------------------------------------------
// The operators from their definition, one row by one warp, in float: lane l
// holds the dims 2l and 2l+1, a key that is not visible is never read.  The
// tiled kernels multiply a hidden key's value by a zero probability; where that
// value is a NaN or an infinity the product is a NaN, and the row is computed
// again here.

template <typename T> __device__ __forceinline__ float2 load2(const T* row);
template <> __device__ __forceinline__ float2 load2<float>(const float* row) {
  return __ldg(reinterpret_cast<const float2*>(row) + (threadIdx.x & 31));
}
template <> __device__ __forceinline__ float2 load2<__nv_bfloat16>(const __nv_bfloat16* row) {
  const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(row) + (threadIdx.x & 31));
  return make_float2(bf16_lo(u), bf16_hi(u));
}
__device__ __forceinline__ void store2(float* row, float2 f) {
  reinterpret_cast<float2*>(row)[threadIdx.x & 31] = f;
}
__device__ __forceinline__ void store2(__nv_bfloat16* row, float2 f) {
  reinterpret_cast<uint32_t*>(row)[threadIdx.x & 31] = pack_bf16x2(f.x, f.y);
}
__device__ __forceinline__ float dot2(float2 a, float2 b) {
  float s = fmaf(a.x, b.x, a.y * b.y);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return s;
}

// Calls f(j) for every key j that position p sees, in order.
template <typename F>
__device__ __forceinline__ void for_visible(const Win& w, int p, F f) {
  const int low = window_low(w, p);
#pragma unroll 1
  for (int j = 0; j < min(w.sinks, low); ++j) f(j);
#pragma unroll 1
  for (int j = low; j <= p; ++j) f(j);
}

// Output (and log-sum-exp) of head h of query row r.
template <typename T>
__device__ __noinline__ void out_row(const Win& w, const Tile& s, int r, int h) {
  const int g = h >> w.gshift, p = position(s, r);
  const size_t at = (size_t)(s.q0 + r) * w.Hq + h;
  const T* k = (const T*)w.k + ((size_t)s.k0 * w.Hkv + g) * kDh;
  const T* v = (const T*)w.v + ((size_t)s.k0 * w.Hkv + g) * kDh;
  const size_t step = (size_t)w.Hkv * kDh;
  const float2 q = load2((const T*)w.q + at * kDh);
  float m = -INFINITY, l = 0.f;
  float2 o = make_float2(0.f, 0.f);
  for_visible(w, p, [&](int j) {
    const float x = dot2(q, load2(k + j * step)) * w.scale;
    const float2 vv = load2(v + j * step);
    float f = 1.f;
    if (x > m) {
      f = expf(m - x);
      m = x;
    }
    // A row whose scores so far are all -infinity keeps weight 0 for them.
    const float e = x == -INFINITY ? 0.f : expf(x - m);
    l = l * f + e;
    o.x = fmaf(e, vv.x, o.x * f);
    o.y = fmaf(e, vv.y, o.y * f);
  });
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  store2((T*)w.out + at * kDh, make_float2(o.x * inv, o.y * inv));
  if (w.lse && (threadIdx.x & 31) == 0) w.lse[at] = m + logf(l);
}

// P and dS of one visible pair, from the row's q, dout, lse and delta.
__device__ __forceinline__ float2 pair_grad(const Win& w, float2 q, float2 d, float lse, float delta, float2 k,
                                            float2 v) {
  const float p = expf(dot2(q, k) * w.scale - lse);
  return make_float2(p, p * (dot2(d, v) - delta));
}

// dq of head h of query row r; delta[at] is up to date.
template <typename T>
__device__ __noinline__ void dq_row(const Win& w, const Tile& s, int r, int h) {
  const int g = h >> w.gshift, p = position(s, r);
  const size_t at = (size_t)(s.q0 + r) * w.Hq + h;
  const T* k = (const T*)w.k + ((size_t)s.k0 * w.Hkv + g) * kDh;
  const T* v = (const T*)w.v + ((size_t)s.k0 * w.Hkv + g) * kDh;
  const size_t step = (size_t)w.Hkv * kDh;
  const float2 q = load2((const T*)w.q + at * kDh), d = load2((const T*)w.dout + at * kDh);
  const float lse = w.lse[at], delta = w.delta[at];
  float2 acc = make_float2(0.f, 0.f);
  for_visible(w, p, [&](int j) {
    const float2 kk = load2(k + j * step);
    const float2 pd = pair_grad(w, q, d, lse, delta, kk, load2(v + j * step));
    acc.x = fmaf(pd.y, kk.x, acc.x);
    acc.y = fmaf(pd.y, kk.y, acc.y);
  });
  store2((T*)w.dq + at * kDh, make_float2(acc.x * w.scale, acc.y * w.scale));
}

// dk and dv of key j of key head g, over every query that sees it.
template <typename T>
__device__ __noinline__ void dkv_row(const Win& w, const Tile& s, int j, int g) {
  const size_t at = (size_t)(s.k0 + j) * w.Hkv + g;
  const float2 k = load2((const T*)w.k + at * kDh), v = load2((const T*)w.v + at * kDh);
  float2 ak = make_float2(0.f, 0.f), av = ak;
  const int first = max(0, j - (s.lk - s.lq));
  int last = s.lq - 1;
  if (w.window > 0 && j >= w.sinks) last = min(last, j + w.window - 1 - (s.lk - s.lq));
  for (int r = first; r <= last; ++r)
    for (int h = g << w.gshift; h < (g + 1) << w.gshift; ++h) {
      const size_t row = (size_t)(s.q0 + r) * w.Hq + h;
      const float2 q = load2((const T*)w.q + row * kDh), d = load2((const T*)w.dout + row * kDh);
      // (The float kernels run both sides at once: there may be no delta yet.)
      const float delta = sizeof(T) == 4 ? dot2(d, load2((const T*)w.out + row * kDh)) : w.delta[row];
      const float2 pd = pair_grad(w, q, d, w.lse[row], delta, k, v);
      ak.x = fmaf(pd.y, q.x, ak.x);
      ak.y = fmaf(pd.y, q.y, ak.y);
      av.x = fmaf(pd.x, d.x, av.x);
      av.y = fmaf(pd.x, d.y, av.y);
    }
  store2((T*)w.dk + at * kDh, make_float2(ak.x * w.scale, ak.y * w.scale));
  store2((T*)w.dv + at * kDh, av);
}

// delta[at] = <dout, out> of one row, by one warp.
template <typename T>
__device__ __forceinline__ void delta_row(const Win& w, size_t at) {
  const float d = dot2(load2((const T*)w.dout + at * kDh), load2((const T*)w.out + at * kDh));
  if ((threadIdx.x & 31) == 0) w.delta[at] = d;
}

// ---- launchers (k_window.cu, k_cache.cu, k_cache_attn.cu) -----------------------

// The tensor-core kernels (bf16; at least one key row and one query row).
cudaError_t launch_window_attn_tc(const Win& w, cudaStream_t st);
cudaError_t launch_window_bwd_tc(const Win& w, cudaStream_t st);
// The float kernels.
cudaError_t launch_window_attn_f32(const Win& w, cudaStream_t st);
cudaError_t launch_window_bwd_f32(const Win& w, cudaStream_t st);
// Bytes of Win::part for a call of this size.
size_t window_bwd_part_bytes(const Win& w, int dtype);
cudaError_t launch_window_attn(const Win& w, int dtype, cudaStream_t st);
cudaError_t launch_window_bwd(const Win& w, int dtype, cudaStream_t st);

// A paged cache call, resolved on the host.
struct Cache {
  int B, Hq, Hkv, G;
  int page, page_shift;
  int max_pages, num_pages, cap;   // cap = max_pages * page
  int window, sinks;
  float scale, scale_log2;
  int elem_bytes;
  const int32_t* table;
  const int32_t* lengths;
  void* k_pages;
  void* v_pages;
  int32_t* err;
};

cudaError_t launch_cache_append(const Cache& c, const int32_t* cu, long rows, const void* k, const void* v,
                                cudaStream_t st);
cudaError_t launch_cache_evict(const Cache& c, const float* weights, int budget, int recent,
                               const int32_t* new_table, int new_max_pages, int32_t* kept, float* new_weights,
                               int32_t* new_lengths, cudaStream_t st);
size_t cache_attn_workspace(int B, int Hq, int Hkv, int cap, bool weights);
cudaError_t launch_cache_attn(const Cache& c, int dtype, const void* q, void* out, float* lse, float* weights,
                              bool accumulate, void* workspace, cudaStream_t st);

// The slots a sequence has, kept inside its capacity.
__device__ __forceinline__ int cached(const Cache& c, int b) {
  const int n = __ldg(c.lengths + b);
  if (n < 0 || n > c.cap) set_err(c.err, PACK3D_DEVERR_LENGTHS);
  return min(max(n, 0), c.cap);
}

// Pool row of slot `at` through a table row, or -1 (and the error bit) for a
// page outside the pool.
__device__ __forceinline__ long pool_row(const Cache& c, const int32_t* row, int at) {
  const int p = __ldg(row + (at >> c.page_shift));
  if (p < 0 || p >= c.num_pages) {
    set_err(c.err, PACK3D_DEVERR_PAGE);
    return -1;
  }
  return ((long)p << c.page_shift) + (at & (c.page - 1));
}

}  // namespace seq
}  // namespace pack3d
