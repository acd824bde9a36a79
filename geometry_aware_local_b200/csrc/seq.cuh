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
// The operators from their definition, one row by one warp, in float: a key that
// is not visible is never read.  Eight lanes (float: 16) share a key's row, 16
// bytes each, so that a load of the warp is of four (two) whole rows; the groups of
// lanes keep sums of their own, joined at the end.

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

// This lane's part of the rows: the dims x .. x + N - 1 of every R-th row from u on.
template <typename T>
struct Part32 {
  static constexpr int N = Elem<T>::kPerChunk, L = kDh / N, R = 32 / L;
  int x, u;
  __device__ __forceinline__ Part32() : x((threadIdx.x & 31) % L * N), u((threadIdx.x & 31) / L) {}
  static __device__ __forceinline__ void floats(const uint4& c, float* f) { chunk_to_float(c, f, T()); }
  // <a, b> of the group's rows.
  static __device__ __forceinline__ float dot(const float* a, const float* b) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) s = fmaf(a[e], b[e], s);
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
  }
  // Sums of the groups' values, in every group.
  template <int n>
  static __device__ __forceinline__ void join(float (&f)[n]) {
#pragma unroll
    for (int d = L; d < 32; d <<= 1)
#pragma unroll
      for (int e = 0; e < n; ++e) f[e] += __shfl_xor_sync(0xffffffffu, f[e], d);
  }
  static __device__ __forceinline__ uint32_t join_bits(uint32_t m) {
#pragma unroll
    for (int d = L; d < 32; d <<= 1) m |= __shfl_xor_sync(0xffffffffu, m, d);
    return m;
  }
  // Which of the lane's dims are not finite, and which are NaNs.
  static __device__ __forceinline__ uint32_t odd(const float* f) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) m |= (uint32_t)!(fabsf(f[e]) < INFINITY) << e;
    return m;
  }
  static __device__ __forceinline__ uint32_t nans(const float* f) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) m |= (uint32_t)(f[e] != f[e]) << e;
    return m;
  }
  __device__ __forceinline__ void store(T* row, const float* f) const {
    if (u == 0) stg16(row + x, float_to_chunk(f, T()));
  }
};

// The keys that position p sees, by number: first the sinks, then the window.
struct Visible {
  int low, sinks, n;
  __device__ __forceinline__ Visible(const Win& w, int p) {
    low = window_low(w, p);
    sinks = min(w.sinks, low);
    n = p < 0 ? 0 : sinks + p + 1 - low;
  }
  __device__ __forceinline__ int key(int i) const { return i < sinks ? i : i - sinks + low; }
};

// Output (and log-sum-exp) of head h of query row r.
template <typename T>
__device__ __noinline__ void out_row(const Win& w, const Tile& s, int r, int h) {
  using P = Part32<T>;
  constexpr int N = P::N, kAhead = 4;           // rows of a group on their way
  const P me;
  const Visible see(w, position(s, r));
  const size_t at = (size_t)(s.q0 + r) * w.Hq + h, first = ((size_t)s.k0 * w.Hkv + (h >> w.gshift)) * kDh + me.x;
  const T *k = (const T*)w.k + first, *v = (const T*)w.v + first;
  const size_t step = (size_t)w.Hkv * kDh;
  const float scale = w.scale;
  float q[N], o[N], m = -INFINITY, l[1] = {0.f};
  P::floats(ldg16((const T*)w.q + at * kDh + me.x), q);
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = 0.f;
#pragma unroll 1
  for (int i0 = me.u; i0 - me.u < see.n; i0 += kAhead * P::R) {
    uint4 kc[kAhead], vc[kAhead];
#pragma unroll
    for (int t = 0; t < kAhead; ++t) {
      const size_t key = see.key(min(i0 + t * P::R, see.n - 1)) * step;
      kc[t] = ldg16(k + key);
      vc[t] = ldg16(v + key);
    }
    float y[kAhead], top = m;
#pragma unroll
    for (int t = 0; t < kAhead; ++t) {
      float f[N];
      P::floats(kc[t], f);
      y[t] = P::dot(q, f) * scale;
      if (i0 + t * P::R >= see.n) y[t] = -INFINITY;
      top = fmaxf(top, y[t]);
    }
    const float f = m == top ? 1.f : expf(m - top);
    m = top;
    l[0] *= f;
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] *= f;
#pragma unroll
    for (int t = 0; t < kAhead; ++t) {
      if (i0 + t * P::R >= see.n) break;
      // A row whose scores so far are all -infinity keeps weight 0 for them.
      const float p = y[t] == -INFINITY ? 0.f : expf(y[t] - top);
      float c[N];
      P::floats(vc[t], c);
      l[0] += p;
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = fmaf(p, c[e], o[e]);
    }
  }
  float top = m;
#pragma unroll
  for (int d = P::L; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const float f = m == top ? 1.f : expf(m - top);
  l[0] *= f;
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] *= f;
  P::join(l);
  P::join(o);
  const float inv = l[0] > 0.f ? 1.f / l[0] : (l[0] == 0.f ? 0.f : l[0]);
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] *= inv;
  me.store((T*)w.out + at * kDh, o);
  if (w.lse && (threadIdx.x & 31) == 0) w.lse[at] = top + logf(l[0]);
}

// dq of head h of query row r; delta[at] is up to date.
template <typename T>
__device__ __noinline__ void dq_row(const Win& w, const Tile& s, int r, int h) {
  using P = Part32<T>;
  constexpr int N = P::N, kAhead = 2;
  const P me;
  const Visible see(w, position(s, r));
  const size_t at = (size_t)(s.q0 + r) * w.Hq + h, first = ((size_t)s.k0 * w.Hkv + (h >> w.gshift)) * kDh + me.x;
  const T *k = (const T*)w.k + first, *v = (const T*)w.v + first;
  const size_t step = (size_t)w.Hkv * kDh;
  const float lse = w.lse[at], delta = w.delta[at], scale = w.scale;
  float q[N], d[N], acc[N];
  P::floats(ldg16((const T*)w.q + at * kDh + me.x), q);
  P::floats(ldg16((const T*)w.dout + at * kDh + me.x), d);
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int i0 = me.u; i0 - me.u < see.n; i0 += kAhead * P::R) {
    uint4 kc[kAhead], vc[kAhead];
#pragma unroll
    for (int t = 0; t < kAhead; ++t) {
      const size_t key = see.key(min(i0 + t * P::R, see.n - 1)) * step;
      kc[t] = ldg16(k + key);
      vc[t] = ldg16(v + key);
    }
#pragma unroll
    for (int t = 0; t < kAhead; ++t) {
      float a[N], b[N];
      P::floats(kc[t], a);
      P::floats(vc[t], b);
      const float p = expf(P::dot(q, a) * scale - lse), ds = p * (P::dot(d, b) - delta);
      if (i0 + t * P::R < see.n) {
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = fmaf(ds, a[e], acc[e]);
      }
    }
  }
  P::join(acc);
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] *= scale;
  me.store((T*)w.dq + at * kDh, acc);
}

// The query rows or keys of a sequence that one tile of any of the kernels takes at most.
constexpr int kTileRows = 128;

// The tiled kernels multiply a hidden key's value (or, for a key's gradients, a
// query's row that does not see it) by a zero probability; where that value is a
// NaN or an infinity the product is a NaN.  So a row of results that is not finite
// is formed again from what it sees, here - but only if something hidden that its
// tile has read, a few hundred rows at most, is not finite in the same dims, and
// what it sees does not make them NaN anyway: a NaN that is the right answer costs
// a look at those rows, not at all that the row sees.

// Whether the rows [from, to) of `base`, `step` apart, are not finite in one of this
// lane's dims of `odd`.
template <typename T>
__device__ __forceinline__ bool met(const Part32<T>& me, uint32_t odd, const T* base, size_t step, int from, int to) {
  uint32_t m = 0;
#pragma unroll 8
  for (int j = from + me.u; j < to; j += Part32<T>::R) {
    float f[Part32<T>::N];
    Part32<T>::floats(ldg16(base + j * step + me.x), f);
    m |= Part32<T>::odd(f);
  }
  return (m & odd) != 0;
}
// The lane's part of a row of results that this kernel has written.
template <typename T>
__device__ __forceinline__ void written(const Part32<T>& me, const T* row, float* f) {
  Part32<T>::floats(*reinterpret_cast<const uint4*>(row + me.x), f);
}

// Whether a hidden key of `keys` (of head g's first key on) that the tile of query
// row r has read is not finite in a dim of `odd`.
template <typename T>
__device__ __forceinline__ bool hidden_key(const Win& w, const Tile& s, int r, const Part32<T>& me, const T* keys,
                                           uint32_t odd) {
  const int tokens = kTileRows >> w.gshift, r0 = r & ~(tokens - 1);
  const int p = position(s, r), p1 = position(s, min(s.lq, r0 + tokens) - 1), low = window_low(w, p);
  const size_t step = (size_t)w.Hkv * kDh;
  int lo = window_low(w, max(position(s, r0), 0));
  if (lo <= 64) lo = 0;                         // the sinks' columns reach it: one range from key 0
  bool hit = met(me, odd, keys, step, max(p + 1, 0), min(p1 + 32, s.lk)) || met(me, odd, keys, step, lo, low);
  if (w.sinks > 0) hit |= met(me, odd, keys, step, w.sinks, min(64, low));
  return __any_sync(0xffffffffu, hit);
}

// out_row of a result that is not finite, whose denominator is a number.
template <typename T>
__device__ __noinline__ void out_again(const Win& w, const Tile& s, int r, int h) {
  using P = Part32<T>;
  constexpr int N = P::N, kAhead = 8;
  const P me;
  const T* v = (const T*)w.v + ((size_t)s.k0 * w.Hkv + (h >> w.gshift)) * kDh;
  float f[N];
  written(me, (const T*)w.out + ((size_t)(s.q0 + r) * w.Hq + h) * kDh, f);
  const uint32_t odd = P::odd(f);
  if (!hidden_key(w, s, r, me, v, odd)) return;
  // Visible values that are not finite, from the nearest key back: a NaN, or
  // infinities of both signs, leave a NaN whatever their weights are.
  const Visible see(w, position(s, r));
#pragma unroll
  for (int e = 0; e < N; ++e) f[e] = 0.f;
#pragma unroll 1
  for (int end = see.n - 1 - me.u; end + me.u >= 0; end -= kAhead * P::R) {
    uint4 c[kAhead];
#pragma unroll
    for (int t = 0; t < kAhead; ++t) c[t] = ldg16(v + see.key(max(end - t * P::R, 0)) * ((size_t)w.Hkv * kDh) + me.x);
#pragma unroll
    for (int t = 0; t < kAhead; ++t) {
      float y[N];
      P::floats(c[t], y);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (!(fabsf(y[e]) < INFINITY)) f[e] += y[e];
    }
    if (__all_sync(0xffffffffu, (odd & ~P::join_bits(P::nans(f))) == 0)) return;
  }
  out_row<T>(w, s, r, h);
}

// dq_row of a result that is not finite.  (Where the row sees a NaN its
// log-sum-exp or its delta is one.)
template <typename T>
__device__ __noinline__ void dq_again(const Win& w, const Tile& s, int r, int h) {
  const Part32<T> me;
  const size_t at = (size_t)(s.q0 + r) * w.Hq + h;
  const float lse = w.lse[at], delta = w.delta[at];
  if (position(s, r) >= 0 && (lse != lse || delta != delta)) return;
  float f[Part32<T>::N];
  written(me, (const T*)w.dq + at * kDh, f);
  const T* k = (const T*)w.k + ((size_t)s.k0 * w.Hkv + (h >> w.gshift)) * kDh;
  if (hidden_key(w, s, r, me, k, Part32<T>::odd(f))) dq_row<T>(w, s, r, h);
}

// dk and dv of key j of key head g, over every query that sees it.  again: of a
// result that is not finite, as above (a query row that sees a NaN has one in its
// log-sum-exp, its delta or its own values).
template <typename T>
__device__ __noinline__ void dkv_row(const Win& w, const Tile& s, int j, int g, bool again) {
  using P = Part32<T>;
  constexpr int N = P::N, kAhead = 2;
  const P me;
  const int shift = s.lk - s.lq;                // position minus row
  const size_t at = ((size_t)(s.k0 + j) * w.Hkv + g) * kDh, heads = (size_t)w.Hq * kDh;
  const size_t row0 = (size_t)s.q0 * w.Hq + (g << w.gshift);
  const T *q = (const T*)w.q + row0 * kDh, *dout = (const T*)w.dout + row0 * kDh;
  const int first = max(0, j - shift);
  const bool windowed = w.window > 0 && j >= w.sinks;
  const int last = windowed ? min(s.lq - 1, j + w.window - 1 - shift) : s.lq - 1;
  uint32_t odd_k = 0, odd_v = 0;
  if (again) {
    float f[N];
    written(me, (const T*)w.dk + at, f);
    odd_k = P::odd(f);
    written(me, (const T*)w.dv + at, f);
    odd_v = P::odd(f);
    // Rows that the key's tile has read besides: before the first that sees the key,
    // and behind the last (for a sink behind those that its own tile takes), to the
    // end of a step of at most 64.
    const int j0 = j & ~(kTileRows - 1), beyond = min(j0 + kTileRows, s.lk) - 1 + w.window - shift;
    const int before = max(0, j0 - shift), before_end = min(first, s.lq);
    const int behind = max(0, windowed ? last + 1 : beyond), behind_end = w.window > 0 ? min(s.lq, beyond + 64) : 0;
    bool hit = false;
#pragma unroll 1
    for (int h = 0; h < w.G; ++h) {
      const T *qh = q + h * kDh, *dh = dout + h * kDh;
      hit |= met(me, odd_k, qh, heads, before, before_end) || met(me, odd_v, dh, heads, before, before_end) ||
             met(me, odd_k, qh, heads, behind, behind_end) || met(me, odd_v, dh, heads, behind, behind_end);
    }
    if (!__any_sync(0xffffffffu, hit)) return;
  }
  float k[N], v[N], ak[N], av[N];
  P::floats(ldg16((const T*)w.k + at + me.x), k);
  P::floats(ldg16((const T*)w.v + at + me.x), v);
#pragma unroll
  for (int e = 0; e < N; ++e) ak[e] = av[e] = 0.f;
  const float scale = w.scale;
  const int n = last >= first ? (last - first + 1) << w.gshift : 0;      // (row, head) pairs
  auto place = [&](int i) { return (size_t)(first + (i >> w.gshift)) * w.Hq + (i & (w.G - 1)); };
  int turn = 0;
#pragma unroll 1
  for (int i0 = me.u; i0 - me.u < n; i0 += kAhead * P::R, ++turn) {
    uint4 qc[kAhead], dc[kAhead];
#pragma unroll
    for (int t = 0; t < kAhead; ++t) {
      const size_t row = place(min(i0 + t * P::R, n - 1));
      qc[t] = ldg16(q + row * kDh + me.x);
      dc[t] = ldg16(dout + row * kDh + me.x);
    }
#pragma unroll
    for (int t = 0; t < kAhead; ++t) {
      const size_t row = row0 + place(min(i0 + t * P::R, n - 1));
      float a[N], b[N];
      P::floats(qc[t], a);
      P::floats(dc[t], b);
      float delta;
      if constexpr (sizeof(T) == 4) {           // both sides run at once: there may be no delta yet
        float c[N];
        P::floats(ldg16((const T*)w.out + row * kDh + me.x), c);
        delta = P::dot(b, c);
      } else {
        delta = w.delta[row];
      }
      const float p = expf(P::dot(a, k) * scale - w.lse[row]), ds = p * (P::dot(b, v) - delta);
      if (i0 + t * P::R < n) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          ak[e] = fmaf(ds, a[e], ak[e]);
          av[e] = fmaf(p, b[e], av[e]);
        }
      }
    }
    // Dims that are NaN stay so, whatever comes; the others are as they were.
    if (again && (turn & 7) == 0) {
      const uint32_t left = (odd_k & ~P::join_bits(P::nans(ak))) | (odd_v & ~P::join_bits(P::nans(av)));
      if (__all_sync(0xffffffffu, left == 0)) {
        written(me, (const T*)w.dk + at, ak);
        written(me, (const T*)w.dv + at, av);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < N; ++e) {
          if ((odd_k >> e) & 1u) ak[e] = NAN;
          if ((odd_v >> e) & 1u) av[e] = NAN;
        }
        me.store((T*)w.dk + at, ak);
        me.store((T*)w.dv + at, av);
        return;
      }
    }
  }
  P::join(ak);
  P::join(av);
#pragma unroll
  for (int e = 0; e < N; ++e) ak[e] *= scale;
  me.store((T*)w.dk + at, ak);
  me.store((T*)w.dv + at, av);
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
