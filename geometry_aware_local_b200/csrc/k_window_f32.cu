// Causal windowed attention of packed sequences and its gradients in float, on
// CUDA cores.
//
// The tiles are those of the tensor-core kernels (rows = (token, query head)
// pairs of one key head's group; key range and sinks; see k_window_tc.cu and
// k_window_bwd_tc.cu), 64 rows by 64 keys.  256 threads hold a 64 x 64 product
// as 4 x 4 values each: thread (ty, tx) = (tid / 16, tid % 16) has the rows
// ty + 16 i and the columns tx + 16 j of S and dP (both operands are read four
// contraction steps at a time, 16 bytes a load, from rows padded to 68 floats),
// and the dims 4 tx .. 4 tx + 3 of O, dQ, dK and dV.  Everything is formed and
// kept in 32 bits, two multiply-adds an instruction.  Bound: the shared-memory
// reads (8 loads of 16 bytes per 64 multiply-adds and thread; 77 % of their
// rate).  128 threads with 8 x 4 values read less, but where a call has few
// tiles their warps are too few.  There the CTAs of a cluster share a tile besides,
// and join what they have through each other's shared memory.  2,050 tokens in
// three sequences, 4 / 2 heads, window 200, one sink: forward 34 us (128 threads, a
// multiply-add an instruction: 42), backward 97 us (166, with the two sides one
// after the other and a CTA a tile).  16,384 tokens, 8 / 2 heads: 0.318 and 1.03 ms.
//
// What is hidden has P = 0; rows that 0 times a NaN or an infinity spoilt are
// computed again (out_again, dq_again, dkv_row), as in the tensor-core kernels.
#include <cooperative_groups.h>

#include "seq_tc.cuh"
#include "window_sinks.cuh"

namespace pack3d {
namespace seq {
namespace {

constexpr int kRows = 64, kKeys = 64, kThreads = 256;
constexpr int kPer = 64 * 16 / kThreads, kSub = kThreads / 16;      // a thread's rows of a product, and their distance
constexpr int kPad = kDh + 4;
constexpr int kTileFloats = 64 * kPad;

typedef float Micro[kPer][4];

__device__ __forceinline__ void zero(Micro c) {
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] = 0.f;
}
__device__ __forceinline__ float4 at4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// c[i][j] += sum_d a[ty + kSub i][d] b[tx + 16 j][d]: both operands' rows run
// along the contraction, even and odd steps apart.
__device__ __forceinline__ void mul_nt(Micro c, const float* a, const float* b) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  float2 e[kPer][4];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) e[i][j] = make_float2(0.f, 0.f);
#pragma unroll 2
  for (int d = 0; d < kDh; d += 4) {
    float4 x[kPer], y[4];
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = at4(a + (ty + kSub * i) * kPad + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = at4(b + (tx + 16 * j) * kPad + d);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        e[i][j] = __ffma2_rn(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), e[i][j]);
        e[i][j] = __ffma2_rn(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), e[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] = e[i][j].x + e[i][j].y;
}
__device__ __forceinline__ void axpy(float* c, float v, float4 y) {
  const float2 p = __ffma2_rn(make_float2(v, v), make_float2(y.x, y.y), make_float2(c[0], c[1]));
  const float2 q = __ffma2_rn(make_float2(v, v), make_float2(y.z, y.w), make_float2(c[2], c[3]));
  c[0] = p.x; c[1] = p.y; c[2] = q.x; c[3] = q.y;
}
// c[i][j] += sum_k a[ty + kSub i][k] b[k][4 tx + j].
__device__ __forceinline__ void mul_nn(Micro c, const float* a, const float* b) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 2
  for (int k = 0; k < 64; k += 4) {
    float4 x[kPer], y[4];
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = at4(a + (ty + kSub * i) * kPad + k);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = at4(b + (k + j) * kPad + 4 * tx);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      axpy(c[i], x[i].x, y[0]);
      axpy(c[i], x[i].y, y[1]);
      axpy(c[i], x[i].z, y[2]);
      axpy(c[i], x[i].w, y[3]);
    }
  }
}
// Row of the product of the transposed operand that c[i] belongs to.
__device__ __forceinline__ int row_tn(int i) { return 4 * (threadIdx.x >> 4) + (i & 3) + 4 * kSub * (i >> 2); }
// c[i][j] += sum_k a[k][row_tn(i)] b[k][4 tx + j].
__device__ __forceinline__ void mul_tn(Micro c, const float* a, const float* b) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 4
  for (int k = 0; k < 64; ++k) {
    const float4 y = at4(b + k * kPad + 4 * tx);
#pragma unroll
    for (int i = 0; i < kPer; i += 4) {
      const float4 x = at4(a + k * kPad + 4 * ty + kSub * i);
      axpy(c[i], x.x, y);
      axpy(c[i + 1], x.y, y);
      axpy(c[i + 2], x.z, y);
      axpy(c[i + 3], x.w, y);
    }
  }
}

// Copies 64 rows of 64 floats into a tile, without waiting: row i is at
// row_of(i), or zeros where that is null.
template <typename RowOf>
__device__ __forceinline__ void load_rows(float* tile, RowOf row_of) {
  const uint32_t base = ptx::smem_u32(tile);
#pragma unroll
  for (int n = 0; n < kPer; ++n) {
    const int i = (threadIdx.x >> 4) + kSub * n, x = threadIdx.x & 15;
    const float* src = row_of(i);
    const uint32_t dst = base + (i * kPad + 4 * x) * 4;
    if (src) ptx::cp_async16(dst, src + 4 * x, 16);
    else ptx::st_shared_v4(dst, 0u, 0u, 0u, 0u);
  }
}
__device__ __forceinline__ void loads_done() {
  ptx::cp_async_commit();
  ptx::cp_async_wait_all();
  __syncthreads();
}

// Query row i of the tile whose first token is r0 (tokens up to r1) of a
// [Tq, Hq, 64] tensor.
__device__ __forceinline__ const float* query_row(const Win& w, const Tile& s, int g, int r0, int r1, const void* t,
                                                  int i) {
  const int r = r0 + (i >> w.gshift);
  if (r > r1) return nullptr;
  return (const float*)t + ((size_t)(s.q0 + r) * w.Hq + (g << w.gshift) + (i & (w.G - 1))) * kDh;
}
__device__ __forceinline__ const float* key_row(const Win& w, const Tile& s, int g, const void* t, int j) {
  if (j >= s.lk) return nullptr;
  return (const float*)t + ((size_t)(s.k0 + j) * w.Hkv + g) * kDh;
}

// Maximum or sum of a value over the 16 threads that share their rows.
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// <dout, out> of the thread's row i, from its four dims of out.
__device__ __forceinline__ float dot_row(const float* dout, int i, float4 y) {
  const float4 x = at4(dout + ((threadIdx.x >> 4) + kSub * i) * kPad + 4 * (threadIdx.x & 15));
  return row_sum(fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, x.w * y.w))));
}

// The query tile x of `grid` of key head g; false where there is none (the rows
// outside are filled).
__device__ __forceinline__ bool query_tile(const Win& w, int x, int grid, int g, Tile* s, void* rows, float* lse) {
  const int tokens = kRows >> w.gshift;
  bool bad;
  if (find_tile(w, x, tokens, false, s, &bad)) {
    s->t = s->n - 1 - s->t;      // the tiles with most keys first
    return true;
  }
  if (bad) {
    if (threadIdx.x == 0) set_err(w.err, PACK3D_DEVERR_LENGTHS);
  } else if (w.zero_outside && g == 0) {
    if (rows) fill_outside(w, w.cu_q, w.Tq, tokens, x, grid, kThreads / 32, rows, w.Hq * kDh, 0u);
    if (lse) fill_outside(w, w.cu_q, w.Tq, tokens, x, grid, kThreads / 32, lse, w.Hq, 0xff800000u);
  }
  return false;
}

// The CTAs of a cluster (kSplit) share a tile's steps: this one takes the steps
// [from, to) of n, and as many of the tile's 64 rows of the joined sums.
template <bool kSplit>
struct Part {
  int rank = 0, size = 1;
  __device__ __forceinline__ Part() {
    if constexpr (kSplit) {
      rank = cooperative_groups::this_cluster().block_rank();
      size = cooperative_groups::this_cluster().num_blocks();
    }
  }
  __device__ __forceinline__ int from(int n) const { return (int)((long)n * rank / size); }
  __device__ __forceinline__ int to(int n) const { return (int)((long)n * (rank + 1) / size); }
  // CTA z's value of what is at `at` in this one's shared memory.
  __device__ __forceinline__ float* of(float* at, int z) const {
    if constexpr (kSplit) return cooperative_groups::this_cluster().map_shared_rank(at, z);
    return at;
  }
  // Sum over the cluster of four floats at `at`, in the steps' order.
  __device__ __forceinline__ float4 sum(float* at) const {
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int z = 0; z < (kSplit ? size : 1); ++z) {
      const float4 y = at4(of(at, z));
      t.x += y.x;
      t.y += y.y;
      t.z += y.z;
      t.w += y.w;
    }
    return t;
  }
  // Before the sums are read, and before a CTA ends.
  __device__ __forceinline__ void meet() const {
    if constexpr (kSplit) cooperative_groups::this_cluster().sync();
    else __syncthreads();
  }
};
__device__ __forceinline__ bool not_finite(float4 c) {
  return !(fmaf(c.x, 0.f, fmaf(c.y, 0.f, fmaf(c.z, 0.f, c.w * 0.f))) == 0.f);
}
__device__ __forceinline__ float4 times(float4 c, float f) { return make_float4(c.x * f, c.y * f, c.z * f, c.w * f); }

template <bool kSplit>
__global__ void __launch_bounds__(kThreads, 2) window_attn_f32_kernel(const __grid_constant__ Win w) {
  extern __shared__ float4 smem4[];
  float* Q = reinterpret_cast<float*>(smem4);
  float *K = Q + kTileFloats, *V = K + kTileFloats, *P = V + kTileFloats;
  __shared__ int redo[kRows];
  Tile s;
  __shared__ float row_m[kRows], row_l[kRows];
  const Part<kSplit> part;
  const bool first = part.rank == 0;
  if (!query_tile(w, blockIdx.x / part.size, gridDim.x / part.size, blockIdx.y, &s, first ? w.out : nullptr,
                  first ? w.lse : nullptr))
    return;
  const int g = blockIdx.y, tokens = kRows >> w.gshift, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int r0 = s.t * tokens, r1 = min(s.lq, r0 + tokens) - 1;
  const KeyTiles<kKeys> kt = key_tiles<kKeys>(w, position(s, r0), position(s, r1));
  load_rows(Q, [&](int i) { return query_row(w, s, g, r0, r1, w.q, i); });
  if (threadIdx.x < kRows) redo[threadIdx.x] = 0;
  float m[kPer], l[kPer];
  Micro o;
  zero(o);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
#pragma unroll 1
  for (int t = part.from(kt.n); t < part.to(kt.n); ++t) {
    const int k0 = kt.begin(t), cols = kt.cols(t);
    load_rows(K, [&](int i) { return i < cols ? key_row(w, s, g, w.k, k0 + i) : nullptr; });
    load_rows(V, [&](int i) { return i < cols ? key_row(w, s, g, w.v, k0 + i) : nullptr; });
    loads_done();
    Micro c;
    mul_nt(c, Q, K);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = r0 + ((ty + kSub * i) >> w.gshift), p = r <= r1 ? position(s, r) : -1, low = window_low(w, p);
      float top = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = tx + 16 * j, key = k0 + col;
        const bool see = col < cols && key <= p && (key >= low || key < w.sinks);
        c[i][j] = see ? c[i][j] * w.scale_log2 : -INFINITY;
        top = fmaxf(top, c[i][j]);
      }
      top = row_max(top);
      const float f = m[i] == top ? 1.f : exp2f(m[i] - top), sub = top == -INFINITY ? 0.f : top;
      m[i] = top;
      l[i] *= f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = exp2f(c[i][j] - sub);
        l[i] += e;                      // of this thread's columns
        o[i][j] *= f;
        P[(ty + kSub * i) * kPad + tx + 16 * j] = e;
      }
    }
    __syncthreads();
    mul_nn(o, P, V);
    __syncthreads();
  }
  if (part.from(kt.n) == part.to(kt.n)) loads_done();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int row = ty + kSub * i;
    const float sum = row_sum(l[i]);
    if (tx == 0) {
      row_m[row] = m[i];
      row_l[row] = sum;
    }
    *reinterpret_cast<float4*>(P + row * kPad + 4 * tx) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
  }
  part.meet();
#pragma unroll 1
  for (int row = part.from(kRows) + ty; row < part.to(kRows); row += kSub) {
    const int r = r0 + (row >> w.gshift);
    if (r > r1) continue;
    // The shares of the row in the keys' order, on their largest maximum.
    float top = -INFINITY, sum = 0.f;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int z = 0; z < (kSplit ? part.size : 1); ++z) top = fmaxf(top, *part.of(row_m + row, z));
    for (int z = 0; z < (kSplit ? part.size : 1); ++z) {
      const float mz = *part.of(row_m + row, z), e = mz == top ? 1.f : exp2f(mz - top);
      const float4 y = at4(part.of(P + row * kPad + 4 * tx, z));
      sum = fmaf(*part.of(row_l + row, z), e, sum);
      f = make_float4(fmaf(y.x, e, f.x), fmaf(y.y, e, f.y), fmaf(y.z, e, f.z), fmaf(y.w, e, f.w));
    }
    // A row that sees no key: its O is 0, or a NaN from a hidden value.
    f = times(f, sum == 0.f ? 0.f : 1.f / sum);
    const size_t at = (size_t)(s.q0 + r) * w.Hq + (g << w.gshift) + (row & (w.G - 1));
    *reinterpret_cast<float4*>((float*)w.out + at * kDh + 4 * tx) = f;
    if (tx == 0 && w.lse) w.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718f;
    if (not_finite(f) && sum == sum) redo[row] = 1;
  }
  part.meet();
#pragma unroll 1
  for (int row = threadIdx.x >> 5; row < kRows; row += kThreads / 32)
    if (redo[row]) out_again<float>(w, s, r0 + (row >> w.gshift), (g << w.gshift) + (row & (w.G - 1)));
}

// P (and dS) of a tile pair from S and dP in registers, stored by row and key.
// Rows past r1 see nothing.
__device__ __forceinline__ void store_grads(const Win& w, const Tile& s, int r0, int r1, int k0, int cols, int keep,
                                            const float* lse2, const float* delta, Micro c, Micro d, float* P,
                                            float* dS) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int row = ty + kSub * i, r = r0 + (row >> w.gshift);
    const int p = r <= r1 ? position(s, r) : -1, low = window_low(w, p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = tx + 16 * j, key = k0 + col;
      const bool see = col < cols && key < keep && key <= p && (key >= low || key < w.sinks);
      const float e = see ? exp2f(fmaf(c[i][j], w.scale_log2, -lse2[i])) : 0.f;
      if (P) P[row * kPad + col] = e;
      dS[row * kPad + col] = see ? e * (d[i][j] - delta[i]) : 0.f;
    }
  }
}

// dQ of query tile x; redo: 64 ints of shared memory.
template <bool kSplit>
__device__ __forceinline__ void query_side(const Win& w, int x, int grid, int g, float* Q, int* redo) {
  float *D = Q + kTileFloats, *K = D + kTileFloats, *V = K + kTileFloats, *dS = V + kTileFloats;
  const Part<kSplit> part;
  Tile s;
  if (!query_tile(w, x, grid, g, &s, part.rank == 0 ? w.dq : nullptr, nullptr)) return;
  const int tokens = kRows >> w.gshift, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int r0 = s.t * tokens, r1 = min(s.lq, r0 + tokens) - 1;
  const KeyTiles<kKeys> kt = key_tiles<kKeys>(w, position(s, r0), position(s, r1));
  load_rows(Q, [&](int i) { return query_row(w, s, g, r0, r1, w.q, i); });
  load_rows(D, [&](int i) { return query_row(w, s, g, r0, r1, w.dout, i); });
  load_rows(K, [&](int i) { return query_row(w, s, g, r0, r1, w.out, i); });      // for <dout, out>
  if (threadIdx.x < kRows) redo[threadIdx.x] = 0;
  loads_done();
  float lse2[kPer], delta[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int row = ty + kSub * i, r = r0 + (row >> w.gshift);
    delta[i] = dot_row(D, i, at4(K + row * kPad + 4 * tx));
    lse2[i] = 0.f;
    if (r <= r1) {
      const size_t at = (size_t)(s.q0 + r) * w.Hq + (g << w.gshift) + (row & (w.G - 1));
      if (tx == 0) w.delta[at] = delta[i];
      lse2[i] = w.lse[at] * 1.4426950408889634f;
    }
  }
  Micro o;
  zero(o);
#pragma unroll 1
  for (int t = part.from(kt.n); t < part.to(kt.n); ++t) {
    const int k0 = kt.begin(t), cols = kt.cols(t);
    __syncthreads();
    load_rows(K, [&](int i) { return i < cols ? key_row(w, s, g, w.k, k0 + i) : nullptr; });
    load_rows(V, [&](int i) { return i < cols ? key_row(w, s, g, w.v, k0 + i) : nullptr; });
    loads_done();
    Micro c, d;
    mul_nt(c, Q, K);
    mul_nt(d, D, V);
    store_grads(w, s, r0, r1, k0, cols, s.lk, lse2, delta, c, d, nullptr, dS);
    __syncthreads();
    mul_nn(o, dS, K);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    *reinterpret_cast<float4*>(dS + (ty + kSub * i) * kPad + 4 * tx) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
  part.meet();
#pragma unroll 1
  for (int row = part.from(kRows) + ty; row < part.to(kRows); row += kSub) {
    const int r = r0 + (row >> w.gshift);
    if (r > r1) continue;
    const float4 f = times(part.sum(dS + row * kPad + 4 * tx), w.scale);
    const size_t at = (size_t)(s.q0 + r) * w.Hq + (g << w.gshift) + (row & (w.G - 1));
    *reinterpret_cast<float4*>((float*)w.dq + at * kDh + 4 * tx) = f;
    if (not_finite(f)) redo[row] = 1;
  }
  part.meet();
#pragma unroll 1
  for (int row = threadIdx.x >> 5; row < kRows; row += kThreads / 32)
    if (redo[row]) dq_again<float>(w, s, r0 + (row >> w.gshift), (g << w.gshift) + (row & (w.G - 1)));
}

// dK and dV of key tile `at`, or from key_grid on of a piece of the sinks' far
// queries.
template <bool kSplit>
__device__ __forceinline__ void key_side(const Win& w, int at, int key_grid, int g, float* K, int* redo) {
  float *V = K + kTileFloats, *Q = V + kTileFloats, *D = Q + kTileFloats, *P = D + kTileFloats, *dS = P + kTileFloats;
  const Part<kSplit> part;
  const bool far = at >= key_grid;
  const int x = far ? at - key_grid : at;
  const int tokens = kRows >> w.gshift, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  Tile s;
  bool bad;
  if (!(far ? find_far<kKeys, kRows>(w, x, &s, &bad) : find_tile(w, x, kKeys, true, &s, &bad))) {
    if (!far && !bad && w.zero_outside && g == 0 && part.rank == 0) {
      fill_outside(w, w.cu_k, w.Tk, kKeys, x, key_grid, kThreads / 32, w.dk, w.Hkv * kDh, 0u);
      fill_outside(w, w.cu_k, w.Tk, kKeys, x, key_grid, kThreads / 32, w.dv, w.Hkv * kDh, 0u);
    }
    return;
  }
  // Keys j0 .. of the sequence and the query rows ra .. rb that see some of them.
  const int shift = s.lk - s.lq;                        // position minus row
  const int j0 = far ? 0 : s.t * kKeys, j1 = min(s.lk, j0 + kKeys) - 1;
  int ra, rb;
  if (far) {
    ra = far_begin<kKeys>(w, s.lq, s.lk) + s.t * far_steps<kRows> * tokens;
    rb = min(s.lq, ra + far_steps<kRows> * tokens) - 1;
  } else {
    ra = max(0, j0 - shift);
    rb = s.lq - 1;
    if (w.window > 0) rb = min(rb, j1 + w.window - 1 - shift);
  }
  // Rows below `split_rows` of this tile leave float partial sums.
  const int split_rows = far || (j0 == 0 && far_pieces<kKeys, kRows>(w, s.lq, s.lk) > 0) ? min(w.sinks, s.lk) : 0;
  load_rows(K, [&](int i) { return key_row(w, s, g, w.k, j0 + i); });
  load_rows(V, [&](int i) { return key_row(w, s, g, w.v, j0 + i); });
  if (threadIdx.x < kKeys) redo[threadIdx.x] = 0;
  const int steps = rb >= ra ? (rb - ra) / tokens + 1 : 0;
  Micro ak, av;
  zero(ak);
  zero(av);
#pragma unroll 1
  for (int t = part.from(steps); t < part.to(steps); ++t) {
    const int rs = ra + t * tokens;
    load_rows(Q, [&](int i) { return query_row(w, s, g, rs, rb, w.q, i); });
    load_rows(D, [&](int i) { return query_row(w, s, g, rs, rb, w.dout, i); });
    float lse2[kPer], delta[kPer];
    float4 out[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int row = ty + kSub * i, r = rs + (row >> w.gshift);
      lse2[i] = 0.f;
      out[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r <= rb) {
        const size_t at = (size_t)(s.q0 + r) * w.Hq + (g << w.gshift) + (row & (w.G - 1));
        lse2[i] = __ldg(w.lse + at) * 1.4426950408889634f;
        out[i] = __ldg(reinterpret_cast<const float4*>((const float*)w.out + at * kDh) + tx);
      }
    }
    loads_done();
#pragma unroll
    for (int i = 0; i < kPer; ++i) delta[i] = dot_row(D, i, out[i]);
    Micro c, d;
    mul_nt(c, Q, K);
    mul_nt(d, D, V);
    store_grads(w, s, rs, rb, j0, kKeys, s.lk, lse2, delta, c, d, P, dS);
    __syncthreads();
    mul_tn(ak, dS, Q);
    mul_tn(av, P, D);
    __syncthreads();
  }
  if (part.from(steps) == part.to(steps)) loads_done();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    *reinterpret_cast<float4*>(P + row_tn(i) * kPad + 4 * tx) = make_float4(ak[i][0], ak[i][1], ak[i][2], ak[i][3]);
    *reinterpret_cast<float4*>(dS + row_tn(i) * kPad + 4 * tx) = make_float4(av[i][0], av[i][1], av[i][2], av[i][3]);
  }
  part.meet();
  const int slot = far ? x + s.b + 1 : part_slot<kRows>(w, s);      // of the sink rows' partial sums
#pragma unroll 1
  for (int row = part.from(kKeys) + ty; row < part.to(kKeys); row += kSub) {
    const float4 fk = times(part.sum(P + row * kPad + 4 * tx), w.scale), fv = part.sum(dS + row * kPad + 4 * tx);
    if (row < split_rows) {
      float4* dst = reinterpret_cast<float4*>(part_row(w, slot, g, row));
      dst[tx] = fk;
      dst[16 + tx] = fv;
    } else if (!far && j0 + row <= j1) {
      const size_t to = ((size_t)(s.k0 + j0 + row) * w.Hkv + g) * kDh + 4 * tx;
      *reinterpret_cast<float4*>((float*)w.dk + to) = fk;
      *reinterpret_cast<float4*>((float*)w.dv + to) = fv;
      if (not_finite(fk) || not_finite(fv)) redo[row] = 1;
    }
  }
  part.meet();
#pragma unroll 1
  for (int row = threadIdx.x >> 5; row < kKeys; row += kThreads / 32)
    if (redo[row]) dkv_row<float>(w, s, j0 + row, g, true);
}

// Both sides in one launch, so that few tiles fill more of the GPU: neither reads
// what the other writes (each forms <dout, out> of its rows).  The key sides come
// first, as the longer ones (behind the query sides 6 % later), and a tile's
// heads side by side (heads one after the other: up to a third later).
template <bool kSplit>
__global__ void __launch_bounds__(kThreads, 2) window_bwd_f32_kernel(const __grid_constant__ Win w, int key_grid, int key_ctas,
                                                                     int query_ctas) {
  extern __shared__ float4 smem4[];
  __shared__ int redo[64];
  float* tiles = reinterpret_cast<float*>(smem4);
  let_next_begin();
  const int x = kSplit ? blockIdx.x / Part<kSplit>().size : blockIdx.x, y = x - key_ctas * w.Hkv;
  if (y < 0) key_side<kSplit>(w, x / w.Hkv, key_grid, x % w.Hkv, tiles, redo);
  else query_side<kSplit>(w, y / w.Hkv, query_ctas, y % w.Hkv, tiles, redo);
}

template <typename K>
cudaError_t allow(K kernel, int tiles) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, tiles * kTileFloats * 4);
}

// CTAs of a cluster that share a tile, of `tiles` in the call: a share should be
// eight steps long, `least` where the SMs would have four CTAs at most (two in the
// backward; the forward's are half as long: four), one where there is a CTA an SM
// at most.  (Backward: 3,000 tokens, 2 / 1 heads, no window, 1 CTA 0.911 ms, 8 CTAs
// 0.294; 1,000, 4 heads: 1, 4, 8 CTAs 161, 84, 112 us; 2,600, 8 / 2 heads, window
// 300: 1, 2, 4: 251, 209, 241; 1,000 in two, 8 heads, window 64, which is two steps:
// 1, 2: 36, 46.  Forward: the first 255 us with 1, 93 with 4; 2,050 in three, window
// 200, four steps: 1, 2: 33, 36.)  The host knows the mean length only: 3,000 tokens
// with 31 sequences of one count as short, 965 us backward with 1 CTA (316 with 4).
int split_of(long tiles, long steps, long least) {
  const long sms = sm_count();
  auto good = [&](long S) {
    return (tiles * S <= sms && steps >= S) || (tiles * S <= 4 * sms && steps >= least * S) ||
           (tiles * S <= 8 * sms && steps >= 8 * S);
  };
  int S = 1;
  while (S < 8 && good(2 * S)) S *= 2;
  return S;
}

// A kernel with `tiles` tiles of shared memory and clusters of S.
template <typename... P, typename... A>
cudaError_t launch_shared(void (*kernel)(P...), dim3 grid, int tiles, int S, cudaStream_t st, A... args) {
  cudaError_t e = allow(kernel, tiles);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = S;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  grid.x *= S;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = tiles * kTileFloats * 4;
  cfg.stream = st;
  cfg.attrs = &cluster;
  cfg.numAttrs = S > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Tokens of a sequence of the mean length, at most those that a window reaches
// from a tile of `tile` tokens.
long reach(const Win& w, long tokens, long tile) {
  const long mean = (tokens + w.B - 1) / w.B;
  return w.window > 0 ? min(mean, (long)w.window + tile) : mean;
}

}  // namespace

size_t window_bwd_part_bytes(const Win& w, int dtype) {
  if (w.sinks == 0 || w.window == 0) return 0;
  // A slot for every sequence's first tile and one for every far piece.
  const long far = dtype == PACK3D_BF16 ? far_grid<kRowsPerTile>(w) : far_grid<kRows>(w);
  return (size_t)(far + w.B) * w.Hkv * w.sinks * 2 * kDh * sizeof(float);
}

cudaError_t launch_window_attn_f32(const Win& w, cudaStream_t st) {
  const int tokens = kRows >> w.gshift;
  const long tiles = tile_grid(w.Tq, tokens, w.B);
  const dim3 grid((unsigned)tiles, w.Hkv);
  const int S = split_of(tiles * w.Hkv, (reach(w, w.Tk, tokens) + kKeys - 1) / kKeys, 4);
  return S > 1 ? launch_shared(window_attn_f32_kernel<true>, grid, 4, S, st, w)
               : launch_shared(window_attn_f32_kernel<false>, grid, 4, 1, st, w);
}

cudaError_t launch_window_bwd_f32(const Win& w, cudaStream_t st) {
  const int key_grid = (int)tile_grid(w.Tk, kKeys, w.B), key_ctas = key_grid + (int)far_grid<kRows>(w);
  const int query_ctas = (int)tile_grid(w.Tq, kRows >> w.gshift, w.B);
  const dim3 grid((unsigned)(key_ctas + query_ctas) * w.Hkv);
  const int S = split_of(grid.x, (reach(w, w.Tq, kKeys) * w.G + kRows - 1) / kRows, 2);
  const cudaError_t e =
      S > 1 ? launch_shared(window_bwd_f32_kernel<true>, grid, 6, S, st, w, key_grid, key_ctas, query_ctas)
            : launch_shared(window_bwd_f32_kernel<false>, grid, 6, 1, st, w, key_grid, key_ctas, query_ctas);
  if (e != cudaSuccess) return e;
  return launch_window_sinks<float, kKeys, kRows>(w, st);
}

}  // namespace seq
}  // namespace pack3d
