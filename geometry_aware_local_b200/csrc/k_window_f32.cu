// Causal windowed attention of packed sequences and its gradients in float, on
// CUDA cores.
//
// The tiles are those of the tensor-core kernels (rows = (token, query head)
// pairs of one key head's group; key range and sinks; see k_window_tc.cu and
// k_window_bwd_tc.cu), 64 rows by 64 keys.  128 threads hold a 64 x 64 product
// as 8 x 4 values each: thread (ty, tx) = (tid / 16, tid % 16) has the rows
// ty + 8 i and the columns tx + 16 j of S and dP (both operands are read four
// contraction steps at a time, 16 bytes a load, from rows padded to 68 floats),
// and the dims 4 tx .. 4 tx + 3 of O, dQ, dK and dV.  Everything is formed and
// kept in 32 bits.  Bound: the shared-memory reads (12 loads of 16 bytes per 128
// multiply-adds and thread) and the multiply-adds themselves.  2,050 tokens in
// three sequences, 4 / 2 heads, window 200, one sink: forward and backward 0.21 ms
// (one warp a row of the definition: 1.27 ms).
//
// What is hidden has P = 0; rows that 0 times a NaN or an infinity spoilt are
// computed again (out_row, dq_row, dkv_row), as in the tensor-core kernels.
#include "seq_tc.cuh"
#include "window_sinks.cuh"

namespace pack3d {
namespace seq {
namespace {

constexpr int kRows = 64, kKeys = 64, kThreads = 128;
constexpr int kPad = kDh + 4;
constexpr int kTileFloats = 64 * kPad;

typedef float Micro[8][4];

__device__ __forceinline__ void zero(Micro c) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] = 0.f;
}
__device__ __forceinline__ float4 at4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// c[i][j] += sum_d a[ty + 8 i][d] b[tx + 16 j][d]: both operands' rows run along
// the contraction.
__device__ __forceinline__ void mul_nt(Micro c, const float* a, const float* b) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 2
  for (int d = 0; d < kDh; d += 4) {
    float4 x[8], y[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = at4(a + (ty + 8 * i) * kPad + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = at4(b + (tx + 16 * j) * kPad + d);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c[i][j] = fmaf(x[i].w, y[j].w, fmaf(x[i].z, y[j].z, fmaf(x[i].y, y[j].y, fmaf(x[i].x, y[j].x, c[i][j]))));
  }
}
// c[i][j] += sum_k a[ty + 8 i][k] b[k][4 tx + j].
__device__ __forceinline__ void mul_nn(Micro c, const float* a, const float* b) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 2
  for (int k = 0; k < 64; k += 4) {
    float4 x[8], y[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = at4(a + (ty + 8 * i) * kPad + k);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = at4(b + (k + j) * kPad + 4 * tx);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[i][0] = fmaf(v[j], y[j].x, c[i][0]);
        c[i][1] = fmaf(v[j], y[j].y, c[i][1]);
        c[i][2] = fmaf(v[j], y[j].z, c[i][2]);
        c[i][3] = fmaf(v[j], y[j].w, c[i][3]);
      }
    }
  }
}
// Row of the product of the transposed operand that c[i] belongs to.
__device__ __forceinline__ int row_tn(int i) { return 4 * (threadIdx.x >> 4) + (i & 3) + 32 * (i >> 2); }
// c[i][j] += sum_k a[k][row_tn(i)] b[k][4 tx + j].
__device__ __forceinline__ void mul_tn(Micro c, const float* a, const float* b) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 4
  for (int k = 0; k < 64; ++k) {
    const float4 x0 = at4(a + k * kPad + 4 * ty), x1 = at4(a + k * kPad + 4 * ty + 32), y = at4(b + k * kPad + 4 * tx);
    const float v[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i][0] = fmaf(v[i], y.x, c[i][0]);
      c[i][1] = fmaf(v[i], y.y, c[i][1]);
      c[i][2] = fmaf(v[i], y.z, c[i][2]);
      c[i][3] = fmaf(v[i], y.w, c[i][3]);
    }
  }
}

// Copies 64 rows of 64 floats into a tile, without waiting: row i is at
// row_of(i), or zeros where that is null.
template <typename RowOf>
__device__ __forceinline__ void load_rows(float* tile, RowOf row_of) {
  const uint32_t base = ptx::smem_u32(tile);
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const int i = (threadIdx.x >> 4) + 8 * n, x = threadIdx.x & 15;
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
__device__ __forceinline__ bool not_finite(const float* c) {
  return !(fmaf(c[0], 0.f, fmaf(c[1], 0.f, fmaf(c[2], 0.f, c[3] * 0.f))) == 0.f);
}

// The query tile of a CTA; false where it has none (the rows outside are filled).
__device__ __forceinline__ bool query_tile(const Win& w, Tile* s, void* rows, float* lse) {
  const int tokens = kRows >> w.gshift;
  bool bad;
  if (find_tile(w, blockIdx.x, tokens, false, s, &bad)) {
    s->t = s->n - 1 - s->t;      // the tiles with most keys first
    return true;
  }
  if (bad) {
    if (threadIdx.x == 0) set_err(w.err, PACK3D_DEVERR_LENGTHS);
  } else if (w.zero_outside && blockIdx.y == 0) {
    fill_outside(w, w.cu_q, w.Tq, tokens, blockIdx.x, gridDim.x, kThreads / 32, rows, w.Hq * kDh, 0u);
    if (lse) fill_outside(w, w.cu_q, w.Tq, tokens, blockIdx.x, gridDim.x, kThreads / 32, lse, w.Hq, 0xff800000u);
  }
  return false;
}

__global__ void __launch_bounds__(kThreads, 3) window_attn_f32_kernel(const Win w) {
  extern __shared__ float4 smem4[];
  float* Q = reinterpret_cast<float*>(smem4);
  float *K = Q + kTileFloats, *V = K + kTileFloats, *P = V + kTileFloats;
  __shared__ int redo[kRows];
  Tile s;
  if (!query_tile(w, &s, w.out, w.lse)) return;
  const int g = blockIdx.y, tokens = kRows >> w.gshift, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int r0 = s.t * tokens, r1 = min(s.lq, r0 + tokens) - 1;
  const KeyTiles<kKeys> kt = key_tiles<kKeys>(w, position(s, r0), position(s, r1));
  load_rows(Q, [&](int i) { return query_row(w, s, g, r0, r1, w.q, i); });
  if (threadIdx.x < kRows) redo[threadIdx.x] = 0;
  float m[8], l[8];
  Micro o;
  zero(o);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
#pragma unroll 1
  for (int t = 0; t < kt.n; ++t) {
    const int k0 = kt.begin(t), cols = kt.cols(t);
    load_rows(K, [&](int i) { return i < cols ? key_row(w, s, g, w.k, k0 + i) : nullptr; });
    load_rows(V, [&](int i) { return i < cols ? key_row(w, s, g, w.v, k0 + i) : nullptr; });
    loads_done();
    Micro c;
    zero(c);
    mul_nt(c, Q, K);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + ((ty + 8 * i) >> w.gshift), p = r <= r1 ? position(s, r) : -1, low = window_low(w, p);
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
        P[(ty + 8 * i) * kPad + tx + 16 * j] = e;
      }
    }
    __syncthreads();
    mul_nn(o, P, V);
    __syncthreads();
  }
  if (kt.n == 0) loads_done();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = ty + 8 * i, r = r0 + (row >> w.gshift);
    const float sum = row_sum(l[i]);
    // A row that sees no key: its O is 0, or a NaN from a hidden value.
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (r > r1) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] *= inv;
    const size_t at = (size_t)(s.q0 + r) * w.Hq + (g << w.gshift) + (row & (w.G - 1));
    *reinterpret_cast<float4*>((float*)w.out + at * kDh + 4 * tx) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
    if (tx == 0 && w.lse) w.lse[at] = sum == 0.f ? -INFINITY : (m[i] + log2f(sum)) * 0.69314718f;
    if (not_finite(o[i])) redo[row] = 1;
  }
  __syncthreads();
#pragma unroll 1
  for (int row = threadIdx.x >> 5; row < kRows; row += kThreads / 32)
    if (redo[row]) out_row<float>(w, s, r0 + (row >> w.gshift), (g << w.gshift) + (row & (w.G - 1)));
}

// P (and dS) of a tile pair from S and dP in registers, stored by row and key.
// Rows past r1 see nothing.
__device__ __forceinline__ void store_grads(const Win& w, const Tile& s, int r0, int r1, int k0, int cols, int keep,
                                            const float* lse2, const float* delta, Micro c, Micro d, float* P,
                                            float* dS) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = ty + 8 * i, r = r0 + (row >> w.gshift), p = r <= r1 ? position(s, r) : -1, low = window_low(w, p);
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

__global__ void __launch_bounds__(kThreads, 2) window_dq_f32_kernel(const Win w) {
  extern __shared__ float4 smem4[];
  float* Q = reinterpret_cast<float*>(smem4);
  float *D = Q + kTileFloats, *K = D + kTileFloats, *V = K + kTileFloats, *dS = V + kTileFloats;
  __shared__ int redo[kRows];
  Tile s;
  if (!query_tile(w, &s, w.dq, nullptr)) return;
  const int g = blockIdx.y, tokens = kRows >> w.gshift, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int r0 = s.t * tokens, r1 = min(s.lq, r0 + tokens) - 1;
  const KeyTiles<kKeys> kt = key_tiles<kKeys>(w, position(s, r0), position(s, r1));
  load_rows(Q, [&](int i) { return query_row(w, s, g, r0, r1, w.q, i); });
  load_rows(D, [&](int i) { return query_row(w, s, g, r0, r1, w.dout, i); });
  load_rows(K, [&](int i) { return query_row(w, s, g, r0, r1, w.out, i); });      // for <dout, out>
  if (threadIdx.x < kRows) redo[threadIdx.x] = 0;
  loads_done();
  float lse2[8], delta[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = ty + 8 * i, r = r0 + (row >> w.gshift);
    const float4 x = at4(D + row * kPad + 4 * tx), y = at4(K + row * kPad + 4 * tx);
    delta[i] = row_sum(fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, x.w * y.w))));
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
  for (int t = 0; t < kt.n; ++t) {
    const int k0 = kt.begin(t), cols = kt.cols(t);
    __syncthreads();
    load_rows(K, [&](int i) { return i < cols ? key_row(w, s, g, w.k, k0 + i) : nullptr; });
    load_rows(V, [&](int i) { return i < cols ? key_row(w, s, g, w.v, k0 + i) : nullptr; });
    loads_done();
    Micro c, d;
    zero(c);
    zero(d);
    mul_nt(c, Q, K);
    mul_nt(d, D, V);
    store_grads(w, s, r0, r1, k0, cols, s.lk, lse2, delta, c, d, nullptr, dS);
    __syncthreads();
    mul_nn(o, dS, K);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = ty + 8 * i, r = r0 + (row >> w.gshift);
    if (r > r1) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] *= w.scale;
    const size_t at = (size_t)(s.q0 + r) * w.Hq + (g << w.gshift) + (row & (w.G - 1));
    *reinterpret_cast<float4*>((float*)w.dq + at * kDh + 4 * tx) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
    if (not_finite(o[i])) redo[row] = 1;
  }
  __syncthreads();
#pragma unroll 1
  for (int row = threadIdx.x >> 5; row < kRows; row += kThreads / 32)
    if (redo[row]) dq_row<float>(w, s, r0 + (row >> w.gshift), (g << w.gshift) + (row & (w.G - 1)));
}

__global__ void __launch_bounds__(kThreads, 2) window_dkv_f32_kernel(const Win w, int key_grid) {
  extern __shared__ float4 smem4[];
  float* K = reinterpret_cast<float*>(smem4);
  float *V = K + kTileFloats, *Q = V + kTileFloats, *D = Q + kTileFloats, *P = D + kTileFloats, *dS = P + kTileFloats;
  __shared__ int redo[kKeys];
  const bool far = (int)blockIdx.x >= key_grid;         // a CTA of the sinks' far queries
  const int x = far ? blockIdx.x - key_grid : blockIdx.x;
  const int g = blockIdx.y, tokens = kRows >> w.gshift, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  Tile s;
  bool bad;
  if (!(far ? find_far<kKeys, kRows>(w, x, &s, &bad) : find_tile(w, x, kKeys, true, &s, &bad))) {
    if (!far && !bad && w.zero_outside && blockIdx.y == 0) {
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
  Micro ak, av;
  zero(ak);
  zero(av);
#pragma unroll 1
  for (int rs = ra; rs <= rb; rs += tokens) {
    load_rows(Q, [&](int i) { return query_row(w, s, g, rs, rb, w.q, i); });
    load_rows(D, [&](int i) { return query_row(w, s, g, rs, rb, w.dout, i); });
    float lse2[8], delta[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = ty + 8 * i, r = rs + (row >> w.gshift);
      lse2[i] = delta[i] = 0.f;
      if (r <= rb) {
        const size_t at = (size_t)(s.q0 + r) * w.Hq + (g << w.gshift) + (row & (w.G - 1));
        lse2[i] = __ldg(w.lse + at) * 1.4426950408889634f;
        delta[i] = __ldg(w.delta + at);
      }
    }
    loads_done();
    Micro c, d;
    zero(c);
    zero(d);
    mul_nt(c, Q, K);
    mul_nt(d, D, V);
    store_grads(w, s, rs, rb, j0, kKeys, s.lk, lse2, delta, c, d, P, dS);
    __syncthreads();
    mul_tn(ak, dS, Q);
    mul_tn(av, P, D);
    __syncthreads();
  }
  if (ra > rb) loads_done();
  const int slot = far ? x + s.b + 1 : part_slot<kRows>(w, s);      // of the sink rows' partial sums
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row_tn(i);
#pragma unroll
    for (int j = 0; j < 4; ++j) ak[i][j] *= w.scale;
    const float4 fk = make_float4(ak[i][0], ak[i][1], ak[i][2], ak[i][3]);
    const float4 fv = make_float4(av[i][0], av[i][1], av[i][2], av[i][3]);
    if (row < split_rows) {
      float4* dst = reinterpret_cast<float4*>(part_row(w, slot, g, row));
      dst[tx] = fk;
      dst[16 + tx] = fv;
    } else if (!far && j0 + row <= j1) {
      const size_t at = ((size_t)(s.k0 + j0 + row) * w.Hkv + g) * kDh + 4 * tx;
      *reinterpret_cast<float4*>((float*)w.dk + at) = fk;
      *reinterpret_cast<float4*>((float*)w.dv + at) = fv;
      if (not_finite(ak[i]) || not_finite(av[i])) redo[row] = 1;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int row = threadIdx.x >> 5; row < kKeys; row += kThreads / 32)
    if (redo[row]) dkv_row<float>(w, s, j0 + row, g);
}

template <typename K>
cudaError_t allow(K kernel, int tiles) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, tiles * kTileFloats * 4);
}

}  // namespace

size_t window_bwd_part_bytes(const Win& w, int dtype) {
  if (w.sinks == 0 || w.window == 0) return 0;
  // A slot for every sequence's first tile and one for every far piece.
  const long far = dtype == PACK3D_BF16 ? far_grid<kRowsPerTile>(w) : far_grid<kRows>(w);
  return (size_t)(far + w.B) * w.Hkv * w.sinks * 2 * kDh * sizeof(float);
}

cudaError_t launch_window_attn_f32(const Win& w, cudaStream_t st) {
  const cudaError_t e = allow(window_attn_f32_kernel, 4);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)tile_grid(w.Tq, kRows >> w.gshift, w.B), w.Hkv);
  window_attn_f32_kernel<<<grid, kThreads, 4 * kTileFloats * 4, st>>>(w);
  return cudaGetLastError();
}

cudaError_t launch_window_bwd_f32(const Win& w, cudaStream_t st) {
  cudaError_t e = allow(window_dq_f32_kernel, 5);
  if (e == cudaSuccess) e = allow(window_dkv_f32_kernel, 6);
  if (e != cudaSuccess) return e;
  const dim3 gq((unsigned)tile_grid(w.Tq, kRows >> w.gshift, w.B), w.Hkv);
  window_dq_f32_kernel<<<gq, kThreads, 5 * kTileFloats * 4, st>>>(w);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int key_grid = (int)tile_grid(w.Tk, kKeys, w.B);
  const dim3 gk((unsigned)(key_grid + far_grid<kRows>(w)), w.Hkv);
  window_dkv_f32_kernel<<<gk, kThreads, 6 * kTileFloats * 4, st>>>(w, key_grid);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_window_sinks<float, kKeys, kRows>(w, st);
}

}  // namespace seq
}  // namespace pack3d
