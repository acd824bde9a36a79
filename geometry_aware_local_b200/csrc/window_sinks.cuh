// The sinks' share of the windowed attention's key gradients (both types).
//
// A sequence's first key tile holds its sinks, which every later query sees.
// The CTA of that tile takes the queries whose window reaches it; those beyond
// ("far") are cut into pieces of far_steps query tiles, one CTA each.  The tile
// and the pieces leave float partial sums of the sink rows in Win::part, at
// slot = (far pieces of the sequences before) + (sequence) for the tile and the
// slots behind it for the pieces; window_sinks_kernel adds them in that order.
#pragma once

#include "seq.cuh"

namespace pack3d {
namespace seq {

// Query tiles (of Rows rows) of a piece: long enough that its partial sums (at
// most 64 rows x 128 floats) are small beside what it reads, and no longer than
// what a CTA of an ordinary key tile takes with a window of a few hundred keys.
template <int Rows>
constexpr int far_steps = Rows == 128 ? 16 : 4;

// First far query row of a sequence, with key tiles of Keys rows; lq where
// there is none.
template <int Keys>
__device__ __forceinline__ int far_begin(const Win& w, int lq, int lk) {
  if (w.sinks == 0 || w.window == 0) return lq;
  const int r = min(Keys, lk) - 1 + w.window - (lk - lq);     // past the last position that sees the tile's last key
  return min(lq, max(0, r));
}
// Pieces of the far queries, with query tiles of Rows rows.
template <int Keys, int Rows>
__device__ __forceinline__ int far_pieces(const Win& w, int lq, int lk) {
  if (lk == 0) return 0;
  const int per = far_steps<Rows> * (Rows >> w.gshift);
  return (lq - far_begin<Keys>(w, lq, lk) + per - 1) / per;
}
// CTAs that cover the far pieces whatever the offsets are.
template <int Rows>
inline long far_grid(const Win& w) {
  if (w.sinks == 0 || w.window == 0) return 0;
  return w.Tq / ((long)far_steps<Rows> * (Rows >> w.gshift)) + w.B;
}
// Partial sums of row `row` (0 .. sinks-1) at a slot: dK's 64 dims, then dV's.
__device__ __forceinline__ float* part_row(const Win& w, int slot, int g, int row) {
  return w.part + (((size_t)slot * w.Hkv + g) * w.sinks + row) * 2 * kDh;
}

// dK and dV of one sink row of one sequence: eight warps add every eighth part,
// then the eight sums in order.
template <typename T, int Keys, int Rows>
__global__ void __launch_bounds__(256) window_sinks_kernel(const Win w) {
  __shared__ float4 sums[8][32];
  const int b = blockIdx.x, g = blockIdx.y, j = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Tile s;
  Tiles all;
  find_tile(w, 0, 1, false, &s, &all);        // checks the offsets
  if (all.bad) return;
  s.b = b;
  s.q0 = __ldg(w.cu_q + b);
  s.lq = __ldg(w.cu_q + b + 1) - s.q0;
  s.k0 = __ldg(w.cu_k + b);
  s.lk = __ldg(w.cu_k + b + 1) - s.k0;
  s.t = 0;
  s.n = far_pieces<Keys, Rows>(w, s.lq, s.lk);
  if (s.n == 0 || j >= s.lk) return;
  const int slot = pieces_before(w, b, [&](int lq, int lk) { return far_pieces<Keys, Rows>(w, lq, lk); }) + b;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = warp; i <= s.n; i += 8) {
    const float4 y = reinterpret_cast<const float4*>(part_row(w, slot + i, g, j))[lane];
    sum.x += y.x;
    sum.y += y.y;
    sum.z += y.z;
    sum.w += y.w;
  }
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp > 0) return;
  for (int i = 1; i < 8; ++i) {
    const float4 y = sums[i][lane];
    sum.x += y.x;
    sum.y += y.y;
    sum.z += y.z;
    sum.w += y.w;
  }
  // Lanes 0-15 hold dK's 64 dims, 16-31 dV's.
  T* dst = (T*)(lane < 16 ? w.dk : w.dv) + ((size_t)(s.k0 + j) * w.Hkv + g) * kDh + 4 * (lane & 15);
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
  else
    *reinterpret_cast<float4*>(dst) = sum;
  const float zero = fmaf(sum.x, 0.f, fmaf(sum.y, 0.f, fmaf(sum.z, 0.f, sum.w * 0.f)));
  const bool again = __any_sync(0xffffffffu, !(zero == 0.f));
  __syncwarp();
  if (again) dkv_row<T>(w, s, j, g);
}

template <typename T, int Keys, int Rows>
cudaError_t launch_window_sinks(const Win& w, cudaStream_t st) {
  if (w.sinks == 0 || w.window == 0) return cudaSuccess;
  window_sinks_kernel<T, Keys, Rows><<<dim3(w.B, w.Hkv, w.sinks), 256, 0, st>>>(w);
  return cudaGetLastError();
}

}  // namespace seq
}  // namespace pack3d
