// The sinks' share of the windowed attention's key gradients (both types).
//
// A sequence's first key tile holds its sinks, which every later query sees.
// The CTA of that tile takes the queries whose window reaches it; those beyond
// ("far") are cut into pieces of far_steps query tiles, one CTA each.  The tile
// and the pieces leave float partial sums of the sink rows in Win::part, the
// tile at slot base(b) + b (base as in find_piece) and the pieces in the slots
// behind it; window_sinks_kernel adds them in that order.
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
// Queries of a piece, and the pieces of the far queries, with query tiles of
// Rows rows.
template <int Rows>
__host__ __device__ __forceinline__ int far_rows(const Win& w) { return far_steps<Rows> * (Rows >> w.gshift); }
template <int Keys, int Rows>
__device__ __forceinline__ int far_pieces(const Win& w, int lq, int lk) {
  const int per = far_rows<Rows>(w);
  return lk == 0 ? 0 : (lq - far_begin<Keys>(w, lq, lk) + per - 1) / per;
}
// The piece of far CTA number x.
template <int Keys, int Rows>
__device__ __forceinline__ bool find_far(const Win& w, int x, Tile* out, bool* bad) {
  return find_piece(w, x, far_rows<Rows>(w), false, [&](int lq, int lk) { return far_pieces<Keys, Rows>(w, lq, lk); },
                    out, bad);
}
// CTAs that cover the far pieces whatever the offsets are.
template <int Rows>
inline long far_grid(const Win& w) {
  return w.sinks == 0 || w.window == 0 ? 0 : w.Tq / far_rows<Rows>(w) + w.B;
}
// The first slot of a sequence's partial sums.
template <int Rows>
__device__ __forceinline__ int part_slot(const Win& w, const Tile& s) {
  return (s.q0 >> log2_of(far_rows<Rows>(w))) + 2 * s.b;
}
// Partial sums of row `row` (0 .. sinks-1) at a slot: dK's 64 dims, then dV's.
__device__ __forceinline__ float* part_row(const Win& w, int slot, int g, int row) {
  return w.part + (((size_t)slot * w.Hkv + g) * w.sinks + row) * 2 * kDh;
}

// Softmax scales below this can make lse / scale, which the bf16 kernels subtract,
// overflow: a row's term is a NaN then, and what it spoils is computed again
// whatever has spoilt it.
constexpr float kLeastScale = 0x1p-100f;

// dK and dV of one sink row of one sequence: eight warps add every eighth part,
// then the eight sums in order.  (With very many sequences a CTA takes several.)
constexpr int kSinksGrid = 1024;
template <typename T, int Keys, int Rows>
__global__ void __launch_bounds__(256) window_sinks_kernel(const __grid_constant__ Win w) {
  __shared__ float4 sums[8][32];
  const int g = blockIdx.y, j = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  wait_for_last();
#pragma unroll 1
  for (int b = blockIdx.x; b < w.B; b += gridDim.x) {
    if (off_range(w, b)) continue;
    Tile s;
    s.b = b;
    s.q0 = __ldg(w.cu_q + b);
    s.lq = __ldg(w.cu_q + b + 1) - s.q0;
    s.k0 = __ldg(w.cu_k + b);
    s.lk = __ldg(w.cu_k + b + 1) - s.k0;
    s.t = 0;
    s.n = far_pieces<Keys, Rows>(w, s.lq, s.lk);
    if (s.n == 0 || j >= s.lk) continue;
    const int slot = part_slot<Rows>(w, s);
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
    if (warp == 0) {
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
      if (again) dkv_row<T>(w, s, j, g, sizeof(T) == 4 || w.scale >= kLeastScale);
    }
    __syncthreads();
  }
}

template <typename T, int Keys, int Rows>
cudaError_t launch_window_sinks(const Win& w, cudaStream_t st) {
  if (w.sinks == 0 || w.window == 0) return cudaSuccess;
  return launch_behind(window_sinks_kernel<T, Keys, Rows>, dim3(min(w.B, kSinksGrid), w.Hkv, w.sinks), 256, 0, st, 1, w);
}

}  // namespace seq
}  // namespace pack3d
