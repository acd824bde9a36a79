// Dispatch of the causal windowed attention of packed sequences: bf16 to the
// tensor-core kernels, float to the CUDA-core ones, and bf16 calls without a
// single key row (or, backwards, query row), which have no tensor a TMA map
// could describe, row by row: one warp owns one query row of one head or one
// key row of one key head.
#include "seq.cuh"

namespace pack3d {
namespace seq {
namespace {

constexpr int kWarps = 8;

// What a CTA without a tile does: it reports wrong offsets, or fills the rows
// that belong to no sequence.
template <typename T>
__device__ __forceinline__ void no_query_tile(const Win& w, bool bad, void* rows, float* lse) {
  if (bad) {
    if (threadIdx.x == 0) set_err(w.err, PACK3D_DEVERR_LENGTHS);
  } else if (w.zero_outside && blockIdx.y == 0) {
    fill_outside(w, w.cu_q, w.Tq, kWarps, blockIdx.x, gridDim.x, kWarps, rows, w.Hq * kDh * (int)sizeof(T) / 4, 0u);
    if (lse) fill_outside(w, w.cu_q, w.Tq, kWarps, blockIdx.x, gridDim.x, kWarps, lse, w.Hq, 0xff800000u);
  }
}
template <typename T>
__device__ __forceinline__ void no_key_tile(const Win& w, bool bad) {
  if (bad || !w.zero_outside || blockIdx.y != 0) return;
  const int words = w.Hkv * kDh * (int)sizeof(T) / 4;
  fill_outside(w, w.cu_k, w.Tk, kWarps, blockIdx.x, gridDim.x, kWarps, w.dk, words, 0u);
  fill_outside(w, w.cu_k, w.Tk, kWarps, blockIdx.x, gridDim.x, kWarps, w.dv, words, 0u);
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) window_rows_kernel(const Win w) {
  Tile s;
  bool bad;
  if (!find_tile(w, blockIdx.x, kWarps, false, &s, &bad)) return no_query_tile<T>(w, bad, w.out, w.lse);
  const int r = s.t * kWarps + (threadIdx.x >> 5);
  if (r < s.lq) out_row<T>(w, s, r, blockIdx.y);
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) window_dq_rows_kernel(const Win w) {
  Tile s;
  bool bad;
  if (!find_tile(w, blockIdx.x, kWarps, false, &s, &bad)) return no_query_tile<T>(w, bad, w.dq, nullptr);
  const int r = s.t * kWarps + (threadIdx.x >> 5);
  if (r >= s.lq) return;
  delta_row<T>(w, (size_t)(s.q0 + r) * w.Hq + blockIdx.y);
  __syncwarp();
  dq_row<T>(w, s, r, blockIdx.y);
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) window_dkv_rows_kernel(const Win w) {
  Tile s;
  bool bad;
  if (!find_tile(w, blockIdx.x, kWarps, true, &s, &bad)) return no_key_tile<T>(w, bad);
  const int j = s.t * kWarps + (threadIdx.x >> 5);
  if (j < s.lk) dkv_row<T>(w, s, j, blockIdx.y, false);
}

}  // namespace

cudaError_t launch_window_attn(const Win& w, int dtype, cudaStream_t st) {
  if (dtype != PACK3D_BF16) return launch_window_attn_f32(w, st);
  if (w.Tk > 0) return launch_window_attn_tc(w, st);
  const dim3 grid((unsigned)tile_grid(w.Tq, kWarps, w.B), w.Hq);
  window_rows_kernel<__nv_bfloat16><<<grid, 32 * kWarps, 0, st>>>(w);
  return cudaGetLastError();
}

cudaError_t launch_window_bwd(const Win& w, int dtype, cudaStream_t st) {
  if (dtype != PACK3D_BF16) return launch_window_bwd_f32(w, st);
  if (w.Tq > 0 && w.Tk > 0) return launch_window_bwd_tc(w, st);
  const dim3 gq((unsigned)tile_grid(w.Tq, kWarps, w.B), w.Hq), gk((unsigned)tile_grid(w.Tk, kWarps, w.B), w.Hkv);
  window_dq_rows_kernel<__nv_bfloat16><<<gq, 32 * kWarps, 0, st>>>(w);
  window_dkv_rows_kernel<__nv_bfloat16><<<gk, 32 * kWarps, 0, st>>>(w);
  return cudaGetLastError();
}

}  // namespace seq
}  // namespace pack3d
