// Attention of one new token per sequence over the paged cache, one warp per
// (sequence, query head).
#include "seq.cuh"

namespace pack3d {
namespace seq {
namespace {

template <typename T>
__global__ void __launch_bounds__(32) cache_attn_row_kernel(const Cache c, const T* __restrict__ q, T* out,
                                                            float* lse, float* row_lse) {
  const int b = blockIdx.x, h = blockIdx.y, g = h / c.G;
  const int n = cached(c, b), low = c.window > 0 ? max(0, n - c.window) : 0;
  const size_t at = (size_t)b * c.Hq + h, step = (size_t)c.Hkv * kDh;
  const T* k = (const T*)c.k_pages + (size_t)g * kDh;
  const T* v = (const T*)c.v_pages + (size_t)g * kDh;
  const int32_t* row = c.table + (size_t)b * c.max_pages;
  const float2 qq = load2(q + at * kDh);
  float m = -INFINITY, l = 0.f;
  float2 o = make_float2(0.f, 0.f);
  for (int j = 0; j < n; ++j) {
    if (j >= c.sinks && j < low) continue;
    const long src = pool_row(c, row, j);
    if (src < 0) continue;
    const float x = dot2(qq, load2(k + src * step)) * c.scale;
    const float2 vv = load2(v + src * step);
    float f = 1.f;
    if (x > m) {
      f = expf(m - x);
      m = x;
    }
    const float e = x == -INFINITY ? 0.f : expf(x - m);
    l = l * f + e;
    o.x = fmaf(e, vv.x, o.x * f);
    o.y = fmaf(e, vv.y, o.y * f);
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  store2(out + at * kDh, make_float2(o.x * inv, o.y * inv));
  if ((threadIdx.x & 31) == 0) {
    if (lse) lse[at] = m + logf(l);
    row_lse[at] = m + logf(l);
  }
}

template <typename T>
__global__ void __launch_bounds__(128) cache_weights_row_kernel(const Cache c, const T* __restrict__ q,
                                                                const float* __restrict__ row_lse, float* weights,
                                                                int accumulate) {
  const int b = blockIdx.y;
  const int n = cached(c, b), low = c.window > 0 ? max(0, n - c.window) : 0;
  const size_t step = (size_t)c.Hkv * kDh;
  const int32_t* row = c.table + (size_t)b * c.max_pages;
  for (int j = blockIdx.x * 4 + (threadIdx.x >> 5); j < n; j += gridDim.x * 4) {
    float total = 0.f;
    if (j < c.sinks || j >= low) {
      const long src = pool_row(c, row, j);
      if (src >= 0)
        for (int h = 0; h < c.Hq; ++h) {
          const size_t at = (size_t)b * c.Hq + h;
          const float x = dot2(load2(q + at * kDh), load2((const T*)c.k_pages + src * step + (h / c.G) * kDh));
          total += expf(x * c.scale - row_lse[at]);
        }
    }
    if ((threadIdx.x & 31) == 0) {
      float* dst = weights + (size_t)b * c.cap + j;
      *dst = accumulate ? *dst + total : total;
    }
  }
}

template <typename T>
cudaError_t launch_t(const Cache& c, const void* q, void* out, float* lse, float* weights, bool accumulate,
                     void* workspace, cudaStream_t st) {
  float* row_lse = (float*)workspace;
  cache_attn_row_kernel<T><<<dim3(c.B, c.Hq), 32, 0, st>>>(c, (const T*)q, (T*)out, lse, row_lse);
  if (weights)
    cache_weights_row_kernel<T><<<dim3((c.cap + 63) / 64, c.B), 128, 0, st>>>(c, (const T*)q, row_lse, weights,
                                                                              accumulate);
  return cudaGetLastError();
}

}  // namespace

size_t cache_attn_workspace(int B, int Hq, int Hkv, int cap, bool weights) {
  return ((size_t)B * Hq * 4 + 1023) / 1024 * 1024;
}

cudaError_t launch_cache_attn(const Cache& c, int dtype, const void* q, void* out, float* lse, float* weights,
                              bool accumulate, void* workspace, cudaStream_t st) {
  if (dtype == PACK3D_BF16) return launch_t<__nv_bfloat16>(c, q, out, lse, weights, accumulate, workspace, st);
  return launch_t<float>(c, q, out, lse, weights, accumulate, workspace, st);
}

}  // namespace seq
}  // namespace pack3d
