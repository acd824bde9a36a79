// Shared parts of the tensor-core kernels of the causal sequence operators: the
// key tiles a query tile reads, the visibility of a 32-key chunk as a bit mask
// and the TMA maps.
#pragma once

#include <cuda.h>

#include "seq.cuh"
#include "tc_ptx.cuh"
#include "tma_host.cuh"

namespace pack3d {
namespace seq {

constexpr int kRowsPerTile = 128;                     // (token, query head) rows of a query tile
constexpr int kChunkBytes = 32 * kDh * 2;             // 32 keys of one head

// mbar_wait with its slow half out of line: the roles' loops stay short.
__device__ __noinline__ inline bool wait_on(uint32_t bar, uint32_t parity, volatile ptx::WaitCtl* ctl) {
  return ptx::mbar_wait(bar, parity, ctl);
}
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile ptx::WaitCtl* ctl) {
  return ptx::mbar_try_wait(bar, parity) || wait_on(bar, parity, ctl);
}

// A box reaches behind the end of its sequence, where the next one's rows lie or rows
// of no sequence; multiplied by zeros in a tile's second products they would be NaNs
// wherever they are not finite.  So the producer's warp, which is idle by then, puts
// zeros into the rows [from, to) of the sequence's last tile (rows of 128 bytes) when
// the tile is there, and says so on a barrier.
__device__ __forceinline__ void clear_rows(uint32_t tile, int from, int to) {
#pragma unroll 1
  for (int i = 8 * from + (threadIdx.x & 31); i < 8 * to; i += 32) ptx::st_shared_v4(tile + 16 * i, 0u, 0u, 0u, 0u);
  ptx::fence_proxy_async_smem();
}
__device__ __forceinline__ void say_cleared(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar);
}

// The key tiles of a query tile: number j starts at key begin(j) of the
// sequence and has cols(j) columns, a multiple of 32, BN at most.
template <int BN>
struct KeyTiles {
  int lo, hi;       // the tile's range of keys
  int sink_cols;    // columns of the sinks' tile in front of it, or 0
  int n;
  __device__ __forceinline__ int begin(int j) const {
    return sink_cols ? (j == 0 ? 0 : lo + (j - 1) * BN) : lo + j * BN;
  }
  __device__ __forceinline__ int cols(int j) const {
    return sink_cols && j == 0 ? sink_cols : min(BN, (hi - begin(j) + 32) & ~31);
  }
};

// Keys of the queries at positions p0 .. p1 (p0 <= p1) of a sequence.
template <int BN>
__device__ __forceinline__ KeyTiles<BN> key_tiles(const Win& w, int p0, int p1) {
  KeyTiles<BN> k;
  k.hi = p1;
  k.sink_cols = 0;
  if (p1 < 0) {
    k.lo = 0;
    k.n = 0;
    return k;
  }
  k.lo = window_low(w, max(p0, 0));
  const int sinks = min(w.sinks, k.lo);
  // One range from key 0 where the sinks' columns would reach the window.
  if (sinks > 0) {
    if (((sinks + 31) & ~31) >= k.lo) k.lo = 0;
    else k.sink_cols = (sinks + 31) & ~31;
  }
  k.n = (k.hi - k.lo) / BN + 1 + (k.sink_cols ? 1 : 0);
  return k;
}

// The same in tiles of 32 columns: the sinks' (one or two) in front.
constexpr int kSmallTile = 32;
struct SmallTiles {
  int lo, sink_tiles, n;
  __device__ __forceinline__ int begin(int j) const {
    return j < sink_tiles ? j * kSmallTile : lo + (j - sink_tiles) * kSmallTile;
  }
  static __device__ __forceinline__ constexpr int cols(int) { return kSmallTile; }
};
__device__ __forceinline__ SmallTiles small_tiles(const Win& w, int p0, int p1) {
  const KeyTiles<2 * kSmallTile> k = key_tiles<2 * kSmallTile>(w, p0, p1);      // a tile holds every sink
  const int sink_tiles = k.sink_cols / kSmallTile;
  return SmallTiles{k.lo, sink_tiles, p1 < 0 ? 0 : (k.hi - k.lo) / kSmallTile + 1 + sink_tiles};
}

// Bit k: the query at position p (window start `low`) sees key c0 + k.  p < 0:
// none.
__device__ __forceinline__ uint32_t visible_bits(const Win& w, int p, int low, int c0) {
  const int a = max(low - c0, 0), z = p - c0;
  const uint32_t upto = z < 0 ? 0u : (z >= 31 ? 0xffffffffu : (2u << z) - 1u);
  const int first = min(max(w.sinks - c0, 0), 32);
  const uint32_t sink = first >= 32 ? 0xffffffffu : (1u << first) - 1u;
  return upto & ((a >= 32 ? 0u : 0xffffffffu << a) | sink);
}

// Query-shaped tensor [Tq][Hq][64] viewed as [Tq][Hkv][G][64]: a box of rows/G
// tokens x G heads x 64 dims of one key head is one tile of `rows` rows.
inline bool map_query_rows(CUtensorMap* m, const Win& w, const void* base, int rows = kRowsPerTile) {
  const cuuint64_t dims[4] = {(cuuint64_t)kDh, (cuuint64_t)w.G, (cuuint64_t)w.Hkv, (cuuint64_t)w.Tq};
  const cuuint64_t strides[3] = {(cuuint64_t)kDh * 2, (cuuint64_t)w.G * kDh * 2, (cuuint64_t)w.Hq * kDh * 2};
  const cuuint32_t box[4] = {(cuuint32_t)kDh, (cuuint32_t)w.G, 1, (cuuint32_t)(rows / w.G)};
  return tma::encode_bf16_sw128(m, base, 4, dims, strides, box);
}

// Key-shaped tensor [Tk][Hkv][64], boxes of `rows` keys of one key head.
inline bool map_key_rows(CUtensorMap* m, const Win& w, const void* base, int rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)kDh, (cuuint64_t)w.Hkv, (cuuint64_t)w.Tk};
  const cuuint64_t strides[2] = {(cuuint64_t)kDh * 2, (cuuint64_t)w.Hkv * kDh * 2};
  const cuuint32_t box[3] = {(cuuint32_t)kDh, 1, (cuuint32_t)rows};
  return tma::encode_bf16_sw128(m, base, 3, dims, strides, box);
}

}  // namespace seq
}  // namespace pack3d
