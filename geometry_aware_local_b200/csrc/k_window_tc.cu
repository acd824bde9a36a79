// Causal windowed attention of packed sequences on sm_100a tensor cores (bf16).
//
//   o[i,h] = sum_{j in V(i)} softmax_j(c <q[i,h], k[j,g]>) v[j,g]
// with V(i) the window behind token i and the sequence's first `sinks` keys.
//
// One CTA = one 128-row query tile of one key head: rows are (token, query
// head) pairs of the group, 128/G tokens of one sequence x G heads, so the
// heads that share keys share every key tile.  The tile's visible keys are one
// range [lo, hi] (the first token's window to the last token) and, where the
// window has moved past them, the sinks in front.  Keys come in tiles of 32 from
// lo on, four CTAs an SM, or where a call has too few CTAs for that in tiles of
// 96, two an SM, the last tile and the sinks' one cut to a multiple of 32 columns
// (narrow() says when).  Masks are evaluated only in the 32-column chunks that
// some row sees in part.
//   * the last warp loads the Q tile and a ring of K / V tiles by TMA (boxes of
//     32 keys x 64 dims, 128-byte swizzle); the first loads are under way
//     before the CTA first meets;
//   * one warp issues tcgen05.mma: S = Q K^T (M=128, N = the tile's columns,
//     K=64) into tensor memory and O += P V (N=64) with P from tensor memory;
//   * four softmax warps (thread = row = TMEM lane) run the online softmax in
//     base 2 with a lazily moved maximum: O is rescaled only when a row maximum
//     grows by more than 2^8.
// Tensor memory of a CTA, 128 or 256 columns: two regions of a tile's width and
// O (64).  Tile j's S and then, over it, its P (packed bf16) are in region
// j % 2: a warp has its rows of S in registers before it writes P.  S of tile
// j + 1 is under way while tile j is exponentiated, and S of tile j + 2 follows
// the product with P of tile j.
//
// At d_h = 64 an exponential pairs with only 256 MMA flops, so the bound is the
// exponentials' rate (16 a clock and SM: 0.115 ms at the size below); what paces
// the kernel is the softmax warps' chain of a tile (wait, load, maximum,
// exponentials, store, arrive), so the number of CTAs that overlap theirs decides:
// narrow tiles let four share an SM's tensor memory and registers, although they
// pay each tile's barriers three times as often.  The code is kept small on
// purpose: the roles' loops evict one another from the instruction cache, and a
// second copy of the softmax body for tiles without masks made the kernel a
// quarter slower.
// 65,536 tokens, 8/2 heads, window 1,024, 4 sinks: 0.228 ms, 600 TFLOP/s, with
// narrow tiles; 0.288 with wide ones (0.298 with S and two P buffers apart, 0.320
// with persistent CTAs that walk the tiles).
//
// Few query tiles before many keys (a piece of a long prompt) would leave most
// SMs idle: then the CTAs of a cluster (2, 4 or 8) share a tile's key tiles and
// join their rows' maxima, sums and O through each other's shared memory.
//
// A key that a row does not see has P = 0 exactly; where its value row holds a
// NaN or an infinity, 0 times it is a NaN.  A row whose result is not finite is
// therefore computed again from its visible keys alone, unless what it sees makes it
// so (out_again).
#include <cooperative_groups.h>

#include "seq_tc.cuh"

namespace pack3d {
namespace seq {
namespace {

constexpr int kBM = kRowsPerTile;
constexpr int kMmaWarp = 4, kTmaWarp = 5, kThreads = 192;
constexpr int kQBytes = kBM * kDh * 2;
constexpr int kWide = 96;                       // columns of a key tile with two CTAs an SM; kSmallTile with four
// What the width of a key tile decides.
template <int BN>
struct Layout {
  using Tiles = KeyTiles<BN>;
  static constexpr int kCtas = 2, kStages = 3, kTmemCols = 256;
  static __device__ __forceinline__ Tiles tiles(const Win& w, int p0, int p1) { return key_tiles<BN>(w, p0, p1); }
};
template <>
struct Layout<kSmallTile> {
  using Tiles = SmallTiles;
  static constexpr int kCtas = 4, kStages = 4, kTmemCols = 128;
  static __device__ __forceinline__ Tiles tiles(const Win& w, int p0, int p1) { return small_tiles(w, p0, p1); }
};
template <int BN>
struct Smem {
  static constexpr int kStages = Layout<BN>::kStages, kTileBytes = BN * kDh * 2;
  static constexpr int kColO = 2 * BN;          // tile j: S, then P over it, at (j & 1) * BN
  static constexpr int kStageOff = kQBytes, kStageBytes = 2 * kTileBytes;      // K at +0, V at +kTileBytes
  static constexpr int kBarOff = kStageOff + kStages * kStageBytes;
  // barriers: full[S], empty[S], qfull, s_full[2], p_full[2], pv_done[2], o_final, drain, cleared
  static constexpr int kNumBars = 2 * kStages + 10;
  static constexpr int kCtlOff = kBarOff + kNumBars * 8;
  static constexpr int kPlanOff = kCtlOff + 32;
  static constexpr int kRedoOff = kPlanOff + 64;        // one byte a row
  static constexpr int kBytes = kRedoOff + kBM + 1024;
  static_assert(kColO + kDh <= Layout<BN>::kTmemCols, "tensor memory plan");
  static_assert(Layout<BN>::kCtas * (kBytes + 1024) <= 228 * 1024, "CTAs per SM");
};
constexpr float kRescaleThreshold = 8.0f;   // log2 units
constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(kBM, kDh, true);   // V MN-major

// What the softmax warps need of the CTA's tile at its edges and its end: kept
// in shared memory, so that it takes no registers in the loop over key tiles.
struct Plan {
  Tile s;
  int r0, r1;       // query rows
};
static_assert(sizeof(Plan) <= 64, "plan slot");

// A CTA's share of a tile that a cluster splits, over its K / V ring (which is
// idle by then): each row's O, maximum and sum.
struct Share {
  float o[kBM][kDh + 4];
  float m[kBM], l[kBM];
};
static_assert(sizeof(Share) <= Smem<kWide>::kStages * Smem<kWide>::kStageBytes, "share slot");

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// kSplit: the CTAs of a cluster along z share the tile's key tiles.
template <int kBN, bool kSplit>
__global__ void __launch_bounds__(kThreads, Layout<kBN>::kCtas)
window_attn_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Win w) {
  using M = Smem<kBN>;
  constexpr int kStages = M::kStages, kStageOff = M::kStageOff, kStageBytes = M::kStageBytes;
  constexpr int kTileBytes = M::kTileBytes, kTmemCols = Layout<kBN>::kTmemCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.y;
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t bar0 = sbase + M::kBarOff;
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto empty = [&](int s) { return bar0 + 8 * (kStages + s); };
  const uint32_t qfull = bar0 + 8 * (2 * kStages);
  const uint32_t o_final = qfull + 8, drain = qfull + 16;
  auto s_full = [&](int b) { return qfull + 24 + 8 * b; };
  auto p_full = [&](int b) { return qfull + 40 + 8 * b; };
  auto pv_done = [&](int b) { return qfull + 56 + 8 * b; };
  const uint32_t cleared = qfull + 72;
  volatile ptx::WaitCtl* ctl = reinterpret_cast<volatile ptx::WaitCtl*>(smem + M::kCtlOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + M::kCtlOff + sizeof(ptx::WaitCtl));
  auto wait = [&](uint32_t bar, uint32_t parity) { return wait_bounded(bar, parity, ctl); };
  const int tokens = kBM >> w.gshift;     // per tile

  // The producer sets the barriers up, and every warp finds the tile for
  // itself, so that the first loads are under way before the CTA meets.
  if (warp == kTmaWarp && lane == 0) {
    ptx::tma_prefetch(&tmQ);
    ptx::tma_prefetch(&tmK);
    ptx::tma_prefetch(&tmV);
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 1);
    }
    ptx::mbar_init(qfull, 1);
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(s_full(b), 1);
      ptx::mbar_init(p_full(b), 4);
      ptx::mbar_init(pv_done(b), 1);
    }
    ptx::mbar_init(o_final, 1);
    ptx::mbar_init(drain, 1);
    ptx::mbar_init(cleared, 1);
    ctl->abort = 0;
    ctl->issued = 0;
    ctl->limit_ns = w.wait_ns;
    ptx::fence_mbar_init();
  }
  __syncwarp();
  Tile s;
  bool bad;
  if (!find_tile(w, blockIdx.x, tokens, false, &s, &bad)) {
    if (bad) {
      if (threadIdx.x == 0) set_err(w.err, PACK3D_DEVERR_LENGTHS);
    } else if (w.zero_outside && blockIdx.y == 0 && blockIdx.z == 0) {
      constexpr int kWarps = kThreads / 32;
      fill_outside(w, w.cu_q, w.Tq, tokens, blockIdx.x, gridDim.x, kWarps, w.out, w.Hq * kDh / 2, 0u);
      if (w.lse) fill_outside(w, w.cu_q, w.Tq, tokens, blockIdx.x, gridDim.x, kWarps, w.lse, w.Hq, 0xff800000u);
    }
    return;
  }
  s.t = s.n - 1 - s.t;      // the tiles with most keys first
  const int r0 = s.t * tokens, r1 = min(s.lq, r0 + tokens) - 1;
  const int p0 = position(s, r0), p1 = position(s, r1);
  const typename Layout<kBN>::Tiles kt = Layout<kBN>::tiles(w, p0, p1);
  // This CTA's key tiles: [jo, jo + T).
  const int jo = kSplit ? (int)((long)kt.n * blockIdx.z / gridDim.z) : 0;
  const int T = kSplit ? (int)((long)kt.n * (blockIdx.z + 1) / gridDim.z) - jo : kt.n;
  const int T_load = w.stall ? max(T - 1, 0) : T;
  // Whether the last tile reaches behind the sequence's end.
  const bool tail = T > 0 && kt.begin(jo + T - 1) + kt.cols(jo + T - 1) > s.lk;
  volatile Plan* plan = reinterpret_cast<volatile Plan*>(smem + M::kPlanOff);
  volatile uint8_t* redo = smem + M::kRedoOff;
  auto load_tile = [&](int j) {
    const int st = j % kStages;
    const uint32_t dst = sbase + kStageOff + st * kStageBytes;
    const int cols = kt.cols(jo + j), row = s.k0 + kt.begin(jo + j);
    ptx::mbar_expect_tx(full(st), 2 * (cols / 32) * kChunkBytes);
#pragma unroll 1
    for (int c = 0; c < cols / 32; ++c) ptx::tma_load_3d(dst + c * kChunkBytes, &tmK, 0, g, row + 32 * c, full(st));
#pragma unroll 1
    for (int c = 0; c < cols / 32; ++c)
      ptx::tma_load_3d(dst + kTileBytes + c * kChunkBytes, &tmV, 0, g, row + 32 * c, full(st));
  };
  if (warp == kTmaWarp && lane == 0 && T > 0) {
    ptx::mbar_expect_tx(qfull, kQBytes);
    ptx::tma_load_4d(sbase, &tmQ, 0, 0, g, s.q0 + r0, qfull);
#pragma unroll 1
    for (int j = 0; j < min(T_load, kStages); ++j) load_tile(j);
    ctl->issued = min(T_load, kStages);
  }
  if (threadIdx.x == 0) *const_cast<Plan*>(plan) = Plan{s, r0, r1};
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  bool again = false;         // a row of this thread's is to be computed again
  if (warp == kTmaWarp) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      int issued = min(T_load, kStages);
#pragma unroll 1
      for (int j = issued; j < T_load; ++j) {
        if (!wait(empty(j % kStages), ((j / kStages) - 1) & 1)) break;
        load_tile(j);
        issued = j + 1;
      }
      ctl->issued = issued;
    }
    __syncwarp();
    if (tail) {
      const int st = (T - 1) % kStages;
      if (__all_sync(0xffffffffu, wait(full(st), ((T - 1) / kStages) & 1))) {
        clear_rows(sbase + kStageOff + st * kStageBytes + kTileBytes, s.lk - kt.begin(jo + T - 1), kt.cols(jo + T - 1));
        say_cleared(cleared);
      }
    }
  } else if (warp == kMmaWarp) {
    // ---------------- MMA issuer ----------------
    if (T > 0 && ptx::elect_one()) {
      const uint32_t tO = tmem + M::kColO;
      auto issue_s = [&](int j) {
        const uint32_t kaddr = sbase + kStageOff + (j % kStages) * kStageBytes;
        const uint32_t idesc = ptx::idesc_bf16_f32(kBM, kt.cols(jo + j), false);
#pragma unroll
        for (int kk = 0; kk < kDh / 16; ++kk)
          ptx::mma_ss(tmem + (j & 1) * kBN, ptx::smem_desc_sw128(sbase + kk * 32, 16, 1024),
                      ptx::smem_desc_sw128(kaddr + kk * 32, 16, 1024), idesc, kk > 0);
        ptx::tc_commit(s_full(j & 1));
      };
      auto issue_pv = [&](int j) {
        const uint32_t vaddr = sbase + kStageOff + (j % kStages) * kStageBytes + kTileBytes;
        const int cols = kt.cols(jo + j);
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          if (kk * 16 < cols)
            ptx::mma_ts(tO, tmem + (j & 1) * kBN + kk * 8, ptx::smem_desc_sw128(vaddr + kk * 2048, 8192, 1024),
                        kIdescPV, (j > 0 || kk > 0) ? 1u : 0u);
        ptx::tc_commit(pv_done(j & 1));
        ptx::tc_commit(empty(j % kStages));
        if (j == T - 1) ptx::tc_commit(o_final);
      };
      const int tail_tile = tail ? T - 1 : T;
      bool ok = wait(qfull, 0);
#pragma unroll 1
      for (int j = -2; ok && j < T; ++j) {
        if (j >= 0) {
          if (!(ok = wait(p_full(j & 1), (j >> 1) & 1))) break;
          if (j == tail_tile && !(ok = wait(cleared, 0))) break;
          ptx::tc_fence_after();
          issue_pv(j);
        }
        if (j + 2 < T) {
          // S of tile j + 2 goes where P of tile j is: once its product is done.
          if (!(ok = (j < 0 || wait(pv_done(j & 1), (j >> 1) & 1)) && wait(full((j + 2) % kStages), ((j + 2) / kStages) & 1)))
            break;
          ptx::tc_fence_after();
          issue_s(j + 2);
        }
      }
    }
    __syncwarp();
  } else {
    // ---------------- softmax warps: thread = row = tensor-memory lane ----------------
    const int lane_base = warp * 32;
    const uint32_t trow = tmem + ((uint32_t)lane_base << 16);
    const uint32_t tO = trow + M::kColO;
    const float c = w.scale_log2;
    // A 32-key chunk is seen in full by every row if it lies in [full_lo,
    // full_hi]: behind the last row's window start and not past the first row's
    // own key (and every row is one of the sequence).
    const int full_lo = window_low(w, p1), full_hi = r0 + tokens > s.lq ? -1 : p0;
    float m_used = -INFINITY, l = 0.f;
    bool ok = true;
    auto warp_arrive = [&](uint32_t bar) {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar);
    };
#pragma unroll 1
    for (int j = 0; j < T; ++j) {
      const int k0 = kt.begin(jo + j), cols = kt.cols(jo + j);
      if (!(ok = __all_sync(0xffffffffu, wait(s_full(j & 1), (j >> 1) & 1)))) break;
      ptx::tc_fence_after();
      const uint32_t tS = trow + (j & 1) * kBN;
      uint32_t sv[kBN];
      if constexpr (kBN == kSmallTile) {
        ptx::tmem_ld32_sync(tS, sv);
      } else {
        if (cols > 32) ptx::tmem_ld64_sync(tS, sv);
        else ptx::tmem_ld32_sync(tS, sv);
        if (cols > 64) ptx::tmem_ld32_sync(tS + 64, sv + 64);
      }
      float mx = -INFINITY;
#pragma unroll
      for (int q = 0; q < kBN / 32; ++q) {
        if (32 * q >= cols) break;
        const int c0 = k0 + 32 * q;
        if (c0 < full_lo || c0 + 31 > full_hi) {
          const int r = plan->r0 + ((lane_base + lane) >> w.gshift);        // this row's token in its sequence
          const int p = r <= plan->r1 ? plan->s.lk - plan->s.lq + r : -1;   // rows past the sequence see nothing
          const uint32_t see = visible_bits(w, p, window_low(w, p), c0);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!((see >> k) & 1u)) sv[32 * q + k] = __float_as_uint(-INFINITY);
        }
        float m4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          m4[e] = fmaxf(__uint_as_float(sv[32 * q + 2 * e]), __uint_as_float(sv[32 * q + 2 * e + 1]));
#pragma unroll
        for (int k = 8; k < 32; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            m4[e] = max3(m4[e], __uint_as_float(sv[32 * q + k + 2 * e]), __uint_as_float(sv[32 * q + k + 2 * e + 1]));
        mx = max3(mx, max3(m4[0], m4[1], m4[2]), m4[3]);
      }
      const float mxs = mx * c;
      float f = 1.f;
      if (j == 0) m_used = mxs;
      else if (mxs > m_used + kRescaleThreshold) {
        f = ptx::ex2(m_used - mxs);
        m_used = mxs;
      }
      const bool rescale = j > 0 && __any_sync(0xffffffffu, f != 1.f);
      // A row that has seen no key yet (maximum -infinity) has only scores of
      // -infinity here: any finite shift gives their weight 0.
      const float shift = m_used == -INFINITY ? 0.f : -m_used;
      const float2 c2 = make_float2(c, c), nm2 = make_float2(shift, shift);
      float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int q = 0; q < kBN / 32; ++q) {
        if (32 * q >= cols) break;
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int e = 32 * q + 2 * k;
          const float2 y = __ffma2_rn(make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), c2, nm2);
          const float2 pr = make_float2(ptx::ex2(y.x), ptx::ex2(y.y));
          rs[k & 1] = __fadd2_rn(rs[k & 1], pr);
          pk[k] = pack_bf16x2(pr.x, pr.y);
        }
        ptx::tmem_st16(tS + 16 * q, pk);
      }
      if (rescale) {
        // After the last tile's O += P V and before this one's.
        if (!(ok = __all_sync(0xffffffffu, wait(pv_done((j - 1) & 1), ((j - 1) >> 1) & 1)))) break;
        ptx::tc_fence_after();
        uint32_t o[16];
#pragma unroll
        for (int q = 0; q < kDh / 16; ++q) {
          ptx::tmem_ld16_sync(tO + 16 * q, o);
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
          ptx::tmem_st16(tO + 16 * q, o);
        }
      }
      ptx::tmem_wait_st();
      warp_arrive(p_full(j & 1));
      l = l * f + ((rs[0].x + rs[0].y) + (rs[1].x + rs[1].y));
    }
    if (T == 0 || (ok && __all_sync(0xffffffffu, wait(o_final, 0)))) {
      const Tile at = *const_cast<const Tile*>(&plan->s);
      const int row = lane_base + lane, r0 = plan->r0, r = r0 + (row >> w.gshift);
      const bool valid = r <= plan->r1;
      const int h = (g << w.gshift) + (row & (w.G - 1));
      const size_t orow = (size_t)(at.q0 + r) * w.Hq + h;
      uint32_t o[kDh];
      if (T > 0) {
        ptx::tc_fence_after();
        ptx::tmem_ld64_sync(tO, o);
      } else {
#pragma unroll
        for (int e = 0; e < kDh; ++e) o[e] = 0u;
      }
      if constexpr (kSplit) {
        Share* mine = reinterpret_cast<Share*>(smem + kStageOff);
#pragma unroll
        for (int e = 0; e < kDh; e += 4)
          *reinterpret_cast<uint4*>(&mine->o[row][e]) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        mine->m[row] = m_used;
        mine->l[row] = l;
      } else {
        // l == 0: the row sees no key (its O is 0, or a NaN from a hidden value).
        const float inv = l == 0.f ? 0.f : 1.f / l;
        float sum = 0.f;                                 // not finite where any element is not
#pragma unroll
        for (int e = 0; e < kDh; ++e) {
          const float x = __uint_as_float(o[e]) * inv;
          sum = fmaf(x, 0.f, sum);
          o[e] = __float_as_uint(x);
        }
        // (A denominator that is a NaN is made of visible scores alone.)
        redo[row] = again = valid && !(sum == 0.f) && l == l;
        if (valid) {
          uint4* dst = reinterpret_cast<uint4*>((__nv_bfloat16*)w.out + orow * kDh);
#pragma unroll
          for (int q = 0; q < kDh / 8; ++q) {
            const float* x = reinterpret_cast<const float*>(o + 8 * q);
            dst[q] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                pack_bf16x2(x[6], x[7]));
          }
          if (w.lse) w.lse[orow] = l == 0.f ? -INFINITY : (m_used + log2f(l)) * 0.69314718f;
        }
      }
    }
  }

  ptx::tc_fence_before();
  const bool some_again = __syncthreads_or(again);
  if (ctl->abort) {
    // Every role has finished.  Before tensor memory and shared memory are
    // released, the MMAs and the loads this CTA started complete.
    if (warp == kMmaWarp && lane == 0) {
      ptx::tc_commit(drain);
      ptx::mbar_wait_drain(drain, 0, ctl->limit_ns);
    }
    if (warp == kTmaWarp && lane == 0) {
      ptx::mbar_wait_drain(qfull, 0, ctl->limit_ns);
      const int issued = ctl->issued;
      for (int j = max(0, issued - kStages); j < issued; ++j)
        ptx::mbar_wait_drain(full(j % kStages), (j / kStages) & 1, ctl->limit_ns);
    }
    ptx::tc_fence_before();
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && ctl->abort) set_err(w.err, PACK3D_DEVERR_TIMEOUT);
  if constexpr (!kSplit) {
    if (!some_again || ctl->abort) return;
#pragma unroll 1
    for (int row = warp; row < kBM; row += kThreads / 32)
      if (redo[row]) out_again<__nv_bfloat16>(w, s, r0 + (row >> w.gshift), (g << w.gshift) + (row & (w.G - 1)));
  } else {
    // Every CTA of the cluster comes here, whatever its waits did.  CTA z joins
    // the rows z * 128 / S .., a warp a row, the shares in the keys' order.
    auto cluster = cooperative_groups::this_cluster();
    cluster.sync();
    Share* mine = reinterpret_cast<Share*>(smem + kStageOff);
    const Tile at = *const_cast<const Tile*>(&plan->s);
    const int S = gridDim.z, rows = kBM / S, r0 = plan->r0, r1 = plan->r1;
#pragma unroll 1
    for (int row = blockIdx.z * rows + warp; row < (int)(blockIdx.z + 1) * rows; row += kThreads / 32) {
      const int r = r0 + (row >> w.gshift), h = (g << w.gshift) + (row & (w.G - 1));
      if (r > r1) continue;
      const Share* other = cluster.map_shared_rank(mine, min(lane, S - 1));
      const float m = lane < S ? other->m[row] : -INFINITY;
      float top = m;
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      top = __shfl_sync(0xffffffffu, top, 0);
      const float f = m == top ? 1.f : ptx::ex2(m - top);
      const float part = lane < S ? other->l[row] * f : 0.f;
      float l = 0.f;
      float2 o = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int z = 0; z < S; ++z) {
        const float fz = __shfl_sync(0xffffffffu, f, z);
        l += __shfl_sync(0xffffffffu, part, z);
        const float2 x = *reinterpret_cast<const float2*>(&cluster.map_shared_rank(mine, z)->o[row][2 * lane]);
        o.x = fmaf(x.x, fz, o.x);
        o.y = fmaf(x.y, fz, o.y);
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      o.x *= inv;
      o.y *= inv;
      const size_t orow = (size_t)(at.q0 + r) * w.Hq + h;
      store2((__nv_bfloat16*)w.out + orow * kDh, o);
      if (w.lse && lane == 0) w.lse[orow] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718f;
      const bool again = l == l && __any_sync(0xffffffffu, !(fmaf(o.x, 0.f, o.y * 0.f) == 0.f));
      __syncwarp();
      if (again) out_again<__nv_bfloat16>(w, at, r, h);
    }
    cluster.sync();           // no CTA ends while another reads its share
  }
}

// CTAs of a cluster per query tile: as many as keep two CTAs an SM busy and
// leave each at least four key tiles (2,048 queries before 16,384 keys, 8 heads
// to one key head: 0.197 ms with 1, 0.130 with 2, 0.138 with 4).
int split_of(const Win& w, long tiles) {
  const long keys = w.window > 0 ? min((long)w.Tk, (long)w.window + 2 * kWide) : w.Tk;
  int S = 1;
  while (S < 8 && tiles * w.Hkv * S * 2 <= 2L * sm_count() && keys / kWide >= 8L * S) S *= 2;
  return S;
}

// Whether the key tiles are narrow, with four CTAs an SM: where there are CTAs
// for them.  Without a window the CTAs' lengths differ, and it takes more than
// four an SM for the short ones to fill the gaps.  Narrow against wide: 65,536
// tokens, window 1,024 0.228 : 0.288 ms; 6,300 tokens, 8 key heads, window 256
// (400 CTAs) 21 : 26 us; 4,096, window 512 (256) 19.3 : 18.6; 8,192, no window
// (512) 162 : 155; the same with 16 heads (1,024) 225 : 238.
bool narrow(const Win& w, long tiles) {
  return tiles * w.Hkv > (w.window > 0 ? 2L : 4L) * sm_count();
}

template <int BN, bool kSplit>
cudaError_t launch_tc(const Win& w, const dim3& grid, cudaStream_t st) {
  constexpr int kBytes = Smem<BN>::kBytes;
  // First, so that a thread that has made no CUDA call yet (autograd's) has the
  // device's context when the tensor maps are encoded.
  cudaError_t e = cudaFuncSetAttribute(window_attn_tc_kernel<BN, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kBytes);
  if (e != cudaSuccess) return e;
  CUtensorMap tq, tk, tv;
  if (!map_query_rows(&tq, w, w.q) || !map_key_rows(&tk, w, w.k, 32) || !map_key_rows(&tv, w, w.v, 32))
    return cudaErrorInvalidValue;
  if constexpr (!kSplit) {
    window_attn_tc_kernel<BN, false><<<grid, kThreads, kBytes, st>>>(tq, tk, tv, w);
    return cudaGetLastError();
  }
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = cluster.val.clusterDim.y = 1;
  cluster.val.clusterDim.z = grid.z;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = st;
  cfg.attrs = &cluster;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, window_attn_tc_kernel<BN, kSplit>, tq, tk, tv, w);
}

}  // namespace

cudaError_t launch_window_attn_tc(const Win& w, cudaStream_t st) {
  const long tiles = tile_grid(w.Tq, kBM >> w.gshift, w.B);
  if (narrow(w, tiles - 1)) return launch_tc<kSmallTile, false>(w, dim3((unsigned)tiles, w.Hkv), st);
  const int S = split_of(w, tiles - 1);
  if (S == 1) return launch_tc<kWide, false>(w, dim3((unsigned)tiles, w.Hkv), st);
  return launch_tc<kWide, true>(w, dim3((unsigned)tiles, w.Hkv, S), st);
}

}  // namespace seq
}  // namespace pack3d
