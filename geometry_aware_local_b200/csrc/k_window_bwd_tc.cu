// Gradients of the causal windowed attention on sm_100a tensor cores (bf16).
//
// With c = scale log2(e), lse2 the row's log-sum-exp in base 2 and
// D = <dout, out>, over the visible pairs:
//   P = 2^(c S - lse2), S = Q K^T (recomputed),  dP = dout V^T,  dS = P (dP - D)
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dout.
//
// window_dq_tc_kernel: one 128-row query tile of one key head per CTA (rows,
//   key range and sinks as in the forward), 32 keys a step, two CTAs per SM.
//   One MMA warp issues S and dP into tensor memory (N = 32 keys, K = 64); two
//   groups of four softmax warps (thread = row) take every other step, each with
//   its own tensor memory, and write dS there as packed bf16; a second MMA warp
//   issues dQ += dS K with the same K tile read MN-major.  It also forms D of its
//   rows and leaves it for the second kernel.  (65,536 tokens, window 1,024, both
//   kernels: one group and 64 keys a step 0.748 ms, two warps a row quarter on the
//   same step 0.751, two groups 0.711.)
//
// window_dkv_tc_kernel: one 128-key tile of one key head per CTA and the
//   queries whose window reaches it, 64 rows a step, one CTA per SM.  S^T and
//   dP^T (M = 128 keys, N = 64 rows) go to tensor memory, already less the rows'
//   lse / scale and D: one more product of K = 16, a column of ones by each term
//   in three bf16 pieces, which the query side leaves beside D.  The softmax warps
//   (thread = key, a 32-row chunk of the step each) write dS^T and P^T beside
//   them as packed bf16, from where a second MMA warp accumulates
//   dK += dS^T Q and dV += P^T dout (M = 128 keys, N = 64, K = 64 rows).  Two
//   groups of eight softmax warps take every other step, each with its own
//   tensor memory.  Where no key of a warp is seen by any row of its chunk it
//   writes zeros without an exponential.  Where there are few key tiles the CTAs
//   of a cluster share a tile's steps and join their dK and dV through each
//   other's shared memory (split_of).
//   65,536 tokens, window 1,024 / 8,192 tokens, 16 / 2 heads, no window, both
//   kernels: S and dP by rows, dS and P through 64 KiB of shared memory for the
//   second product 0.874 / - ms; transposed, with the terms added by the threads
//   from shared memory 0.837 / 0.963; two groups 0.807 / 0.910; the terms added by
//   the tensor cores 0.748 / 0.786.  (A thread's load of 16 bytes that every lane
//   wants is four passes of shared memory, which the products' operands need.)
//
// The first key tile of a sequence holds its sinks, which every later query
// sees.  Their gradients from the queries beyond the tile's window are formed
// by further CTAs of the same kernel, far_steps query tiles each, which like
// the tile itself leave float partial sums of the sink rows; window_sinks_kernel
// adds them in a fixed order.  No atomics: the same inputs give the same bits.
//
// 65,536 tokens, 8 / 2 heads, window 1,024, 4 sinks: 0.69 ms, 498 TFLOP/s (five
// products), about 0.33 ms of it the query side.  As in the forward the pace is
// that of the softmax warps' chains (load, exponentials, store, arrive), not of
// the tensor cores.
//
// A gradient row that is not finite may be spoilt by 0 times a NaN or an
// infinity of a row it does not depend on; it is computed again from its
// visible pairs alone, unless those make it so (dq_again, dkv_row).
#include <cooperative_groups.h>

#include "seq_tc.cuh"
#include "window_sinks.cuh"

namespace pack3d {
namespace seq {
namespace {

constexpr int kQTileBytes = kRowsPerTile * kDh * 2;   // 16 KiB
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  ptx::tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar);
}

// A term of row `orow` for the key side's products, as three bf16 pieces whose sum
// is off by 2^-24 of it: each takes what the ones before leave.  (The largest floats
// would round up to infinity; an infinity or a NaN is a first piece alone.)
__device__ __forceinline__ void write_terms(const Win& w, int plane, size_t orow, float x) {
  constexpr float kMax = 3.3895314e38f;                 // bf16's largest
  const bool finite = fabsf(x) < INFINITY;
  const float hi = finite ? fminf(fmaxf(__bfloat162float(__float2bfloat16(x)), -kMax), kMax) : x;
  const float rest = finite ? x - hi : 0.f, mid = __bfloat162float(__float2bfloat16(rest));
  reinterpret_cast<uint4*>(w.terms)[(size_t)plane * w.Tq * w.Hq + orow] =
      make_uint4(pack_bf16x2(hi, mid), pack_bf16x2(rest - mid, 0.f), 0u, 0u);
}

// The halves of a bf16 pair that bits 2 k and 2 k + 1 of `see` keep.
__device__ __forceinline__ uint32_t kept_pair(uint32_t see, int k) {
  return ((see >> (2 * k)) & 1u ? 0xffffu : 0u) | ((see >> (2 * k + 1)) & 1u ? 0xffff0000u : 0u);
}

// ============================================================================
// Query side
// ============================================================================
namespace q_side {

constexpr int kBN = kSmallTile;
// Two groups of softmax warps on alternate steps; two MMA warps; TMA warp.
constexpr int kSoftmaxWarps = 8, kThreads = 32 * (kSoftmaxWarps + 3);
constexpr int kMmaWarp = kSoftmaxWarps, kMmaWarp2 = kSoftmaxWarps + 1, kTmaWarp = kSoftmaxWarps + 2;
// Group b's S, dP and dS (packed bf16) at 80 b, + 32, + 64.
constexpr int kGroupCols = 2 * kBN + kBN / 2, kColDQ = 2 * kGroupCols, kTmemCols = 256;
static_assert(kColDQ + kDh <= kTmemCols, "tensor memory plan");
constexpr int kKVBytes = kBN * kDh * 2;         // 4 KiB
constexpr int kStages = 8;
constexpr int kQOff = 0, kDOOff = kQTileBytes, kStageOff = 2 * kQTileBytes;
constexpr int kStageBytes = 2 * kKVBytes;       // K at +0, V at +kKVBytes
constexpr int kBarOff = kStageOff + kStages * kStageBytes;
// barriers: full[S], empty[S], qfull, o_final, s_full[2], s_free[2], p_full[2], p_free[2], drain[2], landed
constexpr int kNumBars = 2 * kStages + 13;
constexpr int kCtlOff = kBarOff + kNumBars * 8;
constexpr int kHalfOff = kCtlOff + 32;          // float [2][128]: the groups' shares of D
constexpr int kRedoOff = kHalfOff + 2 * kRowsPerTile * 4;       // one byte per row
constexpr int kSmemBytes = kRedoOff + kRowsPerTile + 1024;
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");
// Row tiles of at most this many key tiles form D from P and dP in a first pass
// over them.  <dout, out> of the rounded out is off by 2^-9 of its terms, which
// where a row sees a few dozen keys is as much as all of dS's rounding (dQ and
// dK off by 1.5 to 1.8 times bf16's own rounding, now 1.4); where it sees more
// it averages out.  The tiles stay in shared memory for the second pass, so
// the first costs two products and the exponentials, and saves the reads of out
// and dout by rows (65,536 tokens, window 65: 245 us without, 218 with it; with 4
// sinks 301, 281).
constexpr int kTwice = 6;
static_assert(kTwice <= kStages, "the first pass's tiles stay");
constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(kRowsPerTile, kBN, false);
constexpr uint32_t kIdescDQ = ptx::idesc_bf16_f32(kRowsPerTile, kDh, true);  // dQ: N = 64 dims, K MN-major

__global__ void __launch_bounds__(kThreads, 2)
window_dq_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ Win w) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.y;
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t bar0 = sbase + kBarOff;
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto empty = [&](int s) { return bar0 + 8 * (kStages + s); };
  const uint32_t qfull = bar0 + 8 * (2 * kStages);
  const uint32_t o_final = qfull + 8;
  auto s_full = [&](int b) { return qfull + 16 + 8 * b; };
  auto s_free = [&](int b) { return qfull + 32 + 8 * b; };
  auto p_full = [&](int b) { return qfull + 48 + 8 * b; };
  auto p_free = [&](int b) { return qfull + 64 + 8 * b; };
  auto drain = [&](int i) { return qfull + 80 + 8 * i; };
  const uint32_t landed = qfull + 96;          // for the tile that is cleared in part
  float* shares = reinterpret_cast<float*>(smem + kHalfOff);
  volatile uint8_t* redo = smem + kRedoOff;
  volatile ptx::WaitCtl* ctl = reinterpret_cast<volatile ptx::WaitCtl*>(smem + kCtlOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kCtlOff + sizeof(ptx::WaitCtl));
  auto wait = [&](uint32_t bar, uint32_t parity) { return wait_bounded(bar, parity, ctl); };
  const int tokens = kRowsPerTile >> w.gshift;

  let_next_begin();
  // The producer sets the barriers up, and every warp finds the tile for
  // itself, so that the first loads are under way before the CTA meets.
  if (warp == kTmaWarp && lane == 0) {
    ptx::tma_prefetch(&tmQ);
    ptx::tma_prefetch(&tmO);
    ptx::tma_prefetch(&tmK);
    ptx::tma_prefetch(&tmV);
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 1);
    }
    ptx::mbar_init(qfull, 1);
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(s_full(b), 1);
      ptx::mbar_init(s_free(b), 4);
      ptx::mbar_init(p_full(b), 4);
      ptx::mbar_init(p_free(b), 1);
      ptx::mbar_init(drain(b), 1);
    }
    ptx::mbar_init(o_final, 1);
    ptx::mbar_init(landed, 1);
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
    } else if (w.zero_outside && blockIdx.y == 0) {
      fill_outside(w, w.cu_q, w.Tq, tokens, blockIdx.x, gridDim.x, kThreads / 32, w.dq, w.Hq * kDh / 2, 0u);
    }
    return;
  }
  s.t = s.n - 1 - s.t;      // the tiles with most keys first
  const int r0 = s.t * tokens, r1 = min(s.lq, r0 + tokens) - 1;
  const int p0 = position(s, r0), p1 = position(s, r1);
  const SmallTiles kt = small_tiles(w, p0, p1);
  const int T = kt.n, T_load = w.stall ? T - 1 : T;
  const int first = T <= kTwice ? T : 0;      // steps of the first pass
  const bool tail = T > 0 && kt.begin(T - 1) + kBN > s.lk;      // the last tile reaches behind the sequence's end
  auto load_tile = [&](int j) {
    const int st = j % kStages;
    const uint32_t dst = sbase + kStageOff + st * kStageBytes;
    const uint32_t bar = tail && j == T - 1 ? landed : full(st);
    ptx::mbar_expect_tx(bar, kStageBytes);
    ptx::tma_load_3d(dst, &tmK, 0, g, s.k0 + kt.begin(j), bar);
    ptx::tma_load_3d(dst + kKVBytes, &tmV, 0, g, s.k0 + kt.begin(j), bar);
  };
  if (warp == kTmaWarp && lane == 0 && T > 0) {
    ptx::mbar_expect_tx(qfull, 2 * kQTileBytes);
    ptx::tma_load_4d(sbase + kQOff, &tmQ, 0, 0, g, s.q0 + r0, qfull);
    ptx::tma_load_4d(sbase + kDOOff, &tmO, 0, 0, g, s.q0 + r0, qfull);
#pragma unroll 1
    for (int j = 0; j < min(T_load, kStages); ++j) load_tile(j);
    ctl->issued = min(T_load, kStages);
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  bool again = false;                   // something of this thread's row is not finite
  if (warp == kTmaWarp) {
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
      if (__all_sync(0xffffffffu, wait(landed, 0))) {
        clear_rows(sbase + kStageOff + st * kStageBytes, s.lk - kt.begin(T - 1), kBN);
        say_cleared(full(st));
      }
    }
  } else if (warp == kMmaWarp || warp == kMmaWarp2) {
    if (T > 0 && ptx::elect_one()) {
      const uint32_t tDQ = tmem + kColDQ;
      auto issue_sdp = [&](int j, int b) {
        const uint32_t kaddr = sbase + kStageOff + (j % kStages) * kStageBytes;
        const uint32_t vaddr = kaddr + kKVBytes;
        const uint32_t tS = tmem + kGroupCols * b;
#pragma unroll
        for (int kk = 0; kk < kDh / 16; ++kk)
          ptx::mma_ss(tS, ptx::smem_desc_sw128(sbase + kQOff + kk * 32, 16, 1024),
                      ptx::smem_desc_sw128(kaddr + kk * 32, 16, 1024), kIdescS, kk > 0);
#pragma unroll
        for (int kk = 0; kk < kDh / 16; ++kk)
          ptx::mma_ss(tS + kBN, ptx::smem_desc_sw128(sbase + kDOOff + kk * 32, 16, 1024),
                      ptx::smem_desc_sw128(vaddr + kk * 32, 16, 1024), kIdescS, kk > 0);
        ptx::tc_commit(s_full(b));
      };
      auto issue_dq = [&](int j, int b) {
        const uint32_t kaddr = sbase + kStageOff + (j % kStages) * kStageBytes;
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          ptx::mma_ts(tDQ, tmem + kGroupCols * b + 2 * kBN + kk * 8,
                      ptx::smem_desc_sw128(kaddr + kk * 2048, 8192, 1024), kIdescDQ, (j > 0 || kk > 0) ? 1u : 0u);
        ptx::tc_commit(p_free(b));
        ptx::tc_commit(empty(j % kStages));
        if (j == T - 1) ptx::tc_commit(o_final);
      };
      bool ok = true;
      if (warp == kMmaWarp) {
        ok = wait(qfull, 0);
        // The first pass's tiles, then all.
#pragma unroll 1
        for (int u = 0; ok && u < first + T; ++u) {
          const int j = u < first ? u : u - first;
          ok = wait(full(j % kStages), (j / kStages) & 1) && (u < 2 || wait(s_free(u & 1), ((u >> 1) - 1) & 1));
          if (!ok) break;
          ptx::tc_fence_after();
          issue_sdp(j, u & 1);
        }
      } else {
#pragma unroll 1
        for (int j = 0; ok && j < T; ++j) {
          const int b = (first + j) & 1;
          if (!(ok = wait(p_full(b), (j >> 1) & 1))) break;
          ptx::tc_fence_after();
          issue_dq(j, b);
        }
      }
    }
    __syncwarp();
  } else {
    // ---------------- softmax warps: thread = row (lane of tensor memory) of every other step ----------------
    const int lane_base = (warp & 3) * 32, group = warp >> 2;
    const uint32_t trow = tmem + ((uint32_t)lane_base << 16);
    const int row = lane_base + lane;
    const int r = r0 + (row >> w.gshift);
    const bool valid = r <= r1;
    const int h = (g << w.gshift) + (row & (w.G - 1));
    const size_t orow = (size_t)(s.q0 + (valid ? r : r0)) * w.Hq + h;
    const int p = valid ? position(s, r) : -1;
    const int low = window_low(w, p), low_last = window_low(w, p1);
    if (group == 0) redo[row] = 0;
    // Rows past the sequence see nothing, whatever their lse2 and D are.
    const float lse = valid && p >= 0 ? w.lse[orow] : 0.f, lse2 = lse * kLog2e;
    const float2 c2 = make_float2(w.scale_log2, w.scale_log2), nl2 = make_float2(-lse2, -lse2);
    // This group's share of D.
    float delta = 0.f;
    bool ok = true;
    const uint32_t ts = trow + kGroupCols * group;
#pragma unroll 1
    for (int j = group; j < first; j += 2) {
      if (!(ok = __all_sync(0xffffffffu, wait(s_full(group), (j >> 1) & 1)))) break;
      ptx::tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < kBN; c += 16) {
        uint32_t sv[16], dv[16];
        ptx::tmem_ld16x2_sync(ts + c, ts + kBN + c, sv, dv);
        const uint32_t see = visible_bits(w, p, low, kt.begin(j) + c);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float pr = ptx::ex2(fmaf(__uint_as_float(sv[k]), w.scale_log2, -lse2));
          if ((see >> k) & 1u) delta = fmaf(pr, __uint_as_float(dv[k]), delta);
        }
      }
      warp_arrive(s_free(group));
    }
    if (valid && first == 0) {
      // In float from the bf16 rows.
      const uint4* a = reinterpret_cast<const uint4*>((const __nv_bfloat16*)w.out + orow * kDh) + 4 * group;
      const uint4* d = reinterpret_cast<const uint4*>((const __nv_bfloat16*)w.dout + orow * kDh) + 4 * group;
      float x[8], y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        chunk_to_float(__ldg(a + i), x, __nv_bfloat16());
        chunk_to_float(__ldg(d + i), y, __nv_bfloat16());
#pragma unroll
        for (int e = 0; e < 8; ++e) delta = fmaf(x[e], y[e], delta);
      }
    }
    shares[group * kRowsPerTile + row] = delta;
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftmaxWarps) : "memory");        // the softmax warps
    delta = shares[row] + shares[kRowsPerTile + row];
    if (valid && group == 0) {
      w.delta[orow] = delta;
      const float term = -lse / w.scale;
      write_terms(w, 0, orow, fabsf(term) == INFINITY && fabsf(lse) < INFINITY ? NAN : term);
      write_terms(w, 1, orow, -delta);
    }
    const float2 nd2 = make_float2(-delta, -delta);
#pragma unroll 1
    for (int j = group ^ (first & 1); ok && j < T; j += 2) {
      if (!(ok = __all_sync(0xffffffffu, wait(s_full(group), ((first + j) >> 1) & 1)))) break;
      ptx::tc_fence_after();
      const int c0 = kt.begin(j);
      uint32_t pk[16];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t sv[16], dv[16];
        ptx::tmem_ld16x2_sync(ts + 16 * q, ts + kBN + 16 * q, sv, dv);
        if (q == 1) warp_arrive(s_free(group));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 x = __ffma2_rn(make_float2(__uint_as_float(sv[2 * k]), __uint_as_float(sv[2 * k + 1])), c2, nl2);
          const float2 t = __fadd2_rn(make_float2(__uint_as_float(dv[2 * k]), __uint_as_float(dv[2 * k + 1])), nd2);
          const float2 ds = __fmul2_rn(make_float2(ptx::ex2(x.x), ptx::ex2(x.y)), t);
          pk[8 * q + k] = pack_bf16x2(ds.x, ds.y);
        }
      }
      if (c0 < low_last || c0 + 31 > p0 || r0 + tokens > s.lq) {   // some row sees the chunk in part
        const uint32_t see = visible_bits(w, p, low, c0);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          pk[k] &= kept_pair(see, k);
        }
      }
      // dS of the group's previous step is read by its dQ MMAs until p_free: wait
      // only now, so this step's exponentials overlap them.
      if (j > 1) {
        if (!(ok = __all_sync(0xffffffffu, wait(p_free(group), ((j >> 1) - 1) & 1)))) break;
        ptx::tc_fence_after();
      }
      ptx::tmem_st16(ts + 2 * kBN, pk);
      ptx::tmem_wait_st();
      warp_arrive(p_full(group));
    }
    if (T == 0 || (ok && __all_sync(0xffffffffu, wait(o_final, 0)))) {
      uint32_t o[32];
      if (T > 0) {
        ptx::tc_fence_after();
        ptx::tmem_ld32_sync(trow + kColDQ + 32 * group, o);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
      }
      float sum = 0.f;                                 // not finite where any element is not
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const float x = __uint_as_float(o[e]) * w.scale;
        sum = fmaf(x, 0.f, sum);
        o[e] = __float_as_uint(x);
      }
      if (valid) {
        uint4* dst = reinterpret_cast<uint4*>((__nv_bfloat16*)w.dq + orow * kDh) + 4 * group;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float* x = reinterpret_cast<const float*>(o + 8 * q);
          dst[q] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                              pack_bf16x2(x[6], x[7]));
        }
        if (!(sum == 0.f)) {
          redo[row] = 1;
          again = true;
        }
      }
    }
  }

  ptx::tc_fence_before();
  const bool some_again = __syncthreads_or(again);
  if (ctl->abort) {
    // Every role has finished: the MMAs and loads this CTA started complete
    // before its tensor and shared memory are released.
    if ((warp == kMmaWarp || warp == kMmaWarp2) && lane == 0) {
      const uint32_t d = drain(warp - kMmaWarp);
      ptx::tc_commit(d);
      ptx::mbar_wait_drain(d, 0, ctl->limit_ns);
    }
    if (warp == kTmaWarp && lane == 0) {
      ptx::mbar_wait_drain(qfull, 0, ctl->limit_ns);
      const int issued = ctl->issued;
      for (int j = max(0, issued - kStages); j < issued; ++j)
        if (tail && j == T - 1) ptx::mbar_wait_drain(landed, 0, ctl->limit_ns);
        else ptx::mbar_wait_drain(full(j % kStages), (j / kStages) & 1, ctl->limit_ns);
    }
    ptx::tc_fence_before();
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
  if (ctl->abort) {
    if (threadIdx.x == 0) set_err(w.err, PACK3D_DEVERR_TIMEOUT);
    return;
  }
  if (!some_again) return;
#pragma unroll 1
  for (int row = warp; row < kRowsPerTile; row += kThreads / 32)
    if (redo[row]) dq_again<__nv_bfloat16>(w, s, r0 + (row >> w.gshift), (g << w.gshift) + (row & (w.G - 1)));
}

}  // namespace q_side

// ============================================================================
// Key side
// ============================================================================
namespace k_side {

constexpr int kKeys = 128;                      // keys per CTA (M of the dK / dV accumulators)
constexpr int kSoftmaxWarps = 16;               // two groups of 128 keys x two 32-row chunks
// Two MMA warps: the first issues each step's S and dP, the second its dK / dV
// accumulation, so that S and dP of the next step never queue behind it.
constexpr int kThreads = 32 * (kSoftmaxWarps + 3);
constexpr int kMmaWarp = kSoftmaxWarps, kMmaWarp2 = kSoftmaxWarps + 1, kTmaWarp = kSoftmaxWarps + 2;
constexpr int kStep = 64;                       // query rows of a step
// Tensor memory: each group's S^T and dP^T (lane = key, column = row), dK, dV,
// and each group's P^T and dS^T as packed bf16.
constexpr int kColDK = 256, kColDV = 320, kTmemCols = 512;
__device__ __forceinline__ constexpr int col_s(int b) { return 128 * b; }
__device__ __forceinline__ constexpr int col_dp(int b) { return 128 * b + 64; }
__device__ __forceinline__ constexpr int col_p(int b) { return 384 + 64 * b; }
__device__ __forceinline__ constexpr int col_ds(int b) { return 416 + 64 * b; }
constexpr int kStepBytes = kStep * kDh * 2;     // 8 KiB
constexpr int kKeyTileBytes = kKeys * kDh * 2;  // 16 KiB
// Two planes of 128 rows x 8 elements: (1, 1, 1, 0, ..), then zeros.
constexpr int kPlaneBytes = kKeys * 16, kOnesOff = 0;
constexpr int kStageOff = 2 * kPlaneBytes;
// Q at +0, dout at +kStepBytes, then the rows' terms: planes of -lse / scale and -D.
constexpr int kTermBytes = kStep * 16, kTermsAt = 2 * kStepBytes;
constexpr int kStageBytes = 2 * kStepBytes + 2 * kTermBytes;
constexpr int kStages = 8;
constexpr int kKOff = kStageOff + kStages * kStageBytes, kVOff = kKOff + kKeyTileBytes;
static_assert(kStageOff % 1024 == 0 && kStageBytes % 1024 == 0, "swizzled tiles");
// A term's second eight elements of K: zeros (the other term there, times zeros,
// would carry its NaNs over).
constexpr int kZeroOff = kVOff + kKeyTileBytes;
constexpr int kBarOff = kZeroOff + kTermBytes;
// barriers: full[S], empty[S], kvfull, o_final, s_full[2], s_free[2], p_full[2], p_free[2], drain[2], landed
constexpr int kNumBars = 2 * kStages + 13;
constexpr int kCtlOff = kBarOff + kNumBars * 8;
constexpr int kTileOff = kCtlOff + 32;
constexpr int kRedoOff = kTileOff + 64;         // one byte per key row
constexpr int kSmemBytes = kRedoOff + kKeys + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(kKeys, kStep, false);             // S^T, dP^T: N = 64 rows
constexpr uint32_t kIdescKV = ptx::idesc_bf16_f32(kKeys, kDh, true);               // dK, dV: B MN-major

// A CTA's share of a tile whose steps a cluster splits, over its stages (which
// are idle by then): each key's dK and dV.
struct Share {
  float o[kKeys][2 * kDh + 4];
};
static_assert(sizeof(Share) <= kStages * kStageBytes, "share slot");

// kSplit: the CTAs of a cluster share the tile's steps.
template <bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
window_dkv_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmT, const __grid_constant__ Win w, int key_grid) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.y;
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t bar0 = sbase + kBarOff;
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto empty = [&](int s) { return bar0 + 8 * (kStages + s); };
  const uint32_t kvfull = bar0 + 8 * (2 * kStages);
  const uint32_t o_final = kvfull + 8;
  auto s_full = [&](int b) { return kvfull + 16 + 8 * b; };
  auto s_free = [&](int b) { return kvfull + 32 + 8 * b; };
  auto p_full = [&](int b) { return kvfull + 48 + 8 * b; };
  auto p_free = [&](int b) { return kvfull + 64 + 8 * b; };
  auto drain = [&](int i) { return kvfull + 80 + 8 * i; };
  const uint32_t landed = kvfull + 96;         // for the step that is cleared in part
  volatile ptx::WaitCtl* ctl = reinterpret_cast<volatile ptx::WaitCtl*>(smem + kCtlOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kCtlOff + sizeof(ptx::WaitCtl));
  Tile* tile_slot = reinterpret_cast<Tile*>(smem + kTileOff);
  int* found_slot = reinterpret_cast<int*>(tile_slot + 1);      // 0: none, 1: one, 2: wrong offsets
  volatile uint8_t* redo = smem + kRedoOff;
  auto wait = [&](uint32_t bar, uint32_t parity) { return wait_bounded(bar, parity, ctl); };
  const int tokens = kStep >> w.gshift;
  let_next_begin();
  int rank = 0, size = 1;
  if constexpr (kSplit) {
    rank = cooperative_groups::this_cluster().block_rank();
    size = cooperative_groups::this_cluster().num_blocks();
  }
  const int at = blockIdx.x / size;
  const bool far = at >= key_grid;                      // a CTA of the sinks' far queries
  const int x = far ? at - key_grid : at;

  if (warp == 0) {
    Tile s;
    bool bad;
    const bool found = far ? find_far<kKeys, kRowsPerTile>(w, x, &s, &bad) : find_tile(w, x, kKeys, true, &s, &bad);
    if (lane == 0) {
      *tile_slot = s;
      *found_slot = bad ? 2 : found;
    }
  }
  if (threadIdx.x == 32) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 1);
    }
    ptx::mbar_init(kvfull, 1);
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(s_full(b), 1);
      ptx::mbar_init(s_free(b), kSoftmaxWarps / 2);
      ptx::mbar_init(p_full(b), kSoftmaxWarps / 2);
      ptx::mbar_init(p_free(b), 1);
    }
    ptx::mbar_init(o_final, 1);
    ptx::mbar_init(landed, 1);
    ptx::mbar_init(drain(0), 1);
    ptx::mbar_init(drain(1), 1);
    ctl->abort = 0;
    ctl->issued = 0;
    ctl->limit_ns = w.wait_ns;
    ptx::fence_mbar_init();
  }
  if (threadIdx.x < kKeys) {
    redo[threadIdx.x] = 0;
    const uint32_t at = sbase + kOnesOff + 16 * threadIdx.x;
    ptx::st_shared_v4(at, 0x3f803f80u, 0x3f80u, 0u, 0u);
    ptx::st_shared_v4(at + kPlaneBytes, 0u, 0u, 0u, 0u);
    if (threadIdx.x < kStep) ptx::st_shared_v4(sbase + kZeroOff + 16 * threadIdx.x, 0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
  }
  __syncthreads();
  wait_for_last();                                      // for delta and the rows' terms
  if (*found_slot != 1) {
    if (!far && *found_slot == 0 && w.zero_outside && blockIdx.y == 0 && rank == 0) {
      fill_outside(w, w.cu_k, w.Tk, kKeys, x, key_grid, kThreads / 32, w.dk, w.Hkv * kDh / 2, 0u);
      fill_outside(w, w.cu_k, w.Tk, kKeys, x, key_grid, kThreads / 32, w.dv, w.Hkv * kDh / 2, 0u);
    }
    return;
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Tile s = *tile_slot;
  // Keys j0 .. of the sequence and the query rows ra .. rb that see some of them.
  const int shift = s.lk - s.lq;                        // position minus row
  const int j0 = far ? 0 : s.t * kKeys, j1 = min(s.lk, j0 + kKeys) - 1;
  int ra, rb;
  if (far) {
    ra = far_begin<kKeys>(w, s.lq, s.lk) + s.t * far_rows<kRowsPerTile>(w);
    rb = min(s.lq, ra + far_rows<kRowsPerTile>(w)) - 1;
  } else {
    ra = max(0, j0 - shift);
    rb = s.lq - 1;
    if (w.window > 0) rb = min(rb, j1 + w.window - 1 - shift);
  }
  const int all = rb >= ra ? (rb - ra) / tokens + 1 : 0;
  // This CTA's steps.
  const int first = kSplit ? (int)((long)all * rank / size) : 0;
  const int nsteps = kSplit ? (int)((long)all * (rank + 1) / size) - first : all;
  ra += first * tokens;
  // Rows below `split_rows` of this tile leave float partial sums.
  const bool shared = far || (j0 == 0 && far_pieces<kKeys, kRowsPerTile>(w, s.lq, s.lk) > 0);
  const int split_rows = shared ? min(w.sinks, s.lk) : 0;
  // Rows of the last step up to the sequence's end, where the step reaches behind it.
  const int left = (s.lq - (ra + (nsteps - 1) * tokens)) << w.gshift;
  const bool tail = nsteps > 0 && left < kStep;

  bool again = false;                   // something of this thread's key is not finite
  if (warp == kTmaWarp) {
    if (lane == 0 && nsteps > 0) {
      ptx::tma_prefetch(&tmQ);
      ptx::tma_prefetch(&tmO);
      ptx::tma_prefetch(&tmK);
      ptx::tma_prefetch(&tmV);
      ptx::tma_prefetch(&tmT);
      ptx::mbar_expect_tx(kvfull, 2 * kKeyTileBytes);
      ptx::tma_load_3d(sbase + kKOff, &tmK, 0, g, s.k0 + j0, kvfull);
      ptx::tma_load_3d(sbase + kVOff, &tmV, 0, g, s.k0 + j0, kvfull);
      const int nsteps_load = w.stall ? nsteps - 1 : nsteps;
      int issued = 0;
#pragma unroll 1
      for (int t = 0; t < nsteps_load; ++t) {
        const int st = t % kStages;
        if (t >= kStages && !wait(empty(st), ((t / kStages) - 1) & 1)) break;
        const uint32_t dst = sbase + kStageOff + st * kStageBytes;
        const int tok0 = s.q0 + ra + t * tokens;
        const uint32_t bar = tail && t == nsteps - 1 ? landed : full(st);
        ptx::mbar_expect_tx(bar, kStageBytes);
        ptx::tma_load_4d(dst, &tmQ, 0, 0, g, tok0, bar);
        ptx::tma_load_4d(dst + kStepBytes, &tmO, 0, 0, g, tok0, bar);
        ptx::tma_load_5d(dst + kTermsAt, &tmT, 0, 0, g, tok0, 0, bar);
        issued = t + 1;
      }
      ctl->issued = issued;
    }
    __syncwarp();
    if (tail) {
      const int st = (nsteps - 1) % kStages;
      if (__all_sync(0xffffffffu, wait(landed, 0))) {
        clear_rows(sbase + kStageOff + st * kStageBytes, left, kStep);
        clear_rows(sbase + kStageOff + st * kStageBytes + kStepBytes, left, kStep);
        say_cleared(full(st));
      }
    }
  } else if (warp == kMmaWarp || warp == kMmaWarp2) {
    if (nsteps > 0 && ptx::elect_one()) {
      const uint32_t tDK = tmem + kColDK, tDV = tmem + kColDV;
      auto issue_sdp = [&](int t) {
        const uint32_t qaddr = sbase + kStageOff + (t % kStages) * kStageBytes;
        const uint32_t oaddr = qaddr + kStepBytes, taddr = qaddr + kTermsAt;
        const uint64_t ones = ptx::smem_desc_plain(sbase + kOnesOff, kPlaneBytes, 128);
        auto terms = [&](uint32_t at) { return ptx::smem_desc_plain(at, sbase + kZeroOff - at, 128); };
#pragma unroll
        for (int kk = 0; kk < kDh / 16; ++kk)
          ptx::mma_ss(tmem + col_s(t & 1), ptx::smem_desc_sw128(sbase + kKOff + kk * 32, 16, 1024),
                      ptx::smem_desc_sw128(qaddr + kk * 32, 16, 1024), kIdescS, kk > 0);
        ptx::mma_ss(tmem + col_s(t & 1), ones, terms(taddr), kIdescS, 1u);
#pragma unroll
        for (int kk = 0; kk < kDh / 16; ++kk)
          ptx::mma_ss(tmem + col_dp(t & 1), ptx::smem_desc_sw128(sbase + kVOff + kk * 32, 16, 1024),
                      ptx::smem_desc_sw128(oaddr + kk * 32, 16, 1024), kIdescS, kk > 0);
        ptx::mma_ss(tmem + col_dp(t & 1), ones, terms(taddr + kTermBytes), kIdescS, 1u);
        ptx::tc_commit(s_full(t & 1));
      };
      auto issue_dkv = [&](int t) {
        const uint32_t qaddr = sbase + kStageOff + (t % kStages) * kStageBytes;
        const uint32_t oaddr = qaddr + kStepBytes;
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk)
          ptx::mma_ts(tDK, tmem + col_ds(t & 1) + kk * 8, ptx::smem_desc_sw128(qaddr + kk * 2048, 8192, 1024), kIdescKV,
                      (t > 0 || kk > 0) ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk)
          ptx::mma_ts(tDV, tmem + col_p(t & 1) + kk * 8, ptx::smem_desc_sw128(oaddr + kk * 2048, 8192, 1024), kIdescKV,
                      (t > 0 || kk > 0) ? 1u : 0u);
        ptx::tc_commit(p_free(t & 1));
        ptx::tc_commit(empty(t % kStages));
        if (t == nsteps - 1) ptx::tc_commit(o_final);
      };
      bool ok = true;
      if (warp == kMmaWarp) {
        ok = wait(kvfull, 0);
#pragma unroll 1
        for (int t = 0; ok && t < nsteps; ++t) {
          if (!(ok = wait(full(t % kStages), (t / kStages) & 1))) break;
          if (t > 1 && !(ok = wait(s_free(t & 1), ((t >> 1) - 1) & 1))) break;
          ptx::tc_fence_after();
          issue_sdp(t);
        }
      } else {
#pragma unroll 1
        for (int t = 0; ok && t < nsteps; ++t) {
          if (!(ok = wait(p_full(t & 1), (t >> 1) & 1))) break;
          ptx::tc_fence_after();
          issue_dkv(t);
        }
      }
    }
    __syncwarp();
  } else {
    // ---------------- softmax warps: thread = key of the tile ----------------
    const int group = warp >> 3;                 // of the even or of the odd steps
    const int c = (warp >> 2) & 1;               // 32-row chunk of the step
    const int lane_base = (warp & 3) * 32;
    const int rl = lane_base + lane;             // key inside the tile
    const uint32_t trow = tmem + ((uint32_t)lane_base << 16);
    const float2 c2 = make_float2(w.scale_log2, w.scale_log2);
    // The rows ka .. kb - 1 of the sequence see this thread's key.
    const int j = j0 + rl;
    const int ka = far && j >= w.sinks ? rb + 1 : max(ra, j - shift);
    const int kb = w.window > 0 && j >= w.sinks ? min(rb, j + w.window - 1 - shift) + 1 : rb + 1;
    bool ok = true;
    const uint32_t tsd = trow + col_s(group) + 32 * c, tp = trow + col_p(group) + 16 * c;
    const uint32_t s_full_g = s_full(group), s_free_g = s_free(group);
    const uint32_t p_full_g = p_full(group), p_free_g = p_free(group);
    uint32_t phase = 0;
#pragma unroll 1
    for (int t = group; t < nsteps; t += 2, phase ^= 1) {
      // Bit k: row 32 c + k of the step sees the key.
      const int rs = ra + t * tokens;
      const int x0 = (min(max(ka - rs, 0), tokens) << w.gshift) - 32 * c;
      const int x1 = (min(max(kb - rs, 0), tokens) << w.gshift) - 32 * c;
      const uint32_t from = x0 >= 32 ? 0u : 0xffffffffu << max(x0, 0);
      const uint32_t see = from & (x1 >= 32 ? 0xffffffffu : (1u << max(x1, 0)) - 1u);
      const bool some = __any_sync(0xffffffffu, see != 0u), whole = __all_sync(0xffffffffu, see == 0xffffffffu);
      if (!(ok = __all_sync(0xffffffffu, wait(s_full_g, phase)))) break;
      ptx::tc_fence_after();
      uint32_t pd[16], pp[16];
      if (some) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t sv[16], dv[16];
          ptx::tmem_ld16x2_sync(tsd + 16 * q, tsd + 64 + 16 * q, sv, dv);
          if (q == 1) warp_arrive(s_free_g);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 x = __fmul2_rn(make_float2(__uint_as_float(sv[2 * k]), __uint_as_float(sv[2 * k + 1])), c2);
            const float2 pr = make_float2(ptx::ex2(x.x), ptx::ex2(x.y));
            const float2 ds = __fmul2_rn(pr, make_float2(__uint_as_float(dv[2 * k]), __uint_as_float(dv[2 * k + 1])));
            pd[8 * q + k] = pack_bf16x2(ds.x, ds.y);
            pp[8 * q + k] = pack_bf16x2(pr.x, pr.y);
          }
        }
        if (!whole) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint32_t keep = kept_pair(see, k);
            pd[k] &= keep;
            pp[k] &= keep;
          }
        }
      } else {
        warp_arrive(s_free_g);
#pragma unroll
        for (int k = 0; k < 16; ++k) pd[k] = pp[k] = 0u;
      }
      // The previous step's dK / dV MMAs read P^T and dS^T: wait for them only
      // now, so this step's exponentials overlap them.
      if (t > 1) {
        if (!(ok = __all_sync(0xffffffffu, wait(p_free_g, phase ^ 1)))) break;
        ptx::tc_fence_after();
      }
      ptx::tmem_st16(tp + 32, pd);
      ptx::tmem_st16(tp, pp);
      ptx::tmem_wait_st();
      warp_arrive(p_full_g);
    }
    if (nsteps == 0 || (ok && __all_sync(0xffffffffu, wait(o_final, 0)))) {
      // Accumulator lane = key of this tile.  The warpgroups share the 128
      // accumulator columns (dK 64, then dV 64): 32 each.
      const int col0 = 32 * (warp >> 2);
      const bool is_k = col0 < kDh;
      uint32_t o[32];
      if (nsteps > 0) {
        ptx::tc_fence_after();
        ptx::tmem_ld32_sync(trow + kColDK + col0, o);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
      }
      if constexpr (kSplit) {
        Share* mine = reinterpret_cast<Share*>(smem + kStageOff);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<uint4*>(&mine->o[rl][col0 + 4 * q]) = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2],
                                                                              o[4 * q + 3]);
      } else {
        const float f = is_k ? w.scale : 1.f;
        float sum = 0.f;                                 // not finite where any element is not
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float y = __uint_as_float(o[e]) * f;
          sum = fmaf(y, 0.f, sum);
          o[e] = __float_as_uint(y);
        }
        const int slot = far ? x + s.b + 1 : part_slot<kRowsPerTile>(w, s);       // of the sink rows' partial sums
        if (rl < split_rows) {
          float4* dst = reinterpret_cast<float4*>(part_row(w, slot, g, rl) + col0);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            dst[q] = make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]), __uint_as_float(o[4 * q + 2]),
                                 __uint_as_float(o[4 * q + 3]));
        } else if (!far && j0 + rl <= j1) {
          __nv_bfloat16* base = (__nv_bfloat16*)(is_k ? w.dk : w.dv);
          uint4* dst = reinterpret_cast<uint4*>(base + ((size_t)(s.k0 + j0 + rl) * w.Hkv + g) * kDh + (col0 % kDh));
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float* y = reinterpret_cast<const float*>(o + 8 * q);
            dst[q] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                pack_bf16x2(y[6], y[7]));
          }
          if (!(sum == 0.f)) {
            redo[rl] = 1;
            again = true;
          }
        }
      }
    }
  }

  ptx::tc_fence_before();
  const bool some_again = __syncthreads_or(again);
  if (ctl->abort) {
    // Every role has finished: the MMAs of both issuing warps and the
    // producer's loads complete before tensor and shared memory are released.
    if ((warp == kMmaWarp || warp == kMmaWarp2) && lane == 0) {
      const uint32_t d = drain(warp - kMmaWarp);
      ptx::tc_commit(d);
      ptx::mbar_wait_drain(d, 0, ctl->limit_ns);
    }
    if (warp == kTmaWarp && lane == 0) {
      ptx::mbar_wait_drain(kvfull, 0, ctl->limit_ns);
      const int issued = ctl->issued;
      for (int t = max(0, issued - kStages); t < issued; ++t)
        if (tail && t == nsteps - 1) ptx::mbar_wait_drain(landed, 0, ctl->limit_ns);
        else ptx::mbar_wait_drain(full(t % kStages), (t / kStages) & 1, ctl->limit_ns);
    }
    ptx::tc_fence_before();
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
  if constexpr (kSplit) {
    // Every CTA of the cluster comes here, whatever its waits did.  Each joins its
    // part of the keys, a warp a key (lanes 0-15 dK, 16-31 dV), in the steps' order.
    auto cluster = cooperative_groups::this_cluster();
    cluster.sync();
    Share* mine = reinterpret_cast<Share*>(smem + kStageOff);
    const int slot = far ? x + s.b + 1 : part_slot<kRowsPerTile>(w, s);
#pragma unroll 1
    for (int row = kKeys * rank / size + warp; row < kKeys * (rank + 1) / size; row += kThreads / 32) {
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int z = 0; z < size; ++z) {
        const float4 a = *reinterpret_cast<const float4*>(&cluster.map_shared_rank(mine, z)->o[row][4 * lane]);
        y = make_float4(y.x + a.x, y.y + a.y, y.z + a.z, y.w + a.w);
      }
      const float f = lane < 16 ? w.scale : 1.f;
      y = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
      if (row < split_rows) {
        reinterpret_cast<float4*>(part_row(w, slot, g, row))[lane] = y;
      } else if (!far && j0 + row <= j1) {
        __nv_bfloat16* base = (__nv_bfloat16*)(lane < 16 ? w.dk : w.dv);
        reinterpret_cast<uint2*>(base + ((size_t)(s.k0 + j0 + row) * w.Hkv + g) * kDh)[lane & 15] =
            make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
        const float zero = fmaf(y.x, 0.f, fmaf(y.y, 0.f, fmaf(y.z, 0.f, y.w * 0.f)));
        if (__any_sync(0xffffffffu, !(zero == 0.f)) && lane == 0) redo[row] = 1;
      }
    }
    cluster.sync();           // no CTA ends while another reads its share
  }
  if (ctl->abort) {
    if (threadIdx.x == 0) set_err(w.err, PACK3D_DEVERR_TIMEOUT);
    return;
  }
  if (!kSplit && !some_again) return;
#pragma unroll 1
  for (int rl = warp; rl < kKeys; rl += kThreads / 32)
    if (redo[rl]) dkv_row<__nv_bfloat16>(w, s, j0 + rl, g, w.scale >= kLeastScale);
}

}  // namespace k_side

// CTAs of a cluster that share a key tile's steps: a share should be four steps
// long where every CTA has an SM of its own, and 64 where some SMs get a second
// one, which pays where the tiles' lengths differ.  (Both kernels, no window:
// 2,048 tokens, 8 / 2 heads, 1, 4, 8 CTAs 99, 56, 71 us; 4,096, 1, 2, 4 CTAs 195, 137,
// 115; 8,192, 16 / 2 heads, 1, 2 CTAs 747, 524; window 512, 2,048 tokens, 1, 4, 8 CTAs
// 46, 34, 56.)  The host knows the mean length only: 4,096 tokens with 31 sequences of
// one count as short and get 1 CTA, 202 us (143 with 2).
int split_of(const Win& w, long key_ctas) {
  const long mean = (w.Tq + w.B - 1) / w.B, rows = w.window > 0 ? min(mean, (long)w.window + k_side::kKeys) : mean;
  const long steps = (rows * w.G + k_side::kStep - 1) / k_side::kStep, tiles = key_ctas * w.Hkv, sms = sm_count();
  auto good = [&](long S) {
    return (tiles * S <= sms && steps >= 4 * S) || (tiles * S <= 2 * sms && steps >= 64 * S);
  };
  int S = 1;
  while (S < 8 && good(2 * S)) S *= 2;
  return S;
}

// Win::terms viewed as [2][Tq][Hkv][G][8]: boxes of both planes of a step's rows.
inline bool map_terms(CUtensorMap* m, const Win& w) {
  const cuuint64_t dims[5] = {8, (cuuint64_t)w.G, (cuuint64_t)w.Hkv, (cuuint64_t)w.Tq, 2};
  const cuuint64_t strides[4] = {16, (cuuint64_t)w.G * 16, (cuuint64_t)w.Hq * 16, (cuuint64_t)w.Tq * w.Hq * 16};
  const cuuint32_t box[5] = {8, (cuuint32_t)w.G, 1, (cuuint32_t)(k_side::kStep / w.G), 2};
  return tma::encode_bf16(m, w.terms, 5, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

}  // namespace

cudaError_t launch_window_bwd_tc(const Win& w, cudaStream_t st) {
  // First, so that a thread that has made no CUDA call yet (autograd's) has the
  // device's context when the tensor maps are encoded.
  cudaError_t e = cudaFuncSetAttribute(q_side::window_dq_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       q_side::kSmemBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_side::window_dkv_tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             k_side::kSmemBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_side::window_dkv_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             k_side::kSmemBytes);
  if (e != cudaSuccess) return e;
  CUtensorMap tq, to, tk, tv, tk128, tv128, tq64, to64, tt;
  if (!map_query_rows(&tq, w, w.q) || !map_query_rows(&to, w, w.dout) || !map_key_rows(&tk, w, w.k, 32) ||
      !map_key_rows(&tv, w, w.v, 32) || !map_key_rows(&tk128, w, w.k, k_side::kKeys) ||
      !map_key_rows(&tv128, w, w.v, k_side::kKeys) || !map_query_rows(&tq64, w, w.q, k_side::kStep) ||
      !map_query_rows(&to64, w, w.dout, k_side::kStep) || !map_terms(&tt, w))
    return cudaErrorInvalidValue;
  const dim3 gq((unsigned)tile_grid(w.Tq, kRowsPerTile >> w.gshift, w.B), w.Hkv);
  q_side::window_dq_tc_kernel<<<gq, q_side::kThreads, q_side::kSmemBytes, st>>>(tq, to, tk, tv, w);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int key_grid = (int)tile_grid(w.Tk, k_side::kKeys, w.B);
  const long key_ctas = key_grid + far_grid<kRowsPerTile>(w);
  const int S = split_of(w, key_ctas);
  const dim3 gk((unsigned)(key_ctas * S), w.Hkv);
  e = S > 1 ? launch_behind(k_side::window_dkv_tc_kernel<true>, gk, k_side::kThreads, k_side::kSmemBytes, st, S, tq64, to64,
                            tk128, tv128, tt, w, key_grid)
            : launch_behind(k_side::window_dkv_tc_kernel<false>, gk, k_side::kThreads, k_side::kSmemBytes, st, 1, tq64,
                            to64, tk128, tv128, tt, w, key_grid);
  if (e != cudaSuccess) return e;
  return launch_window_sinks<__nv_bfloat16, k_side::kKeys, kRowsPerTile>(w, st);
}

}  // namespace seq
}  // namespace pack3d
