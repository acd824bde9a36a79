// Attention of one new token per sequence over the paged cache.
//
// Every visible key and value row is read once and serves the G query heads of
// its key head; there is no reuse beyond that, so HBM bounds the work and the
// kernels are built to keep enough reads in flight.  Each warp copies (cp.async)
// whole rows into a queue of its own in shared memory, 4 KiB a stage, ahead of
// their use: no warp waits for another, and the reads in flight (16 warps an
// SM) take no registers.
//
// Split and join.  The work is one line of units - (sequence, key head, tile of
// 16 visible slots), sequences of very different lengths behind one another -
// cut into equal runs, one per CTA: every processor reads the same number of
// rows whatever the lengths are.  The eight warps of a CTA take every eighth
// tile, or an eighth of the run each where it holds many short sequences.  A
// warp keeps the online softmax (maximum, sum, weighted values) of the piece of
// a (sequence, key head) it is in.  A piece that is whole is written out; the
// others of a CTA are joined in shared memory, a warp a head, and what is still
// part of a longer one goes to the workspace (two slots a CTA at most: the
// run's first and last), where cache_join_kernel adds the parts in order.
// Short caches, and batches that fill the GPU by themselves, take one CTA per
// (sequence, key head) and no second launch.
//
// bf16: mma.sync m16n8k16 with the heads as rows.  The tile's keys are the B
// operand of S = Q K^T and its values that of O += P V, both as they come from
// memory: a lane's 16-byte chunks are the fragments of a permuted contraction
// index (Q is permuted the same way), and the values' token pairs are formed
// with byte permutes.  The tensor cores matter little here; they keep the issue
// slots free for the loads.  P is rounded to bf16 for the product.
// float: 16 lanes share a row, two rows at a time, on CUDA cores.
//
// Measured: 48 sequences of 1 to 32,768 slots, 8 / 2 heads, bf16, 371 MB: 80 us,
// 4.6 TB/s, and 3 us more for the join, which begins behind it.  On a like batch of
// 407 MB (89 us) the arithmetic is 5 us of it and the look-up of the pages 8: what
// bounds it is reading rows of 128 bytes and the two turns' starts (between two
// sizes the rate is 5.4 TB/s, 7.1 in float).  One sequence of 311 slots: 7 us.
#include "seq.cuh"
#include "tc_ptx.cuh"

namespace pack3d {
namespace seq {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kSlots = 16;                 // visible slots of a unit

// Softmax state of one piece: for each head the maximum (log2 units), the sum
// and the weighted values.
template <int G>
struct alignas(16) Piece {
  float o[G][kDh];
  float m[G], l[G];
};

struct DecodeArgs {
  Cache c;
  const void* q;
  void* out;
  float* lse;        // nullable
  float* row_lse2;   // with weights: log2 of each row's denominator
  float* logits;     // with weights: scaled log2 scores [B * Hq][cap], by visible slot
  void* part;        // Piece [CTAs][2]
  int2* joins;       // [B * Hkv]: first CTA and number of CTAs that have a part
  int split;         // 0: one CTA per (sequence, key head)
};

// The visible slots of a sequence: first the sinks [0, s0), then [lo, n).
struct Seen {
  int lo, s0, count;
  __device__ __forceinline__ int slot(int i) const { return i < s0 ? i : i - s0 + lo; }
};
__device__ __forceinline__ Seen seen(const Cache& c, int n) {
  Seen v;
  v.lo = c.window > 0 && n > c.window ? n - c.window : 0;
  v.s0 = min(c.sinks, v.lo);
  v.count = v.s0 + n - v.lo;
  return v;
}

__device__ __forceinline__ int units_of(const Cache& c, int b) {
  return (seen(c, cached(c, b)).count + kSlots - 1) / kSlots;
}

// Where a unit lies: tile t of a (sequence, key head) with so many tiles.
struct Unit {
  int b, g, t, tiles;
};
// The tiles [t0, t1) of a (sequence, key head) that a piece covers; b < 0: none.
struct Span {
  int b, g, t0, t1;
};

// All sequences' units, and where unit number first(total) lies: found by the
// whole CTA, kThreads sequences at a time.  A split call has fewer than 2^31
// units (is_split).
struct Scan {
  int warp_sum[kWarps];
  Unit at;
  int start;        // first unit of at's (sequence, key head)
};
template <typename First>
__device__ __forceinline__ int find_unit(const Cache& c, Scan* sc, First first) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int total = 0, tiles = 0, own = 0, before = 0;
  // With more sequences than threads the sum comes first and the place in a
  // second pass.
  for (int pass = c.B > kThreads ? 0 : 1; pass < 2; ++pass) {
    int base = 0, u = pass ? (c.B > kThreads ? first(total) : 0) : -1;
#pragma unroll 1
    for (int b0 = 0; b0 < c.B; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      tiles = b < c.B ? units_of(c, b) : 0;
      own = tiles * c.Hkv;
      int incl = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += up;
      }
      __syncthreads();
      if (lane == 31) sc->warp_sum[warp] = incl;
      __syncthreads();
      before = base + incl - own;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const int n = sc->warp_sum[i];
        if (i < warp) before += n;
        base += n;
      }
      if (c.B <= kThreads) u = first(base);
      if (u >= before && u < before + own) {
        Unit at;
        at.b = b;
        at.tiles = tiles;
        at.g = (u - before) / tiles;
        at.t = (u - before) - at.g * tiles;
        sc->at = at;
      }
    }
    total = base;
  }
  __syncthreads();
  return total;
}

// Units of one CTA's run: at least four a warp.
__device__ __forceinline__ int run_units(int total, int ctas) {
  return max((int)(((unsigned)total + ctas - 1) / ctas), 4 * kWarps);
}

// d += A B for the rows 0-7 of A (8-15 are zero, and so is what they give).
__device__ __forceinline__ void mma_16816(float* d, uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  float z0, z1;
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, {%9,%10,%11,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(z0), "=f"(z1)
      : "r"(a0), "r"(0u), "r"(a2), "r"(b0), "r"(b1), "f"(d[0]), "f"(d[1]), "f"(0.f));
  (void)z0;
  (void)z1;
}

// Pages and pool rows of a tile's 16 slots, lane i < 16 for slot i; -1 where
// there is none (past the end, or a page outside the pool: reported and left
// out).  The page is read a turn before the row is formed, so that no branch
// waits for it.
__device__ __forceinline__ int tile_pages(const Cache& c, const int32_t* table, const Seen& v, int t) {
  const int i = t * kSlots + (threadIdx.x & 15);
  return i < v.count ? __ldg(table + (v.slot(i) >> c.page_shift)) : 0;
}
__device__ __forceinline__ int tile_rows(const Cache& c, const Seen& v, int t, int page) {
  const int i = t * kSlots + (threadIdx.x & 15);
  if (i >= v.count) return -1;
  if ((unsigned)page >= (unsigned)c.num_pages) {
    set_err(c.err, PACK3D_DEVERR_PAGE);
    return -1;
  }
  return (page << c.page_shift) + (v.slot(i) & (c.page - 1));
}

// A stage of a warp's queue: 4 KiB, the keys in its first half.
constexpr int kStageBytes = 4096, kDepth = 3;

template <typename T, int G> struct Worker;

// ---- bf16: a stage is a unit -------------------------------------------------------
// Lane (r, x) = (lane / 4, lane % 4): head row r; of the keys, token r (and
// 8 + r) and the 16-byte chunks x and x + 4; of the values, the tokens 2x, 2x+1,
// 8+2x, 8+2x+1 and the chunk r.
template <int G> struct Worker<__nv_bfloat16, G> {
  static constexpr int kStages = 1;      // per unit
  uint32_t q[8];
  float o[8][2];
  float m, l;

  __device__ __forceinline__ void begin(const DecodeArgs& a, int b, int g) {
    const int r = (threadIdx.x & 31) >> 2, x = threadIdx.x & 3;
    uint4 c0 = make_uint4(0, 0, 0, 0), c1 = c0;
    if (r < G) {
      const uint4* p = reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.q + ((size_t)b * a.c.Hq + g * G + r) * kDh);
      c0 = __ldg(p + x);
      c1 = __ldg(p + x + 4);
    }
    q[0] = c0.x; q[1] = c0.y; q[2] = c0.z; q[3] = c0.w;
    q[4] = c1.x; q[5] = c1.y; q[6] = c1.z; q[7] = c1.w;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = 0.f;
    m = -INFINITY;
    l = 0.f;
  }
  // Copies of one unit whose pool rows are `rows`; a row that is not there gives zeros.
  __device__ __forceinline__ static void issue(const DecodeArgs& a, int g, int rows, int, uint32_t stage) {
    const int lane = threadIdx.x & 31, r = lane >> 2, x = lane & 3;
    const long step = (long)a.c.Hkv * 8;      // 16-byte chunks a pool row
    const uint4* k = reinterpret_cast<const uint4*>(a.c.k_pages) + g * 8;
    const uint4* v = reinterpret_cast<const uint4*>(a.c.v_pages) + g * 8;
    // Keys: four rows an instruction, chunk c of row i at 128 i + 16 (c ^ 4 (i & 1)).
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = 4 * i + (lane >> 3), row = __shfl_sync(0xffffffffu, rows, at);
      ptx::cp_async16(stage + 128 * at + 16 * ((lane & 7) ^ ((at & 1) << 2)), k + max(row, 0) * step + (lane & 7),
                      row >= 0 ? 16 : 0);
    }
    // Values: the lane's own chunks, chunk i of lane l at 2048 + 512 i + 16 l.
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = __shfl_sync(0xffffffffu, rows, (i >> 1) * 8 + 2 * x + (i & 1));
      ptx::cp_async16(stage + 2048 + 512 * i + 16 * lane, v + max(row, 0) * step + r, row >= 0 ? 16 : 0);
    }
  }
  __device__ __forceinline__ void compute(const DecodeArgs& a, int count, uint32_t stage, int t, int, float* logits) {
    const int lane = threadIdx.x & 31, r = lane >> 2, x = lane & 3;
    float s[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[h][0] = s[h][1] = 0.f;
      const uint32_t at = stage + 128 * (8 * h + r), flip = (r & 1) << 2;
      const uint4 a0 = ptx::ld_shared_v4(at + 16 * (x ^ flip)), a1 = ptx::ld_shared_v4(at + 16 * ((x + 4) ^ flip));
      mma_16816(s[h], q[0], q[1], a0.x, a0.y);
      mma_16816(s[h], q[2], q[3], a0.z, a0.w);
      mma_16816(s[h], q[4], q[5], a1.x, a1.y);
      mma_16816(s[h], q[6], q[7], a1.z, a1.w);
    }
    float y[4] = {s[0][0] * a.c.scale_log2, s[0][1] * a.c.scale_log2, s[1][0] * a.c.scale_log2,
                  s[1][1] * a.c.scale_log2};
    if (count < kSlots) {       // slots past the end
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((i >> 1) * 8 + 2 * x + (i & 1) >= count) y[i] = -INFINITY;
    }
    if (logits && r < G) {
      float* p = logits + (size_t)r * a.c.cap + t * kSlots + 2 * x;   // cap is a multiple of 16
      *reinterpret_cast<float2*>(p) = make_float2(y[0], y[1]);
      *reinterpret_cast<float2*>(p + 8) = make_float2(y[2], y[3]);
    }
    float mx = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    if (__any_sync(0xffffffffu, mx > m)) {
      const float top = fmaxf(m, mx);
      const float f = top == -INFINITY ? 1.f : ptx::ex2(m - top);
      m = top;
      l *= f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i][0] *= f;
        o[i][1] *= f;
      }
    }
    const float sub = m == -INFINITY ? 0.f : m;
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = ptx::ex2(y[i] - sub);
    l += (p[0] + p[1]) + (p[2] + p[3]);
    const uint32_t p0 = pack_bf16x2(p[0], p[1]), p1 = pack_bf16x2(p[2], p[3]);
    uint32_t v[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 y4 = ptx::ld_shared_v4(stage + 2048 + 512 * i + 16 * lane);
      v[4 * i] = y4.x; v[4 * i + 1] = y4.y; v[4 * i + 2] = y4.z; v[4 * i + 3] = y4.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t pick = (i & 1) ? 0x7632u : 0x5410u;   // high or low halves: one dim of a token pair
      mma_16816(o[i], p0, p1, __byte_perm(v[i >> 1], v[4 + (i >> 1)], pick),
                __byte_perm(v[8 + (i >> 1)], v[12 + (i >> 1)], pick));
    }
  }
  // The lane's row total; o[i][e] of row r is dim 16 x + 8 e + i.
  __device__ __forceinline__ void finish() {
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
  }
  __device__ __forceinline__ void store(Piece<G>* p) const {
    const int r = (threadIdx.x & 31) >> 2, x = threadIdx.x & 3;
    if (r >= G) return;
    if (x == 0) {
      p->m[r] = m;
      p->l[r] = l;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        *reinterpret_cast<float4*>(&p->o[r][16 * x + 8 * e + i]) =
            make_float4(o[i][e], o[i + 1][e], o[i + 2][e], o[i + 3][e]);
  }
};

// ---- float: a stage is half a unit ---------------------------------------------------
// Lane (u, x) = (lane / 16, lane % 16): of every pair of slots, slot u, and the
// dims 4x .. 4x+3.  The two halves of a warp keep separate softmax states,
// joined at the end of a piece.
template <int G> struct Worker<float, G> {
  static constexpr int kStages = 2;
  float4 q[G], o[G];
  float m[G], l[G];

  __device__ __forceinline__ void begin(const DecodeArgs& a, int b, int g) {
    const int x = threadIdx.x & 15;
    const float4* p = reinterpret_cast<const float4*>((const float*)a.q + ((size_t)b * a.c.Hq + g * G) * kDh);
#pragma unroll
    for (int h = 0; h < G; ++h) {
      q[h] = __ldg(p + h * 16 + x);
      o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
      m[h] = -INFINITY;
      l[h] = 0.f;
    }
  }
  __device__ __forceinline__ static void issue(const DecodeArgs& a, int g, int rows, int half, uint32_t stage) {
    const int u = (threadIdx.x >> 4) & 1, x = threadIdx.x & 15;
    stage += 16 * (threadIdx.x & 31);         // chunk i of lane l at 512 i + 16 l
    const long step = (long)a.c.Hkv * 16;
    const float4* k = reinterpret_cast<const float4*>(a.c.k_pages) + g * 16 + x;
    const float4* v = reinterpret_cast<const float4*>(a.c.v_pages) + g * 16 + x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = __shfl_sync(0xffffffffu, rows, 8 * half + 2 * i + u);
      ptx::cp_async16(stage + 512 * i, k + max(row, 0) * step, row >= 0 ? 16 : 0);
      ptx::cp_async16(stage + 2048 + 512 * i, v + max(row, 0) * step, row >= 0 ? 16 : 0);
    }
  }
  __device__ __forceinline__ static float4 chunk(uint32_t at) {
    const uint4 u = ptx::ld_shared_v4(at);
    return make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
  }
  __device__ __forceinline__ void compute(const DecodeArgs& a, int count, uint32_t stage, int t, int half,
                                          float* logits) {
    const int u = (threadIdx.x >> 4) & 1, x = threadIdx.x & 15;
    stage += 16 * (threadIdx.x & 31);
    float y[G][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 k = chunk(stage + 512 * i);
      const int slot = 8 * half + 2 * i + u;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        float s = fmaf(q[h].x, k.x, fmaf(q[h].y, k.y, fmaf(q[h].z, k.z, q[h].w * k.w)));
#pragma unroll
        for (int e = 8; e > 0; e >>= 1) s += __shfl_xor_sync(0xffffffffu, s, e);
        y[h][i] = slot < count ? s * a.c.scale_log2 : -INFINITY;
        if (logits && x == 0) logits[(size_t)h * a.c.cap + t * kSlots + slot] = y[h][i];
      }
    }
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const float top = fmaxf(fmaxf(fmaxf(y[h][0], y[h][1]), fmaxf(y[h][2], y[h][3])), m[h]);
      const float f = m[h] == top ? 1.f : ptx::ex2(m[h] - top);
      const float sub = top == -INFINITY ? 0.f : top;
      m[h] = top;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[h][i] = ptx::ex2(y[h][i] - sub);
      l[h] = fmaf(l[h], f, (y[h][0] + y[h][1]) + (y[h][2] + y[h][3]));
      o[h].x *= f;
      o[h].y *= f;
      o[h].z *= f;
      o[h].w *= f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = chunk(stage + 2048 + 512 * i);
#pragma unroll
      for (int h = 0; h < G; ++h) {
        o[h].x = fmaf(y[h][i], v.x, o[h].x);
        o[h].y = fmaf(y[h][i], v.y, o[h].y);
        o[h].z = fmaf(y[h][i], v.z, o[h].z);
        o[h].w = fmaf(y[h][i], v.w, o[h].w);
      }
    }
  }
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const float mo = __shfl_xor_sync(0xffffffffu, m[h], 16);
      const float top = fmaxf(m[h], mo);
      const float f = m[h] == top ? 1.f : ptx::ex2(m[h] - top);     // also for two empty halves
      float* acc[5] = {&l[h], &o[h].x, &o[h].y, &o[h].z, &o[h].w};
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        const float mine = *acc[i] * f;
        *acc[i] = mine + __shfl_xor_sync(0xffffffffu, mine, 16);
      }
      m[h] = top;
    }
  }
  __device__ __forceinline__ void store(Piece<G>* p) const {
    const int lane = threadIdx.x & 31;
    if (lane >= 16) return;
#pragma unroll
    for (int h = 0; h < G; ++h) {
      if (lane == 0) {
        p->m[h] = m[h];
        p->l[h] = l[h];
      }
      *reinterpret_cast<float4*>(&p->o[h][4 * lane]) = o[h];
    }
  }
};

// Tiles t0, t0 + step, .. below t1 of one (sequence, key head) through the warp's
// queue: copies kDepth - 1 stages ahead of their use, the pages one tile ahead
// of that.
template <typename T, int G>
__device__ __forceinline__ void run_tiles(Worker<T, G>& k, const DecodeArgs& a, int b, int g, const Seen& v, int t0,
                                          int t1, int step, float* logits, uint32_t queue) {
  constexpr int S = Worker<T, G>::kStages;
  const int32_t* table = a.c.table + (size_t)b * a.c.max_pages;
  const int end = (t1 - t0 + step - 1) / step * S;      // stages
  int rows = tile_rows(a.c, v, t0, tile_pages(a.c, table, v, t0));
  int next = tile_pages(a.c, table, v, t0 + step);
  int in = 0, in_t = t0, t = t0, in_slot = 0, out_slot = 0;   // the next stage to copy; its tile, the tile in use; ring slots
#pragma unroll 1
  for (int s = 1 - kDepth; s < end; ++s) {
    if (s >= 0) {
      ptx::cp_async_wait_one();                    // all but the newest group: stage s is here,
      __syncwarp();                                // every lane's part of it
      k.compute(a, v.count - t * kSlots, queue + out_slot * kStageBytes, t, s % S, logits);
      out_slot = out_slot + 1 == kDepth ? 0 : out_slot + 1;
      if ((s + 1) % S == 0) t += step;
    }
    if (in < end) {
      __syncwarp();                                // the slot's last stage has been read by every lane
      Worker<T, G>::issue(a, g, rows, in % S, queue + in_slot * kStageBytes);
      in_slot = in_slot + 1 == kDepth ? 0 : in_slot + 1;
      if (++in % S == 0) {
        in_t += step;
        rows = tile_rows(a.c, v, in_t, next);
        next = tile_pages(a.c, table, v, in_t + step);
      }
    }
    ptx::cp_async_commit();                        // a group a turn, empty or not
  }
}

// Final values of head h: lane holds the dims 2 lane, 2 lane + 1 of the sum o.
template <typename T>
__device__ __forceinline__ void write_row(const DecodeArgs& a, int b, int h, float m, float l, float2 o) {
  const size_t at = (size_t)b * a.c.Hq + h;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  store2((T*)a.out + at * kDh, make_float2(o.x * inv, o.y * inv));
  if ((threadIdx.x & 31) == 0) {
    const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
    if (a.lse) a.lse[at] = lse2 * 0.69314718f;
    if (a.row_lse2) a.row_lse2[at] = lse2;
  }
}

// A CTA's shared memory: per warp its queue and two pieces, the run's first and
// last (the ones that may not be whole).  The second piece lies over the queue,
// which is empty when it is written.
template <int G>
struct CtaSmem {
  alignas(128) uint8_t queue[kWarps][kDepth * kStageBytes];
  Piece<G> first[kWarps];
  Span spans[2 * kWarps];
  Scan scan;
  __device__ __forceinline__ Piece<G>* piece(int i) {
    return i & 1 ? reinterpret_cast<Piece<G>*>(queue[i >> 1]) : &first[i >> 1];
  }
};

// Joins head h of the pieces in `mask` (bit i: piece i), all of one (sequence,
// key head), in order: into `to`, or where to is null into the results.  One
// warp; lane i < 16 holds piece i's maximum and sum.
template <typename T, int G>
__device__ __forceinline__ void join_head(const DecodeArgs& a, CtaSmem<G>* sm, int b, int g, int h, uint32_t mask,
                                          Piece<G>* to) {
  const int lane = threadIdx.x & 31;
  const bool in = (mask >> lane) & 1u;
  const float m = in ? sm->piece(lane)->m[h] : -INFINITY;
  float top = m;
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  top = __shfl_sync(0xffffffffu, top, 0);
  const float f = m == top ? 1.f : ptx::ex2(m - top);
  float l = in ? sm->piece(lane)->l[h] * f : 0.f;
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  l = __shfl_sync(0xffffffffu, l, 0);
  float2 o = make_float2(0.f, 0.f);
#pragma unroll 4
  for (uint32_t left = mask; left; left &= left - 1) {
    const int i = __ffs(left) - 1;
    const float fi = __shfl_sync(0xffffffffu, f, i);
    const float2 x = *reinterpret_cast<const float2*>(&sm->piece(i)->o[h][2 * lane]);
    o.x = fmaf(x.x, fi, o.x);
    o.y = fmaf(x.y, fi, o.y);
  }
  if (to) {
    if (lane == 0) {
      to->m[h] = top;
      to->l[h] = l;
    }
    *reinterpret_cast<float2*>(&to->o[h][2 * lane]) = o;
  } else {
    write_row<T>(a, b, g * G + h, top, l, o);
  }
}

template <typename T, int G>
__global__ void __launch_bounds__(kThreads, 2) cache_attn_kernel(const DecodeArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  CtaSmem<G>* sm = reinterpret_cast<CtaSmem<G>*>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Cache& c = a.c;
  let_next_begin();
  if (threadIdx.x < 2 * kWarps) sm->spans[threadIdx.x].b = -1;
  // This CTA's run of units: where it begins, and how many.
  Unit at;
  int first = 0, count, per = 1;
  if (a.split) {
    const int total = find_unit(c, &sm->scan, [&](int total) {
      per = run_units(total, gridDim.x);
      return (int)min((unsigned)total, blockIdx.x * (unsigned)per);
    });
    first = (int)min((unsigned)total, blockIdx.x * (unsigned)per);
    count = min(total - first, per);
    if (count == 0) return;
    at = sm->scan.at;
  } else {
    at.b = blockIdx.x / c.Hkv;
    at.g = blockIdx.x % c.Hkv;
    at.t = 0;
    count = at.tiles = units_of(c, at.b);
    if (count == 0) {        // nothing cached: zeros, for every head of the group
      if (warp < G) write_row<T>(a, at.b, at.g * G + warp, -INFINITY, 0.f, make_float2(0.f, 0.f));
      return;
    }
  }
  __syncthreads();
  const uint32_t queue = ptx::smem_u32(sm->queue[warp]);
  int used = 0;              // pieces this warp left in shared memory
  Worker<T, G> k;
  // One piece: the tiles t0, t0 + step, .. of [t0, t1) of at's (sequence, key
  // head), left in the warp's next slot as a part of its tiles [p0, p1).
  auto piece = [&](int t0, int t1, int step, int p0, int p1) {
    float* logits = a.logits ? a.logits + ((size_t)at.b * c.Hq + at.g * G) * c.cap : nullptr;
    k.begin(a, at.b, at.g);
    run_tiles(k, a, at.b, at.g, seen(c, cached(c, at.b)), t0, t1, step, logits, queue);
    k.finish();
    __syncwarp();            // the queue's last stage has been read by every lane
    k.store(sm->piece(2 * warp + used));
    if (lane == 0) sm->spans[2 * warp + used] = Span{at.b, at.g, p0, p1};
    __syncwarp();
  };
  // To the next (sequence, key head) with units.
  auto advance = [&]() {
    at.t = 0;
    if (++at.g == c.Hkv) {
      at.g = 0;
      do at.tiles = units_of(c, ++at.b);
      while (at.tiles == 0 && at.b + 1 < c.B);
    }
  };
  const int part0 = min(at.tiles - at.t, count);
  bool few = part0 == count;      // at most two (sequence, key head)s in the run
  if (!few) {
    const Unit was = at;
    advance();
    few = at.tiles >= count - part0;
    at = was;
  }
  int u = few ? 0 : (int)((unsigned)count * warp / kWarps);
  const int end = few ? count : (int)((unsigned)count * (warp + 1) / kWarps);
  // Few: the warps take every eighth tile of each, so that the CTA reads one
  // stretch of the cache at a time.  Many short ones: a stretch of the run each.
  if (!few)
    for (int skip = u; skip > 0;) {
      const int n = min(skip, at.tiles - at.t);
      at.t += n;
      skip -= n;
      if (at.t == at.tiles) advance();
    }
#pragma unroll 1
  while (u < end) {
    const int t0 = at.t, t1 = min(at.tiles, t0 + (end - u));
    if (a.split && t0 == 0 && lane == 0 && (!few || warp == 0)) {
      // The beginning of a (sequence, key head): which CTAs have parts of it.
      const int start = first + u, c0 = start / per;
      a.joins[at.b * c.Hkv + at.g] = make_int2(c0, (start + at.tiles - 1) / per - c0 + 1);
    }
    if (few) {
      if (t0 + warp < t1) piece(t0 + warp, t1, kWarps, t0, t1);
      ++used;
    } else {
      piece(t0, t1, 1, t0, t1);
      if (t0 == 0 && t1 == at.tiles) {       // whole: the slot is free again
#pragma unroll 1
        for (int h = 0; h < G; ++h) join_head<T, G>(a, sm, at.b, at.g, h, 1u << (2 * warp + used), nullptr);
        __syncwarp();
        if (lane == 0) sm->spans[2 * warp + used].b = -1;
      } else {
        ++used;
      }
    }
    u += t1 - t0;
    if (u < end) advance();
  }
  __syncthreads();
  // Pieces of one (sequence, key head) lie behind one another.  Every warp looks
  // at the groups (lane i < 16: piece i) and joins every eighth head of each.
  // What is still not whole goes to the workspace: slot 1 of the CTA if it
  // begins its (sequence, key head), slot 0 if it continues one.
  const Span me = lane < 2 * kWarps ? sm->spans[lane] : Span{-1, 0, 0, 0};
  const int key = me.b < 0 ? -1 - lane : me.b * c.Hkv + me.g;
  const uint32_t mask = __match_any_sync(0xffffffffu, key);
  uint32_t groups = __ballot_sync(0xffffffffu, me.b >= 0 && __ffs(mask) - 1 == lane);
  for (int n = 0; groups; groups &= groups - 1, n += G) {
    const int i = __ffs(groups) - 1;
    const uint32_t of = __shfl_sync(0xffffffffu, mask, i);
    const int b = __shfl_sync(0xffffffffu, me.b, i), g = __shfl_sync(0xffffffffu, me.g, i);
    const int t0 = __shfl_sync(0xffffffffu, me.t0, i), t1 = __shfl_sync(0xffffffffu, me.t1, 31 - __clz(of));
    const bool whole = t0 == 0 && t1 == units_of(c, b);
    Piece<G>* to = whole ? nullptr : (Piece<G>*)a.part + 2 * (size_t)blockIdx.x + (t0 == 0 ? 1 : 0);
#pragma unroll 1
    for (int h = (warp - n) & (kWarps - 1); h < G; h += kWarps) join_head<T, G>(a, sm, b, g, h, of, to);
  }
}

// Joins the CTAs' parts of one (sequence, head) in the order of the cache: 16
// groups of 16 threads each add every 16th part, a thread four dims.
template <typename T, int G>
__global__ void __launch_bounds__(256) cache_join_kernel(const DecodeArgs a) {
  __shared__ float s_top[8];
  __shared__ float4 s_o[16][16];
  __shared__ float s_l[16];
  const Cache& c = a.c;
  const int b = blockIdx.x / c.Hq, hq = blockIdx.x % c.Hq, g = hq / G, h = hq % G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  let_next_begin();
  wait_for_last();
  const int2 from = a.joins[b * c.Hkv + g];
  if (units_of(c, b) == 0) {          // nothing cached: no CTA had it
    if (warp == 0) write_row<T>(a, b, hq, -INFINITY, 0.f, make_float2(0.f, 0.f));
    return;
  }
  const int c0 = from.x, n = from.y;
  if (n == 1) return;       // one CTA had all of it and wrote the results
  const Piece<G>* part = (const Piece<G>*)a.part + 2 * (size_t)c0;
  auto piece = [&](int i) { return part + 2 * i + (i == 0 ? 1 : 0); };
  float top = -INFINITY;
  for (int i = threadIdx.x; i < n; i += 256) top = fmaxf(top, piece(i)->m[h]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, s_top[i]);
  const int part_of = threadIdx.x >> 4, x = threadIdx.x & 15;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 4
  for (int i = part_of; i < n; i += 16) {
    const Piece<G>* p = piece(i);
    const float f = p->m[h] == top ? 1.f : ptx::ex2(p->m[h] - top);
    const float4 y = *reinterpret_cast<const float4*>(&p->o[h][4 * x]);
    l = fmaf(p->l[h], f, l);
    o.x = fmaf(y.x, f, o.x);
    o.y = fmaf(y.y, f, o.y);
    o.z = fmaf(y.z, f, o.z);
    o.w = fmaf(y.w, f, o.w);
  }
  s_o[part_of][x] = o;
  if (x == 0) s_l[part_of] = l;
  __syncthreads();
  if (warp > 0) return;
  float2 sum = make_float2(0.f, 0.f);
  l = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 y = reinterpret_cast<const float2*>(s_o[i])[lane];
    sum.x += y.x;
    sum.y += y.y;
    l += s_l[i];
  }
  write_row<T>(a, b, hq, top, l, sum);
}

// The token's weight of every slot: softmax weights from the kept scores and
// the rows' denominators, summed over the heads.
__global__ void __launch_bounds__(256) cache_weights_kernel(const Cache c, const float* logits, const float* row_lse2,
                                                            float* weights, int accumulate) {
  const int b = blockIdx.y;
  const int n = cached(c, b);
  const Seen v = seen(c, n);
  wait_for_last();
  for (int j = blockIdx.x * 256 + threadIdx.x; j < n; j += gridDim.x * 256) {
    const int i = j < v.s0 ? j : (j >= v.lo ? j - v.lo + v.s0 : -1);
    float total = 0.f;
    if (i >= 0)
      for (int h = 0; h < c.Hq; ++h) {
        const size_t at = (size_t)b * c.Hq + h;
        // A head whose scores are all -infinity has no weight to give, as its output is 0.
        const float lse2 = row_lse2[at];
        if (lse2 != -INFINITY) total += ptx::ex2(logits[at * c.cap + i] - lse2);
      }
    float* dst = weights + (size_t)b * c.cap + j;
    *dst = accumulate ? *dst + total : total;
  }
}

// ---- host side ------------------------------------------------------------------

// One CTA per (sequence, key head) where a cache of at most 64 units (eight a
// warp) leaves nothing to split for, or a batch of at least 4,096 such pairs fills
// the GPU if its lengths are alike.  (One sequence of 32,768 slots, the others of 10,
// 8 key heads: 511 sequences, split, 40 us; 512, not split, 198.)  Also where the
// units would not fit 31 bits.
bool is_split(int B, int Hkv, int cap) {
  return cap > 64 * kSlots && (long)B * Hkv < 4096 && (long)B * Hkv * (cap / kSlots) < (1L << 31) - 4096;
}

// CTAs of a split call: two turns of two an SM (the SMs do not all get the same
// share of the memory's bandwidth, so the second turn goes where there is time:
// 407 MB in 93.5 us with one turn, 92.0 with two, 94.4 with three), fewer where
// the capacity has fewer runs.  The workspace has room for the most there can be
// on any GPU.
constexpr int kMaxCtas = 1024;
int split_ctas(int B, int Hkv, int cap) {
  const long runs = ((long)B * Hkv * (cap / kSlots) + 4 * kWarps - 1) / (4 * kWarps);
  return (int)min((long)min(4 * sm_count(), kMaxCtas), max(1L, runs));
}

size_t up1k(size_t n) { return (n + 1023) / 1024 * 1024; }
size_t parts_bytes(int G) { return up1k((size_t)2 * kMaxCtas * (((size_t)G * (2 + kDh) * sizeof(float) + 15) / 16 * 16)); }

template <typename T, int G>
cudaError_t launch_g(DecodeArgs& a, cudaStream_t st) {
  const Cache& c = a.c;
  constexpr int kSmem = sizeof(CtaSmem<G>);
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
  cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<T, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int ctas = a.split ? split_ctas(c.B, c.Hkv, c.cap) : c.B * c.Hkv;
  cache_attn_kernel<T, G><<<ctas, kThreads, kSmem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.split) return e;
  return launch_behind(cache_join_kernel<T, G>, c.B * c.Hq, 256, 0, st, 1, a);
}

template <typename T>
cudaError_t launch_t(DecodeArgs& a, cudaStream_t st) {
  switch (a.c.G) {
    case 1: return launch_g<T, 1>(a, st);
    case 2: return launch_g<T, 2>(a, st);
    case 4: return launch_g<T, 4>(a, st);
    default: return launch_g<T, 8>(a, st);
  }
}

}  // namespace

// The split's parts and the table for their join, then with weights the rows' denominators and the scores.
size_t cache_attn_workspace(int B, int Hq, int Hkv, int cap, bool weights) {
  size_t n = 0;
  if (is_split(B, Hkv, cap)) n = parts_bytes(Hq / Hkv) + up1k((size_t)B * Hkv * sizeof(int2));
  if (weights) n += up1k((size_t)B * Hq * 4) + (size_t)B * Hq * cap * 4;
  return n;
}

cudaError_t launch_cache_attn(const Cache& c, int dtype, const void* q, void* out, float* lse, float* weights,
                              bool accumulate, void* workspace, cudaStream_t st) {
  DecodeArgs a;
  a.c = c;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.split = is_split(c.B, c.Hkv, c.cap);
  a.part = workspace;
  a.joins = (int2*)((char*)workspace + parts_bytes(c.G));
  a.row_lse2 = nullptr;
  a.logits = nullptr;
  if (weights) {
    char* p = (char*)workspace + cache_attn_workspace(c.B, c.Hq, c.Hkv, c.cap, false);
    a.row_lse2 = (float*)p;
    a.logits = (float*)(p + up1k((size_t)c.B * c.Hq * 4));
  }
  cudaError_t e = dtype == PACK3D_BF16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
  if (e != cudaSuccess || !weights || c.cap == 0) return e;
  const dim3 grid((unsigned)((c.cap + 255) / 256), c.B);
  return launch_behind(cache_weights_kernel, grid, 256, 0, st, 1, c, a.logits, a.row_lse2, weights, (int)accumulate);
}

}  // namespace seq
}  // namespace pack3d
