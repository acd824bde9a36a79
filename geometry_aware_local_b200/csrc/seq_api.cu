// C ABI of the causal sequence operators (pack3d_seq.h): host-side validation
// and stream-ordered launches.  Nothing allocates, frees or synchronises.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <initializer_list>

#include "seq.cuh"

using namespace pack3d;

namespace {

constexpr int64_t kMaxRows = 1 << 24;      // packed rows, as the lattice's token limit
constexpr int32_t kMaxBatch = 65535;
constexpr int32_t kMaxSinks = 64;          // one key tile holds every sink

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

pack3d_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return PACK3D_OK;
  cudaGetLastError();  // clear a sticky launch-configuration error
  return PACK3D_ERR_CUDA;
}

// A buffer of a call: `n` elements of `size` bytes (none where p is null).
struct Span {
  uintptr_t from, to;
  Span(const void* p, int64_t n, int size) : from((uintptr_t)p), to(p ? from + (uintptr_t)n * size : from) {}
  bool meets(const Span& o) const { return from < to && o.from < o.to && from < o.to && o.from < to; }
};
// Whether a written buffer meets a read one or another written one.  (Other CTAs
// still read the inputs when the first results are written.)
bool overlap(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  for (const Span* a = written.begin(); a != written.end(); ++a) {
    for (const Span* b = written.begin(); b != a; ++b)
      if (a->meets(*b)) return true;
    for (const Span& b : read)
      if (a->meets(b)) return true;
  }
  return false;
}

int shift_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

int elem_bytes(const pack3d_seq_config& c) { return c.dtype == PACK3D_BF16 ? 2 : 4; }

// Counts every windowed call checks: PACK3D_OK, and *empty where nothing is to do.
pack3d_status check_rows(int32_t batch, int64_t q_rows, int64_t k_rows) {
  if (batch < 0 || q_rows < 0 || k_rows < 0) return PACK3D_ERR_INVALID_ARG;
  if (batch > kMaxBatch || q_rows >= kMaxRows || k_rows >= kMaxRows) return PACK3D_ERR_SHAPE;
  return PACK3D_OK;
}

seq::Win make_win(const pack3d_seq_config& c, int32_t batch, int64_t q_rows, int64_t k_rows, const int32_t* cu_q,
                  const int32_t* cu_k) {
  seq::Win w;
  memset(&w, 0, sizeof(w));
  w.cu_q = cu_q;
  w.cu_k = cu_k;
  w.B = batch;
  w.Tq = (int)q_rows;
  w.Tk = (int)k_rows;
  w.Hq = c.Hq;
  w.Hkv = c.Hkv;
  w.G = c.Hq / c.Hkv;
  w.gshift = shift_of(w.G);
  w.window = c.window >= kMaxRows ? 0 : c.window;     // longer than any sequence
  w.sinks = w.window ? c.sinks : 0;
  w.scale = c.softmax_scale;
  w.scale_log2 = (float)((double)c.softmax_scale * 1.4426950408889634);
  w.wait_ns = c.wait_limit_us > 0 ? (unsigned long long)c.wait_limit_us * 1000ull : 2000000000ull;
  w.stall = (c.flags & PACK3D_FLAG_DIAG_STALL) ? 1 : 0;
  return w;
}

// The counts and pointers every cache call shares.
pack3d_status check_cache(const pack3d_seq_config& c, int32_t batch, int32_t max_pages, int32_t num_pages) {
  if (batch < 0 || max_pages < 0 || num_pages < 0) return PACK3D_ERR_INVALID_ARG;
  if (batch > kMaxBatch) return PACK3D_ERR_SHAPE;
  if ((int64_t)max_pages * c.page >= (1LL << 31) || (int64_t)num_pages * c.page >= (1LL << 31))
    return PACK3D_ERR_SHAPE;
  return PACK3D_OK;
}

seq::Cache make_cache(const pack3d_seq_config& c, int32_t batch, const int32_t* lengths, const int32_t* table,
                      int32_t max_pages, int32_t num_pages, const void* k_pages, const void* v_pages, int32_t* err) {
  seq::Cache r;
  memset(&r, 0, sizeof(r));
  r.B = batch;
  r.Hq = c.Hq;
  r.Hkv = c.Hkv;
  r.G = c.Hq / c.Hkv;
  r.page = c.page;
  r.page_shift = shift_of(c.page);
  r.max_pages = max_pages;
  r.num_pages = num_pages;
  r.cap = max_pages * c.page;
  r.window = c.window;
  r.sinks = c.sinks;
  r.scale = c.softmax_scale;
  r.scale_log2 = (float)((double)c.softmax_scale * 1.4426950408889634);
  r.elem_bytes = elem_bytes(c);
  r.table = table;
  r.lengths = lengths;
  r.k_pages = const_cast<void*>(k_pages);
  r.v_pages = const_cast<void*>(v_pages);
  r.err = err;
  return r;
}

// The backward's workspace: Win::delta, in bf16 Win::terms, then Win::part.
size_t delta_bytes(const seq::Win& w) { return ((size_t)w.Tq * w.Hq * 4 + 1023) / 1024 * 1024; }
size_t terms_bytes(const seq::Win& w, int dtype) {
  return dtype == PACK3D_BF16 ? ((size_t)w.Tq * w.Hq * 32 + 1023) / 1024 * 1024 : 0;
}
size_t bwd_bytes(const seq::Win& w, int dtype) {
  return delta_bytes(w) + terms_bytes(w, dtype) + (seq::window_bwd_part_bytes(w, dtype) + 1023) / 1024 * 1024;
}

}  // namespace

extern "C" {

void pack3d_default_seq_config(pack3d_seq_config* cfg) {
  if (!cfg) return;
  memset(cfg, 0, sizeof(*cfg));
  cfg->Hq = 8;
  cfg->Hkv = 2;
  cfg->d_h = 64;
  cfg->dtype = PACK3D_BF16;
  cfg->softmax_scale = 0.125f;
  cfg->page = 64;
}

pack3d_status pack3d_validate_seq_config(const pack3d_seq_config* c) {
  if (!c) return PACK3D_ERR_INVALID_ARG;
  if (c->reserved0 != 0 || c->reserved1 != 0 || c->wait_limit_us < 0) return PACK3D_ERR_INVALID_ARG;
  if (c->dtype != PACK3D_F32 && c->dtype != PACK3D_BF16) return PACK3D_ERR_DTYPE;
  if (c->d_h != kDh) return PACK3D_ERR_SHAPE;
  if (c->Hq <= 0 || c->Hkv <= 0 || c->Hq % c->Hkv != 0 || c->Hq > 1024) return PACK3D_ERR_SHAPE;
  const int G = c->Hq / c->Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8) return PACK3D_ERR_SHAPE;
  if (!(c->softmax_scale > 0.f) || !isfinite(c->softmax_scale)) return PACK3D_ERR_INVALID_ARG;
  if (c->window < 0) return PACK3D_ERR_INVALID_ARG;
  if (c->sinks < 0 || c->sinks > kMaxSinks) return PACK3D_ERR_SHAPE;
  if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1))) return PACK3D_ERR_SHAPE;
  if (c->flags & ~PACK3D_FLAG_DIAG_STALL) return PACK3D_ERR_INVALID_ARG;
  return PACK3D_OK;
}

pack3d_status pack3d_window_attn(const pack3d_seq_config* cfg, int32_t batch, int64_t q_rows, int64_t k_rows,
                                 const int32_t* cu_q, const int32_t* cu_k, const void* q, const void* k,
                                 const void* v, void* out, float* lse, int32_t zero_outside, int32_t* err_word,
                                 void* stream) {
  pack3d_status st = pack3d_validate_seq_config(cfg);
  if (st == PACK3D_OK) st = check_rows(batch, q_rows, k_rows);
  if (st != PACK3D_OK) return st;
  if (batch == 0 || q_rows == 0) return PACK3D_OK;
  if (!cu_q || !cu_k || !q || !out || (k_rows > 0 && (!k || !v))) return PACK3D_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(cu_q, 4) ||
      !aligned(cu_k, 4) || !aligned(lse, 4))
    return PACK3D_ERR_ALIGNMENT;
  const int e = elem_bytes(*cfg) * kDh;
  const int64_t nq = q_rows * cfg->Hq, nk = k_rows * cfg->Hkv;
  if (overlap({{out, nq, e}, {lse, nq, 4}},
              {{q, nq, e}, {k, nk, e}, {v, nk, e}, {cu_q, batch + 1, 4}, {cu_k, batch + 1, 4}}))
    return PACK3D_ERR_INVALID_ARG;
  seq::Win w = make_win(*cfg, batch, q_rows, k_rows, cu_q, cu_k);
  w.q = q;
  w.k = k;
  w.v = v;
  w.out = out;
  w.lse = lse;
  w.zero_outside = zero_outside != 0;
  w.err = err_word;
  return cuda_status(seq::launch_window_attn(w, cfg->dtype, (cudaStream_t)stream));
}

size_t pack3d_window_attn_bwd_workspace_bytes(const pack3d_seq_config* cfg, int32_t batch, int64_t q_rows,
                                              int64_t k_rows) {
  if (pack3d_validate_seq_config(cfg) != PACK3D_OK || check_rows(batch, q_rows, k_rows) != PACK3D_OK) return 0;
  return bwd_bytes(make_win(*cfg, batch, q_rows, k_rows, nullptr, nullptr), cfg->dtype);
}

pack3d_status pack3d_window_attn_bwd(const pack3d_seq_config* cfg, int32_t batch, int64_t q_rows, int64_t k_rows,
                                     const int32_t* cu_q, const int32_t* cu_k, const void* q, const void* k,
                                     const void* v, const void* out, const float* lse, const void* dout, void* dq,
                                     void* dk, void* dv, int32_t zero_outside, void* workspace,
                                     size_t workspace_bytes, int32_t* err_word, void* stream) {
  pack3d_status st = pack3d_validate_seq_config(cfg);
  if (st == PACK3D_OK) st = check_rows(batch, q_rows, k_rows);
  if (st != PACK3D_OK) return st;
  if (batch == 0 || (q_rows == 0 && k_rows == 0)) return PACK3D_OK;
  if (!cu_q || !cu_k || (q_rows > 0 && (!q || !out || !lse || !dout || !dq)) ||
      (k_rows > 0 && (!k || !v || !dk || !dv)))
    return PACK3D_ERR_INVALID_ARG;
  seq::Win w = make_win(*cfg, batch, q_rows, k_rows, cu_q, cu_k);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < bwd_bytes(w, cfg->dtype))
    return PACK3D_ERR_WORKSPACE;
  const void* ptrs[] = {q, k, v, out, dout, dq, dk, dv};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return PACK3D_ERR_ALIGNMENT;
  if (!aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(lse, 4)) return PACK3D_ERR_ALIGNMENT;
  const int e = elem_bytes(*cfg) * kDh;
  const int64_t nq = q_rows * cfg->Hq, nk = k_rows * cfg->Hkv;
  if (overlap({{dq, nq, e}, {dk, nk, e}, {dv, nk, e}, {workspace, (int64_t)bwd_bytes(w, cfg->dtype), 1}},
              {{q, nq, e}, {k, nk, e}, {v, nk, e}, {out, nq, e}, {lse, nq, 4}, {dout, nq, e}, {cu_q, batch + 1, 4},
               {cu_k, batch + 1, 4}}))
    return PACK3D_ERR_INVALID_ARG;
  w.q = q;
  w.k = k;
  w.v = v;
  w.out = const_cast<void*>(out);
  w.lse = const_cast<float*>(lse);
  w.dout = dout;
  w.dq = dq;
  w.dk = dk;
  w.dv = dv;
  w.delta = (float*)workspace;
  w.terms = (char*)workspace + delta_bytes(w);
  w.part = (float*)((char*)w.terms + terms_bytes(w, cfg->dtype));
  w.zero_outside = zero_outside != 0;
  w.err = err_word;
  return cuda_status(seq::launch_window_bwd(w, cfg->dtype, (cudaStream_t)stream));
}

pack3d_status pack3d_cache_append(const pack3d_seq_config* cfg, int32_t batch, int64_t rows, const int32_t* cu,
                                  const int32_t* lengths, const int32_t* table, int32_t max_pages,
                                  int32_t num_pages, const void* k, const void* v, void* k_pages, void* v_pages,
                                  int32_t* err_word, void* stream) {
  pack3d_status st = pack3d_validate_seq_config(cfg);
  if (st == PACK3D_OK) st = check_cache(*cfg, batch, max_pages, num_pages);
  if (st != PACK3D_OK) return st;
  if (rows < 0 || (!cu && rows != batch)) return PACK3D_ERR_INVALID_ARG;
  if (rows >= kMaxRows) return PACK3D_ERR_SHAPE;
  if (batch == 0 || rows == 0) return PACK3D_OK;
  if (!lengths || !table || !k || !v || !k_pages || !v_pages) return PACK3D_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(cu, 4) ||
      !aligned(lengths, 4) || !aligned(table, 4))
    return PACK3D_ERR_ALIGNMENT;
  const seq::Cache c = make_cache(*cfg, batch, lengths, table, max_pages, num_pages, k_pages, v_pages, err_word);
  return cuda_status(seq::launch_cache_append(c, cu, (long)rows, k, v, (cudaStream_t)stream));
}

size_t pack3d_cache_attn_workspace_bytes(const pack3d_seq_config* cfg, int32_t batch, int32_t max_pages,
                                         int32_t with_weights) {
  if (pack3d_validate_seq_config(cfg) != PACK3D_OK || check_cache(*cfg, batch, max_pages, 0) != PACK3D_OK) return 0;
  return seq::cache_attn_workspace(batch, cfg->Hq, cfg->Hkv, max_pages * cfg->page, with_weights != 0);
}

pack3d_status pack3d_cache_attn(const pack3d_seq_config* cfg, int32_t batch, const void* q, const void* k_pages,
                                const void* v_pages, const int32_t* table, int32_t max_pages, int32_t num_pages,
                                const int32_t* lengths, void* out, float* lse, float* weights, int32_t accumulate,
                                void* workspace, size_t workspace_bytes, int32_t* err_word, void* stream) {
  pack3d_status st = pack3d_validate_seq_config(cfg);
  if (st == PACK3D_OK) st = check_cache(*cfg, batch, max_pages, num_pages);
  if (st != PACK3D_OK) return st;
  if (batch == 0) return PACK3D_OK;
  if (!q || !lengths || !out) return PACK3D_ERR_INVALID_ARG;
  if (max_pages > 0 && (!k_pages || !v_pages || !table)) return PACK3D_ERR_INVALID_ARG;
  const size_t need = seq::cache_attn_workspace(batch, cfg->Hq, cfg->Hkv, max_pages * cfg->page, weights != nullptr);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return PACK3D_ERR_WORKSPACE;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(lse, 4) ||
      !aligned(weights, 4) || !aligned(lengths, 4) || !aligned(table, 4))
    return PACK3D_ERR_ALIGNMENT;
  const int e = elem_bytes(*cfg) * kDh;
  const int64_t nq = (int64_t)batch * cfg->Hq, pool = (int64_t)num_pages * cfg->page * cfg->Hkv;
  // The results may take the queries' place: a head's are written when it has been read.
  const bool in_place = out == q;
  if (overlap({{out, nq, e}, {lse, nq, 4}, {weights, (int64_t)batch * max_pages * cfg->page, 4},
               {workspace, (int64_t)need, 1}},
              {{in_place ? nullptr : q, nq, e}, {k_pages, pool, e}, {v_pages, pool, e},
               {table, (int64_t)batch * max_pages, 4}, {lengths, batch, 4}}))
    return PACK3D_ERR_INVALID_ARG;
  const seq::Cache c = make_cache(*cfg, batch, lengths, table, max_pages, num_pages, k_pages, v_pages, err_word);
  return cuda_status(seq::launch_cache_attn(c, cfg->dtype, q, out, lse, weights, accumulate != 0, workspace,
                                            (cudaStream_t)stream));
}

pack3d_status pack3d_cache_evict(const pack3d_seq_config* cfg, int32_t batch, void* k_pages, void* v_pages,
                                 int32_t num_pages, const int32_t* table, int32_t max_pages, const int32_t* lengths,
                                 const float* weights, int32_t budget, int32_t recent, const int32_t* new_table,
                                 int32_t new_max_pages, int32_t* kept, float* new_weights, int32_t* new_lengths,
                                 int32_t* err_word, void* stream) {
  pack3d_status st = pack3d_validate_seq_config(cfg);
  if (st == PACK3D_OK) st = check_cache(*cfg, batch, max_pages, num_pages);
  if (st == PACK3D_OK) st = check_cache(*cfg, batch, new_max_pages, num_pages);
  if (st != PACK3D_OK) return st;
  if (budget < 1 || recent < 0 || (int64_t)cfg->sinks + recent > budget ||
      (int64_t)new_max_pages * cfg->page < budget)
    return PACK3D_ERR_INVALID_ARG;
  if (batch == 0) return PACK3D_OK;
  if (!k_pages || !v_pages || !table || !lengths || !weights || !new_table || !kept || !new_weights || !new_lengths)
    return PACK3D_ERR_INVALID_ARG;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16)) return PACK3D_ERR_ALIGNMENT;
  const void* words[] = {table, lengths, weights, new_table, kept, new_weights, new_lengths};
  for (const void* p : words)
    if (!aligned(p, 4)) return PACK3D_ERR_ALIGNMENT;
  const int64_t old_slots = (int64_t)batch * max_pages, new_slots = (int64_t)batch * new_max_pages;
  if (overlap({{kept, (int64_t)batch * budget, 4}, {new_weights, new_slots * cfg->page, 4}, {new_lengths, batch, 4}},
              {{table, old_slots, 4}, {lengths, batch, 4}, {weights, old_slots * cfg->page, 4}, {new_table, new_slots, 4}}))
    return PACK3D_ERR_INVALID_ARG;
  const seq::Cache c = make_cache(*cfg, batch, lengths, table, max_pages, num_pages, k_pages, v_pages, err_word);
  return cuda_status(seq::launch_cache_evict(c, weights, budget, recent, new_table, new_max_pages, kept, new_weights,
                                             new_lengths, (cudaStream_t)stream));
}

}  // extern "C"
