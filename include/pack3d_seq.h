/*
 * pack3d_seq.h - C ABI of the causal sequence operators of libpack3d.so
 * (sm_100a): attention of packed one-dimensional token sequences with a
 * sliding window and a few first tokens that stay visible, its backward, and
 * the paged key-value cache that serves the same attention one token at a
 * time.  A model that reads packed 3D tokens with pack3d_forward and writes or
 * reads a token sequence next to them (a caption, a report, a conversation
 * about the volume) needs both; they share the head layout, the types, the
 * status codes and the conventions of pack3d.h:
 *
 * - DEVICE pointers unless stated, owned by the caller, contiguous; tensors of
 *   the operator's type 16-byte aligned, index and float tensors 4-byte
 *   aligned.  Nothing is allocated, freed or kept.  Every call is asynchronous
 *   on `stream`, runs on the current device and can be captured into a CUDA
 *   graph (workspaces of calls that may overlap must be distinct).  What a call
 *   writes overlaps none of its inputs and nothing else that it writes
 *   (PACK3D_ERR_INVALID_ARG; the pages are the caller's to keep apart), but
 *   pack3d_cache_attn's out may be its q.
 * - T = float or bf16 (config.dtype); d_h = 64; Hq / Hkv in {1, 2, 4, 8};
 *   query head h reads key head floor(h * Hkv / Hq).  Rotations (or any other
 *   position code) are applied to q and k by the caller.
 * - Sequences are packed one after another: sequence b holds the rows
 *   cu[b] .. cu[b+1]-1 of a packed tensor, cu int32 [batch + 1] on the device,
 *   0 <= cu[b] <= cu[b+1] <= rows.  Rows outside [cu[0], cu[batch]) belong to
 *   no sequence: they are not read for a result, and outputs there stay as
 *   they were or, with zero_outside != 0, become 0 (the log-sum-exp -infinity).
 * - Errors only the device can see are OR-ed into err_word (int32, nullable):
 *   PACK3D_DEVERR_LENGTHS (offsets or lengths out of order or out of range)
 *   and PACK3D_DEVERR_PAGE (a page number outside the pool); no address
 *   outside the given buffers is touched, and the outputs of that call are
 *   unspecified.  pack3d_check_status reads them back.
 * - Limits: packed rows < 2^24; batch <= 65,535; a pool below 2^31 rows
 *   (num_pages * page).  batch == 0 or no rows: PACK3D_OK, nothing launched.
 *
 * Visible keys: the query of a sequence with Lq queries and Lk keys that sits
 * at row r of its sequence has position p = Lk - Lq + r (queries are the last
 * Lq tokens of the sequence) and sees the keys
 *   V(p) = { j : 0 <= j <= p and (window == 0 or p - j < window or j < sinks) }.
 * With Lq > Lk the first queries see no key; their output is 0 and their
 * log-sum-exp -infinity.  What a query does not see never reaches its results,
 * not even a NaN or an infinity.  (Results that a hidden one has spoilt are formed
 * again, on a slower path: a tile's rows for each such token.)
 */
#ifndef PACK3D_SEQ_H
#define PACK3D_SEQ_H

#include "pack3d.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int32_t Hq, Hkv, d_h;     /* query heads, key/value heads, head dim (64)          */
    int32_t dtype;            /* pack3d_dtype of q, k, v, the pages, out               */
    float   softmax_scale;    /* logit scale (1/sqrt(d_h))                             */
    int32_t window;           /* keys a query sees behind it, itself among them; 0 =
                                 every earlier key                                     */
    int32_t sinks;            /* first keys of a sequence that stay visible, 0..64     */
    int32_t page;             /* tokens per cache page: a power of two, 16..256        */
    int32_t flags;            /* 0 or PACK3D_FLAG_DIAG_STALL (pack3d.h)                */
    int32_t wait_limit_us;    /* as in pack3d_config                                   */
    int32_t reserved0, reserved1; /* must be 0                                         */
} pack3d_seq_config;

/* Hq=8, Hkv=2, d_h=64, bf16, scale 1/8, no window, no sinks, pages of 64. */
void pack3d_default_seq_config(pack3d_seq_config *cfg);

/* Checks a config without touching the device. */
pack3d_status pack3d_validate_seq_config(const pack3d_seq_config *cfg);

/* Causal attention of `batch` packed sequences:
 *   o[i,h] = sum_{j in V(i)} softmax_j(scale <q[i,h], k[j,g]>) v[j,g]
 * q, out T [q_rows,Hq,64]; k, v T [k_rows,Hkv,64]; cu_q, cu_k int32 [batch+1]
 * (the same pointer where queries and keys are the same tokens); lse float
 * [q_rows,Hq] (nullable): the natural log of the softmax denominator, which the
 * backward reads.  Float accumulation and softmax; bf16 runs on tcgen05 tensor
 * cores with the probabilities rounded to bf16 for the product with v, float
 * on CUDA cores. */
pack3d_status pack3d_window_attn(const pack3d_seq_config *cfg, int32_t batch, int64_t q_rows, int64_t k_rows,
                                 const int32_t *cu_q, const int32_t *cu_k, const void *q, const void *k,
                                 const void *v, void *out, float *lse, int32_t zero_outside, int32_t *err_word,
                                 void *stream);

/* Bytes of device workspace pack3d_window_attn_bwd needs (0 on an invalid
 * config or count). */
size_t pack3d_window_attn_bwd_workspace_bytes(const pack3d_seq_config *cfg, int32_t batch, int64_t q_rows,
                                              int64_t k_rows);

/* Gradients of <dout, out> of pack3d_window_attn with respect to q, k and v,
 * from that call's out and lse:
 *   P = exp(scale <q,k> - lse), dS = P (<dout,v> - <dout,out>),
 *   dq = scale dS k, dk = scale dS^T q, dv = P^T dout,
 * summed over the query heads of a key head.  dq T [q_rows,Hq,64], dk, dv T
 * [k_rows,Hkv,64]; rows of keys that no query sees get 0.  Float accumulation
 * in a fixed order: the same inputs give the same bits.  bf16 runs on tcgen05
 * tensor cores with P and dS rounded to bf16 for the products with dout, q and k.
 * workspace: 256-byte aligned, contents on entry do not matter. */
pack3d_status pack3d_window_attn_bwd(const pack3d_seq_config *cfg, int32_t batch, int64_t q_rows, int64_t k_rows,
                                     const int32_t *cu_q, const int32_t *cu_k, const void *q, const void *k,
                                     const void *v, const void *out, const float *lse, const void *dout, void *dq,
                                     void *dk, void *dv, int32_t zero_outside, void *workspace,
                                     size_t workspace_bytes, int32_t *err_word, void *stream);

/* ---- the paged cache ---------------------------------------------------------
 * Pools k_pages, v_pages T [num_pages,page,Hkv,64]; table int32
 * [batch,max_pages]: entry p of row b is the page that holds the slots
 * p*page .. (p+1)*page-1 of sequence b.  A sequence has at most max_pages*page
 * slots, its capacity.  Several rows of the table may name the same page (a
 * shared prompt) as long as no call writes there.  lengths int32 [batch]: the
 * slots in use. */

/* Writes new rows behind the cached ones: row cu[b] + i of k and v (T
 * [rows,Hkv,64]) goes to slot lengths[b] + i of sequence b.  cu NULL: one row
 * per sequence (rows == batch).  `lengths` is the number of slots in use
 * before the call and is not changed.  A row that does not fit the capacity
 * sets PACK3D_DEVERR_LENGTHS and is not written. */
pack3d_status pack3d_cache_append(const pack3d_seq_config *cfg, int32_t batch, int64_t rows, const int32_t *cu,
                                  const int32_t *lengths, const int32_t *table, int32_t max_pages,
                                  int32_t num_pages, const void *k, const void *v, void *k_pages, void *v_pages,
                                  int32_t *err_word, void *stream);

/* Bytes of device workspace pack3d_cache_attn needs; with_weights != 0 where
 * the call gets a weights buffer.  0 where it needs none (a short capacity
 * without weights; workspace may then be NULL), and on an invalid config or
 * count. */
size_t pack3d_cache_attn_workspace_bytes(const pack3d_seq_config *cfg, int32_t batch, int32_t max_pages,
                                         int32_t with_weights);

/* Attention of one new token per sequence over the cache.  lengths[b] counts
 * the new token, whose key and value were appended before: q[b] has position
 * lengths[b] - 1 and sees V(position) of the slots.  q, out T [batch,Hq,64];
 * lse float [batch,Hq] (nullable).  A sequence of length 0 gives out = 0 and
 * lse = -infinity.  weights float [batch, max_pages*page] (nullable): the
 * softmax weights of this token, summed over the Hq heads, are written
 * (accumulate == 0) or added (accumulate != 0) to the slots below lengths[b];
 * other slots stay as they were.  Float accumulation and softmax; with bf16 the
 * probabilities are rounded to bf16 for the product with v (not the weights).
 * A head whose visible scores are all -infinity gives 0 and no weight, its
 * log-sum-exp is -infinity.  The cache's length is split over the GPU's
 * processors and the parts are joined in a fixed order: the same inputs give
 * the same bits on the same GPU.  workspace: 256-byte aligned, contents on
 * entry do not matter. */
pack3d_status pack3d_cache_attn(const pack3d_seq_config *cfg, int32_t batch, const void *q, const void *k_pages,
                                const void *v_pages, const int32_t *table, int32_t max_pages, int32_t num_pages,
                                const int32_t *lengths, void *out, float *lse, float *weights, int32_t accumulate,
                                void *workspace, size_t workspace_bytes, int32_t *err_word, void *stream);

/* Cuts every sequence to at most `budget` slots by accumulated attention
 * weight.  A sequence of n > budget slots keeps its first `sinks` (config), its
 * last `recent` and, of the slots between them, those with the largest
 * weights[b][slot] (equal weights: the lower slot; -0 equals 0; a NaN is below
 * every number); a shorter one keeps all.  The kept rows are copied, in slot order, to the pages that new_table
 * (int32 [batch,new_max_pages]) names, which must be distinct and named by no
 * row of `table` (the old pages are only read, so shared ones are safe); then
 *   kept        int32 [batch,budget]: the old slot of every new slot, -1 behind
 *               the last one;
 *   new_weights float [batch, new_max_pages*page]: the kept weights, 0 behind;
 *   new_lengths int32 [batch].
 * sinks + recent <= budget <= new_max_pages*page; budget >= 1. */
pack3d_status pack3d_cache_evict(const pack3d_seq_config *cfg, int32_t batch, void *k_pages, void *v_pages,
                                 int32_t num_pages, const int32_t *table, int32_t max_pages, const int32_t *lengths,
                                 const float *weights, int32_t budget, int32_t recent, const int32_t *new_table,
                                 int32_t new_max_pages, int32_t *kept, float *new_weights, int32_t *new_lengths,
                                 int32_t *err_word, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PACK3D_SEQ_H */
