/*
 * cskvx - attention over bounded and shared caches, and the eviction that keeps
 * them bounded: the part of libcskv.so beside the compressed-KV calls of cskv.h,
 * whose conventions (cskv_paged, formats, ownership, asynchrony, status codes,
 * cskv_device_status) hold here too.
 *
 * The calls work together in a decode loop:
 *   cskvx_prefix_decode_attn  attends and gives each head's log-sum-exp,
 *   cskvx_attn_weights        turns it into each entry's attention weight and
 *                             accumulates that,
 *   cskvx_evict               drops the entries of least accumulated weight once
 *                             a request has outgrown its budget; the next step's
 *                             n_entries is its n_out, and cskv_compress appends
 *                             there.
 * cskvx_window_attn serves the layers that keep raw rows: a sliding window, and the
 * first rows of the request that stay visible.
 *
 * Every pointer is device memory.  Alignment: q, out, swa, q_rope_cs 16 bytes,
 * workspaces 256 bytes, the rest their element's size.  Arguments are checked on the
 * host before anything is launched (CSKV_ERR_INVALID).  A length beyond the host's
 * bound is cut to it, an index outside its table or pool is skipped; both set
 * CSKV_ERR_BOUNDS on the device.  A workspace belongs to one call at a time.
 * Limits: 2^23 queries or requests of a call (65,535 requests in attn_weights and
 * evict), lengths and positions up to 2^30; softmax_scale is above 0, 1e38 at most.  Logits
 * are up to 2^30 in magnitude: above, where a rounding of fp32 is a factor of 2^64 between
 * weights, outputs may be NaN.
 * A wait inside a kernel that runs out (cskv_set_spin_limit) ends the kernel with
 * CSKV_ERR_TIMEOUT on the device; its outputs are then not defined.
 */
#ifndef CSKVX_H
#define CSKVX_H

#include "cskv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * cskvx_window_attn: attention over a sliding window and the first rows.
 * Query i (of T) belongs to request req_of[i] (NULL: request i) and sits at
 * position t = pos1[i] - 1; its keys are the rows j of its request in `rows` (raw
 * rows by position) with
 *   j <= t  and  (j < first  or  j > t - window),
 * each once.  For every head h:
 *   q' = q[i,h] with its last 64 dims rotated by q_rope_cs[i],
 *   z_j = (q' . c_j) * softmax_scale,   lse = ln(sum_j exp(z_j) + exp(sink[h])),
 *   out[i,h] = sum_j exp(z_j - lse) c_j with its last 64 dims rotated back.
 * One query per request is the decode step; the queries of prompts may come in any
 * order and from any requests (neighbours of one request at neighbouring positions
 * share their keys' loads).  pos1[i] <= 0 marks a padding query: no key, out 0,
 * lse the sink (-inf without one).  A row that no query sees never counts, whatever it
 * holds, and no page without a visible row is looked up: pages wholly behind the window
 * may be reused, with any table entry left behind.  (Where queries of one request lie up
 * to 64 positions apart, the rows between their windows may be read; they share pages with
 * visible ones.)
 * q, out: bf16 [T, H, 512]; rows: 512-d, format BF16, FP8 or FP4, its block table
 * [num_reqs, max_pages] (NULL: one flat array of rows for every request);
 * pos1, req_of: int32 [T]; sink: fp32 [H] or NULL; q_rope_cs: fp32 [T, 32, 2];
 * lse: fp32 [T, H] or NULL.  window >= 1, first >= 0, H in [1, 128], every pos1[i]
 * <= max_ctx_len.  A key row with a value that is not finite makes the outputs of
 * the queries that see it NaN, and no others.
 * The query is kept as the sum of two bf16 numbers after its rotation (logits of N(0, 2)
 * are exact to about 2e-6, rms), products run as bf16 tensor-core MMAs with fp32
 * accumulation, weights enter the second product
 * as bf16 and the output is divided by the sum of the rounded ones; lse is made of the
 * fp32 weights; sums, maxima and partial outputs are fp32.  The same call gives the
 * same bits each time.
 * ------------------------------------------------------------------------ */
CSKV_API size_t cskvx_window_attn_workspace_size(int32_t T, int32_t H, int32_t max_ctx_len, int32_t window,
                                                 int32_t first);
CSKV_API int32_t cskvx_window_attn(const void* q, cskv_paged rows, int32_t num_reqs, const int32_t* req_of,
                                   const int32_t* pos1, int32_t window, int32_t first, int32_t max_ctx_len,
                                   const float* sink, float softmax_scale, const float* q_rope_cs, int32_t T,
                                   int32_t H, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* ------------------------------------------------------------------------
 * cskvx_prefix_decode_attn: decode attention of a batch whose requests share
 * their first n_prefix entries.
 * Request b's keys are its entries j < n_entries[b] of main_kv and, with swa, the
 * rows of its 128-slot window ring (slot r holds a key when r < ctx_len[b]); one
 * softmax with the sink, rotations, out and lse as in cskvx_window_attn.  The
 * entries j < n_prefix are read through request 0's block-table row, once for blocks of
 * 64 (request, head) rows, or with each request's own entries where that takes less
 * time; the entries from n_prefix on through the request's own row.  n_prefix need not
 * be a multiple of the page: rows of request 0 stand for everybody's below it.  A
 * request with fewer than n_prefix entries sees those it has (request 0's pages hold
 * all n_prefix of them in any case).  n_prefix = 0: nothing is shared.  Unlike
 * cskv_sparse_decode_attn the number of entries does not follow from a context
 * length, so a cache that cskvx_evict has cut is read as it is.
 * n_entries: int32 [B], 0 .. max_entries (0: none); ctx_len: int32 [B], <= 0: empty
 * ring (may be NULL without swa); n_prefix in [0, max_entries].  main_kv: 512-d,
 * BF16, FP8 or FP4, block table [B, max_pages] or NULL; swa: [B, 128,
 * row_bytes(swa_fmt, 512)] BF16 or FP8, or NULL.  A request without any key: out
 * 0, lse the sink (-inf without one).
 * ------------------------------------------------------------------------ */
CSKV_API size_t cskvx_prefix_decode_attn_workspace_size(int32_t B, int32_t H, int32_t n_prefix,
                                                        int32_t max_entries, int32_t with_swa);
CSKV_API int32_t cskvx_prefix_decode_attn(const void* q, cskv_paged main_kv, const int32_t* n_entries,
                                          int32_t n_prefix, int32_t max_entries, const void* swa, int32_t swa_fmt,
                                          const int32_t* ctx_len, const float* sink, float softmax_scale,
                                          const float* q_rope_cs, int32_t B, int32_t H, void* out, float* lse,
                                          void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * cskvx_attn_weights: accumulated attention weights.  For every request b and
 * entry j with first <= j < n_entries[b]:
 *   acc_out[b, j] = decay * acc[b, j] + sum_h exp(z_{b,h,j} - lse[b, h]),
 * z of the entry's row in request b's own pages, lse what cskvx_prefix_decode_attn gave (a
 * row whose lse is -inf adds nothing); other elements of acc_out are left as they are.
 * After a call with n_prefix > 0 take first >= n_prefix: entries below n_prefix were
 * attended to in request 0's pages, and have their weights here only where every
 * request's table row and pages hold the prefix too.  acc, acc_out: fp32 [B, stride],
 * stride >= max_entries; acc_out may be acc itself.  decay finite.  H in [1, 128].  The
 * rotated query is kept as three bf16 numbers and a logit summed in four parts (two above
 * 64 heads), so that logits of N(0, 2) are exact to about 2e-7 (rms; 6e-7 above 64 heads).
 * ------------------------------------------------------------------------ */
CSKV_API int32_t cskvx_attn_weights(const void* q, cskv_paged main_kv, const int32_t* n_entries, int32_t first,
                                    int32_t max_entries, float softmax_scale, const float* q_rope_cs,
                                    const float* lse, int32_t B, int32_t H, float decay, const float* acc,
                                    int64_t acc_stride, float* acc_out, int64_t acc_out_stride, void* stream);

/* ------------------------------------------------------------------------
 * cskvx_evict: cuts each request's entries to a budget by accumulated weight.
 * A request with n = n_entries[b] <= budget keeps everything.  Otherwise `budget`
 * slots stay, in this order of preference: the protected ones (slots below `fixed`,
 * and with age the entries whose age is above newest - recent, newest the largest
 * age among the n), then larger acc, at equal acc the lower slot (+0 and -0 are
 * equal, NaN is below everything).  With m = min(n, budget) entries kept, a kept
 * slot below m stays where it is; the kept slots from m on move, in ascending
 * order, into the slots below m that were given up, in ascending order: the fewest
 * rows move, and slots below `fixed` are not written: pages that requests share hold slots
 * below `fixed` alone (a shared prefix of n_prefix entries: fixed >= n_prefix, and the slots
 * from `fixed` on in pages of the request's own).
 * The rows of all `ncaches` caches (1..4; any format, tables of their own, NULL only with
 * B = 1) move, and
 *   src[b, i]      = the slot whose entry slot i now holds (i < m), -1 for m <= i < budget,
 *   acc_out[b, i]  = acc[b, src[b, i]],  age_out likewise, for i < m,
 *   n_out[b]       = m.
 * acc_out may be acc, age_out age and n_out n_entries (each wholly, same stride, or
 * not overlapping at all).  age: int32 [B, stride], a number that grows with every
 * entry the caller appends; NULL: none, recent must be 0.  src: int32 [B, budget].
 * budget >= 1, fixed, recent >= 0, fixed + recent <= budget.
 * ------------------------------------------------------------------------ */
CSKV_API size_t cskvx_evict_workspace_size(int32_t B, int32_t max_entries, int32_t budget);
CSKV_API int32_t cskvx_evict(const cskv_paged* caches, int32_t ncaches, const float* acc, int64_t acc_stride,
                             const int32_t* age, int64_t age_stride, const int32_t* n_entries, int32_t B,
                             int32_t max_entries, int32_t budget, int32_t fixed, int32_t recent, int32_t* src,
                             float* acc_out, int64_t acc_out_stride, int32_t* age_out, int64_t age_out_stride,
                             int32_t* n_out, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CSKVX_H */
