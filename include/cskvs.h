/*
 * cskvs - one step of a server: from the requests' lengths to the attention of the
 * step's new tokens.  The part of libcskv.so beside cskv.h and cskvx.h, whose
 * conventions (cskv_paged, formats, ownership, asynchrony, status codes,
 * cskv_device_status) hold here too.
 *
 * The calls work together; nothing in between goes through the host:
 *   cskvs_plan_step   lengths -> block tables, slots, positions of the step's tokens,
 *   cskvs_rope_cs     positions -> their (cos, sin) table,
 *   cskvs_norm_rope   normed queries (not rotated: every attention call turns its own), normed
 *                     and rotated index queries; normed, rotated and coded cache rows in
 *                     those slots (raw rows; cskv_compress writes entries, with first_row as
 *                     its first_entry),
 *   cskvs_chunk_attn  the new tokens' attention over all visible entries and a window.
 *
 * Every pointer is device memory unless it says host.  Arguments are checked on the
 * host before anything is launched (CSKV_ERR_INVALID).  What only the device can see
 * (a length beyond its bound, an index outside its table or pool) is cut or skipped and
 * sets CSKV_ERR_BOUNDS.  A workspace belongs to one call at a time.  A wait inside a
 * kernel that runs out (cskv_set_spin_limit) ends the kernel with CSKV_ERR_TIMEOUT on
 * the device; its outputs are then not defined.  The same call gives the same bits each
 * time.
 */
#ifndef CSKVS_H
#define CSKVS_H

#include "cskv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * cskvs_plan_step: block tables and slot maps of a step, from the requests' lengths.
 * Request b has ctx_len[b] tokens and gets n_new[b] more; n_new[b] = 0: none this step,
 * n_new[b] < 0: the request ends (its new length is 0).  The new tokens are numbered
 * request by request, cu_new[b] .. cu_new[b+1] - 1 of request b; those from T on are cut
 * off (CSKV_ERR_BOUNDS).  With new_len[b] = ctx_len[b] + its new tokens:
 *   first_row[b] = floor(ctx_len[b] / ratio), n_rows[b] = floor(new_len[b] / ratio): the
 *     rows (raw rows at ratio 1, entries of a compressor otherwise) before the step and
 *     after it, so that it writes rows first_row .. n_rows - 1; both 0 where a request ends;
 *   token i < cu_new[B]: req_of[i], pos1[i] = its position + 1; slot[i] = the physical row
 *     (page * 64 + row % 64) of the row that it completes (position + 1 a multiple of
 *     ratio), -1 if it completes none or has no page; ring_slot[i] = b * ring_rows +
 *     position % ring_rows for the request's last ring_rows tokens, -1 for those that later
 *     tokens of the step overwrite;
 *   tokens cu_new[B] <= i < T: req_of -1, pos1 0, slot -1, ring_slot -1 (padding).
 * Pages.  block_table (NULL: none, and no slots) is int32 [B, max_pages]; free_pages is a
 * ring of `capacity` ids of free pages, state[0] the place of the first one, state[1] how
 * many there are.  A request that outgrows its pages gets new ones, requests in order, its
 * pages in order, from the front of the ring, written into its row of the table; where
 * none is left the table gets -1 and state_out[2] counts the missing pages.  No later step
 * fills such a hole: the rows of that page were not kept (their slots are -1), and the request
 * goes on behind it; a caller that needs them ends the request and begins it again.  The
 * pages of a request that ends go behind the last one, requests in order, except the first
 * shared_pages[b] places of its row (pages that are not its own; NULL: none) and those that
 * hold no page (negative ids); they can be taken from the next step on.  The table's row of
 * such a request stays as it is.  state_out, int32 [4]: the
 * ring after the step (place, count), the missing pages, 0; it may be state itself.  Ids
 * outside the table or beyond the ring's capacity set CSKV_ERR_BOUNDS.
 * ctx_len, n_new, shared_pages: int32 [B]; cu_new: int32 [B + 1]; new_len (may be ctx_len
 * itself), first_row, n_rows: int32 [B]; req_of, pos1: int32 [T]; slot, ring_slot: int64
 * [T] (ring_slot NULL with ring_rows 0).  B in [1, 65535], T in [0, 2^27], ratio in
 * [1, 2^20], ring_rows in [0, 2^20], lengths up to 2^30, capacity, max_pages >= 1.
 * workspace: cskvs_plan_step_workspace_size(B) bytes, 256-byte aligned.
 * ------------------------------------------------------------------------ */
CSKV_API size_t cskvs_plan_step_workspace_size(int32_t B);
CSKV_API int32_t cskvs_plan_step(const int32_t* ctx_len, const int32_t* n_new, int32_t B, int32_t ratio, int32_t T,
                                 int32_t ring_rows, int32_t* block_table, int32_t max_pages,
                                 const int32_t* shared_pages, int32_t* free_pages, int32_t capacity,
                                 const int32_t* state, int32_t* state_out, int32_t* cu_new, int32_t* new_len,
                                 int32_t* first_row, int32_t* n_rows, int32_t* req_of, int32_t* pos1, int64_t* slot,
                                 int64_t* ring_slot, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * cskvs_rope_cs: the (cos, sin) table of positions on the device, for one axis or several
 * (time, height and width of images and video).  Pair k of the 32 turns by
 *   angle = (positions[axis[k]][i] + shift) * f_k,
 * f_k = theta^(-2k/64), with YaRN as in cskv_rope_table.  cskvs_rope_init (host code, no
 * GPU needed) fills a plan that the caller keeps: the pairs' speeds f_k / 2 pi as 96-bit
 * fractions of a turn and the axis of each (axis_of: host uint8 [32], NULL: all 0).
 *   out[i, k] = (cos, sin) fp32, off by less than an ulp (and 1.1e-18) from those of the
 * exact angle (pos * f_k with f_k in double precision; an angle that is computed in double
 * precision is itself off by 2^-53 of it), for every int32 position and every sum of one
 * with the shift, negative ones too.
 * positions: int32, axis a at positions + a * axis_stride, [T] each; out: fp32 [T, 32, 2],
 * 16-byte aligned.  axes in [1, 4]; T in [0, 2^27].
 * ------------------------------------------------------------------------ */
typedef struct {
  uint32_t speed[32][3]; /* f_k / 2 pi: bits 2^-1 .. 2^-32, 2^-33 .. 2^-64, 2^-65 .. 2^-96 */
  uint8_t axis[32];
  int32_t axes;
} cskvs_rope_plan;
CSKV_API int32_t cskvs_rope_init(cskvs_rope_plan* plan, double theta, double yarn_factor, double yarn_original,
                                 double beta_fast, double beta_slow, int32_t axes, const uint8_t* axis_of);
CSKV_API int32_t cskvs_rope_cs(const cskvs_rope_plan* plan, const int32_t* positions, int64_t axis_stride,
                               int32_t shift, int32_t T, float* out, void* stream);

/* ------------------------------------------------------------------------
 * cskvs_norm_rope: norms of queries and rows for each head, with the rotation and the
 * coding in the same pass.  Up to 4 jobs over the same T tokens in one launch.  For every
 * token i and head h of a job, x = x[i, h, :] (bf16, `dim` values):
 *   norm:    y = (x * (1 / sqrt(sum x^2 / dim + eps))) * norm_w (NULL: 1), else y = x;
 *   rotate:  the last 64 dims of y by rope_cs[i];
 *   out:     y as bf16 to out[i, h, :], or, with slot, one row (H = 1) coded into physical
 *            row slot[i] (page slot / 64, place slot % 64) of `cache`, whose block table is
 *            not looked at; slot[i] < 0: skipped; a page outside the pool: CSKV_ERR_BOUNDS.
 * Arithmetic: the fp32 operations of cskv_compress in its order (a pairwise sum of squares,
 * no fused multiply-add): the same bits as cskv_decode_append's ratio-1 job.
 * x: heads `dim` apart, tokens x_stride apart (elements, a multiple of 8, at least H * dim);
 * out likewise with out_stride; out may be x itself (same stride).  The jobs run in no order: an
 * out that overlaps its own x otherwise, or another job's x or out, is refused (columns of one
 * buffer do not overlap; pieces of two strides in one stretch of memory are refused unless no
 * multiples of the strides could meet), and no job's x lies in rows that the call codes.  No two tokens have
 * the same slot, nor two jobs the same row of one pool.  norm_w: fp32 [dim]; rope_cs: fp32 [T, 32, 2] (NULL: no job rotates); slot:
 * int64 [T].  dim 128 or 512, H in [1, 1024], T in [0, 2^27]; cache: any format of that dim
 * (dim 128: the index-key formats or BF16).  Alignment: x, out, norm_w, rope_cs 16 bytes.
 * ------------------------------------------------------------------------ */
typedef struct {
  const void* x;
  int64_t x_stride;
  int32_t H, dim;
  int32_t norm;
  const float* norm_w;
  float eps;
  int32_t rotate;
  void* out;
  int64_t out_stride;
  cskv_paged cache;    /* read only when slot != NULL */
  const int64_t* slot;
} cskvs_norm_job;
CSKV_API int32_t cskvs_norm_rope(const cskvs_norm_job* jobs, int32_t njobs, const float* rope_cs, int32_t T,
                                 void* stream);

/* ------------------------------------------------------------------------
 * cskvs_chunk_attn: attention of chunks of new tokens over everything their requests keep.
 * The queries cu_q[r] .. cu_q[r+1] - 1 are the last tokens of request r, at positions
 * t = ctx_len[r] - (cu_q[r+1] - cu_q[r]), ..., ctx_len[r] - 1 (a single token: the decode
 * step).  Query at t of request r sees, each once,
 *   the entries j < floor((t + 1) / ratio) of `entries` (ratio 1: every raw row up to its
 *   own; ratio 0: all n_entries[r] entries, as in attention to the states of an encoder,
 *   which are of another length), never more than n_entries[r], where that is given, and
 *   with `rows` the raw rows max(0, t - window + 1) .. t of its request.
 * One softmax with the sink, rotations, out and lse as in cskvx_window_attn (q comes without
 * its rotation, which the call does by q_rope_cs, and out goes with it undone); a query
 * without any key: out 0, lse the sink (-inf without one).  Queries from cu_q[R] on are
 * left as they were.  A row that no query sees never counts; no page wholly behind the
 * windows is looked up.  A key row with a value that is not finite makes the outputs of
 * the queries that see it NaN, and no others.
 * q, out: bf16 [T, H, 512]; cu_q: int32 [R + 1], from 0, not decreasing, at most T (else no
 * query is computed, CSKV_ERR_BOUNDS);
 * ctx_len: int32 [R], at most max_ctx_len; n_entries: int32 [R] (NULL: no such bound;
 * required with ratio 0); entries (NULL: none), rows (NULL: none; one of the two is
 * given): 512-d, BF16, FP8 or FP4, block tables [R, max_pages] or NULL (one flat array of
 * rows for every request); max_entries: no request's entries that count are more; sink:
 * fp32 [H] or NULL; q_rope_cs: fp32 [T, 32, 2]; lse: fp32 [T, H] or NULL.  H in [1, 128],
 * R in [1, 65535], T in [1, 2^23], ratio in [0, 2^20], window >= 1 with rows, lengths up to
 * 2^30.
 * The rows that the chunks see are first decoded into the workspace, once for all queries.
 * max_keys bounds their number over all requests: sum over r of (its entries, rounded up to
 * 16, + min(ctx_len, chunk + window - 1), rounded up to 16); a request that finds no room
 * is left without keys (CSKV_ERR_BOUNDS).  cskvs_chunk_attn_max_keys gives a bound that
 * always holds.  Alignment: q, out, q_rope_cs 16 bytes, workspace 256.
 * Precision as in cskvx_window_attn: the rotated query in two bf16 numbers, weights of the
 * second product in bf16 over their own sum, the rest fp32; logits up to 2^30 in magnitude.
 * ------------------------------------------------------------------------ */
CSKV_API int64_t cskvs_chunk_attn_max_keys(int32_t R, int32_t T, int32_t max_entries, int32_t window,
                                           int32_t max_ctx_len);
CSKV_API size_t cskvs_chunk_attn_workspace_size(int32_t R, int32_t T, int32_t H, int64_t max_keys);
CSKV_API int32_t cskvs_chunk_attn(const void* q, const int32_t* cu_q, const int32_t* ctx_len, int32_t R, int32_t T,
                                  int32_t H, const cskv_paged* entries, int32_t ratio, const int32_t* n_entries,
                                  int32_t max_entries, const cskv_paged* rows, int32_t window, int32_t max_ctx_len,
                                  const float* sink, float softmax_scale, const float* q_rope_cs, void* out,
                                  float* lse, int64_t max_keys, void* workspace, size_t workspace_bytes,
                                  void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CSKVS_H */
