// Launchers and per-translation-unit error readers shared between the C-ABI
// front end (cskv_api.cu) and the kernel files.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/cskv.h"
#include "../../include/cskvs.h"

namespace cskv {

// default bound of every mbarrier spin-wait, in SM cycles (about 1 s at 2 GHz)
constexpr unsigned long long kDefaultSpinLimit = 1ull << 31;
unsigned long long spin_limit();
// measurement hook around the indexer score kernel (may be null)
void timing_events(cudaEvent_t* begin, cudaEvent_t* end);
void record_timing_event(cudaEvent_t ev, cudaStream_t stream);
void record_timing_branch(cudaEvent_t ev, cudaStream_t stream);

cudaError_t launch_compress(const void* kv, const void* gate, const void* prev_kv,
                            const void* prev_gate, const float* ape, const float* norm_w, float eps,
                            const float* rope_cs, int S, int T, int ratio, int overlap, int dim,
                            const int32_t* req, const int32_t* first_entry, const cskv_paged& out,
                            int out_row_bytes, cudaStream_t stream);

cudaError_t launch_compress_many(const cskv_compress_job* jobs, int njobs, cudaStream_t stream,
                                 bool dependent = false);
cudaError_t launch_decode_append(const cskv_decode_job* jobs, int njobs, const int32_t* pos, int B,
                                 cudaStream_t stream);

cudaError_t launch_encode_rows(const void* src, int src_bf16, int n, int dim, const int32_t* req,
                               const int32_t* row, const cskv_paged& out, int out_row_bytes,
                               cudaStream_t stream);

size_t index_workspace_bytes(int B, int n_max, int Hi, int k);
cudaError_t launch_index_topk(const void* q_idx, const float* w, const cskv_paged& keys,
                              const int32_t* ctx_len, int B, int Hi, int ratio, int k,
                              int max_ctx_len, int32_t* topk_idx, float* topk_score,
                              void* workspace, cudaStream_t stream);

// One decode step's compressor and indexer, overlapped (cskv_decode_layer): the query
// prep, then compress_many(jobs) as a programmatic dependent of it, then the score
// kernel, which reads the index keys these jobs write only after they are complete.
// *ready receives the per-request flags that the selection raises (nullptr when the
// batch takes the cooperative large-batch kernel; the attention then waits for the
// whole indexer instead).
cudaError_t launch_index_topk_fused(const void* q_idx, const float* w, const cskv_paged& keys,
                                    const int32_t* ctx_len, int B, int Hi, int ratio, int k, int max_ctx_len,
                                    int32_t* topk_idx, float* topk_score, void* workspace,
                                    const cskv_compress_job* jobs, int njobs, cudaStream_t stream,
                                    const uint32_t** ready);

cudaError_t launch_index_topk_noalloc(const void* q_idx, const float* w, const cskv_paged& keys,
                                      const int32_t* ctx_len, int B, int Hi, int ratio, int k,
                                      int max_ctx_len, int32_t* topk_idx, float* topk_score,
                                      cudaStream_t stream);

size_t attn_workspace_bytes(int B, int H, int max_ctx, int ratio, int k);
cudaError_t launch_sparse_decode_attn(const void* q, const cskv_paged& kv, const void* swa, int swa_fmt,
                                      const int32_t* ctx_len, const int32_t* topk, int k, int ratio,
                                      int max_ctx, const float* sink, float softmax_scale,
                                      const float* q_rope, int B, int H, void* out, void* workspace,
                                      cudaStream_t stream, void* out_host = nullptr,
                                      const uint32_t* ready = nullptr);
cudaError_t launch_sparse_prefill_attn(const void* q, const cskv_paged& kv, const cskv_paged& win,
                                       const int32_t* req_of, const int32_t* pos1, const int32_t* topk, int k,
                                       int ratio, int max_ctx, const float* sink, float softmax_scale,
                                       const float* q_rope, int T, int H, void* out, void* workspace,
                                       cudaStream_t stream);

// Lets `kernel` use `bytes` of dynamic shared memory, asked of the driver once per device (a
// request costs as much as a third of a launch); `again` asks in any case, after a launch that
// failed (a device reset forgets it).
inline cudaError_t allow_shared_memory(const void* kernel, std::atomic<uint64_t>& done, size_t bytes, bool again) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!again && (done.load(std::memory_order_relaxed) & bit) != 0) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}
// A launch of a kernel whose shared memory was allowed before (at most max_bytes of it).
template <class Kernel, class... Args>
inline cudaError_t launch_with_shared_memory(const cudaLaunchConfig_t& cfg, Kernel kernel, std::atomic<uint64_t>& done,
                                             size_t max_bytes, const Args&... args) {
  cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kernel), done, max_bytes, false);
  if (e != cudaSuccess) return e;
  e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaErrorInvalidValue) return e;
  cudaGetLastError();
  e = allow_shared_memory(reinterpret_cast<const void*>(kernel), done, max_bytes, true);
  return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, kernel, args...);
}

// include/cskvx.h
size_t window_attn_workspace_bytes(int T, int H, int max_ctx, int window, int first);
cudaError_t launch_window_attn(const void* q, const cskv_paged& rows, int num_reqs, const int32_t* req_of,
                               const int32_t* pos1, int window, int first, int max_ctx, const float* sink, float scale,
                               const float* q_rope, int T, int H, void* out, float* lse, void* workspace,
                               cudaStream_t stream);
size_t prefix_attn_workspace_bytes(int B, int H, int n_prefix, int max_entries, int with_swa);
cudaError_t launch_prefix_attn(const void* q, const cskv_paged& kv, const int32_t* n_entries, int n_prefix,
                               int max_entries, const void* swa, int swa_fmt, const int32_t* ctx_len, const float* sink,
                               float scale, const float* q_rope, int B, int H, void* out, float* lse, void* workspace,
                               cudaStream_t stream);
cudaError_t launch_attn_weights(const void* q, const cskv_paged& kv, const int32_t* n_entries, int first,
                                int max_entries, float scale, const float* q_rope, const float* lse, int B, int H,
                                float decay, const float* acc, long long acc_stride, float* acc_out,
                                long long acc_out_stride, cudaStream_t stream);
size_t evict_workspace_bytes(int B, int max_entries, int budget);
cudaError_t launch_evict(const cskv_paged* caches, int ncaches, const float* acc, long long acc_stride,
                         const int32_t* age, long long age_stride, const int32_t* n_entries, int B, int max_entries,
                         int budget, int fixed, int recent, int32_t* src, float* acc_out, long long acc_out_stride,
                         int32_t* age_out, long long age_out_stride, int32_t* n_out, void* workspace,
                         cudaStream_t stream);

// include/cskvs.h
// the pairs' angles per position, as cskv_rope_table has them; false: bad arguments
bool rope_speeds(double theta, double yarn_factor, double yarn_original, double beta_fast, double beta_slow,
                 double (&f)[32]);
size_t plan_step_workspace_bytes(int B);
cudaError_t launch_plan_step(const int32_t* ctx_len, const int32_t* n_new, int B, int ratio, int T, int ring_rows,
                             int32_t* table, int max_pages, const int32_t* shared, int32_t* free_pages, int capacity,
                             const int32_t* state, int32_t* state_out, int32_t* cu_new, int32_t* new_len,
                             int32_t* first_row, int32_t* n_rows, int32_t* req_of, int32_t* pos1, int64_t* slot,
                             int64_t* ring_slot, void* workspace, cudaStream_t stream);
cudaError_t launch_rope_cs(const cskvs_rope_plan& plan, const int32_t* pos, int64_t axis_stride, int shift, int T,
                           float* out, cudaStream_t stream);
cudaError_t launch_norm_rope(const cskvs_norm_job* jobs, int njobs, const float* rope_cs, int T, cudaStream_t stream);
size_t chunk_attn_workspace_bytes(int R, int T, int H, int64_t max_keys);
cudaError_t launch_chunk_attn(const void* q, const int32_t* cu_q, const int32_t* ctx_len, int R, int T, int H,
                              const cskv_paged* entries, int ratio, const int32_t* n_entries, int max_entries,
                              const cskv_paged* rows, int window, int max_ctx, const float* sink, float scale,
                              const float* q_rope, void* out, float* lse, int64_t max_keys, void* workspace,
                              cudaStream_t stream);

unsigned int take_err_compress();
unsigned int take_err_index();
unsigned int take_err_attention();
unsigned int take_err_list_attn();
unsigned int take_err_evict();
unsigned int take_err_step();
unsigned int take_err_chunk_attn();

}  // namespace cskv
