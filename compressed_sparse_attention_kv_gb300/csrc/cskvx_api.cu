// C-ABI front end of include/cskvx.h: synchronous argument checks, then launches.
#include <cmath>

#include "../../include/cskvx.h"
#include "internal.h"

using namespace cskv;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int32_t cuda_status(cudaError_t e) { return e == cudaSuccess ? CSKV_OK : CSKV_ERR_CUDA; }

constexpr unsigned kRowFormats =
    (1u << CSKV_FMT_BF16) | (1u << CSKV_FMT_FP8_E4M3_E8M0_B32) | (1u << CSKV_FMT_FP4_E2M1_E4M3_B16);
constexpr int kMaxRows = 1 << 30;  // (query, head) rows of a call
constexpr int kMaxLen = 1 << 30;   // positions and entries: sums of two stay within 32 bits
constexpr float kMaxScale = 1e38f; // finite in base 2 (times 1.4427) as well

bool cache_ok(const cskv_paged& c, unsigned formats) {
  if (c.pool == nullptr || !aligned(c.pool, 16)) return false;
  if (c.fmt < 0 || c.fmt > 4 || !((formats >> c.fmt) & 1u)) return false;
  const size_t rb = cskv_row_bytes(c.fmt, c.dim);
  const bool key = c.fmt == CSKV_FMT_FP8_E4M3_ROWSCALE_PAGESPLIT || c.fmt == CSKV_FMT_FP4_E2M1_E8M0_HADAMARD_PAGESPLIT;
  if (rb == 0 || (key && c.dim != 128)) return false;
  if (c.page_bytes < static_cast<int64_t>(64 * rb) || c.page_bytes % 16 != 0 || c.num_pages <= 0) return false;
  if (c.block_table != nullptr && (c.max_pages <= 0 || !aligned(c.block_table, 4))) return false;
  return true;
}

bool rows_ok(const cskv_paged& c) { return cache_ok(c, kRowFormats) && c.dim == 512; }

// what the three attention calls share; rows = queries
int32_t query_check(const void* q, const cskv_paged& kv, float scale, const float* q_rope_cs, int32_t rows, int32_t H) {
  if (q == nullptr || q_rope_cs == nullptr || rows < 1 || rows > kMaxRows / 128 || H < 1 || H > 128)
    return CSKV_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(q_rope_cs, 16)) return CSKV_ERR_INVALID;
  if (!(scale > 0.0f && scale <= kMaxScale) || !rows_ok(kv)) return CSKV_ERR_INVALID;
  return CSKV_OK;
}

bool workspace_ok(const void* w, size_t have, size_t need) {
  return need == 0 || (w != nullptr && aligned(w, 256) && have >= need);
}

}  // namespace

extern "C" {

size_t cskvx_window_attn_workspace_size(int32_t T, int32_t H, int32_t max_ctx_len, int32_t window, int32_t first) {
  if (T < 1 || T > kMaxRows / 128 || H < 1 || H > 128 || max_ctx_len < 0 || window < 1 || first < 0) return 0;
  return window_attn_workspace_bytes(T, H, max_ctx_len, window, first);
}

int32_t cskvx_window_attn(const void* q, cskv_paged rows, int32_t num_reqs, const int32_t* req_of,
                          const int32_t* pos1, int32_t window, int32_t first, int32_t max_ctx_len, const float* sink,
                          float softmax_scale, const float* q_rope_cs, int32_t T, int32_t H, void* out, float* lse,
                          void* workspace, size_t workspace_bytes, void* stream) {
  const int32_t st = query_check(q, rows, softmax_scale, q_rope_cs, T, H);
  if (st != CSKV_OK) return st;
  if (pos1 == nullptr || out == nullptr || !aligned(out, 16) || num_reqs < 1) return CSKV_ERR_INVALID;
  if (req_of == nullptr && num_reqs < T) return CSKV_ERR_INVALID;
  if (window < 1 || first < 0 || max_ctx_len < 0 || max_ctx_len > kMaxLen) return CSKV_ERR_INVALID;
  if (!workspace_ok(workspace, workspace_bytes, window_attn_workspace_bytes(T, H, max_ctx_len, window, first)))
    return CSKV_ERR_INVALID;
  return cuda_status(launch_window_attn(q, rows, num_reqs, req_of, pos1, window, first, max_ctx_len, sink,
                                        softmax_scale, q_rope_cs, T, H, out, lse, workspace,
                                        static_cast<cudaStream_t>(stream)));
}

size_t cskvx_prefix_decode_attn_workspace_size(int32_t B, int32_t H, int32_t n_prefix, int32_t max_entries,
                                               int32_t with_swa) {
  if (B < 1 || B > kMaxRows / 128 || H < 1 || H > 128 || n_prefix < 0 || max_entries < n_prefix) return 0;
  return prefix_attn_workspace_bytes(B, H, n_prefix, max_entries, with_swa != 0);
}

int32_t cskvx_prefix_decode_attn(const void* q, cskv_paged main_kv, const int32_t* n_entries, int32_t n_prefix,
                                 int32_t max_entries, const void* swa, int32_t swa_fmt, const int32_t* ctx_len,
                                 const float* sink, float softmax_scale, const float* q_rope_cs, int32_t B, int32_t H,
                                 void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const int32_t st = query_check(q, main_kv, softmax_scale, q_rope_cs, B, H);
  if (st != CSKV_OK) return st;
  if (n_entries == nullptr || out == nullptr || !aligned(out, 16)) return CSKV_ERR_INVALID;
  if (n_prefix < 0 || max_entries < n_prefix || max_entries > kMaxLen) return CSKV_ERR_INVALID;
  if (swa != nullptr) {
    if (!aligned(swa, 16) || ctx_len == nullptr) return CSKV_ERR_INVALID;
    if (swa_fmt != CSKV_FMT_BF16 && swa_fmt != CSKV_FMT_FP8_E4M3_E8M0_B32) return CSKV_ERR_INVALID;
  }
  if (!workspace_ok(workspace, workspace_bytes,
                    prefix_attn_workspace_bytes(B, H, n_prefix, max_entries, swa != nullptr)))
    return CSKV_ERR_INVALID;
  return cuda_status(launch_prefix_attn(q, main_kv, n_entries, n_prefix, max_entries, swa, swa_fmt, ctx_len, sink,
                                        softmax_scale, q_rope_cs, B, H, out, lse, workspace,
                                        static_cast<cudaStream_t>(stream)));
}

int32_t cskvx_attn_weights(const void* q, cskv_paged main_kv, const int32_t* n_entries, int32_t first,
                           int32_t max_entries, float softmax_scale, const float* q_rope_cs, const float* lse,
                           int32_t B, int32_t H, float decay, const float* acc, int64_t acc_stride, float* acc_out,
                           int64_t acc_out_stride, void* stream) {
  const int32_t st = query_check(q, main_kv, softmax_scale, q_rope_cs, B, H);
  if (st != CSKV_OK) return st;
  if (n_entries == nullptr || lse == nullptr || acc == nullptr || acc_out == nullptr || !std::isfinite(decay))
    return CSKV_ERR_INVALID;
  if (first < 0 || max_entries < 0 || max_entries > kMaxLen || B > 65535) return CSKV_ERR_INVALID;
  if (acc_stride < max_entries || acc_out_stride < max_entries) return CSKV_ERR_INVALID;
  if (acc == acc_out && acc_stride != acc_out_stride) return CSKV_ERR_INVALID;
  return cuda_status(launch_attn_weights(q, main_kv, n_entries, first, max_entries, softmax_scale, q_rope_cs, lse, B,
                                         H, decay, acc, acc_stride, acc_out, acc_out_stride,
                                         static_cast<cudaStream_t>(stream)));
}

size_t cskvx_evict_workspace_size(int32_t B, int32_t max_entries, int32_t budget) {
  if (B < 1 || B > 65535 || max_entries < 0 || budget < 1) return 0;
  return evict_workspace_bytes(B, max_entries, budget);
}

int32_t cskvx_evict(const cskv_paged* caches, int32_t ncaches, const float* acc, int64_t acc_stride,
                    const int32_t* age, int64_t age_stride, const int32_t* n_entries, int32_t B, int32_t max_entries,
                    int32_t budget, int32_t fixed, int32_t recent, int32_t* src, float* acc_out,
                    int64_t acc_out_stride, int32_t* age_out, int64_t age_out_stride, int32_t* n_out,
                    void* workspace, size_t workspace_bytes, void* stream) {
  if (caches == nullptr || ncaches < 1 || ncaches > 4 || acc == nullptr || n_entries == nullptr) return CSKV_ERR_INVALID;
  for (int32_t c = 0; c < ncaches; ++c)
    if (!cache_ok(caches[c], 0x1Fu)) return CSKV_ERR_INVALID;
  if (src == nullptr || acc_out == nullptr || n_out == nullptr) return CSKV_ERR_INVALID;
  if (B < 1 || B > 65535 || max_entries < 0 || max_entries > kMaxLen) return CSKV_ERR_INVALID;
  for (int32_t c = 0; c < ncaches; ++c)   // without a table all requests would move the same rows
    if (caches[c].block_table == nullptr && B > 1) return CSKV_ERR_INVALID;
  if (budget < 1 || budget > kMaxLen || fixed < 0 || recent < 0 || fixed > budget || recent > budget - fixed)
    return CSKV_ERR_INVALID;
  if (age == nullptr ? (recent != 0 || age_out != nullptr) : (age_out == nullptr || age_stride < max_entries))
    return CSKV_ERR_INVALID;
  const int64_t kept = max_entries < budget ? max_entries : budget;
  if (acc_stride < max_entries || acc_out_stride < kept || (age != nullptr && age_out_stride < kept))
    return CSKV_ERR_INVALID;
  if ((acc == acc_out && acc_stride != acc_out_stride) ||
      (age != nullptr && age == age_out && age_stride != age_out_stride))
    return CSKV_ERR_INVALID;
  if (!workspace_ok(workspace, workspace_bytes, evict_workspace_bytes(B, max_entries, budget))) return CSKV_ERR_INVALID;
  return cuda_status(launch_evict(caches, ncaches, acc, acc_stride, age, age_stride, n_entries, B, max_entries, budget,
                                  fixed, recent, src, acc_out, acc_out_stride, age_out, age_out_stride, n_out,
                                  workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
