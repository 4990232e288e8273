// C-ABI front end of include/cskvs.h: synchronous argument checks, then launches.
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <numeric>

#include "../../include/cskvs.h"
#include "internal.h"

using namespace cskv;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool words(std::initializer_list<const void*> p) {   // arrays of 32-bit numbers (or none)
  return std::all_of(p.begin(), p.end(), [](const void* x) { return aligned(x, 4); });
}

int32_t cuda_status(cudaError_t e) { return e == cudaSuccess ? CSKV_OK : CSKV_ERR_CUDA; }

constexpr int kMaxTokens = 1 << 27;
constexpr int kMaxLen = 1 << 30;
constexpr int kMaxRatio = 1 << 20;
constexpr int kMaxReqs = 65535;
constexpr int kMaxQueries = 1 << 23;
constexpr float kMaxScale = 1e38f;   // finite in base 2 (times 1.4427) as well

bool index_key(int fmt) {
  return fmt == CSKV_FMT_FP8_E4M3_ROWSCALE_PAGESPLIT || fmt == CSKV_FMT_FP4_E2M1_E8M0_HADAMARD_PAGESPLIT;
}

bool cache_ok(const cskv_paged& c, int dim) {
  if (c.pool == nullptr || !aligned(c.pool, 16)) return false;
  if (c.fmt < 0 || c.fmt > 4 || c.dim != dim || (index_key(c.fmt) && dim != 128)) return false;
  const size_t rb = cskv_row_bytes(c.fmt, c.dim);
  if (rb == 0) return false;
  if (c.page_bytes < static_cast<int64_t>(64 * rb) || c.page_bytes % 16 != 0 || c.num_pages <= 0) return false;
  if (c.block_table != nullptr && (c.max_pages <= 0 || !aligned(c.block_table, 4))) return false;
  return true;
}

bool workspace_ok(const void* w, size_t have, size_t need) {
  return need == 0 || (w != nullptr && aligned(w, 256) && have >= need);
}

// What a norm job reads or writes: T pieces of `width` bytes, `stride` apart (at least the width).
struct Pieces {
  uintptr_t at;
  int64_t stride, width;
};
Pieces pieces_of(const cskvs_norm_job& j, const void* at, int64_t stride) {
  return {reinterpret_cast<uintptr_t>(at), 2 * stride, 2 * static_cast<int64_t>(j.H) * j.dim};
}
// Whether some piece i of a and some piece k of b share a byte: -a.width < d + i a.stride - k b.stride < b.width.
// With equal strides exactly; else whether the whole stretches meet and some multiple of the strides' common
// divisor lies between (pieces that pass one another in one stretch, as columns of one buffer do, do not).
bool meet(const Pieces& a, const Pieces& b, int64_t T) {
  using wide = __int128;
  const wide d = static_cast<wide>(a.at) - static_cast<wide>(b.at), last = T - 1;
  if (d + last * a.stride + a.width <= 0 || d >= last * b.stride + b.width) return false;
  const wide step = a.stride == b.stride ? a.stride : std::gcd(a.stride, b.stride);
  // the least m with d + m step > -a.width
  const wide over = -a.width - d;
  wide m = over / step - (over % step < 0) + 1;
  if (a.stride == b.stride) {
    m = std::max(m, -last);
    if (m > last) return false;
  }
  return d + m * step < b.width;
}

// 1 / 2 pi = kInvTwoPi / 2^128
constexpr uint64_t kInvTwoPi[2] = {0x28BE60DB9391054Aull, 0x7F09D5F47D4D3770ull};

// floor(f / 2 pi * 2^96) for 0 <= f <= 1, in three words
void turn_fraction(double f, uint32_t (&word)[3]) {
  int e;
  const uint64_t m = static_cast<uint64_t>(std::ldexp(std::frexp(f, &e), 53));   // f = m 2^(e - 53)
  const unsigned __int128 low = static_cast<unsigned __int128>(m) * kInvTwoPi[1];
  const unsigned __int128 high = static_cast<unsigned __int128>(m) * kInvTwoPi[0] + static_cast<uint64_t>(low >> 64);
  const int shift = 53 - e + 32;   // of the 192-bit product, whose upper 128 bits are `high`
  // product >> shift: f <= 1 makes it at least 84, and leaves less than 96 bits
  const unsigned __int128 r = shift < 192 ? high >> (shift - 64) : 0;
  word[0] = static_cast<uint32_t>(r >> 64);
  word[1] = static_cast<uint32_t>(r >> 32);
  word[2] = static_cast<uint32_t>(r);
}

}  // namespace

extern "C" {

size_t cskvs_plan_step_workspace_size(int32_t B) { return B < 1 || B > kMaxReqs ? 0 : plan_step_workspace_bytes(B); }

int32_t cskvs_plan_step(const int32_t* ctx_len, const int32_t* n_new, int32_t B, int32_t ratio, int32_t T,
                        int32_t ring_rows, int32_t* block_table, int32_t max_pages, const int32_t* shared_pages,
                        int32_t* free_pages, int32_t capacity, const int32_t* state, int32_t* state_out,
                        int32_t* cu_new, int32_t* new_len, int32_t* first_row, int32_t* n_rows, int32_t* req_of,
                        int32_t* pos1, int64_t* slot, int64_t* ring_slot, void* workspace, size_t workspace_bytes,
                        void* stream) {
  if (B < 1 || B > kMaxReqs || T < 0 || T > kMaxTokens || ratio < 1 || ratio > kMaxRatio) return CSKV_ERR_INVALID;
  if (ring_rows < 0 || ring_rows > kMaxRatio || (ring_rows > 0 ? T > 0 && ring_slot == nullptr : ring_slot != nullptr))
    return CSKV_ERR_INVALID;
  if (ctx_len == nullptr || n_new == nullptr || cu_new == nullptr || new_len == nullptr || first_row == nullptr ||
      n_rows == nullptr)
    return CSKV_ERR_INVALID;
  if (T > 0 && (req_of == nullptr || pos1 == nullptr)) return CSKV_ERR_INVALID;
  if (!words({ctx_len, n_new, block_table, shared_pages, free_pages, state, state_out, cu_new, new_len, first_row, n_rows,
              req_of, pos1}) || !aligned(slot, 8) || !aligned(ring_slot, 8))
    return CSKV_ERR_INVALID;
  if (block_table != nullptr) {
    if (max_pages < 1 || free_pages == nullptr || capacity < 1 || state == nullptr || state_out == nullptr)
      return CSKV_ERR_INVALID;
    if (T > 0 && slot == nullptr) return CSKV_ERR_INVALID;
  } else if (shared_pages != nullptr || free_pages != nullptr || state != nullptr || state_out != nullptr ||
             slot != nullptr) {
    return CSKV_ERR_INVALID;
  }
  if (!workspace_ok(workspace, workspace_bytes, plan_step_workspace_bytes(B))) return CSKV_ERR_INVALID;
  return cuda_status(launch_plan_step(ctx_len, n_new, B, ratio, T, ring_rows, block_table, max_pages, shared_pages,
                                      free_pages, capacity, state, state_out, cu_new, new_len, first_row, n_rows,
                                      req_of, pos1, slot, ring_slot, workspace, static_cast<cudaStream_t>(stream)));
}

int32_t cskvs_rope_init(cskvs_rope_plan* plan, double theta, double yarn_factor, double yarn_original, double beta_fast,
                        double beta_slow, int32_t axes, const uint8_t* axis_of) {
  if (plan == nullptr || axes < 1 || axes > 4) return CSKV_ERR_INVALID;
  double f[32];
  if (!rope_speeds(theta, yarn_factor, yarn_original, beta_fast, beta_slow, f)) return CSKV_ERR_INVALID;
  for (int k = 0; k < 32; ++k) {
    const int axis = axis_of != nullptr ? axis_of[k] : 0;
    if (axis >= axes || !(f[k] >= 0.0 && f[k] <= 1.0)) return CSKV_ERR_INVALID;
    plan->axis[k] = static_cast<uint8_t>(axis);
    turn_fraction(f[k], plan->speed[k]);
  }
  plan->axes = axes;
  return CSKV_OK;
}

int32_t cskvs_rope_cs(const cskvs_rope_plan* plan, const int32_t* positions, int64_t axis_stride, int32_t shift,
                      int32_t T, float* out, void* stream) {
  if (plan == nullptr || plan->axes < 1 || plan->axes > 4 || T < 0 || T > kMaxTokens) return CSKV_ERR_INVALID;
  for (int k = 0; k < 32; ++k)
    if (plan->axis[k] >= plan->axes) return CSKV_ERR_INVALID;
  if (T > 0 && (positions == nullptr || out == nullptr)) return CSKV_ERR_INVALID;
  if (!words({positions}) || !aligned(out, 16)) return CSKV_ERR_INVALID;
  if (plan->axes > 1 && axis_stride < T) return CSKV_ERR_INVALID;
  return cuda_status(launch_rope_cs(*plan, positions, axis_stride, shift, T, out, static_cast<cudaStream_t>(stream)));
}

int32_t cskvs_norm_rope(const cskvs_norm_job* jobs, int32_t njobs, const float* rope_cs, int32_t T, void* stream) {
  if (jobs == nullptr || njobs < 1 || njobs > 4 || T < 0 || T > kMaxTokens) return CSKV_ERR_INVALID;
  if (rope_cs != nullptr && !aligned(rope_cs, 16)) return CSKV_ERR_INVALID;
  int64_t warps = 0;
  for (int32_t i = 0; i < njobs; ++i) {
    const cskvs_norm_job& j = jobs[i];
    if ((j.dim != 128 && j.dim != 512) || j.H < 1 || j.H > 1024) return CSKV_ERR_INVALID;
    const int64_t least = static_cast<int64_t>(j.H) * j.dim;
    if (j.x_stride < least || j.x_stride % 8 != 0 || j.x_stride > (int64_t(1) << 40)) return CSKV_ERR_INVALID;
    if (T > 0 && (j.x == nullptr || !aligned(j.x, 16))) return CSKV_ERR_INVALID;
    if (j.norm_w != nullptr && (!aligned(j.norm_w, 16) || j.norm == 0)) return CSKV_ERR_INVALID;
    if (j.norm != 0 && !(j.eps >= 0.0f && std::isfinite(j.eps))) return CSKV_ERR_INVALID;
    if (j.rotate != 0 && rope_cs == nullptr) return CSKV_ERR_INVALID;
    if (j.slot != nullptr) {
      if (j.H != 1 || j.out != nullptr || !aligned(j.slot, 8) || !cache_ok(j.cache, j.dim)) return CSKV_ERR_INVALID;
    } else {
      if (T > 0 && (j.out == nullptr || !aligned(j.out, 16))) return CSKV_ERR_INVALID;
      if (j.out_stride < least || j.out_stride % 8 != 0 || j.out_stride > (int64_t(1) << 40)) return CSKV_ERR_INVALID;
      if (j.out == j.x && j.out_stride != j.x_stride) return CSKV_ERR_INVALID;
    }
    warps += static_cast<int64_t>(T) * j.H;
  }
  if (warps > (int64_t(1) << 33)) return CSKV_ERR_INVALID;   // of one launch
  // the jobs run in any order: what one writes no other one reads or writes, and itself only in place
  for (int32_t i = 0; i < njobs && T > 0; ++i) {
    if (jobs[i].slot != nullptr) continue;
    const Pieces out = pieces_of(jobs[i], jobs[i].out, jobs[i].out_stride);
    for (int32_t k = 0; k < njobs; ++k) {
      const cskvs_norm_job& o = jobs[k];
      if (!(k == i && o.x == o.out) && meet(out, pieces_of(o, o.x, o.x_stride), T)) return CSKV_ERR_INVALID;
      if (k < i && o.slot == nullptr && meet(out, pieces_of(o, o.out, o.out_stride), T)) return CSKV_ERR_INVALID;
    }
  }
  return cuda_status(launch_norm_rope(jobs, njobs, rope_cs, T, static_cast<cudaStream_t>(stream)));
}

int64_t cskvs_chunk_attn_max_keys(int32_t R, int32_t T, int32_t max_entries, int32_t window, int32_t max_ctx_len) {
  if (R < 1 || R > kMaxReqs || T < 1 || T > kMaxQueries || max_entries < 0 || max_entries > kMaxLen || window < 0 ||
      max_ctx_len < 0 || max_ctx_len > kMaxLen)
    return 0;
  // a request with queries has rows of its chunk and the window before it, or its whole length
  const int64_t reqs = std::min<int64_t>(R, T);
  const int64_t rows = window == 0 ? 0 : std::min<int64_t>(reqs * max_ctx_len, T + reqs * (static_cast<int64_t>(window) - 1));
  return reqs * ((static_cast<int64_t>(max_entries) + 15) / 16 * 16) + rows + (window == 0 ? 0 : reqs * 15);
}

size_t cskvs_chunk_attn_workspace_size(int32_t R, int32_t T, int32_t H, int64_t max_keys) {
  if (R < 1 || R > kMaxReqs || T < 1 || T > kMaxQueries || H < 1 || H > 128 || max_keys < 0 ||
      max_keys > (int64_t(1) << 40))
    return 0;
  return chunk_attn_workspace_bytes(R, T, H, max_keys);
}

int32_t cskvs_chunk_attn(const void* q, const int32_t* cu_q, const int32_t* ctx_len, int32_t R, int32_t T, int32_t H,
                         const cskv_paged* entries, int32_t ratio, const int32_t* n_entries, int32_t max_entries,
                         const cskv_paged* rows, int32_t window, int32_t max_ctx_len, const float* sink,
                         float softmax_scale, const float* q_rope_cs, void* out, float* lse, int64_t max_keys,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (R < 1 || R > kMaxReqs || T < 1 || T > kMaxQueries || H < 1 || H > 128) return CSKV_ERR_INVALID;
  if (q == nullptr || cu_q == nullptr || q_rope_cs == nullptr || out == nullptr) return CSKV_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(q_rope_cs, 16)) return CSKV_ERR_INVALID;
  if (!words({cu_q, ctx_len, n_entries, sink, lse})) return CSKV_ERR_INVALID;
  if (entries == nullptr && rows == nullptr) return CSKV_ERR_INVALID;
  const unsigned formats = (1u << CSKV_FMT_BF16) | (1u << CSKV_FMT_FP8_E4M3_E8M0_B32) | (1u << CSKV_FMT_FP4_E2M1_E4M3_B16);
  for (const cskv_paged* c : {entries, rows})
    if (c != nullptr && (!cache_ok(*c, 512) || !((formats >> c->fmt) & 1u))) return CSKV_ERR_INVALID;
  if (ratio < 0 || ratio > kMaxRatio || max_entries < 0 || max_entries > kMaxLen) return CSKV_ERR_INVALID;
  if (entries != nullptr && ratio == 0 && n_entries == nullptr) return CSKV_ERR_INVALID;
  if (rows != nullptr ? window < 1 : window != 0) return CSKV_ERR_INVALID;
  if (max_ctx_len < 0 || max_ctx_len > kMaxLen) return CSKV_ERR_INVALID;
  if (ctx_len == nullptr && (rows != nullptr || ratio != 0)) return CSKV_ERR_INVALID;   // positions count
  if (!(softmax_scale > 0.0f && softmax_scale <= kMaxScale)) return CSKV_ERR_INVALID;
  if (max_keys < 0 || max_keys > (int64_t(1) << 40)) return CSKV_ERR_INVALID;
  if (!workspace_ok(workspace, workspace_bytes, chunk_attn_workspace_bytes(R, T, H, max_keys))) return CSKV_ERR_INVALID;
  return cuda_status(launch_chunk_attn(q, cu_q, ctx_len, R, T, H, entries, ratio, n_entries, max_entries, rows, window,
                                       max_ctx_len, sink, softmax_scale, q_rope_cs, out, lse, max_keys, workspace,
                                       static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
