// Attention of chunks of new tokens over all visible entries of a paged cache and a window of raw
// rows (cskvs_chunk_attn): a warp for each (query, head), the keys one after the other with a
// running maximum and sum, everything in fp32.
#include <cmath>

#include "codec.cuh"
#include "internal.h"

namespace cskv {

namespace {

constexpr int kD = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct ChunkArgs {
  const uint8_t* q;
  const int32_t* cu_q;
  const int32_t* ctx_len;
  int R, T, H;
  cskv_paged entries, rows;
  int has_entries, has_rows, entry_bytes, row_bytes;
  int ratio;
  const int32_t* n_entries;
  int max_entries, window, max_ctx;
  const float* sink;
  float scale_log2;
  const float* q_rope;
  uint8_t* out;
  float* lse;
};

// 16 neighbouring dims of a row
__device__ __forceinline__ void row_values(const cskv_paged& c, const RowPtr& r, int lane, float (&v)[16]) {
  if (c.fmt == CSKV_FMT_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = load_bf16x4(r.data + lane * 32 + i * 8);
      v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
    }
  } else if (c.fmt == CSKV_FMT_FP8_E4M3_E8M0_B32) {
    const float s = exp2i(static_cast<int>(r.scale[lane >> 1]) - 127);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = e4m3_to_f32(r.data[lane * 16 + i]) * s;
  } else {
    const float s = e4m3_to_f32(r.scale[lane]);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int code = (r.data[lane * 8 + (i >> 1)] >> (4 * (i & 1))) & 15, m = code & 7;
      const float mag = m < 4 ? 0.5f * m : m == 4 ? 2.f : m == 5 ? 3.f : m == 6 ? 4.f : 6.f;
      v[i] = (code & 8 ? -mag : mag) * s;
    }
  }
}

__global__ void __launch_bounds__(256) chunk_attn_simple_kernel(const __grid_constant__ ChunkArgs a) {
  const long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int i = static_cast<int>(w / a.H), h = static_cast<int>(w - static_cast<long long>(i) * a.H);
  if (i >= a.T || i >= a.cu_q[a.R]) return;
  int r = 0, n = a.R;
  while (n > 1) {
    const int half = n / 2;
    const bool le = a.cu_q[r + half] <= i;
    r = le ? r + half : r;
    n = le ? n - half : half;
  }
  int len = a.ctx_len != nullptr ? a.ctx_len[r] : 0;
  if (len < 0 || len > a.max_ctx) { set_err(CSKV_ERR_BOUNDS); len = max(0, min(len, a.max_ctx)); }
  const int p1 = len - (a.cu_q[r + 1] - i) + 1;
  int see = 0;
  if (a.has_entries) {
    see = a.ratio > 0 ? max(p1, 0) / a.ratio : a.max_entries;
    if (a.n_entries != nullptr) {
      int m = a.n_entries[r];
      if (m < 0 || m > a.max_entries) { set_err(CSKV_ERR_BOUNDS); m = max(0, min(m, a.max_entries)); }
      see = min(see, m);
    }
    if (see > a.max_entries) { set_err(CSKV_ERR_BOUNDS); see = a.max_entries; }
  }
  const int lo = a.has_rows ? max(0, p1 - a.window) : 0, hi = a.has_rows ? max(0, p1) : 0;
  float q[16], o[16];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 x = load_bf16x4(a.q + ((static_cast<size_t>(i) * a.H + h) * kD + lane * 16 + k * 4) * 2);
    q[4 * k] = x.x; q[4 * k + 1] = x.y; q[4 * k + 2] = x.z; q[4 * k + 3] = x.w;
  }
  const float* cs = a.q_rope + static_cast<size_t>(i) * 64 + (lane - 28) * 16;
  if (lane >= 28) {
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      const float c = cs[k], s = cs[k + 1], y0 = q[k], y1 = q[k + 1];
      q[k] = y0 * c - y1 * s;
      q[k + 1] = y0 * s + y1 * c;
    }
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) o[k] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < see + (hi - lo); ++j) {
    const bool entry = j < see;
    const cskv_paged& c = entry ? a.entries : a.rows;
    const RowPtr row = paged_row(c, r, entry ? j : lo + j - see, entry ? a.entry_bytes : a.row_bytes);
    if (row.data == nullptr) continue;
    float v[16], z = 0.f;
    row_values(c, row, lane, v);
#pragma unroll
    for (int k = 0; k < 16; ++k) z = fmaf(q[k], v[k], z);
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, s);
    z *= a.scale_log2;
    const float now = fmaxf(m, z), f = m == -INFINITY ? 0.f : exp2f(m - now), p = exp2f(z - now);
    l = l * f + p;
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = o[k] * f + p * v[k];
    m = now;
  }
  const float sink = a.sink != nullptr ? a.sink[h] : -INFINITY, s2 = sink * kLog2e;
  const float M = fmaxf(m, s2), e = exp2f(m - M);
  const bool none = l == 0.f || s2 == INFINITY;
  const float total = l * e + (s2 == -INFINITY ? 0.f : exp2f(s2 - M));
  const float f = none ? 0.f : l != l ? l : e / total;
#pragma unroll
  for (int k = 0; k < 16; ++k) o[k] *= f;
  if (lane >= 28) {
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      const float c = cs[k], s = cs[k + 1], y0 = o[k], y1 = o[k + 1];
      o[k] = y0 * c + y1 * s;
      o[k + 1] = y1 * c - y0 * s;
    }
  }
  __nv_bfloat162* out = reinterpret_cast<__nv_bfloat162*>(a.out + ((static_cast<size_t>(i) * a.H + h) * kD + lane * 16) * 2);
#pragma unroll
  for (int k = 0; k < 8; ++k) out[k] = __floats2bfloat162_rn(o[2 * k], o[2 * k + 1]);
  if (lane == 0 && a.lse != nullptr)
    a.lse[static_cast<size_t>(i) * a.H + h] = none ? sink : l != l ? l : (M + log2f(total)) * kLn2;
}

}  // namespace

size_t chunk_attn_workspace_bytes(int R, int T, int H, int64_t max_keys) { return 0; }

cudaError_t launch_chunk_attn(const void* q, const int32_t* cu_q, const int32_t* ctx_len, int R, int T, int H,
                              const cskv_paged* entries, int ratio, const int32_t* n_entries, int max_entries,
                              const cskv_paged* rows, int window, int max_ctx, const float* sink, float scale,
                              const float* q_rope, void* out, float* lse, int64_t max_keys, void* workspace,
                              cudaStream_t stream) {
  ChunkArgs a = {};
  a.q = static_cast<const uint8_t*>(q);
  a.cu_q = cu_q;
  a.ctx_len = ctx_len;
  a.R = R;
  a.T = T;
  a.H = H;
  if (entries != nullptr) {
    a.has_entries = 1;
    a.entries = *entries;
    a.entry_bytes = static_cast<int>(cskv_row_bytes(entries->fmt, kD));
  }
  if (rows != nullptr) {
    a.has_rows = 1;
    a.rows = *rows;
    a.row_bytes = static_cast<int>(cskv_row_bytes(rows->fmt, kD));
  }
  a.ratio = ratio;
  a.n_entries = n_entries;
  a.max_entries = max_entries;
  a.window = window;
  a.max_ctx = max_ctx;
  a.sink = sink;
  a.scale_log2 = scale * kLog2e;
  a.q_rope = q_rope;
  a.out = static_cast<uint8_t*>(out);
  a.lse = lse;
  const long long warps = static_cast<long long>(T) * H;
  chunk_attn_simple_kernel<<<static_cast<unsigned>((warps + 7) / 8), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

unsigned int take_err_chunk_attn() { return take_dev_err(); }

}  // namespace cskv
