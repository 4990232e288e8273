// Attention over sliding windows with first rows, over shared prefixes, and the
// accumulated attention weights (cskvx_window_attn, cskvx_prefix_decode_attn,
// cskvx_attn_weights).
//
// One warp per (query, head) row, 16 dims per lane, one pass over the row's keys with
// a running maximum and sum.
#include "codec.cuh"
#include "internal.h"

namespace cskv {

namespace {

constexpr int kD = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct ListArgs {
  const uint8_t* q;
  cskv_paged kv;
  int row_bytes;
  const float* sink;
  float scale_log2;
  const float* q_rope;
  int T, H;
  uint8_t* out;
  float* lse;
  // window: queries of requests, raw rows by position
  const int32_t* req_of;
  const int32_t* pos1;
  int num_reqs, window, first, max_ctx;
  // entries of requests
  const int32_t* n_entries;
  int n_prefix, max_entries;
  const uint8_t* swa;
  int swa_fmt, swa_row_bytes;
  const int32_t* ctx_len;
  // weights
  const float* lse_in;
  const float* acc;
  long long acc_stride;
  float* acc_out;
  long long acc_out_stride;
  float decay;
};

// dims 16 l .. 16 l + 15 of a row
__device__ __forceinline__ void row16(int fmt, const uint8_t* p, int l, float (&v)[16]) {
  if (fmt == CSKV_FMT_BF16) {
    for (int i = 0; i < 4; ++i) {
      const float4 x = load_bf16x4(p + 32 * l + 8 * i);
      v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
    }
  } else if (fmt == CSKV_FMT_FP8_E4M3_E8M0_B32) {
    const float s = exp2i(static_cast<int>(p[kD + (l >> 1)]) - 127);
    for (int i = 0; i < 16; ++i) v[i] = e4m3_to_f32(p[16 * l + i]) * s;
  } else {
    const float s = e4m3_to_f32(p[kD / 2 + l]);
    for (int i = 0; i < 8; ++i) {
      uint32_t h;
      asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
          : "=r"(h) : "r"(static_cast<uint32_t>(p[8 * l + i])));
      v[2 * i] = __half2float(__ushort_as_half(h & 0xFFFF)) * s;
      v[2 * i + 1] = __half2float(__ushort_as_half(h >> 16)) * s;
    }
  }
}

struct RowState {
  float q[16], o[16], m, l;
};

__device__ __forceinline__ void rotate16(const float* cs, int lane, float sign, float (&v)[16]) {
  if (lane < 28) return;
  for (int i = 0; i < 8; ++i) {
    const int k = 8 * (lane - 28) + i;
    const float c = cs[2 * k], s = sign * cs[2 * k + 1];
    const float y0 = v[2 * i], y1 = v[2 * i + 1];
    v[2 * i] = y0 * c - y1 * s;
    v[2 * i + 1] = y0 * s + y1 * c;
  }
}

// the key's logit in base 2 (all lanes), its values in v
__device__ __forceinline__ float logit(const ListArgs& a, int fmt, const uint8_t* p, int lane, const float (&q)[16],
                                       float (&v)[16]) {
  row16(fmt, p, lane, v);
  float z = 0.f;
  for (int i = 0; i < 16; ++i) z += q[i] * v[i];
  for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
  bool fine = true;   // a row that is not finite makes its logits NaN
  for (int i = 0; i < 16; ++i) fine = fine && fabsf(v[i]) < INFINITY;
  if (!__all_sync(0xFFFFFFFFu, fine)) return __int_as_float(0x7FC00000);
  return z * a.scale_log2;
}

__device__ __forceinline__ void attend(const ListArgs& a, int fmt, const uint8_t* p, int lane, RowState& r) {
  if (p == nullptr) return;
  float v[16];
  const float z = logit(a, fmt, p, lane, r.q, v);
  const float m = fmaxf(r.m, z);
  const float f = r.m == -INFINITY ? 0.f : exp2f(r.m - m);
  const float e = exp2f(z - m);
  r.l = r.l * f + e;
  for (int i = 0; i < 16; ++i) r.o[i] = r.o[i] * f + e * v[i];
  r.m = m;
}

__device__ __forceinline__ void load_query(const ListArgs& a, int t, int h, int lane, float (&q)[16]) {
  row16(CSKV_FMT_BF16, a.q + (size_t(t) * a.H + h) * kD * 2, lane, q);
  rotate16(a.q_rope + size_t(t) * 64, lane, 1.f, q);
}

__device__ __forceinline__ int cut(int n, int most) {
  if (n > most) { set_err(CSKV_ERR_BOUNDS); n = most; }
  return n;
}

__global__ void __launch_bounds__(256) list_attn_kernel(const ListArgs a) {
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= (long long)a.T * a.H) return;
  const int t = static_cast<int>(row / a.H), h = static_cast<int>(row % a.H);
  RowState r;
  load_query(a, t, h, lane, r.q);
  for (int i = 0; i < 16; ++i) r.o[i] = 0.f;
  r.m = -INFINITY;
  r.l = 0.f;
  if (a.pos1 != nullptr) {
    const int pos = cut(a.pos1[t], a.max_ctx) - 1;
    const int req = a.req_of ? a.req_of[t] : t;
    if (pos >= 0 && (req < 0 || req >= a.num_reqs)) {
      set_err(CSKV_ERR_BOUNDS);
    } else {
      const int lo = max(0, pos - a.window + 1);
      for (int j = 0; j < min(a.first, lo); ++j) attend(a, a.kv.fmt, paged_row(a.kv, req, j, a.row_bytes).data, lane, r);
      for (int j = lo; j <= pos; ++j) attend(a, a.kv.fmt, paged_row(a.kv, req, j, a.row_bytes).data, lane, r);
    }
  } else {
    int n = a.n_entries[t];
    if (n < 0) { set_err(CSKV_ERR_BOUNDS); n = 0; }
    n = cut(n, a.max_entries);
    for (int j = 0; j < n; ++j)
      attend(a, a.kv.fmt, paged_row(a.kv, j < a.n_prefix ? 0 : t, j, a.row_bytes).data, lane, r);
    if (a.swa != nullptr) {
      const int w = min(a.ctx_len[t], kWindow);
      for (int j = 0; j < w; ++j)
        attend(a, a.swa_fmt, a.swa + (size_t(t) * kWindow + j) * a.swa_row_bytes, lane, r);
    }
  }
  const bool empty = r.l == 0.f;   // no key: out 0, lse the sink itself
  if (a.sink != nullptr) {
    const float s = a.sink[h] * kLog2e, m = fmaxf(r.m, s);
    if (m > -INFINITY) {
      const float f = r.m == -INFINITY ? 0.f : exp2f(r.m - m);
      r.l = r.l * f + exp2f(s - m);
      for (int i = 0; i < 16; ++i) r.o[i] *= f;
      r.m = m;
    }
  }
  const float inv = r.l == 0.f ? 0.f : 1.0f / r.l;
  for (int i = 0; i < 16; ++i) r.o[i] *= inv;
  rotate16(a.q_rope + size_t(t) * 64, lane, -1.f, r.o);
  __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(a.out + (size_t(row) * kD + 16 * lane) * 2);
  for (int i = 0; i < 8; ++i) o[i] = __floats2bfloat162_rn(r.o[2 * i], r.o[2 * i + 1]);
  if (a.lse != nullptr && lane == 0) a.lse[row] = empty ? (a.sink ? a.sink[h] : -INFINITY) : (r.m + log2f(r.l)) * kLn2;
}

// one warp per (request, entry)
__global__ void __launch_bounds__(256) weights_kernel(const ListArgs a) {
  const int b = blockIdx.y;
  const int j = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  int n = a.n_entries[b];
  if (n < 0) { set_err(CSKV_ERR_BOUNDS); n = 0; }
  n = cut(n, a.max_entries);
  if (j < a.first || j >= n) return;
  const uint8_t* p = paged_row(a.kv, b, j, a.row_bytes).data;
  float w = 0.f;
  for (int h = 0; h < a.H && p != nullptr; ++h) {
    float q[16], v[16];
    load_query(a, b, h, lane, q);
    const float z = logit(a, a.kv.fmt, p, lane, q, v);
    const float l = a.lse_in[size_t(b) * a.H + h];
    if (l != -INFINITY) w += exp2f(z - l * kLog2e);
  }
  if (lane == 0) a.acc_out[b * a.acc_out_stride + j] = a.decay * a.acc[b * a.acc_stride + j] + w;
}

ListArgs common_args(const void* q, const cskv_paged& kv, const float* sink, float scale, const float* q_rope, int T,
                     int H, void* out, float* lse) {
  ListArgs a = {};
  a.q = static_cast<const uint8_t*>(q);
  a.kv = kv;
  a.row_bytes = static_cast<int>(cskv_row_bytes(kv.fmt, kv.dim));
  a.sink = sink;
  a.scale_log2 = scale * kLog2e;
  a.q_rope = q_rope;
  a.T = T;
  a.H = H;
  a.out = static_cast<uint8_t*>(out);
  a.lse = lse;
  return a;
}

cudaError_t launch_list(const ListArgs& a, cudaStream_t stream) {
  const long long rows = (long long)a.T * a.H;
  list_attn_kernel<<<static_cast<unsigned>((rows + 7) / 8), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t window_attn_workspace_bytes(int, int, int, int, int) { return 0; }
size_t prefix_attn_workspace_bytes(int, int, int, int, int) { return 0; }

cudaError_t launch_window_attn(const void* q, const cskv_paged& rows, int num_reqs, const int32_t* req_of,
                               const int32_t* pos1, int window, int first, int max_ctx, const float* sink, float scale,
                               const float* q_rope, int T, int H, void* out, float* lse, void*, cudaStream_t stream) {
  ListArgs a = common_args(q, rows, sink, scale, q_rope, T, H, out, lse);
  a.req_of = req_of;
  a.pos1 = pos1;
  a.num_reqs = num_reqs;
  a.window = window;
  a.first = first;
  a.max_ctx = max_ctx;
  return launch_list(a, stream);
}

cudaError_t launch_prefix_attn(const void* q, const cskv_paged& kv, const int32_t* n_entries, int n_prefix,
                               int max_entries, const void* swa, int swa_fmt, const int32_t* ctx_len, const float* sink,
                               float scale, const float* q_rope, int B, int H, void* out, float* lse, void*,
                               cudaStream_t stream) {
  ListArgs a = common_args(q, kv, sink, scale, q_rope, B, H, out, lse);
  a.n_entries = n_entries;
  a.n_prefix = n_prefix;
  a.max_entries = max_entries;
  a.swa = static_cast<const uint8_t*>(swa);
  a.swa_fmt = swa_fmt;
  a.swa_row_bytes = static_cast<int>(cskv_row_bytes(swa_fmt, kD));
  a.ctx_len = ctx_len;
  return launch_list(a, stream);
}

cudaError_t launch_attn_weights(const void* q, const cskv_paged& kv, const int32_t* n_entries, int first,
                                int max_entries, float scale, const float* q_rope, const float* lse, int B, int H,
                                float decay, const float* acc, long long acc_stride, float* acc_out,
                                long long acc_out_stride, cudaStream_t stream) {
  if (max_entries <= first) return cudaSuccess;
  ListArgs a = common_args(q, kv, nullptr, scale, q_rope, B, H, nullptr, nullptr);
  a.n_entries = n_entries;
  a.first = first;
  a.max_entries = max_entries;
  a.lse_in = lse;
  a.decay = decay;
  a.acc = acc;
  a.acc_stride = acc_stride;
  a.acc_out = acc_out;
  a.acc_out_stride = acc_out_stride;
  weights_kernel<<<dim3((max_entries + 7) / 8, B), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

unsigned int take_err_list_attn() { return take_dev_err(); }

}  // namespace cskv
