// Eviction of cache entries by accumulated attention weight (cskvx_evict).
//
// Per request: the budget-th largest key (protected entries above every weight), by a
// radix select over order-preserving 32-bit keys, ties to the lower slot; then one
// ordered scan that lists the given-up slots below m (holes) and the kept slots from m
// on (movers), pairwise; then the movers' rows are copied into the holes.  A mover's
// slot is at least m and a hole's below m, so no copy reads what another one writes.
#include "common.cuh"
#include "internal.h"

namespace cskv {

namespace {

constexpr int kSelThreads = 1024;

struct EvictArgs {
  cskv_paged cache[4];
  int row_bytes[4];
  int ncaches;
  const float* acc;
  long long acc_stride;
  const int32_t* age;
  long long age_stride;
  const int32_t* n_entries;
  int max_entries, budget, fixed, recent;
  int32_t* src;
  float* acc_out;
  long long acc_out_stride;
  int32_t* age_out;
  long long age_out_stride;
  int32_t* n_out;
  int32_t* npairs;   // [B]
  int32_t* hole;     // [B, max_pairs]
  int32_t* mover;    // [B, max_pairs]
  int max_pairs;
};

__host__ __device__ inline size_t a256(size_t x) { return (x + 255) & ~size_t(255); }

// Larger weight, larger key: the float's bits made order-preserving, NaN lowest, -0 as
// +0; 0xFFFFFFFF (above +inf's key) is a protected entry.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// inclusive scan of one value per thread over the block; *total = the sum
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += x;
  }
  if (lane == 31) warp_sums[w] = v;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) {
    if (i < w) before += warp_sums[i];
    all += warp_sums[i];
  }
  *total = all;
  __syncthreads();
  return v + before;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int warp_sums[32];
  __shared__ int s_newest, s_need;
  __shared__ uint32_t s_prefix;
  const int b = blockIdx.x, tid = threadIdx.x;
  int n = a.n_entries[b];
  if (n < 0 || n > a.max_entries) {
    if (tid == 0) set_err(CSKV_ERR_BOUNDS);
    n = max(0, min(n, a.max_entries));
  }
  const int m = min(n, a.budget);
  const float* acc = a.acc + b * a.acc_stride;
  const int32_t* age = a.age ? a.age + b * a.age_stride : nullptr;
  int32_t* src = a.src + (long long)b * a.budget;
  int32_t* hole = a.hole + (long long)b * a.max_pairs;
  int32_t* mover = a.mover + (long long)b * a.max_pairs;
  if (n <= a.budget) {
    for (int i = tid; i < a.budget; i += blockDim.x) src[i] = i < n ? i : -1;
    if (tid == 0) a.npairs[b] = 0;
  } else {
    // newest age
    if (tid == 0) { s_newest = INT32_MIN; s_prefix = 0; s_need = m; }
    __syncthreads();
    if (age != nullptr && a.recent > 0) {
      int mx = INT32_MIN;
      for (int i = tid; i < n; i += blockDim.x) mx = max(mx, age[i]);
      mx = __reduce_max_sync(0xFFFFFFFFu, mx);
      if ((tid & 31) == 0) atomicMax(&s_newest, mx);
      __syncthreads();
    }
    const long long bar = static_cast<long long>(s_newest) - a.recent;
    auto key_of = [&](int i) -> uint32_t {
      if (i < a.fixed || (age != nullptr && a.recent > 0 && age[i] > bar)) return 0xFFFFFFFFu;
      return weight_key(acc[i]);
    };
    // the m-th largest key, eight bits at a time from the top
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
      const uint32_t prefix = s_prefix;
      for (int i = tid; i < n; i += blockDim.x) {
        const uint32_t k = key_of(i);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int need = s_need, d = 255;
        while (hist[d] < need) need -= hist[d--];
        s_need = need;
        s_prefix = prefix | (static_cast<uint32_t>(d) << shift);
      }
      __syncthreads();
    }
    const uint32_t T = s_prefix;
    const int ties = s_need;   // of the keys equal to T, this many (the lowest slots) stay
    int ties_before = 0, holes = 0, movers = 0;
    for (int i0 = 0; i0 < n; i0 += blockDim.x) {
      const int i = i0 + tid;
      const uint32_t k = i < n ? key_of(i) : 0u;
      int total;
      const int tie = i < n && k == T ? 1 : 0;
      const int tr = block_scan(tie, warp_sums, &total) + ties_before;
      ties_before += total;
      const bool keep = i < n && (k > T || (tie && tr <= ties));
      const int is_hole = i < m && !keep ? 1 : 0;
      const int hr = block_scan(is_hole, warp_sums, &total) + holes;
      holes += total;
      const int is_mover = i >= m && keep ? 1 : 0;
      const int mr = block_scan(is_mover, warp_sums, &total) + movers;
      movers += total;
      if (is_hole) hole[hr - 1] = i;
      else if (i < m) src[i] = i;
      if (is_mover) mover[mr - 1] = i;
    }
    __syncthreads();
    for (int i = tid; i < holes; i += blockDim.x) src[hole[i]] = mover[i];
    if (tid == 0) a.npairs[b] = holes;
  }
  __syncthreads();
  if (tid == 0) a.n_out[b] = m;
  // weights and ages follow their entries; in place only the holes change
  for (int i = tid; i < m; i += blockDim.x) {
    const int s = src[i];
    if (s != i || a.acc_out != a.acc) a.acc_out[b * a.acc_out_stride + i] = acc[s];
    if (age != nullptr && (s != i || a.age_out != a.age)) a.age_out[b * a.age_out_stride + i] = age[s];
  }
}

// one warp per (request, pair): the rows of every cache, 4 bytes a lane
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int np = a.npairs[b];
  for (int i = blockIdx.x * 8 + (threadIdx.x >> 5); i < np; i += gridDim.x * 8) {
    const int to = a.hole[(long long)b * a.max_pairs + i], from = a.mover[(long long)b * a.max_pairs + i];
    for (int c = 0; c < a.ncaches; ++c) {
      const cskv_paged& p = a.cache[c];
      const RowPtr d = paged_row(p, b, to, a.row_bytes[c]), s = paged_row(p, b, from, a.row_bytes[c]);
      if (d.data == nullptr || s.data == nullptr) continue;
      const bool split = p.fmt == CSKV_FMT_FP8_E4M3_ROWSCALE_PAGESPLIT || p.fmt == CSKV_FMT_FP4_E2M1_E8M0_HADAMARD_PAGESPLIT;
      const int words = (split ? a.row_bytes[c] - 4 : a.row_bytes[c]) / 4;
      for (int x = lane; x < words; x += 32)
        reinterpret_cast<uint32_t*>(d.data)[x] = reinterpret_cast<const uint32_t*>(s.data)[x];
      if (split && lane == 0) *reinterpret_cast<uint32_t*>(d.scale) = *reinterpret_cast<const uint32_t*>(s.scale);
    }
  }
}

int max_pairs_of(int max_entries, int budget) {
  const int over = max_entries - budget;
  return over <= 0 ? 0 : (over < budget ? over : budget);
}

}  // namespace

size_t evict_workspace_bytes(int B, int max_entries, int budget) {
  const size_t pairs = max_pairs_of(max_entries, budget);
  return a256(size_t(B) * 4) + 2 * a256(size_t(B) * pairs * 4);
}

cudaError_t launch_evict(const cskv_paged* caches, int ncaches, const float* acc, long long acc_stride,
                         const int32_t* age, long long age_stride, const int32_t* n_entries, int B, int max_entries,
                         int budget, int fixed, int recent, int32_t* src, float* acc_out, long long acc_out_stride,
                         int32_t* age_out, long long age_out_stride, int32_t* n_out, void* workspace,
                         cudaStream_t stream) {
  EvictArgs a = {};
  for (int c = 0; c < ncaches; ++c) {
    a.cache[c] = caches[c];
    a.row_bytes[c] = static_cast<int>(cskv_row_bytes(caches[c].fmt, caches[c].dim));
  }
  a.ncaches = ncaches;
  a.acc = acc;
  a.acc_stride = acc_stride;
  a.age = age;
  a.age_stride = age_stride;
  a.n_entries = n_entries;
  a.max_entries = max_entries;
  a.budget = budget;
  a.fixed = fixed;
  a.recent = recent;
  a.src = src;
  a.acc_out = acc_out;
  a.acc_out_stride = acc_out_stride;
  a.age_out = age_out;
  a.age_out_stride = age_out_stride;
  a.n_out = n_out;
  a.max_pairs = max_pairs_of(max_entries, budget);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.npairs = reinterpret_cast<int32_t*>(w);
  w += a256(size_t(B) * 4);
  a.hole = reinterpret_cast<int32_t*>(w);
  w += a256(size_t(B) * a.max_pairs * 4);
  a.mover = reinterpret_cast<int32_t*>(w);
  evict_select_kernel<<<B, kSelThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.max_pairs == 0) return e;
  const int blocks = (a.max_pairs + 7) / 8;
  evict_move_kernel<<<dim3(blocks, B), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

unsigned int take_err_evict() { return take_dev_err(); }

}  // namespace cskv
