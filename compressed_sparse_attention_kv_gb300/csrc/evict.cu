// Eviction of cache entries by accumulated attention weight (cskvx_evict).
//
// Per request: the m-th largest key, m the budget (order-preserving 32-bit keys of the
// weights, protected entries above every weight), by a radix select of three digits
// (11 + 11 + 10 bits); ties go to the lower slot; then an ordered pass pairs the given-up
// slots below m (holes) with the kept slots from m on (movers), both ascending; then the
// movers' rows are copied into the holes.  A mover's slot is at least m and a hole's below m,
// so no copy reads what another one writes, and the order of the copies does not matter.
//
// What it needs: a weight and an age read per entry (8 bytes) and two row copies per evicted
// entry of the head; the selection is latency-bound (a request's 65,536 entries are 0.5 MB),
// the copies are bound by HBM.
//
// A request is selected by one cluster of 1, 2, 4 or 8 blocks, each with a slice of the
// entries whose keys it keeps in shared memory (a slice too large for it is read again, from
// L2, for every digit).  Histograms of the blocks are added up through distributed shared
// memory; every block takes the same decision.  Warps walk contiguous stretches with
// ballots, so that ranks need one scan over the warps' counts.  Few pairs are copied by the
// cluster itself; many by a second kernel
// over the whole device.  The counts of kept entries on either side of slot m give every warp
// its place in both lists in one exchange between the blocks.
//
// Measured: 8 requests of 65,536 entries cut to half (1 KB rows) 78 us, 29 of them the
// selection and 48 the copies (5.7 TB/s); 32 requests of 4,160 cut by a page 16 us, one
// request of 333 entries 12 us, both the chain of barriers and memory latencies of a selection.
#include <algorithm>

#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace cskv {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
// Entries per block before a request takes another block: 65,536 entries took 112 us in one block
// and 30 in eight, 16,384 took 26 in one and 20 in four; 4,096 took 15 in one and 18 in four.
constexpr int kSliceTarget = 4096;
// Entries of a slice whose keys fit in shared memory (4 requests of 65,536: 49 us, read again for
// every digit 56).
constexpr int kKeysInSmem = 48 * 1024;
// Pairs that the selecting cluster copies itself: 64, 512 and 1,024 pairs of one request took 16, 20
// and 25 us, by a second kernel 19 each; of 32 requests 17, 21 and 27 us, by a second kernel 20, 22 and 26.
constexpr int kFusedPairs = 512;

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
  int max_pairs, fused, cached;
};

__host__ __device__ inline size_t a256(size_t x) { return (x + 255) & ~size_t(255); }

// Larger weight, larger key: the float's bits made order-preserving, NaN lowest, -0 as
// +0; 0xFFFFFFFF (above +inf's key) is a protected entry.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Of a stretch of entries, by slot (below m, from m on): keys above the m-th largest one, and equal to it.
struct Counts {
  int above[2], equal[2];
};

struct SelSmem {
  __align__(16) int hist[2048];
  int sums[kSelWarps];
  Counts warps[kSelWarps];
  Counts total;              // of the slice
  int newest;                // of the slice, then of the request
  int digit, need;
};

// Copies the rows of pair (to, from) of request b in every cache; one warp.
__device__ __forceinline__ void move_pair(const EvictArgs& a, int b, int to, int from, int lane) {
  for (int c = 0; c < a.ncaches; ++c) {
    const cskv_paged& p = a.cache[c];
    const RowPtr d = paged_row(p, b, to, a.row_bytes[c]), s = paged_row(p, b, from, a.row_bytes[c]);
    if (d.data == nullptr || s.data == nullptr) continue;
    const bool split = p.fmt == CSKV_FMT_FP8_E4M3_ROWSCALE_PAGESPLIT || p.fmt == CSKV_FMT_FP4_E2M1_E8M0_HADAMARD_PAGESPLIT;
    const int bytes = split ? a.row_bytes[c] - 4 : a.row_bytes[c];
    if ((bytes & 15) == 0) {   // rows start on 16 bytes then (128 and 64 bytes of page-split codes too)
      uint4 v[2];
      const int n = bytes >> 4;   // at most 64
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (lane + 32 * u < n) v[u] = reinterpret_cast<const uint4*>(s.data)[lane + 32 * u];
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (lane + 32 * u < n) reinterpret_cast<uint4*>(d.data)[lane + 32 * u] = v[u];
    } else {                   // 132 or 72 bytes
      for (int x = lane; x < bytes >> 2; x += 32)
        reinterpret_cast<uint32_t*>(d.data)[x] = reinterpret_cast<const uint32_t*>(s.data)[x];
    }
    if (split && lane == 0) *reinterpret_cast<uint32_t*>(d.scale) = *reinterpret_cast<const uint32_t*>(s.scale);
  }
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint32_t keys[];   // the slice's keys, if they fit
  __shared__ SelSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int blocks = cluster.num_blocks(), rank = cluster.block_rank();
  auto sync_all = [&]() {   // a cluster of one block needs its block's barrier only
    if (blocks == 1) __syncthreads();
    else cluster.sync();
  };
  const int b = blockIdx.x / blocks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  // the blocks' slices: contiguous, whole warp stretches of 32
  const int per_warp = (((n + blocks - 1) / blocks + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int slice0 = min(n, rank * per_warp * kSelWarps), slice1 = min(n, (rank + 1) * per_warp * kSelWarps);
  const int w0 = min(slice1, slice0 + warp * per_warp), w1 = min(slice1, w0 + per_warp);
  const bool acc_in_place = a.acc_out == a.acc, age_in_place = a.age_out == a.age;
  int pairs = 0;

  if (n > a.budget) {
    const bool aged = age != nullptr && a.recent > 0;
    const bool cached = a.cached != 0;
    if (tid == 0) sm.newest = INT32_MIN;
    __syncthreads();
    // One pass over the slice: the weights' keys, the newest age, and the tables' entries to where
    // they stay if nothing moves into their slots (movers follow several barriers later).
    int mx = INT32_MIN;
    constexpr int kBatch = 8;   // loads in flight per thread
    for (int i0 = slice0 + tid; i0 < slice1; i0 += kBatch * kSelThreads) {
      float w[kBatch];
      int32_t g[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * kSelThreads;
        w[u] = 0.f;
        g[u] = INT32_MIN;
        if (i < slice1) {
          w[u] = acc[i];
          if (age != nullptr) g[u] = age[i];
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * kSelThreads;
        if (i < slice1 && cached) keys[i - slice0] = weight_key(w[u]);
        if (i < min(m, slice1)) {
          if (!acc_in_place) a.acc_out[b * a.acc_out_stride + i] = w[u];
          if (age != nullptr && !age_in_place) a.age_out[b * a.age_out_stride + i] = g[u];
        }
        mx = max(mx, g[u]);
      }
    }
    if (aged) {   // the newest age of the request
      mx = __reduce_max_sync(0xFFFFFFFFu, mx);
      if (lane == 0) atomicMax(&sm.newest, mx);
      sync_all();
      mx = INT32_MIN;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < blocks) mx = max(mx, *cluster.map_shared_rank(&sm.newest, r));   // (not written again)
    }
    const long long bar = static_cast<long long>(mx) - a.recent;
    auto guarded = [&](int i) { return i < a.fixed || (aged && age[i] > bar); };
    if (cached) {   // (a thread reads back its own keys only)
#pragma unroll 4
      for (int i = slice0 + tid; i < slice1; i += kSelThreads)
        if (guarded(i)) keys[i - slice0] = 0xFFFFFFFFu;
    }
    auto key_of = [&](int i) -> uint32_t {
      return cached ? keys[i - slice0] : guarded(i) ? 0xFFFFFFFFu : weight_key(acc[i]);
    };
    // the m-th largest key, digit by digit from the top
    uint32_t prefix = 0, mask = 0;
    int need = m;
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
      const int bits = d == 2 ? 10 : 11, shift = d == 0 ? 21 : d == 1 ? 10 : 0;
      const int bins = 1 << bits;
      for (int x = tid; x < bins; x += kSelThreads) sm.hist[x] = 0;
      __syncthreads();
#pragma unroll 4
      for (int i = slice0 + tid; i < slice1; i += kSelThreads) {
        const uint32_t k = key_of(i);
        if ((k & mask) == prefix) atomicAdd(&sm.hist[(k >> shift) & (bins - 1)], 1);
      }
      sync_all();
      // this thread's two bins (from the top), over all blocks
      int c[2] = {0, 0};
      if (2 * tid < bins) {
        const int* two = &sm.hist[bins - 2 - 2 * tid];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          if (r < blocks) {
            const int2 x = *reinterpret_cast<const int2*>(cluster.map_shared_rank(two, r));
            c[0] += x.y;
            c[1] += x.x;
          }
        }
      }
      int v = c[0] + c[1];   // inclusive scan over the threads
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += x;
      }
      if (lane == 31) sm.sums[warp] = v;
      __syncthreads();
      int before = 0;
      {
        int x = lane < warp ? sm.sums[lane] : 0;
        before = __reduce_add_sync(0xFFFFFFFFu, x);
      }
      const int upto = before + v, above = upto - c[0] - c[1];
      if (above < need && upto >= need) {   // the digit lies in one of this thread's bins
        const bool second = above + c[0] < need;
        sm.digit = bins - 1 - (2 * tid + (second ? 1 : 0));
        sm.need = need - above - (second ? c[0] : 0);
      }
      sync_all();   // the decision, and every block is done with the histograms
      prefix |= static_cast<uint32_t>(sm.digit) << shift;
      mask |= static_cast<uint32_t>(bins - 1) << shift;
      need = sm.need;
    }
    // keys above `prefix` stay, and the first `need` of those equal to it
    // ---- counts of the warps' stretches
    Counts mine = {};
#pragma unroll 4
    for (int i = w0 + lane; i < w1; i += 32) {
      const uint32_t k = key_of(i);
      const int late = i >= m;
      mine.above[0] += (k > prefix) & !late;
      mine.above[1] += (k > prefix) & late;
      mine.equal[0] += (k == prefix) & !late;
      mine.equal[1] += (k == prefix) & late;
    }
    auto sum_up = [&](Counts& c) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        c.above[u] = __reduce_add_sync(0xFFFFFFFFu, c.above[u]);
        c.equal[u] = __reduce_add_sync(0xFFFFFFFFu, c.equal[u]);
      }
    };
    sum_up(mine);
    if (lane == 0) sm.warps[warp] = mine;
    __syncthreads();
    if (warp == 0) {
      Counts c = sm.warps[lane];
      sum_up(c);
      if (lane == 0) sm.total = c;
    }
    Counts before = lane < warp ? sm.warps[lane] : Counts{};   // of this warp's stretch: the block's, then all
    sum_up(before);
    sync_all();
    Counts all = {};
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      if (r >= blocks) continue;
      const Counts c = *cluster.map_shared_rank(&sm.total, r);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        all.above[u] += c.above[u];
        all.equal[u] += c.equal[u];
        if (r < rank) {
          before.above[u] += c.above[u];
          before.equal[u] += c.equal[u];
        }
      }
    }
    // kept slots before this stretch, below m and from m on: those above, and the first `need` equal ones
    const int ties = before.equal[0] + before.equal[1];
    int h0 = min(w0, m) - (before.above[0] + min(need, before.equal[0]));
    int v0 = before.above[1] + min(max(need - all.equal[0], 0), before.equal[1]);
    pairs = m - (all.above[0] + min(need, all.equal[0]));
    // ---- holes and movers, in order
    int t = ties;
#pragma unroll 1
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t below = (1u << lane) - 1u;
      const uint32_t k = i < w1 ? key_of(i) : 0u;
      const uint32_t eq = __ballot_sync(0xFFFFFFFFu, i < w1 && k == prefix);
      const bool keep = i < w1 && (k > prefix || (k == prefix && t + __popc(eq & below) < need));
      const uint32_t h = __ballot_sync(0xFFFFFFFFu, i < min(m, w1) && !keep), v = __ballot_sync(0xFFFFFFFFu, i >= m && keep);
      if ((h >> lane) & 1u) hole[h0 + __popc(h & below)] = i;
      else if (i < min(m, w1)) src[i] = i;   // keeps its entry
      if ((v >> lane) & 1u) mover[v0 + __popc(v & below)] = i;
      t += __popc(eq);
      h0 += __popc(h);
      v0 += __popc(v);
    }
    __threadfence();
    sync_all();   // the lists are complete, and no block reads another's shared memory any more
  } else {
    for (int i = rank * kSelThreads + tid; i < a.budget; i += blocks * kSelThreads) {
      src[i] = i < n ? i : -1;
      if (i < n && !acc_in_place) a.acc_out[b * a.acc_out_stride + i] = acc[i];
      if (i < n && age != nullptr && !age_in_place) a.age_out[b * a.age_out_stride + i] = age[i];
    }
  }
  // the movers' weights and ages (those of the slots that keep their entry: above, unless in place)
#pragma unroll 2
  for (int i = rank * kSelThreads + tid; i < pairs; i += blocks * kSelThreads) {
    const int to = hole[i], from = mover[i];
    src[to] = from;
    a.acc_out[b * a.acc_out_stride + to] = acc[from];
    if (age != nullptr) a.age_out[b * a.age_out_stride + to] = age[from];
  }
  if (rank == 0 && tid == 0) {
    a.npairs[b] = pairs;
    if (a.n_out != a.n_entries) a.n_out[b] = m;
  }
  if (a.fused) {
    for (int i = rank * kSelWarps + warp; i < pairs; i += blocks * kSelWarps) move_pair(a, b, hole[i], mover[i], lane);
  }
  if (a.n_out == a.n_entries) {   // every block has read n_entries
    sync_all();
    if (rank == 0 && tid == 0) a.n_out[b] = m;
  }
}

// The rows of many pairs: a warp moves four pairs, one after the other.
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  grid_dep_wait();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int np = a.npairs[b];
  const int i0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * 4;
#pragma unroll 1
  for (int i = i0; i < min(i0 + 4, np); ++i)
    move_pair(a, b, a.hole[(long long)b * a.max_pairs + i], a.mover[(long long)b * a.max_pairs + i], lane);
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
  a.fused = a.max_pairs <= kFusedPairs;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.npairs = reinterpret_cast<int32_t*>(w);
  w += a256(size_t(B) * 4);
  a.hole = reinterpret_cast<int32_t*>(w);
  w += a256(size_t(B) * a.max_pairs * 4);
  a.mover = reinterpret_cast<int32_t*>(w);
  int blocks = 1;
  while (blocks < kMaxCluster && static_cast<long long>(blocks) * kSliceTarget < max_entries) blocks *= 2;
  // the largest slice: whole warp stretches of 32
  const int slice = ((((max_entries + blocks - 1) / blocks + kSelWarps - 1) / kSelWarps + 31) & ~31) * kSelWarps;
  a.cached = slice <= kKeysInSmem;
  const size_t smem = a.cached ? size_t(slice) * 4 : 0;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B) * blocks);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = blocks > 1;
  static std::atomic<uint64_t> allowed;
  const cudaError_t e = launch_with_shared_memory(cfg, evict_select_kernel, allowed, kKeysInSmem * 4, a);
  if (e != cudaSuccess || a.max_pairs == 0 || a.fused) return e;
  // starts while the selection ends; waits for it before it reads the pairs
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>((a.max_pairs + 31) / 32), B);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, a);
}

unsigned int take_err_evict() { return take_dev_err(); }

}  // namespace cskv
