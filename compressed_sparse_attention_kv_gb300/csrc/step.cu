// What a step of new tokens needs before its attention (include/cskvs.h): block tables and slot
// maps from the requests' lengths, the (cos, sin) table of positions on the device, and the
// norms of queries and rows with the rotation and the coding in the same pass.
#include <algorithm>
#include <cmath>

#include "codec.cuh"
#include "internal.h"

namespace cskv {

namespace {

// ---------------------------------------------------------------------------
// cskvs_plan_step.  Three prefix sums over the requests (their new tokens, the pages they need,
// the pages they give back), then every token finds its request among the sums and every new
// page its place in the ring of free pages.  A request that ends gives back the ids of its row that are
// pages: where none was left it has -1, and its row is counted before the sum of what comes back.  Nothing
// is carried between blocks but the sums, so
// a page's place follows from its number alone: the k-th new page of the step is the k-th of the
// ring, and the j-th page given back goes j places behind the ring's last one.  The two stretches
// do not meet, so that blocks read and write the ring without waiting for one another.
// Bound: latency (24 bytes a token; 262,144 tokens of 512 requests take 14.7 us, their 4.5 MB 0.7): the chain of
// loads, barriers and scans of one block, with which the other SMs wait.
// One block does a small step in one launch; beyond that one block makes the sums and a launch of
// many blocks, started meanwhile, the maps (in one launch and in two: 1 request of 1 token 5.3 and
// 6.3 us, 64 of one 7.7 and 9.2, 64 and 256 tokens 8.5 and 9.5, 64 and 1,024 9.0 and 9.5, 256 of one 15.1
// and 10.5).
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kMapThreads = 256;
constexpr int kStaged = 2048;            // requests of a block's tokens that fit into shared memory
constexpr int kMaxLen = 1 << 30;
constexpr int kSmallStep = 256, kSmallBatch = 64;   // tokens and requests of one launch at most

struct PlanRecord {        // of a request
  int tok0;                // its first token
  int ctx;                 // its length before the step
  int first, last;         // its pages before and after the step
  int used, own;           // a request that ends: of its row's places [own, used) the pages are given back
  long long take, give;    // the number of its first new page, and of its first page given back
};
struct PlanHead {
  int tokens;              // new tokens of the step
  int head, count;         // the ring before the step
  int pad;
};

struct PlanArgs {
  const int32_t* ctx_len;
  const int32_t* n_new;
  int B, ratio, T, ring_rows;
  int32_t* table;
  int max_pages;
  const int32_t* shared;
  int32_t* free_pages;
  int capacity;
  const int32_t* state;
  int32_t* state_out;
  int32_t* cu_new;
  int32_t* new_len;
  int32_t* first_row;
  int32_t* n_rows;
  int32_t* req_of;
  int32_t* pos1;
  long long* slot;
  long long* ring_slot;
  PlanHead* head;
  PlanRecord* rec;
};

__device__ __forceinline__ int pages_of(int rows) { return (rows + kPageRows - 1) / kPageRows; }

// Inclusive sums of a block's values; `total` gets the last one.
__device__ __forceinline__ long long block_scan(long long v, long long* part, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += x;
  }
  if (lane == 31) part[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long x = lane < warps ? part[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    part[lane] = x;
  }
  __syncthreads();
  if (warp > 0) v += part[warp - 1];
  *total = part[warps - 1];
  __syncthreads();   // part is used again
  return v;
}

__device__ __forceinline__ int bounded_len(int n) {
  if (n >= 0 && n <= kMaxLen) return n;
  set_err(CSKV_ERR_BOUNDS);
  return n < 0 ? 0 : kMaxLen;
}

// The pages among the places [own, used) of the rows of requests that end in this round: a warp reads 512 places
// of a row at once, 16 bytes a lane; with fewer rows than warps several warps share one.  (262,144 tokens of
// 512 requests, 64 of which end with 512 places on average: 14.7 us, with 4 bytes a lane 19 to 23.)
constexpr int kCountAtOnce = 4;          // 16-byte pieces of a lane
constexpr int kMoveAtOnce = 8;           // places of a lane
struct Ended {
  int thread, own, used;   // of a request that ends: its thread
};
__device__ __forceinline__ int pages_in(const int4& v) {
  return 4 + (v.x >> 31) + (v.y >> 31) + (v.z >> 31) + (v.w >> 31);
}
__device__ void count_pages(const PlanArgs& a, int b0, const Ended* ended, int n, int* pages) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int each = max(1, warps / n), groups = warps / each, part = warp % each;
  for (int e = warp / each; e < n; e += groups) {   // (fewer rows than warps: one each, groups >= n)
    const Ended r = ended[e];
    const int32_t* line = a.table + static_cast<long long>(b0 + r.thread) * a.max_pages;
    // the places before the first 16-byte border, whole pieces, and the places behind the last one
    const int ahead = min(r.used - r.own, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(line + r.own) & 15)) & 15) / 4);
    const int4* piece = reinterpret_cast<const int4*>(line + r.own + ahead);
    const int whole = (r.used - r.own - ahead) / 4, behind = r.own + ahead + 4 * whole;
    int have = 0;
    if (part == 0) {
      if (lane < ahead) have += line[r.own + lane] >= 0;
      if (behind + lane < r.used) have += line[behind + lane] >= 0;
    }
    for (int x = part * (32 * kCountAtOnce) + lane; x < whole; x += each * (32 * kCountAtOnce)) {
      int4 v[kCountAtOnce];
#pragma unroll
      for (int u = 0; u < kCountAtOnce; ++u) v[u] = x + 32 * u < whole ? piece[x + 32 * u] : make_int4(-1, -1, -1, -1);
#pragma unroll
      for (int u = 0; u < kCountAtOnce; ++u) have += pages_in(v[u]);
    }
    have = __reduce_add_sync(0xFFFFFFFFu, have);
    if (lane == 0) atomicAdd(&pages[r.thread], have);
  }
}

// The sums, the lengths and the ring's new state; one block.  first_tokens (shared memory, may be
// null): the requests' first tokens once more.
__device__ void plan_sums(const PlanArgs& a, int* first_tokens) {
  __shared__ long long part[32];
  __shared__ Ended ended[kPlanThreads];
  __shared__ int pages[kPlanThreads], n_ended;
  long long tok = 0, take = 0, give = 0;   // before this round of requests
  int head = a.state != nullptr ? a.state[0] : 0, count = a.state != nullptr ? a.state[1] : 0;
  if (a.state != nullptr && (head < 0 || head >= a.capacity || count < 0 || count > a.capacity)) {
    if (threadIdx.x == 0) set_err(CSKV_ERR_BOUNDS);
    head = head < 0 || head >= a.capacity ? 0 : head;
    count = max(0, min(count, a.capacity));
  }
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    const bool there = b < a.B;
    int ctx = 0, n = 0;
    bool ends = false;
    if (there) {
      ctx = bounded_len(a.ctx_len[b]);
      n = a.n_new[b];
      ends = n < 0;
      n = ends ? 0 : n;
      if (n > kMaxLen - ctx) { set_err(CSKV_ERR_BOUNDS); n = kMaxLen - ctx; }
    }
    pages[threadIdx.x] = 0;
    if (threadIdx.x == 0) n_ended = 0;
    long long total;
    const long long upto = tok + block_scan(n, part, &total);
    const int tok0 = static_cast<int>(min(upto - n, static_cast<long long>(a.T)));
    if (upto > a.T && n > 0) { set_err(CSKV_ERR_BOUNDS); n = min(n, a.T - tok0); }
    tok += total;
    const int len = ends ? 0 : ctx + n;
    const int row0 = ends ? 0 : ctx / a.ratio, row1 = len / a.ratio;
    PlanRecord r;
    r.tok0 = tok0;
    r.ctx = ctx;
    r.first = pages_of(row0);
    r.last = pages_of(row1);
    r.used = ends ? pages_of(ctx / a.ratio) : 0;
    if (a.table != nullptr && max(r.last, r.used) > a.max_pages) {
      set_err(CSKV_ERR_BOUNDS);
      r.first = min(r.first, a.max_pages);
      r.last = min(r.last, a.max_pages);
      r.used = min(r.used, a.max_pages);
    }
    r.own = there && ends && a.shared != nullptr ? max(0, min(a.shared[b], r.used)) : 0;
    const int need = there && a.table != nullptr ? r.last - r.first : 0;
    if (a.table != nullptr && r.used > r.own) ended[atomicAdd(&n_ended, 1)] = Ended{static_cast<int>(threadIdx.x), r.own, r.used};
    r.take = take + block_scan(need, part, &total) - need;
    take += total;
    if (n_ended > 0) {   // (in any order: their counts are their own)
      count_pages(a, b0, ended, n_ended, pages);
      __syncthreads();
    }
    const int back = pages[threadIdx.x];
    r.give = give + block_scan(back, part, &total) - back;
    give += total;
    if (there) {
      a.rec[b] = r;
      a.cu_new[b] = tok0;
      if (first_tokens != nullptr) first_tokens[b] = tok0;
      a.new_len[b] = len;
      a.first_row[b] = row0;
      a.n_rows[b] = row1;
    }
  }
  if (threadIdx.x == 0) {
    const int tokens = static_cast<int>(min(tok, static_cast<long long>(a.T)));
    a.cu_new[a.B] = tokens;
    *a.head = PlanHead{tokens, head, count, 0};
    if (a.table != nullptr) {
      const int taken = static_cast<int>(min(take, static_cast<long long>(count)));
      if (give > a.capacity - count) { set_err(CSKV_ERR_BOUNDS); give = a.capacity - count; }
      a.state_out[0] = static_cast<int>((static_cast<long long>(head) + taken) % a.capacity);
      a.state_out[1] = static_cast<int>(count - taken + give);
      a.state_out[2] = static_cast<int>(min(take - taken, static_cast<long long>(INT32_MAX)));
      a.state_out[3] = 0;
    }
  }
}

// The ring's place k behind its first one (k up to its capacity).
__device__ __forceinline__ int32_t* ring_place(const PlanArgs& a, const PlanHead& h, long long k) {
  const long long at = h.head + k;
  return a.free_pages + (at >= a.capacity ? at - a.capacity : at);
}
// The id of the step's k-th new page, -1: none is left.
__device__ __forceinline__ int new_page(const PlanArgs& a, const PlanHead& h, long long k) {
  return k < h.count ? *ring_place(a, h, k) : -1;
}

// The maps of the tokens of blocks block, block + blocks, ...; staged: shared memory, which holds the
// requests' first tokens already (kWhole) or gets those of the block's tokens.
template <bool kWhole>
__device__ void plan_tokens(const PlanArgs& a, const PlanHead& h, int block, int blocks, int* staged) {
  for (long long base = static_cast<long long>(block) * blockDim.x; base < a.T;
       base += static_cast<long long>(blocks) * blockDim.x) {
    const int i0 = static_cast<int>(base), i = i0 + threadIdx.x;
    // the requests of the block's tokens: [lo, hi], the last ones whose first token is not behind them
    int lo = 0, hi = kWhole ? a.B - 1 : 0;
    bool stage = kWhole;
    if constexpr (!kWhole) {
      const int end = min(i0 + static_cast<int>(blockDim.x), h.tokens) - 1;
      if (i0 < h.tokens) {
#pragma unroll
        for (int side = 0; side < 2; ++side) {   // 32 places at a time; every warp for itself
          const int key = side == 0 ? i0 : end;
          int from = 0, n = a.B;                 // the last b in [from, from + n) with a first token <= key
          while (n > 1) {
            const int step = (n + 31) / 32, at = from + static_cast<int>(threadIdx.x & 31) * step;
            const bool le = at < from + n && a.cu_new[at] <= key;
            const int k = __popc(__ballot_sync(0xFFFFFFFFu, le)) - 1;   // (from itself is one)
            const int next = from + k * step;
            n = min(step, from + n - next);
            from = next;
          }
          (side == 0 ? lo : hi) = from;
        }
      }
      stage = hi - lo < kStaged && hi > lo;
      __syncthreads();   // the tokens before are mapped
      if (stage)
        for (int x = threadIdx.x; x <= hi - lo; x += blockDim.x) staged[x] = a.cu_new[lo + x];
      __syncthreads();
    }
    if (i >= a.T) continue;
    int req = -1, p1 = 0;
    long long slot = -1, ring = -1;
    if (i < h.tokens) {
      int b = lo, n = hi - lo + 1;
      while (n > 1) {
        const int half = n / 2, at = b + half;
        const bool le = (stage ? staged[at - lo] : a.cu_new[at]) <= i;
        b = le ? at : b;
        n = le ? n - half : half;
      }
      const PlanRecord r = a.rec[b];
      const int p = r.ctx + (i - r.tok0), len = a.new_len[b];
      req = b;
      p1 = p + 1;
      if (a.table != nullptr && p1 % a.ratio == 0) {
        const int row = p1 / a.ratio - 1, lp = row / kPageRows;
        int page = -1;
        if (lp < a.max_pages)
          page = lp < r.first ? a.table[static_cast<long long>(b) * a.max_pages + lp] : new_page(a, h, r.take + lp - r.first);
        if (page >= 0) slot = static_cast<long long>(page) * kPageRows + row % kPageRows;
      }
      if (a.ring_rows > 0 && len - p <= a.ring_rows) ring = static_cast<long long>(b) * a.ring_rows + p % a.ring_rows;
    }
    a.req_of[i] = req;
    a.pos1[i] = p1;
    if (a.slot != nullptr) a.slot[i] = slot;
    if (a.ring_slot != nullptr) a.ring_slot[i] = ring;
  }
}

__device__ void plan_pages(const PlanArgs& a, const PlanHead& h, int warp, int warps) {
  if (a.table == nullptr) return;
  const int lane = threadIdx.x & 31;
  for (int b = warp; b < a.B; b += warps) {
    const PlanRecord r = a.rec[b];
    int32_t* line = a.table + static_cast<long long>(b) * a.max_pages;
    for (int lp = r.first + lane; lp < r.last; lp += 32) line[lp] = new_page(a, h, r.take + lp - r.first);
    long long give = r.give;   // the number of the next page
    for (int lp = r.own; lp < r.used; lp += 32 * kMoveAtOnce) {
      int id[kMoveAtOnce];
#pragma unroll
      for (int u = 0; u < kMoveAtOnce; ++u) id[u] = lp + 32 * u + lane < r.used ? line[lp + 32 * u + lane] : -1;
#pragma unroll
      for (int u = 0; u < kMoveAtOnce; ++u) {
        const uint32_t there = __ballot_sync(0xFFFFFFFFu, id[u] >= 0);
        const long long j = give + __popc(there & ((1u << lane) - 1u));
        if (id[u] >= 0 && j < a.capacity - h.count) *ring_place(a, h, h.count + j) = id[u];
        give += __popc(there);
      }
    }
  }
}

template <bool kWhole>   // kWhole: the maps too
__global__ void __launch_bounds__(kPlanThreads) plan_sums_kernel(const __grid_constant__ PlanArgs a) {
  grid_dep_launch();
  if constexpr (kWhole) {
    __shared__ int first_tokens[kSmallBatch];
    plan_sums(a, first_tokens);
    __syncthreads();   // (the records are this block's own writes)
    const PlanHead h = *a.head;
    plan_tokens<true>(a, h, 0, 1, first_tokens);
    plan_pages(a, h, threadIdx.x >> 5, kPlanThreads / 32);
  } else {
    plan_sums(a, nullptr);
  }
}

__global__ void __launch_bounds__(kMapThreads) plan_maps_kernel(const __grid_constant__ PlanArgs a) {
  __shared__ int staged[kStaged];
  grid_dep_wait();
  const PlanHead h = *a.head;
  plan_pages(a, h, (blockIdx.x * kMapThreads + threadIdx.x) >> 5, gridDim.x * (kMapThreads / 32));
  plan_tokens<false>(a, h, blockIdx.x, gridDim.x, staged);
}

// ---------------------------------------------------------------------------
// cskvs_rope_cs.  The angle in turns is position * (f / 2 pi), of which the fraction alone
// matters: a 32-bit position times a 96-bit fraction, kept to 64 bits, is exact to 2^-63 turns at
// any position, in two integer products (double precision has a 64th of the fp32 rate here, and
// its reduction by 2 pi would take most of it).  What is left of the nearest quarter turn, in
// [-1/8, 1/8], becomes two floats; times 2 pi that is the angle t + d, |t| <= pi / 4, and
//   sin = t + (t^3 (-1/6 + t^2/120 - ...) + d),  cos = (1 - t^2/2) + (t^4 (1/24 - ...) - t d + what
// the rounding of 1 - t^2/2 lost): Taylor polynomials to t^11 and t^12 (remainders 7e-12 and
// 1e-12), the error below one ulp of the result.
// Bound: neither memory nor issue slots.  131,071 positions take 12.0 us (their 35 MB 5.2): 58 instructions a warp
// and position, with fp32 operations on two numbers at once, use 53 % of an SM's issue slots while it has
// warps; at each issue as many warps wait for the arithmetic pipes (3.2) as for their positions
// (3.0), 64 % of the warps are there, and of the 7.7 rounds of the grid the last is partly empty.
// ---------------------------------------------------------------------------
constexpr int kRopeThreads = 256;
constexpr int kRopeBlocks = 7;                   // of an SM: all are resident (32 registers a thread, 8 bytes of spills), none waits for a place
constexpr int kRopeAtOnce = kRopeThreads / 16;   // positions of a block at a time: a thread has two pairs

struct RopeArgs {
  cskvs_rope_plan plan;
  const int32_t* pos;
  long long axis_stride;
  int shift, T;
  float* out;
};

// a number below 2^23 as a float: the last bits of 2^23 + n
__device__ __forceinline__ float float23(uint32_t n) { return __uint_as_float(0x4B000000u | n) - 8388608.0f; }

// Two numbers in one register pair, and the fp32 operations on both at once (each rounded as alone).
struct Two {
  float a, b;
};
__device__ __forceinline__ Two both(float x) { return Two{x, x}; }
__device__ __forceinline__ Two mul(const Two& x, const Two& y) {
  Two r;
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(r.a), "=f"(r.b) : "f"(x.a), "f"(x.b), "f"(y.a), "f"(y.b));
  return r;
}
__device__ __forceinline__ Two add(const Two& x, const Two& y) {
  Two r;
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tadd.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(r.a), "=f"(r.b) : "f"(x.a), "f"(x.b), "f"(y.a), "f"(y.b));
  return r;
}
__device__ __forceinline__ Two fma(const Two& x, const Two& y, const Two& z) {
  Two r = z;
  fma2(r.a, r.b, x.a, x.b, y.a, y.b);
  return r;
}
__device__ __forceinline__ Two neg(const Two& x) { return Two{-x.a, -x.b}; }

// (cos, sin) of two angles in turns of 2^64
__device__ __forceinline__ float4 cos_sin_of_turns(const uint64_t (&t)[2]) {
  uint32_t q[2];
  float part[2][3];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint32_t low = static_cast<uint32_t>(t[u]);
    uint32_t high = static_cast<uint32_t>(t[u] >> 32);
    q[u] = (high + 0x20000000u) >> 30;
    high -= q[u] << 30;   // what is left, signed: [-2^61, 2^61) with the low word
    // in three pieces, each a float without rounding (conversions of 64 bits run at a quarter of the
    // rate: 25.5 us instead of 16)
    part[u][0] = __uint_as_float(0x4B400000u + (static_cast<int>(high) >> 14)) - 12582912.0f;
    part[u][1] = float23(__funnelshift_l(low, high, 9) & 0x7FFFFFu);
    part[u][2] = float23(low & 0x7FFFFFu);
  }
  const Two r2 = mul(Two{part[0][0], part[1][0]}, both(0x1p46f)), r1 = mul(Two{part[0][1], part[1][1]}, both(0x1p23f));
  const Two rh = add(r2, r1);
  const Two rl = add(add(r1, neg(add(rh, neg(r2)))), Two{part[0][2], part[1][2]});
  constexpr float kTurn = 0x1.921fb6p-62f, kTurnLow = -0x1.777a5cp-87f;   // 2 pi / 2^64
  const Two x = mul(rh, both(kTurn));
  const Two d = add(fma(rh, both(kTurn), neg(x)), fma(rh, both(kTurnLow), mul(rl, both(kTurn))));
  const Two s = mul(x, x), sl = fma(x, x, neg(s));
  Two p = fma(both(-1.0f / 39916800.0f), s, both(1.0f / 362880.0f));
  p = fma(p, s, both(-1.0f / 5040.0f));
  p = fma(p, s, both(1.0f / 120.0f));
  p = fma(p, s, both(-1.0f / 6.0f));
  const Two sn = add(x, fma(mul(x, s), p, d));
  Two c = fma(both(1.0f / 479001600.0f), s, both(-1.0f / 3628800.0f));
  c = fma(c, s, both(1.0f / 40320.0f));
  c = fma(c, s, both(-1.0f / 720.0f));
  c = fma(c, s, both(1.0f / 24.0f));
  const Two w = fma(both(-0.5f), s, both(1.0f));
  const Two lost = add(fma(both(-0.5f), s, add(both(1.0f), neg(w))), neg(fma(x, d, mul(both(0.5f), sl))));
  const Two cs = add(w, fma(mul(s, s), c, lost));
  float o[4];
  const float cc[2] = {cs.a, cs.b}, ss[2] = {sn.a, sn.b};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float a = (q[u] & 1) ? ss[u] : cc[u], b = (q[u] & 1) ? cc[u] : ss[u];
    o[2 * u] = __uint_as_float(__float_as_uint(a) ^ (((q[u] + 1) & 2) << 30));
    o[2 * u + 1] = __uint_as_float(__float_as_uint(b) ^ ((q[u] & 2) << 30));
  }
  return make_float4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) rope_cs_kernel(const __grid_constant__ RopeArgs a) {
  const int two = threadIdx.x & 15;
  uint64_t speed[2], more[2];   // bits 2^-1 .. 2^-64 of a turn; 2^-33 .. 2^-96
  const int32_t* pos[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint32_t* w = a.plan.speed[2 * two + u];
    speed[u] = static_cast<uint64_t>(w[0]) << 32 | w[1];
    more[u] = static_cast<uint64_t>(w[1]) << 32 | w[2];
    pos[u] = a.pos + a.plan.axis[2 * two + u] * a.axis_stride;
  }
  const int step = gridDim.x * kRopeAtOnce;
  int i = blockIdx.x * kRopeAtOnce + (threadIdx.x >> 4);
  float4* out = reinterpret_cast<float4*>(a.out) + static_cast<long long>(i) * 16 + two;
  int next[2] = {0, 0};
  if (i < a.T) {
    next[0] = __ldg(pos[0] + i);
    next[1] = __ldg(pos[1] + i);
  }
  for (; i < a.T; i += step, out += static_cast<long long>(step) * 16) {
    const int now[2] = {next[0], next[1]};
    if (i + step < a.T) {
      next[0] = __ldg(pos[0] + i + step);
      next[1] = __ldg(pos[1] + i + step);
    }
    uint64_t t[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // position p = low - (p < 0) 2^32, in [-2^32, 2^32)
      const long long p = static_cast<long long>(now[u]) + a.shift;
      const uint32_t low = static_cast<uint32_t>(p);
      t[u] = speed[u] * low + __umulhi(low, static_cast<uint32_t>(more[u])) - (p < 0 ? more[u] : 0);
    }
    *out = cos_sin_of_turns(t);
  }
}

// ---------------------------------------------------------------------------
// cskvs_norm_rope: y = x r w, r = (mean of x^2 + eps)^-1/2, the last 64 dims turned by the
// token's angles; bf16 out, or coded into a page.  The order of the sums is that of the calls that
// norm rows one by one, and products and sums are rounded one at a time, so that the bits
// agree.
// Bound: memory, one read and one write of everything: a warp keeps its heads in registers between
// the sum and the product.  8,192 tokens of 64 heads of 512, 64 of 128 and their rows: 1.36 GB in
// 214 us, 6.3 TB/s, 93 % of a copy; in three resident blocks an SM (two: 228 us; 80 registers, which costs 84 bytes
// of spills a thread), with heads loaded
// and stored as what leaves the cache first (plain: 219 us; 1,037 tokens of 20 heads 10.2 -> 8.7 us).
// ---------------------------------------------------------------------------
constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kMaxNormJobs = 4;
// Heads of 512 dims from which on a warp takes four of them, so that their loads are on their way together: 8 warps
// an SM.  With fewer, warps hide more (one and four a warp, tokens of 80 heads: 1 token 3.2 and 4.0 us, 32
// 3.95 and 4.1, 64 5.2 and 5.0, 512 18.6 and 14.8, 4,096 158 and 112).
constexpr long long kManyHeads = 152 * 32;

struct NormJob {
  const uint8_t* x;
  long long x_stride;   // bytes
  int H, dim, norm, rotate;
  const float* norm_w;
  float eps;
  uint8_t* out;
  long long out_stride;
  cskv_paged cache;
  int row_bytes;
  const long long* slot;
  int per_token;        // warps of a token
};
struct NormArgs {
  NormJob job[kMaxNormJobs];
  long long first[kMaxNormJobs + 1];   // warps of the jobs before
  int njobs;
  int T;
  const float* rope_cs;
};

__device__ __forceinline__ void turn2(float& y0, float& y1, float c, float s) {
  const float z0 = __fsub_rn(__fmul_rn(y0, c), __fmul_rn(y1, s));
  y1 = __fadd_rn(__fmul_rn(y0, s), __fmul_rn(y1, c));
  y0 = z0;
}

// N heads of one token (dim 512) or 4 N (dim 128).  A lane has pieces of 8 neighbouring dims: of a head
// of 512 the pieces lane and lane + 32; of a head of 128 piece lane % 16 of head lane / 16 and of
// head lane / 16 + 2, so that every access of a warp is 512 contiguous bytes.  All of a warp's
// loads are on their way before the first is used.
__device__ __forceinline__ void unpack8(const uint4& v, float (&y)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = bf16lo(u[i]);
    y[2 * i + 1] = bf16hi(u[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
    o[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// neighbours first
__device__ __forceinline__ float squares8(const float (&y)[8]) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __fadd_rn(__fmul_rn(y[2 * i], y[2 * i]), __fmul_rn(y[2 * i + 1], y[2 * i + 1]));
  return __fadd_rn(__fadd_rn(v[0], v[1]), __fadd_rn(v[2], v[3]));
}
__device__ __forceinline__ void scale8(float (&y)[8], float r, const float4& w0, const float4& w1) {
  const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(__fmul_rn(y[i], r), w[i]);
}
__device__ __forceinline__ void turn8(float (&y)[8], const float4& c0, const float4& c1) {
  turn2(y[0], y[1], c0.x, c0.y);
  turn2(y[2], y[3], c0.z, c0.w);
  turn2(y[4], y[5], c1.x, c1.y);
  turn2(y[6], y[7], c1.z, c1.w);
}

template <int D, int N>
__device__ __forceinline__ void norm_heads(const NormArgs& a, const NormJob& j, long long w) {
  constexpr int kLanes = D == 512 ? 32 : 16;            // of a piece of a head
  constexpr int kStep = D == 512 ? 1 : 4;               // heads of two pieces of a warp
  const int lane = threadIdx.x & 31;
  const long long t = w / j.per_token;
  const int h0 = static_cast<int>(w - t * j.per_token) * (N * kStep);
  const int at = (lane & (kLanes - 1)) * 8;             // the first piece's first dim
  const uint8_t* from = j.x + t * j.x_stride;
  uint8_t* to = j.out + t * j.out_stride;
  // piece p of head group n: its head, its byte
  auto head = [&](int n, int p) { return D == 512 ? h0 + n : h0 + 4 * n + 2 * p + lane / 16; };
  auto byte = [&](int n, int p) {
    return (static_cast<long long>(head(n, p)) * D + at + (D == 512 ? 256 * p : 0)) * 2;
  };
  uint4 v[N][2];
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      v[n][p] = make_uint4(0u, 0u, 0u, 0u);
      if (head(n, p) < j.H) v[n][p] = __ldcs(reinterpret_cast<const uint4*>(from + byte(n, p)));
    }
  const bool turn = j.rotate && at >= (D == 512 ? 192 : 64);   // of the last piece (512), of either (128)
  float4 c0 = make_float4(1.f, 0.f, 1.f, 0.f), c1 = c0;
  if (turn) {
    const float4* cs = reinterpret_cast<const float4*>(a.rope_cs + t * 64 + (at - (D == 512 ? 192 : 64)));
    c0 = __ldg(cs);
    c1 = __ldg(cs + 1);
  }
  const float4 one = make_float4(1.f, 1.f, 1.f, 1.f);
  float4 g[2][2] = {{one, one}, {one, one}};
  if (j.norm_w != nullptr) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const float4* wp = reinterpret_cast<const float4*>(j.norm_w + at + (D == 512 ? 256 * p : 0));
      g[p][0] = __ldg(wp);
      g[p][1] = __ldg(wp + 1);
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float y[2][8];
    unpack8(v[n][0], y[0]);
    unpack8(v[n][1], y[1]);
    if (j.norm) {
      float ss[2] = {squares8(y[0]), squares8(y[1])};
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) {
        ss[0] = __fadd_rn(ss[0], __shfl_xor_sync(0xFFFFFFFFu, ss[0], o));
        ss[1] = __fadd_rn(ss[1], __shfl_xor_sync(0xFFFFFFFFu, ss[1], o));
      }
      if (D == 512) ss[0] = ss[1] = __fadd_rn(ss[0], ss[1]);
      // one square root and division for all pieces of a head: lane-wise they are the same numbers
#pragma unroll
      for (int p = 0; p < (D == 512 ? 1 : 2); ++p)
        ss[p] = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss[p], static_cast<float>(D)), j.eps)));
      if (D == 512) ss[1] = ss[0];
      scale8(y[0], ss[0], g[0][0], g[0][1]);
      scale8(y[1], ss[1], g[1][0], g[1][1]);
    }
    if (turn) {
      if (D == 128) turn8(y[0], c0, c1);
      turn8(y[1], c0, c1);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p)
      if (head(n, p) < j.H) __stcs(reinterpret_cast<uint4*>(to + byte(n, p)), pack8(y[p]));
  }
}

// A row of D dims into the cache: a lane has four neighbouring dims of every 128.
template <int D>
__device__ __forceinline__ void norm_row(const NormArgs& a, const NormJob& j, long long t) {
  constexpr int N = D / 128;
  const int lane = threadIdx.x & 31;
  const long long slot = j.slot[t];
  if (slot < 0) return;   // (the whole warp)
  const long long page = slot / kPageRows;
  if (page >= j.cache.num_pages) {
    if (lane == 0) set_err(CSKV_ERR_BOUNDS);
    return;
  }
  const RowPtr dst = page_row(j.cache, page, static_cast<int>(slot % kPageRows), j.row_bytes);
  float4 y[N];
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = load_bf16x4(j.x + t * j.x_stride + (128 * i + 4 * lane) * 2);
  if (j.norm) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = __fadd_rn(__fadd_rn(__fmul_rn(y[i].x, y[i].x), __fmul_rn(y[i].y, y[i].y)),
                       __fadd_rn(__fmul_rn(y[i].z, y[i].z), __fmul_rn(y[i].w, y[i].w)));
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) v[i] = __fadd_rn(v[i], __shfl_xor_sync(0xFFFFFFFFu, v[i], o));
    }
    float ss = v[0];
    if constexpr (N == 4) ss = __fadd_rn(__fadd_rn(v[0], v[1]), __fadd_rn(v[2], v[3]));
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(D)), j.eps)));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float4 w = make_float4(1.f, 1.f, 1.f, 1.f);
      if (j.norm_w != nullptr) w = __ldg(reinterpret_cast<const float4*>(j.norm_w + 128 * i + 4 * lane));
      y[i].x = __fmul_rn(__fmul_rn(y[i].x, r), w.x);
      y[i].y = __fmul_rn(__fmul_rn(y[i].y, r), w.y);
      y[i].z = __fmul_rn(__fmul_rn(y[i].z, r), w.z);
      y[i].w = __fmul_rn(__fmul_rn(y[i].w, r), w.w);
    }
  }
  if (j.rotate && lane >= 16) {   // dims 64 .. 127 of the last 128
    const float4 cs = __ldg(reinterpret_cast<const float4*>(a.rope_cs + t * 64) + (lane - 16));
    turn2(y[N - 1].x, y[N - 1].y, cs.x, cs.y);
    turn2(y[N - 1].z, y[N - 1].w, cs.z, cs.w);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) store_row_values(y[i], 32 * i + lane, j.cache.fmt, D, dst, true);
}

// N: heads of 512 dims a warp has at a time
template <int N>
__global__ void __launch_bounds__(kNormThreads, N == 4 ? 3 : 1) norm_rope_kernel(const __grid_constant__ NormArgs a) {
  const long long w = static_cast<long long>(blockIdx.x) * kNormWarps + (threadIdx.x >> 5);
  int k = 0;
  while (k + 1 < a.njobs && w >= a.first[k + 1]) ++k;
  if (w >= a.first[a.njobs]) return;
  const NormJob& j = a.job[k];
  if (j.slot == nullptr) {
    if (j.dim == 512) norm_heads<512, N>(a, j, w - a.first[k]);
    else norm_heads<128, N>(a, j, w - a.first[k]);
  } else if (j.dim == 512) {
    norm_row<512>(a, j, w - a.first[k]);
  } else {
    norm_row<128>(a, j, w - a.first[k]);
  }
}

inline size_t a256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

size_t plan_step_workspace_bytes(int B) { return 256 + a256(sizeof(PlanRecord) * static_cast<size_t>(B)); }

cudaError_t launch_plan_step(const int32_t* ctx_len, const int32_t* n_new, int B, int ratio, int T, int ring_rows,
                             int32_t* table, int max_pages, const int32_t* shared, int32_t* free_pages, int capacity,
                             const int32_t* state, int32_t* state_out, int32_t* cu_new, int32_t* new_len,
                             int32_t* first_row, int32_t* n_rows, int32_t* req_of, int32_t* pos1, int64_t* slot,
                             int64_t* ring_slot, void* workspace, cudaStream_t stream) {
  PlanArgs a = {};
  a.ctx_len = ctx_len;
  a.n_new = n_new;
  a.B = B;
  a.ratio = ratio;
  a.T = T;
  a.ring_rows = ring_slot != nullptr ? ring_rows : 0;
  a.table = table;
  a.max_pages = max_pages;
  a.shared = shared;
  a.free_pages = free_pages;
  a.capacity = capacity;
  a.state = table != nullptr ? state : nullptr;
  a.state_out = state_out;
  a.cu_new = cu_new;
  a.new_len = new_len;
  a.first_row = first_row;
  a.n_rows = n_rows;
  a.req_of = req_of;
  a.pos1 = pos1;
  a.slot = reinterpret_cast<long long*>(slot);
  a.ring_slot = reinterpret_cast<long long*>(ring_slot);
  a.head = static_cast<PlanHead*>(workspace);
  a.rec = reinterpret_cast<PlanRecord*>(static_cast<uint8_t*>(workspace) + 256);
  const bool whole = T <= kSmallStep && B <= kSmallBatch;
  if (whole) {
    plan_sums_kernel<true><<<1, kPlanThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }
  plan_sums_kernel<false><<<1, kPlanThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int blocks = std::max((T + kMapThreads - 1) / kMapThreads, (B + kMapThreads / 32 - 1) / (kMapThreads / 32));
  cfg.gridDim = dim3(static_cast<unsigned>(std::min(std::max(blocks, 1), 152 * 8)));
  cfg.blockDim = dim3(kMapThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_maps_kernel, a);
}

cudaError_t launch_rope_cs(const cskvs_rope_plan& plan, const int32_t* pos, int64_t axis_stride, int shift, int T,
                           float* out, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  RopeArgs a;
  a.plan = plan;
  a.pos = pos;
  a.axis_stride = axis_stride;
  a.shift = shift;
  a.T = T;
  a.out = out;
  const int blocks = std::min((T + kRopeAtOnce - 1) / kRopeAtOnce, 152 * kRopeBlocks);
  rope_cs_kernel<<<blocks, kRopeThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_norm_rope(const cskvs_norm_job* jobs, int njobs, const float* rope_cs, int T, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  NormArgs a = {};
  a.njobs = njobs;
  a.T = T;
  a.rope_cs = rope_cs;
  long long heads = 0;
  for (int i = 0; i < njobs; ++i)
    if (jobs[i].slot == nullptr) heads += static_cast<long long>(T) * jobs[i].H * jobs[i].dim / 512;
  const int n = heads >= kManyHeads ? 4 : 1;
  for (int i = 0; i < njobs; ++i) {
    const cskvs_norm_job& s = jobs[i];
    NormJob& j = a.job[i];
    j.x = static_cast<const uint8_t*>(s.x);
    j.x_stride = s.x_stride * 2;
    j.H = s.H;
    j.dim = s.dim;
    j.norm = s.norm != 0;
    j.norm_w = s.norm_w;
    j.eps = s.eps;
    j.rotate = s.rotate != 0;
    j.slot = reinterpret_cast<const long long*>(s.slot);
    j.per_token = 1;
    if (s.slot != nullptr) {
      j.cache = s.cache;
      j.row_bytes = static_cast<int>(cskv_row_bytes(s.cache.fmt, s.cache.dim));
    } else {
      j.out = static_cast<uint8_t*>(s.out);
      j.out_stride = s.out_stride * 2;
      const int step = s.dim == 512 ? n : 4 * n;
      j.per_token = (s.H + step - 1) / step;
    }
    a.first[i + 1] = a.first[i] + static_cast<long long>(T) * j.per_token;
  }
  const long long blocks = (a.first[njobs] + kNormWarps - 1) / kNormWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  if (n == 4) norm_rope_kernel<4><<<static_cast<unsigned>(blocks), kNormThreads, 0, stream>>>(a);
  else norm_rope_kernel<1><<<static_cast<unsigned>(blocks), kNormThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

unsigned int take_err_step() { return take_dev_err(); }

}  // namespace cskv
