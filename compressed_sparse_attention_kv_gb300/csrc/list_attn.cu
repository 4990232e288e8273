// Attention over sliding windows with first rows, over shared prefixes, and the
// accumulated attention weights (cskvx_window_attn, cskvx_prefix_decode_attn,
// cskvx_attn_weights).
//
// The mathematics.  A key row c_j is key and value of every head.  For a (query, head)
// row r with rotated query q'_r: z_rj = (q'_r . c_j) * scale over the keys the row sees,
// and out_r = rot^-1(sum_j exp(z_rj) c_j / (sum_j exp(z_rj) + exp(sink))).  The keys are
// taken in tiles of 128; a running reference m_r (base 2) stands for the maximum, and
//   l_r <- l_r 2^(m - m') + sum_j 2^(z_rj - m'),  O_r <- O_r 2^(m - m') + sum_j 2^(z_rj - m') c_j
// where m moves only when a logit exceeds it by more than kSlack: until then the weights
// stay below 2^kSlack, and O need not be touched.  Parts of a row's keys that different
// blocks take are joined by attn_join_kernel in a fixed order.
//
// What bounds it.  A tile of 128 keys for 64 rows is 16.8 MFLOP (1.3 us of one SM's tensor core) on
// 67 KB of FP8 rows (1.5 us of an SM's share of HBM, where no other block reads them): either, with
// the dequantisation of the tile (65,536 values) and the softmax of 8,192 logits beside them, which
// take longer than both; short windows are bound by the queries and outputs.
//
// The tiling.  One block holds 64 rows: 64 / H queries of a request (or one query's heads),
// or 64 consecutive (request, head) rows over a shared prefix.  Both products run with the
// keys or the dims as the 128 MMA rows and the 64 query rows as the MMA columns:
//   S^T = K Q^T    (128 keys x 64, K = 512 dims, K-major operands), 64 TMEM columns,
//   O^T += V^T P^T (4 blocks of 128 dims x 64, K = 128 keys, MN-major operands; V is the
//                   same shared-memory tile as K), 4 x 64 TMEM columns,
// since a 512-d fp32 output of 128 rows would take the whole tensor memory.  Few rows need
// no padding to 128.  The tile lives in eight 16 KiB chunks of 64 dims.  Roles:
//   warps 0-15  load and rotate the queries; then for each tile: dequantise the tile's rows
//               exactly to bf16 into the two chunks that four warps share, as soon as the O product
//               has released it (the rows' bytes have been on their way since the tile
//               before); then softmax: a thread has one key and 16 rows, straight from TMEM;
//               P^T to shared memory as bf16; at the end the epilogue;
//   warp 16     one thread issues the MMAs of a chunk as soon as it is full;
//   warp 17     finds what the block's next 64 rows see (their runs of keys) and, a tile or two
//               ahead of the others, looks the addresses of a tile's rows up.
// A block takes one row block after the other (prompts have many more of them than the device
// has SMs): the queries and the first keys of the next one are on their way while the last
// products and the epilogue of this one run.
// Loading and softmax take turns in the same warps: a tile's products wait for both anyway,
// and sixteen warps hide the latency of either better than eight warps for each.
//
// Roundings: the rotated query is kept as hi + lo, two bf16 numbers (the lo part of the 64
// rotated dims is a ninth chunk of Q), so that logits of N(0, 2) and the log-sum-exp are off by
// 2.1e-6 (rms: 1.7e-6 the two numbers, the rest the tensor core's sums; one number 1.2e-3);
// P is rounded to bf16 (2^-8 relative at most, the operand type of the product), and the output
// divided by the sum of the rounded weights, so that the roundings of a few large ones cancel
// (outputs of 237 keys and N(0, 2) logits are off by 1.9e-3 after their own rounding to bf16, by
// 2.1e-3 over the exact sum, up to 2.6e-3 in single requests; plain fp32 1.7e-3; the second sum costs
// a prompt chunk 5 %, 732 us without it); the log-sum-exp has the exact weights' sum; what the
// rounding took from a sum, 2^-8 of it at most, is handed on as bf16 (2^-16 of the sum); partial
// outputs, sums and maxima stay fp32.
//
// Measured: a prompt chunk of 8,192 tokens, 64 heads, a window of 128 and 4 first rows (FP8)
// 768 us; 32 single tokens over 4,160 FP8 keys, 64 heads, 56 us (1.3 TB/s); 64 requests of 64 heads
// over a prefix of 8,192 FP4 entries and 512 of their own 142 us (0.51 PFLOP/s).  A tile takes 3.5
// to 4 us, of which the products are 1.5: its rows' loads, their conversion (about 7,000
// warp instructions), the softmax and the barriers between them follow one another, and one block's
// tile, queries and weights fill the shared memory of an SM.  A row block of one short tile takes 10 us.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "attn.cuh"
#include "internal.h"

namespace cskv {

namespace {

constexpr int kD = 512;
constexpr int kKeys = 128;
constexpr int kRows = 64;
constexpr int kRuns = 32;                // runs of keys of a row block (of one query each at most)
constexpr int kChunk = kKeys * 128;      // bytes of 64 dims of a tile
constexpr int kWorkWarps = 16;
constexpr int kWorkThreads = kWorkWarps * 32;
constexpr int kThreads = kWorkThreads + 64;
constexpr int kWorkBarrier = 1;          // named barrier of warps 0-15
constexpr uint32_t kTmemS = 256;         // TMEM columns: O 0..255, S from here
constexpr float kSlack = 8.0f;           // base 2: weights stay below 2^8

enum Kind { kWindowRows, kPrefixEntries, kOwnEntries, kRing };

struct ListArgs {
  const uint8_t* q;
  cskv_paged kv;
  int row_bytes;
  const float* sink;
  float scale_log2;
  const float* q_rope;
  int T, H;                  // queries (requests) and heads
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
  int balanced;              // the blocks share all requests' tiles evenly
  // the grid's work: row blocks of per-query items, and how often each key list is split
  int group;                 // queries per block (H <= 64)
  int head_blocks, heads_per_block;
  int split, prefix_split, prefix_blocks, own_blocks;
  int prefix_in_own, ring_in_own;   // the prefix, the ring belong to each request's own list
  int rings_only, lead, beside;     // the call's launch for the rings; before it; beside another
  int items;                        // row blocks of the launch
  int q_rows;                       // rows of its largest one, padded to 16
  int prefetch;                     // no other block reads this block's keys: send for them early
  int parts;                 // partial outputs of a row (1: written straight to out)
  float* opart;              // [row][part][512]
  float* ml;                 // [row][part][2]: m (base 2) and l
  float slack;               // kSlack in units of q'.c
  unsigned long long spin;
};

// A stretch of keys that rows of one request share: positions 0 .. f1-1, then base, base+1, ...
struct Run {
  int req, f1, base, nkeys, tile0;
  int q0, q1;                // the block's queries [q0, q1) that belong to it
  int ring;                  // the keys are slots of request req's window ring, not of the cache
  int whole;                 // every row of the block belongs to it
  int min_f, max_lo, min_hi; // over its rows: positions that all of them see
};

struct __align__(16) RowSees {   // position p of run `run` is seen when p < f or lo <= p <= hi;
  int f, lo, hi, run;            // entries: hi = -1, and lo is the number of ring slots
};

struct Item {
  int kind;
  int row_bytes;
  cskv_paged pages;
  const uint8_t* ring;   // rings of all requests, for runs of ring slots
  int n_prefix;          // positions below it are looked up in request 0's row
  int r0, nr;            // rows [r0, r0 + nr) of the [T * H] rows
  int t0, one;           // the first row's query; all rows are that query's
  int split, nsplit;     // this block takes the split-th of nsplit shares of the tiles
  int part;              // its partial output
};

// A row block's work, made by the planning warp.
struct Plan {
  Item item;
  int nruns, begin, nt, nq;          // runs; its tiles [begin, begin + nt); rows padded to 16
  Run runs[kRuns];
  RowSees sees[kRows];
};

struct TileInfo {
  int n, k0, run;                    // keys; key index of the first one within the run
  int plain;                         // every row sees every one of 128 keys
};

struct ListSmem {
  unsigned long long rowp[2][kKeys]; // addresses of a tile's rows (g_zero_row: no such row), by tile parity
  TileInfo info[2];
  Plan plan[2];                      // of the row block at hand and of the next one
  uint64_t full[4], free_[4],        // of a pair of chunk slots; of a block of 128 dims
      bar_s[2], bar_p[2], bar_q[2], plan_full[2], plan_free[2], rows_full[2], rows_free[2], drained;
  uint32_t tmem;
  int abort;
  __align__(16) float m[kRows];      // running reference in units of q'.c, -inf: no key yet
  __align__(16) float limit[kRows];  // a logit above it moves the reference
  __align__(16) float msub[kRows];   // the reference in base 2, 0 for none
  __align__(16) float fac[kRows];
  float part[4][kRows];
  __nv_bfloat16 cut[4][kRows];       // what the rounding of the weights took from the sums
  // rows of tile i that could not be read: bit r & 31 of word [i & 3][r >> 5] (four tiles:
  // weights_kernel's loads run ahead of its weights)
  uint32_t none[4][4];
};

__host__ __device__ inline int tiles_of(long long keys) { return static_cast<int>((keys + kKeys - 1) / kKeys); }

// ---------------------------------------------------------------------------
// small wrappers
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool wait_on(ListSmem* sm, uint64_t* bar, uint32_t parity, unsigned long long limit) {
  const unsigned long long t0 = clock64();
  while (!try_wait_long(bar, parity)) {
    if (*reinterpret_cast<volatile int*>(&sm->abort)) return false;
    if (clock64() - t0 > limit) {   // gave up: every role leaves its loop
      set_err(CSKV_ERR_TIMEOUT);
      *reinterpret_cast<volatile int*>(&sm->abort) = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_bar(ListSmem* sm, uint64_t* bar, uint32_t parity, unsigned long long limit) {
  return try_wait_long(bar, parity) || wait_on(sm, bar, parity, limit);
}
// wait_bar for a whole warp: all lanes take the same decision
__device__ __forceinline__ bool wait_warp(ListSmem* sm, uint64_t* bar, uint32_t parity, unsigned long long limit) {
  return __all_sync(0xFFFFFFFFu, wait_bar(sm, bar, parity, limit)) != 0;
}
// Before the tensor memory is given back: the issuing lane's products are complete (at once,
// unless a wait gave up while some were in flight).
__device__ __forceinline__ void drain_products(ListSmem* sm) {
  mma_commit(&sm->drained);
  mbar_wait(&sm->drained, 0, kDefaultSpinLimit);
}
// The named barrier of the working warps has no limit: every one of them reaches each of its
// uses, because they all take the same loops (a plan is accepted by all or by none, and after a
// wait that gave up they go on through the same tiles without waiting).
__device__ __forceinline__ void work_sync() {
  asm volatile("bar.sync %0, %1;" ::"n"(kWorkBarrier), "n"(kWorkThreads) : "memory");
}
__device__ __forceinline__ bool work_any(bool p) {
  int r;
  asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.s32 a, %1, 0;\n\tbar.red.or.pred b, %2, %3, a;\n\tselp.s32 %0, 1, 0, b;\n\t}"
               : "=r"(r) : "r"(static_cast<int>(p)), "n"(kWorkBarrier), "n"(kWorkThreads) : "memory");
  return r != 0;
}
// Transposing butterfly: of N columns, lanes (32 / N) c to (32 / N) (c + 1) - 1 end with op over the
// warp's lanes of their v[c] (v is spent).
template <int N, class Op>
__device__ __forceinline__ float reduce_columns(float (&v)[N], Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = N / 2; w >= 1; w >>= 1) {
    const int bit = w * (32 / N);
    const bool hi = (lane & bit) != 0;
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const float send = hi ? v[j] : v[j + w];
      const float keep = hi ? v[j + w] : v[j];
      v[j] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, send, bit));
    }
  }
#pragma unroll
  for (int bit = 16 / N; bit >= 1; bit >>= 1) v[0] = op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], bit));
  return v[0];
}
// Adds a warp's rounded weights up: lane k's b[2 q], b[2 q + 1] are key k's bf16 weights of rows 4 q .. 4 q + 3;
// sum[0], sum[1] end with row lane / 4's sums over some of the keys, sum[2], sum[3] with row lane / 4 + 8's.
// A warp-wide product with a matrix that picks the rows apart: rows 4 q + c of the result take the
// elements of class c (the first or second number of b[2 q] or of b[2 q + 1]).  No shuffles, and no
// sums outside the registers.
// (NaN weights, of a row whose sum is NaN anyway, count as 0: the product would spread them.)
__device__ __forceinline__ uint32_t number(uint32_t x) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0u));
  return r;
}
__device__ __forceinline__ void sum_weights(float (&sum)[4], const uint32_t (&b)[4], int half) {
  const int lane = threadIdx.x & 31, c = (lane >> 2) & 3;
  const uint32_t one = (c & 1) != 0 ? 0x3F800000u : 0x00003F80u;
#pragma unroll
  for (int x = 0; x < 2; ++x) {   // q = 2 half + x: rows 4 q + c are rows lane / 4 (+ 8: half 1) of the lanes with lane / 16 == x
    const uint32_t mine = (lane >> 4) == x ? one : 0u, first = c < 2 ? mine : 0u, second = c < 2 ? 0u : mine;
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(sum[0]), "+f"(sum[1]), "+f"(sum[2]), "+f"(sum[3])
        : "r"(half == 0 ? first : 0u), "r"(half == 0 ? 0u : first), "r"(half == 0 ? second : 0u),
          "r"(half == 0 ? 0u : second), "r"(number(b[2 * x])), "r"(number(b[2 * x + 1])));
  }
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void mma_if(uint32_t d, uint64_t da, uint64_t db, uint32_t id, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(da), "l"(db), "r"(id), "r"(add)
      : "memory");
}
// ---------------------------------------------------------------------------
// rows: 16 dims of a row from its bytes to bf16, exactly
// ---------------------------------------------------------------------------
// a lane's share of a row: the codes of 16 dims; and the scales of a row's block of 128 dims
template <int FMT>
struct Raw;
template <>
struct Raw<CSKV_FMT_FP8_E4M3_E8M0_B32> {
  using Codes = uint4;
  using Scales = uint32_t;   // four e8m0
};
template <>
struct Raw<CSKV_FMT_FP4_E2M1_E4M3_B16> {
  using Codes = uint2;
  using Scales = uint2;      // eight e4m3
};
template <>
struct Raw<CSKV_FMT_BF16> {   // copied straight into the chunk
  using Codes = char;
  using Scales = char;
};

// Rows that do not exist read as zeros from here, so that loads and conversions have no branch.
__device__ uint4 g_zero_row[64];

// ---------------------------------------------------------------------------
// a block's work
// ---------------------------------------------------------------------------
__device__ __forceinline__ Item item_of(const ListArgs& a, int x) {
  Item it;
  it.row_bytes = a.row_bytes;
  it.pages = a.kv;
  it.ring = a.swa;
  it.n_prefix = a.pos1 == nullptr && a.prefix_in_own ? a.n_prefix : 0;
  it.split = 0;
  it.nsplit = 1;
  it.part = 0;
  const int rows = a.T * a.H;
  if (a.pos1 != nullptr) {
    it.kind = kWindowRows;
    it.nsplit = a.split;
    it.split = it.part = x % a.split;
    x /= a.split;
  } else if (a.rings_only) {
    it.kind = kRing;
    it.part = a.parts - 1;
    it.row_bytes = a.swa_row_bytes;
  } else if (x < a.prefix_blocks * a.prefix_split) {
    it.kind = kPrefixEntries;
    it.nsplit = a.prefix_split;
    it.split = it.part = x % a.prefix_split;
    it.r0 = x / a.prefix_split * kRows;
    it.nr = min(kRows, rows - it.r0);
    it.t0 = it.r0 / a.H;
    it.one = (it.r0 + it.nr - 1) / a.H == it.t0;
    return it;
  } else {
    x -= a.prefix_blocks * a.prefix_split;
    it.kind = kOwnEntries;
    it.nsplit = a.split;
    it.split = x % a.split;
    it.part = (a.prefix_blocks > 0 ? a.prefix_split : 0) + it.split;
    x /= a.split;
  }
  it.t0 = x * a.group;
  it.one = a.group == 1;
  if (a.head_blocks == 1) {
    it.r0 = it.t0 * a.H;
    it.nr = min(a.group * a.H, rows - it.r0);
  } else {
    const int q = x / a.head_blocks, h0 = (x - q * a.head_blocks) * a.heads_per_block;
    it.t0 = q;
    it.r0 = q * a.H + h0;
    it.nr = min(a.heads_per_block, a.H - h0);
  }
  return it;
}

__device__ __forceinline__ int entries_of(const ListArgs& a, int b) {
  int n = a.n_entries[b];
  if (n < 0 || n > a.max_entries) {
    set_err(CSKV_ERR_BOUNDS);
    n = max(0, min(n, a.max_entries));
  }
  return n;
}

// What the rows of row block x see, and their runs of keys; one warp.
__device__ void make_plan(const ListArgs& a, int x, Plan* pl) {
  const int lane = threadIdx.x & 31;
  const Item it = item_of(a, x);
  const int t0 = it.t0;
  int fmax = -1;
  unsigned fmin = 0xFFFFFFFFu;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = lane + 32 * u;
    RowSees s{0, 0, -1, -1};   // nothing
    if (r < it.nr) {
      const int t = it.one ? t0 : (it.r0 + r) / a.H;
      if (it.kind == kWindowRows) {
        int p1 = a.pos1[t];
        const int req = a.req_of ? a.req_of[t] : t;
        if (p1 > a.max_ctx) { set_err(CSKV_ERR_BOUNDS); p1 = a.max_ctx; }
        if (p1 > 0 && (req < 0 || req >= a.num_reqs)) { set_err(CSKV_ERR_BOUNDS); p1 = 0; }
        if (p1 > 0) s = RowSees{min(a.first, p1), max(0, p1 - a.window), p1 - 1, req};
      } else {
        const int ring = a.swa != nullptr ? max(0, min(a.ctx_len[t], kWindow)) : 0;
        const int n = it.kind == kRing ? 0 : entries_of(a, t);
        s = RowSees{it.kind == kPrefixEntries ? min(n, a.n_prefix) : n, ring, -1, 0};
        fmax = max(fmax, s.f);
        fmin = min(fmin, static_cast<unsigned>(s.f));
      }
    }
    pl->sees[r] = s;   // window: .run holds the request until the runs are built
  }
  fmax = __reduce_max_sync(0xFFFFFFFFu, fmax);
  fmin = __reduce_min_sync(0xFFFFFFFFu, fmin);
  __syncwarp();
  if (lane == 0) {
    int nruns = 0, tiles = 0;
    if (it.kind != kWindowRows) {
      const int from = it.kind == kOwnEntries && !a.prefix_in_own ? a.n_prefix : 0;
      const int req = it.kind == kPrefixEntries ? 0 : t0;
      if (fmax > from && it.kind != kRing) {
        pl->runs[nruns++] = Run{req, 0, from, fmax - from, 0, 0, it.nr, 0, 1, static_cast<int>(fmin), 1, 0};
        tiles = tiles_of(fmax - from);
      }
      const int ring = pl->sees[0].lo;   // one request's rows
      if ((it.kind == kRing || (it.kind == kOwnEntries && a.ring_in_own)) && ring > 0) {
        pl->runs[nruns++] = Run{req, 0, 0, ring, tiles, 0, it.nr, 1, 1, ring, 1, 0};
        ++tiles;
      }
    } else {
      // neighbouring queries of one request at neighbouring positions share a run
      const int nq = it.one ? 1 : (it.r0 + it.nr - 1) / a.H - t0 + 1;
      int q = 0;
      while (q < nq) {
        const RowSees first = pl->sees[q * a.H < it.nr ? q * a.H : 0];
        if (first.run < 0) { ++q; continue; }
        int lo = first.lo, hi = first.hi, f = first.f, last = first.hi;
        int minf = first.f, maxlo = first.lo, minhi = first.hi;
        int e = q + 1;
        for (; e < nq; ++e) {
          const RowSees s = pl->sees[e * a.H];
          if (s.run != first.run || s.hi > last + 64 || s.hi < last - 64) break;
          last = s.hi;
          lo = min(lo, s.lo); hi = max(hi, s.hi); f = max(f, s.f);
          minf = min(minf, s.f); maxlo = max(maxlo, s.lo); minhi = min(minhi, s.hi);
        }
        const int f1 = min(f, lo);        // first rows before the windows; the rest of them lie inside
        pl->runs[nruns++] = Run{first.run, f1, lo, f1 + hi - lo + 1, tiles, q, e, 0, q == 0 && e == nq, minf, maxlo, minhi};
        tiles += tiles_of(f1 + hi - lo + 1);
        q = e;
      }
    }
    pl->item = it;
    pl->nruns = nruns;
    pl->nq = (it.nr + 15) & ~15;
    pl->begin = static_cast<int>(static_cast<long long>(tiles) * it.split / it.nsplit);
    pl->nt = static_cast<int>(static_cast<long long>(tiles) * (it.split + 1) / it.nsplit) - pl->begin;
  }
  __syncwarp();
  if (it.kind == kWindowRows) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = lane + 32 * u;
      int run = -1;
      const int q = it.one ? 0 : (it.r0 + r) / a.H - t0;
      for (int i = 0; i < pl->nruns; ++i)
        if (r < it.nr && q >= pl->runs[i].q0 && q < pl->runs[i].q1) run = i;
      pl->sees[r].run = run;
    }
  }
}

// Walks a block's tiles in order.
struct TileWalk {
  const Plan* pl;
  int run = 0;
  __device__ __forceinline__ explicit TileWalk(const Plan* p) : pl(p) {}
  // key index of the tile's first key within its run, and the number of keys it holds
  __device__ __forceinline__ void seek(int tile, int* k0, int* n) {
    while (run + 1 < pl->nruns && tile >= pl->runs[run + 1].tile0) ++run;
    *k0 = (tile - pl->runs[run].tile0) * kKeys;
    *n = min(kKeys, pl->runs[run].nkeys - *k0);
  }
  __device__ __forceinline__ int position(int key) const {
    const Run& u = pl->runs[run];
    return key < u.f1 ? key : u.base + (key - u.f1);
  }
};

// ---------------------------------------------------------------------------
// loading.  Warps 4m .. 4m + 3 have the dims 128 m .. 128 m + 127 (two chunks, one block of
// the O product) of every tile, 32 rows each; lane l the 16-dim group l & 3 of chunk l / 16 of
// the rows (l / 4) & 3, + 4, ...: an instruction reads 128 bytes of four rows (whole sectors,
// few cache lines), and eight neighbouring lanes store to different banks.  A tile's bytes are
// requested while the tile before it is in its products.  NS chunk slots; the fills of a pair of
// slots wait for its release.
// ---------------------------------------------------------------------------
// Waits until the slots of a block of dims are free for tile g: the block that had them last has
// been used.  (A release barrier per block of dims, not per pair of slots: a wait sees every phase
// of its barrier, so that none is mistaken for another by its parity.)
template <int NS>
__device__ __forceinline__ bool wait_released(ListSmem* sm, int block, int g, unsigned long long spin) {
  constexpr int kAtOnce = NS / 2;   // blocks of dims in the slots
  const int last = (block + 4 - kAtOnce) & 3, tile = block < kAtOnce ? g - 1 : g;   // kAtOnce blocks before it
  return tile < 0 || wait_bar(sm, &sm->free_[last], tile & 1, spin);
}

template <int FMT, int NS>
struct RowLoader {
  ListSmem* sm;
  uint8_t* slot;
  typename Raw<FMT>::Codes raw[2][4];
  typename Raw<FMT>::Scales scales;   // of row row0 + lane
  int block, row0, lane, group;       // group: of 16 dims
  // of the tile requested; -1 for good after a wait that gave up (a later wait might pass by its
  // parity, before there are addresses)
  int keys = 0;

  __device__ __forceinline__ RowLoader(ListSmem* s, uint8_t* slots) : sm(s) {
    const int warp = threadIdx.x >> 5;
    block = warp >> 2;
    row0 = 32 * (warp & 3);
    lane = threadIdx.x & 31;
    slot = slots + (2 * block % NS + (lane >> 4)) * kChunk + (row0 + ((lane >> 2) & 3)) * 128;
    group = 8 * block + 4 * (lane >> 4) + (lane & 3);
  }
  __device__ __forceinline__ const uint8_t* row_of(int g, int j, int u) const {
    return reinterpret_cast<const uint8_t*>(sm->rowp[g & 1][row0 + 16 * j + 4 * u + ((lane >> 2) & 3)]);
  }
  __device__ __forceinline__ void load(int g, int j) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint8_t* from = row_of(g, j, u);
      if constexpr (FMT == CSKV_FMT_BF16) {   // the block's 256 bytes of the row: into L2, until the chunks are free
        if ((lane & 3) == 0) prefetch_l2(from + 32 * group);
      } else {
        using C = typename Raw<FMT>::Codes;
        raw[j][u] = __ldg(reinterpret_cast<const C*>(from) + group);
      }
    }
  }
  __device__ __forceinline__ void store(int g, int j) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = 16 * j + 4 * u, src = r + ((lane >> 2) & 3);   // of the warp's 32 rows
      const int swz = src & 7, c = 2 * (lane & 3);                // row0 is a multiple of 8
      uint8_t* first = slot + r * 128 + ((c ^ swz) << 4);
      uint8_t* second = slot + r * 128 + (((c + 1) ^ swz) << 4);
      if constexpr (FMT == CSKV_FMT_BF16) {
        const uint8_t* from = row_of(g, j, u) + 32 * group;
        cp_async16(first, from);
        cp_async16(second, from + 16);
      } else {
        uint32_t scale, w[8];
        if constexpr (FMT == CSKV_FMT_FP8_E4M3_E8M0_B32) {
          scale = byte_of(__shfl_sync(0xFFFFFFFFu, scales, src), (group >> 1) & 3);
        } else {
          const uint32_t s0 = __shfl_sync(0xFFFFFFFFu, scales.x, src), s1 = __shfl_sync(0xFFFFFFFFu, scales.y, src);
          scale = byte_of((lane & 16) ? s1 : s0, lane & 3);
        }
        convert(raw[j][u], scale, w);
        *reinterpret_cast<uint4*>(first) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(second) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  }
  // requests the bytes of the block's tile g, whose addresses have been looked up
  __device__ __forceinline__ bool request(int g, unsigned long long spin) {
    const bool ok = keys >= 0 && wait_warp(sm, &sm->rows_full[g & 1], (g >> 1) & 1, spin);
    keys = ok ? sm->info[g & 1].n : -1;
    if (row0 >= keys) return ok;   // none of this warp's rows
    const uint8_t* x = reinterpret_cast<const uint8_t*>(sm->rowp[g & 1][row0 + lane]);
    if constexpr (FMT == CSKV_FMT_FP8_E4M3_E8M0_B32) scales = __ldg(reinterpret_cast<const uint32_t*>(x + kD) + block);
    if constexpr (FMT == CSKV_FMT_FP4_E2M1_E4M3_B16) scales = __ldg(reinterpret_cast<const uint2*>(x + kD / 2) + block);
    load(g, 0);
    load(g, 1);
    return ok;
  }
  // the tile's rows into the chunks once they are free
  __device__ __forceinline__ bool fill(int g, unsigned long long spin) {
    const bool ok = wait_released<NS>(sm, block, g, spin);
    __syncwarp();
    if (row0 < keys) {   // (rows behind the last key: zeros up to this warp's 32, beyond them nothing is read)
      store(g, 0);
      store(g, 1);
    }
    if (FMT == CSKV_FMT_BF16) cp_async_wait_all();
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm->full[block % (NS / 2)]);
    return ok;
  }
};

// Tile `tile` of a plan, the block's tile g: looks its rows up in the block table and hands their
// addresses on, once the tile two before it has been used; one warp.
__device__ __forceinline__ bool look_up_tile(const ListArgs& a, ListSmem* sm, const Plan* pl, TileWalk& walk, int tile,
                                             int g) {
  const int lane = threadIdx.x & 31;
  const Item& it = pl->item;
  int k0, n;
  walk.seek(tile, &k0, &n);
  const Run& u = pl->runs[walk.run];
  int row[4], page[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = 32 * j + lane;
    row[j] = page[j] = -1;
    if (r < n) {
      row[j] = walk.position(k0 + r);
      page[j] = row[j] / kPageRows;
      if (!u.ring && it.pages.block_table != nullptr) {
        const int req = row[j] < it.n_prefix ? 0 : u.req;
        page[j] = page[j] < it.pages.max_pages
                      ? __ldg(it.pages.block_table + static_cast<long long>(req) * it.pages.max_pages + page[j]) : -1;
      }
    }
  }
  const uint8_t* x[4];
  uint32_t none[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[j] = reinterpret_cast<const uint8_t*>(g_zero_row);
    bool bad = false;
    if (row[j] >= 0) {
      if (u.ring) x[j] = it.ring + (static_cast<long long>(u.req) * kWindow + row[j]) * it.row_bytes;
      else if (page[j] >= 0 && page[j] < it.pages.num_pages)
        x[j] = page_row(it.pages, page[j], row[j] % kPageRows, it.row_bytes).data;
      else bad = true;
    }
    if (bad) set_err(CSKV_ERR_BOUNDS);
    none[j] = __ballot_sync(0xFFFFFFFFu, bad);
  }
  if (a.prefetch) {   // into L2, until the loading warps have registers for them
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (row[j] >= 0)
        for (int o = 0; o < it.row_bytes; o += 128) prefetch_l2(x[j] + o);
  }
  // all 128 keys seen by all rows: inside every window, or all first rows
  const int pa = walk.position(k0), pb = walk.position(k0 + n - 1);
  const int plain = u.whole && n == kKeys && (none[0] | none[1] | none[2] | none[3]) == 0u &&
                    ((pb < u.min_f) || (pa >= u.max_lo && pb <= u.min_hi && pb - pa == kKeys - 1));
  if (g >= 2 && !wait_warp(sm, &sm->rows_free[g & 1], ((g >> 1) - 1) & 1, a.spin)) return false;
#pragma unroll
  for (int j = 0; j < 4; ++j) sm->rowp[g & 1][32 * j + lane] = reinterpret_cast<unsigned long long>(x[j]);
  if (lane < 4) sm->none[g & 3][lane] = lane == 0 ? none[0] : lane == 1 ? none[1] : lane == 2 ? none[2] : none[3];
  if (lane == 0) sm->info[g & 1] = TileInfo{n, k0, walk.run, plain};
  __syncwarp();
  if (lane == 0) mbar_arrive(&sm->rows_full[g & 1]);
  return true;
}

// The block's query rows into the K-major chunks of Q (rows nq apart); warps 0-15.  The rows
// come in by asynchronous copies; the last 64 dims are then rotated in place, chunk 8 holds
// the second bf16 of each rotated value.
__device__ __forceinline__ void request_queries(const ListArgs& a, int r0, int nr, int nq, uint8_t* qtile) {
  const uint8_t* q = a.q + static_cast<size_t>(r0) * kD * 2;
#pragma unroll 1
  for (int x = threadIdx.x; x < nq * 64; x += kWorkThreads) {
    const int r = x >> 6, c = x & 63;   // dims 8c .. 8c + 7
    uint8_t* dst = qtile + (c >> 3) * (nq * 128) + sw128_offset(r, c & 7);
    if (r < nr) cp_async16(dst, q + static_cast<size_t>(x) * 16);
    else *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
  }
}
// kTerms: bf16 numbers that a rotated value is kept as (the third one in chunk 9).
template <int kTerms>
__device__ __forceinline__ void rotate_queries(const ListArgs& a, int r0, int nr, int nq, uint8_t* qtile) {
  static_assert(kRows * 8 <= kWorkThreads, "a thread per 8 dims of 64 rows, two passes for 128");
#pragma unroll 1
  for (int x = threadIdx.x; x - static_cast<int>(threadIdx.x) < nq * 8; x += kWorkThreads) {
    const int r = x >> 3, c = x & 7;
    float4 t0 = make_float4(1.f, 0.f, 1.f, 0.f), t1 = t0;
    if (r < nr) {   // on their way while the queries are awaited
      const float* cs = a.q_rope + static_cast<size_t>(static_cast<unsigned>(r0 + r) / static_cast<unsigned>(a.H)) * 64 + c * 8;
      t0 = __ldg(reinterpret_cast<const float4*>(cs));
      t1 = __ldg(reinterpret_cast<const float4*>(cs + 4));
    }
    if (x < kWorkThreads) {
      cp_async_wait_all();
      work_sync();
    }
    if (r < nq) {
      uint4* hi = reinterpret_cast<uint4*>(qtile + 7 * (nq * 128) + sw128_offset(r, c));
      uint4 v = *hi, lo = make_uint4(0u, 0u, 0u, 0u), rest = lo;
      if (r < nr) {
        const float co[4] = {t0.x, t0.z, t1.x, t1.z}, si[4] = {t0.y, t0.w, t1.y, t1.w};
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
        uint32_t* l = reinterpret_cast<uint32_t*>(&lo);
        uint32_t* e = reinterpret_cast<uint32_t*>(&rest);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float y0 = bf16lo(w[k]), y1 = bf16hi(w[k]);
          const float z0 = y0 * co[k] - y1 * si[k], z1 = y0 * si[k] + y1 * co[k];
          w[k] = pack_bf16(z0, z1);
          const float l0 = z0 - bf16lo(w[k]), l1 = z1 - bf16hi(w[k]);   // (exact)
          l[k] = pack_bf16(l0, l1);
          if (kTerms == 3) e[k] = pack_bf16(l0 - bf16lo(l[k]), l1 - bf16hi(l[k]));
        }
        *hi = v;
      }
      *reinterpret_cast<uint4*>(qtile + 8 * (nq * 128) + sw128_offset(r, c)) = lo;
      if (kTerms == 3) *reinterpret_cast<uint4*>(qtile + 9 * (nq * 128) + sw128_offset(r, c)) = rest;
    }
  }
  fence_proxy_async_smem();
}

// S^T of chunk c: 128 keys x nq rows (TMEM d), K = 64 dims; dk, dq: the chunk's descriptors,
// dl: those of the query's second halves, on the same keys' rotated dims
__device__ __forceinline__ void issue_s_chunk(uint32_t d, uint64_t dk, uint64_t dq, uint64_t dl, int c, uint32_t id) {
  if (c == 0) mma_set(d, dk, dq, id);
  else mma_add(d, dk, dq, id);
#pragma unroll
  for (int k = 1; k < 4; ++k) mma_add(d, dk + 2 * k, dq + 2 * k, id);
  if (c == 7) {
#pragma unroll
    for (int k = 0; k < 4; ++k) mma_add(d, dk + 2 * k, dl + 2 * k, id);
  }
}

// For the weights, which are fp32: block m of 128 dims (chunks 2m, 2m + 1; dk, dq: its first chunk's
// descriptors) into a sum of its own, or on top of the block before it (`add`).  The tensor core
// cuts the low bits off at every step, so short sums are more exact, and the small terms of the
// rotated dims (dl: the query's second and third) come before the large ones.
__device__ __forceinline__ void issue_s_block(uint32_t d, uint64_t dk, uint64_t dq, uint64_t dl, uint32_t qstep, int m,
                                              uint32_t add, uint32_t id) {
  if (m == 3) {
    mma_if(d, dk + (kChunk >> 4), dl + qstep, id, add);
#pragma unroll
    for (int k = 1; k < 8; ++k) mma_add(d, dk + (kChunk >> 4) + 2 * (k & 3), dl + (k < 4 ? qstep : 0u) + 2 * (k & 3), id);
    mma_add(d, dk, dq, id);
  } else {
    mma_if(d, dk, dq, id, add);
  }
#pragma unroll
  for (int k = 1; k < 4; ++k) mma_add(d, dk + 2 * k, dq + 2 * k, id);
#pragma unroll
  for (int k = 0; k < 4; ++k) mma_add(d, dk + (kChunk >> 4) + 2 * k, dq + qstep + 2 * k, id);
}

// ---------------------------------------------------------------------------
// the attention kernel
// ---------------------------------------------------------------------------
// Bits [0, n) of a word, for n of any size.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// Which of a warp's 32 rows see which of its 32 keys: the lane with column c makes row cb + c's
// bits over the keys k0 .. k0 + 31 of the run (the seen positions are at most three stretches
// of key indices), then the 32 x 32 bit matrix is transposed; lane k ends with key k0 + k's
// bits over the rows.  (16 rows: lanes c and c + 16 make the same row's bits.)
__device__ __forceinline__ uint32_t seen_by(const Plan* pl, int run, int k0, int col) {
  const int lane = threadIdx.x & 31;
  const RowSees s = pl->sees[col];
  const Run& u = pl->runs[run];
  uint32_t x = 0;
  if (u.ring) {
    x = s.run >= 0 ? low_bits(s.lo - k0) : 0u;
  } else if (s.run == run) {
    const int shift = u.f1 - u.base - k0;   // bit of a position in the second stretch
    const uint32_t second = ~low_bits(u.f1 - k0);
    x = low_bits(min(s.f, u.f1) - k0);
    x |= second & low_bits(s.f + shift);
    x |= second & low_bits(s.hi + 1 + shift) & ~low_bits(s.lo + shift);
  }
#pragma unroll
  for (int j = 16; j >= 1; j >>= 1) {
    const uint32_t m = j == 16 ? 0x0000FFFFu : j == 8 ? 0x00FF00FFu : j == 4 ? 0x0F0F0F0Fu : j == 2 ? 0x33333333u : 0x55555555u;
    const uint32_t y = __shfl_xor_sync(0xFFFFFFFFu, x, j);
    x = (lane & j) ? (x & ~m) | ((y & ~m) >> j) : (x & m) | ((y & m) << j);
  }
  return x;
}

// A key row with a value that is not finite makes every logit of its key not finite, so one
// column is looked at, and only then the row.  Such a row leaves the tile (zeros, for the O
// product) and the key's logits become NaN.
__device__ __forceinline__ bool unfit_row(const uint8_t* ktile, int key) {
  uint32_t bad = 0;
#pragma unroll 1
  for (int x = 0; x < 64; ++x) {
    const uint4 v = *reinterpret_cast<const uint4*>(ktile + (x >> 3) * kChunk + sw128_offset(key, x & 7));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    // an exponent of all ones carries into the sign bit when its lowest bit is added
    for (int i = 0; i < 4; ++i) bad |= ((w[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
  }
  return bad != 0u;
}
__device__ __forceinline__ void clear_row(uint8_t* ktile, int key) {
#pragma unroll 1
  for (int x = 0; x < 64; ++x)
    *reinterpret_cast<uint4*>(ktile + (x >> 3) * kChunk + sw128_offset(key, x & 7)) = make_uint4(0u, 0u, 0u, 0u);
}

// The softmax of the block's tile g (`first`: no tile of these rows before it): l accumulates the warp's keys' weights of row cb + lane / 2.
__device__ __forceinline__ bool weigh_tile(const ListArgs& a, const Plan* pl, ListSmem* sm, uint8_t* ktile,
                                           uint8_t* ptile, uint32_t tmem, int g, bool first, float& l, float (&hat)[4]) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quarter = warp & 3, group = warp >> 2;
  const int cb = group * 16;        // this thread's rows (columns of S^T)
  const int nq = pl->nq;
  const int key = quarter * 32 + lane;
  const uint32_t tlane = static_cast<uint32_t>(quarter * 32) << 16;
  const TileInfo t = sm->info[g & 1];
  const int n = t.n;
  // whether the warp has rows and keys: a short tile's weights behind its last key are not read
  const bool rows = cb < nq, has = rows && quarter * 32 < n;
  uint32_t bits = 0xFFFFu;
  if (t.plain == 0 && has) {   // before S is complete
    bits = seen_by(pl, t.run, t.k0 + quarter * 32, cb + (lane & 15));
    if (key >= n || ((sm->none[g & 3][quarter] >> lane) & 1u) != 0u) bits = 0u;
  }
  const bool ok = wait_bar(sm, &sm->bar_s[0], g & 1, a.spin);
  __syncwarp();
  tc_fence_after();
  float z[16];
  if (has) {
    tmem_ld16(tmem + kTmemS + tlane + cb, z);
    tmem_wait_ld();
  }
  bool unfit = false;
  if (has && key < n && !(fabsf(z[0]) < INFINITY)) {
    unfit = unfit_row(ktile, key);
#pragma unroll
    for (int c = 0; c < 16; ++c)
      if (unfit) z[c] = __int_as_float(0x7FC00000);
  }
  __syncwarp();
  if (t.plain == 0) {
#pragma unroll
    for (int c = 0; c < 16; ++c)
      if (((bits >> c) & 1u) == 0u) z[c] = -INFINITY;
  }
  bool above = false;
  if (has) {
#pragma unroll
    for (int c = 0; c < 16; c += 4) {
      const float4 m = *reinterpret_cast<const float4*>(&sm->limit[cb + c]);
      above |= (z[c] > m.x) | (z[c + 1] > m.y) | (z[c + 2] > m.z) | (z[c + 3] > m.w);
    }
  }
  const bool moves = work_any(above);
  if (unfit && group == 0) clear_row(ktile, key);   // every group has looked at it
  if (moves) {   // some row's reference moves: the tile's maxima, exactly
    if (has) {
#pragma unroll
      for (int h = 0; h < 16; h += 8) {   // (in halves: registers)
        float t[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) t[c] = z[h + c];
        const float mine = reduce_columns(t, [](float x, float y) { return fmaxf(x, y); });
        if ((lane & 3) == 0) sm->part[quarter][cb + h + (lane >> 2)] = mine;
      }
    } else if (rows && lane < 16) {
      sm->part[quarter][cb + lane] = -INFINITY;
    }
    work_sync();
    if (tid < nq) {
      const float old = sm->m[tid], old_sub = sm->msub[tid];
      const float now = fmaxf(fmaxf(fmaxf(sm->part[0][tid], sm->part[1][tid]), fmaxf(sm->part[2][tid], sm->part[3][tid])), old);
      const float sub = now == -INFINITY ? 0.f : now * a.scale_log2;
      sm->fac[tid] = old == -INFINITY ? 0.f : exp2f(old_sub - sub);
      sm->m[tid] = now;
      sm->limit[tid] = now + a.slack;
      sm->msub[tid] = sub;
    }
    work_sync();
    if (rows) {
      l *= sm->fac[cb + (lane >> 1)];
#pragma unroll
      for (int c = 0; c < 4; ++c) hat[c] *= sm->fac[cb + (lane >> 2) + 8 * (c >> 1)];
    }
    if (!first) {   // the S commit says that the O products so far are complete
#pragma unroll 1
      for (int r = 0; r < nq; r += 16) {   // this warp's 32 dims of block `group`, 16 rows at a time
        float o[16];
        const uint32_t at = tmem + tlane + group * kRows + r;
        tmem_ld16(at, o);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) o[c] *= sm->fac[r + c];
        tmem_st16(at, o);
      }
      tmem_wait_st();
    }
  }
  if (has) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 m0 = *reinterpret_cast<const float4*>(&sm->msub[cb + 8 * h]);
      const float4 m1 = *reinterpret_cast<const float4*>(&sm->msub[cb + 8 * h + 4]);
      const float mm[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
      for (int c = 0; c < 8; ++c) z[8 * h + c] = exp2_fast(fmaf(z[8 * h + c], a.scale_log2, -mm[c]));
      const float* p = z + 8 * h;
      const uint32_t b[4] = {pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7])};
      *reinterpret_cast<uint4*>(ptile + sw128_offset(key, group * 2 + h)) = make_uint4(b[0], b[1], b[2], b[3]);
      sum_weights(hat, b, h);
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sm->bar_p[0]);
  if (lane == 0) mbar_arrive(&sm->rows_free[g & 1]);
  // while the O product starts: lanes 2c and 2c + 1 keep the sum of the warp's keys for row cb + c
  if (has) l += reduce_columns(z, [](float x, float y) { return x + y; });
  return ok;
}


// The epilogue of a row block, first part (while its last O product runs): the rows' sums, their
// log-sum-exps, and the factors that their outputs take.
__device__ __forceinline__ void finish_sums(const ListArgs& a, const Plan* pl, ListSmem* sm, float l, const float (&hat)[4]) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quarter = warp & 3, cb = (warp >> 2) * 16;
  const Item& it = pl->item;
  const unsigned r = it.r0 + tid;
  float sink = -INFINITY;
  if (a.sink != nullptr && tid < it.nr) sink = __ldg(a.sink + r % static_cast<unsigned>(a.H));
  if (cb < pl->nq) {
    if ((lane & 1) == 0) sm->part[quarter][cb + (lane >> 1)] = l;
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float x = hat[2 * c] + hat[2 * c + 1];
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
      const int row = cb + (lane >> 2) + 8 * c;
      if ((lane & 3) == 0) sm->cut[quarter][row] = __float2bfloat16(sm->part[quarter][row] - x);
    }
  }
  work_sync();
  if (tid < kRows) {
    float f = 0.f;
    if (tid < it.nr) {
      const float sum = ((sm->part[0][tid] + sm->part[1][tid]) + sm->part[2][tid]) + sm->part[3][tid];
      // the output is made of rounded weights: over their own sum a few large ones' roundings cancel
      const float cut = (__bfloat162float(sm->cut[0][tid]) + __bfloat162float(sm->cut[1][tid])) +
                        (__bfloat162float(sm->cut[2][tid]) + __bfloat162float(sm->cut[3][tid]));
      const float ratio = sum == 0.f ? 1.f : sum / (sum - cut);
      const float m = sm->m[tid] == -INFINITY ? -INFINITY : sm->msub[tid];
      if (a.parts > 1) {
        *reinterpret_cast<float2*>(a.ml + (static_cast<size_t>(r) * a.parts + it.part) * 2) = make_float2(m, sum);
        f = ratio;
      } else {
        const float s2 = sink * kLog2e;
        const float M = fmaxf(m, s2);
        const float e = exp2f(m - M);
        const float total = sum * e + (s2 == -INFINITY ? 0.f : exp2f(s2 - M));
        // no key, or a sink above fp32 in base 2 (which leaves the keys nothing): out 0, lse the sink itself
        const bool none = sum == 0.f || s2 == INFINITY;
        f = none ? 0.f : e / total * ratio;
        if (sum != sum) f = sum;
        if (a.lse != nullptr) a.lse[r] = none ? sink : sum != sum ? sum : (M + log2f(total)) * kLn2;
      }
    }
    sm->fac[tid] = f;
    sm->m[tid] = sm->limit[tid] = -INFINITY;   // for the next rows
    sm->msub[tid] = 0.f;
  }
  work_sync();
}

// Second part: O^T out, in units of 8 rows of a block of 128 dims (the next tile's bytes hold
// most registers); a thread has one dim of them,
// a row's 32 dims of a warp are one 64-byte run.  With 64 rows a warp has 16 rows of every
// block, so that the turned dims (twice the instructions) are spread over eight warps.
__device__ __forceinline__ void write_rows(const ListArgs& a, const Plan* pl, ListSmem* sm, uint32_t tmem, int nt) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;
  const int r0 = pl->item.r0, nr = pl->item.nr;
  const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const unsigned H = a.H, t0 = r0 / H;
  const bool one = pl->item.one;   // the rows of one query
  const int sets = (nr + 7) >> 3;
#pragma unroll 1
  for (int x = warp >> 2; x < 4 * sets; x += 4) {
    const int block = x / sets, g = (x - block * sets) * 8;
    const int d = block * 128 + quarter * 32 + lane;
    const bool turn = block == 3 && quarter >= 2 && a.parts == 1;   // dims 448..511, turned back
    const float2* cs = reinterpret_cast<const float2*>(a.q_rope) + ((d - (kD - 64)) >> 1);
    float2 w = make_float2(1.f, 0.f);
    if (turn && one) w = __ldg(cs + static_cast<size_t>(t0) * 32);
    float o[8];
    if (nt > 0) {
      tmem_ld8(from + block * kRows + g, o);   // (columns behind the last row hold nothing of use)
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < 8; c += 4) {
      const float4 f = *reinterpret_cast<const float4*>(&sm->fac[g + c]);   // 0 behind the last row
      o[c] *= f.x;
      o[c + 1] *= f.y;
      o[c + 2] *= f.z;
      o[c + 3] *= f.w;
    }
    if (a.parts > 1) {
      float* to = a.opart + ((static_cast<size_t>(r0) + g) * a.parts + pl->item.part) * kD + d;
      const size_t step = static_cast<size_t>(a.parts) * kD;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (g + c < nr) to[c * step] = o[c];
      continue;
    }
    if (turn) {
      // even lanes turn and store the pair of dims (d, d + 1) of row c, odd lanes (d - 1, d) of row c + 1
      const bool odd = (lane & 1) != 0;
#pragma unroll
      for (int c = 0; c < 8; c += 2) {
        const int r = g + c + (odd ? 1 : 0);
        if (!one) w = __ldg(cs + static_cast<size_t>((r0 + min(r, nr - 1)) / H) * 32);
        const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? o[c] : o[c + 1], 1);
        const float y0 = odd ? other : o[c], y1 = odd ? o[c + 1] : other;
        const uint32_t v = pack_bf16(y0 * w.x + y1 * w.y, y1 * w.x - y0 * w.y);
        if (r < nr)
          *reinterpret_cast<uint32_t*>(a.out + ((static_cast<size_t>(r0) + r) * kD + (d & ~1)) * 2) = v;
      }
      continue;
    }
    uint16_t* to = reinterpret_cast<uint16_t*>(a.out) + (static_cast<size_t>(r0) + g) * kD + d;
#pragma unroll
    for (int c = 0; c < 8; c += 2) {
      const uint32_t v = pack_bf16(o[c], o[c + 1]);
      if (g + c < nr) to[c * kD] = static_cast<uint16_t>(v);
      if (g + c + 1 < nr) to[(c + 1) * kD] = static_cast<uint16_t>(v >> 16);
    }
  }
}

// One kernel per row format: a call whose rings have another format than its cache launches two
// (a block's code stays within its registers and the instruction cache).
template <int FMT>
__global__ void __launch_bounds__(kThreads, 1) list_attn_kernel(const __grid_constant__ ListArgs a) {
  if (a.lead) grid_dep_launch();   // the call's launch for the rings may start
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* ktile = base;                              // 8 chunks of 128 rows x 128 B
  uint8_t* qtile = ktile + 8 * kChunk;                // 9 chunks of nq rows x 128 B
  uint8_t* ptile = qtile + 9 * a.q_rows * 128;        // 128 keys x 128 B
  ListSmem* sm = reinterpret_cast<ListSmem*>(ptile + kChunk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // this block's row blocks: blockIdx.x, + gridDim.x, ...
  const int items = (a.items - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm->full[i], 4);
      mbar_init(&sm->free_[i], 1);
    }
    mbar_init(&sm->bar_s[0], 2);
    mbar_init(&sm->bar_p[0], kWorkWarps);
    mbar_init(&sm->drained, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->bar_q[i], kWorkWarps);
      mbar_init(&sm->plan_full[i], 1);
      mbar_init(&sm->plan_free[i], kWorkWarps + 1);
      mbar_init(&sm->rows_full[i], 1);
      mbar_init(&sm->rows_free[i], kWorkWarps);
    }
    sm->abort = 0;
    sm->info[0] = sm->info[1] = TileInfo{0, 0, 0, 0};   // (what a wait that gave up leaves is never wild)
    fence_mbar_init();
  }
  if (tid < kRows) {
    sm->m[tid] = sm->limit[tid] = -INFINITY;
    sm->msub[tid] = 0.f;
  }
  if (warp == kWorkWarps) tmem_alloc(&sm->tmem, 512);
  if (warp == kWorkWarps + 1) make_plan(a, blockIdx.x, &sm->plan[0]);
  if (warp < kWorkWarps) {
    const Item it = item_of(a, blockIdx.x);
    request_queries(a, it.r0, it.nr, (it.nr + 15) & ~15, qtile);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sm->tmem, 0);

  if (warp == kWorkWarps + 1) {          // ---- plans and addresses
    bool ok = true;
    int g = 0;
    for (int e = 0; e < items && ok; ++e) {
      if (e >= 2) ok = wait_warp(sm, &sm->plan_free[e & 1], ((e >> 1) - 1) & 1, a.spin);
      if (!ok) break;
      Plan* pl = &sm->plan[e & 1];
      if (e > 0) make_plan(a, blockIdx.x + e * gridDim.x, pl);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->plan_full[e & 1]);
      TileWalk walk(pl);
      for (int i = 0; i < pl->nt && ok; ++i, ++g) ok = look_up_tile(a, sm, pl, walk, pl->begin + i, g);
    }
  } else if (warp == kWorkWarps) {       // ---- products
    if (elect_lane()) {
      const uint64_t dk = smem_desc_sw128(smem_u32(ktile), 16, 1024);
      const uint64_t dq = smem_desc_sw128(smem_u32(qtile), 16, 1024);
      const uint64_t dv = smem_desc_sw128(smem_u32(ktile), kChunk, 1024);
      const uint64_t dp = smem_desc_sw128(smem_u32(ptile), kChunk, 1024);
      bool ok = true;
      int g = 0;
      for (int e = 0; e < items && ok; ++e) {
        ok = wait_bar(sm, &sm->plan_full[e & 1], (e >> 1) & 1, a.spin);
        if (!ok) break;
        const Plan* pl = &sm->plan[e & 1];
        const int nt = pl->nt, nq = pl->nq;
        const uint32_t ids = make_idesc(1, 1, 0, 0, 128, 0) | (static_cast<uint32_t>(nq >> 3) << 17);
        const uint32_t ido = make_idesc(1, 1, 1, 1, 128, 0) | (static_cast<uint32_t>(nq >> 3) << 17);
        const uint32_t qstep = nq * 8;   // a chunk of Q, in the descriptors' 16-byte units
        ok = wait_bar(sm, &sm->bar_q[e & 1], (e >> 1) & 1, a.spin);
        for (int i = 0; i < nt && ok; ++i, ++g) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if ((c & 1) == 0) {
              ok = ok && wait_bar(sm, &sm->full[c >> 1], g & 1, a.spin);
              tc_fence_after();
            }
            if (ok) issue_s_chunk(tmem + kTmemS, dk + c * (kChunk >> 4), dq + c * qstep, dq + 8 * qstep, c, ids);
          }
          const int ks = (min(sm->info[g & 1].n, kKeys) + 15) >> 4;   // (the tile's, until its weights are there)
          mma_commit(&sm->bar_s[0]);
          mbar_arrive(&sm->bar_s[0]);   // hands on what the loading warps wrote (none)
          ok = ok && wait_bar(sm, &sm->bar_p[0], g & 1, a.spin);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int mb = 0; mb < 4; ++mb) {
            const uint64_t dvb = dv + mb * (kChunk >> 3);
            if (i == 0) mma_set(tmem + mb * kRows, dvb, dp, ido);
            else mma_add(tmem + mb * kRows, dvb, dp, ido);
            if (ks == 8) {
#pragma unroll
              for (int k = 1; k < 8; ++k) mma_add(tmem + mb * kRows, dvb + k * 128, dp + k * 128, ido);
            } else {
#pragma unroll 1
              for (int k = 1; k < ks; ++k) mma_add(tmem + mb * kRows, dvb + k * 128, dp + k * 128, ido);
            }
            mma_commit(&sm->free_[mb]);
          }
        }
        mbar_arrive(&sm->plan_free[e & 1]);
      }
      drain_products(sm);
    }
    __syncwarp();
  } else {                               // ---- loads, softmax, epilogue
    RowLoader<FMT, 8> rows(sm, ktile);
    bool ok = true, requested = false;
    int g = 0;
    auto plan_of = [&](int e) -> const Plan* {   // nullptr: not there in time
      return wait_warp(sm, &sm->plan_full[e & 1], (e >> 1) & 1, a.spin) ? &sm->plan[e & 1] : nullptr;
    };
    for (int e = 0; e < items; ++e) {
      const Plan* pl = plan_of(e);
      if (work_any(pl == nullptr)) break;
      rotate_queries<2>(a, pl->item.r0, pl->item.nr, pl->nq, qtile);
      tc_fence_before();
      __syncwarp();
      // (a barrier per plan slot: nothing else keeps these warps from completing the phase of the row
      // block behind one without tiles before the issuing thread has seen this one)
      if (lane == 0) mbar_arrive(&sm->bar_q[e & 1]);
      float l = 0.f, hat[4] = {0.f, 0.f, 0.f, 0.f};   // sums of the weights, and of the rounded ones
      const int nt = pl->nt;
      if (nt > 0 && !requested) ok = rows.request(g, a.spin) && ok;
      for (int i = 0; i < nt; ++i, ++g) {
        ok = rows.fill(g, a.spin) && ok;
        // the next tile's bytes, this row block's or the next one's
        const bool last = i + 1 == nt;
        const Plan* np = !last ? pl : e + 1 < items ? plan_of(e + 1) : nullptr;
        requested = np != nullptr && (!last || np->nt > 0);
        if (requested) ok = rows.request(g + 1, a.spin) && ok;
        ok = weigh_tile(a, pl, sm, ktile, ptile, tmem, g, i == 0, l, hat) && ok;
        // the last S product on these queries is complete: the next ones may come
        if (last && np != nullptr) request_queries(a, np->item.r0, np->item.nr, np->nq, qtile);
      }
      finish_sums(a, pl, sm, l, hat);
      if (nt > 0 && ok) wait_bar(sm, &sm->free_[3], (g - 1) & 1, a.spin);
      if (nt == 0 && e + 1 < items) {
        const Plan* np = plan_of(e + 1);
        work_sync();   // everybody has rotated these rows
        if (np != nullptr) request_queries(a, np->item.r0, np->item.nr, np->nq, qtile);
      }
      __syncwarp();
      tc_fence_after();
      write_rows(a, pl, sm, tmem, nt);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->plan_free[e & 1]);
    }
    cp_async_wait_all();   // (queries on their way, if a wait gave up)
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWorkWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (a.rings_only && a.beside) grid_dep_wait();   // this grid completes after the one it runs beside
}

// Joins a row's partial outputs in order, adds the sink, turns the output back: 64 threads of
// 8 dims, and where there are many parts four times as many, each with every fourth part (128
// parts of 8 rows took 45 us longer with 64 threads that read them one after the other).
// Up to 8 parts one share: four take longer where there are many rows (16 requests of 64 heads and
// 4 parts: 31.2 us, with four shares 32.6); beyond, 30.6 us against 18.3 (16 heads, 8,192 keys).
constexpr int kFewParts = 8;
template <int kShares>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ ListArgs a) {
  __shared__ float shares[kShares > 1 ? kShares - 1 : 1][kD];
  grid_dep_wait();
  const int sub = threadIdx.x >> 6, share = kShares > 1 ? sub : 0, lane = threadIdx.x & 31;
  const size_t row = kShares > 1 ? blockIdx.x : static_cast<size_t>(blockIdx.x) * 4 + sub;
  if (row >= static_cast<size_t>(a.T) * a.H) return;   // (one row per block: never)
  const int d = (threadIdx.x & 63) * 8;
  const float2* ml = reinterpret_cast<const float2*>(a.ml) + row * a.parts;
  const float sink = a.sink ? a.sink[row % a.H] : -INFINITY;
  const float s2 = sink * kLog2e;
  auto weight = [&](float2 x, float M) { return x.y == 0.f ? 0.f : x.y != x.y ? x.y : exp2f(x.x - M); };
  // the maximum and the sum: each thread by itself, or a part per lane
  const int first = kShares > 1 ? lane : 0, step = kShares > 1 ? 32 : 1;
  float M = s2, total = 0.f, o[8];
#pragma unroll 4
  for (int p = first; p < a.parts; p += step) {
    const float2 x = __ldg(ml + p);
    if (x.y != 0.f) M = fmaxf(M, x.x);
  }
  if constexpr (kShares > 1) {
    for (int w = 16; w >= 1; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, w));
    for (int p = lane; p < a.parts; p += 32) {
      const float2 x = __ldg(ml + p);
      total += x.y * weight(x, M);
    }
    for (int w = 16; w >= 1; w >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, w);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
#pragma unroll 4
  for (int p = share; p < a.parts; p += kShares) {
    const float2 x = __ldg(ml + p);
    const float e = weight(x, M);   // 0: a part without keys, whose output is 0
    if constexpr (kShares == 1) total += x.y * e;
    const float4* v = reinterpret_cast<const float4*>(a.opart + (row * a.parts + p) * kD + d);
    const float4 v0 = __ldg(v), v1 = __ldg(v + 1);
    o[0] += e * v0.x; o[1] += e * v0.y; o[2] += e * v0.z; o[3] += e * v0.w;
    o[4] += e * v1.x; o[5] += e * v1.y; o[6] += e * v1.z; o[7] += e * v1.w;
  }
  if constexpr (kShares > 1) {
    if (share > 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) shares[share - 1][d + i] = o[i];
    }
    __syncthreads();
    if (share > 0) return;
    for (int x = 0; x < kShares - 1; ++x) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] += shares[x][d + i];
    }
  }
  const bool none = total == 0.f;   // no key that counts beside the sink
  if (s2 != -INFINITY) total += exp2f(s2 - M);
  const float inv = none ? 0.f : 1.0f / total;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] *= inv;
  if (d >= kD - 64) {
    const float* cs = a.q_rope + row / a.H * 64 + (d - (kD - 64));
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float c = cs[i], s = cs[i + 1], y0 = o[i], y1 = o[i + 1];
      o[i] = y0 * c + y1 * s;
      o[i + 1] = y1 * c - y0 * s;
    }
  }
  *reinterpret_cast<uint4*>(a.out + (row * kD + d) * 2) =
      make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
  if (a.lse != nullptr && d == 0) a.lse[row] = none ? sink : (M + log2f(total)) * kLn2;
}

// ---------------------------------------------------------------------------
// accumulated weights: S^T of every tile, then a thread sums its key's weights over the
// heads.  Up to 128 heads are the MMA columns, two S buffers in TMEM, four chunk slots
// (released as soon as the chunk's products are complete).  Eight slots would hold a tile, but the
// rows' bytes on their way wait for lines of what shared memory leaves of L1: 32 x 8192 FP8 entries
// of 64 heads took 52 us with eight slots (28 KB of L1) and 45 us with four (64 KB).
// Two, where the queries of more than 112 heads leave room for no more.  The weights are fp32: with
// a rotated query in three bf16 numbers and the S product in four sums logits of N(0, 2) are off by
// 2.3e-7 (rms), in the two sums that 128 columns leave room for by 6.4e-7; in two numbers and one sum
// they were off by 2.1e-6, and no faster.
// ---------------------------------------------------------------------------
constexpr int kTileSums = 256;   // TMEM columns of a tile: 4 sums of up to 64 columns, or 2 of up to 128
__device__ __forceinline__ int tile_sums(int nq) { return nq <= 64 ? 4 : 2; }

// Request b's queries and log-sum-exps (base 2; +inf: adds nothing); warps 0-15.
__device__ __forceinline__ void load_request(const ListArgs& a, ListSmem* sm, int b, int nq, uint8_t* qtile, float* lse) {
  work_sync();   // the request before it is weighed
  request_queries(a, b * a.H, a.H, nq, qtile);
  if (threadIdx.x < 128) {
    const float v = threadIdx.x < a.H ? a.lse_in[static_cast<size_t>(b) * a.H + threadIdx.x] : -INFINITY;
    lse[threadIdx.x] = v == -INFINITY ? INFINITY : v * kLog2e;
  }
  rotate_queries<3>(a, b * a.H, a.H, nq, qtile);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sm->bar_q[0]);   // (every run has a tile: one barrier does)
}

// The block's runs: an even share of all requests' tiles (up to kRuns requests), or of one
// request's.  One warp calls this.
__device__ __forceinline__ void plan_weights(const ListArgs& a, ListSmem* sm) {
  const int lane = threadIdx.x & 31;
  int keys[2] = {0, 0}, before[2];
  long long lo, hi;
  int req[2];
  if (a.balanced) {
    int sum = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      req[u] = 2 * lane + u;
      if (req[u] < a.T) keys[u] = max(0, entries_of(a, req[u]) - a.first);
      before[u] = sum;
      sum += tiles_of(keys[u]);
    }
    int upto = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += x;
    }
    const long long total = __shfl_sync(0xFFFFFFFFu, upto, 31);
    before[0] += upto - sum;
    before[1] += upto - sum;
    lo = total * blockIdx.x / gridDim.x;
    hi = total * (blockIdx.x + 1) / gridDim.x;
  } else {
    req[0] = blockIdx.x / a.split;
    req[1] = 0;
    before[0] = before[1] = 0;
    if (lane == 0) keys[0] = max(0, entries_of(a, req[0]) - a.first);
    const long long total = __shfl_sync(0xFFFFFFFFu, tiles_of(keys[0]), 0);
    lo = total * (blockIdx.x % a.split) / a.split;
    hi = total * (blockIdx.x % a.split + 1) / a.split;
  }
  int nruns = 0;
  uint32_t have[2];
  long long from[2], to[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    from[u] = max(lo, static_cast<long long>(before[u]));
    to[u] = min(hi, static_cast<long long>(before[u]) + tiles_of(keys[u]));
    have[u] = __ballot_sync(0xFFFFFFFFu, from[u] < to[u]);
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if (from[u] < to[u]) {
      const uint32_t below = (1u << lane) - 1u;
      const int at = __popc(have[0] & below) + __popc(have[1] & below) + (u == 1 ? (have[0] >> lane) & 1 : 0);
      const long long k0 = (from[u] - before[u]) * kKeys, k1 = min(static_cast<long long>(keys[u]), (to[u] - before[u]) * kKeys);
      sm->plan[0].runs[at] = Run{req[u], 0, static_cast<int>(a.first + k0), static_cast<int>(k1 - k0),
                         static_cast<int>(from[u] - lo), 0, 1, 0, 1, 0, 0, 0};
    }
  }
  nruns = __popc(have[0]) + __popc(have[1]);
  if (lane == 0) {
    sm->plan[0].nruns = nruns;
    sm->plan[0].begin = 0;
    sm->plan[0].nt = static_cast<int>(hi - lo);
  }
}

// The block's nt tiles (runs of one or several requests): while the S product of a tile runs,
// the tile before it is weighed.
template <int FMT, int NS>
__device__ __forceinline__ void weigh_tiles(const ListArgs& a, ListSmem* sm, uint8_t* slots, uint8_t* qtile,
                                            float* lse, uint32_t tmem, int nq, int nt) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, group = warp >> 2;
  const int key = quarter * 32 + lane;
  const uint32_t tlane = static_cast<uint32_t>(quarter * 32) << 16;
  RowLoader<FMT, NS> rows(sm, slots);
  const Plan* pl = &sm->plan[0];
  const int sums = tile_sums(nq);
  TileWalk walk(pl);
  rows.request(0, a.spin);
  int next_run = 1, i = 0, t = 0;   // tiles to fill and to weigh next
  while (t < nt) {
    // The first tile of another request's run is filled after the tile before it has been weighed
    // and the queries replaced: with four slots its first chunks have to be used before the last
    // ones can be filled.
    const bool turn = next_run < pl->nruns && i == pl->runs[next_run].tile0;
    if (i < nt && (i == t || !turn)) {
      if (turn) load_request(a, sm, pl->runs[next_run++].req, nq, qtile, lse);
      rows.fill(i, a.spin);
      if (lane == 0) mbar_arrive(&sm->rows_free[i & 1]);
      ++i;
      if (i < nt) rows.request(i, a.spin);
      if (i < nt && i - t < 2) continue;
    }
    const int buf = t & 1;
    int k0, n;
    walk.seek(t, &k0, &n);
    const Run& u = pl->runs[walk.run];
    wait_bar(sm, &sm->bar_s[buf], (t >> 1) & 1, a.spin);
    __syncwarp();
    tc_fence_after();
    // columns group * 16, group * 16 + 64, ...: this warp's share of the heads
    float w = 0.f;
    for (int c = group * 16; c < nq; c += 64) {
      float z[16], more[16];
      const uint32_t at = tmem + tlane + buf * kTileSums + c;
      tmem_ld16(at, z);
      for (int x = kTileSums / sums; x < kTileSums; x += kTileSums / sums) {
        tmem_ld16(at + x, more);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) z[k] += more[k];
      }
#pragma unroll
      for (int k = 0; k < 16; k += 4) {
        const float4 s = *reinterpret_cast<const float4*>(&lse[c + k]);
        w += (exp2_fast(fmaf(z[k], a.scale_log2, -s.x)) + exp2_fast(fmaf(z[k + 1], a.scale_log2, -s.y))) +
             (exp2_fast(fmaf(z[k + 2], a.scale_log2, -s.z)) + exp2_fast(fmaf(z[k + 3], a.scale_log2, -s.w)));
      }
    }
    tc_fence_before();
    const uint32_t none = sm->none[t & 3][quarter];
    float* part = lse + 128 + buf * (3 * kKeys);   // three groups' shares, two tiles in turn
    if (group > 0) part[(group - 1) * kKeys + key] = w;
    work_sync();
    if (lane == 0) mbar_arrive(&sm->bar_p[buf]);
    if (group == 0 && key < n) {
      w = (w + part[key]) + (part[kKeys + key] + part[2 * kKeys + key]);
      if ((none >> lane) & 1u) w = 0.f;
      const long long b = u.req, j = walk.position(k0 + key);
      a.acc_out[b * a.acc_out_stride + j] = a.decay * a.acc[b * a.acc_stride + j] + w;
    }
    ++t;
  }
}

template <int kWeightSlots>
__global__ void __launch_bounds__(kThreads, 1) weights_kernel(const __grid_constant__ ListArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* slots = base;
  const int nq = (a.H + 15) & ~15;
  uint8_t* qtile = slots + kWeightSlots * kChunk;
  ListSmem* sm = reinterpret_cast<ListSmem*>(qtile + 10 * nq * 128);
  float* lse = reinterpret_cast<float*>(sm + 1);   // [128], then the groups' shares of two tiles
  const int tid = threadIdx.x, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm->full[i], 4);
      mbar_init(&sm->free_[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->rows_full[i], 1);
      mbar_init(&sm->rows_free[i], kWorkWarps);
      mbar_init(&sm->bar_s[i], 2);
      mbar_init(&sm->bar_p[i], kWorkWarps);
    }
    mbar_init(&sm->bar_q[0], kWorkWarps);
    mbar_init(&sm->drained, 1);
    sm->abort = 0;
    fence_mbar_init();
    sm->plan[0].item.row_bytes = a.row_bytes;
    sm->plan[0].item.pages = a.kv;
    sm->plan[0].item.n_prefix = 0;
  }
  if (warp == 1) plan_weights(a, sm);
  if (warp == kWorkWarps) tmem_alloc(&sm->tmem, 2 * kTileSums);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sm->tmem, 0);
  const int nt = sm->plan[0].nt;

  if (nt > 0) {
    if (warp == kWorkWarps + 1) {
      TileWalk walk(&sm->plan[0]);
      bool ok = true;
      for (int g = 0; g < nt && ok; ++g) ok = look_up_tile(a, sm, &sm->plan[0], walk, g, g);
    } else if (warp == kWorkWarps) {
      if (elect_lane()) {
        const uint32_t ids = make_idesc(1, 1, 0, 0, 128, 0) | (static_cast<uint32_t>(nq >> 3) << 17);
        const uint64_t dk = smem_desc_sw128(smem_u32(slots), 16, 1024);
        const uint64_t dq = smem_desc_sw128(smem_u32(qtile), 16, 1024);
        const uint32_t qstep = nq * 8;
        const int sums = tile_sums(nq);
        bool ok = true;
        int run = -1;
        for (int i = 0; i < nt && ok; ++i) {
          const int buf = i & 1;
          if (run + 1 < sm->plan[0].nruns && i == sm->plan[0].runs[run + 1].tile0) {
            ++run;
            ok = wait_bar(sm, &sm->bar_q[0], run & 1, a.spin);
          }
          if (i >= 2) ok = ok && wait_bar(sm, &sm->bar_p[buf], ((i >> 1) - 1) & 1, a.spin);
          tc_fence_after();
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int slot = 2 * m % kWeightSlots, fill = i * (8 / kWeightSlots) + 2 * m / kWeightSlots;
            ok = ok && wait_bar(sm, &sm->full[slot >> 1], fill & 1, a.spin);
            tc_fence_after();
            if (ok)
              issue_s_block(tmem + buf * kTileSums + (m * sums >> 2) * (kTileSums / sums), dk + slot * (kChunk >> 4),
                            dq + 2 * m * qstep, dq + 8 * qstep, qstep, m, (m & 1) != 0 && sums == 2, ids);
            mma_commit(&sm->free_[m]);
          }
          mma_commit(&sm->bar_s[buf]);
          mbar_arrive(&sm->bar_s[buf]);   // hands on what the loading warps wrote (none)
        }
        drain_products(sm);
      }
      __syncwarp();
    } else {
      load_request(a, sm, sm->plan[0].runs[0].req, nq, qtile, lse);
      if (a.kv.fmt == CSKV_FMT_FP8_E4M3_E8M0_B32)
        weigh_tiles<CSKV_FMT_FP8_E4M3_E8M0_B32, kWeightSlots>(a, sm, slots, qtile, lse, tmem, nq, nt);
      else if (a.kv.fmt == CSKV_FMT_FP4_E2M1_E4M3_B16)
        weigh_tiles<CSKV_FMT_FP4_E2M1_E4M3_B16, kWeightSlots>(a, sm, slots, qtile, lse, tmem, nq, nt);
      else
        weigh_tiles<CSKV_FMT_BF16, kWeightSlots>(a, sm, slots, qtile, lse, tmem, nq, nt);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWorkWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kTileSums);
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// Only as much as the rows need: the rest is L1, which the keys on their way wait for.
constexpr size_t attn_smem(int q_rows) { return 1024 + 9 * size_t(kChunk) + 9 * size_t(q_rows) * 128 + sizeof(ListSmem); }
static_assert(attn_smem(kRows) <= 227 * 1024, "one block per SM");

constexpr size_t weights_smem(int H, int slots) {
  return 1024 + slots * size_t(kChunk) + 10 * size_t((H + 15) & ~15) * 128 + sizeof(ListSmem) + (128 + 6 * kKeys) * sizeof(float);
}
constexpr int kMostHeads = 112;   // with four slots
static_assert(weights_smem(kMostHeads, 4) <= 227 * 1024 && weights_smem(128, 2) <= 227 * 1024, "one block per SM");

__host__ __device__ inline size_t a256(size_t x) { return (x + 255) & ~size_t(255); }

// How blocks, splits and partial outputs follow from the sizes alone (so that a workspace of
// the size that was asked for always fits).  Lengths and costs are in tiles of 128 keys.
struct ListPlan {
  int group, head_blocks, heads_per_block, blocks;   // per-query blocks
  int split, prefix_blocks, prefix_split, own_blocks, ring_blocks, parts;
  int prefix_in_own, ring_in_own;
};

constexpr int kSmsPlanned = 152;
constexpr double kBlockCost = 2.0;   // a block's set-up and epilogue

// The time of groups of equal blocks started one after the other on all SMs.
struct Schedule {
  double time = 0, idle = 0;
  void add(double n, double length) {
    const double work = n * length;
    if (work <= idle) {
      idle -= work;
    } else {
      const double left = work - idle, waves = std::ceil(left / length / kSmsPlanned);
      time += waves * length;
      idle = waves * length * kSmsPlanned - left;
    }
    if (time < length) {   // blocks beside shorter ones
      idle += (length - time) * kSmsPlanned;
      time = length;
    }
  }
};

// The join's launch (on the host too: two tiles of one row block in two blocks and a join took
// 26 us a call, in one block 20 us), and writing and reading partial outputs: 4 KB a row and part.
double join_cost(double rows, int parts) { return parts <= 1 ? 0.0 : 2.0 + rows * parts * 4096.0 / 15e6; }

int shares(int tiles, int len) { return len > 0 ? (tiles + len - 1) / len : 0; }

// the share length of least cost among tiles, tiles / 2, ... (every count to 16, then in steps of an eighth)
template <class Cost>
int best_length(int tiles, Cost&& cost) {
  int best_len = tiles;
  double best = cost(tiles);
  for (int n = 2; n <= tiles && n <= 4 * kSmsPlanned; n += n < 16 ? 1 : n / 8) {
    const int len = (tiles + n - 1) / n;
    const double c = cost(len);
    if (c < best) {
      best = c;
      best_len = len;
    }
  }
  return best_len;
}

ListPlan base_plan(int T, int H, bool grouped) {
  ListPlan p = {};
  p.head_blocks = (H + kRows - 1) / kRows;
  p.heads_per_block = (H + p.head_blocks - 1) / p.head_blocks;
  p.group = p.head_blocks == 1 && grouped ? std::min(kRuns, kRows / H) : 1;
  p.blocks = (T + p.group - 1) / p.group * p.head_blocks;
  p.split = p.prefix_split = 1;
  return p;
}

// `several`: the queries are of more than one request, so that a row block may see two lists.
ListPlan window_plan(int T, int H, bool grouped, bool several, int max_ctx, int window, int first) {
  ListPlan p = base_plan(T, H, grouped);
  const long long keys = std::min<long long>(max_ctx, static_cast<long long>(window) + first + p.group - 1);
  const int tiles = std::max(1, tiles_of(keys));
  const int len = best_length(tiles, [&](int l) {
    Schedule s;
    s.add(double(p.blocks) * shares(tiles, l), l + kBlockCost);
    if (several && p.group > 1) s.time = std::max(s.time, 2 * l + kBlockCost);
    return s.time + join_cost(double(T) * H, shares(tiles, l));
  });
  p.split = p.parts = shares(tiles, len);
  return p;
}

// The prefix once for blocks of 64 (request, head) rows beside each request's own list, or as
// the first part of every request's list (the better one when a block's 64 rows are one
// request's heads anyway, or when there is little of it: fewer partial outputs).  Apart and in the
// lists: 64 requests of 64 heads and 8,192 + 512 entries 133 and 152 us, of 16 heads and 1,024 + 64
// 22 and 28 us, 32 requests of 896 + 128 the same 26.  The ring in the request's list when its rows
// have the cache's format (`merge`; those 32 requests: 26 us, as blocks of their own 35), else as a
// block of its own.
ListPlan prefix_plan(int B, int H, int n_prefix, int max_entries, bool ring, bool merge) {
  ListPlan best = {};
  double best_cost = -1;
  const int rows = B * H;
  for (int in_own = n_prefix > 0 ? 0 : 1; in_own < 2; ++in_own) {
    ListPlan p = base_plan(B, H, false);
    const int ptiles = in_own ? 0 : tiles_of(n_prefix);
    const int entries = in_own ? max_entries : max_entries - n_prefix;
    p.prefix_in_own = in_own;
    p.own_blocks = entries > 0 || (ptiles == 0 && !ring) ? p.blocks : 0;
    p.ring_in_own = ring && merge && p.own_blocks > 0;
    p.ring_blocks = ring && !p.ring_in_own ? p.blocks : 0;
    p.prefix_blocks = ptiles > 0 ? (rows + kRows - 1) / kRows : 0;
    const int otiles = p.own_blocks > 0 ? tiles_of(entries) + p.ring_in_own : 0;
    auto cost = [&](int l) {
      Schedule s;
      if (ptiles > 0) s.add(double(p.prefix_blocks) * shares(ptiles, l), std::min(l, ptiles) + kBlockCost);
      if (otiles > 0) s.add(double(p.own_blocks) * shares(otiles, l), std::min(l, otiles) + kBlockCost);
      if (p.ring_blocks > 0) s.add(p.ring_blocks, 1 + kBlockCost);
      return s.time + join_cost(rows, shares(ptiles, l) + shares(otiles, l) + (p.ring_blocks > 0));
    };
    const int len = best_length(std::max(1, std::max(ptiles, otiles)), cost);
    p.prefix_split = std::max(1, shares(ptiles, len));
    p.split = std::max(1, shares(otiles, len));
    p.parts = (p.prefix_blocks > 0 ? p.prefix_split : 0) + (p.own_blocks > 0 ? p.split : 0) + (p.ring_blocks > 0);
    const double c = cost(len);
    if (best_cost < 0 || c < best_cost) {
      best_cost = c;
      best = p;
    }
  }
  return best;
}

size_t plan_workspace(const ListPlan& p, int T, int H) {
  if (p.parts <= 1) return 0;
  const size_t n = static_cast<size_t>(T) * H * p.parts;
  return a256(n * kD * 4) + a256(n * 2 * 4);
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
  // finite for the smallest scales too: the reference of a row without keys is -inf, and has to stay so
  a.slack = std::min(kSlack / a.scale_log2, FLT_MAX);
  a.spin = spin_limit();
  return a;
}

// One launch of list_attn_kernel for rows of format fmt; `beside`: it may start while the
// launch before it runs.
cudaError_t launch_kind(const ListArgs& a, int fmt, unsigned grid, bool beside, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed[3];
  auto kernel = fmt == CSKV_FMT_FP8_E4M3_E8M0_B32 ? list_attn_kernel<CSKV_FMT_FP8_E4M3_E8M0_B32>
                : fmt == CSKV_FMT_FP4_E2M1_E4M3_B16 ? list_attn_kernel<CSKV_FMT_FP4_E2M1_E4M3_B16>
                                                    : list_attn_kernel<CSKV_FMT_BF16>;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = attn_smem(a.q_rows);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = beside ? 1 : 0;
  static_assert(CSKV_FMT_BF16 == 0 && CSKV_FMT_FP8_E4M3_E8M0_B32 == 1 && CSKV_FMT_FP4_E2M1_E4M3_B16 == 2, "an index");
  return launch_with_shared_memory(cfg, kernel, allowed[fmt], attn_smem(kRows), a);
}

cudaError_t launch_list(ListArgs& a, const ListPlan& p, void* workspace, cudaStream_t stream) {
  a.group = p.group;
  a.head_blocks = p.head_blocks;
  a.heads_per_block = p.heads_per_block;
  a.split = p.split;
  a.prefix_split = p.prefix_split;
  a.prefix_blocks = p.prefix_blocks;
  a.own_blocks = p.own_blocks;
  a.prefix_in_own = p.prefix_in_own;
  a.ring_in_own = p.ring_in_own;
  a.parts = p.parts;
  const size_t rows = static_cast<size_t>(a.T) * a.H;
  a.opart = static_cast<float*>(workspace);
  a.ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + a256(rows * p.parts * kD * 4));
  // few blocks: a request's keys come from HBM (32 requests of 4,160 keys: 52 us, without it 56); many
  // blocks read them again and again from L2 (a prefix of 896 entries: 26.0 us, without it 25.2)
  a.prefetch = a.req_of == nullptr && p.prefix_blocks == 0 && p.head_blocks == 1;
  a.rings_only = a.lead = a.beside = 0;
  a.q_rows = p.prefix_blocks > 0 ? kRows : (p.group * p.heads_per_block + 15) & ~15;
  const int blocks = p.prefix_blocks * p.prefix_split + (a.pos1 != nullptr ? p.blocks : p.own_blocks) * p.split;
  cudaError_t e = cudaSuccess;
  if (blocks > 0) {
    a.items = blocks;
    a.lead = p.ring_blocks > 0;
    // prompts: one block per SM, each with several row blocks (8,192 tokens of 16 heads, a window of
    // 128: 212 us, with a block each 253); otherwise the row blocks differ in length, and the
    // hardware's order balances them better
    e = launch_kind(a, a.kv.fmt, a.pos1 != nullptr ? std::min(blocks, kSmsPlanned) : blocks, false, stream);
    if (e != cudaSuccess) return e;
  }
  if (p.ring_blocks > 0) {
    ListArgs r = a;
    r.rings_only = 1;
    r.lead = 0;
    r.beside = blocks > 0;
    r.items = p.ring_blocks;
    e = launch_kind(r, a.swa_fmt, p.ring_blocks, r.beside != 0, stream);
  }
  if (e != cudaSuccess || p.parts <= 1) return e;
  // launched while the kernel before it ends; waits for it before it reads anything
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const bool many = p.parts > kFewParts;
  cfg.gridDim = dim3(static_cast<unsigned>(many ? rows : (rows + 3) / 4));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, many ? attn_join_kernel<4> : attn_join_kernel<1>, a);
}

}  // namespace

size_t window_attn_workspace_bytes(int T, int H, int max_ctx, int window, int first) {
  // one query per request, queries of one prompt or of several: the largest
  return std::max({plan_workspace(window_plan(T, H, false, false, max_ctx, window, first), T, H),
                   plan_workspace(window_plan(T, H, true, false, max_ctx, window, first), T, H),
                   plan_workspace(window_plan(T, H, true, true, max_ctx, window, first), T, H)});
}

size_t prefix_attn_workspace_bytes(int B, int H, int n_prefix, int max_entries, int with_swa) {
  // with a ring of the cache's format or of another: the larger of the two
  return std::max(plan_workspace(prefix_plan(B, H, n_prefix, max_entries, with_swa != 0, false), B, H),
                  plan_workspace(prefix_plan(B, H, n_prefix, max_entries, with_swa != 0, true), B, H));
}

cudaError_t launch_window_attn(const void* q, const cskv_paged& rows, int num_reqs, const int32_t* req_of,
                               const int32_t* pos1, int window, int first, int max_ctx, const float* sink, float scale,
                               const float* q_rope, int T, int H, void* out, float* lse, void* workspace,
                               cudaStream_t stream) {
  ListArgs a = common_args(q, rows, sink, scale, q_rope, T, H, out, lse);
  a.req_of = req_of;
  a.pos1 = pos1;
  a.num_reqs = num_reqs;
  a.window = window;
  a.first = first;
  a.max_ctx = max_ctx;
  // without req_of every query is a request of its own: no two share keys
  return launch_list(a, window_plan(T, H, req_of != nullptr, num_reqs > 1, max_ctx, window, first), workspace, stream);
}

cudaError_t launch_prefix_attn(const void* q, const cskv_paged& kv, const int32_t* n_entries, int n_prefix,
                               int max_entries, const void* swa, int swa_fmt, const int32_t* ctx_len, const float* sink,
                               float scale, const float* q_rope, int B, int H, void* out, float* lse, void* workspace,
                               cudaStream_t stream) {
  ListArgs a = common_args(q, kv, sink, scale, q_rope, B, H, out, lse);
  a.n_entries = n_entries;
  a.n_prefix = n_prefix;
  a.max_entries = max_entries;
  a.swa = static_cast<const uint8_t*>(swa);
  a.swa_fmt = swa_fmt;
  a.swa_row_bytes = swa != nullptr ? static_cast<int>(cskv_row_bytes(swa_fmt, kD)) : 0;
  a.ctx_len = ctx_len;
  return launch_list(a, prefix_plan(B, H, n_prefix, max_entries, swa != nullptr, swa_fmt == kv.fmt), workspace, stream);
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
  a.prefetch = 1;
  // up to kRuns requests: the blocks, one per SM, share all their tiles evenly, whatever their
  // lengths (32 requests of 256 to 8,192 entries: 33 us; 58 in blocks of one request's tiles each,
  // as more requests are)
  const int tiles = tiles_of(max_entries - first);
  a.balanced = B <= kRuns;
  unsigned grid = static_cast<unsigned>(std::min<long long>(kSmsPlanned, static_cast<long long>(B) * tiles));
  if (!a.balanced) {
    a.split = shares(tiles, best_length(tiles, [&](int l) {
      Schedule s;
      s.add(double(B) * shares(tiles, l), l + kBlockCost);
      return s.time;
    }));
    grid = static_cast<unsigned>(B) * a.split;
  }
  static std::atomic<uint64_t> allowed[2];
  const bool most = H > kMostHeads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = weights_smem(H, most ? 2 : 4);
  cfg.stream = stream;
  return launch_with_shared_memory(cfg, most ? weights_kernel<2> : weights_kernel<4>, allowed[most],
                                   most ? weights_smem(128, 2) : weights_smem(kMostHeads, 4), a);
}

unsigned int take_err_list_attn() { return take_dev_err(); }

}  // namespace cskv
