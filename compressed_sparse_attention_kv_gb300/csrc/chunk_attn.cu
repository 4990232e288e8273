// Attention of chunks of new tokens over all visible entries of a paged cache and a window of raw
// rows (cskvs_chunk_attn).
//
// The mathematics.  A key row c_j is key and value of every head.  For a (query, head) row r with
// rotated query q'_r: z_rj = (q'_r . c_j) * scale over the keys the row sees, and
// out_r = rot^-1(sum_j exp(z_rj) c_j / (sum_j exp(z_rj) + exp(sink))).  A running reference m_r
// (base 2) stands for the maximum: l_r <- l_r 2^(m - m') + sum_j 2^(z_rj - m'), O_r likewise, and m
// moves only when a logit exceeds it by more than kSlack (weights stay below 2^kSlack).
//
// What bounds it.  Every key is read by all the queries of its chunk, so the products: 4 * 512
// flops for each (query, head, key).  On an SM a 128 x 64 x 16 product takes 50 cycles and a
// 64 x 64 x 16 one 35 (operands from shared memory, measured), so that 64 rows on 64 keys cost
// 36 * 35 + 16 * 51 = 2,060 cycles, half of the tensor core's peak rate; a 512-d fp32 output of more
// than 64 rows and the logits beside it do not fit the tensor memory.
//
// Four kernels, each started while the one before it ends:
//   chunk_plan_kernel    the requests' key lists, the row blocks and their tiles as one line of
//                        work, cut into equal shares;
//   chunk_decode_kernel  every key that some query sees, once, from its paged row to bf16 in the
//                        order that the tensor core reads (the same rows are read by hundreds of row
//                        blocks: decoding a tile takes longer than its products);
//   chunk_attn_kernel    one block per SM, its share of the work;
//   chunk_join_kernel    the row blocks that a share's border cuts in two or more.
//
// chunk_attn_kernel.  A row block is up to 64 rows of one request: 64 / H queries, or one query's
// heads.  Its keys come in tiles of 64, two tiles in shared memory; P is one of two buffers; tensor
// memory holds the output (4 blocks of 128 dims x 64 rows, dims as lanes) and two tiles' logits
// (rows as lanes: a row's sums stay within four threads).  Roles:
//   warps 0-7    softmax of a tile, 16 rows and 32 keys each: logits from tensor memory, P to shared
//                memory (four warps of 64 keys each took 2,000 cycles a tile: 5.76 ms);
//   warps 8-15   the next row block's queries (loaded and rotated while the last products of this one
//                run), and the outputs;
//   warp 16      one thread issues the products: S S O O of two tiles in turn, so that the softmax of
//                one runs beside the products of the other, and the next two tiles' keys come while
//                the O products run;
//   warp 17      plans row blocks and sends for their keys (bulk copies, a pair of chunks of 64 dims
//                at a time, as soon as the O product on the pair two tiles before is complete).
// Roundings as in list_attn.cu: the rotated query as two bf16 numbers, P in bf16 over the sum of the
// rounded weights, all sums, references and partial outputs fp32.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "attn.cuh"
#include "internal.h"

namespace cskv {

namespace {

constexpr int kD = 512;
constexpr int kTile = 64;                 // keys of a tile
constexpr int kRows = 64;                 // rows of a row block
constexpr int kChunk = kTile * 128;       // bytes of 64 dims of a tile
constexpr int kPair = 2 * kChunk;         // of 128 dims: groups of 8 keys, each [64 dims][8 keys][128 B] twice
constexpr int kStage = 4 * kPair;
constexpr int kSoftWarps = 8, kOutWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kOutWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = (kLoadWarp + 1) * 32;
constexpr int kOutThreads = kOutWarps * 32;
constexpr uint32_t kTmemS = 256;          // TMEM columns: O 0..255, S from here, 64 for each tile
constexpr float kSlack = 8.0f;            // base 2
constexpr int kSms = 152;
constexpr int kPlanThreads = 1024;
constexpr int kPlanItems = 4;             // row blocks of a thread at a time
constexpr int kItemUnits = 3;             // a row block's cost beside its tiles, a tile being 2
constexpr int kLeastShare = 8;            // units of a share

struct ReqPlan {
  int q0, nq, len;          // its queries [q0, q0 + nq), its length
  int entries, entries16;   // entries that count, and rounded up to 16 (decoded rows)
  int row0, rows, rows16;   // its first decoded raw row, how many, rounded up
  long long base;           // its first decoded row
  int item0;                // its first row block
  int bad;                  // a row of it could not be read or is not finite
};
struct SplitPlan {
  int item, b0, b1, pad;    // a row block that blocks b0 .. b1 share
};
struct ChunkHead {
  int items, blocks, splits, pad;
  long long units;          // of all row blocks
  long long keys;           // decoded rows
};

struct ChunkArgs {
  const uint8_t* q;
  const int32_t* cu_q;
  const int32_t* ctx_len;
  int R, T, H;
  cskv_paged entries, rows;
  int has_entries, has_rows;
  int ratio;
  const int32_t* n_entries;
  int max_entries, window, max_ctx;
  const float* sink;
  float scale_log2, slack;
  const float* q_rope;
  uint8_t* out;
  float* lse;
  long long max_keys;
  int group, head_blocks, heads_per_block;
  int most_blocks;          // shares at most
  // workspace
  ChunkHead* head;
  ReqPlan* req;
  long long* unit0;         // [items + 1]
  SplitPlan* split;         // [most_blocks]
  uint8_t* flags;           // of every decoded row: 0, kNone, kUnfit
  uint8_t* images;          // decoded rows: of each request 4 blocks of 128 dims as they lie in a stage
  float* opart;             // [2 * most_blocks][kRows][512]
  float2* ml;               // [2 * most_blocks][kRows]: m (base 2) and l
  unsigned long long spin;
};
constexpr uint8_t kNone = 1, kUnfit = 2;

__host__ __device__ inline int up16(int n) { return (n + 15) & ~15; }

// ---------------------------------------------------------------------------
// row blocks
// ---------------------------------------------------------------------------
// The request of row block e, by the first row blocks of the requests.
__device__ __forceinline__ int request_of_item(const ChunkArgs& a, int e) {
  int r = 0, n = a.R;
  while (n > 1) {   // the last request whose first row block is not behind e
    const int half = n / 2;
    const bool le = a.req[r + half].item0 <= e;
    r = le ? r + half : r;
    n = le ? n - half : half;
  }
  return r;
}

// What row block e of request p sees: entries [0, seen) and decoded raw rows [lo, hi) (counted from
// the request's first decoded one), both as lists of whole 16 rows: entries16 of them, then raw
// rows from raw0.
struct BlockKeys {
  int i0, i1;               // queries of the request
  int seen16, raw0, keys;   // keys: rows of the list
};
__device__ __forceinline__ int seen_entries(const ChunkArgs& a, const ReqPlan& p, int pos1) {
  return a.ratio > 0 ? min(p.entries, max(pos1, 0) / a.ratio) : p.entries;
}
__device__ __forceinline__ BlockKeys block_keys(const ChunkArgs& a, const ReqPlan& p, int x) {
  BlockKeys k;
  const int g = a.head_blocks == 1 ? x : x / a.head_blocks;
  k.i0 = g * a.group;
  k.i1 = min(p.nq, k.i0 + a.group);
  const int p0 = p.len - p.nq + k.i0 + 1, p1 = p.len - p.nq + k.i1;   // position + 1 of the first and last one
  k.seen16 = up16(seen_entries(a, p, p1));
  k.raw0 = 0;
  k.keys = k.seen16;
  if (p.rows > 0 && p1 > 0) {
    const int lo = max(0, p0 - a.window) - p.row0, hi = p1 - p.row0;
    k.raw0 = max(0, lo) & ~15;
    k.keys += up16(hi) - k.raw0;
  }
  return k;
}
__device__ __forceinline__ int tiles_of(int keys) { return (keys + kTile - 1) / kTile; }
__device__ __forceinline__ int units_of(int tiles) { return 2 * max(tiles, 1) + kItemUnits; }

// Shares: block b has the units [units * b / blocks, units * (b + 1) / blocks); tile t of a row block
// begins at its unit 2 t and belongs to the block that has this unit.
__device__ __forceinline__ long long share_begin(long long units, int blocks, int b) { return units * b / blocks; }
__device__ __forceinline__ int block_of_unit(long long units, int blocks, long long u) {
  return static_cast<int>(((u + 1) * blocks - 1) / units);
}
// the last row block that begins at or before unit u
__device__ __forceinline__ int item_of_unit(const long long* unit0, int items, long long u) {
  int e = 0, n = items;
  while (n > 1) {
    const int half = n / 2;
    const bool le = unit0[e + half] <= u;
    e = le ? e + half : e;
    n = le ? n - half : half;
  }
  return e;
}

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

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ ChunkArgs a) {
  __shared__ long long part[32];
  grid_dep_launch();
  const int tid = threadIdx.x;
  long long keys = 0, items = 0, total;
  for (int r0 = 0; r0 < a.R; r0 += kPlanThreads) {
    const int r = r0 + tid;
    ReqPlan p = {};
    if (r < a.R) {
      const int lo = a.cu_q[r], hi = a.cu_q[r + 1];
      if (lo < 0 || hi < lo || hi > a.T) set_err(CSKV_ERR_BOUNDS);
      else { p.q0 = lo; p.nq = hi - lo; }
      if (p.nq > 0) {
        int len = a.ctx_len != nullptr ? a.ctx_len[r] : 0;
        if (len < 0 || len > a.max_ctx) { set_err(CSKV_ERR_BOUNDS); len = max(0, min(len, a.max_ctx)); }
        p.len = len;
        if (a.has_entries) {
          int n = a.ratio > 0 ? len / a.ratio : a.max_entries;
          if (a.n_entries != nullptr) {
            int m = a.n_entries[r];
            if (m < 0 || m > a.max_entries) { set_err(CSKV_ERR_BOUNDS); m = max(0, min(m, a.max_entries)); }
            n = min(n, m);
          }
          if (n > a.max_entries) { set_err(CSKV_ERR_BOUNDS); n = a.max_entries; }
          p.entries = n;
        }
        if (a.has_rows) {
          p.rows = static_cast<int>(min(static_cast<long long>(len), static_cast<long long>(p.nq) + a.window - 1));
          p.row0 = len - p.rows;
        }
        p.entries16 = up16(p.entries);
        p.rows16 = up16(p.rows);
      }
    }
    const long long mine = static_cast<long long>(p.entries16) + p.rows16;
    const long long upto = keys + block_scan(mine, part, &total);
    keys += total;
    p.base = upto - mine;
    if (upto > a.max_keys && mine > 0) {   // no room
      set_err(CSKV_ERR_BOUNDS);
      p.entries = p.entries16 = p.rows = p.rows16 = 0;
    }
    const int blocks = (p.nq + a.group - 1) / a.group * a.head_blocks;
    p.item0 = static_cast<int>(items + block_scan(blocks, part, &total) - blocks);
    items += total;
    if (r < a.R) a.req[r] = p;
  }
  // the last request that has room ends the decoded rows
  keys = min(keys, a.max_keys);
  __syncthreads();
  long long units = 0;
  for (int e0 = 0; e0 < items; e0 += kPlanThreads * kPlanItems) {
    int mine[kPlanItems], sum = 0;
    const int e1 = e0 + tid * kPlanItems;
    int r = e1 < items ? request_of_item(a, e1) : 0;
#pragma unroll
    for (int u = 0; u < kPlanItems; ++u) {
      mine[u] = 0;
      if (e1 + u < items) {
        while (r + 1 < a.R && a.req[r + 1].item0 <= e1 + u) ++r;
        const ReqPlan& p = a.req[r];
        mine[u] = units_of(tiles_of(block_keys(a, p, e1 + u - p.item0).keys));
      }
      sum += mine[u];
    }
    long long at = units + block_scan(sum, part, &total) - sum;
    units += total;
#pragma unroll
    for (int u = 0; u < kPlanItems; ++u) {
      if (e1 + u < items) a.unit0[e1 + u] = at;
      at += mine[u];
    }
  }
  if (tid == 0) a.unit0[items] = units;
  __syncthreads();
  const int blocks = static_cast<int>(max(1ll, min(static_cast<long long>(a.most_blocks), units / kLeastShare)));
  // row blocks that a border cuts: listed at the last border inside
  int splits = 0;
  for (int b0 = 1; b0 < blocks; b0 += kPlanThreads) {
    const int b = b0 + tid;
    bool last = false;
    int e = 0;
    if (b < blocks) {
      const long long u = share_begin(units, blocks, b);
      e = item_of_unit(a.unit0, static_cast<int>(items), u);
      const int tiles = (static_cast<int>(a.unit0[e + 1] - a.unit0[e]) - kItemUnits) / 2;
      const long long end = a.unit0[e] + 2ll * (tiles - 1);   // its last tile
      last = u > a.unit0[e] && u <= end && block_of_unit(units, blocks, end) == b;
    }
    const long long at = splits + block_scan(last, part, &total) - 1;
    if (last) a.split[at] = SplitPlan{e, block_of_unit(units, blocks, a.unit0[e]), b, 0};
    splits += static_cast<int>(total);
  }
  if (tid == 0) *a.head = ChunkHead{static_cast<int>(items), blocks, splits, 0, units, keys};
}

// ---------------------------------------------------------------------------
// the keys
// ---------------------------------------------------------------------------
// 16 neighbouring dims of a row (lane's) as bf16 pairs
__device__ __forceinline__ void decode16(const cskv_paged& c, const uint8_t* row, int lane, uint32_t (&w)[8]) {
  if (c.fmt == CSKV_FMT_BF16) {
    const uint4* p = reinterpret_cast<const uint4*>(row) + 2 * lane;
    const uint4 x = __ldg(p), y = __ldg(p + 1);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
  } else if (c.fmt == CSKV_FMT_FP8_E4M3_E8M0_B32) {
    convert(__ldg(reinterpret_cast<const uint4*>(row) + lane), __ldg(row + kD + (lane >> 1)), w);
  } else {
    convert(__ldg(reinterpret_cast<const uint2*>(row) + lane), __ldg(row + kD / 2 + lane), w);
  }
}

constexpr int kDecodeThreads = 256;
constexpr int kDecodeRows = 16;   // of a warp at a time (a request's rows are whole 16s)

__global__ void __launch_bounds__(kDecodeThreads) chunk_decode_kernel(const __grid_constant__ ChunkArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const long long keys = a.head->keys;
  const long long warps = static_cast<long long>(gridDim.x) * (kDecodeThreads / 32);
  for (long long x = (static_cast<long long>(blockIdx.x) * kDecodeThreads + threadIdx.x) / 32 * kDecodeRows; x < keys;
       x += warps * kDecodeRows) {
    int r = 0, n = a.R;
    while (n > 1) {   // the last request whose rows begin at or before x
      const int half = n / 2;
      const bool le = a.req[r + half].base <= x;
      r = le ? r + half : r;
      n = le ? n - half : half;
    }
    const ReqPlan p = a.req[r];
    const long long rows = p.entries16 + p.rows16;
    if (x - p.base >= rows) continue;   // no room for this request
    const int first = static_cast<int>(x - p.base);
    const bool raw = first >= p.entries16;
    const cskv_paged& c = raw ? a.rows : a.entries;
    const int k0 = raw ? first - p.entries16 : first, have = raw ? p.rows : p.entries;
    const int row_bytes = c.fmt == CSKV_FMT_BF16 ? 2 * kD : c.fmt == CSKV_FMT_FP8_E4M3_E8M0_B32 ? kD + kD / 32 : kD / 2 + kD / 16;
    // lane i < 16 looks row i up
    const uint8_t* mine = nullptr;
    if (lane < kDecodeRows && k0 + lane < have)
      mine = paged_row(c, r, (raw ? p.row0 : 0) + static_cast<long long>(k0) + lane, row_bytes).data;
    uint8_t* image = a.images + p.base * (2 * kD) + (lane >> 3) * (rows * 256) + static_cast<long long>(first) * 256 +
                     ((lane >> 2) & 1) * 1024;
    uint32_t unfit = 0;
#pragma unroll 4
    for (int i = 0; i < kDecodeRows; ++i) {
      const uint8_t* row = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(mine), i));
      uint32_t w[8] = {};
      if (row != nullptr) {
        decode16(c, row, lane, w);
        uint32_t bad = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) bad |= ((w[k] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
        if (__any_sync(0xFFFFFFFFu, bad != 0u)) {   // (an exponent of all ones carries into the sign bit)
          unfit |= 1u << i;
#pragma unroll
          for (int k = 0; k < 8; ++k) w[k] = 0u;
        }
      }
      const int swz = i & 7, at = 2 * (lane & 3);
      uint8_t* to = image + (i >> 3) * 2048 + swz * 128;
      *reinterpret_cast<uint4*>(to + ((at ^ swz) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(to + (((at + 1) ^ swz) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
    }
    const uint32_t none = __ballot_sync(0xFFFFFFFFu, lane < kDecodeRows && mine == nullptr);
    if (lane < kDecodeRows) a.flags[x + lane] = (none >> lane) & 1u ? kNone : (unfit >> lane) & 1u ? kUnfit : 0;
    // rows that are there but cannot be used; those behind the last one are seen by nobody
    const uint32_t there = k0 + kDecodeRows <= have ? 0xFFFFu : (1u << max(0, have - k0)) - 1u;
    if (lane == 0 && ((none & there) | unfit) != 0u) a.req[r].bad = 1;
  }
}

// ---------------------------------------------------------------------------
// the attention kernel
// ---------------------------------------------------------------------------
struct __align__(16) RowSees {   // key k of the block's list is seen when k < seen or lo <= k <= hi
  int seen, lo, hi, pad;
};

struct Item {
  int r0, nr, nq;                // rows [r0, r0 + nr) of the [T * H] rows; padded to 16
  int t0, one;                   // the first row's query; all rows are that query's
  int seen16, raw0, keys;        // the list (BlockKeys); raw0 counted among all decoded rows of the request
  int begin, nt;                 // this block's tiles
  int plain;                     // keys below it are seen by every row
  int bad;
  int part;                      // partial output, -1: none
  long long base, stride;        // the request's first decoded row, bytes between its blocks of dims
  RowSees sees[kRows];
};

struct ChunkSmem {
  Item item[2];
  uint64_t full[2][4], free_[2][4];        // of a stage's pairs of chunks
  uint64_t s_full[2], p_full[2];
  uint64_t q_full, q_free, o_free, l_full[2], item_full[2], item_free[2], drained;
  uint32_t tmem;
  int abort;
  __align__(16) float fac[kRows];          // a moved reference's factors
  float top[2][kRows];                     // a tile's largest logits, of either half of its keys
  float4 sums[2][2][kRows];                // of a row block and a half: m (base 2), l, sum of the rounded weights
  __align__(16) float out_fac[kRows];
};

__device__ __forceinline__ bool wait_on(ChunkSmem* sm, uint64_t* bar, uint32_t parity, unsigned long long limit) {
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
__device__ __forceinline__ bool wait_bar(ChunkSmem* sm, uint64_t* bar, uint32_t parity, unsigned long long limit) {
  return try_wait_long(bar, parity) || wait_on(sm, bar, parity, limit);
}
__device__ __forceinline__ bool wait_warp(ChunkSmem* sm, uint64_t* bar, uint32_t parity, unsigned long long limit) {
  return __all_sync(0xFFFFFFFFu, wait_bar(sm, bar, parity, limit)) != 0;
}
// Named barriers of the softmax warps (1) and of the output warps (2).  They have no limit: all of
// a role's warps take the same loops (a row block is accepted by all or by none, and after a wait
// that gave up they go on through its tiles without waiting).
template <int kId, int kCount>
__device__ __forceinline__ void role_sync() {
  asm volatile("bar.sync %0, %1;" ::"n"(kId), "n"(kCount) : "memory");
}
template <int kId, int kCount>
__device__ __forceinline__ bool role_any(bool p) {
  int r;
  asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.s32 a, %1, 0;\n\tbar.red.or.pred b, %2, %3, a;\n\tselp.s32 %0, 1, 0, b;\n\t}"
               : "=r"(r) : "r"(static_cast<int>(p)), "n"(kId), "n"(kCount) : "memory");
  return r != 0;
}
constexpr int kSoftId = 1, kOutId = 2;

// 16 lanes x 32 columns: thread l has columns 8 j + 2 (l & 3) and + 1 of lane l / 4 in v[4 j], v[4 j + 1],
// of lane l / 4 + 8 in v[4 j + 2], v[4 j + 3].
__device__ __forceinline__ void tmem_ld16x32(uint32_t taddr, float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Row block e of this block's share; one warp.
__device__ void make_item(const ChunkArgs& a, Item* it, int e, long long units, int blocks) {
  const int lane = threadIdx.x & 31;
  const ReqPlan p = a.req[request_of_item(a, e)];
  const int x = e - p.item0;
  const BlockKeys k = block_keys(a, p, x);
  const int h0 = a.head_blocks == 1 ? 0 : (x % a.head_blocks) * a.heads_per_block;
  const int nr = a.head_blocks == 1 ? (k.i1 - k.i0) * a.H : min(a.heads_per_block, a.H - h0);
  const int raw0 = k.raw0 + p.row0;   // position of the list's first raw row
  int least = INT32_MAX;
  for (int r = lane; r < kRows; r += 32) {
    RowSees s{0, 0, -1, 0};
    if (r < nr) {
      const int pos1 = p.len - p.nq + k.i0 + (a.head_blocks == 1 ? r / a.H : 0) + 1;
      s.seen = seen_entries(a, p, pos1);
      if (p.rows > 0 && pos1 > 0) {
        s.lo = k.seen16 + max(0, pos1 - a.window) - raw0;
        s.hi = k.seen16 + pos1 - 1 - raw0;
      }
      least = min(least, s.seen);
    }
    it->sees[r] = s;
  }
  least = __reduce_min_sync(0xFFFFFFFFu, least);
  if (lane == 0) {
    it->t0 = p.q0 + k.i0;
    it->one = a.head_blocks != 1 || a.group == 1;
    it->r0 = it->t0 * a.H + h0;
    it->nr = nr;
    it->nq = up16(nr);
    it->seen16 = k.seen16;
    it->raw0 = p.entries16 + k.raw0;
    it->keys = k.keys;
    it->plain = least;
    it->bad = p.bad;
    it->base = p.base;
    it->stride = static_cast<long long>(p.entries16 + p.rows16) * 256;
    // its tiles between the share's borders
    const long long u0 = a.unit0[e];
    const int tiles = tiles_of(k.keys);
    const long long lo = share_begin(units, blocks, blockIdx.x), hi = share_begin(units, blocks, blockIdx.x + 1);
    const int begin = static_cast<int>(min(static_cast<long long>(tiles), max(0ll, (lo - u0 + 1) / 2)));
    const int end = static_cast<int>(min(static_cast<long long>(tiles), max(0ll, (hi - u0 + 1) / 2)));
    it->begin = begin;
    it->nt = end - begin;
    it->part = begin > 0 || end < tiles ? 2 * blockIdx.x + (u0 > lo) : -1;
  }
}

// The row blocks of this block's share: [first, last].
__device__ __forceinline__ void share_items(const ChunkArgs& a, const ChunkHead& h, int* first, int* last) {
  const long long lo = share_begin(h.units, h.blocks, blockIdx.x), hi = share_begin(h.units, h.blocks, blockIdx.x + 1);
  int e = item_of_unit(a.unit0, h.items, lo);
  const int tiles = (static_cast<int>(a.unit0[e + 1] - a.unit0[e]) - kItemUnits) / 2;
  if (a.unit0[e] + 2ll * (tiles - 1) < lo) ++e;   // its tiles are all before the border
  *first = e;
  *last = item_of_unit(a.unit0, h.items, hi - 1);
}

// Queries into the K-major chunks of Q (64 rows apart; rows behind the last one zero).  A thread
// rotates what it loaded itself: chunk 7 holds the first bf16 of each rotated value, chunk 8 the second.
__device__ __forceinline__ void request_queries(const ChunkArgs& a, const Item* it, uint8_t* qtile) {
  const int tid = threadIdx.x - kSoftWarps * 32;
  const uint8_t* q = a.q + static_cast<size_t>(it->r0) * kD * 2;
  const int nr = it->nr;
#pragma unroll 4
  for (int x = tid; x < kRows * 64; x += kOutThreads) {
    const int r = x >> 6, c = x & 63;
    uint8_t* dst = qtile + (c >> 3) * kChunk + sw128_offset(r, c & 7);
    if (r < nr) cp_async16(dst, q + static_cast<size_t>(x) * 16);
    else *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
  }
}
__device__ __forceinline__ void rotate_queries(const ChunkArgs& a, const Item* it, uint8_t* qtile) {
  const int tid = threadIdx.x - kSoftWarps * 32;
  const int c = tid & 63;   // of all of the thread's pieces (kOutThreads is a multiple of 64)
  cp_async_wait_all();
  if (c >= 56) {
#pragma unroll 1
    for (int r = tid >> 6; r < kRows; r += kOutThreads / 64) {
      uint4* hi = reinterpret_cast<uint4*>(qtile + 7 * kChunk + sw128_offset(r, c & 7));
      uint4 lo = make_uint4(0u, 0u, 0u, 0u);
      if (r < it->nr) {
        const float* cs = a.q_rope + static_cast<size_t>(static_cast<unsigned>(it->r0 + r) / static_cast<unsigned>(a.H)) * 64 + (c & 7) * 8;
        const float4 t0 = __ldg(reinterpret_cast<const float4*>(cs)), t1 = __ldg(reinterpret_cast<const float4*>(cs + 4));
        const float co[4] = {t0.x, t0.z, t1.x, t1.z}, si[4] = {t0.y, t0.w, t1.y, t1.w};
        uint4 v = *hi;
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
        uint32_t* l = reinterpret_cast<uint32_t*>(&lo);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float y0 = bf16lo(w[k]), y1 = bf16hi(w[k]);
          const float z0 = y0 * co[k] - y1 * si[k], z1 = y0 * si[k] + y1 * co[k];
          w[k] = pack_bf16(z0, z1);
          l[k] = pack_bf16(z0 - bf16lo(w[k]), z1 - bf16hi(w[k]));
        }
        *hi = v;
      }
      *reinterpret_cast<uint4*>(qtile + 8 * kChunk + sw128_offset(r, c & 7)) = lo;
    }
  }
  fence_proxy_async_smem();
}

// The softmax warps' state of two rows: r = 16 * (warp & 3) + lane / 4, and r + 8.
struct RowState {
  float m[2], limit[2], msub[2];   // reference in units of q'.c; a logit above limit moves it; in base 2
  float l[2], hat[2];              // this thread's sums of the weights, and of the rounded ones
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[i] = limit[i] = -INFINITY;
      msub[i] = l[i] = hat[i] = 0.f;
    }
  }
};

// Logits of the keys k0 .. k0 + 31 that a row does not see become -inf, those of unfit rows NaN.
__device__ __forceinline__ void mask_keys(const ChunkArgs& a, const Item* it, int k0, const RowSees (&sees)[2], float (&z)[16]) {
  const int c = 2 * (threadIdx.x & 3);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k = k0 + 8 * j + c + u;
      int flag = 0;
      if (it->bad && k < it->keys) {
        const int row = k < it->seen16 ? k : it->raw0 + k - it->seen16;
        flag = a.flags[it->base + row];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool see = (k < sees[i].seen || (k >= sees[i].lo && k <= sees[i].hi)) && flag != kNone;
        float& x = z[4 * j + 2 * i + u];
        x = !see ? -INFINITY : flag == kUnfit ? __int_as_float(0x7FC00000) : x;
      }
    }
  }
}

// The softmax of the block's tile g, the row block's tile t: this warp's 16 rows and 32 keys.
__device__ __forceinline__ void weigh_tile(const ChunkArgs& a, ChunkSmem* sm, const Item* it, uint8_t* ptile, uint32_t tmem,
                                           int g, int t, bool first, const RowSees (&sees)[2], RowState& s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, half = warp >> 2;
  const uint32_t tlane = static_cast<uint32_t>(quarter * 32) << 16;
  const int buf = g & 1, k0 = t * kTile + 32 * half, r = 16 * quarter + (lane >> 2);
  wait_warp(sm, &sm->s_full[buf], (g >> 1) & 1, a.spin);
  tc_fence_after();
  float z[16];
  tmem_ld16x32(tmem + kTmemS + 64 * buf + 32 * half + tlane, z);
  tmem_wait_ld();
  if (k0 + 32 > it->plain || it->bad) mask_keys(a, it, k0, sees, z);
  float top[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    top[i] = fmaxf(fmaxf(fmaxf(z[2 * i], z[2 * i + 1]), fmaxf(z[4 + 2 * i], z[4 + 2 * i + 1])),
                   fmaxf(fmaxf(z[8 + 2 * i], z[8 + 2 * i + 1]), fmaxf(z[12 + 2 * i], z[12 + 2 * i + 1])));
  if (role_any<kSoftId, kSoftWarps * 32>(top[0] > s.limit[0] || top[1] > s.limit[1])) {   // some row's reference moves
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 1));
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 2));
      if ((lane & 3) == 0) sm->top[half][r + 8 * i] = top[i];
    }
    role_sync<kSoftId, kSoftWarps * 32>();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float now = fmaxf(fmaxf(top[i], sm->top[half ^ 1][r + 8 * i]), s.m[i]);
      const float sub = now == -INFINITY ? 0.f : now * a.scale_log2;
      const float f = s.m[i] == -INFINITY ? 0.f : exp2f(s.msub[i] - sub);
      s.m[i] = now;
      s.limit[i] = now + a.slack;
      s.msub[i] = sub;
      s.l[i] *= f;
      s.hat[i] *= f;
      if (half == 0 && (lane & 3) == 0) sm->fac[r + 8 * i] = f;
    }
    if (!first) {
      role_sync<kSoftId, kSoftWarps * 32>();
      wait_warp(sm, &sm->free_[(g - 1) & 1][3], ((g - 1) >> 1) & 1, a.spin);   // the O product before is complete
      tc_fence_after();
#pragma unroll 1
      for (int block = 2 * half; block < 2 * half + 2; ++block) {   // this warp's 32 dims of two blocks, 16 rows at a time
#pragma unroll 1
        for (int x = 0; x < it->nq; x += 16) {
          float o[16];
          const uint32_t at = tmem + tlane + block * kRows + x;
          tmem_ld16(at, o);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 16; ++c) o[c] *= sm->fac[x + c];
          tmem_st16(at, o);
        }
      }
      tmem_wait_st();
    }
  }
  uint8_t* to = ptile + buf * kChunk + r * 128 + 4 * (lane & 3);
  const int swz = lane >> 2;   // of both rows
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float x = exp2_fast(fmaf(z[4 * j + 2 * i], a.scale_log2, -s.msub[i]));
      const float y = exp2_fast(fmaf(z[4 * j + 2 * i + 1], a.scale_log2, -s.msub[i]));
      const uint32_t w = pack_bf16(x, y);
      s.l[i] += x + y;
      s.hat[i] += bf16lo(w) + bf16hi(w);
      *reinterpret_cast<uint32_t*>(to + i * 1024 + (((4 * half + j) ^ swz) << 4)) = w;
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sm->p_full[buf]);
}

// O^T out, in units of 8 rows of a block of 128 dims: a thread has one dim of them, a row's 32 dims
// of a warp are one 64-byte run.
__device__ __forceinline__ void write_rows(const ChunkArgs& a, const Item* it, ChunkSmem* sm, uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;
  const int r0 = it->r0, nr = it->nr;
  const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const unsigned H = a.H;
  const int sets = (nr + 7) >> 3;
#pragma unroll 1
  for (int x = (warp - kSoftWarps) >> 2; x < 4 * sets; x += kOutWarps / 4) {
    const int block = x / sets, g = (x - block * sets) * 8;
    const int d = block * 128 + quarter * 32 + lane;
    const bool turn = block == 3 && quarter >= 2 && it->part < 0;   // dims 448..511, turned back
    const float2* cs = reinterpret_cast<const float2*>(a.q_rope) + ((d - (kD - 64)) >> 1);
    float2 w = make_float2(1.f, 0.f);
    if (turn && it->one) w = __ldg(cs + static_cast<size_t>(it->t0) * 32);
    float o[8];
    if (it->nt > 0) {
      tmem_ld8(from + block * kRows + g, o);   // (columns behind the last row hold nothing of use)
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < 8; c += 4) {
      const float4 f = *reinterpret_cast<const float4*>(&sm->out_fac[g + c]);
      o[c] *= f.x;
      o[c + 1] *= f.y;
      o[c + 2] *= f.z;
      o[c + 3] *= f.w;
    }
    if (it->part >= 0) {
      float* to = a.opart + (static_cast<size_t>(it->part) * kRows + g) * kD + d;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (g + c < nr) to[c * kD] = o[c];
      continue;
    }
    if (turn) {
      // even lanes turn and store the pair of dims (d, d + 1) of row c, odd lanes (d - 1, d) of row c + 1
      const bool odd = (lane & 1) != 0;
#pragma unroll
      for (int c = 0; c < 8; c += 2) {
        const int r = g + c + (odd ? 1 : 0);
        if (!it->one) w = __ldg(cs + static_cast<size_t>((r0 + min(r, nr - 1)) / H) * 32);
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

// The factors that the rows' outputs take, their log-sum-exps or partial sums.
__device__ __forceinline__ void finish_sums(const ChunkArgs& a, const Item* it, ChunkSmem* sm, int e) {
  const int r = threadIdx.x - kSoftWarps * 32;
  if (r >= kRows) return;
  float f = 0.f;
  if (r < it->nr) {
    float4 s = sm->sums[e & 1][0][r];   // m, l, sum of the rounded weights
    const float4 more = sm->sums[e & 1][1][r];
    s.y += more.y;
    s.z += more.z;
    const unsigned row = it->r0 + r;
    // the output is made of rounded weights: over their own sum a few large ones' roundings cancel
    const float ratio = s.y == 0.f ? 1.f : s.y / s.z;
    if (it->part >= 0) {
      a.ml[static_cast<size_t>(it->part) * kRows + r] = make_float2(s.x, s.y);
      f = ratio;
    } else {
      const float sink = a.sink != nullptr ? __ldg(a.sink + row % static_cast<unsigned>(a.H)) : -INFINITY;
      const float s2 = sink * kLog2e;
      const float M = fmaxf(s.x, s2);
      const float w = exp2f(s.x - M);
      const float total = s.y * w + (s2 == -INFINITY ? 0.f : exp2f(s2 - M));
      // no key, or a sink above fp32 in base 2 (which leaves the keys nothing): out 0, lse the sink itself
      const bool none = s.y == 0.f || s2 == INFINITY;
      f = none ? 0.f : w / total * ratio;
      if (s.y != s.y) f = s.y;
      if (a.lse != nullptr) a.lse[row] = none ? sink : s.y != s.y ? s.y : (M + log2f(total)) * kLn2;
    }
  }
  sm->out_fac[r] = f;
}

// S of a tile: 64 rows x 64 keys, K = 512 dims and the second halves of the 64 rotated ones
__device__ __forceinline__ void issue_s_chunk(uint32_t d, uint64_t dq, uint64_t dk, int c, uint32_t id) {
  const uint64_t q = dq + c * (kChunk >> 4), k = dk + (c >> 1) * (kPair >> 4) + (c & 1) * (1024 >> 4);
  if (c == 0) mma_set(d, q, k, id);
  else mma_add(d, q, k, id);
#pragma unroll
  for (int x = 1; x < 4; ++x) mma_add(d, q + 2 * x, k + 2 * x, id);
  if (c == 7) {
#pragma unroll
    for (int x = 0; x < 4; ++x) mma_add(d, q + (kChunk >> 4) + 2 * x, k + 2 * x, id);
  }
}

constexpr size_t kChunkSmemBytes = 1024 + 2 * size_t(kStage) + 9 * size_t(kChunk) + 2 * size_t(kChunk) + sizeof(ChunkSmem);
static_assert(kChunkSmemBytes <= 227 * 1024, "one block per SM");

__global__ void __launch_bounds__(kThreads, 1) chunk_attn_kernel(const __grid_constant__ ChunkArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ktile = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);   // 2 stages of 64 keys
  uint8_t* qtile = ktile + 2 * kStage;                                            // 9 chunks
  uint8_t* ptile = qtile + 9 * kChunk;                                            // 2 of 64 rows x 64 keys
  ChunkSmem* sm = reinterpret_cast<ChunkSmem*>(ptile + 2 * kChunk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      for (int m = 0; m < 4; ++m) {
        mbar_init(&sm->full[i][m], 1);
        mbar_init(&sm->free_[i][m], 1);
      }
      mbar_init(&sm->s_full[i], 1);
      mbar_init(&sm->p_full[i], kSoftWarps);
      mbar_init(&sm->l_full[i], kSoftWarps);
      mbar_init(&sm->item_full[i], 1);
      mbar_init(&sm->item_free[i], 1 + kSoftWarps + kOutWarps);
    }
    mbar_init(&sm->q_full, kOutWarps);
    mbar_init(&sm->q_free, 1);
    mbar_init(&sm->o_free, kOutWarps);
    mbar_init(&sm->drained, 1);
    sm->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&sm->tmem, 512);
  grid_dep_wait();
  grid_dep_launch();
  const ChunkHead head = *a.head;
  int first = 0, last = -1;
  if (blockIdx.x < head.blocks && head.items > 0) share_items(a, head, &first, &last);
  const int items = last - first + 1;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sm->tmem, 0);

  if (warp == kLoadWarp) {                 // ---- row blocks and keys
    bool ok = true;
    int g = 0, pairs = 0;                  // tiles sent for, and pairs of chunks of one more
    fence_proxy_async_global();            // (the decoded rows, by another kernel's plain stores)
    for (int e = 0; e < items && ok; ++e) {
      Item* it = &sm->item[e & 1];
      if (e >= 2) ok = wait_warp(sm, &sm->item_free[e & 1], ((e >> 1) - 1) & 1, a.spin);
      if (!ok) break;
      make_item(a, it, first + e, head.units, head.blocks);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->item_full[e & 1]);
      if (lane == 0) {
        const uint8_t* image = a.images + it->base * (2 * kD);
        const long long stride = it->stride;
        const int nt = it->nt, keys = it->keys, seen16 = it->seen16, raw0 = it->raw0;
        for (int t = 0; t < nt && ok; ++t) {
          const int k0 = (it->begin + t) * kTile, n = min(kTile, keys - k0);
          const int ne = max(0, min(n, seen16 - k0)), nr = n - ne;   // entries, raw rows (whole 16s)
          const uint8_t* from = image + static_cast<long long>(ne > 0 ? k0 : raw0 + k0 - seen16) * 256;
          const int stage = g & 1;
          uint8_t* to = ktile + stage * kStage;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            uint64_t* full = &sm->full[stage][m];
            if (g >= 2) ok = ok && wait_bar(sm, &sm->free_[stage][m], ((g >> 1) - 1) & 1, a.spin);
            if (ok) {
              mbar_expect_tx(full, n * 256);
              bulk_g2s(to + m * kPair, from + m * stride, (ne > 0 ? ne : nr) * 256, full);
              if (ne > 0 && nr > 0)
                bulk_g2s(to + m * kPair + ne * 256, image + m * stride + static_cast<long long>(raw0) * 256, nr * 256, full);
              pairs = m + 1;
            }
          }
          if (ok) { ++g; pairs = 0; }
        }
      }
      g = __shfl_sync(0xFFFFFFFFu, g, 0);
      pairs = __shfl_sync(0xFFFFFFFFu, pairs, 0);
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    }
    // copies in flight (there are none, unless a wait gave up): the last ones to each pair of chunks
    if (lane == 0) {
      for (int i = 0; i < 8; ++i) {
        const int stage = i >> 2, m = i & 3;
        const int sent = (g + 1 - stage) / 2 + (stage == (g & 1) && m < pairs);
        if (sent > 0) mbar_wait(&sm->full[stage][m], (sent - 1) & 1, kDefaultSpinLimit);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {           // ---- products
    if (elect_lane()) {
      const uint32_t ids = make_idesc(1, 1, 0, 0, 64, 64);
      const uint64_t dq = smem_desc_sw128(smem_u32(qtile), 16, 1024);
      const uint64_t dk = smem_desc_sw128(smem_u32(ktile), 16, 2048);
      const uint64_t dv = smem_desc_sw128(smem_u32(ktile), 1024, 2048);
      const uint64_t dp = smem_desc_sw128(smem_u32(ptile), 16, 1024);
      bool ok = true;
      int g = 0;
      for (int e = 0; e < items && ok; ++e) {
        ok = wait_bar(sm, &sm->item_full[e & 1], (e >> 1) & 1, a.spin);
        if (!ok) break;
        const Item* it = &sm->item[e & 1];
        const int nt = it->nt, keys = it->keys - it->begin * kTile;
        const uint32_t ido = make_idesc(1, 1, 1, 0, 128, 0) | (static_cast<uint32_t>(it->nq >> 3) << 17);
        ok = wait_bar(sm, &sm->q_full, e & 1, a.spin);
        tc_fence_after();
        // before this row block's first O product the outputs of the one before are read (a row block
        // without tiles waits too: its own outputs would be told from those by nothing)
        bool waited = e == 0;
        auto outputs_read = [&]() {
          if (!waited) {
            ok = ok && wait_bar(sm, &sm->o_free, (e - 1) & 1, a.spin);
            tc_fence_after();
            waited = true;
          }
        };
        if (nt == 0) {
          outputs_read();
          mma_commit(&sm->q_free);
        }
        for (int t = 0; t < nt && ok; t += 2) {
          const int two = min(2, nt - t);
          for (int u = 0; u < two && ok; ++u) {
            const int i = g + u, stage = i & 1;
            const uint64_t k = dk + stage * (kStage >> 4);
            const uint32_t d = tmem + kTmemS + 64 * stage;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              if ((c & 1) == 0) {
                ok = ok && wait_bar(sm, &sm->full[stage][c >> 1], (i >> 1) & 1, a.spin);
                tc_fence_after();
              }
              if (ok) issue_s_chunk(d, dq, k, c, ids);
            }
            mma_commit(&sm->s_full[stage]);
          }
          if (t + two == nt) mma_commit(&sm->q_free);
          outputs_read();
          for (int u = 0; u < two && ok; ++u) {
            const int i = g + u, stage = i & 1;
            const int ks = min(kTile, keys - (t + u) * kTile) >> 4;
            ok = ok && wait_bar(sm, &sm->p_full[stage], (i >> 1) & 1, a.spin);
            if (!ok) break;
            tc_fence_after();
            const uint64_t v = dv + stage * (kStage >> 4), p = dp + stage * (kChunk >> 4);
#pragma unroll
            for (int mb = 0; mb < 4; ++mb) {
              const uint64_t vb = v + mb * (kPair >> 4);
              if (t + u == 0) mma_set(tmem + mb * kRows, vb, p, ido);
              else mma_add(tmem + mb * kRows, vb, p, ido);
              if (ks == 4) {
#pragma unroll
                for (int k = 1; k < 4; ++k) mma_add(tmem + mb * kRows, vb + k * 256, p + 2 * k, ido);
              } else {
#pragma unroll 1
                for (int k = 1; k < ks; ++k) mma_add(tmem + mb * kRows, vb + k * 256, p + 2 * k, ido);
              }
              mma_commit(&sm->free_[stage][mb]);
            }
          }
          g += two;
        }
        mbar_arrive(&sm->item_free[e & 1]);
      }
      mma_commit(&sm->drained);   // before the tensor memory is given back (and shared memory)
      mbar_wait(&sm->drained, 0, kDefaultSpinLimit);
    }
    __syncwarp();
  } else if (warp < kSoftWarps) {          // ---- softmax
    int g = 0;
    for (int e = 0; e < items; ++e) {
      const bool there = wait_warp(sm, &sm->item_full[e & 1], (e >> 1) & 1, a.spin);
      if (role_any<kSoftId, kSoftWarps * 32>(!there)) break;
      const Item* it = &sm->item[e & 1];
      const int r = 16 * (warp & 3) + (lane >> 2);
      const RowSees sees[2] = {it->sees[r], it->sees[r + 8]};
      RowState s;
      s.reset();
      const int nt = it->nt;
      for (int t = 0; t < nt; ++t, ++g) weigh_tile(a, sm, it, ptile, tmem, g, it->begin + t, t == 0, sees, s);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          s.l[i] += __shfl_xor_sync(0xFFFFFFFFu, s.l[i], o);
          s.hat[i] += __shfl_xor_sync(0xFFFFFFFFu, s.hat[i], o);
        }
        if ((lane & 3) == 0)
          sm->sums[e & 1][warp >> 2][r + 8 * i] = make_float4(s.m[i] == -INFINITY ? -INFINITY : s.msub[i], s.l[i], s.hat[i], 0.f);
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm->l_full[e & 1]);
        mbar_arrive(&sm->item_free[e & 1]);
      }
    }
  } else {                                 // ---- queries and outputs
    int g = 0;
    auto item_there = [&](int e) {
      const bool there = wait_warp(sm, &sm->item_full[e & 1], (e >> 1) & 1, a.spin);
      return !role_any<kOutId, kOutThreads>(!there);
    };
    auto queries = [&](int e) {
      const Item* it = &sm->item[e & 1];
      request_queries(a, it, qtile);
      rotate_queries(a, it, qtile);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->q_full);
    };
    bool there = items > 0 && item_there(0);
    if (there) queries(0);
    for (int e = 0; e < items && there; ++e) {
      const Item* it = &sm->item[e & 1];
      g += it->nt;
      wait_warp(sm, &sm->q_free, e & 1, a.spin);   // the last S product on these queries is complete
      if (e + 1 < items) {
        there = item_there(e + 1);
        if (there) queries(e + 1);
      }
      wait_warp(sm, &sm->l_full[e & 1], (e >> 1) & 1, a.spin);
      finish_sums(a, it, sm, e);
      role_sync<kOutId, kOutThreads>();
      if (it->nt > 0) wait_warp(sm, &sm->free_[(g - 1) & 1][3], ((g - 1) >> 1) & 1, a.spin);
      tc_fence_after();
      write_rows(a, it, sm, tmem);
      tc_fence_before();
      role_sync<kOutId, kOutThreads>();   // (out_fac is read; this row block's sums too)
      if (lane == 0) {
        mbar_arrive(&sm->o_free);
        mbar_arrive(&sm->item_free[e & 1]);
      }
    }
    cp_async_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// the join: the parts of a row in order, the sink, the rotation back.  64 threads of 8 dims, four
// times as many, each with every fourth part, for a row.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;
constexpr int kShares = 4;

__global__ void __launch_bounds__(kJoinThreads) chunk_join_kernel(const __grid_constant__ ChunkArgs a) {
  __shared__ float shares[kShares - 1][kD];
  grid_dep_wait();
  const ChunkHead head = *a.head;
  const int share = threadIdx.x >> 6, lane = threadIdx.x & 31, d = (threadIdx.x & 63) * 8;
  for (int x = blockIdx.x; x < head.splits * kRows; x += gridDim.x) {
    const SplitPlan sp = a.split[x / kRows];
    const int r = x % kRows;
    const ReqPlan p = a.req[request_of_item(a, sp.item)];
    const int y = sp.item - p.item0;
    const int g = a.head_blocks == 1 ? y : y / a.head_blocks, h0 = a.head_blocks == 1 ? 0 : (y % a.head_blocks) * a.heads_per_block;
    const int nr = a.head_blocks == 1 ? min(p.nq - g * a.group, a.group) * a.H : min(a.heads_per_block, a.H - h0);
    if (r >= nr) continue;   // (the whole block)
    const size_t row = static_cast<size_t>(p.q0 + g * a.group) * a.H + h0 + r;
    const bool late = a.unit0[sp.item] > share_begin(head.units, head.blocks, sp.b0);
    const int parts = sp.b1 - sp.b0 + 1;
    auto slot = [&](int k) { return (2 * static_cast<size_t>(sp.b0 + k) + (k == 0 && late)) * kRows + r; };
    const float sink = a.sink != nullptr ? __ldg(a.sink + row % a.H) : -INFINITY;
    const float s2 = sink * kLog2e;
    auto weight = [&](float2 v, float M) { return v.y == 0.f ? 0.f : v.y != v.y ? v.y : exp2f(v.x - M); };
    float M = s2, total = 0.f, o[8];
    for (int k = lane; k < parts; k += 32) {
      const float2 v = a.ml[slot(k)];
      if (v.y != 0.f) M = fmaxf(M, v.x);
    }
    for (int w = 16; w >= 1; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, w));
    for (int k = lane; k < parts; k += 32) {
      const float2 v = a.ml[slot(k)];
      total += v.y * weight(v, M);
    }
    for (int w = 16; w >= 1; w >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = 0.f;
#pragma unroll 4
    for (int k = share; k < parts; k += kShares) {
      const float e = weight(a.ml[slot(k)], M);   // 0: a part without keys, whose output is 0
      const float4* v = reinterpret_cast<const float4*>(a.opart + slot(k) * kD + d);
      const float4 v0 = v[0], v1 = v[1];
      o[0] += e * v0.x; o[1] += e * v0.y; o[2] += e * v0.z; o[3] += e * v0.w;
      o[4] += e * v1.x; o[5] += e * v1.y; o[6] += e * v1.z; o[7] += e * v1.w;
    }
    if (share > 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) shares[share - 1][d + i] = o[i];
    }
    __syncthreads();
    if (share == 0) {
      for (int k = 0; k < kShares - 1; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += shares[k][d + i];
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
    __syncthreads();   // shares are used again
  }
}

inline size_t a256(size_t x) { return (x + 255) & ~size_t(255); }

// How the row blocks and the workspace follow from the sizes alone.
struct Layout {
  int group, head_blocks, heads_per_block, most_blocks;
  size_t head, req, unit0, split, flags, images, opart, ml, bytes;
};
Layout layout_of(int R, int T, int H, int64_t max_keys) {
  Layout l = {};
  l.head_blocks = (H + kRows - 1) / kRows;
  l.heads_per_block = (H + l.head_blocks - 1) / l.head_blocks;
  l.group = l.head_blocks == 1 ? kRows / H : 1;
  // each request's last row block may be a short one
  const int64_t items = (static_cast<int64_t>(T) / l.group + std::min(R, T)) * l.head_blocks;
  const int64_t tiles = items * ((max_keys + kTile - 1) / kTile + 1);
  l.most_blocks = static_cast<int>(std::min<int64_t>(kSms, std::max<int64_t>(1, (2 * tiles + kItemUnits * items) / kLeastShare)));
  const size_t keys = static_cast<size_t>(max_keys + 15) & ~size_t(15);
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t x = at; at += a256(bytes); return x; };
  l.head = take(sizeof(ChunkHead));
  l.req = take(sizeof(ReqPlan) * static_cast<size_t>(R));
  l.unit0 = take(8 * static_cast<size_t>(items + 1));
  l.split = take(sizeof(SplitPlan) * l.most_blocks);
  l.flags = take(keys);
  l.images = take(keys * (2 * kD));
  l.opart = take(2 * static_cast<size_t>(l.most_blocks) * kRows * kD * 4);
  l.ml = take(2 * static_cast<size_t>(l.most_blocks) * kRows * 8);
  l.bytes = at;
  return l;
}

template <class... Args>
cudaError_t launch_next(void (*kernel)(Args...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                        std::atomic<uint64_t>* allowed, const ChunkArgs& a) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return allowed != nullptr ? launch_with_shared_memory(cfg, kernel, *allowed, smem, a) : cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

size_t chunk_attn_workspace_bytes(int R, int T, int H, int64_t max_keys) { return layout_of(R, T, H, max_keys).bytes; }

cudaError_t launch_chunk_attn(const void* q, const int32_t* cu_q, const int32_t* ctx_len, int R, int T, int H,
                              const cskv_paged* entries, int ratio, const int32_t* n_entries, int max_entries,
                              const cskv_paged* rows, int window, int max_ctx, const float* sink, float scale,
                              const float* q_rope, void* out, float* lse, int64_t max_keys, void* workspace,
                              cudaStream_t stream) {
  const Layout l = layout_of(R, T, H, max_keys);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
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
  }
  if (rows != nullptr) {
    a.has_rows = 1;
    a.rows = *rows;
  }
  a.ratio = ratio;
  a.n_entries = n_entries;
  a.max_entries = max_entries;
  a.window = window;
  a.max_ctx = max_ctx;
  a.sink = sink;
  a.scale_log2 = scale * kLog2e;
  a.slack = std::min(kSlack / a.scale_log2, FLT_MAX);   // finite for the smallest scales too
  a.q_rope = q_rope;
  a.out = static_cast<uint8_t*>(out);
  a.lse = lse;
  a.max_keys = max_keys;
  a.group = l.group;
  a.head_blocks = l.head_blocks;
  a.heads_per_block = l.heads_per_block;
  a.most_blocks = l.most_blocks;
  a.head = reinterpret_cast<ChunkHead*>(ws + l.head);
  a.req = reinterpret_cast<ReqPlan*>(ws + l.req);
  a.unit0 = reinterpret_cast<long long*>(ws + l.unit0);
  a.split = reinterpret_cast<SplitPlan*>(ws + l.split);
  a.flags = ws + l.flags;
  a.images = ws + l.images;
  a.opart = reinterpret_cast<float*>(ws + l.opart);
  a.ml = reinterpret_cast<float2*>(ws + l.ml);
  a.spin = spin_limit();
  chunk_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t decode_warps = (max_keys + kDecodeRows - 1) / kDecodeRows;
  const unsigned decode_blocks = static_cast<unsigned>(
      std::min<int64_t>(8 * kSms, std::max<int64_t>(1, (decode_warps + kDecodeThreads / 32 - 1) / (kDecodeThreads / 32))));
  e = launch_next(chunk_decode_kernel, decode_blocks, kDecodeThreads, 0, stream, nullptr, a);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> allowed;
  e = launch_next(chunk_attn_kernel, l.most_blocks, kThreads, kChunkSmemBytes, stream, &allowed, a);
  if (e != cudaSuccess || l.most_blocks == 1) return e;
  return launch_next(chunk_join_kernel, 4 * kSms, kJoinThreads, 0, stream, nullptr, a);
}

unsigned int take_err_chunk_attn() { return take_dev_err(); }

}  // namespace cskv
