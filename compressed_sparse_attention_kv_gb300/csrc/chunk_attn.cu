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
// flops for each (query, head, key).  A 512-d fp32 output of more than 64 rows and the logits beside
// it do not fit an SM's tensor memory, and products of 64 rows are bound by shared memory (128
// bytes a cycle for operands): on one SM 36 products of 64 x 64 x 16 and 16 of 128 x 64 x 16 for 64 rows on
// 64 keys take 2,060 cycles (measured: 35 and 51 each), half of the tensor core's peak rate, and the
// copies' writes come on top.  Two SMs that share 128 rows and their keys read half of it:
// 36 products of 128 x 128 x 16 (34 cycles) and 16 of 256 x 128 x 16 (69) for 128 rows on 128 keys.
//
// Four kernels, each started while the one before it ends:
//   chunk_plan_kernel    the requests' key lists, the row blocks and their tiles as one line of
//                        work, cut into equal shares;
//   chunk_decode_kernel  every key that some query sees, once, from its paged row to bf16 in the
//                        order that the tensor core reads (the same rows are read by hundreds of row
//                        blocks: decoding a tile takes longer than its products);
//   chunk_attn_kernel    one pair of blocks (a cluster) per two SMs, its share of the work;
//   chunk_join_kernel    the row blocks that a share's border cuts in two or more.
//
// chunk_attn_kernel.  A row block is up to 128 rows of one request, 128 / H queries; the even block of
// the pair has the first half of its rows, the odd one the second.  The keys come in tiles of 128.
//   S  = Q K^T     each block gets its own rows x 128 keys; it holds its rows of Q and half of the
//                  tile's keys, all dims (64 KB);
//   O^T += V^T P^T each block gets all rows x two of the four blocks of 128 dims; it holds these dims of
//                  all the tile's keys (64 KB) and its own rows of P (16 KB).
// The products are issued for both by the even block.  Tensor memory: O in columns 0..255 (dims as
// lanes), the logits of two tiles behind it (rows as lanes, 64 to 127 with the second half of
// the keys).  Roles in each block:
//   warps 0-7    softmax of a tile: a thread has one row and 32 keys; P to shared memory;
//   warps 8-15   the next row block's queries (loaded and rotated while the last products of this one
//                run), and the outputs;
//   warp 16      in the even block one thread issues the products, S of the next tile before O of this
//                one, so that the softmax runs beside products; in the odd block one thread tells the
//                even one which copies have arrived;
//   warp 17      sends for the keys (bulk copies of a block of 128 dims), as soon as the product on the
//                same place's keys before is complete;
//   warp 18      plans the row blocks, two at a time.
// A row's reference belongs to its block, its output's columns to both: when a reference moves, the
// factors go to the other block's shared memory, and a flag for every tile says whether they did.
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
constexpr int kTile = 128;                // keys of a tile
constexpr int kRows = 64;                 // rows of a block, at most; a row block has twice as many
constexpr int kChunk = kRows * 128;       // bytes of 64 dims of the queries, of 64 keys of P
constexpr int kKeyPart = 64 * 256;        // bytes of 128 dims of half a tile: groups of 8 keys, each [64 dims][8 keys][128 B] twice
constexpr int kDimPart = kTile * 256;     // of a tile
constexpr int kSoftWarps = 8, kOutWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kOutWarps, kLoadWarp = kMmaWarp + 1, kPlanWarp = kMmaWarp + 2;
constexpr int kThreads = (kPlanWarp + 1) * 32;
constexpr int kOutThreads = kOutWarps * 32;
constexpr uint32_t kTmemS = 256;          // TMEM columns: O 0..255, S from here, 64 for each tile
constexpr float kSlack = 8.0f;            // base 2
constexpr int kPairs = 76;                // of SMs
constexpr int kPlanThreads = 1024;
constexpr int kPlanItems = 4;             // row blocks of a thread at a time
constexpr int kItemUnits = 3;             // a row block's cost beside its tiles, a tile being 2
constexpr int kLeastShare = 8;            // units of a share
constexpr unsigned long long kDrainLimit = 1ull << 27;   // cycles that a block which gives up waits for its own copies

struct ReqPlan {
  int q0, nq, len;          // its queries [q0, q0 + nq), its length
  int entries, entries16;   // entries that count, and rounded up to 16 (decoded rows)
  int row0, rows, rows16;   // its first decoded raw row, how many, rounded up
  long long base;           // its first decoded row
  int item0;                // its first row block
  int bad;                  // a row of it could not be read or is not finite
};
struct SharePlan {
  int first, last;          // the row blocks of a pair's share
};
struct SplitPlan {
  int item, b0, b1, pad;    // a row block that pairs b0 .. b1 share
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
  int group;                // queries of a row block
  int most_blocks;          // shares at most
  // workspace
  ChunkHead* head;
  ReqPlan* req;
  long long* unit0;         // [items + 1]
  SharePlan* share;         // [most_blocks]
  SplitPlan* split;         // [most_blocks]
  uint8_t* flags;           // of every decoded row: 0, kNone, kUnfit
  uint8_t* images;          // decoded rows: of each request 4 blocks of 128 dims as they lie in a stage
  float* opart;             // [2 * most_blocks][2 * kRows][512]
  float2* ml;               // [2 * most_blocks][2 * kRows]: m (base 2) and l
  unsigned long long spin;
};
constexpr uint8_t kNone = 1, kUnfit = 2;

__host__ __device__ inline int up16(int n) { return (n + 15) & ~15; }
// Products of a pair of blocks have whole 32s of columns: each block has half of a tile's keys, rounded
// up to 16 (columns behind the last key are seen by nobody).
__device__ __forceinline__ int half_keys(int n) { return up16((n + 1) / 2); }

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
  k.i0 = x * a.group;
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

// Shares: pair b has the units [units * b / blocks, units * (b + 1) / blocks); tile t of a row block
// begins at its unit 2 t and belongs to the pair that has this unit.
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

constexpr int kPlanStaged = 4096;         // row blocks whose places are searched in shared memory

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ ChunkArgs a) {
  __shared__ long long part[32], staged[kPlanStaged];
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
    const int blocks = (p.nq + a.group - 1) / a.group;
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
      if (e1 + u < items) {
        a.unit0[e1 + u] = at;
        if (e1 + u < kPlanStaged) staged[e1 + u] = at;
      }
      at += mine[u];
    }
  }
  if (tid == 0) {
    a.unit0[items] = units;
    if (items < kPlanStaged) staged[items] = units;
  }
  __syncthreads();
  const int blocks = static_cast<int>(max(1ll, min(static_cast<long long>(a.most_blocks), units / kLeastShare)));
  // the row blocks of each share; those that a border cuts are listed at the last border inside
  if (items == 0) {
    if (tid == 0) a.share[0] = SharePlan{0, -1};
  } else if (tid == 0) {
    a.share[0].first = 0;
    a.share[blocks - 1].last = static_cast<int>(items) - 1;
  }
  const long long* unit0 = items < kPlanStaged ? staged : a.unit0;
  int splits = 0;
  for (int b0 = 1; b0 < blocks; b0 += kPlanThreads) {
    const int b = b0 + tid;
    bool last = false;
    int e = 0;
    if (b < blocks) {
      const long long u = share_begin(units, blocks, b);
      e = item_of_unit(unit0, static_cast<int>(items), u);
      const int tiles = (static_cast<int>(unit0[e + 1] - unit0[e]) - kItemUnits) / 2;
      const long long end = unit0[e] + 2ll * (tiles - 1);   // its last tile
      a.share[b].first = e + (end < u);                     // (its tiles are all before the border)
      a.share[b - 1].last = e - (unit0[e] == u);
      last = u > unit0[e] && u <= end && block_of_unit(units, blocks, end) == b;
    }
    const long long at = splits + block_scan(last, part, &total) - 1;
    if (last) a.split[at] = SplitPlan{e, block_of_unit(units, blocks, unit0[e]), b, 0};
    splits += static_cast<int>(total);
  }
  if (tid == 0) *a.head = ChunkHead{static_cast<int>(items), blocks, splits, 0, units, keys};
}

// ---------------------------------------------------------------------------
// the keys
// ---------------------------------------------------------------------------
constexpr int kDecodeThreads = 256;
constexpr int kDecodeRows = 8;    // of a warp at a time: a group of the image (a request's rows are whole 16s)

// The bytes of 16 neighbouring dims of a row, and their scale.
template <int FMT>
struct RawRow;
template <>
struct RawRow<CSKV_FMT_BF16> {
  uint4 x, y;
  __device__ __forceinline__ void load(const uint8_t* row, int lane) {
    x = __ldg(reinterpret_cast<const uint4*>(row) + 2 * lane);
    y = __ldg(reinterpret_cast<const uint4*>(row) + 2 * lane + 1);
  }
  __device__ __forceinline__ void to_bf16(uint32_t (&w)[8]) const {
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
  }
};
template <>
struct RawRow<CSKV_FMT_FP8_E4M3_E8M0_B32> {
  uint4 codes;
  uint32_t scale;
  __device__ __forceinline__ void load(const uint8_t* row, int lane) {
    codes = __ldg(reinterpret_cast<const uint4*>(row) + lane);
    scale = __ldg(row + kD + (lane >> 1));
  }
  __device__ __forceinline__ void to_bf16(uint32_t (&w)[8]) const { convert(codes, scale, w); }
};
template <>
struct RawRow<CSKV_FMT_FP4_E2M1_E4M3_B16> {
  uint2 codes;
  uint32_t scale;
  __device__ __forceinline__ void load(const uint8_t* row, int lane) {
    codes = __ldg(reinterpret_cast<const uint2*>(row) + lane);
    scale = __ldg(row + kD / 2 + lane);
  }
  __device__ __forceinline__ void to_bf16(uint32_t (&w)[8]) const { convert(codes, scale, w); }
};

// Eight rows (lane i < 8 has row i's address, nullptr: none) into their group of the image; returns
// a bit for each that is not finite, whose values become 0.  All loads are on their way before the
// first is used.
template <int FMT>
__device__ __forceinline__ uint32_t decode_rows(const uint8_t* mine, uint8_t* image) {
  const int lane = threadIdx.x & 31;
  RawRow<FMT> raw[kDecodeRows] = {};
#pragma unroll
  for (int i = 0; i < kDecodeRows; ++i) {
    const uint8_t* row = reinterpret_cast<const uint8_t*>(
        __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(mine), i));
    if (row != nullptr) raw[i].load(row, lane);
  }
  const uint32_t there = __ballot_sync(0xFFFFFFFFu, mine != nullptr);
  uint32_t unfit = 0;
#pragma unroll
  for (int i = 0; i < kDecodeRows; ++i) {
    uint32_t w[8] = {}, bad = 0;
    if ((there >> i) & 1u) raw[i].to_bf16(w);
#pragma unroll
    for (int k = 0; k < 8; ++k) bad |= ((w[k] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
    if (__any_sync(0xFFFFFFFFu, bad != 0u)) {   // (an exponent of all ones carries into the sign bit)
      unfit |= 1u << i;
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = 0u;
    }
    const int at = 2 * (lane & 3);
    uint8_t* to = image + i * 128;
    *reinterpret_cast<uint4*>(to + ((at ^ i) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(to + (((at + 1) ^ i) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
  }
  return unfit;
}

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
    const bool exists = lane < kDecodeRows && k0 + lane < have;
    const uint8_t* mine = nullptr;
    if (exists) mine = paged_row(c, r, (raw ? p.row0 : 0) + static_cast<long long>(k0) + lane, row_bytes).data;
    uint8_t* image = a.images + p.base * (2 * kD) + (lane >> 3) * (rows * 256) + static_cast<long long>(first) * 256 +
                     ((lane >> 2) & 1) * 1024;
    const uint32_t unfit = c.fmt == CSKV_FMT_BF16 ? decode_rows<CSKV_FMT_BF16>(mine, image)
                           : c.fmt == CSKV_FMT_FP8_E4M3_E8M0_B32 ? decode_rows<CSKV_FMT_FP8_E4M3_E8M0_B32>(mine, image)
                                                                : decode_rows<CSKV_FMT_FP4_E2M1_E4M3_B16>(mine, image);
    if (lane < kDecodeRows) a.flags[x + lane] = mine == nullptr ? kNone : (unfit >> lane) & 1u ? kUnfit : 0;
    // a row that is there and cannot be used (those behind the last one are seen by nobody)
    if (__any_sync(0xFFFFFFFFu, exists && mine == nullptr) || unfit != 0u) {
      if (lane == 0) a.req[r].bad = 1;
    }
  }
}

// ---------------------------------------------------------------------------
// the attention kernel
// ---------------------------------------------------------------------------
struct __align__(16) RowSees {   // key k of the block's list is seen when k < seen or lo <= k <= hi
  int seen, lo, hi, pad;
};

struct Item {
  int row0, rows, half;          // rows [row0, row0 + rows) of the [T * H] rows, the first `half` of them in the even block
  int r0, nr;                    // this block's
  int nq;                        // columns of O for a block's rows: half, rounded up to 16
  int t0, one;                   // the first row's query; all rows are that query's
  int seen16, raw0, keys;        // the list (BlockKeys); raw0 counted among all decoded rows of the request
  int begin, nt;                 // this pair's tiles
  int plain;                     // keys below it are seen by every row
  int bad;
  int part;                      // partial output, -1: none
  long long base, stride;        // the request's first decoded row, bytes between its blocks of dims
  RowSees sees[kRows];
};

struct ChunkSmem {
  Item item[2];
  uint64_t k_full[4], k_free[4];           // keys: blocks of 128 dims
  uint64_t v_full[2], v_free[2];           // this block's dims
  uint64_t s_full[2], moved[2], p_full, q_full, q_free, o_free[2], l_full[2], f_full[2], item_full[2], item_free[2], drained;
  uint32_t tmem;
  int abort;
  int flag[2];                             // by tile: the other block's references moved
  __align__(16) float fac[2][2][kRows];    // by tile and block: a moved reference's factors
  float top[4][kRows];                     // a tile's largest logits, of each quarter of its keys
  float ref[2][kRows];                     // of a row block: m (base 2)
  float2 sums[2][4][kRows];                // and of a quarter of its keys: l, the sum of the rounded weights
  __align__(16) float out_fac[2][2][kRows];   // of a row block, by block
};

// Another block of the cluster's shared memory.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t of_block(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
// 4 bytes into it, counted on its barrier (the wait for the barrier is all that they need).
__device__ __forceinline__ void send_to(uint32_t at, uint32_t v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(at), "r"(v), "r"(bar) : "memory");
}
// Says that something is done: what the products read (P and the queries in their own block's shared
// memory, tensor memory) is ordered before it by the proxy and tcgen05 fences.  With a release at
// cluster scope, which waits for every write of the warp, a tile took 1.8 times as long.
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Products for both blocks of the pair (issued by the even one) and their completion, on the barrier
// of both.
__device__ __forceinline__ void mma2_add(uint32_t d, uint64_t da, uint64_t db, uint32_t id) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, 0, 0;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(da), "l"(db), "r"(id)
      : "memory");
}
__device__ __forceinline__ void mma2_set(uint32_t d, uint64_t da, uint64_t db, uint32_t id) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, 0, 0;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(da), "l"(db), "r"(id)
      : "memory");
}
__device__ __forceinline__ void mma2_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
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
// a role's warps take the same loops (a row block is accepted by all or by none; after a wait that gave
// up a warp goes on through its tiles to these barriers alone).
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

// Row block e of this pair's share, and this block's rows of it; one warp.
__device__ void make_item(const ChunkArgs& a, Item* it, int e, long long units, int blocks, int pair, int rank) {
  const int lane = threadIdx.x & 31;
  const ReqPlan p = a.req[request_of_item(a, e)];
  const BlockKeys k = block_keys(a, p, e - p.item0);
  const int rows = (k.i1 - k.i0) * a.H, half = (rows + 1) / 2;
  const int at = rank == 0 ? 0 : half, nr = rank == 0 ? half : rows - half;   // of the row block
  const int raw0 = k.raw0 + p.row0;   // position of the list's first raw row
  int least = INT32_MAX;
  for (int r = lane; r < kRows; r += 32) {
    RowSees s{0, 0, -1, 0};
    if (r < nr) {
      const int pos1 = p.len - p.nq + k.i0 + (at + r) / a.H + 1;
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
    it->one = k.i1 - k.i0 == 1;
    it->row0 = it->t0 * a.H;
    it->rows = rows;
    it->half = half;
    it->r0 = it->row0 + at;
    it->nr = nr;
    it->nq = up16(half);
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
    const long long lo = share_begin(units, blocks, pair), hi = share_begin(units, blocks, pair + 1);
    const int begin = static_cast<int>(min(static_cast<long long>(tiles), max(0ll, (lo - u0 + 1) / 2)));
    const int end = static_cast<int>(min(static_cast<long long>(tiles), max(0ll, (hi - u0 + 1) / 2)));
    it->begin = begin;
    it->nt = end - begin;
    it->part = begin > 0 || end < tiles ? 2 * pair + (u0 > lo) : -1;
  }
}

// Queries into the K-major chunks of Q (64 rows apart; rows behind the last one zero); the output
// warps.  The last 64 dims are then rotated in place: chunk 7 holds the first bf16 of each rotated
// value, chunk 8 the second.  (The angles are on their way while the queries are awaited: loaded row by
// row, they took 5,600 cycles.)
__device__ __forceinline__ void load_queries(const ChunkArgs& a, const Item* it, uint8_t* qtile) {
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
  static_assert(kRows * 8 == 2 * kOutThreads, "a thread rotates 8 dims of two rows");
  float4 cs[2][2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = (tid >> 3) + 32 * u;
    if (r < nr) {
      const float4* from = reinterpret_cast<const float4*>(
          a.q_rope + static_cast<size_t>(static_cast<unsigned>(it->r0 + r) / static_cast<unsigned>(a.H)) * 64 + (tid & 7) * 8);
      cs[u][0] = __ldg(from);
      cs[u][1] = __ldg(from + 1);
    }
  }
  cp_async_wait_all();
  role_sync<kOutId, kOutThreads>();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = (tid >> 3) + 32 * u, c = tid & 7;
    uint4 lo = make_uint4(0u, 0u, 0u, 0u);
    if (r < nr) {
      uint4* hi = reinterpret_cast<uint4*>(qtile + 7 * kChunk + sw128_offset(r, c));
      const float co[4] = {cs[u][0].x, cs[u][0].z, cs[u][1].x, cs[u][1].z}, si[4] = {cs[u][0].y, cs[u][0].w, cs[u][1].y, cs[u][1].w};
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
    *reinterpret_cast<uint4*>(qtile + 8 * kChunk + sw128_offset(r, c)) = lo;
  }
  fence_proxy_async_smem();
}

// A softmax thread's state of its row.
struct RowState {
  float m, limit, msub;   // reference in units of q'.c; a logit above limit moves it; in base 2
  float l, hat;           // this thread's sums of the weights, and of the rounded ones
  __device__ __forceinline__ void reset() {
    m = limit = -INFINITY;
    msub = l = hat = 0.f;
  }
};

// Logits of the keys k0 .. k0 + 31 that the row does not see become -inf, those of unfit rows NaN.
__device__ __forceinline__ void mask_keys(const ChunkArgs& a, const Item* it, int k0, const RowSees& s, float (&z)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const int k = k0 + j;
    if (!(k < s.seen || (k >= s.lo && k <= s.hi))) z[j] = -INFINITY;
  }
  if (it->bad) {
#pragma unroll 1
    for (int j0 = 0; j0 < 32; j0 += 8) {   // eight rows' flags lie together (k0 and the list's parts are whole 8s)
      const int k = k0 + j0;
      if (k >= it->keys) break;
      const uint8_t* at = a.flags + it->base + (k < it->seen16 ? k : it->raw0 + k - it->seen16);
      const uint2 f = *reinterpret_cast<const uint2*>(at);
      if ((f.x | f.y) == 0u) continue;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        if ((j & ~7) != j0) continue;
        const uint32_t x = byte_of((j & 4) ? f.y : f.x, j & 3);
        if (x == kNone) z[j] = -INFINITY;
        if (x == kUnfit && z[j] != -INFINITY) z[j] = __int_as_float(0x7FC00000);
      }
    }
  }
}

// The softmax of the pair's tile g, the row block's tile t: this thread's row and 32 keys.
__device__ __forceinline__ void weigh_tile(const ChunkArgs& a, ChunkSmem* sm, const Item* it, uint8_t* ptile, uint32_t tmem,
                                           int rank, int g, int t, bool first, const RowSees& sees, RowState& s, bool& ok) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, side = warp >> 2;        // lanes of tensor memory; columns 32 side .. + 31
  const int r = 32 * (quarter & 1) + lane;
  const uint32_t tlane = static_cast<uint32_t>(quarter * 32) << 16;
  const int buf = g & 1;
  const int n2 = half_keys(min(kTile, it->keys - t * kTile));
  const int c0 = 32 * side;                              // the thread's first key within its half
  const int k0 = (quarter >> 1) * n2 + c0;               // within the tile
  ok = ok && wait_warp(sm, &sm->s_full[buf], (g >> 1) & 1, a.spin);
  const bool has = ok && c0 < n2;
  tc_fence_after();
  float z[32];
  if (has) {
    tmem_ld32(tmem + kTmemS + 64 * buf + c0 + tlane, z);
    tmem_wait_ld();
    if (n2 - c0 < 32) {   // a short tile: columns behind its last key
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (c0 + j >= n2) z[j] = -INFINITY;
    }
    if (t * kTile + k0 + 32 > it->plain || it->bad) mask_keys(a, it, t * kTile + k0, sees, z);
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) z[j] = -INFINITY;
  }
  float top = z[0];
#pragma unroll
  for (int j = 1; j < 32; ++j) top = fmaxf(top, z[j]);
  float fac = 1.f;
  const bool moves = role_any<kSoftId, kSoftWarps * 32>(top > s.limit);
  if (moves) {   // some row's reference moves
    sm->top[2 * side + (quarter >> 1)][r] = top;
    role_sync<kSoftId, kSoftWarps * 32>();
    const float now = fmaxf(fmaxf(fmaxf(sm->top[0][r], sm->top[1][r]), fmaxf(sm->top[2][r], sm->top[3][r])), s.m);
    const float sub = now == -INFINITY ? 0.f : __fmul_rn(now, a.scale_log2);
    const float f = s.m == -INFINITY ? 0.f : exp2f(s.msub - sub);
    s.m = now;
    s.limit = now + a.slack;
    s.msub = sub;
    s.l *= f;
    s.hat *= f;
    if (side == 0 && quarter < 2) sm->fac[buf][rank][r] = fac = f;
    role_sync<kSoftId, kSoftWarps * 32>();
  }
  if (!ok) return;
  // to the other block: each row's factor, and whether there is one
  const uint32_t theirs = of_block(&sm->moved[buf], rank ^ 1);
  if (side == 0 && quarter < 2) send_to(of_block(&sm->fac[buf][rank][r], rank ^ 1), __float_as_uint(fac), theirs);
  if (threadIdx.x == 0) {
    send_to(of_block(&sm->flag[buf], rank ^ 1), moves, theirs);
    mbar_expect_tx(&sm->moved[buf], kRows * 4 + 4);
  }
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float x = exp2_fast(fmaf(z[2 * j], a.scale_log2, -s.msub));
    const float y = exp2_fast(fmaf(z[2 * j + 1], a.scale_log2, -s.msub));
    w[j] = pack_bf16(x, y);
    s.l += x + y;
    s.hat += bf16lo(w[j]) + bf16hi(w[j]);
  }
  // the O product before has read P, and its output may be rescaled
  if (g > 0) {
    ok = wait_warp(sm, &sm->v_free[1], (g - 1) & 1, a.spin);
    tc_fence_after();
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = k0 + 8 * j;
    if (c0 + 8 * j < n2)
      *reinterpret_cast<uint4*>(ptile + (k >> 6) * kChunk + r * 128 + ((((k >> 3) & 7) ^ (r & 7)) << 4)) =
          make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  }
  ok = ok && wait_warp(sm, &sm->moved[buf], (g >> 1) & 1, a.spin);
  if (!ok) return;
  if (!first) {
    const bool other = *reinterpret_cast<volatile int*>(&sm->flag[buf]) != 0;
#pragma unroll 1
    for (int u = 0; u < 2; ++u) {
      if (!(u == rank ? moves : other)) continue;
#pragma unroll 1
      for (int x = 0; x < it->nq; x += 16) {   // 32 dims of block `side`, 16 rows at a time
        float o[16];
        const uint32_t at = tmem + tlane + side * (2 * kRows) + u * it->nq + x;
        tmem_ld16(at, o);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) o[c] *= sm->fac[buf][u][x + c];
        tmem_st16(at, o);
      }
      tmem_wait_st();
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) arrive_at(of_block(&sm->p_full, 0));
}

// Block j of O^T out (128 dims x all rows of the row block), 16 rows at a time: a thread has one dim, a
// row's 32 dims of a warp are one 64-byte run; warps 8-11 have the even block's rows, 12-15 the odd one's.
// `read` is called once the block is out of tensor memory: the next row block's products go on with
// it while the other block is read.  Dims 448..511 are turned back on the way: even lanes have the
// pair of dims (d, d + 1) of row c, odd lanes (d - 1, d) of row c + 1.  A partial output goes out in fp32 as
// it is.  (Rolled: with all 64 rows unrolled the block's first outputs waited 12,000 cycles for
// instructions.)
template <class Read>
__device__ __forceinline__ void write_block(const ChunkArgs& a, const Item* it, ChunkSmem* sm, uint32_t tmem, int rank, int e,
                                            int j, Read&& read) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, u = (warp - kSoftWarps) >> 2, odd = lane & 1;
  const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + j * (2 * kRows) + u * it->nq;
  const int at = u == 0 ? 0 : it->half, rows = u == 0 ? it->half : it->rows - it->half;   // of the row block
  const unsigned row0 = it->row0 + at, H = a.H;
  const int d = (2 * j + rank) * 128 + quarter * 32 + lane;
  const bool whole = it->part < 0, turn = whole && d >= kD - 64, tiles = it->nt > 0;
  // the angles of the thread's pair of dims for its row's query, and for the next query, on their way
  const float2* cs = reinterpret_cast<const float2*>(a.q_rope) + ((d - (kD - 64)) >> 1);
  const unsigned final_query = rows > 0 ? (row0 + rows - 1) / H : 0;
  unsigned query = (row0 + odd) / H, border = (query + 1) * H;
  float2 w = make_float2(1.f, 0.f), next = w;
  if (turn && rows > 0) {
    w = __ldg(cs + static_cast<size_t>(min(query, final_query)) * 32);
    next = __ldg(cs + static_cast<size_t>(min(query + 1, final_query)) * 32);
  }
  float* part = whole ? nullptr : a.opart + (static_cast<size_t>(it->part) * (2 * kRows) + at) * kD + d;
  uint8_t* out = a.out + (static_cast<size_t>(row0) * kD + d) * 2;
#pragma unroll 1
  for (int g = 0; g < rows; g += 16) {
    float o[16];
    if (tiles) {
      tmem_ld16(from + g, o);   // (columns behind the last row hold nothing of use)
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c) o[c] = 0.f;
    }
    if (g + 16 >= rows) read();
    const int left = rows - g;
#pragma unroll
    for (int c = 0; c < 16; c += 4) {
      const float4 f = *reinterpret_cast<const float4*>(&sm->out_fac[e & 1][u][g + c]);
      o[c] *= f.x;
      o[c + 1] *= f.y;
      o[c + 2] *= f.z;
      o[c + 3] *= f.w;
    }
    if (!whole) {
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (c < left) part[(g + c) * kD] = o[c];
    } else if (turn) {
      uint8_t* to = out + (static_cast<size_t>(g + odd) * kD - odd) * 2;
#pragma unroll
      for (int c = 0; c < 16; c += 2) {
        while (row0 + g + c + odd >= border && query < final_query) {
          w = next;
          ++query;
          border += H;
          next = __ldg(cs + static_cast<size_t>(min(query + 1, final_query)) * 32);
        }
        const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? o[c] : o[c + 1], 1);
        const float y0 = odd ? other : o[c], y1 = odd ? o[c + 1] : other;
        if (c + odd < left) *reinterpret_cast<uint32_t*>(to + c * (2 * kD)) = pack_bf16(y0 * w.x + y1 * w.y, y1 * w.x - y0 * w.y);
      }
    } else {
      uint16_t* to = reinterpret_cast<uint16_t*>(out) + g * kD;
#pragma unroll
      for (int c = 0; c < 16; c += 2) {
        const uint32_t v = pack_bf16(o[c], o[c + 1]);
        if (c < left) to[c * kD] = static_cast<uint16_t>(v);
        if (c + 1 < left) to[(c + 1) * kD] = static_cast<uint16_t>(v >> 16);
      }
    }
  }
  if (rows == 0) read();
}

// The factors that this block's rows' outputs take (to both blocks), their log-sum-exps or partial sums.
__device__ __forceinline__ void finish_sums(const ChunkArgs& a, const Item* it, ChunkSmem* sm, int rank, int e) {
  const int r = threadIdx.x - kSoftWarps * 32;
  if (r >= kRows) return;
  float f = 0.f;
  if (r < it->nr) {
    const float m = sm->ref[e & 1][r];
    float2 s = sm->sums[e & 1][0][r];
#pragma unroll
    for (int k = 1; k < 4; ++k) {
      const float2 more = sm->sums[e & 1][k][r];
      s.x += more.x;
      s.y += more.y;
    }
    const unsigned row = it->r0 + r;
    // the output is made of rounded weights: over their own sum a few large ones' roundings cancel
    const float ratio = s.x == 0.f ? 1.f : s.x / s.y;
    if (it->part >= 0) {
      a.ml[static_cast<size_t>(it->part) * (2 * kRows) + (it->r0 - it->row0) + r] = make_float2(m, s.x);
      f = ratio;
    } else {
      const float sink = a.sink != nullptr ? __ldg(a.sink + row % static_cast<unsigned>(a.H)) : -INFINITY;
      const float s2 = __fmul_rn(sink, kLog2e);   // (not part of a fused difference: s2 - M is 0 where s2 is the larger)
      const float M = fmaxf(m, s2);
      const float w = exp2f(m - M);
      const float total = s.x * w + (s2 == -INFINITY ? 0.f : exp2f(s2 - M));
      // no key, or a sink above fp32 in base 2 (which leaves the keys nothing): out 0, lse the sink itself
      const bool none = s.x == 0.f || s2 == INFINITY;
      f = none ? 0.f : w / total * ratio;
      if (s.x != s.x) f = s.x;
      if (a.lse != nullptr) a.lse[row] = none ? sink : s.x != s.x ? s.x : (M + log2f(total)) * kLn2;
    }
  }
  float* to = &sm->out_fac[e & 1][rank][r];
  *to = f;
  send_to(of_block(to, rank ^ 1), __float_as_uint(f), of_block(&sm->f_full[e & 1], rank ^ 1));
  if (r == 0) mbar_expect_tx(&sm->f_full[e & 1], kRows * 4);
}

// S of a tile: 64 dims (chunk c) of the queries and the keys, with chunk 7 the second halves of its
// rotated queries
__device__ __forceinline__ void issue_s_chunk(uint32_t d, uint64_t dq, uint64_t dk, int c, uint32_t id) {
  const uint64_t q = dq + c * (kChunk >> 4), k = dk + (c >> 1) * (kKeyPart >> 4) + (c & 1) * (1024 >> 4);
  if (c == 0) mma2_set(d, q, k, id);
  else mma2_add(d, q, k, id);
#pragma unroll
  for (int x = 1; x < 4; ++x) mma2_add(d, q + 2 * x, k + 2 * x, id);
  if (c == 7) {
#pragma unroll
    for (int x = 0; x < 4; ++x) mma2_add(d, q + (kChunk >> 4) + 2 * x, k + 2 * x, id);
  }
}

// `rows` rows of the list from `k` on, `bytes` each of 16 (a block of dims at `image`, 256 bytes a row)
// into shared memory: entries, raw rows, or both.
__device__ __forceinline__ void send_for(const Item* it, uint8_t* to, const uint8_t* image, int k, int rows, uint64_t* full) {
  const int ne = max(0, min(rows, it->seen16 - k)), nr = rows - ne;
  if (ne > 0) bulk_g2s(to, image + static_cast<long long>(k) * 256, ne * 256, full);
  if (nr > 0)
    bulk_g2s(to + ne * 256, image + static_cast<long long>(it->raw0 + k + ne - it->seen16) * 256, nr * 256, full);
}

constexpr size_t kChunkSmemBytes = 1024 + 9 * size_t(kChunk) + 4 * size_t(kKeyPart) + 2 * size_t(kDimPart) + 2 * size_t(kChunk) + sizeof(ChunkSmem);
static_assert(kChunkSmemBytes <= 227 * 1024, "one block per SM");

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) chunk_attn_kernel(const __grid_constant__ ChunkArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* qtile = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);   // 9 chunks (the same place in both blocks)
  uint8_t* ktile = qtile + 9 * kChunk;       // half a tile's keys, four blocks of 128 dims
  uint8_t* vtile = ktile + 4 * kKeyPart;     // a tile's keys, two blocks of 128 dims
  uint8_t* ptile = vtile + 2 * kDimPart;     // this block's rows x 2 x 64 keys
  ChunkSmem* sm = reinterpret_cast<ChunkSmem*>(ptile + 2 * kChunk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = cluster_rank(), pair = blockIdx.x >> 1;

  if (tid == 0) {
    const int both = rank == 0 ? 2 : 1;      // the even block hears of the odd one's copies
    for (int m = 0; m < 4; ++m) {
      mbar_init(&sm->k_full[m], both);
      mbar_init(&sm->k_free[m], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->v_full[i], both);
      mbar_init(&sm->v_free[i], 1);
      mbar_init(&sm->s_full[i], 1);
      mbar_init(&sm->moved[i], 1);
      mbar_init(&sm->l_full[i], kSoftWarps);
      mbar_init(&sm->f_full[i], 1);
      mbar_init(&sm->item_full[i], 1);
      mbar_init(&sm->item_free[i], 2 + kSoftWarps + kOutWarps);
    }
    mbar_init(&sm->p_full, 2 * kSoftWarps);
    mbar_init(&sm->q_full, 2 * kOutWarps);
    mbar_init(&sm->q_free, 1);
    for (int j = 0; j < 2; ++j) mbar_init(&sm->o_free[j], 2 * kOutWarps);
    mbar_init(&sm->drained, 1);
    sm->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm->tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  grid_dep_wait();
  grid_dep_launch();
  const ChunkHead head = *a.head;
  const SharePlan share = pair < head.blocks ? a.share[pair] : SharePlan{0, -1};
  const int items = share.last - share.first + 1;
  tc_fence_before();
  __syncthreads();
  cluster_sync();                          // the other block's barriers are there
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sm->tmem, 0);

  if (warp == kPlanWarp) {                 // ---- row blocks
    for (int e = 0; e < items; ++e) {
      if (e >= 2 && !wait_warp(sm, &sm->item_free[e & 1], ((e >> 1) - 1) & 1, a.spin)) break;
      make_item(a, &sm->item[e & 1], share.first + e, head.units, head.blocks, pair, rank);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->item_full[e & 1]);
    }
  } else if (warp == kLoadWarp) {          // ---- keys
    if (elect_lane()) {
      bool ok = true;
      int gk = 0, gv = 0, parts = 0;         // tiles sent for: keys, dims; and parts of one more (4 + of dims)
      fence_proxy_async_global();            // (the decoded rows, by another kernel's plain stores)
      auto send_keys = [&](const Item* it, int t) {
        const int k0 = (it->begin + t) * kTile, n = min(kTile, it->keys - k0), n2 = half_keys(n);
        const int mine = rank == 0 ? min(n, n2) : n - min(n, n2);
        const uint8_t* image = a.images + it->base * (2 * kD);
#pragma unroll 1
        for (int m = 0; m < 4 && ok; ++m) {
          if (gk > 0) ok = wait_bar(sm, &sm->k_free[m], (gk - 1) & 1, a.spin);
          if (!ok) break;
          mbar_expect_tx(&sm->k_full[m], mine * 256);
          send_for(it, ktile + m * kKeyPart, image + m * it->stride, k0 + rank * n2, mine, &sm->k_full[m]);
          parts = m + 1;
        }
        if (ok) { ++gk; parts = 0; }
      };
      auto send_dims = [&](const Item* it, int t) {
        const int k0 = (it->begin + t) * kTile, n = min(kTile, it->keys - k0);
        const uint8_t* image = a.images + it->base * (2 * kD);
#pragma unroll 1
        for (int j = 0; j < 2 && ok; ++j) {
          if (gv > 0) ok = wait_bar(sm, &sm->v_free[j], (gv - 1) & 1, a.spin);
          if (!ok) break;
          mbar_expect_tx(&sm->v_full[j], n * 256);
          send_for(it, vtile + j * kDimPart, image + (2 * j + rank) * it->stride, k0, n, &sm->v_full[j]);
          parts = 4 + j + 1;
        }
        if (ok) { ++gv; parts = 0; }
      };
      bool sent = false;                     // the keys of this row block's first tile have been sent for
      for (int e = 0; e < items && ok; ++e) {
        if (e == 0) ok = wait_bar(sm, &sm->item_full[0], 0, a.spin);
        if (!ok) break;
        const Item* it = &sm->item[e & 1];
        const int nt = it->nt;
        if (nt > 0 && !sent) send_keys(it, 0);
        for (int t = 0; t + 1 < nt && ok; ++t) {
          send_keys(it, t + 1);
          send_dims(it, t);
        }
        // the next row block's first keys before this one's last dims
        if (ok && e + 1 < items) ok = wait_bar(sm, &sm->item_full[(e + 1) & 1], ((e + 1) >> 1) & 1, a.spin);
        sent = ok && nt > 0 && e + 1 < items && sm->item[(e + 1) & 1].nt > 0;
        if (sent) send_keys(&sm->item[(e + 1) & 1], 0);
        if (nt > 0 && ok) send_dims(it, nt - 1);
        mbar_arrive(&sm->item_free[e & 1]);
      }
      // copies in flight (there are none, unless a wait gave up): the last ones to each place
      {
        for (int m = 0; m < 4; ++m) {
          const int n = gk + (parts < 4 && m < parts ? 1 : 0);
          if (n > 0) mbar_wait(&sm->k_full[m], (n - 1) & 1, kDrainLimit);
        }
        for (int j = 0; j < 2; ++j) {
          const int n = gv + (parts > 4 + j ? 1 : 0);
          if (n > 0) mbar_wait(&sm->v_full[j], (n - 1) & 1, kDrainLimit);
        }
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp && rank == 1) {   // ---- tells the even block of this one's copies
    if (elect_lane()) {
      bool ok = true;
      int g = 0;
      auto keys = [&](int i) {
#pragma unroll 1
        for (int m = 0; m < 4 && ok; ++m) {
          ok = wait_bar(sm, &sm->k_full[m], i & 1, a.spin);
          if (ok) arrive_at(of_block(&sm->k_full[m], 0));
        }
      };
      auto dims = [&](int i) {
#pragma unroll 1
        for (int j = 0; j < 2 && ok; ++j) {
          ok = wait_bar(sm, &sm->v_full[j], i & 1, a.spin);
          if (ok) arrive_at(of_block(&sm->v_full[j], 0));
        }
      };
      for (int e = 0; e < items && ok; ++e) {
        ok = wait_bar(sm, &sm->item_full[e & 1], (e >> 1) & 1, a.spin);
        if (!ok) break;
        const int nt = sm->item[e & 1].nt;
        mbar_arrive(&sm->item_free[e & 1]);
        if (nt > 0) keys(g);
        for (int t = 0; t < nt && ok; ++t, ++g) {
          if (t + 1 < nt) keys(g + 1);
          dims(g);
        }
      }
      mbar_wait(&sm->drained, 0, 2 * kDefaultSpinLimit);   // the even block's last commit has come (before this block ends)
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {           // ---- products
    if (elect_lane()) {
      const uint64_t dq = smem_desc_sw128(smem_u32(qtile), 16, 1024);
      const uint64_t dk = smem_desc_sw128(smem_u32(ktile), 16, 2048);
      const uint64_t dv = smem_desc_sw128(smem_u32(vtile), 1024, 2048);
      const uint64_t dp = smem_desc_sw128(smem_u32(ptile), 16, 1024);
      bool ok = true;
      int g = 0;
      for (int e = 0; e < items && ok; ++e) {
        ok = wait_bar(sm, &sm->item_full[e & 1], (e >> 1) & 1, a.spin);
        if (!ok) break;
        const Item* it = &sm->item[e & 1];
        const int nt = it->nt, keys = it->keys - it->begin * kTile;
        const uint32_t ido = make_idesc(1, 1, 1, 0, 256, 0) | (static_cast<uint32_t>(it->nq >> 2) << 17);   // 2 nq columns
        ok = wait_bar(sm, &sm->q_full, e & 1, a.spin);
        tc_fence_after();
        auto issue_s = [&](int t) {
          const int i = g + t;
          const uint32_t ids = make_idesc(1, 1, 0, 0, 128, 0) |
                               (static_cast<uint32_t>(half_keys(min(kTile, keys - t * kTile)) >> 2) << 17);
          const uint32_t d = tmem + kTmemS + 64 * (i & 1);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if ((c & 1) == 0) {
              ok = ok && wait_bar(sm, &sm->k_full[c >> 1], i & 1, a.spin);
              tc_fence_after();
            }
            if (ok) issue_s_chunk(d, dq, dk, c, ids);
            if ((c & 1) == 1) mma2_commit(&sm->k_free[c >> 1]);
          }
          mma2_commit(&sm->s_full[i & 1]);
          if (t == nt - 1) mma2_commit(&sm->q_free);
        };
        // before this row block's first O products the outputs of the one before are read (a row block
        // without tiles waits too: its own outputs would be told from those by nothing)
        auto outputs_read = [&](int j) {
          if (e > 0) {
            ok = ok && wait_bar(sm, &sm->o_free[j], (e - 1) & 1, a.spin);
            tc_fence_after();
          }
        };
        if (nt == 0) {
          outputs_read(0);
          outputs_read(1);
          mma2_commit(&sm->q_free);
        }
        for (int t = -1; t < nt && ok; ++t) {   // (issue_s once: its code is long)
          const int i = g + t;
          if (t + 1 < nt) issue_s(t + 1);
          if (t < 0) continue;
          const int ks = min(kTile, keys - t * kTile) >> 4;
          ok = ok && wait_bar(sm, &sm->p_full, i & 1, a.spin);
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (t == 0) outputs_read(j);
            ok = ok && wait_bar(sm, &sm->v_full[j], i & 1, a.spin);
            tc_fence_after();
            if (!ok) break;
            const uint64_t v = dv + j * (kDimPart >> 4);
            const uint32_t d = tmem + j * (2 * kRows);
            if (t == 0) mma2_set(d, v, dp, ido);
            else mma2_add(d, v, dp, ido);
            if (ks == 8) {
#pragma unroll
              for (int k = 1; k < 8; ++k) mma2_add(d, v + k * 256, dp + (k >> 2) * (kChunk >> 4) + 2 * (k & 3), ido);
            } else {
#pragma unroll 1
              for (int k = 1; k < ks; ++k) mma2_add(d, v + k * 256, dp + (k >> 2) * (kChunk >> 4) + 2 * (k & 3), ido);
            }
            mma2_commit(&sm->v_free[j]);
          }
        }
        g += nt;
        mbar_arrive(&sm->item_free[e & 1]);
      }
      mma2_commit(&sm->drained);   // before the tensor memory is given back (and shared memory)
      mbar_wait(&sm->drained, 0, kDefaultSpinLimit);
    }
    __syncwarp();
  } else if (warp < kSoftWarps) {          // ---- softmax
    int g = 0;
    bool ok = true;
    for (int e = 0; e < items; ++e) {
      const bool there = ok && wait_warp(sm, &sm->item_full[e & 1], (e >> 1) & 1, a.spin);
      if (role_any<kSoftId, kSoftWarps * 32>(!there)) break;
      const Item* it = &sm->item[e & 1];
      const int r = 32 * (warp & 1) + lane;
      const RowSees sees = it->sees[r];
      RowState s;
      s.reset();
      const int nt = it->nt;
      for (int t = 0; t < nt; ++t, ++g) weigh_tile(a, sm, it, ptile, tmem, rank, g, it->begin + t, t == 0, sees, s, ok);
      const int quarter = 2 * (warp >> 2) + ((warp >> 1) & 1);   // of the keys
      if (quarter == 0) sm->ref[e & 1][r] = s.m == -INFINITY ? -INFINITY : s.msub;
      sm->sums[e & 1][quarter][r] = make_float2(s.l, s.hat);
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm->l_full[e & 1]);
        mbar_arrive(&sm->item_free[e & 1]);
      }
    }
  } else {                                 // ---- queries and outputs
    int g = 0;
    bool ok = true;
    auto item_there = [&](int e) {
      ok = ok && wait_warp(sm, &sm->item_full[e & 1], (e >> 1) & 1, a.spin);
      return !role_any<kOutId, kOutThreads>(!ok);
    };
    auto queries = [&](int e) {
      const Item* it = &sm->item[e & 1];
      load_queries(a, it, qtile);
      __syncwarp();
      if (lane == 0) arrive_at(of_block(&sm->q_full, 0));
    };
    bool there = items > 0 && item_there(0);
    if (there) queries(0);
    for (int e = 0; e < items && there; ++e) {
      const Item* it = &sm->item[e & 1];
      g += it->nt;
      ok = ok && wait_warp(sm, &sm->q_free, e & 1, a.spin);   // the last S product on these queries is complete
      if (e + 1 < items) {
        there = item_there(e + 1);
        if (there) queries(e + 1);
      }
      ok = ok && wait_warp(sm, &sm->l_full[e & 1], (e >> 1) & 1, a.spin);
      if (ok) finish_sums(a, it, sm, rank, e);
      role_sync<kOutId, kOutThreads>();
      ok = ok && wait_warp(sm, &sm->f_full[e & 1], (e >> 1) & 1, a.spin);   // the other rows' factors
      if (it->nt > 0) ok = ok && wait_warp(sm, &sm->v_free[1], (g - 1) & 1, a.spin);
      if (!ok) continue;
      tc_fence_after();
#pragma unroll 1
      for (int j = 0; j < 2; ++j)
        write_block(a, it, sm, tmem, rank, e, j, [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_at(of_block(&sm->o_free[j], 0));
        });
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->item_free[e & 1]);
    }
    cp_async_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                          // nobody writes into or reads from a block that has ended
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// ---------------------------------------------------------------------------
// the join: the parts of a row in order, the sink, the rotation back.  64 threads of 8 dims for a row;
// where there are many parts four times as many, each with every fourth part.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;
constexpr int kShares = 4;
constexpr int kFewParts = 8;

__global__ void __launch_bounds__(kJoinThreads) chunk_join_kernel(const __grid_constant__ ChunkArgs a) {
  __shared__ float shares[kShares - 1][kD];
  grid_dep_wait();
  const ChunkHead head = *a.head;
  const int sub = threadIdx.x >> 6, lane = threadIdx.x & 31, d = (threadIdx.x & 63) * 8;
  constexpr int kSets = 2 * kRows / 4;   // of four rows of a row block
  for (int x = blockIdx.x; x < head.splits * kSets; x += gridDim.x) {
    const SplitPlan sp = a.split[x / kSets];
    const ReqPlan p = a.req[request_of_item(a, sp.item)];
    const int i0 = (sp.item - p.item0) * a.group;
    const int nr = min(p.nq - i0, a.group) * a.H;
    const bool late = a.unit0[sp.item] > share_begin(head.units, head.blocks, sp.b0);
    const int parts = sp.b1 - sp.b0 + 1;
    const bool few = parts <= kFewParts;
    for (int y = 0; y < (few ? 1 : 4); ++y) {   // (the whole block)
      const int r = (x % kSets) * 4 + (few ? sub : y), share = few ? 0 : sub;
      const bool there = r < nr;
      auto slot = [&](int k) { return (2 * static_cast<size_t>(sp.b0 + k) + (k == 0 && late)) * (2 * kRows) + r; };
      auto weight = [&](float2 v, float M) { return v.y == 0.f ? 0.f : v.y != v.y ? v.y : exp2f(v.x - M); };
      const size_t row = static_cast<size_t>(p.q0 + i0) * a.H + r;
      const float sink = a.sink != nullptr && there ? __ldg(a.sink + row % a.H) : -INFINITY;
      const float s2 = __fmul_rn(sink, kLog2e);   // (not part of a fused difference: s2 - M is 0 where s2 is the larger)
      float M = s2, total = 0.f, o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = 0.f;
      if (there) {
        if (few) {
          for (int k = 0; k < parts; ++k) {
            const float2 v = a.ml[slot(k)];
            if (v.y != 0.f) M = fmaxf(M, v.x);
          }
        } else {
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
        }
#pragma unroll 4
        for (int k = share; k < parts; k += few ? 1 : kShares) {
          const float2 ml = a.ml[slot(k)];
          const float e = weight(ml, M);   // 0: a part without keys, whose output is 0
          if (few) total += ml.y * e;
          const float4* v = reinterpret_cast<const float4*>(a.opart + slot(k) * kD + d);
          const float4 v0 = v[0], v1 = v[1];
          o[0] += e * v0.x; o[1] += e * v0.y; o[2] += e * v0.z; o[3] += e * v0.w;
          o[4] += e * v1.x; o[5] += e * v1.y; o[6] += e * v1.z; o[7] += e * v1.w;
        }
      }
      if (!few) {
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
        }
        __syncthreads();   // shares are used again
      }
      if (!there || share > 0) continue;
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
  }
}

inline size_t a256(size_t x) { return (x + 255) & ~size_t(255); }

// How the row blocks and the workspace follow from the sizes alone.
struct Layout {
  int group, most_blocks;
  size_t head, req, unit0, share, split, flags, images, opart, ml, bytes;
};
Layout layout_of(int R, int T, int H, int64_t max_keys) {
  Layout l = {};
  l.group = std::max(1, 2 * kRows / H);
  // each request's last row block may be a short one
  const int64_t items = static_cast<int64_t>(T) / l.group + std::min(R, T);
  const int64_t tiles = items * ((max_keys + kTile - 1) / kTile + 1);
  l.most_blocks = static_cast<int>(std::min<int64_t>(kPairs, std::max<int64_t>(1, (2 * tiles + kItemUnits * items) / kLeastShare)));
  const size_t keys = static_cast<size_t>(max_keys + 15) & ~size_t(15);
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t x = at; at += a256(bytes); return x; };
  l.head = take(sizeof(ChunkHead));
  l.req = take(sizeof(ReqPlan) * static_cast<size_t>(R));
  l.unit0 = take(8 * static_cast<size_t>(items + 1));
  l.share = take(sizeof(SharePlan) * l.most_blocks);
  l.split = take(sizeof(SplitPlan) * l.most_blocks);
  l.flags = take(keys);
  l.images = take(keys * (2 * kD));
  l.opart = take(2 * static_cast<size_t>(l.most_blocks) * (2 * kRows) * kD * 4);
  l.ml = take(2 * static_cast<size_t>(l.most_blocks) * (2 * kRows) * 8);
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
  a.window = std::min(window, 1 << 30);   // (no length is more; differences stay within 32 bits)
  a.max_ctx = max_ctx;
  a.sink = sink;
  a.scale_log2 = scale * kLog2e;
  a.slack = std::min(kSlack / a.scale_log2, FLT_MAX);   // finite for the smallest scales too
  a.q_rope = q_rope;
  a.out = static_cast<uint8_t*>(out);
  a.lse = lse;
  a.max_keys = max_keys;
  a.group = l.group;
  a.most_blocks = l.most_blocks;
  a.head = reinterpret_cast<ChunkHead*>(ws + l.head);
  a.req = reinterpret_cast<ReqPlan*>(ws + l.req);
  a.unit0 = reinterpret_cast<long long*>(ws + l.unit0);
  a.share = reinterpret_cast<SharePlan*>(ws + l.share);
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
      std::min<int64_t>(16 * kPairs, std::max<int64_t>(1, (decode_warps + kDecodeThreads / 32 - 1) / (kDecodeThreads / 32))));
  e = launch_next(chunk_decode_kernel, decode_blocks, kDecodeThreads, 0, stream, nullptr, a);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> allowed;
  e = launch_next(chunk_attn_kernel, 2 * l.most_blocks, kThreads, kChunkSmemBytes, stream, &allowed, a);
  if (e != cudaSuccess || l.most_blocks == 1) return e;
  return launch_next(chunk_join_kernel, 32 * l.most_blocks, kJoinThreads, 0, stream, nullptr, a);
}

unsigned int take_err_chunk_attn() { return take_dev_err(); }

}  // namespace cskv
