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
// Three kernels, each started while the one before it ends:
//   chunk_prepare_kernel its first block plans: the requests' key lists, the row blocks and their tiles as one line
//                        of work, cut into equal shares, or dealt out whole where that is as short.  The others
//                        decode meanwhile: every key that some query
//                        sees, once, from its paged row to bf16 in the order that the tensor core reads (the
//                        same rows are read by hundreds of row blocks: decoding a tile takes longer than
//                        its products).  (Two kernels one after the other for very many requests.)
//   chunk_attn_kernel    one pair of blocks (a cluster) per two SMs, its share of the work;
//   chunk_join_kernel    the row blocks that a share's border cuts in two or more.
//
// A pair of blocks.  A row block has up to 128 (query, head) rows, whole queries of a request; the even block of
// the pair has the first half of its rows, the odd one the second.  The keys come in tiles of 128.
//   S  = Q K^T     each block gets its own rows x 128 keys; it holds its rows of Q and half of the
//                  tile's keys, all dims (64 KB);
//   O^T += V^T P^T each block gets all rows x two of the four blocks of 128 dims; it holds these dims of
//                  all the tile's keys (64 KB) and its own rows of P (16 KB).
// The products are issued for both by the even block.  Tensor memory: three places of outputs (a block of 128
// dims as lanes), by turns, so that a row block's products begin while the one before is read; the logits of
// two tiles behind them (rows as lanes, 64 to 127 with the second half of the keys).  Roles in each block:
//   warps 0-7    softmax of a tile: a thread has one row and 32 keys; P to shared memory;
//   warps 8-15   the next row block's queries (loaded and rotated ahead), and the outputs;
//   warp 16      in the even block one thread issues the products, S of the next tile before O of this
//                one, also from row block to row block, so that the softmax runs beside products; in the odd
//                block one thread tells the even one which copies have arrived;
//   warp 17      sends for the keys (bulk copies of a block of 128 dims), as soon as the product on the
//                same place's keys before is complete;
//   warp 18      plans the row blocks, two at a time.
// Measured: two tiles take O + S + the softmax and what lies between, 5,400 cycles; the products alone are 4,660
// of them.  What the single threads do between a barrier and the next product or copy counts in full, and
// so does code that drops out of the instruction caches: a clock read before every wait cost 16 % (4,096
// queries on 8,320 keys: 2.72 -> 3.3 ms), the give-up path of every wait in line 8 % of three short prompts.
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
constexpr int kPlaces = 3;                // of outputs in tensor memory: 128 dims of a row block (128 columns)
constexpr uint32_t kTmemS = kPlaces * 2 * kRows;   // TMEM columns: O, then S, 64 for each tile
constexpr float kSlack = 8.0f;            // base 2
constexpr int kPairs = 76;                // of SMs
constexpr int kPlanThreads = 1024;         // of the plan alone
constexpr int kPrepThreads = 256;          // of the plan beside the decoding, and of the decoding
// Requests whose rows every decoding block sums up itself, beside the plan.  (64 requests of one token on 500 entries: 31.6 us,
// waiting for a plan of its own 37.4; 1,000: 292 and 298.)
constexpr int kOwnReqs = 1024;
constexpr int kPlanItems = 4;             // row blocks of a thread at a time
// A row block's cost beside its tiles, a tile being 2 (three ragged prompts, 173 row blocks: 71.6, 69.4, 67.7 and
// 68.4 us with 2, 3, 4 and 5).
constexpr int kItemUnits = 4;
// Units of a share at least (5 tokens on 288 keys, 3 tiles: 18.4 us on several pairs with 4, 17.6 us on one with 8;
// with 16 the same).
constexpr int kLeastShare = 8;
// Row blocks are dealt out whole, largest first, where the longest share is at most this many units longer than an equal
// one: what cutting row blocks and joining their parts costs.  (45 calls of 2 to 640 row blocks, BF16, cut and whole: 336
// row blocks, equal shares of 39.8 units and at most 46, 75.9 and 60.1 us; 138, 79.9 and 88: 77.7 and 76.1; 120, 44.2 and 56: 57.7
// and 55.7; 96, 22.7 and 36: 41.3 and 41.4; 90, 22 and 36: 40.6 and 41.3; 411, 149.5 and 164: 136.1 and 142.4; 232, 61.1
// and 80: 75.3 and 79.5.  Below 11 units' difference whole ones are shorter by up to 16 us and longer by 0.6 at most, from 14 on
// shorter in two of 21 calls, by 2.4 at most.)
constexpr int kSplitCost = 13;
// Parts of a row that one warp joins; more are a block's.  (64 queries of 64 heads on 65,536 entries, two or three parts:
// 360 us, by blocks 372; one on 262,144, seventy: 146 us, by warps 187.)
constexpr int kFewParts = 8;
constexpr unsigned long long kDrainLimit = 1ull << 27;   // cycles that a block which gives up waits for its own copies

struct ReqPlan {
  int q0, nq, len;          // its queries [q0, q0 + nq), its length
  int entries, entries16;   // entries that count, and rounded up to 16 (decoded rows)
  int row0, rows, rows16;   // its first decoded raw row, how many, rounded up
  long long base;           // its first decoded row
  int item0;                // its first row block
};
struct ItemPlan {           // of a row block
  long long unit0;          // its first unit of work
  int req, item;            // its request; its number
};
struct SharePlan {
  ItemPlan plan;            // of its first row block
  long long lo, hi;         // a pair's units [lo, hi)
  int first, last;          // the row blocks that have some of them
};
struct SplitPlan {          // a row block that several pairs share
  int row0, rows;           // its rows of [T * H]
  int first, next;          // its first part, and its second one: each further one is two behind
  int parts, pad[3];
};
struct ChunkHead {
  int items, blocks;
  int few, many;            // split[0 .. few): row blocks of kFewParts parts at most; split[most_blocks - many ..): of more
  int whole, pad;           // shares of whole row blocks, in `list`'s order
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
  int head_inv;             // 2^16 / H, rounded up: row / H is row * head_inv >> 16 for rows of a row block
  int most_blocks;          // shares at most
  // workspace
  ChunkHead* head;
  ReqPlan* req;
  ItemPlan* item;           // [items + 1]; the last one ends the units
  ItemPlan* list;           // [items]: the row blocks share by share, where shares are of whole ones
  SharePlan* share;         // [most_blocks]
  SplitPlan* split;         // [most_blocks]
  uint8_t* flags;           // of every decoded row: 0, kNone, kUnfit
  uint8_t* bad;             // of every eight of them: whether a row that is there cannot be used
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

// a / b, most often of 32 bits (b's are below 2^31)
__device__ __forceinline__ long long divide(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}
// Shares: pair b has the units [units * b / blocks, units * (b + 1) / blocks); tile t of a row block
// begins at its unit 2 t and belongs to the pair that has this unit.
__device__ __forceinline__ long long share_begin(long long units, int blocks, int b) { return divide(units * b, blocks); }
__device__ __forceinline__ int block_of_unit(long long units, int blocks, long long u) {
  return static_cast<int>(divide((u + 1) * blocks - 1, units));
}
// the last row block that begins at or before unit u
template <class Unit0>
__device__ __forceinline__ int item_of_unit(Unit0&& unit0, int items, long long u) {
  int e = 0, n = items;
  while (n > 1) {
    const int half = n / 2;
    const bool le = unit0(e + half) <= u;
    e = le ? e + half : e;
    n = le ? n - half : half;
  }
  return e;
}

// Inclusive sums of a block's pairs of values; `total` gets the last ones.
struct Pair {
  long long x;
  int y;
};
__device__ __forceinline__ Pair block_scan(Pair v, Pair* part, Pair* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  auto warp_scan = [&](Pair& p) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xFFFFFFFFu, p.x, o);
      const int y = __shfl_up_sync(0xFFFFFFFFu, p.y, o);
      if (lane >= o) {
        p.x += x;
        p.y += y;
      }
    }
  };
  warp_scan(v);
  if (lane == 31) part[warp] = v;
  __syncthreads();
  if (warp == 0) {
    Pair p = lane < warps ? part[lane] : Pair{0, 0};
    warp_scan(p);
    part[lane] = p;
  }
  __syncthreads();
  if (warp > 0) {
    v.x += part[warp - 1].x;
    v.y += part[warp - 1].y;
  }
  *total = part[warps - 1];
  __syncthreads();   // part is used again
  return v;
}

// Whether request r's queries are none: a border outside [0, T], or before the one before it.
__device__ __forceinline__ bool wrong_queries(const ChunkArgs& a, int lo, int hi) { return lo < 0 || hi < lo || hi > a.T; }

// What request r has, nq -1 with wrong queries (one such request leaves all without any: the sum of their
// queries is no longer bounded by T); what is wrong is told by the plan alone.
template <bool kTell>
__device__ __forceinline__ ReqPlan request_of(const ChunkArgs& a, int r) {
  auto wrong = [] { if constexpr (kTell) set_err(CSKV_ERR_BOUNDS); };
  ReqPlan p = {};
  const int lo = a.cu_q[r], hi = a.cu_q[r + 1];
  int len = a.ctx_len != nullptr ? a.ctx_len[r] : 0, given = a.n_entries != nullptr ? a.n_entries[r] : 0;
  if (wrong_queries(a, lo, hi)) {
    wrong();
    p.nq = -1;
    return p;
  }
  p.q0 = lo;
  p.nq = hi - lo;
  if (p.nq == 0) return p;
  if (len < 0 || len > a.max_ctx) { wrong(); len = max(0, min(len, a.max_ctx)); }
  p.len = len;
  if (a.has_entries) {
    int n = a.ratio > 0 ? len / a.ratio : a.max_entries;
    if (a.n_entries != nullptr) {
      if (given < 0 || given > a.max_entries) { wrong(); given = max(0, min(given, a.max_entries)); }
      n = min(n, given);
    }
    if (n > a.max_entries) { wrong(); n = a.max_entries; }
    p.entries = n;
  }
  if (a.has_rows) {
    p.rows = static_cast<int>(min(static_cast<long long>(len), static_cast<long long>(p.nq) + a.window - 1));
    p.row0 = len - p.rows;
  }
  p.entries16 = up16(p.entries);
  p.rows16 = up16(p.rows);
  return p;
}

constexpr int kPlanStaged = 2048;         // row blocks whose places are searched in shared memory
constexpr int kSizes = 1024;              // sizes of row blocks that are told apart
struct PlanSmem {
  Pair part[32];
  long long staged[kPlanStaged];
  int item0[kOwnReqs];
  int sizes[kSizes];
  uint16_t rank[kPlanStaged];
  int load[kPairs];
};

// Deals the row blocks out whole, if that is no longer than equal shares with their join: largest first, to the
// pairs in order and back again in turn (row blocks of one size in any order: every one's results are its own).
__device__ __forceinline__ bool deal_whole(const ChunkArgs& a, PlanSmem& sm, int items, int most) {
  const int tid = threadIdx.x, pairs = min(items, a.most_blocks), rounds = items / pairs, rest = items % pairs;
  auto units_at = [&](int e) { return static_cast<int>(sm.staged[e + 1] - sm.staged[e]); };
  auto pair_of = [&](int rank) { return (rank / pairs) & 1 ? pairs - 1 - rank % pairs : rank % pairs; };
  const bool single = pairs == items;    // one for each pair: in any order
  bool longer = false;
  if (single) {
    for (int e = tid; e < items; e += blockDim.x) longer |= units_at(e) > most;
  } else {
    for (int i = tid; i < kSizes; i += blockDim.x) sm.sizes[i] = 0;
    for (int i = tid; i < pairs; i += blockDim.x) sm.load[i] = 0;
    __syncthreads();
    auto size_of = [&](int e) { return kSizes - 1 - min(units_at(e) / 2, kSizes - 1); };
    for (int e = tid; e < items; e += blockDim.x) {
      atomicAdd(&sm.sizes[size_of(e)], 1);
      longer |= units_at(e) / 2 >= kSizes;   // not told apart: their order, and with it the longest share, would be any
    }
    __syncthreads();
    const int each = kSizes / blockDim.x;
    int mine = 0;
    for (int i = 0; i < each; ++i) mine += sm.sizes[tid * each + i];
    Pair total;
    int at = block_scan(Pair{0, mine}, sm.part, &total).y - mine;
    for (int i = 0; i < each; ++i) {
      const int n = sm.sizes[tid * each + i];
      sm.sizes[tid * each + i] = at;
      at += n;
    }
    __syncthreads();
    for (int e = tid; e < items; e += blockDim.x) {
      const int rank = atomicAdd(&sm.sizes[size_of(e)], 1);
      sm.rank[e] = static_cast<uint16_t>(rank);
      atomicAdd(&sm.load[pair_of(rank)], units_at(e));
    }
    __syncthreads();
    longer |= tid < pairs && sm.load[tid] > most;
  }
  if (__syncthreads_or(longer)) return false;
  // row blocks of the pairs before: whole rounds, and those of the last one
  auto first_of = [&](int pair) { return pair * rounds + ((rounds & 1) ? max(0, pair - (pairs - rest)) : min(pair, rest)); };
  for (int e = tid; e < items; e += blockDim.x) {
    const int rank = single ? e : sm.rank[e], pair = pair_of(rank), first = first_of(pair);
    const ItemPlan plan = {0, a.item[e].req, e};
    a.list[first + rank / pairs] = plan;
    if (rank < pairs) {
      a.share[pair].plan = plan;
      a.share[pair].lo = 0;
      a.share[pair].hi = 1ll << 40;   // (beyond every tile)
      a.share[pair].first = first;
      a.share[pair].last = first_of(pair + 1) - 1;
    }
  }
  return true;
}

__device__ void plan_chunks(const ChunkArgs& a, PlanSmem& sm) {
  Pair* part = sm.part;
  const int tid = threadIdx.x;
  long long keys = 0;
  int items = 0;
  Pair total;
  const bool once = a.R <= static_cast<int>(blockDim.x);
  bool sound = true;
  if (!once) {
    bool wrong = false;
    for (int r = tid; r < a.R; r += blockDim.x) wrong |= wrong_queries(a, a.cu_q[r], a.cu_q[r + 1]);
    sound = __syncthreads_or(wrong) == 0;
  }
  for (int r0 = 0; r0 < a.R; r0 += blockDim.x) {
    const int r = r0 + tid;
    ReqPlan p = {};
    if (r < a.R) p = request_of<true>(a, r);
    if (once) sound = __syncthreads_or(p.nq < 0) == 0;
    if (!sound) p = ReqPlan{};
    const long long mine = static_cast<long long>(p.entries16) + p.rows16;
    const int blocks = (p.nq + a.group - 1) / a.group;
    const Pair upto = block_scan(Pair{mine, blocks}, part, &total);
    p.base = keys + upto.x - mine;
    p.item0 = items + upto.y - blocks;
    if (p.base + mine > a.max_keys && mine > 0) {   // no room
      set_err(CSKV_ERR_BOUNDS);
      p.entries = p.entries16 = p.rows = p.rows16 = 0;
    }
    keys += total.x;
    items += total.y;
    if (r < a.R) a.req[r] = p;
    if (r < kOwnReqs) sm.item0[r] = p.item0;
  }
  // the last request that has room ends the decoded rows
  keys = min(keys, a.max_keys);
  __syncthreads();
  auto item0 = [&](int r) { return a.R <= kOwnReqs ? sm.item0[r] : a.req[r].item0; };
  long long units = 0;
  for (int e0 = 0; e0 < items; e0 += blockDim.x * kPlanItems) {
    int mine[kPlanItems], req[kPlanItems], sum = 0;
    const int e1 = e0 + tid * kPlanItems;
    int r = 0;
    if (e1 < items) {
      for (int n = a.R; n > 1;) {   // the last request whose first row block is not behind e1
        const int half = n / 2;
        const bool le = item0(r + half) <= e1;
        r = le ? r + half : r;
        n = le ? n - half : half;
      }
    }
#pragma unroll
    for (int u = 0; u < kPlanItems; ++u) {
      mine[u] = req[u] = 0;
      if (e1 + u < items) {
        while (r + 1 < a.R && item0(r + 1) <= e1 + u) ++r;
        const ReqPlan& p = a.req[r];
        mine[u] = units_of(tiles_of(block_keys(a, p, e1 + u - p.item0).keys));
        req[u] = r;
      }
      sum += mine[u];
    }
    long long at = units + block_scan(Pair{sum, 0}, part, &total).x - sum;
    units += total.x;
#pragma unroll
    for (int u = 0; u < kPlanItems; ++u) {
      if (e1 + u < items) {
        a.item[e1 + u] = ItemPlan{at, req[u], e1 + u};
        if (e1 + u < kPlanStaged) sm.staged[e1 + u] = at;
      }
      at += mine[u];
    }
  }
  if (tid == 0) {
    a.item[items] = ItemPlan{units, 0, 0};
    if (items < kPlanStaged) sm.staged[items] = units;
  }
  __syncthreads();
  // may the row blocks be dealt out whole?  A first test needs no order: as many average ones as some pair gets at least
  bool whole = false;
  if (items > 1 && items < kPlanStaged) {
    const float all = static_cast<float>(units), most = fmaxf(__fdividef(all, a.most_blocks), kLeastShare) + kSplitCost;
    whole = __fdividef(all, items) * ceilf(__fdividef(items, min(items, a.most_blocks))) <= most;
    if (whole) whole = deal_whole(a, sm, items, static_cast<int>(most));
  }
  if (whole) {
    if (tid == 0) *a.head = ChunkHead{items, min(items, a.most_blocks), 0, 0, 1, 0, units, keys};
    return;
  }
  const int blocks = static_cast<int>(max(1ll, min(static_cast<long long>(a.most_blocks), units / kLeastShare)));
  // the row blocks of each share; those that a border cuts are listed at the last border inside
  if (items == 0) {
    if (tid == 0) a.share[0].first = 0, a.share[0].last = -1;
  } else if (tid == 0) {
    a.share[0].first = 0;
    a.share[0].plan = a.item[0];
    a.share[0].lo = 0;
    a.share[blocks - 1].hi = units;
    a.share[blocks - 1].last = items - 1;
  }
  auto unit0 = [&](int e) { return items < kPlanStaged ? sm.staged[e] : a.item[e].unit0; };
  static_assert(kPairs <= kPrepThreads, "a thread for each border");
  const int b = tid + 1;
  SplitPlan split = {};
  if (b < blocks) {
    const long long u = share_begin(units, blocks, b);
    const int e = item_of_unit(unit0, items, u);
    const long long u0 = unit0(e);
    const int tiles = (static_cast<int>(unit0(e + 1) - u0) - kItemUnits) / 2;
    const long long end = u0 + 2ll * (tiles - 1);   // its last tile
    const int first = e + (end < u);                // (its tiles are all before the border)
    a.share[b].first = first;
    a.share[b].plan = a.item[first];
    a.share[b].lo = u;
    a.share[b - 1].hi = u;
    a.share[b - 1].last = e - (u0 == u);
    if (u > u0 && u <= end && block_of_unit(units, blocks, end) == b) {
      const int b0 = block_of_unit(units, blocks, u0);
      const ReqPlan& p = a.req[a.item[e].req];
      const int i0 = (e - p.item0) * a.group;
      split.row0 = (p.q0 + i0) * a.H;
      split.rows = min(p.nq - i0, a.group) * a.H;
      split.first = 2 * b0 + (u0 > share_begin(units, blocks, b0));
      split.next = 2 * (b0 + 1);
      split.parts = b - b0 + 1;
    }
  }
  const bool few = split.parts > 0 && split.parts <= kFewParts, many = split.parts > kFewParts;
  const Pair at = block_scan(Pair{few, many}, part, &total);
  if (few) a.split[at.x - 1] = split;
  if (many) a.split[a.most_blocks - at.y] = split;
  if (tid == 0) *a.head = ChunkHead{items, blocks, static_cast<int>(total.x), total.y, 0, 0, units, keys};
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ ChunkArgs a) {
  __shared__ PlanSmem sm;
  grid_dep_launch();
  plan_chunks(a, sm);
}

// ---------------------------------------------------------------------------
// the keys
// ---------------------------------------------------------------------------
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
// a bit for each that is not finite, whose values become 0.  All loads (of four rows, if they are long
// ones) are on their way before the first is used.
template <int FMT>
__device__ __forceinline__ uint32_t decode_rows(const uint8_t* mine, uint8_t* image) {
  constexpr int kAtOnce = FMT == CSKV_FMT_BF16 ? kDecodeRows / 2 : kDecodeRows;
  const int lane = threadIdx.x & 31;
  const uint32_t there = __ballot_sync(0xFFFFFFFFu, mine != nullptr);
  uint32_t unfit = 0;
#pragma unroll
  for (int i0 = 0; i0 < kDecodeRows; i0 += kAtOnce) {
    RawRow<FMT> raw[kAtOnce] = {};
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const uint8_t* row = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(mine), i0 + i));
      if (row != nullptr) raw[i].load(row, lane);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      uint32_t w[8] = {}, bad = 0;
      if ((there >> (i0 + i)) & 1u) raw[i].to_bf16(w);
#pragma unroll
      for (int k = 0; k < 8; ++k) bad |= ((w[k] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
      if (__any_sync(0xFFFFFFFFu, bad != 0u)) {   // (an exponent of all ones carries into the sign bit)
        unfit |= 1u << (i0 + i);
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = 0u;
      }
      const int at = 2 * (lane & 3);
      uint8_t* to = image + (i0 + i) * 128;
      // the two pieces of 16 bytes are a sector, the second one first in every other row
      const int o = (i0 + i) & 1 ? 4 : 0;
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to + (((at ^ (i0 + i)) & ~1) << 4)), "r"(w[o]),
                   "r"(w[o + 1]), "r"(w[o + 2]), "r"(w[o + 3]), "r"(w[4 - o]), "r"(w[5 - o]), "r"(w[6 - o]), "r"(w[7 - o])
                   : "memory");
    }
  }
  return unfit;
}

struct ReqRows {            // of a request: its decoded rows
  long long base;
  int entries, rows, row0, pad;
};
struct DecodeSmem {
  Pair part[32];
  ReqRows req[kOwnReqs];
};

// Eight rows a warp, from block `block` of `blocks` on (32,000 FP4 rows of 16 requests to 33 MB: 7 us, bound by the chain
// page, row, conversion, store of the warps that are resident).  kOwn: the requests' places are the sums of this block itself (they
// are made in the time that a wait for the plan would take); else the plan's.
template <bool kOwn>
__device__ __forceinline__ void decode_chunks(const ChunkArgs& a, DecodeSmem* sm, int block, int blocks) {
  const int lane = threadIdx.x & 31;
  long long keys;
  if constexpr (kOwn) {
    Pair total;
    const int each = (a.R + kPrepThreads - 1) / kPrepThreads, r0 = threadIdx.x * each;
    long long mine = 0;
    bool wrong = false;
    for (int r = r0; r < min(a.R, r0 + each); ++r) {
      const ReqPlan p = request_of<false>(a, r);
      wrong |= p.nq < 0;
      sm->req[r] = ReqRows{mine, p.entries, p.rows, p.row0, 0};
      mine += p.entries16 + p.rows16;
    }
    const long long before = block_scan(Pair{mine, 0}, sm->part, &total).x - mine;
    for (int r = r0; r < min(a.R, r0 + each); ++r) {
      ReqRows& p = sm->req[r];
      p.base += before;
      if (p.base + up16(p.entries) + up16(p.rows) > a.max_keys) p.entries = p.rows = 0;   // no room
    }
    keys = __syncthreads_or(wrong) != 0 ? 0 : min(total.x, a.max_keys);
  } else {
    keys = a.head->keys;
  }
  const long long warps = static_cast<long long>(blocks) * (kPrepThreads / 32);
  for (long long x = (static_cast<long long>(block) * kPrepThreads + threadIdx.x) / 32 * kDecodeRows; x < keys;
       x += warps * kDecodeRows) {
    int r = 0, n = a.R;
    while (n > 1) {   // the last request whose rows begin at or before x
      const int half = n / 2;
      const bool le = (kOwn ? sm->req[r + half].base : a.req[r + half].base) <= x;
      r = le ? r + half : r;
      n = le ? n - half : half;
    }
    ReqRows p;
    if constexpr (kOwn) p = sm->req[r];
    else p = ReqRows{a.req[r].base, a.req[r].entries, a.req[r].rows, a.req[r].row0, 0};
    const int entries16 = up16(p.entries);
    const long long rows = entries16 + up16(p.rows);
    if (x - p.base >= rows) continue;   // no room for this request
    const int first = static_cast<int>(x - p.base);
    const bool raw = first >= entries16;
    const cskv_paged& c = raw ? a.rows : a.entries;
    const int k0 = raw ? first - entries16 : first, have = raw ? p.rows : p.entries;
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
    // (rows behind the last one are seen by nobody)
    const bool bad = __any_sync(0xFFFFFFFFu, exists && mine == nullptr) || unfit != 0u;
    if (lane == 0) a.bad[x / kDecodeRows] = bad;
  }
}

// Of an SM: all are resident, so that the next kernel's blocks come as these end.  (Four, with 64 registers a thread: up to 3 %
// longer; five: 9 %.)
constexpr int kPrepBlocks = 3;
// The first block plans, the others decode.
__global__ void __launch_bounds__(kPrepThreads, kPrepBlocks) chunk_prepare_kernel(const __grid_constant__ ChunkArgs a) {
  __shared__ union Smem {
    PlanSmem plan;
    DecodeSmem decode;
    __device__ Smem() {}
  } sm;
  grid_dep_launch();
  if (blockIdx.x == 0) plan_chunks(a, sm.plan);
  else decode_chunks<true>(a, &sm.decode, blockIdx.x - 1, gridDim.x - 1);
}

__global__ void __launch_bounds__(kPrepThreads, kPrepBlocks) chunk_decode_kernel(const __grid_constant__ ChunkArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  decode_chunks<false>(a, nullptr, blockIdx.x, gridDim.x);
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
  int t0;                        // the first row's query
  int seen16, raw0, keys;        // the list (BlockKeys); raw0 counted among all decoded rows of the request
  int begin, nt;                 // this pair's tiles
  int part;                      // partial output, -1: none
  long long base, stride;        // the request's first decoded row, bytes between its blocks of dims
  // of the softmax alone:
  int plain;                     // keys below it are seen by every row
  int bad;                       // a row of these tiles could not be read or is not finite
  RowSees sees[kRows];
};

struct ChunkSmem {
  Item item[2];
  uint64_t k_full[4], k_free[4];           // keys: blocks of 128 dims
  uint64_t v_full[2], v_free[2];           // this block's dims
  uint64_t s_full[2], moved[2], p_full, q_full, q_free, o_free[kPlaces], l_full[2], f_full[2], item_full[2], sees_full[2], item_free[2], drained;
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
// Says that something is done.  Nothing that plain loads of the other block read stands behind it (those numbers
// come by send_to): what it announces is read by the tensor core alone, P and the queries in their own
// block's shared memory and tensor memory, behind this block's proxy and tcgen05 fences, or it frees a
// place.  The arrival and the waits have the default scope, the block; that these fences also order what the
// products, which the other block issues, read of this block's memory is an assumption on the
// hardware, not a promise of the memory model.  The model's form, a release at cluster scope, waits
// for every write of the warp: a tile took 1.8 times as long.
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
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {   // at once
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return done != 0u;
}
// A wait that gives up makes every role leave its loop.
__device__ __noinline__ bool wait_on(ChunkSmem* sm, uint64_t* bar, uint32_t parity, unsigned long long limit) {
  const unsigned long long t0 = clock64();
  do {
    if (*reinterpret_cast<volatile int*>(&sm->abort) != 0 || clock64() - t0 > limit) {
      *reinterpret_cast<volatile int*>(&sm->abort) = 1;
      return false;
    }
  } while (!try_wait_long(bar, parity));
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

// A row block of this pair's share, and this block's rows of it; one warp.  First what all others wait for.
__device__ void make_item(const ChunkArgs& a, ChunkSmem* sm, int place, const ItemPlan& plan, long long lo, long long hi,
                          int pair, int rank) {
  const int lane = threadIdx.x & 31;
  Item* it = &sm->item[place];
  const ReqPlan p = a.req[plan.req];
  const BlockKeys k = block_keys(a, p, plan.item - p.item0);
  const int rows = (k.i1 - k.i0) * a.H, half = (rows + 1) / 2;
  const int at = rank == 0 ? 0 : half, nr = rank == 0 ? half : rows - half;   // of the row block
  // its tiles between the share's borders
  const int tiles = tiles_of(k.keys);
  const int begin = static_cast<int>(min(static_cast<long long>(tiles), max(0ll, (lo - plan.unit0 + 1) / 2)));
  const int end = static_cast<int>(min(static_cast<long long>(tiles), max(0ll, (hi - plan.unit0 + 1) / 2)));
  const int raw_at = p.entries16 + k.raw0;
  if (lane == 0) {
    it->t0 = p.q0 + k.i0;
    it->row0 = (p.q0 + k.i0) * a.H;
    it->rows = rows;
    it->half = half;
    it->r0 = (p.q0 + k.i0) * a.H + at;
    it->nr = nr;
    it->nq = up16(half);
    it->seen16 = k.seen16;
    it->raw0 = raw_at;
    it->keys = k.keys;
    it->base = p.base;
    it->stride = static_cast<long long>(p.entries16 + p.rows16) * 256;
    it->begin = begin;
    it->nt = end - begin;
    it->part = begin > 0 || end < tiles ? 2 * pair + (plan.unit0 > lo) : -1;
    mbar_arrive(&sm->item_full[place]);
  }
  const int raw0 = k.raw0 + p.row0;   // position of the list's first raw row
  int least = INT32_MAX;
  for (int r = lane; r < kRows; r += 32) {
    RowSees s{0, 0, -1, 0};
    if (r < nr) {
      const int pos1 = p.len - p.nq + k.i0 + ((at + r) * a.head_inv >> 16) + 1;
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
  uint32_t bad = 0;
  const uint8_t* groups = a.bad + p.base / kDecodeRows;
#pragma unroll 4
  for (int g = begin * (kTile / kDecodeRows) + lane; g < min(end * kTile, k.keys) / kDecodeRows; g += 32) {
    const int k0 = g * kDecodeRows;
    bad |= groups[(k0 < k.seen16 ? k0 : raw_at + k0 - k.seen16) / kDecodeRows];
  }
  bad = __any_sync(0xFFFFFFFFu, bad != 0u);
  if (lane == 0) {
    it->plain = least;
    it->bad = bad;
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(&sm->sees_full[place]);
}

// The next row block's queries wait in the output warps' registers for the last product on this one's (loaded
// from memory then, they took 4,000 cycles, in which nothing was multiplied): a thread has 8 dims of
// every 64 of two rows.  Of the last 64 dims `v` has the first bf16 of each rotated value, `low` the second.
struct NextQueries {
  uint4 v[2][8], low[2];
};
__device__ __forceinline__ void load_queries(const ChunkArgs& a, const Item* it, bool any, NextQueries& n) {
  const int tid = threadIdx.x - kSoftWarps * 32, nr = any ? it->nr : 0;
  const uint8_t* q = a.q + (static_cast<size_t>(it->r0) + (tid >> 3)) * (2 * kD) + (tid & 7) * 16;
  static_assert(kRows * 8 == 2 * kOutThreads, "a thread has 8 dims of two rows");
  float4 cs[2][2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = (tid >> 3) + 32 * u;
    const bool there = r < nr;
    // (the row's query: rows of a row block are counted from its first query's first head)
    const int query = it->t0 + ((it->r0 - it->row0 + r) * a.head_inv >> 16);
    const float4* from = reinterpret_cast<const float4*>(a.q_rope + static_cast<size_t>(query) * 64 + (tid & 7) * 8);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      n.v[u][k] = make_uint4(0u, 0u, 0u, 0u);
      if (there) n.v[u][k] = __ldg(reinterpret_cast<const uint4*>(q + u * 32 * (2 * kD) + k * 128));
    }
    cs[u][0] = cs[u][1] = make_float4(1.f, 0.f, 1.f, 0.f);
    if (there) {
      cs[u][0] = __ldg(from);
      cs[u][1] = __ldg(from + 1);
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float co[4] = {cs[u][0].x, cs[u][0].z, cs[u][1].x, cs[u][1].z}, si[4] = {cs[u][0].y, cs[u][0].w, cs[u][1].y, cs[u][1].w};
    uint32_t* w = reinterpret_cast<uint32_t*>(&n.v[u][7]);
    uint32_t* l = reinterpret_cast<uint32_t*>(&n.low[u]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float y0 = bf16lo(w[k]), y1 = bf16hi(w[k]);
      const float z0 = y0 * co[k] - y1 * si[k], z1 = y0 * si[k] + y1 * co[k];
      w[k] = pack_bf16(z0, z1);
      l[k] = pack_bf16(z0 - bf16lo(w[k]), z1 - bf16hi(w[k]));
    }
  }
}
// Into the K-major chunks of Q (rows behind the last one are zero).
__device__ __forceinline__ void store_queries(const NextQueries& n, uint8_t* qtile) {
  const int tid = threadIdx.x - kSoftWarps * 32;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint8_t* to = qtile + sw128_offset((tid >> 3) + 32 * u, tid & 7);
#pragma unroll
    for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(to + k * kChunk) = n.v[u][k];
    *reinterpret_cast<uint4*>(to + 8 * kChunk) = n.low[u];
  }
  fence_proxy_async_smem();
}

// The place of row block e's block j of outputs in tensor memory, of three by turns: the next row block's
// products begin in the third one while this one's are read.
__device__ __forceinline__ uint32_t place_of(int e, int j) { return static_cast<uint32_t>((2 * e + j) % kPlaces) * (2 * kRows); }

// A softmax thread's state of its row.
struct RowState {
  float m, limit, msub;   // reference in units of q'.c; a logit above limit moves it; in base 2
  float l, hat;           // this thread's sums of the weights, and of the rounded ones
  __device__ __forceinline__ void reset() {
    m = limit = -INFINITY;
    msub = l = hat = 0.f;
  }
};

// bits [0, n)
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }
// the lowest bits of four bytes
__device__ __forceinline__ uint32_t bit_of_bytes(uint32_t x) { return ((x & 0x01010101u) * 0x01020408u) >> 24; }
// Logits of the keys k0 .. k0 + n - 1 that the row does not see, and those behind, become -inf; says whether
// it sees an unfit row (whose values are 0): its sum is NaN then, and with it its output.
__device__ __forceinline__ bool mask_keys(const ChunkArgs& a, const Item* it, int k0, int n, const RowSees& s, float (&z)[32]) {
  uint32_t seen = (low_bits(s.seen - k0) | (low_bits(s.hi + 1 - k0) & ~low_bits(s.lo - k0))) & low_bits(n), unfit = 0;
  if (it->bad) {
    uint32_t none = 0;
#pragma unroll 1
    for (int j = 0; j < 32; j += 8) {   // eight rows' flags lie together (k0 and the list's parts are whole 8s)
      const int k = k0 + j;
      if (k >= it->keys) break;
      const uint8_t* at = a.flags + it->base + (k < it->seen16 ? k : it->raw0 + k - it->seen16);
      const uint2 f = *reinterpret_cast<const uint2*>(at);
      static_assert(kNone == 1 && kUnfit == 2, "a bit of each");
      none |= (bit_of_bytes(f.x) | bit_of_bytes(f.y) << 4) << j;
      unfit |= (bit_of_bytes(f.x >> 1) | bit_of_bytes(f.y >> 1) << 4) << j;
    }
    seen &= ~none;
    unfit &= seen;
  }
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (!(seen & (1u << j))) z[j] = -INFINITY;
  return unfit != 0u;
}

// The softmax of the pair's tile g, the row block's tile t: this thread's row and 32 keys.
__device__ __forceinline__ void weigh_tile(const ChunkArgs& a, ChunkSmem* sm, const Item* it, uint8_t* ptile, uint32_t tmem,
                                           int rank, uint32_t place, int left, int masked, int g, int t, bool first, const RowSees& sees, RowState& s, bool& ok) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, side = warp >> 2;        // lanes of tensor memory; columns 32 side .. + 31
  const int r = 32 * (quarter & 1) + lane;
  const uint32_t tlane = static_cast<uint32_t>(quarter * 32) << 16;
  const int buf = g & 1;
  const int n2 = half_keys(min(kTile, left));
  const int c0 = 32 * side;                              // the thread's first key within its half
  const int k0 = (quarter >> 1) * n2 + c0;               // within the tile
  ok = ok && wait_warp(sm, &sm->s_full[buf], (g >> 1) & 1, a.spin);
  const bool has = ok && c0 < n2;   // (a warp's columns may all lie behind the last key)
  tc_fence_after();
  float z[32];
  if (has) {
    tmem_ld32(tmem + kTmemS + 64 * buf + c0 + tlane, z);
    tmem_wait_ld();
  }
  bool spoilt = false;
  if (n2 - c0 < 32 || t * kTile + k0 + 32 > masked || !has)
    spoilt = mask_keys(a, it, t * kTile + k0, has ? n2 - c0 : 0, sees, z);
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
  if (spoilt) s.l = __int_as_float(0x7FC00000);
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
        const uint32_t at = tmem + tlane + place + u * it->nq + x;
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
  const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + place_of(e, j) + u * it->nq;
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

// What the loading thread needs of a row block, in its registers: its reads of shared memory wait behind the
// products', and whatever it does between a place that is free and its copy is time without products.
struct Source {
  const uint8_t* image;     // the request's first block of dims
  long long stride;         // to the next one
  int seen16, raw0;         // (BlockKeys)
  int keys, begin, nt;
  __device__ __forceinline__ void load(const ChunkArgs& a, const Item* it) {
    image = a.images + it->base * (2 * kD);
    stride = it->stride;
    seen16 = it->seen16;
    raw0 = it->raw0;
    keys = it->keys;
    begin = it->begin;
    nt = it->nt;
  }
};
// `rows` rows of a list from `k` on, entries, raw rows, or both: where they lie in a block of dims (256 bytes a row).
struct Stretch {
  const uint8_t *entries, *raw;
  int entry_bytes, raw_bytes;
  __device__ __forceinline__ Stretch(const Source& s, int k, int rows, long long at) {
    const int ne = max(0, min(rows, s.seen16 - k));
    entry_bytes = ne * 256;
    raw_bytes = (rows - ne) * 256;
    entries = s.image + at + static_cast<long long>(k) * 256;
    raw = s.image + at + static_cast<long long>(s.raw0 + k + ne - s.seen16) * 256;
  }
  __device__ __forceinline__ void send(uint8_t* to, uint64_t* full) const {
    mbar_expect_tx(full, entry_bytes + raw_bytes);
    if (entry_bytes > 0) bulk_g2s(to, entries, entry_bytes, full);
    if (raw_bytes > 0) bulk_g2s(to + entry_bytes, raw, raw_bytes, full);
  }
  __device__ __forceinline__ void move(long long bytes) {
    entries += bytes;
    raw += bytes;
  }
};

// The order in which a share's tiles are sent for (and told of): a tile's keys before the dims of the tile before it,
// as the products need them, also from row block to row block; the very first tile's dims at once, as their
// place is free.
template <class Source, class Keys, class Dims>
__device__ __forceinline__ void walk_tiles(const ChunkArgs& a, ChunkSmem* sm, int items, bool& ok, Source s, Keys&& keys, Dims&& dims) {
  int e = 0, t = -1;                       // the row block, its tile
  bool fresh = true, first = true, early = false;
#pragma unroll 1
  while (e < items) {
    if (fresh) {
      ok = wait_bar(sm, &sm->item_full[e & 1], (e >> 1) & 1, a.spin);
      if (!ok) break;
      s.load(a, &sm->item[e & 1]);
      t = -1;
    }
    fresh = s.nt == 0;
    bool next = false;
    if (!fresh) {
      Source of = s;
      int kt = t + 1;
      bool send = kt < s.nt;
      if (!send && e + 1 < items) {
        ok = wait_bar(sm, &sm->item_full[(e + 1) & 1], ((e + 1) >> 1) & 1, a.spin);
        if (!ok) break;
        of.load(a, &sm->item[(e + 1) & 1]);
        kt = 0;
        send = next = of.nt > 0;
      }
      if (send) keys(of, kt);
      if (!ok) break;
      if (first || (t >= 0 && !early)) dims(s, max(t, 0));
      if (!ok) break;
      early = first;
      first = false;
      if (t + 1 < s.nt) {
        ++t;
        continue;
      }
      s = of;
      t = 0;
      fresh = !next;
    }
    mbar_arrive(&sm->item_free[e & 1]);
    ++e;
  }
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
      mbar_init(&sm->sees_full[i], 1);
      mbar_init(&sm->item_free[i], 2 + kSoftWarps + kOutWarps);
    }
    mbar_init(&sm->p_full, 2 * kSoftWarps);
    mbar_init(&sm->q_full, 2 * kOutWarps);
    mbar_init(&sm->q_free, 1);
    for (int j = 0; j < kPlaces; ++j) mbar_init(&sm->o_free[j], 2 * kOutWarps);
    mbar_init(&sm->drained, 1);
    sm->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm->tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                          // the other block's barriers are there
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sm->tmem, 0);
  grid_dep_wait();
  grid_dep_launch();
  const ChunkHead head = *a.head;
  const SharePlan share = a.share[pair];         // (there is room for every pair's; on its way beside the head)
  const int items = pair < head.blocks ? share.last - share.first + 1 : 0;

  if (warp == kPlanWarp) {                 // ---- row blocks
    ItemPlan plan = share.plan;
    for (int e = 0; e < items; ++e) {
      if (e >= 2 && !wait_warp(sm, &sm->item_free[e & 1], ((e >> 1) - 1) & 1, a.spin)) break;
      if (e > 0) plan = (head.whole ? a.list : a.item)[share.first + e];
      make_item(a, sm, e & 1, plan, share.lo, share.hi, pair, rank);
    }
  } else if (warp == kLoadWarp) {          // ---- keys
    if (elect_lane()) {
      bool ok = true;
      int gk = 0, gv = 0, parts = 0;         // tiles sent for: keys, dims; and parts of one more (4 + of dims)
      fence_proxy_async_global();            // (the decoded rows, by another kernel's plain stores)
      walk_tiles(
          a, sm, items, ok, Source{},
          [&](const Source& s, int t) {
            const int k0 = (s.begin + t) * kTile, n = min(kTile, s.keys - k0), n2 = half_keys(n);
            Stretch x(s, k0 + rank * n2, rank == 0 ? min(n, n2) : n - min(n, n2), 0);
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
              if (gk > 0) ok = wait_bar(sm, &sm->k_free[m], (gk - 1) & 1, a.spin);
              if (!ok) return;
              x.send(ktile + m * kKeyPart, &sm->k_full[m]);
              x.move(s.stride);
              parts = m + 1;
            }
            ++gk;
            parts = 0;
          },
          [&](const Source& s, int t) {
            const int k0 = (s.begin + t) * kTile;
            Stretch x(s, k0, min(kTile, s.keys - k0), rank * s.stride);
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {
              if (gv > 0) ok = wait_bar(sm, &sm->v_free[j], (gv - 1) & 1, a.spin);
              if (!ok) return;
              x.send(vtile + j * kDimPart, &sm->v_full[j]);
              x.move(2 * s.stride);
              parts = 4 + j + 1;
            }
            ++gv;
            parts = 0;
          });
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
      int gk = 0, gv = 0;
      struct Count {
        int nt;
        __device__ __forceinline__ void load(const ChunkArgs&, const Item* it) { nt = it->nt; }
      };
      walk_tiles(
          a, sm, items, ok, Count{},
          [&](const Count&, int) {
#pragma unroll 1
            for (int m = 0; m < 4 && ok; ++m) {
              ok = wait_bar(sm, &sm->k_full[m], gk & 1, a.spin);
              if (ok) arrive_at(of_block(&sm->k_full[m], 0));
            }
            ++gk;
          },
          [&](const Count&, int) {
#pragma unroll 1
            for (int j = 0; j < 2 && ok; ++j) {
              ok = wait_bar(sm, &sm->v_full[j], gv & 1, a.spin);
              if (ok) arrive_at(of_block(&sm->v_full[j], 0));
            }
            ++gv;
          });
      mbar_wait(&sm->drained, 0, 2 * kDefaultSpinLimit);   // the even block's last commit has come (before this block ends)
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {           // ---- products
    if (elect_lane()) {
      const uint64_t dq = smem_desc_sw128(smem_u32(qtile), 16, 1024);
      const uint64_t dk = smem_desc_sw128(smem_u32(ktile), 16, 2048);
      const uint64_t dv = smem_desc_sw128(smem_u32(vtile), 1024, 2048);
      const uint64_t dp = smem_desc_sw128(smem_u32(ptile), 16, 1024);
      bool ok = true, ahead = false;         // ahead: S of this row block's first tile has been issued
      int g = 0;
      for (int e = 0; e < items && ok; ++e) {
        ok = wait_bar(sm, &sm->item_full[e & 1], (e >> 1) & 1, a.spin);
        if (!ok) break;
        const Item* it = &sm->item[e & 1];
        const int nt = it->nt, keys = it->keys - it->begin * kTile;
        const uint32_t ido = make_idesc(1, 1, 1, 0, 256, 0) | (static_cast<uint32_t>(it->nq >> 2) << 17);   // 2 nq columns
        if (!ahead) {
          ok = wait_bar(sm, &sm->q_full, e & 1, a.spin);
          tc_fence_after();
        }
        // before this row block's first O products the outputs in their places before are read (a row block
        // without tiles waits too: its own outputs would be told from those by nothing)
        auto outputs_read = [&](int j) {
          const int n = 2 * e + j;
          if (n >= kPlaces) {
            ok = ok && wait_bar(sm, &sm->o_free[n % kPlaces], (n / kPlaces - 1) & 1, a.spin);
            tc_fence_after();
          }
        };
        if (nt == 0) {
          outputs_read(0);
          outputs_read(1);
          mma2_commit(&sm->q_free);
        }
        int t = ahead ? 0 : -1;
        ahead = false;
        for (; t < nt && ok; ++t) {
          const int i = g + t;
          // S of the next tile before O of this one, so that the softmax runs beside products; behind the last
          // tile that is the next row block's first one, if its queries are there before this one's weights
          const int k = i + 1;
          bool more = t + 1 < nt;
          int left = keys - (t + 1) * kTile, tiles = nt - (t + 1);   // of the row block from that tile on
          if (!more && nt > 0 && e + 1 < items) {
            const int f = e + 1;
            const unsigned long long t0 = clock64();
            while (!more && !mbar_test(&sm->p_full, i & 1) && clock64() - t0 < a.spin &&
                   !*reinterpret_cast<volatile int*>(&sm->abort)) {
              if (mbar_test(&sm->item_full[f & 1], (f >> 1) & 1)) {
                const Item* of = &sm->item[f & 1];
                left = of->keys - of->begin * kTile;
                tiles = of->nt;
                if (tiles == 0) break;
                more = mbar_test(&sm->q_full, f & 1);
              }
            }
            tc_fence_after();
            ahead = more;
          }
          if (more) {   // (here alone: its code is long)
            const uint32_t ids =
                make_idesc(1, 1, 0, 0, 128, 0) | (static_cast<uint32_t>(half_keys(min(kTile, left)) >> 2) << 17);
            const uint32_t d = tmem + kTmemS + 64 * (k & 1);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              if ((c & 1) == 0) {
                ok = ok && wait_bar(sm, &sm->k_full[c >> 1], k & 1, a.spin);
                tc_fence_after();
              }
              if (ok) issue_s_chunk(d, dq, dk, c, ids);
              if ((c & 1) == 1) mma2_commit(&sm->k_free[c >> 1]);
            }
            mma2_commit(&sm->s_full[k & 1]);
            if (tiles == 1) mma2_commit(&sm->q_free);
          }
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
            const uint32_t d = tmem + place_of(e, j);
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
      const bool there = ok && wait_warp(sm, &sm->sees_full[e & 1], (e >> 1) & 1, a.spin);
      if (role_any<kSoftId, kSoftWarps * 32>(!there)) break;
      const Item* it = &sm->item[e & 1];
      const int r = 32 * (warp & 1) + lane;
      const RowSees sees = it->sees[r];
      RowState s;
      s.reset();
      const int nt = it->nt;
      const int keys = it->keys, begin = it->begin, masked = it->bad ? 0 : it->plain;
      const uint32_t place = place_of(e, warp >> 2);
      for (int t = 0; t < nt; ++t, ++g)
        weigh_tile(a, sm, it, ptile, tmem, rank, place, keys - (begin + t) * kTile, masked, g, begin + t, t == 0, sees, s, ok);
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
    bool there = items > 0;
    for (int e = -1; e < items && there; ++e) {   // (-1: the first queries)
      const bool more = e + 1 < items;
      if (more) there = item_there(e + 1);
      NextQueries next;
      load_queries(a, &sm->item[(e + 1) & 1], more && there, next);
      if (e >= 0) ok = ok && wait_warp(sm, &sm->q_free, e & 1, a.spin);   // the last S product on these queries is complete
      if (more && there && ok) {
        store_queries(next, qtile);
        __syncwarp();
        if (lane == 0) arrive_at(of_block(&sm->q_full, 0));
      }
      if (e < 0) continue;
      const Item* it = &sm->item[e & 1];
      g += it->nt;
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
          if (lane == 0) arrive_at(of_block(&sm->o_free[(2 * e + j) % kPlaces], 0));
        });
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->item_free[e & 1]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && sm->abort != 0) set_err(CSKV_ERR_TIMEOUT);
  cluster_sync();                          // nobody writes into or reads from a block that has ended
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// ---------------------------------------------------------------------------
// the join: the parts of a row in order, the sink, the rotation back.  A lane has four dims of every 128.
// A row of few parts is one warp's, one of more (few queries on a long cache) a block's, whose warps have every
// eighth part.  75 row blocks of two or three parts, 38 MB: 7 to 10 us and 1.9 us between the kernels.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
// Blocks for a row block of few parts, a warp for each row.  The launch has as many for each share: fewer row blocks than
// shares are cut, so that a block of the launch meets one of few parts at most, its own.
constexpr int kJoinSets = 2 * kRows / kJoinWarps;

__global__ void __launch_bounds__(kJoinThreads, 4) chunk_join_kernel(const __grid_constant__ ChunkArgs a) {
  __shared__ float shares[kJoinWarps - 1][kD];
  grid_dep_wait();
  const ChunkHead head = *a.head;
  SplitPlan sp = a.split[blockIdx.x / kJoinSets]; // (there is room for as many; on its way beside the head)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int few = head.few * kJoinSets, all = few + head.many * (2 * kRows);
  for (int x = blockIdx.x; x < all; x += gridDim.x) {
    const bool alone = x < few;   // (the whole block)
    if (!alone) sp = a.split[a.most_blocks - 1 - (x - few) / (2 * kRows)];
    const int r = alone ? x % kJoinSets * kJoinWarps + warp : (x - few) % (2 * kRows);
    const int share = alone ? 0 : warp, step = alone ? 1 : kJoinWarps;
    if (r >= sp.rows) continue;   // (a warp alone, or the whole block)
    auto slot = [&](int k) { return static_cast<size_t>(k == 0 ? sp.first : sp.next + 2 * (k - 1)) * (2 * kRows) + r; };
    auto weight = [&](float2 v, float M) { return v.y == 0.f ? 0.f : v.y != v.y ? v.y : exp2f(v.x - M); };
    const unsigned row = sp.row0 + r;
    const float sink = a.sink != nullptr ? __ldg(a.sink + row % static_cast<unsigned>(a.H)) : -INFINITY;
    const float s2 = __fmul_rn(sink, kLog2e);   // (not part of a fused difference: s2 - M is 0 where s2 is the larger)
    float M = s2, total = 0.f;
    for (int k = lane; k < sp.parts; k += 32) {
      const float2 v = a.ml[slot(k)];
      if (v.y != 0.f) M = fmaxf(M, v.x);
    }
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, w));
    float4 o[4] = {};
#pragma unroll 2
    for (int k = share; k < sp.parts; k += step) {
      const float2 ml = a.ml[slot(k)];
      const float e = weight(ml, M);   // 0: a part without keys, whose output is 0
      total += ml.y * e;
      const float4* v = reinterpret_cast<const float4*>(a.opart + slot(k) * kD) + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 y = v[32 * i];
        o[i].x += e * y.x;
        o[i].y += e * y.y;
        o[i].z += e * y.z;
        o[i].w += e * y.w;
      }
    }
    if (!alone) {
      __shared__ float totals[kJoinWarps];
      if (lane == 0) totals[warp] = total;
      if (share > 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) reinterpret_cast<float4*>(shares[share - 1])[32 * i + lane] = o[i];
      }
      __syncthreads();
      if (share == 0) {
        for (int k = 1; k < kJoinWarps; ++k) {
          total += totals[k];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 y = reinterpret_cast<const float4*>(shares[k - 1])[32 * i + lane];
            o[i].x += y.x;
            o[i].y += y.y;
            o[i].z += y.z;
            o[i].w += y.w;
          }
        }
      }
      __syncthreads();   // shares are used again
      if (share > 0) continue;
    }
    const bool none = total == 0.f;   // no key that counts beside the sink
    if (s2 != -INFINITY) total += exp2f(s2 - M);
    const float inv = none ? 0.f : 1.0f / total;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float4 y = make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv);
      if (i == 3 && lane >= 16) {   // dims 448 .. 511, back
        const float4 w = __ldg(reinterpret_cast<const float4*>(a.q_rope + static_cast<size_t>(row / static_cast<unsigned>(a.H)) * 64) + (lane - 16));
        y = make_float4(y.x * w.x + y.y * w.y, y.y * w.x - y.x * w.y, y.z * w.z + y.w * w.w, y.w * w.z - y.z * w.w);
      }
      *reinterpret_cast<uint2*>(a.out + (static_cast<size_t>(row) * kD + 128 * i + 4 * lane) * 2) =
          make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
    }
    if (a.lse != nullptr && lane == 0) a.lse[row] = none ? sink : (M + log2f(total)) * kLn2;
  }
}

inline size_t a256(size_t x) { return (x + 255) & ~size_t(255); }

// How the row blocks and the workspace follow from the sizes alone.
struct Layout {
  int group, most_blocks;
  size_t head, req, item, list, share, split, flags, bad, images, opart, ml, bytes;
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
  l.item = take(sizeof(ItemPlan) * static_cast<size_t>(items + 1));
  l.list = take(sizeof(ItemPlan) * static_cast<size_t>(std::min<int64_t>(items, kPlanStaged)));
  l.share = take(sizeof(SharePlan) * l.most_blocks);
  l.split = take(sizeof(SplitPlan) * l.most_blocks);
  l.flags = take(keys);
  l.bad = take(keys / kDecodeRows);
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
  a.head_inv = (65535 + H) / H;
  a.most_blocks = l.most_blocks;
  a.head = reinterpret_cast<ChunkHead*>(ws + l.head);
  a.req = reinterpret_cast<ReqPlan*>(ws + l.req);
  a.item = reinterpret_cast<ItemPlan*>(ws + l.item);
  a.list = reinterpret_cast<ItemPlan*>(ws + l.list);
  a.share = reinterpret_cast<SharePlan*>(ws + l.share);
  a.split = reinterpret_cast<SplitPlan*>(ws + l.split);
  a.flags = ws + l.flags;
  a.bad = ws + l.bad;
  a.images = ws + l.images;
  a.opart = reinterpret_cast<float*>(ws + l.opart);
  a.ml = reinterpret_cast<float2*>(ws + l.ml);
  a.spin = spin_limit();
  const int64_t decode_warps = (max_keys + kDecodeRows - 1) / kDecodeRows;
  const unsigned decode_blocks = static_cast<unsigned>(std::min<int64_t>(
      2 * kPairs * kPrepBlocks - 1, std::max<int64_t>(1, (decode_warps + kPrepThreads / 32 - 1) / (kPrepThreads / 32))));
  cudaError_t e;
  if (R <= kOwnReqs) {
    chunk_prepare_kernel<<<1 + decode_blocks, kPrepThreads, 0, stream>>>(a);
    e = cudaGetLastError();
  } else {
    chunk_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_next(chunk_decode_kernel, decode_blocks, kPrepThreads, 0, stream, nullptr, a);
  }
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> allowed;
  e = launch_next(chunk_attn_kernel, 2 * l.most_blocks, kThreads, kChunkSmemBytes, stream, &allowed, a);
  if (e != cudaSuccess || l.most_blocks == 1) return e;
  return launch_next(chunk_join_kernel, kJoinSets * l.most_blocks, kJoinThreads, 0, stream, nullptr, a);
}

unsigned int take_err_chunk_attn() { return take_dev_err(); }

}  // namespace cskv
