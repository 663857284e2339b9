// Prefill attention over the block-scaled 8-bit cache.
//
// Mathematics as in kv8_decode.cu: s_i = scale * a * (q . K_i), out = sum_i
// 2^(s_i - M) b V_i / L with the page scales a (keys) and b (values). Both
// products run in f16: E4M3 codes are exact in f16, and so is a bf16 q times a
// power of two of its own row (2^14 for the row's largest |q|: 8 significant
// bits down to 2^-28 of that). A weight is held as 8 b 2^(s_i - m) <= 2^15 in
// f16: 11 significant bits down to 2^-17 of the reference, 8 down to 2^-20; its
// exponent comes from one multiply-add, y = S g + (log2 8b - m), and the sum L
// is kept in fp32 of the unrounded weights, page by page (a page's sum divided
// by 8 b).
//
// The reference m of a row is the largest s_i + log2 b_i of its first tile with
// anything to see and moves only when a tile passes it by more than 2^12. Every
// decision is the row's own, tiles start at multiples of 128 positions, and a
// tile in which a row sees nothing adds zeros: a token's bits depend on its
// request's cache and its own q alone.
//
// Work split: query rows are (token, head of the group) pairs of one kv head,
// in order, so that a K/V tile serves the whole group; an item is 256 rows (two
// row tiles of 128), one kv head, and all positions they see. A small kernel
// first numbers the tiles of all items; one CTA per SM then takes an equal run
// of them. A run that ends inside an item hands the rows' state (reference,
// sum and fp32 outputs) to the next CTA, which continues where it stopped: the
// same operations in the same order, so that where runs are cut changes no
// bit. A CTA does the piece that it hands over first and the piece that it
// takes over last, so that nobody waits where runs are longer than items, and
// the launch is cooperative (every CTA resident), so that a wait always ends.
// (512 equal items on 152 SMs would otherwise take 4 rounds for 3.4 rounds of
// work.) What this does not do is walk one item's positions in parallel: the
// grid has at most as many CTAs as there are items, and the CTAs of an item
// longer than a run follow one another. 16 tokens on 32768 positions, 64 / 8 heads
// x 128, are 8 items: 450 us (decode, which cuts contexts, takes 75).
//   softmax warps    thread = row = TMEM lane; with dim 64 two threads share a
//                    row, a page of the tile each. With dim 128, P over S, the
//                    tensor pipe and the memory of S and O bound the loop, and
//                    reading S twice for want of registers costs more than the
//                    shorter way to P gives: ragged prompts of dim 64 took 293 us
//                    so and 332 with one thread a row, a chunk of dim 128 took
//                    1767 us with one thread and 1965 with two;
//   4 loader warps   codes from global memory, through registers, to f16 tiles
//                    of K and V in shared memory (two buffers each): the copy
//                    engine cannot widen them, and staging the codes in shared
//                    memory first would cost 64 KB of its bandwidth a tile;
//   MMA issuer       (a warp) S = Q K^T (M 128, N 128), O += P V with P from
//                    TMEM. One row tile's products run under the other's
//                    softmax. With dim 128 P lies over S; with dim 64 there is
//                    room for P apart, and the next S is computed under this
//                    one's softmax. (An M 128 product takes 64 cycles a K of 16
//                    from N 64 to N 128, so that S by pages of 64 positions, two
//                    in flight, took 2073 us.)
//   a last warp      looks the pieces up ahead of the others.
//
// The bound is the way S -> softmax -> P -> O of a row tile: two of them in turn
// keep the tensor pipe busy half the time (dim 128; the last 2048 of 32768
// positions, 64 / 8 heads: 1769 us, 1204 TFLOP/s; 12 ragged prompts of dim 64, 28 /
// 4 heads: 292 us). Shared memory is near: an M 128 x N 128 x K 16 product reads
// 8 KB in its 64 cycles, and without the loader's stores the chunk took 1486 us,
// without the softmax 1410.

#include <cuda_runtime.h>
#include <stdint.h>

#include "kv8_common.cuh"
#include "kv8_join.cuh"

namespace dsmla {

namespace {

constexpr int kTile = 128;               // positions per K/V tile (two pages)
constexpr int kRows = 256;               // query rows per CTA
constexpr int kErrPage = DS_DEVERR_PAGE, kErrTimeout = DS_DEVERR_TIMEOUT;
constexpr int kMaxCtas = 192;
// Trees of drafts: contexts are cut so that few requests fill the GPU too, into at most
// 8 spans. An item costs about 8 us beside its tiles (q, the first S, partial outputs), the
// join about 20. us with at most 1 / 4 / 8 / 16 spans, 64 / 8 heads x 128, one build, inputs
// not in L2:
//   16 requests on 4096 to 32768 positions   24 nodes 614 / 399 / 440 / 507   12: 576 / 330 / 363 / 413
//   one on 32768                             24 nodes 607 / 189 / 116 / 80    12: 564 / 174 / 105 / 75
//   4 on 3000 to 8000                        24 nodes 165 /  86 /  79 / 78    12: 165 /  76 /  76 / 72
// 8 lie between: 4 are 10 % faster for the batch and 60 % slower for one request.
using TreeSpans = SpanRule<1024, 1 << 28, 8>;

// What the first kernel writes: item (unit u of one kv head) has weight
// first[u + 1] - first[u]: its tiles and kItemCost for its queries and outputs
// (about that many tiles' time), 0 for a unit without rows.
constexpr int kItemCost = 5;
// (Rows of a request are counted in 31 bits: num_tokens * group < 2^31.)
struct alignas(32) UnitInfo {
  int32_t r, t0, n;      // request, its first token, its tokens
  int32_t row0;          // first row of the request's rows; < 0: none
  int32_t raw_len;
  int32_t jb, span;      // first tile, and number of the span (trees; else 0)
};
struct Plan {
  int64_t* first;        // [units + 1]
  UnitInfo* info;        // [units]
  int32_t* flags;        // [kMaxCtas]
  uint8_t* state;        // [kMaxCtas] x state_bytes
};
// O [dim / 4][256 rows] float4, then (reference, sum, unset, NaN) for either
// half (unset 2: the row has seen scores too low for a reference) and the NaN
// bits.
__host__ __device__ constexpr int64_t state_bytes(int dim) {
  return (int64_t)kRows * (dim * 4 + 32 + dim / 8);
}

template <int DIM>
struct Layout {
  static constexpr int kBlock = kTile * 128;              // 64 dims of 128 rows in f16
  static constexpr int kTileBytes = DIM / 64 * kBlock;
  static constexpr int kQ = 0;                            // two row tiles
  static constexpr int kK = kQ + 2 * kTileBytes;          // two buffers
  static constexpr int kV = kK + 2 * kTileBytes;          // two buffers
  static constexpr int kBars = kV + 2 * kTileBytes;
  static constexpr int kMeta = kBars + 32 * 8;            // 4 tiles x 2 pages x float4
  static constexpr int kPiece = kMeta + 4 * 32;           // 2 x 64 bytes
  static constexpr int kNanMap = kPiece + 128;            // 2 x [128][DIM / 16] u16
  static constexpr int kNanMapBytes = kTile * (DIM / 16) * 2;
  static constexpr int kRowNan = kNanMap + 2 * kNanMapBytes;   // [256][DIM / 16] u16
  static constexpr int kFactor = kRowNan + kRows * (DIM / 16) * 2;   // [256] floats
  static constexpr int kSwap = kFactor + kRows * 4;              // [256][2] floats
  static constexpr int kMisc = kSwap + kRows * 8;
  static constexpr int kEnd = kMisc + 64;
  static constexpr int kSmem = kEnd + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // Warps: kShare threads share a row (warps of 32 rows: 4 * kShare a row tile),
  // then 4 loader warps and the MMA issuer's four.
  static constexpr int kShare = DIM == 64 ? 2 : 1;
  static constexpr int kLoaderWarp = 8 * kShare, kMmaWarp = kLoaderWarp + 4;
  static constexpr int kRowThreads = 128 * kShare;          // of a row tile
  static constexpr int kThreads = 32 * (kMmaWarp + 4);
  static constexpr int kPieceReaders = 2 * kRowThreads + 128 + 32;
  // Registers: 512 threads launch with 128 each, 768 with 80.
  static constexpr int kRegsSoftmax = kShare == 2 ? 80 : 160;
  static constexpr int kRegsLoader = 120, kRegsMma = kShare == 2 ? 40 : 72;
  static_assert(2 * kRowThreads * kRegsSoftmax + 128 * (kRegsLoader + kRegsMma) <=
                kThreads * (65536 / kThreads / 8 * 8), "registers of the launch");
  // TMEM columns: S and O of both row tiles and, where there is room, P; else P
  // lies over the upper half of S.
  static constexpr bool kApart = DIM == 64;
  static constexpr uint32_t kS = 0, kO = 2 * kTile;
  static constexpr uint32_t kP = kApart ? kO + 2 * DIM : kS + 64, kPStep = kApart ? 64 : kTile;
  static constexpr uint32_t kCols = 512u;
  static_assert((kApart ? kP + 2 * kPStep : kO + 2 * DIM) <= kCols, "TMEM columns");
};

enum Bar {
  kQFull = 0,       // 2 (row tile): its softmax threads
  kKFull = 2,       // 2: the 128 loader threads
  kKEmpty = 4,      // 2: commit
  kVFull = 6,       // 2: the 128 loader threads
  kVEmpty = 8,      // 2: commit
  kSFull = 10,      // 2 (row tile): commit
  kPFull = 12,      // 2: the row tile's softmax threads
  kPvDone = 14,     // 2: commit
  kPieceFull = 16,  // 2: the scheduling lane
  kPieceEmpty = 18, // 2: every thread that reads pieces
  kSFree = 20,      // 2: the row tile's softmax threads have read S (P apart)
  kDrain = 22,
  kNumBars = 23
};

// One run of tiles [j0, j1) of an item. r < 0 ends the list.
struct alignas(64) Piece {
  int32_t r, t0, n, row0, raw_len;
  int32_t kvh, nt, j0, j1;
  int32_t take, give;    // state slots to continue from / to hand over to, or -1
  int32_t jb, span;      // tile j of the piece is tile jb + j of the request
};

struct Params {
  const __nv_bfloat16* q;
  int64_t q_stride;
  int64_t tokens;
  const int32_t* starts;
  int heads, group;
  int64_t units;         // items of one kv head, an upper bound
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  Plan plan;
  Kv8Cache c;
  // Trees of drafts: every request has next_n tokens, its context is cut into spans,
  // and a unit is (request, span, 256 rows).
  int next_n, row_units, rows;   // units of a span; rows of a unit's slot
  const uint64_t* masks;         // [requests, next_n]
  int64_t spans;                 // slots of a request
  float* part_o;
  float2* part_ml;
};

__device__ __forceinline__ int clamp_pos(const Params& p, int64_t v) {
  const int64_t most = p.c.bt_stride * kPage;
  return (int)(v < 0 ? 0 : (v > most ? most : v));
}
// Positions that a row of the request sees.
__device__ __forceinline__ int visible(const Params& p, int raw_len, int n, int row) {
  return clamp_pos(p, (int64_t)raw_len - n + 1 + row / p.group);
}
__device__ __forceinline__ int last_row_of(const Params& p, int row0, int n) {
  const int left = n * p.group - row0;
  return row0 + (left < kRows ? left : kRows) - 1;
}
// Tiles of an item.
__device__ __forceinline__ int item_tiles(const Params& p, int raw_len, int n, int row0) {
  return (visible(p, raw_len, n, last_row_of(p, row0, n)) + kTile - 1) / kTile;
}

// Trees: unit (request, span, 256 rows).
__device__ __forceinline__ UnitInfo tree_unit(const Params& p, int64_t u, int* weight) {
  UnitInfo i;
  const int64_t rs = u / p.row_units;
  i.r = (int)(rs / p.spans);
  i.span = (int)(rs % p.spans);
  i.t0 = i.r * p.next_n;
  i.n = p.next_n;
  i.raw_len = p.c.lens[i.r];
  const int len = clamp_pos(p, i.raw_len), span = TreeSpans::of(len);
  const int tiles = (len + kTile - 1) / kTile;
  i.jb = i.span * (span / kTile);
  const int left = tiles - i.jb;
  i.row0 = -1;
  *weight = 0;
  if (i.span == 0 || left > 0) {     // (an empty request has one unit, for its outputs)
    i.row0 = (int)(u % p.row_units) * kRows;
    *weight = (left < span / kTile ? left : span / kTile) + kItemCost;
  }
  return i;
}

// Units of request r are numbered from floor(starts[r] * group / 256) + r (at
// least as many as it has); one CTA finds each unit's request and numbers the
// tiles.
template <bool TREE>
__global__ void __launch_bounds__(1024) kv8_prefill_plan_kernel(const Params p) {
  __shared__ int64_t part[32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < kMaxCtas) p.plan.flags[tid] = 0;
  auto start_of = [&](int64_t r) {
    const int64_t s = p.starts[r];
    return s < 0 ? 0 : (s > p.tokens ? p.tokens : s);
  };
  const int64_t per = (p.units + 1023) / 1024;
  const int64_t u0 = tid * per, u1 = u0 + per < p.units ? u0 + per : p.units;
  int64_t sum = 0;
  if constexpr (TREE) {
    for (int64_t u = u0; u < u1; ++u) {
      int w;
      p.plan.info[u] = tree_unit(p, u, &w);
      p.plan.first[u] = sum;     // within the thread's run; completed below
      sum += w;
    }
  } else if (u0 < u1) {
    // The request of the first unit; the others follow.
    int64_t lo = 0, hi = p.c.requests - 1;
    while (lo < hi) {
      const int64_t mid = (lo + hi + 1) >> 1;
      if (start_of(mid) * p.group / kRows + mid <= u0)
        lo = mid;
      else
        hi = mid - 1;
    }
    int64_t r = lo, t0 = start_of(r), t1 = start_of(r + 1);
    int raw = p.c.lens[r];
    for (int64_t u = u0; u < u1; ++u) {
      while (r + 1 < p.c.requests && t1 * p.group / kRows + r + 1 <= u) {
        ++r;
        t0 = t1;
        t1 = start_of(r + 1);
        raw = p.c.lens[r];
      }
      UnitInfo i;
      i.r = (int)r;
      i.t0 = (int)t0;
      i.n = (int)(t1 > t0 ? t1 - t0 : 0);
      i.raw_len = raw;
      i.jb = i.span = 0;
      const int64_t row0 = (u - (t0 * p.group / kRows + r)) * kRows;
      i.row0 = -1;
      int w = 0;
      if (row0 >= 0 && row0 < (int64_t)i.n * p.group) {
        i.row0 = (int)row0;
        w = item_tiles(p, raw, i.n, i.row0) + kItemCost;
      }
      p.plan.info[u] = i;
      p.plan.first[u] = sum;     // within the thread's run; completed below
      sum += w;
    }
  }
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  int64_t before = inc - sum, total = 0;
  for (int w = 0; w < 32; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  if (before != 0)
    for (int64_t u = u0; u < u1; ++u) p.plan.first[u] += before;
  if (tid == 0) p.plan.first[p.units] = total;
}

// The pieces of CTA `blockIdx.x`, one after the other.
struct Scheduler {
  const Params& p;
  int64_t per_head, lo, hi;       // weight of a kv head; the CTA's run
  int64_t i0, i1, at;             // items kvh * units + u of its ends; the next one
  int phase;

  // The item that holds weight x.
  __device__ int64_t find(int64_t x) const {
    const int64_t head = x / per_head;
    x -= head * per_head;
    int64_t a = 0, b = p.units - 1;   // last unit with first[u] <= x
    while (a < b) {
      const int64_t mid = (a + b + 1) >> 1;
      if (p.plan.first[mid] <= x)
        a = mid;
      else
        b = mid - 1;
    }
    return head * p.units + a;        // (its weight is not 0)
  }
  // The first item with a weight behind item i, which has none (requests without
  // tokens are such units, any number of them in a row). The one at i1 has.
  __device__ int64_t skip(int64_t i) const {
    return find(i / p.units * per_head + p.plan.first[i % p.units]);
  }
  __device__ explicit Scheduler(const Params& params) : p(params) {
    per_head = p.plan.first[p.units];
    const int64_t total = per_head * p.c.kv_heads;
    // Every run holds something, so that the CTA before is the one that hands over:
    // where the call's requests have less than a weight a CTA (most of them
    // without tokens), the last CTAs have no run.
    const int64_t n = total < gridDim.x ? total : gridDim.x;
    phase = 3;
    if (blockIdx.x >= n) return;
    lo = total * blockIdx.x / n;
    hi = total * (blockIdx.x + 1) / n;
    i0 = find(lo);
    i1 = find(hi - 1);
    at = i0;
    phase = 0;
  }
  // The CTA's tiles of item i: from its own start where the run begins in the
  // item's cost, none where it ends there. r < 0: no piece; nt < 0: no such item.
  __device__ Piece piece(int64_t i) const {
    Piece x;
    x.r = -1;
    const int64_t u = i % p.units;
    const int64_t s = i / p.units * per_head + p.plan.first[u];
    const int nt = (int)(p.plan.first[u + 1] - p.plan.first[u]) - kItemCost;
    x.nt = nt;
    if (nt < 0) return x;
    auto tile_of = [&](int64_t w) {
      const int64_t t = w - s - kItemCost;
      return (int)(t < 0 ? 0 : (t > nt ? nt : t));
    };
    x.j0 = tile_of(lo);
    x.j1 = tile_of(hi);
    if (nt > 0 ? x.j0 >= x.j1 : (s < lo || s >= hi)) return x;
    const UnitInfo info = p.plan.info[u];
    x.r = info.r;
    x.row0 = info.row0;
    x.t0 = info.t0;
    x.n = info.n;
    x.raw_len = info.raw_len;
    x.jb = info.jb;
    x.span = info.span;
    x.kvh = (int)(i / p.units);
    x.take = x.j0 > 0 ? (int)blockIdx.x - 1 : -1;
    x.give = x.j1 < nt ? (int)blockIdx.x : -1;
    return x;
  }
  // First what the next CTA waits for, last what the CTA before has begun.
  __device__ Piece next() {
    Piece x;
    if (phase == 0) {
      phase = 1;
      if (i1 != i0) {
        x = piece(i1);
        if (x.r >= 0 && x.give >= 0) return x;
      }
    }
    while (phase == 1) {
      if (at > i1) {
        phase = 2;
        break;
      }
      x = piece(at);
      at = x.nt < 0 ? skip(at) : at + 1;
      if (x.r < 0 || (i0 != i1 && (x.take >= 0 || x.give >= 0))) continue;
      return x;
    }
    if (phase == 2) {
      phase = 3;
      if (i0 != i1) {
        x = piece(i0);
        if (x.r >= 0 && x.take >= 0) return x;
      }
    }
    x.r = -1;
    return x;
  }
};

// TREE: the rows are nodes of a tree of drafts: all see the positions before the
// drafts, and draft i where bit i of their mask is set; items are spans, and a span
// of several gives its part to the join.
template <int DIM, bool TREE>
__global__ void __launch_bounds__(Layout<DIM>::kThreads, 1) kv8_prefill_kernel(const Params p) {
  using LY = Layout<DIM>;
  constexpr int kMmaWarp = LY::kMmaWarp, kLoaderWarp = LY::kLoaderWarp, H = LY::kShare;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + LY::kBars);
  float4* meta = reinterpret_cast<float4*>(smem + LY::kMeta);
  Piece* pieces = reinterpret_cast<Piece*>(smem + LY::kPiece);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + LY::kMisc);
  volatile uint32_t* nan_tag = reinterpret_cast<volatile uint32_t*>(smem + LY::kMisc + 8);   // 2
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t count = 1u;
      if ((i >= kKFull && i < kKEmpty) || (i >= kVFull && i < kVEmpty)) count = 128u;
      if (i < kKFull || (i >= kPFull && i < kPvDone) || (i >= kSFree && i < kDrain)) count = LY::kRowThreads;
      if (i >= kPieceEmpty && i < kSFree) count = LY::kPieceReaders;
      mbar_init(&bars[i], count);
    }
    mbar_fence_init();
    nan_tag[0] = nan_tag[1] = 0;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, LY::kCols);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The next piece, in shared memory until piece_done() (every reader calls both
  // in step; r < 0: no more).
  uint32_t np = 0;
  bool failed = false;
  auto next_piece = [&]() {
    const bool ok = mbar_wait_long(&bars[kPieceFull + (np & 1)], (np >> 1) & 1);
    if (!__all_sync(0xffffffffu, ok)) failed = true;
    return const_cast<const volatile Piece*>(&pieces[np & 1]);
  };
  auto piece_done = [&]() {
    mbar_arrive(&bars[kPieceEmpty + (np & 1)]);
    ++np;
  };

  if (warp < kLoaderWarp) {
    // ----------------------------------------------------------- softmax
    if constexpr (LY::kRegsSoftmax > 80) regs_inc<LY::kRegsSoftmax>();
    // Row tile; with two threads a row, which page of a tile and half of the dims
    // is this one's (else both).
    const int m = warp / (4 * H), half = H == 2 ? (warp >> 2) & 1 : 0;
    const int row = (warp & 3) * 32 + lane;          // TMEM lane
    const int pair = 1 + m * 4 + (warp & 3);         // named barrier of the rows' two warps
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_base + LY::kS + m * kTile + half * kPage;
    const uint32_t t_o = tmem + lane_base + LY::kO + m * DIM + half * (DIM / H);
    const uint32_t t_p = tmem + lane_base + LY::kP + m * LY::kPStep + half * (kPage / 2);
    constexpr int NB = DIM / 16 / H;                 // words of NaN bits of this thread's dims
    uint16_t* const row_bits = reinterpret_cast<uint16_t*>(smem + LY::kRowNan) +
                               (m * kTile + row) * (DIM / 16) + half * NB;
    float* const factor = reinterpret_cast<float*>(smem + LY::kFactor) + m * kTile;
    float* const swap = reinterpret_cast<float*>(smem + LY::kSwap) + (m * kTile + row) * 2;
    // Waits are the warp's, and none follows one that gave up: the piece runs to
    // its end without meaning.
    auto wait = [&](int bar, uint32_t phase) {
      if (!failed && !__all_sync(0xffffffffu, mbar_wait_long(&bars[bar], phase & 1)))
        failed = true;
    };
    uint32_t tiles = 0;        // tiles of this row tile so far
    uint32_t kv = 0;           // tiles of the CTA so far
    while (true) {
      const volatile Piece& x = *next_piece();
      // (Two warps of the same rows give up together: neither waits for one that left.)
      if constexpr (H == 2) failed = named_bar_or(pair, 64, failed);
      if (failed || x.r < 0) break;
      const int first = x.row0 + m * kTile;            // rows of the row tile
      const int rows = x.n * p.group - first;          // at most 128 of them exist
      const bool any = rows > 0;
      // TREE: the first draft's position and the row's drafts; a row sees something
      // up to `vis`.
      const int64_t base = (int64_t)x.raw_len - x.n;
      uint64_t drafts = 0;
      int vis, min_vis;
      if constexpr (TREE) {
        if (row < rows) {
          drafts = p.masks[(int64_t)x.r * p.next_n + (first + row) / p.group];
          if (p.next_n < 64) drafts &= (1ull << p.next_n) - 1;
        }
        vis = row < rows ? clamp_pos(p, base + 64 - __clzll((long long)drafts)) : 0;
        min_vis = clamp_pos(p, base);
      } else {
        vis = row < rows ? visible(p, x.raw_len, x.n, first + row) : 0;
        min_vis = visible(p, x.raw_len, x.n, x.row0);
      }
      // TREE: what the row sees of the 64 positions from `from` on, a bit each.
      auto sees = [&](int from) {
        if (row >= rows) return (uint64_t)0;
        const int64_t e = base - from;
        if (e >= 64) return ~(uint64_t)0;
        if (e > 0) return ((uint64_t)1 << e) - 1 | drafts << e;
        return e > -64 ? drafts >> -e : (uint64_t)0;
      };
      // Element offset of a row of this warp in q (stride q_stride) or out.
      auto offset = [&](int i, int64_t stride) {
        const int rr = first + (warp & 3) * 32 + i;
        return (x.t0 + rr / p.group) * stride + (x.kvh * p.group + rr % p.group) * DIM;
      };
      const int left = rows - (warp & 3) * 32;         // rows of this warp that exist
      float f = 0.0f;
      if (any && x.j1 > x.j0) {
        // The rows' q, each times a power of two of its own, in f16. A warp does
        // its 32 rows, or 16 of them, RI at a time.
        constexpr int RL = DIM / 8, RI = 32 / RL;      // lanes of a row; rows of a step
        constexpr int NR = RL / H;                     // steps
        const int sub = lane / RL, ch = lane % RL;     // row of the step, 16-byte chunk
        uint4 v[NR];
        {
          // From a row to the one RI behind it without a division each (half of this
          // stretch's instructions, which took 8000 cycles of an item).
          const int r0 = first + (warp & 3) * 32 + half * 16 + sub;
          const int tokens = RI / p.group, heads = RI % p.group;
          const int64_t step = tokens * p.q_stride + heads * DIM;
          const int64_t wrap = p.q_stride - (int64_t)p.group * DIM;
          int head = r0 % p.group;
          const __nv_bfloat16* at = p.q + offset(half * 16 + sub, p.q_stride) + ch * 8;
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (half * 16 + i * RI + sub < left) v[i] = *reinterpret_cast<const uint4*>(at);
            head += heads;
            at += step;
            if (head >= p.group) {
              head -= p.group;
              at += wrap;
            }
          }
        }
        // Largest magnitude bits of the rows (NaN above infinity), two values a word:
        // reduced over a row's lanes so that lane ch ends with step ch / H's alone, and
        // works its factors out for all.
        uint32_t t[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i)
          t[i] = __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                          __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
#pragma unroll
        for (int o = RL / 2, n = NR; o > 0; o >>= 1) {
          if (n > 1) {
            n /= 2;
            const bool upper = (ch & o) != 0;
#pragma unroll
            for (int i = 0; i < NR / 2; ++i)
              if (i < n) {
                const uint32_t keep = upper ? t[i + n] : t[i], give = upper ? t[i] : t[i + n];
                t[i] = __vmaxu2(keep, __shfl_xor_sync(0xffffffffu, give, o));
              }
          } else {
            t[0] = __vmaxu2(t[0], __shfl_xor_sync(0xffffffffu, t[0], o));
          }
        }
        const uint32_t top = max(t[0] << 16, t[0] & 0xFFFF0000u);
        // Largest |q| 2^k in [2^14, 2^15); 2^k stays a normal float.
        int k = top > 0u ? 14 - ((int)(top >> 23) - 127) : 0;
        k = k > 120 ? 120 : (k < -120 ? -120 : k);
        const float up = copysignf(__uint_as_float((uint32_t)(k + 127) << 23), p.scale_log2);
        const float mine =
            top >= 0x7F800000u
                ? NAN
                : __uint_as_float((uint32_t)(127 - k) << 23) * fabsf(p.scale_log2);
        if constexpr (H == 2) {
          if (ch % H == 0) factor[(warp & 3) * 32 + half * 16 + ch / H * RI + sub] = mine;
        } else {
          f = __shfl_sync(0xffffffffu, mine, (lane % RI) * RL + lane / RI);
        }
        uint8_t* dst = smem + LY::kQ + m * LY::kTileBytes + (ch >> 3) * LY::kBlock;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int rr = (warp & 3) * 32 + half * 16 + i * RI + sub;
          const float by = __shfl_sync(0xffffffffu, up, sub * RL + i * H);
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          uint32_t h[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const __half2 y = __floats2half2_rn(__uint_as_float(w[u] << 16) * by,
                                                __uint_as_float(w[u] & 0xFFFF0000u) * by);
            h[u] = *reinterpret_cast<const uint32_t*>(&y);
          }
          *reinterpret_cast<uint4*>(dst + swz<128>(rr, (ch & 7) * 16)) =
              make_uint4(h[0], h[1], h[2], h[3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(&bars[kQFull + m]);
        if constexpr (H == 2) {
          named_bar_sync(pair, 64);
          f = factor[row];
        }
      }
      float ref = 0.0f, l = 0.0f;              // l: of this half's page
      bool unset = vis > 0, row_nan = false;   // (a row that sees nothing needs no reference)
      bool low = false;                        // without one, the row saw scores too low for it
      if (x.take >= 0) {
        // Continue from the CTA before: it does this piece first.
        const uint8_t* st = p.plan.state + x.take * state_bytes(DIM);
        const uint64_t began = clock64();
        bool there = true;
        while (true) {
          int flag;
          asm volatile("ld.acquire.gpu.global.s32 %0, [%1];"
                       : "=r"(flag)
                       : "l"(p.plan.flags + x.take)
                       : "memory");
          if (flag == 2 * LY::kRowThreads) break;   // all softmax threads have written theirs
          if ((uint64_t)(clock64() - began) > (1ull << 32)) {
            there = false;
            break;
          }
          __nanosleep(200);
        }
        if (!__all_sync(0xffffffffu, there)) failed = true;
        const int rr = m * kTile + row;
        const float4* so = reinterpret_cast<const float4*>(st) + half * (DIM / 4 / H) * kRows;
#pragma unroll 4
        for (int d = 0; d < DIM / H; d += 4) {
          const float4 o = so[(d / 4) * kRows + rr];
          const float v[4] = {o.x, o.y, o.z, o.w};
          tmem_st4(t_o + d, v);
        }
        tmem_wait_st();
        const float4 ml =
            reinterpret_cast<const float4*>(st + kRows * DIM * 4)[half * kRows + rr];
        ref = ml.x;
        l = ml.y;
        unset = ml.z != 0.0f;
        low = ml.z == 2.0f;
        row_nan = ml.w != 0.0f;
        const uint16_t* sn =
            reinterpret_cast<const uint16_t*>(st + kRows * (DIM * 4 + 32)) + half * NB * kRows;
        if (row_nan)
          for (int c = 0; c < NB; ++c) row_bits[c] = sn[c * kRows + rr];
      }
      // Moves the reference by a whole number of powers of two to 3 above the row's
      // largest exponent y, and the sum and the outputs of the tiles before with it
      // (PV of the last one may still run). Returns the outputs' factor.
      auto move_reference = [&](bool move, float y, int j) {
        const float by = move ? reference_step(ref, ceilf(y)) : 0.0f;
        const float al = by == 0.0f ? 1.0f
                         : unset || by > 126.0f
                             ? 0.0f
                             : __uint_as_float((uint32_t)(127 - (int)by) << 23);
        if (move) {
          ref += by;
          l *= al;
          unset = false;
        }
        if (j > 0 && __any_sync(0xffffffffu, al != 1.0f)) {
          if (j > x.j0) wait(kPvDone + m, tiles - 1);
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < DIM / H; c += 16) {
            float o[16];
            tmem_ld<16>(t_o + c, o);
            tmem_fence<16>(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= al;
#pragma unroll
            for (int i = 0; i < 16; i += 4) tmem_st4(t_o + c + i, o + i);
          }
          tmem_wait_st();
        }
        return al;
      };
      uint32_t g = kv;         // tile of the CTA
      for (int j = any ? x.j0 : x.j1; j < x.j1; ++j, ++g) {
        const int pos0 = (TREE ? x.jb + j : j) * kTile;
        if constexpr (H == 2) {
          wait(kSFull + m, tiles);
        } else if (!__all_sync(0xffffffffu, mbar_wait_long(&bars[kSFull + m], tiles & 1))) {
          failed = true;
          break;
        }
        tc_fence_after();
        if constexpr (H == 2) {
          // This thread's page: (key scale, log2 of 8 times the value scale, its
          // reciprocal, valid). Its S is read twice, for the largest and for the
          // weights: 64 values do not fit in the registers of 24 warps.
          const float4 mt = meta[(g & 3) * 2 + half];
          const int end = mt.w != 0.0f ? vis - pos0 - half * kPage : 0;
          const uint64_t bits = TREE && mt.w != 0.0f ? sees(pos0 + half * kPage) : 0;
          const float gg = f * mt.x;
          float s[32];
          // 32 columns of S, what the row does not see at -infinity.
          auto load = [&](int q) {
            tmem_ld32(t_s + 32 * q, s);
            tmem_fence<32>(s);
          };
          auto mask = [&](int q) {
            if constexpr (TREE) {
              const uint32_t b = (uint32_t)(bits >> (32 * q));
              if (b != 0xFFFFFFFFu) {
#pragma unroll
                for (int i = 0; i < 32; ++i) s[i] = (b >> i) & 1u ? s[i] : -INFINITY;
              }
            } else if (end < kPage) {
#pragma unroll
              for (int i = 0; i < 32; ++i) s[i] = 32 * q + i < end ? s[i] : -INFINITY;
            }
          };
          // Rarely a weight would pass 2^15 (or the row has no reference yet): again,
          // with a new one (3 above the largest, or NaN: the loop ends).
          while (true) {
            // (gg is not negative: the largest exponent is that of the largest S.)
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              load(q);
              mask(q);
#pragma unroll
              for (int i = 0; i < 32; i += 8)
#pragma unroll
                for (int k = 0; k < 4; ++k) top[k] = fmaxf(fmaxf(top[k], s[i + k]), s[i + 4 + k]);
            }
            float y =
                __fmaf_rn(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), gg, mt.y - ref);
            const float most = unset ? kLowest : 15.0f;
            low |= unset && y > -INFINITY;
            if (!named_bar_or(pair, 64, y > most)) break;
            swap[half] = y;
            named_bar_sync(pair, 64);
            y = fmaxf(swap[0], swap[1]);
            move_reference(y > most, y, j);
          }
          // The weights; P's columns are free once PV of the last tile has ended.
          if (tiles > 0) wait(kPvDone + m, tiles - 1);
          tc_fence_after();
          const float cc = mt.y - ref;
          const float2 g2 = make_float2(gg, gg), c2 = make_float2(cc, cc);
          float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            load(q);
            if (q == 1) {
              tc_fence_before();
              mbar_arrive(&bars[kSFree + m]);
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 e = fma2(make_float2(s[i], s[i + 1]), g2, c2);
              s[i] = e.x;
              s[i + 1] = e.y;
            }
            mask(q);
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 e = make_float2(ex2(s[i]), ex2(s[i + 1]));
              sum = add2(sum, e);
              const __half2 z = __floats2half2_rn(e.x, e.y);
              w[i / 2] = *reinterpret_cast<const uint32_t*>(&z);
            }
            tmem_st16u(t_p + 16 * q, w);
          }
          l = __fmaf_rn(sum.x + sum.y, mt.z, l);
        } else {
          // 64 columns (one page, one scale) at a time, positions 64-127 first: P
          // may go over the upper half of S, which is in registers by then.
          float2 s[32];
          float* const s1 = reinterpret_cast<float*>(s);
          const float4 mt0 = meta[(g & 3) * 2], mt1 = meta[(g & 3) * 2 + 1];
          // (key scale, log2 of 8 times the value scale, its reciprocal, valid)
          const int end0 = mt0.w != 0.0f ? vis - pos0 : 0, end1 = mt1.w != 0.0f ? vis - pos0 - 64 : 0;
          const uint64_t bits0 = TREE && mt0.w != 0.0f ? sees(pos0) : 0;
          const uint64_t bits1 = TREE && mt1.w != 0.0f ? sees(pos0 + kPage) : 0;
          const float g0 = f * mt0.x, g1 = f * mt1.x;
          // s = exponents relative to the reference; returns the largest.
          auto exponents = [&](int page) {
            tmem_ld32(t_s + 64 * page, s1);
            tmem_ld32(t_s + 64 * page + 32, s1 + 32);
            const float gg = page ? g1 : g0, cc = (page ? mt1.y : mt0.y) - ref;
            const float2 g2 = make_float2(gg, gg), c2 = make_float2(cc, cc);
            const int end = page ? end1 : end0;
            tmem_fence<64>(s1);
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] = fma2(s[i], g2, c2);
            if constexpr (TREE) {
              const uint64_t b = page ? bits1 : bits0;
              if (b != ~(uint64_t)0) {
#pragma unroll
                for (int i = 0; i < 64; ++i) s1[i] = (b >> i) & 1u ? s1[i] : -INFINITY;
              }
            } else if (end < 64) {
#pragma unroll
              for (int i = 0; i < 64; ++i) s1[i] = i < end ? s1[i] : -INFINITY;
            }
            float top[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) top[u] = fmaxf(s1[u], s1[4 + u]);
#pragma unroll
            for (int i = 8; i < 64; i += 8)
#pragma unroll
              for (int u = 0; u < 4; ++u) top[u] = fmaxf(fmaxf(top[u], s1[i + u]), s1[i + 4 + u]);
            return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          };
          // P of this tile's page 1, which nobody has read yet, moves with a reference
          // that page 0 moves.
          auto rebase = [&](bool move, float y, bool upper_in) {
            const float al = move_reference(move, y, j);
            if (upper_in && __any_sync(0xffffffffu, al != 1.0f)) {
#pragma unroll 1
              for (int c = 32; c < 64; c += 16) {
                float o[16];
                tmem_ld<16>(t_p + c, o);
                tmem_fence<16>(o);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  // (In fp32: al may be below f16's range where a weight times it is not.)
                  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&o[i]));
                  const __half2 w = __floats2half2_rn(x.x * al, x.y * al);
                  o[i] = *reinterpret_cast<const float*>(&w);
                }
#pragma unroll
                for (int i = 0; i < 16; i += 4) tmem_st4(t_p + c + i, o + i);
              }
              tmem_wait_st();
            }
          };
#pragma unroll
          for (int page = 1; page >= 0; --page) {
            // Rarely a weight would pass 2^15 (or the row has no reference yet): the
            // exponents again, with a new one (3 above the largest, or NaN: the loop
            // ends).
            while (true) {
              const float y = exponents(page);
              const bool move = y > (unset ? kLowest : 15.0f);
              low |= unset && y > -INFINITY;
              if (!__any_sync(0xffffffffu, move)) break;
              rebase(move, y, page == 0);
            }
            uint32_t h[32];
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float2 e = make_float2(ex2(s[i].x), ex2(s[i].y));
              sum = add2(sum, e);
              const __half2 w = __floats2half2_rn(e.x, e.y);
              h[i] = *reinterpret_cast<const uint32_t*>(&w);
            }
            tmem_st16u(t_p + 32 * page, h);
            tmem_st16u(t_p + 16 + 32 * page, h + 16);
            l = __fmaf_rn(sum.x + sum.y, page ? mt1.z : mt0.z, l);
            if (page == 1) tmem_wait_st();   // (page 0 may read it back)
          }
        }
        // Where rows see different lengths, NaN values were taken out of the tile
        // and listed: the rows that see one get a NaN in that dim.
        if (pos0 + kTile > min_vis) {
          wait(kVFull + (g & 1), g >> 1);
          if (nan_tag[g & 1] == g + 1) {
            const uint16_t* map =
                reinterpret_cast<const uint16_t*>(smem + LY::kNanMap + (g & 1) * LY::kNanMapBytes) +
                half * NB;
            if (!row_nan)
              for (int c = 0; c < NB; ++c) row_bits[c] = 0;
            row_nan = true;
            for (int i = 0; i < kTile && pos0 + i < vis; ++i) {
              if (TREE && !((sees(pos0 + i / 64 * 64) >> (i & 63)) & 1u)) continue;
              for (int c = 0; c < NB; ++c) row_bits[c] |= map[i * (DIM / 16) + c];
            }
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars[kPFull + m]);
        ++tiles;
      }
      kv += (uint32_t)(x.j1 - x.j0);
      if (any && x.j1 > x.j0) wait(kPvDone + m, tiles - 1);
      if constexpr (H == 2) failed = named_bar_or(pair, 64, failed);
      if (failed) break;
      tc_fence_after();
      if (x.give >= 0) {
        uint8_t* st = p.plan.state + x.give * state_bytes(DIM);
        const int rr = m * kTile + row;
        float4* so = reinterpret_cast<float4*>(st) + half * (DIM / 4 / H) * kRows;
        if (any) {
#pragma unroll 1
          for (int d = 0; d < DIM / H; d += 16) {
            float o[16];
            tmem_ld<16>(t_o + d, o);
            tmem_fence<16>(o);
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              so[(d + i) / 4 * kRows + rr] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        reinterpret_cast<float4*>(st + kRows * DIM * 4)[half * kRows + rr] =
            make_float4(ref, l, unset ? (low ? 2.0f : 1.0f) : 0.0f, row_nan ? 1.0f : 0.0f);
        uint16_t* sn = reinterpret_cast<uint16_t*>(st + kRows * (DIM * 4 + 32)) + half * NB * kRows;
        if (row_nan)
          for (int c = 0; c < NB; ++c) sn[c * kRows + rr] = row_bits[c];
        __threadfence();
        asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p.plan.flags + x.give)
                     : "memory");
        piece_done();
        continue;
      }
      if (!any) {
        piece_done();
        continue;
      }
      bool part = false;         // TREE: one of several spans
      if constexpr (TREE) part = clamp_pos(p, x.raw_len) > TreeSpans::of(clamp_pos(p, x.raw_len));
      if (unset && low && !part) l = NAN;
      if constexpr (H == 2) {
        // (Each thread has seen one page of a tile; a span reports for both.)
        if (part) low = named_bar_or(pair, 64, low);
        swap[half] = l;
        named_bar_sync(pair, 64);
        l = swap[0] + swap[1];
      }
      if (part) {
        // The row's part of the join: outputs relative to its reference, dims [dim / 4][rows]
        // so that a warp writes 512 bytes in a piece (rows of their own, 16 bytes each,
        // cost an item 4 us more), and (reference, sum). (The loads are the warp's, also
        // where only some of its rows exist.)
        const int64_t group = ((int64_t)x.r * p.c.kv_heads + x.kvh) * p.row_units + x.row0 / kRows;
        const int64_t slot0 = (group * p.spans + x.span) * p.rows;
        const int rr = m * kTile + row;
        float4* to = reinterpret_cast<float4*>(p.part_o + slot0 * DIM) +
                     half * (DIM / 4 / H) * p.rows + rr;
#pragma unroll 1
        for (int c = 0; c < DIM / H; c += 32) {
          float o[32];
          tmem_ld32(t_o + c, o);
          tmem_fence<32>(o);
          if (row_nan) {
            const uint32_t bits = row_bits[c >> 4] | (uint32_t)row_bits[(c >> 4) + 1] << 16;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((bits >> i) & 1) o[i] = NAN;
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= 0.125f;
          if (row < rows) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              to[(c + i) / 4 * p.rows] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
          __syncwarp();
        }
        if (half == 0 && row < rows)
          p.part_ml[slot0 + rr] = make_float2(unset ? (low ? kOnlyLow : -INFINITY) : ref, l);
        if constexpr (H == 2)
          named_bar_sync(pair, 64);
        else
          __syncwarp();
        piece_done();
        continue;
      }
      // Outputs by way of the row tile's Q buffer (its last S is long done), so
      // that rows are written in long pieces. A warp does its half of the dims.
      const float inv = l == 0.0f ? 0.0f : __fdiv_rn(0.125f, l);
      uint8_t* stage = smem + LY::kQ + m * LY::kTileBytes;
#pragma unroll 1
      for (int c = 0; c < DIM / H; c += 16) {
        const int d0 = half * (DIM / H) + c;
        float o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = 0.0f;
        if (x.nt > 0) {
          tmem_ld<16>(t_o + c, o);
          tmem_fence<16>(o);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = l == 0.0f ? 0.0f : o[i] * inv;
        if (row_nan) {
          const uint32_t bits = row_bits[c >> 4];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if ((bits >> i) & 1) o[i] = NAN;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t h[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const __nv_bfloat162 y = __floats2bfloat162_rn(o[8 * i + 2 * u], o[8 * i + 2 * u + 1]);
            h[u] = *reinterpret_cast<const uint32_t*>(&y);
          }
          *reinterpret_cast<uint4*>(stage + (d0 >> 6) * LY::kBlock +
                                    swz<128>(row, ((d0 >> 3) & 7) * 16 + i * 16)) =
              make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      __syncwarp();
      constexpr int OL = DIM / 8 / H, OI = 32 / OL;    // lanes of the row's part; rows of a step
#pragma unroll
      for (int i = 0; i < OL; ++i) {
        const int rr = i * OI + lane / OL, ch = half * OL + lane % OL;
        const uint4 y = *reinterpret_cast<const uint4*>(
            stage + (ch >> 3) * LY::kBlock + swz<128>((warp & 3) * 32 + rr, (ch & 7) * 16));
        if (rr < left)
          *reinterpret_cast<uint4*>(p.out + offset(rr, (int64_t)p.heads * DIM) + ch * 8) = y;
      }
      if (half == 0 && lane < left)
        p.lse[offset(lane, (int64_t)p.heads * DIM) / DIM] =
            l == 0.0f ? -INFINITY : (ref + log2f(l)) * kLn2;
      // The next Q goes over what the other warp may still read.
      if constexpr (H == 2)
        named_bar_sync(pair, 64);
      else
        __syncwarp();
      piece_done();
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------ loader
    if constexpr (LY::kRegsLoader > 65536 / LY::kThreads)
      regs_inc<LY::kRegsLoader>();
    else
      regs_dec<LY::kRegsLoader>();
    constexpr int NC = kTile * DIM / 16 / 128;     // 16-code chunks per thread and tile
    constexpr int RC = DIM / 16;                   // chunks per position
    const int lt = tid - kLoaderWarp * 32;
    const int64_t side = (int64_t)p.c.kv_heads * kPage * DIM;
    int err_bits = 0;
    uint32_t g = 0;                                // tiles so far
    while (true) {
      const volatile Piece& x = *next_piece();
      if (failed || x.r < 0) break;
      const int j0 = x.j0, j1 = x.j1, kvh = x.kvh;
      const int32_t* table = p.c.block_table + x.r * p.c.bt_stride;
      const int len = clamp_pos(p, x.raw_len);
      const int min_vis = TREE ? clamp_pos(p, (int64_t)x.raw_len - x.n)
                               : visible(p, x.raw_len, x.n, x.row0);
      const int jb = TREE ? x.jb : 0;
      // The pages of tile j (-1: none, or outside the pool).
      auto pages_of = [&](int j, int* pg) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          pg[h] = -1;
          const int b = (jb + j) * 2 + h;
          if (j < j1 && b * kPage < len) {
            const int v = table[b];
            if (v >= 0 && v < p.c.num_pages)
              pg[h] = v;
            else
              err_bits |= kErrPage;
          }
        }
      };
      // Chunk e of this thread: position lt / RC + e * 128 / RC of the tile.
      auto load = [&](const int* pg, int64_t off, uint4* v) {
#pragma unroll
        for (int e = 0; e < NC; ++e) {
          const int64_t page = pg[e / (NC / 2)];
          v[e] = make_uint4(0u, 0u, 0u, 0u);
          if (page >= 0)
            v[e] = __ldg(reinterpret_cast<const uint4*>(
                             p.c.pages +
                             ((page * 2) * p.c.kv_heads + kvh) * (int64_t)(kPage * DIM) + off) +
                         lt + (e % (NC / 2)) * 128);
        }
      };
      auto store = [&](uint8_t* dst, const uint4* v) {
#pragma unroll
        for (int e = 0; e < NC; ++e) {
          const int row = lt / RC + e * (128 / RC), c = lt % RC;
          const uint2 a = codes_to_f16(v[e].x), b = codes_to_f16(v[e].y),
                      d = codes_to_f16(v[e].z), h = codes_to_f16(v[e].w);
          // Lanes of the second column block store their upper 16 bytes first:
          // eight lanes then write eight different bank groups.
          uint8_t* at = dst + (c >> 2) * LY::kBlock + row * 128;
          const int o = (c >> 2) & 1, ch = (c & 3) * 2;
          const uint4 lo = make_uint4(a.x, a.y, b.x, b.y), hi = make_uint4(d.x, d.y, h.x, h.y);
          *reinterpret_cast<uint4*>(at + (((ch + o) ^ (row & 7)) << 4)) = o ? hi : lo;
          *reinterpret_cast<uint4*>(at + (((ch + 1 - o) ^ (row & 7)) << 4)) = o ? lo : hi;
        }
      };
      uint4 kx[NC], vx[NC];
      int now[2], next[2];
      float ks = 0.0f, vs = 1.0f;      // scales of page lt of the tile (threads 0 and 1)
      auto scales_of = [&](const int* pg) {
        ks = 0.0f;
        vs = 1.0f;
        const int64_t page = lt == 0 ? pg[0] : pg[1];
        if (lt < 2 && page >= 0) {
          const int64_t part = page * 2 * p.c.kv_heads + kvh;
          ks = p.c.scales[part];
          vs = p.c.scales[part + p.c.kv_heads];
        }
      };
      pages_of(j0, now);
      pages_of(j0 + 1, next);
      load(now, 0, kx);
      load(now, side, vx);
      scales_of(now);
      for (int j = j0; j < j1; ++j, ++g) {
        const int st = (int)(g & 1);
        if (!__all_sync(0xffffffffu,
                        g < 2 || mbar_wait_long(&bars[kKEmpty + st], ((g >> 1) - 1) & 1))) {
          failed = true;
          break;
        }
        store(smem + LY::kK + st * LY::kTileBytes, kx);
        if (lt < 2)
          meta[(g & 3) * 2 + lt] =
              make_float4(ks, log2f(vs) + 3.0f, __fdiv_rn(0.125f, vs),
                          (lt == 0 ? now[0] : now[1]) >= 0 ? 1.0f : 0.0f);
        fence_proxy_async_smem();
        mbar_arrive(&bars[kKFull + st]);
        load(next, 0, kx);
        scales_of(next);
        if (!__all_sync(0xffffffffu,
                        g < 2 || mbar_wait_long(&bars[kVEmpty + st], ((g >> 1) - 1) & 1))) {
          failed = true;
          break;
        }
        // Positions behind the context hold anything: zeros in their place (a
        // weight of 0 times NaN is NaN). Where the item's rows see different
        // lengths, NaN codes become 0 too, and are listed.
        if ((jb + j + 1) * kTile > min_vis) {
#pragma unroll
          for (int e = 0; e < NC; ++e) {
            const int row = lt / RC + e * (128 / RC), pos = (jb + j) * kTile + row;
            uint32_t bits = 0u;
            if (pos >= len) {
              vx[e] = make_uint4(0u, 0u, 0u, 0u);
            } else if (pos >= min_vis && has_nan_code(vx[e])) {
              uint32_t w[4] = {vx[e].x, vx[e].y, vx[e].z, vx[e].w};
#pragma unroll
              for (int u = 0; u < 16; ++u)
                if (((w[u >> 2] >> (8 * (u & 3))) & 0x7Fu) == 0x7Fu) {
                  bits |= 1u << u;
                  w[u >> 2] &= ~(0xFFu << (8 * (u & 3)));
                }
              vx[e] = make_uint4(w[0], w[1], w[2], w[3]);
              nan_tag[st] = g + 1;
            }
            reinterpret_cast<uint16_t*>(smem + LY::kNanMap +
                                        st * LY::kNanMapBytes)[row * RC + lt % RC] = (uint16_t)bits;
          }
        }
        store(smem + LY::kV + st * LY::kTileBytes, vx);
        fence_proxy_async_smem();
        mbar_arrive(&bars[kVFull + st]);
        load(next, side, vx);
        now[0] = next[0];
        now[1] = next[1];
        pages_of(j + 2, next);
      }
      if (failed) break;
      piece_done();
    }
    if (err_bits && lt == 0 && p.c.err != nullptr) atomicOr(p.c.err, err_bits);
  } else {
    regs_dec<LY::kRegsMma>();
    if (warp == kMmaWarp) {
      // -------------------------------------------------------- MMA issuer
      // (the whole warp; one lane issues)
      constexpr uint32_t idesc_s = make_idesc_f16(128, kTile, 0, 0);
      constexpr uint32_t idesc_o = make_idesc_f16(128, DIM, 0, 1);
      const uint64_t q_desc = make_sw128_desc(sbase + LY::kQ, 16, 1024);
      const uint64_t k_desc = make_sw128_desc(sbase + LY::kK, 16, 1024);
      const uint64_t v_desc = make_sw128_desc(sbase + LY::kV, LY::kBlock, 1024);
      const bool leader = elect_one();
      uint32_t g = 0;                    // tiles of the CTA so far
      uint32_t done[2] = {0u, 0u};       // tiles of each row tile
      uint32_t items[2] = {0u, 0u};      // Q of each row tile
      while (true) {
        const volatile Piece& x = *next_piece();
        if (failed || x.r < 0) break;
        const int nt = x.j1 - x.j0;
        const bool begins = x.j0 == 0;
        const int mts = x.n * p.group - x.row0 > kTile ? 2 : 1;
        piece_done();
        if (nt <= 0) continue;
        auto issue_s = [&](int m, uint32_t t) {
          const uint64_t kd = k_desc + (uint64_t)(((t & 1) * LY::kTileBytes) >> 4);
          if (leader) {
#pragma unroll
            for (int k = 0; k < DIM / 16; ++k) {
              const uint32_t off = (uint32_t)((k >> 2) * LY::kBlock + (k & 3) * 32);
              mma_bf16_ss(tmem + LY::kS + m * kTile, q_desc + ((m * LY::kTileBytes + off) >> 4),
                          kd + (off >> 4), idesc_s, k > 0 ? 1u : 0u);
            }
            mma_commit(&bars[kSFull + m]);
            if (m == mts - 1) mma_commit(&bars[kKEmpty + (t & 1)]);
          }
          __syncwarp();
        };
        // Waits are the warp's: one lane's failure is everyone's.
        auto wait = [&](int bar, uint32_t phase) {
          if (!failed && !__all_sync(0xffffffffu, mbar_wait_long(&bars[bar], phase & 1)))
            failed = true;
        };
        // The first S of the piece, behind the last PV of the piece before.
        wait(kKFull + (g & 1), g >> 1);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (m >= mts) break;
          wait(kQFull + m, items[m]);
          if (!LY::kApart && done[m] != 0) wait(kPvDone + m, done[m] - 1);
          ++items[m];
          if (failed) break;
          tc_fence_after();
          issue_s(m, g);
        }
        for (int j = 0; j < nt && !failed; ++j, ++g) {
          const uint64_t vd = v_desc + (uint64_t)(((g & 1) * LY::kTileBytes) >> 4);
          const bool fresh = j == 0 && begins;
          wait(kVFull + (g & 1), g >> 1);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (m >= mts) break;
            if (LY::kApart && j + 1 < nt) {
              // The next S as soon as this one is read.
              if (m == 0) wait(kKFull + ((g + 1) & 1), (g + 1) >> 1);
              wait(kSFree + m, done[m]);
              if (failed) break;
              tc_fence_after();
              issue_s(m, g + 1);
            }
            wait(kPFull + m, done[m]);
            if (failed) break;
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int k = 0; k < kTile / 16; ++k)
                mma_f16_ts(tmem + LY::kO + m * DIM,
                           tmem + LY::kP + m * LY::kPStep + k * 8,
                           vd + ((k * 16 * 128) >> 4), idesc_o, k > 0 ? 1u : (fresh ? 0u : 1u));
              mma_commit(&bars[kPvDone + m]);
              if (m == mts - 1) mma_commit(&bars[kVEmpty + (g & 1)]);
            }
            __syncwarp();
            ++done[m];
            if (!LY::kApart && j + 1 < nt) {
              // The next S overwrites this P: only once PV has ended.
              if (m == 0) wait(kKFull + ((g + 1) & 1), (g + 1) >> 1);
              wait(kPvDone + m, done[m] - 1);
              if (failed) break;
              tc_fence_after();
              issue_s(m, g + 1);
            }
          }
        }
        if (failed) break;
      }
      if (leader) mma_commit(&bars[kDrain]);
      __syncwarp();
      if (!mbar_wait_long(&bars[kDrain], 0)) failed = true;
    } else if (warp == kMmaWarp + 1) {
      // ----------------------------------------------------- piece lookups
      // (every lane alike; the lanes then ask for the piece's q, which is read when
      // the one before has ended)
      Scheduler sched(p);
      for (uint32_t i = 0;; ++i) {
        const Piece x = sched.next();
        if (i >= 2 && !__all_sync(0xffffffffu, mbar_wait_long(&bars[kPieceEmpty + (i & 1)],
                                                              ((i >> 1) - 1) & 1))) {
          failed = true;
          break;
        }
        if (lane == 0) {
          pieces[i & 1] = x;
          mbar_arrive(&bars[kPieceFull + (i & 1)]);
        }
        if (x.r < 0) break;
        const int last = last_row_of(p, x.row0, x.n);
        for (int rr = x.row0 + lane; rr <= last; rr += 32) {
          const __nv_bfloat16* at = p.q + (x.t0 + rr / p.group) * p.q_stride +
                                    (x.kvh * p.group + rr % p.group) * DIM;
#pragma unroll
          for (int d = 0; d < DIM; d += 64)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at + d));
        }
      }
    }
    __syncwarp();
  }
  if (failed && p.c.err != nullptr) atomicOr(p.c.err, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, LY::kCols);
}

template <int DIM, bool TREE>
cudaError_t launch(const Params& p, int dev, cudaStream_t stream) {
  static PerDeviceOnce once;
  auto kern = kv8_prefill_kernel<DIM, TREE>;
  cudaError_t e = set_max_dynamic_smem(once, dev, kern, Layout<DIM>::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kv8_prefill_plan_kernel<TREE>, dim3(1), dim3(1024), 0, stream, 1u, p);
  if (e != cudaSuccess) return e;
  const int64_t items = p.units * p.c.kv_heads;
  int64_t ctas = kv8_sm_count(dev);
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  if (ctas > items) ctas = items;
  // CTAs wait for the state of the one before: a cooperative launch keeps all of
  // them resident.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(Layout<DIM>::kThreads);
  cfg.dynamicSmemBytes = Layout<DIM>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeCooperative;
  attr.val.cooperative = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

size_t carve(Plan* plan, void* base, int64_t units, int dim) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* x = base ? static_cast<uint8_t*>(base) + at : nullptr;
    at += pad256(bytes);
    return x;
  };
  Plan r;
  r.first = reinterpret_cast<int64_t*>(take((size_t)(units + 1) * 8));
  r.info = reinterpret_cast<UnitInfo*>(take((size_t)units * sizeof(UnitInfo)));
  r.flags = reinterpret_cast<int32_t*>(take(kMaxCtas * 4));
  r.state = take((size_t)kMaxCtas * state_bytes(dim));
  if (plan) *plan = r;
  return at;
}

}  // namespace

int64_t kv8_prefill_units(int64_t tokens, int64_t requests, int group) {
  return tokens * group / kRows + requests;
}

size_t kv8_prefill_workspace_bytes(int64_t tokens, int64_t requests, int heads, int kv_heads,
                                   int dim) {
  if (tokens == 0 || requests == 0) return 0;
  return carve(nullptr, nullptr, kv8_prefill_units(tokens, requests, heads / kv_heads), dim);
}

cudaError_t launch_kv8_prefill(const Kv8AttnArgs& a, cudaStream_t stream) {
  int dev = 0;
  const cudaError_t e = stream_device(stream, &dev);
  if (e != cudaSuccess) return e;
  Params p{};
  p.q = reinterpret_cast<const __nv_bfloat16*>(a.q);
  p.q_stride = a.q_stride;
  p.tokens = a.tokens;
  p.starts = a.starts;
  p.heads = a.heads;
  p.group = a.heads / a.c.kv_heads;
  p.units = kv8_prefill_units(a.tokens, a.c.requests, p.group);
  p.scale_log2 = a.scale * kLog2e;
  p.out = reinterpret_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.c = a.c;
  carve(&p.plan, a.workspace, p.units, a.c.dim);
  return a.c.dim == 128 ? launch<128, false>(p, dev, stream) : launch<64, false>(p, dev, stream);
}

namespace {

// Shape of a tree call: spans of a request, units of a span, rows of a unit.
struct TreeShape {
  int64_t spans, units, slots;
  int row_units, rows;
};
TreeShape tree_shape(int64_t requests, int next_n, int heads, int kv_heads, int64_t bt_stride) {
  const int total = next_n * (heads / kv_heads);
  TreeShape s;
  s.row_units = (total + kRows - 1) / kRows;
  s.rows = total < kRows ? total : kRows;
  s.spans = TreeSpans::most(bt_stride * kPage);
  s.units = requests * s.spans * s.row_units;
  s.slots = requests * kv_heads * s.row_units * s.spans * s.rows;
  return s;
}

}  // namespace

size_t kv8_tree_workspace_bytes(int64_t requests, int next_n, int heads, int kv_heads, int dim,
                                int64_t bt_stride) {
  const TreeShape s = tree_shape(requests, next_n, heads, kv_heads, bt_stride);
  return carve(nullptr, nullptr, s.units, dim) + pad256((size_t)s.slots * dim * 4) +
         pad256((size_t)s.slots * 8) + 256;
}

namespace {

// Joins the spans of a tree's rows, in order. A block has 32 rows of a unit, one a
// lane, and each warp an eighth of the dims. Requests with one span (or none) are
// complete already.
template <int DIM>
__global__ void __launch_bounds__(256) kv8_tree_join_kernel(const JoinArgs p) {
  constexpr int V = DIM / 4 / 8;        // float4s of a thread
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = (p.rows + 31) / 32;
  const int64_t group = blockIdx.x / blocks;                  // (request, kv head, unit)
  const int rr = blockIdx.x % blocks * 32 + lane;
  const int row = (int)(group % p.row_groups) * kRows + rr;   // of the kv head's
  const int64_t rk = group / p.row_groups, r = rk / p.c.kv_heads;
  const int kvh = (int)(rk % p.c.kv_heads);
  pdl_wait();
  pdl_trigger();
  const int64_t most = p.c.bt_stride * kPage, raw = p.c.lens[r];
  const int len = (int)(raw < 0 ? 0 : (raw > most ? most : raw));
  const int span = TreeSpans::of(len);
  const int spans = (len + span - 1) / span;
  if (spans <= 1 || rr >= p.rows || row >= p.next_n * p.group) return;
  const int64_t slot0 = group * p.spans * p.rows;
  const float2* ml = p.part_ml + slot0 + rr;
  const float4* o = reinterpret_cast<const float4*>(p.part_o + slot0 * DIM) +
                    (int64_t)warp * V * p.rows + rr;
  constexpr int S = TreeSpans::kMost;
  float2 x[S];
  float M = -INFINITY;
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (s < spans) x[s] = ml[s * p.rows];
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (s < spans) M = fmaxf(M, x[s].x);
  const float m0 = M == -INFINITY ? 0.0f : M;
  float L = 0.0f;
  float4 acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    if (s >= spans) break;
    const float wt = ex2(x[s].x - m0);
    L = __fmaf_rn(wt, x[s].y, L);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float4 v = o[(s * (DIM / 4) + i) * p.rows];
      acc[i] = make_float4(__fmaf_rn(wt, v.x, acc[i].x), __fmaf_rn(wt, v.y, acc[i].y),
                           __fmaf_rn(wt, v.z, acc[i].z), __fmaf_rn(wt, v.w, acc[i].w));
    }
  }
  if (M == kOnlyLow) L = NAN;
  const float inv = L == 0.0f ? 0.0f : __fdiv_rn(1.0f, L);
  const int64_t w =
      (r * p.next_n + row / p.group) * p.heads + kvh * p.group + row % p.group;
  uint4* out = reinterpret_cast<uint4*>(p.out + w * DIM + warp * V * 4);
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    const __nv_bfloat162 b[4] = {__floats2bfloat162_rn(acc[i].x * inv, acc[i].y * inv),
                                 __floats2bfloat162_rn(acc[i].z * inv, acc[i].w * inv),
                                 __floats2bfloat162_rn(acc[i + 1].x * inv, acc[i + 1].y * inv),
                                 __floats2bfloat162_rn(acc[i + 1].z * inv, acc[i + 1].w * inv)};
    out[i / 2] = *reinterpret_cast<const uint4*>(b);
  }
  if (warp == 0) p.lse[w] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
}

template <int DIM>
cudaError_t launch_tree(const Params& p, int dev, cudaStream_t stream) {
  const cudaError_t e = launch<DIM, true>(p, dev, stream);
  if (e != cudaSuccess || p.spans == 1) return e;   // no table holds a row of two spans
  const JoinArgs a{p.part_o, p.part_ml, p.out,  p.lse,       p.c,    p.next_n,
                   p.heads,  p.group,   p.rows, p.row_units, p.spans};
  const int64_t blocks = p.c.requests * p.c.kv_heads * p.row_units * ((p.rows + 31) / 32);
  return launch_pdl(kv8_tree_join_kernel<DIM>, dim3((unsigned)blocks), dim3(256), 0, stream, 1u, a);
}

}  // namespace

cudaError_t launch_kv8_tree(const Kv8AttnArgs& a, cudaStream_t stream) {
  int dev = 0;
  const cudaError_t e = stream_device(stream, &dev);
  if (e != cudaSuccess) return e;
  const TreeShape s = tree_shape(a.c.requests, a.next_n, a.heads, a.c.kv_heads, a.c.bt_stride);
  Params p{};
  p.q = reinterpret_cast<const __nv_bfloat16*>(a.q);
  p.q_stride = a.q_stride;
  p.tokens = a.tokens;
  p.heads = a.heads;
  p.group = a.heads / a.c.kv_heads;
  p.units = s.units;
  p.scale_log2 = a.scale * kLog2e;
  p.out = reinterpret_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.c = a.c;
  p.next_n = a.next_n;
  p.row_units = s.row_units;
  p.rows = s.rows;
  p.masks = a.masks;
  p.spans = s.spans;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace) + carve(&p.plan, a.workspace, p.units, a.c.dim);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + pad256((size_t)s.slots * a.c.dim * 4));
  return a.c.dim == 128 ? launch_tree<128>(p, dev, stream) : launch_tree<64>(p, dev, stream);
}

}  // namespace dsmla
