// Attention mass over the block-scaled 8-bit cache: how much weight each cached
// position got from new tokens.
//
// Mathematics. With codes K (E4M3), key scale a and a token's lse as attention
// gave it,
//   mass[p] += sum over rows (token, head of the group) that see p of
//              2^(scale * log2e * a * (q . K_p) - lse * log2e).
// S^T = K Q^T, positions on the rows of the product: a TMEM lane is a position,
// so its sum over the query rows stays in one thread (or two, with every other
// step), nothing is reduced across threads, and the order of the additions follows
// from the request alone.
//
// Work goes by tiles of 128 positions of a (request, kv head), their codes brought
// by TMA. Two forms, by the request's number of rows R = tokens * heads of the
// group:
//
// - Few rows (R <= 24): K is multiplied as it lies, on the 8-bit tensor cores,
//   with q as three E4M3 pieces, each a column of its own under the row's power of
//   two: q = 2^-k (q0 + q1 / 32 + q2 / 1024). A bf16 number has 8 significant
//   bits, so this is exact down to 2^-19 of the row's largest |q| and off by up to
//   2^-27 of that below. The pieces are made once per (request, kv head) and
//   serve all its tiles; a tile is then a product of 3 R columns and 128 R
//   exponentials, and up to four of them are an item, so that the walk and the waits
//   are paid once and a thread has two positions to work on. The bound is HBM, dim
//   bytes a position and head.
//
// - More: K becomes bf16 (an E4M3 code has 4 significant bits and an exponent that
//   bf16 holds: exponent and mantissa bits are placed under bf16's, subnormals
//   included, and multiplied by 2^120) and lies in TMEM as the A operand, two tiles
//   for an item; the query rows stream past both in steps of up to 192, by TMA as
//   they lie, and both operands are exact. Each of the two tiles has its eight warps
//   and its buffer of S. The bound is the tensor core (2 dim flops a position and
//   row) and the exponentials beside it.
//
// Sums are fp32: of a step first, then over the steps.
//
// Work split: a persistent grid, each CTA a run of items of equal cost. A
// request's tiles are taken from both ends in turn, since the last ones are seen
// by fewer rows.
//
// Measured: one token of 32 requests with 4096 to 32768 positions, 64 / 8 heads x 128:
// 132 us (684 MB, 5.2 TB/s: 76 % of a plain copy; bf16 products of the same took 319,
// one tile an item 153); 6 tokens of each 322, 24 tokens 372. The last 2048 of 32768
// positions: 838 us, 1270 TFLOP/s, 66 % (the tensor pipe 57 % busy, issue slots 55 %:
// exponentials, and the products of the two tiles take turns with them; of it 20 us since
// rows of lse -inf are looked for behind the wait for S. Looked for before it the chunk
// takes 806 and 48 to 192 rows 5 to 8 % more, dim 64 the other way round: registers
// spill). 12 ragged prompts of dim 64, 28 / 4 heads: 226 us, where exponentials alone
// take 87: a product of dim 64 is half as long, so that issuing and waiting count twice,
// and a quarter of the steps is masked. Not kept, each against the build of its time: S
// in three buffers that both tiles share (chunk 938 us, 883 without), eight warps that sum
// (919, 883), lse read four steps ahead (1560: registers), steps of 128 rows (863, 821).
//
// Per CTA: warps 0-15 convert and sum (enough of them that the exponentials of some
// run while others wait for their product), warp 16 brings K, warp 17 issues the
// products, warp 18 walks the items, lists them for the others and brings Q, warp 19
// lse and the pieces of q.

#include <cuda.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "kv8_common.cuh"

namespace dsmla {

namespace {

constexpr int kTile = 128;                 // positions of a tile
constexpr int kStep = 192;                 // query rows of a step
constexpr int kFewCols = 128;              // columns of an S buffer with few rows
constexpr int kSumWarps = 16;
constexpr int kProducerWarp = 16, kMmaWarp = 17, kQWarp = 18, kLWarp = 19;
constexpr int kThreads = 32 * (kLWarp + 1);   // (96 registers a thread)
constexpr int kMetaSlots = 32;
constexpr int kItems = 32;                 // slots of the list of items
constexpr int kLook = 4;                   // items whose pages are looked up at once
// Items listed ahead of the one whose Q is being brought: K is looked up to 2 kLook
// ahead of the one in work, and waits for the list.
constexpr int kAhead = 3 * kLook;
constexpr int kReaders = kSumWarps + 3;    // warps that read the list
constexpr int kNS = 3;                     // S buffers of few rows (more: one for each place)
constexpr int kNL = 8;                     // slots of lse (more than stages of Q: they are let go
                                           // when a step is summed, Q once its product is done)
// Most rows that are multiplied in pieces. us by pieces / as bf16, 64 / 8 heads x 128, inputs
// not in L2:
//   rows                                       8      16      24      32      40
//   32 requests on 4096 to 32768 positions  148/298 192/300 277/301 294/310 314/337
//   one on 32768                             29/40   34/40   39/40   42/40   46/42
//   32 on 300 to 1000                        36/36   46/33   56/36   68/36   76/36
// (Dim 64 is much the same: 120/275 and 31/33 with 8 rows, 282/300 and 54/36 with 24.) Beyond
// 24 a long batch has 2 to 7 % of it, and a short one pays twice.
constexpr int kFewRows = 24;
// Word of an lse slot (behind the factors, of which few rows need kFewRows) that tells
// whether a row of the step is left out: the paths without masks are not for it then.
constexpr int kLeftOut = 3 * kStep - 1;
constexpr int kErrPage = DS_DEVERR_PAGE, kErrTimeout = DS_DEVERR_TIMEOUT;

template <int DIM>
struct Layout {
  static constexpr int kKBytes = kTile * DIM;
  static constexpr int kQBytes = kStep * DIM * 2;
  static constexpr int kNK = DIM == 128 ? 6 : 8;    // stages
  static constexpr int kNQ = DIM == 128 ? 2 : 4;
  static constexpr int kK = 0;
  static constexpr int kQ = kK + kNK * kKBytes;
  static constexpr int kLse = kQ + kNQ * kQBytes;   // per slot: lse, visible, factors; kStep each
  static constexpr int kBars = kLse + kNL * kStep * 12;
  static constexpr int kMeta = kBars + 136 * 8;               // kMetaSlots x float4
  static constexpr int kList = kMeta + kMetaSlots * 16;       // kItems x Item
  static constexpr int kOther = kList + kItems * 64;          // 4 x kTile sums
  static constexpr int kMisc = kOther + 4 * kTile * 4;        // tmem slot, start of work, scan
  static constexpr int kEnd = kMisc + 32 + 8 * (kThreads / 32);
  static constexpr int kSmem = kEnd + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  // TMEM columns: the S buffers, then K of two tiles.
  static constexpr int kA = 2 * kStep;
  static_assert(kNS * kFewCols <= kA, "the buffers of few rows");
  static constexpr int kACols = DIM / 2;
  static constexpr uint32_t kCols = 512;
  static_assert(kA + 2 * kACols <= 512, "TMEM columns");
};

enum Bar {
  kKFull = 0,       // <= 8: K landed
  kKEmpty = 8,      // K converted, or its product done
  kQFull = 16,      // <= 8: Q landed, and its lse is written
  kQEmpty = 24,     // product done
  kLFull = 32,      // kNL: lse written
  kLEmpty = 40,     // lse read
  kAFull = 48,      // 2: A of a tile written
  kSFull = 50,      // kNS: few rows: S of an item ready
  kSFree = 53,      // kNS: S read
  kCFull = 56,      // 2: more rows: S of a set ready
  kCFree = 58,      // 2: read
  kXFull = 60,      // 4: the other half's sums of a tile written, two slots each
  kXFree = 64,      // 4: read
  kDrain = 68,
  kIFull = 69,      // kItems: an item is in the list
  kIEmpty = 101,    // every reader is done with it
  kNumBars = 133
};

struct Params {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const float* lse;
  const int32_t* starts;
  int64_t tokens;
  int heads, group;
  // A step: `tokens` tokens of `heads` heads each; of `chunks` steps of a token
  // where its heads do not fit one.
  int step_tokens, step_heads, chunks;
  float scale_log2;
  float* mass;
  int64_t mass_stride;
  Kv8Cache c;
};

// One request, and the CTA's place in it.
struct Walk {
  int64_t at, end;       // cost before the present item; end of the CTA's share
  int r;                 // request
  int item_r, item_kvh;  // of the last item loaded
  int raw, len, n;       // lens[r], clamped, new tokens
  int64_t t0;            // first token
  int tiles;
  bool few;              // multiplied in pieces
  // Units: a tile with few rows, else two (the last may be one). An item is a unit,
  // or with few rows up to `batch` of them.
  int units, cost;       // of a head; cost of one
  int batch;
  int i, items;          // first unit of the present item; units of the request
  int j;                 // its number among its head's
  int kvh, tile;         // of the present item: its first tile
  int nb;                // its tiles
  int first;             // first token that sees them (few: 0)
  int steps;
  bool same;             // one step, of the rows that the item before it had in its one step
};

__device__ __forceinline__ int64_t start_of(const Params& p, int64_t r) {
  const int64_t s = p.starts[r];
  return s < 0 ? 0 : (s > p.tokens ? p.tokens : s);
}

// (len, n, first token) of a request; n = 0 where there is nothing to do.
__device__ __forceinline__ void load_request(const Params& p, int64_t r, Walk& w) {
  w.raw = p.c.lens[r];
  const int64_t most = p.c.bt_stride * kPage;
  w.len = w.raw < 0 ? 0 : (w.raw > most ? (int)most : w.raw);
  w.t0 = start_of(p, r);
  const int64_t n = start_of(p, r + 1) - w.t0;
  w.n = n < 0 || w.len == 0 ? 0 : (int)n;
  w.tiles = w.n > 0 ? (w.len + kTile - 1) / kTile : 0;
  const int rows = w.n * p.group;   // (below 2^31 - 256)
  // (The pieces stay clear of the rows of a stage that no step writes.)
  w.few = rows <= kFewRows && 3 * ((rows + 7) & ~7) <= p.step_tokens * p.step_heads;
  // As many tiles as S columns of one buffer: products of 32 columns with up to 8
  // rows, 48 with 16.
  w.batch = !w.few || rows > 16 ? 1 : (rows > 8 ? 2 : 4);
  w.units = w.few ? w.tiles : (w.tiles + 1) / 2;
  w.items = w.units * p.c.kv_heads;
  w.cost = w.few ? 1 : 2 + 2 * ((w.n + p.step_tokens - 1) / p.step_tokens) * p.chunks;
}

// A head's units from both ends in turn: the first tile of the j-th.
__device__ __forceinline__ int tile_of(const Walk& w, int j) {
  const int u = j & 1 ? w.units - 1 - (j >> 1) : j >> 1;
  return w.few ? u : 2 * u;
}

__device__ __forceinline__ void load_item(const Params& p, Walk& w) {
  w.tile = tile_of(w, w.j);   // (the first of a batch)
  const bool one = w.steps == 1 && w.item_r == w.r && w.item_kvh == w.kvh;
  if (w.few) {
    w.same = one;
    w.first = 0;
    w.steps = 1;
    const int left = w.units - w.j < w.batch ? w.units - w.j : w.batch;
    w.nb = w.end - w.at < left ? (int)(w.end - w.at) : left;   // (cost 1 each)
  } else {
    // Token i sees position p if p <= base + i.
    const int before = w.first;
    const int64_t first = (int64_t)w.tile * kTile - ((int64_t)w.raw - w.n);
    w.first = first > 0 ? (int)first : 0;
    w.steps = (w.n - w.first + p.step_tokens - 1) / p.step_tokens * p.chunks;
    w.same = one && w.steps == 1 && before == w.first;
    w.nb = w.tiles - w.tile < 2 ? w.tiles - w.tile : 2;
  }
  w.item_r = w.r;
  w.item_kvh = w.kvh;
}

// What the warps are told of an item.
struct __align__(16) Item {
  int nb;                // tiles; 0 ends the list
  int steps;
  int n, first;          // new tokens; the first that sees the tiles
  int tile[4];
  int raw, len;          // lens[r], and clamped
  int r, kvh;
  int t0;                // the request's first token
  int few, same, single; // in pieces; Q as it is; in pieces and one tile an item
};
static_assert(sizeof(Item) == 64, "an item's slot");

// Step s of an item: its first token, its chunk of heads and its rows.
struct Step {
  int token, head, rows;
};
__device__ __forceinline__ Step step_of(const Params& p, int n, int first, int s) {
  Step x;
  if (p.chunks == 1) {
    x.token = first + s * p.step_tokens;
    x.head = 0;
    const int left = n - x.token;
    x.rows = (left < p.step_tokens ? left : p.step_tokens) * p.step_heads;
  } else {
    x.token = first + s / p.chunks;
    x.head = s % p.chunks * kStep;
    const int left = p.group - x.head;
    x.rows = left < kStep ? left : kStep;
  }
  return x;
}

// The next item from w.i on, in later requests where need be. (Whole warps call it
// with one state: behind a request without tokens the lanes look at 32 at a time,
// since the other warps wait for the list, and a batch may be empty but for a few.)
__device__ __forceinline__ bool walk_settle(const Params& p, Walk& w) {
  while (w.i >= w.items) {
    if (++w.r >= p.c.requests) return false;
    load_request(p, w.r, w);
    w.i = w.j = w.kvh = 0;
    if (w.items > 0) break;
    const int64_t r = (int64_t)w.r + 1 + (threadIdx.x & 31);
    const uint32_t in = __ballot_sync(
        0xffffffffu, r < p.c.requests && p.c.lens[r] > 0 && start_of(p, r + 1) > start_of(p, r));
    w.r += in ? __ffs((int)in) - 1 : 32;
  }
  if (w.at >= w.end) return false;
  load_item(p, w);
  return true;
}
// Moves on by a number of units: those of the present item, or more.
__device__ __forceinline__ int item_units(const Walk& w) { return w.few ? w.nb : 1; }
__device__ __forceinline__ bool walk_next(const Params& p, Walk& w, int units) {
  w.at += (int64_t)units * w.cost;
  w.i += units;
  w.j += units;
  while (w.j >= w.units && w.i < w.items) {
    w.j -= w.units;
    ++w.kvh;
  }
  if (w.at >= w.end) return false;
  return walk_settle(p, w);
}

// Two codes (bytes 0 and 1, or 2 and 3, of w) as a bf16 pair: sign, exponent
// and mantissa bits in place, times 2^120 (exact, subnormal codes included). The
// NaN codes become +-480.
template <int HI>
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t w) {
  const uint32_t x = __byte_perm(w, 0u, HI ? 0x3424 : 0x1404);
  const uint32_t y = ((x >> 4) & 0x07F007F0u) | (x & 0x80008000u);
  const uint32_t up = 0x7B807B80u;
  const __nv_bfloat162 z = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&y),
                                   *reinterpret_cast<const __nv_bfloat162*>(&up));
  return *reinterpret_cast<const uint32_t*>(&z);
}
// Nonzero in a byte's highest bit where w's byte is a NaN code.
__device__ __forceinline__ uint32_t nan_bits(uint32_t w) {
  return (w & 0x7F7F7F7Fu) + 0x01010101u;
}

// The power of two that brings a row's largest |q|, a, to [128, 256); it stays a
// normal float.
__device__ __forceinline__ int q_exponent(float a) {
  const int k = a > 0.0f ? 7 - ((int)(__float_as_uint(a) >> 23) - 127) : 0;
  return k > 120 ? 120 : (k < -120 ? -120 : k);
}
__device__ __forceinline__ float pow2f(int k) {
  return __uint_as_float((uint32_t)(k + 127) << 23);
}
// Two values as E4M3, and 32 times what that leaves of them.
__device__ __forceinline__ uint16_t piece(float& u0, float& u1) {
  const __nv_fp8x2_storage_t b =
      __nv_cvt_float2_to_fp8x2(make_float2(u0, u1), __NV_SATFINITE, __NV_E4M3);
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(b, __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  u0 = (u0 - f.x) * 32.0f;
  u1 = (u1 - f.y) * 32.0f;
  return b;
}

template <int DIM>
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
  if constexpr (DIM == 128)
    return make_sw128_desc(addr, 16, 1024);
  else
    return make_sw64_desc(addr, 16, 512);
}

// Whether one of tokens from .. n - 1 has a head that is not left out; lse is the group's
// of token 0. (The last token first: it sees all of the others' positions.)
__device__ __noinline__ bool weighs(const float* lse, int heads, int group, int from, int n) {
  for (int i = n - 1; i >= 0 && i >= from; --i)
    for (int h = 0; h < group; ++h)
      if (lse[(int64_t)i * heads + h] != -INFINITY) return true;
  return false;
}

template <int DIM>
__global__ void __launch_bounds__(kThreads, 1) kv8_mass_kernel(
    const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap q_map,
    const Params p) {
  using LY = Layout<DIM>;
  constexpr int NK = LY::kNK, NQ = LY::kNQ;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + LY::kBars);
  float4* meta = reinterpret_cast<float4*>(smem + LY::kMeta);
  Item* list = reinterpret_cast<Item*>(smem + LY::kList);
  float* other = reinterpret_cast<float*>(smem + LY::kOther);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + LY::kMisc);
  int64_t* start_s = reinterpret_cast<int64_t*>(smem + LY::kMisc + 8);   // request, cost before it
  int64_t* scan_s = reinterpret_cast<int64_t*>(smem + LY::kMisc + 32);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t n = 1;
      if (i >= kAFull && i < kAFull + 2) n = 2 * kTile;
      if (i >= kXFull && i < kXFree + 4) n = kTile;
      if (i >= kIEmpty && i < kIEmpty + kItems) n = kReaders;
      if (i >= kLFull && i < kLFull + kNL) n = 32;
      if (i >= kQFull && i < kQFull + NQ) n = 2;
      if (i >= kLEmpty && i < kLEmpty + kNL) n = kSumWarps;
      if (i >= kSFree && i < kSFree + kNS) n = kSumWarps;
      if (i >= kCFree && i < kCFree + 2) n = kSumWarps / 2;   // of one place
      mbar_init(&bars[i], n);
    }
    mbar_fence_init();
    start_s[0] = -1;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, LY::kCols);
    tmem_relinquish();
  }
  // Rows that no step writes stay 0, so that their scores are.
  const int capacity = p.step_tokens * p.step_heads;
  for (int i = tid; i < NQ * (DIM / 64) * (kStep - capacity) * 8; i += kThreads) {
    const int block = i / ((kStep - capacity) * 8), at = i % ((kStep - capacity) * 8);
    *reinterpret_cast<uint4*>(smem + LY::kQ + (block * kStep + capacity) * 128 + at * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's share: thread t sums the cost of a run of requests, and a
  // scan over the block finds the request that holds the share's start.
  const int64_t per = (p.c.requests + kThreads - 1) / kThreads;
  Walk w;
  int64_t sum = 0;
  for (int64_t r = tid * per; r < p.c.requests && r < (tid + 1) * per; ++r) {
    load_request(p, r, w);
    sum += (int64_t)w.items * w.cost;
  }
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) scan_s[warp] = inc;
  __syncthreads();
  int64_t total = 0, before = inc - sum;
#pragma unroll
  for (int v = 0; v < kThreads / 32; ++v) {
    if (v < warp) before += scan_s[v];
    total += scan_s[v];
  }
  const int64_t lo = (int64_t)((double)total * blockIdx.x / gridDim.x);
  const int64_t hi = blockIdx.x + 1 == gridDim.x
                         ? total
                         : (int64_t)((double)total * (blockIdx.x + 1) / gridDim.x);
  if (lo < hi && lo >= before && lo < before + sum) {
    int64_t base = before;
    for (int64_t r = tid * per; r < p.c.requests; ++r) {
      load_request(p, r, w);
      const int64_t n = (int64_t)w.items * w.cost;
      if (lo < base + n) {
        start_s[0] = r;
        start_s[1] = base;
        break;
      }
      base += n;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool some = start_s[0] >= 0;
  w.end = hi;
  if (some) {
    // The first item that begins in the share.
    w.r = (int)start_s[0];
    load_request(p, w.r, w);
    w.steps = 0;           // no item before the first
    w.i = (int)((lo - start_s[1] + w.cost - 1) / w.cost);
    w.at = start_s[1] + (int64_t)w.i * w.cost;
    w.kvh = w.i / w.units;
    w.j = w.i % w.units;
    some = walk_settle(p, w);
  }

  bool failed = false;
  // The number-th item of the list, for a reading warp as a whole; nb is 0 behind
  // the last (and if a wait gave up).
  auto take = [&](uint32_t number) {
    const uint32_t slot = number % kItems;
    Item x;
    x.nb = 0;
    if (__all_sync(0xffffffffu, mbar_wait_long(&bars[kIFull + slot], (number / kItems) & 1u))) {
      x = list[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kIEmpty + slot]);
    } else {
      failed = true;
    }
    return x;
  };
  if (warp == kProducerWarp) {
    // ---------------------------------------------------------- K producer
    const int none = (int)(p.c.num_pages * 2 * p.c.kv_heads * kPage);   // a row past the pool: zeros
    int err_bits = 0;
    uint32_t g = 0, issued = 0, looked = 0;
    // Lane 8 e + i looks up the i-th page of the e-th of kLook items; the next ones'
    // while these are brought.
    struct Batch {
      int y;
      float ks;
      int places;            // page places of the lane's item; 0 behind the last
    };
    bool ok = true, more = true;
    auto look = [&] {
      Batch b;
      b.y = none;
      b.ks = 0.0f;
      b.places = 0;
      int tile = 0, r = 0, kvh = 0, len = 0;
#pragma unroll 1
      for (int e = 0; e < kLook && more && ok; ++e, ++looked) {
        const uint32_t slot = looked % kItems;
        ok = __all_sync(0xffffffffu, mbar_wait_long(&bars[kIFull + slot], (looked / kItems) & 1u));
        if (!ok) break;
        const Item& x = list[slot];
        more = x.nb > 0;
        if (lane >> 3 == e) {
          b.places = 2 * x.nb;
          tile = x.tile[(lane >> 1) & 3];
          r = x.r;
          kvh = x.kvh;
          len = x.len;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kIEmpty + slot]);
      }
      const int block = 2 * tile + (lane & 1);
      if ((lane & 7) < b.places && (int64_t)block * kPage < len) {
        const int64_t page = p.c.block_table[(int64_t)r * p.c.bt_stride + block];
        if (page >= 0 && page < p.c.num_pages) {
          const int64_t part = page * 2 * p.c.kv_heads + kvh;
          b.y = (int)(part * kPage);
          b.ks = p.c.scales[part] * p.scale_log2;
        } else {
          err_bits |= kErrPage;
        }
      }
      return b;
    };
    Batch next = look();
    while (ok && __any_sync(0xffffffffu, next.places > 0)) {
      const Batch now = next;
      next = look();
      for (int e = 0; e < 32 && ok; e += 2) {
        if ((e & 7) >= __shfl_sync(0xffffffffu, now.places, e)) continue;
        const int y0 = __shfl_sync(0xffffffffu, now.y, e);
        const int y1 = __shfl_sync(0xffffffffu, now.y, e + 1);
        const float k0 = __shfl_sync(0xffffffffu, now.ks, e);
        const float k1 = __shfl_sync(0xffffffffu, now.ks, e + 1);
        if (lane == 0) {
          const int st = (int)(g % NK);
          if (g >= NK) ok = mbar_wait_long(&bars[kKEmpty + st], (uint32_t)((g / NK - 1) & 1));
          if (ok) {
            meta[g & (kMetaSlots - 1)] =
                make_float4(k0, y0 == none ? 0.0f : 1.0f, k1, y1 == none ? 0.0f : 1.0f);
            mbar_arrive_expect_tx(&bars[kKFull + st], LY::kKBytes);
            const uint32_t dst = sbase + LY::kK + st * LY::kKBytes;
            tma_load_box(dst, &map, 0, y0, &bars[kKFull + st]);
            tma_load_box(dst + kPage * DIM, &map, 0, y1, &bars[kKFull + st]);
            issued = g + 1;
          }
        }
        ++g;
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    failed = !ok;
    if (lane == 0)   // every copy has landed before the CTA can exit
      for (uint32_t i = issued > NK ? issued - NK : 0; i < issued; ++i)
        if (!mbar_wait_long(&bars[kKFull + i % NK], (uint32_t)((i / NK) & 1))) failed = true;
    if (err_bits && p.c.err != nullptr) atomicOr(p.c.err, err_bits);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer
    const uint64_t q_desc = make_sw128_desc(sbase + LY::kQ, 16, 1024);
    const uint64_t q8_desc = tile_desc<DIM>(sbase + LY::kQ);
    const uint64_t k_desc = tile_desc<DIM>(sbase + LY::kK);
    const bool leader = elect_one();
    // The loop runs on values from one lane (a shuffle): the compiler sees that they
    // are uniform then, keeps them and the descriptors in uniform registers, and
    // the warp gets to the next product in a third of a product's time instead of two
    // of them, which was the bound.
    auto uni = [](auto x) { return __shfl_sync(0xffffffffu, x, 0); };
    const uint32_t t_d = uni(tmem), bar0 = uni(smem_u32(bars));
    // A ring's place and phase.
    struct Ring {
      uint32_t at = 0, phase = 0;
    };
    auto next = [](Ring& r, uint32_t n) {
      if (++r.at == n) {
        r.at = 0;
        r.phase ^= 1u;
      }
    };
    auto wait = [&](int bar, uint32_t at, uint32_t phase) {
      return mbar_wait_at(bar0 + (uint32_t)(bar + at) * 8u, phase);
    };
    auto commit = [&](int bar, uint32_t at) { mma_commit_at(bar0 + (uint32_t)(bar + at) * 8u); };
    // An item of one step may use the load of Q of the one before it (`held`), which
    // is let go when the next comes. `phases`: bit u is that of place u's tiles.
    // (A buffer's first use waits for nothing: the phase before the first is over.)
    Ring tile, s_free, load;
    uint32_t phases = 0, held_at = 0, c_free[2] = {1u, 1u};
    s_free.phase = 1u;
    bool held = false, was_few = false;
    for (uint32_t item = 0;; ++item) {
      const Item x = take(item);
      const int nb = uni(x.nb);
      if (nb == 0) break;
      const int steps = uni(x.steps), few = uni(x.few), same = uni(x.same);
      const int rows = uni(x.n * p.group);
      bool ok = true;
      if (held && !same) {
        if (leader) commit(kQEmpty, held_at);
        __syncwarp();
      }
      if (few != (int)was_few) {
        // The two forms share the buffers: all of the other one are read first.
        was_few = few;
        if (few)
          ok = wait(kCFree, 0, c_free[0]) && wait(kCFree, 1, c_free[1]);
        else
          for (uint32_t i = 0; i < kNS; ++i)
            ok = wait(kSFree, i, i < s_free.at ? s_free.phase ^ 1u : s_free.phase) && ok;
      }
      if (few) {
        // One buffer of S for all tiles of the item.
        const int n = (3 * ((rows + 7) & ~7) + 15) & ~15;
        const uint32_t idesc = make_idesc_e4m3(kTile, n, 0, 0);
        if (!same) {
          ok = wait(kQFull, load.at, load.phase) && ok;
          held_at = load.at;
          next(load, NQ);
        }
        ok = wait(kSFree, s_free.at, s_free.phase) && ok;
        const uint64_t b = q8_desc + (uint64_t)(held_at * (LY::kQBytes >> 4));
        for (int u = 0; u < nb; ++u) {
          ok = wait(kKFull, tile.at, tile.phase) && ok;
          tc_fence_after();
          if (leader) {
            const uint64_t a = k_desc + (uint64_t)(tile.at * (LY::kKBytes >> 4));
#pragma unroll
            for (int k = 0; k < DIM / 32; ++k)
              mma_f8_ss(t_d + s_free.at * kFewCols + u * n, a + ((k * 32) >> 4), b + ((k * 32) >> 4),
                        idesc, k > 0 ? 1u : 0u);
            commit(kKEmpty, tile.at);
          }
          __syncwarp();
          next(tile, NK);
        }
        if (leader) commit(kSFull, s_free.at);
        __syncwarp();
        next(s_free, kNS);
      } else {
        for (int s = 0; s < steps; ++s) {
          if (!same) {
            ok = wait(kQFull, load.at, load.phase) && ok;
            held_at = load.at;
            next(load, NQ);
          }
          const int n = s + 1 < steps && p.chunks == 1 ? (capacity + 15) & ~15
                                                       : uni((step_of(p, x.n, x.first, s).rows + 15) & ~15);
          const uint32_t idesc = make_idesc_bf16(kTile, n, 0, 0);
          const uint64_t b = q_desc + (uint64_t)(held_at * (LY::kQBytes >> 4));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (u >= nb) break;
            ok = wait(kCFree, u, c_free[u]) && ok;
            c_free[u] ^= 1u;
            if (s == 0) {
              // K of the tile is in TMEM: its stage is free.
              ok = wait(kAFull, u, (phases >> u) & 1u) && ok;
              if (lane == 0) mbar_arrive(&bars[kKEmpty + tile.at]);
              phases ^= 1u << u;
              next(tile, NK);
            }
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int k = 0; k < DIM / 16; ++k)
                mma_f16_ts(t_d + u * kStep, t_d + LY::kA + u * LY::kACols + 8 * k,
                           b + (((k >> 2) * (kStep * 128) + (k & 3) * 32) >> 4), idesc,
                           k > 0 ? 1u : 0u);
              commit(kCFull, u);
            }
            __syncwarp();
          }
          if (leader && steps > 1) commit(kQEmpty, held_at);
          __syncwarp();
          if (!__all_sync(0xffffffffu, ok)) break;
        }
      }
      if (!__all_sync(0xffffffffu, ok)) {
        failed = true;
        break;
      }
      held = steps == 1;
    }
    if (leader) mma_commit(&bars[kDrain]);
    __syncwarp();
    if (!mbar_wait_long(&bars[kDrain], 0)) failed = true;
    __syncwarp();
  } else if (warp == kQWarp) {
    // ------------------------------------------------------------------ Q
    const uint32_t bytes = (uint32_t)(capacity * DIM * 2);
    uint32_t ql = 0, listed = 0;
    bool ended = false;
    // Adds an item to the list, or its end.
    auto list_one = [&] {
      const uint32_t slot = listed % kItems;
      if (!__all_sync(0xffffffffu, listed < kItems ||
                                       mbar_wait_long(&bars[kIEmpty + slot],
                                                      (listed / kItems - 1) & 1u))) {
        failed = true;
        return;
      }
      if (lane == 0) {
        Item& x = list[slot];
        x.nb = some ? w.nb : 0;
        if (some) {
          x.steps = w.steps;
          x.n = w.n;
          x.first = w.first;
          x.raw = w.raw;
          x.len = w.len;
          x.r = w.r;
          x.kvh = w.kvh;
          x.t0 = (int)w.t0;
          x.few = w.few;
          x.same = w.same;
          x.single = w.few && w.batch == 1;
          x.tile[0] = w.tile;
          for (int u = 1; u < w.nb; ++u) x.tile[u] = w.few ? tile_of(w, w.j + u) : w.tile + u;
        } else {
          x.few = x.same = x.single = 0;
        }
        mbar_arrive(&bars[kIFull + slot]);
      }
      __syncwarp();
      ++listed;
      ended = !some;
      if (some) some = walk_next(p, w, item_units(w));
    };
    for (uint32_t item = 0; !failed; ++item) {
      while (!ended && !failed && listed <= item + kAhead) list_one();
      if (failed) break;
      const Item x = list[item % kItems];   // (its own: nobody else writes)
      if (x.nb == 0) break;
      if (x.same) continue;
      for (int s = 0; s < x.steps; ++s, ++ql) {
        const uint32_t st = ql % NQ;
        if (!__all_sync(0xffffffffu,
                        ql < NQ || mbar_wait_long(&bars[kQEmpty + st], (ql / NQ - 1) & 1u))) {
          failed = true;
          break;
        }
        if (lane == 0) {
          if (x.few) {
            mbar_arrive(&bars[kQFull + st]);   // (the pieces come with the lse)
          } else {
            const Step y = step_of(p, x.n, x.first, s);
            mbar_arrive_expect_tx(&bars[kQFull + st], bytes);
#pragma unroll
            for (int b = 0; b < DIM / 64; ++b)
              tma_load_box3(sbase + LY::kQ + st * LY::kQBytes + b * (kStep * 128), &q_map, 64 * b,
                            x.kvh * p.group + y.head, x.t0 + y.token, &bars[kQFull + st]);
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0)   // every copy has landed before the CTA can exit
      for (uint32_t i = ql > NQ ? ql - NQ : 0; i < ql; ++i)
        if (!mbar_wait_long(&bars[kQFull + i % NQ], (i / NQ) & 1u)) failed = true;
    __syncwarp();
  } else if (warp == kLWarp) {
    // --------------------------------------------- lse, and pieces of few rows
    constexpr int N = kStep / 32;              // rows of a lane: lane, lane + 32, ...
    constexpr int D = 2;                       // steps whose lse is read at once
    int t_token[N], t_head[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      t_token[i] = (lane + 32 * i) / p.step_heads;
      t_head[i] = (lane + 32 * i) % p.step_heads;
    }
    uint32_t ql = 0;
    for (uint32_t item = 0; !failed; ++item) {
      const Item w = take(item);
      if (w.nb == 0) break;
      if (w.same) continue;
      const int seen = w.raw - w.n + 1;        // by token 0
      const float* lse0 = p.lse + (int64_t)w.t0 * p.heads + w.kvh * p.group;
      // A row that there is not sees nothing, nor does one of lse -inf: its q may hold
      // anything, and infinity or NaN less infinity is NaN.
      bool out = false;      // some row of this lane's is left out
      auto put = [&](uint32_t slot, int i, bool in, int token, float l) {
        float* ls = reinterpret_cast<float*>(smem + LY::kLse + slot * (kStep * 12)) + lane + 32 * i;
        out |= in && l == -INFINITY;
        in &= l != -INFINITY;
        ls[0] = in ? -l * kLog2e : -INFINITY;
        reinterpret_cast<int*>(ls)[kStep] = in ? seen + token : INT_MIN;
      };
      // (Its arrival counts for Q's stage too, which has to be free for that.)
      auto wait_slot = [&] {
        const bool ok = (ql < NQ || mbar_wait_long(&bars[kQEmpty + ql % NQ], (ql / NQ - 1) & 1u)) &&
                        (ql < kNL || mbar_wait_long(&bars[kLEmpty + ql % kNL], (ql / kNL - 1) & 1u));
        return __all_sync(0xffffffffu, ok);
      };
      auto arrive = [&] {
        out = __any_sync(0xffffffffu, out);
        if (lane == 0)
          reinterpret_cast<int*>(smem + LY::kLse + ql % kNL * (kStep * 12))[kLeftOut] = out;
        out = false;
        mbar_arrive(&bars[kLFull + ql % kNL]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kQFull + ql % NQ]);
        ++ql;
      };
      if (w.few) {
        const uint32_t st = ql % NQ, sl = ql % kNL;
        const int rows = w.n * p.group, r8 = (rows + 7) & ~7;
        if (!wait_slot()) {
          failed = true;
          break;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int row = lane + 32 * i, token = row / p.group;
          const bool in = row < rows;
          put(sl, i, in, token, in ? lse0[(int64_t)token * p.heads + row % p.group] : 0.0f);
        }
        // (What lies behind the rows is anything: columns of the product that nobody
        // reads.)
        constexpr int E = DIM / 32;
        uint8_t* q8 = smem + LY::kQ + st * LY::kQBytes;
        float* factor = reinterpret_cast<float*>(smem + LY::kLse + sl * (kStep * 12)) + 2 * kStep;
        const __nv_bfloat16* q0 = p.q + (int64_t)w.t0 * p.q_stride + (int64_t)w.kvh * p.group * DIM + lane * E;
        for (int r0 = 0; r0 < rows; r0 += 4) {
          float x[4][E];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = r0 + u < rows ? r0 + u : rows - 1;
            const __nv_bfloat16* src = q0 + (r / p.group) * p.q_stride + (r % p.group) * DIM;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              const uint32_t v = reinterpret_cast<const uint32_t*>(src)[e / 2];
              x[u][e] = __uint_as_float(v << 16);
              x[u][e + 1] = __uint_as_float(v & 0xFFFF0000u);
            }
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = r0 + u;
            float a = 0.0f;
            bool nan = false;
#pragma unroll
            for (int e = 0; e < E; ++e) {
              a = fmaxf(a, fabsf(x[u][e]));
              nan |= x[u][e] != x[u][e];
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            nan = __any_sync(0xffffffffu, nan) || a == INFINITY;
            if (r >= rows) continue;
            const int k = q_exponent(a);
            const float up = pow2f(k);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              float u0 = x[u][e] * up, u1 = x[u][e + 1] * up;
#pragma unroll
              for (int z = 0; z < 3; ++z)
                *reinterpret_cast<uint16_t*>(q8 + swz<DIM>(z * r8 + r, lane * E + e)) =
                    piece(u0, u1);
            }
            if (lane == 0) factor[r] = nan ? NAN : pow2f(-k);
          }
        }
        fence_proxy_async_smem();
        arrive();
        continue;
      }
      for (int s0 = 0; s0 < w.steps && !failed; s0 += D) {
        float l[D][N];
#pragma unroll
        for (int d = 0; d < D; ++d) {
          const Step x = step_of(p, w.n, w.first, s0 + d);
#pragma unroll
          for (int i = 0; i < N; ++i)
            l[d][i] = s0 + d < w.steps && lane + 32 * i < x.rows
                          ? lse0[(int64_t)(x.token + t_token[i]) * p.heads + x.head + t_head[i]]
                          : 0.0f;
        }
        for (int d = 0; d < D && s0 + d < w.steps; ++d) {
          if (!wait_slot()) {
            failed = true;
            break;
          }
          const Step x = step_of(p, w.n, w.first, s0 + d);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            float v = l[0][i];
#pragma unroll
            for (int e = 1; e < D; ++e)
              if (d == e) v = l[e][i];
            put(ql % kNL, i, lane + 32 * i < x.rows, x.token + t_token[i], v);
          }
          arrive();
        }
      }
    }
  } else {
    // --------------------------------------------------- convert and sum
    // Four sets of a warp for each 32 positions. Few rows: a set has a tile of the
    // item. More: sets 0 and 2 have the first tile, 1 and 3 the second, each half of
    // the dims to convert and half of a step's columns to sum.
    const int quad = warp & 3, set = warp >> 2, place = set & 1, half = set >> 1;
    const int tok = quad * 32 + lane;          // position of the tile (TMEM lane)
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    // Items, tiles, S buffers and loads of Q so far (as the issuer counts), and items
    // of more rows that had a tile for this place.
    uint32_t item = 0, tile = 0, g = 0, buf = 0, ql = 0, c_phase = 0, summed = 0;
    const uint32_t c_full = smem_u32(&bars[kCFull + place]);
    bool held = false;
    struct Keys {
      float scale;
      bool there, nan;     // the page is; a NaN among this thread's codes
    };
    auto read_meta = [&](uint32_t it) {
      const float4 m = meta[it & (kMetaSlots - 1)];
      return Keys{tok < kPage ? m.x : m.z, (tok < kPage ? m.y : m.w) != 0.0f, false};
    };
    // K of tile number `it` to bf16, this thread's half of the dims, into its place.
    auto convert = [&](uint32_t it, Keys* keys) {
      const int st = (int)(it % NK);
      if (!__all_sync(0xffffffffu, mbar_wait_long(&bars[kKFull + st], (it / NK) & 1u))) return false;
      *keys = read_meta(it);
      const uint8_t* src = smem + LY::kK + st * LY::kKBytes;
      uint32_t bad = 0;
      const uint32_t t_a = tmem + lane_base + LY::kA + place * LY::kACols + half * (DIM / 4);
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < DIM / 64; ++c) {
        uint32_t v[16];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint4 x = *reinterpret_cast<const uint4*>(
              src + swz<DIM>(tok, half * (DIM / 2) + c * 32 + e * 16));
          const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[8 * e + 2 * i] = codes_to_bf16<0>(y[i]);
            v[8 * e + 2 * i + 1] = codes_to_bf16<1>(y[i]);
            bad |= nan_bits(y[i]);
          }
        }
        tmem_st16u(t_a + 16 * c, v);
      }
      keys->nan = (bad & 0x80808080u) != 0u;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars[kAFull + place]);
      return true;
    };
    // The tile of an item whose mass this thread adds to, or -1. (Where few rows have
    // one tile an item, the sets take the items in turn.)
    auto mine = [&](const Item& v, uint32_t it) {
      if (v.single) return (int)(it & 3) == set ? 0 : -1;
      return set < v.nb && (v.few || half == 0) ? set : -1;
    };
    // What the mass held before is read an item ahead.
    float* row = nullptr;      // this thread's position of the next item's head's tile 0
    auto held_mass = [&](const Item& v, uint32_t it) {
      if (!v.same)
        row = p.mass + ((int64_t)v.r * p.c.kv_heads + v.kvh) * p.mass_stride + tok;
      const int u = mine(v, it);
      if (u < 0) return 0.0f;
      const int t0 = v.tile[u] * kTile;
      return t0 + tok < v.len && t0 + tok < v.raw - v.n ? row[t0] : 0.0f;
    };
    // The item after the present one is looked at early (and read again when it is
    // its turn: kept in registers it would push others out).
    Keys keys{0.0f, false, false}, next{0.0f, false, false};
    float old = 0.0f, old_next = 0.0f;
    bool more = false, ahead = false;
    auto look_ahead = [&](uint32_t it) {
      const uint32_t slot = it % kItems;
      if (!__all_sync(0xffffffffu, mbar_wait_long(&bars[kIFull + slot], (it / kItems) & 1u))) {
        failed = true;
        return;
      }
      const Item& v = list[slot];
      more = v.nb > 0;
      ahead = !v.few && place < v.nb;
      if (more) old_next = held_mass(v, it);
    };
    look_ahead(0);
    if (ahead && !failed && !convert(place, &next)) failed = true;
    while (more && !failed) {
      const Item now = take(item);
      keys = next;
      old = old_next;
      const int rows = now.n * p.group, base = now.raw - now.n;
      if (held && !now.same && lane == 0) mbar_arrive(&bars[kLEmpty + (ql - 1) % kNL]);
      held = now.steps == 1;
      float* const at = row;
      look_ahead(item + 1);
      if (failed) break;
      // The next item's K, as soon as the last product of this one's is done.
      if (ahead && now.few && !convert(tile + now.nb + place, &next)) {
        failed = true;
        break;
      }
      // (A page outside the pool adds nothing.)
      auto put = [&](int pos0, bool there, float total) {
        const int pos = pos0 + tok;
        if (pos < now.len && (there || pos >= base)) at[pos0] = old + (there ? total : 0.0f);
      };
      if (now.few) {
        if (!now.same) ++ql;
        const uint32_t sl = (ql - 1) % kNL;
        const bool ok = (now.same || mbar_wait_long(&bars[kLFull + sl], ((ql - 1) / kNL) & 1u)) &&
                        mbar_wait_long(&bars[kSFull + buf], (g / kNS) & 1u);
        if (!__all_sync(0xffffffffu, ok)) {
          failed = true;
          break;
        }
        tc_fence_after();
        const int u = mine(now, item);
        if (u >= 0) {
          const float* ls = reinterpret_cast<const float*>(smem + LY::kLse + sl * (kStep * 12));
          const int* vs = reinterpret_cast<const int*>(ls) + kStep;
          const int r8 = (rows + 7) & ~7, cols = (3 * r8 + 15) & ~15;
          const uint32_t t_s = tmem + lane_base + buf * kFewCols + u * cols;
          const Keys k0 = read_meta(tile + u);
          const int tile_u = u == 0 ? now.tile[0] : (u == 1 ? now.tile[1] : (u == 2 ? now.tile[2]
                                                                                 : now.tile[3]));
          const int pos0 = tile_u * kTile, pos = pos0 + tok;
          const float2 ks = make_float2(k0.scale, k0.scale), w5 = make_float2(0x1p-5f, 0x1p-5f);
          float2 acc[2] = {};
          const bool all = pos0 + kTile - 1 <= base && vs[kLeftOut - kStep] == 0;
          for (int c = 0; c < rows; c += 8) {
            float x[3][8];
#pragma unroll
            for (int z = 0; z < 3; ++z) tmem_ld<8>(t_s + z * r8 + c, x[z]);
            const float4 l0 = *reinterpret_cast<const float4*>(ls + c);
            const float4 l1 = *reinterpret_cast<const float4*>(ls + c + 4);
            const float4 f0 = *reinterpret_cast<const float4*>(ls + 2 * kStep + c);
            const float4 f1 = *reinterpret_cast<const float4*>(ls + 2 * kStep + c + 4);
            const float2 l[4] = {make_float2(l0.x, l0.y), make_float2(l0.z, l0.w),
                                 make_float2(l1.x, l1.y), make_float2(l1.z, l1.w)};
            const float2 f[4] = {make_float2(f0.x, f0.y), make_float2(f0.z, f0.w),
                                 make_float2(f1.x, f1.y), make_float2(f1.z, f1.w)};
#pragma unroll
            for (int z = 0; z < 3; ++z) tmem_fence<8>(x[z]);
            float2 y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[e] = fma2(make_float2(x[2][2 * e], x[2][2 * e + 1]), w5,
                          make_float2(x[1][2 * e], x[1][2 * e + 1]));
              y[e] = fma2(y[e], w5, make_float2(x[0][2 * e], x[0][2 * e + 1]));
              y[e] = fma2(y[e], mul2(f[e], ks), l[e]);
            }
            // Rows that do not see the position; columns behind the rows hold anything.
            if (!all || c + 8 > rows) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int2 v = *reinterpret_cast<const int2*>(vs + c + 2 * e);
                if (pos >= v.x) y[e].x = -INFINITY;
                if (pos >= v.y) y[e].y = -INFINITY;
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[e & 1] = add2(acc[e & 1], make_float2(ex2(y[e].x), ex2(y[e].y)));
          }
          tc_fence_before();
          put(pos0, k0.there, (acc[0].x + acc[1].x) + (acc[0].y + acc[1].y));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kSFree + buf]);
        ++g;
        buf = buf + 1 == kNS ? 0 : buf + 1;
        tile += now.nb;
        ++item;
        continue;
      }
      const int pos0 = (place ? now.tile[1] : now.tile[0]) * kTile, pos = pos0 + tok;
      const bool edge = pos0 + kTile - 1 > base;   // some row does not see all of the tile
      const bool work = place < now.nb;
      const float2 ks = make_float2(keys.scale, keys.scale);
      float total = 0.0f;
      for (int s = 0; s < now.steps; ++s) {
        if (!now.same) ++ql;
        const uint32_t sl = (ql - 1) % kNL;
        const float* ls = reinterpret_cast<const float*>(smem + LY::kLse + sl * (kStep * 12));
        const int* vs = reinterpret_cast<const int*>(ls) + kStep;
        // (A set without a tile only goes along.)
        const bool ok = (!work || mbar_wait_at(c_full, c_phase)) &&
                              mbar_wait_long(&bars[kLFull + sl], ((ql - 1) / kNL) & 1u);
        if (!__all_sync(0xffffffffu, ok)) {
          failed = true;
          break;
        }
        if (ahead && s + 1 == now.steps && !convert(tile + now.nb + place, &next)) {
          failed = true;
          break;
        }
        if (work) {
          c_phase ^= 1u;
          tc_fence_after();
          float2 acc0 = make_float2(0.0f, 0.0f), acc1 = acc0;
          const uint32_t t_s = tmem + lane_base + place * kStep;
          // Columns of 8. ls holds minus the lse.
          auto add8 = [&](const float* x, int c, bool masked) {
            const float4 l0 = *reinterpret_cast<const float4*>(ls + c);
            const float4 l1 = *reinterpret_cast<const float4*>(ls + c + 4);
            float2 a = fma2(make_float2(x[0], x[1]), ks, make_float2(l0.x, l0.y));
            float2 b = fma2(make_float2(x[2], x[3]), ks, make_float2(l0.z, l0.w));
            float2 d = fma2(make_float2(x[4], x[5]), ks, make_float2(l1.x, l1.y));
            float2 e = fma2(make_float2(x[6], x[7]), ks, make_float2(l1.z, l1.w));
            if (masked) {
              const int4 v0 = *reinterpret_cast<const int4*>(vs + c);
              const int4 v1 = *reinterpret_cast<const int4*>(vs + c + 4);
              if (pos >= v0.x) a.x = -INFINITY;
              if (pos >= v0.y) a.y = -INFINITY;
              if (pos >= v0.z) b.x = -INFINITY;
              if (pos >= v0.w) b.y = -INFINITY;
              if (pos >= v1.x) d.x = -INFINITY;
              if (pos >= v1.y) d.y = -INFINITY;
              if (pos >= v1.z) e.x = -INFINITY;
              if (pos >= v1.w) e.y = -INFINITY;
            }
            acc0 = add2(acc0, make_float2(ex2(a.x), ex2(a.y)));
            acc1 = add2(acc1, make_float2(ex2(b.x), ex2(b.y)));
            acc0 = add2(acc0, make_float2(ex2(d.x), ex2(d.y)));
            acc1 = add2(acc1, make_float2(ex2(e.x), ex2(e.y)));
          };
          auto let_go = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kCFree + place]);
          };
          const int here =
              s + 1 < now.steps && p.chunks == 1 ? capacity : step_of(p, now.n, now.first, s).rows;
          const int c0 = half * (kStep / 2);
          if (here == capacity && capacity > kStep - 16 && !(edge && vs[0] < pos0 + kTile) &&
              vs[kLeftOut - kStep] == 0) {
#pragma unroll
            for (int c = 0; c < kStep / 2; c += 32) {
              float x[32];
              tmem_ld32(t_s + c0 + c, x);
              tmem_fence<32>(x);
              if (c + 32 == kStep / 2) let_go();
#pragma unroll
              for (int e = 0; e < 32; e += 8) add8(x + e, c0 + c + e, false);
            }
          } else {
            // (Columns behind the rows hold anything; no row of theirs sees a position.)
#pragma unroll 1
            for (int c = c0; c < here && c < c0 + kStep / 2; c += 16) {
              float x[16];
              tmem_ld<16>(t_s + c, x);
              tmem_fence<16>(x);
              add8(x, c, true);
              add8(x + 8, c + 8, true);
            }
            let_go();
          }
          total += (acc0.x + acc1.x) + (acc0.y + acc1.y);
        }
        if (now.steps > 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kLEmpty + sl]);
        }
      }
      if (failed) break;
      if (work) {
        // Both halves together; a NaN key makes its position NaN.
        if (keys.nan) total = NAN;
        const uint32_t slot = place * 2 + (summed & 1);
        bool ok;
        if (half == 1) {
          ok = summed < 2 || mbar_wait_long(&bars[kXFree + slot], ((summed >> 1) - 1) & 1u);
          if (ok) {
            other[slot * kTile + tok] = total;
            mbar_arrive(&bars[kXFull + slot]);
          }
        } else {
          ok = mbar_wait_long(&bars[kXFull + slot], (summed >> 1) & 1u);
          if (ok) {
            total += other[slot * kTile + tok];
            mbar_arrive(&bars[kXFree + slot]);
            // (Rarely: unless only rows that are left out see the position.)
            if (total != total && !weighs(p.lse + (int64_t)now.t0 * p.heads + now.kvh * p.group,
                                          p.heads, p.group, pos - base, now.n))
              total = 0.0f;
            put(pos0, keys.there, total);
          }
        }
        ++summed;
        if (!__all_sync(0xffffffffu, ok)) {
          failed = true;
          break;
        }
      }
      tile += now.nb;
      ++item;
    }
  }
  if (failed && p.c.err != nullptr) atomicOr(p.c.err, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, LY::kCols);
}

template <int DIM>
cudaError_t launch_dim(const CUtensorMap& map, const CUtensorMap& q_map, const Params& p, int dev,
                       cudaStream_t stream) {
  static PerDeviceOnce once;
  auto kern = kv8_mass_kernel<DIM>;
  const cudaError_t e = set_max_dynamic_smem(once, dev, kern, Layout<DIM>::kSmem);
  if (e != cudaSuccess) return e;
  // At most one CTA per item.
  const int64_t items = p.c.requests * p.c.kv_heads * ((p.c.bt_stride + 1) / 2);
  const int64_t sms = kv8_sm_count(dev);
  return launch_pdl(kern, dim3((unsigned)(items < sms ? items : sms)), dim3(kThreads),
                    Layout<DIM>::kSmem, stream, 1u, map, q_map, p);
}

}  // namespace

cudaError_t launch_kv8_mass(const Kv8MassArgs& a, cudaStream_t stream) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return cudaErrorNotSupported;
  const int dim = a.c.dim;
  CUtensorMap map;
  const cuuint64_t gdim[2] = {(cuuint64_t)dim,
                              (cuuint64_t)(a.c.num_pages * 2 * a.c.kv_heads * kPage)};
  const cuuint64_t gstride[1] = {(cuuint64_t)dim};
  const cuuint32_t box[2] = {(cuuint32_t)dim, (cuuint32_t)kPage};
  const cuuint32_t estride[2] = {1, 1};
  if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.c.pages, gdim, gstride, box, estride,
          CU_TENSOR_MAP_INTERLEAVE_NONE,
          dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  int dev = 0;
  const cudaError_t e = stream_device(stream, &dev);
  if (e != cudaSuccess) return e;
  Params p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_stride = a.q_stride;
  p.lse = a.lse;
  p.starts = a.starts;
  p.tokens = a.tokens;
  p.heads = a.heads;
  p.group = a.heads / a.c.kv_heads;
  p.step_heads = p.group < kStep ? p.group : kStep;
  p.step_tokens = kStep / p.step_heads;
  p.chunks = (p.group + kStep - 1) / kStep;
  // q as [tokens][heads][dim], in boxes of a step's rows by 64 dims.
  CUtensorMap q_map;
  const cuuint64_t qdim[3] = {(cuuint64_t)dim, (cuuint64_t)a.heads, (cuuint64_t)a.tokens};
  // (One token's stride is never used, and might be none that a map takes.)
  const cuuint64_t qstride[2] = {(cuuint64_t)dim * 2,
                                 (cuuint64_t)(a.tokens > 1 ? a.q_stride : (int64_t)a.heads * dim) * 2};
  const cuuint32_t qbox[3] = {64, (cuuint32_t)p.step_heads, (cuuint32_t)p.step_tokens};
  const cuuint32_t qestride[3] = {1, 1, 1};
  if (enc(&q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), qdim, qstride, qbox,
          qestride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  p.scale_log2 = a.scale * kLog2e;
  p.mass = a.mass;
  p.mass_stride = a.mass_stride;
  p.c = a.c;
  return dim == 128 ? launch_dim<128>(map, q_map, p, dev, stream)
                    : launch_dim<64>(map, q_map, p, dev, stream);
}

}  // namespace dsmla
