// Attention mass over the block-scaled 8-bit cache: how much weight each cached
// position got from new tokens.
//
// Mathematics. With codes K (E4M3), key scale a and a token's lse as attention
// gave it,
//   mass[p] += sum over rows (token, head of the group) that see p of
//              2^(scale * log2e * a * (q . K_p) - lse * log2e).
// S^T = K Q^T, positions on the rows of the product: a TMEM lane is a position,
// so its sum over the query rows stays in one thread (two, each with half of the
// rows), nothing is reduced across threads, and the order of the additions
// follows from the request alone.
//
// Both operands are bf16: an E4M3 code has 4 significant bits and an exponent
// that bf16 holds, so K and q enter the product exactly, whatever their
// magnitudes; sums are fp32. A code becomes bf16 by placing its exponent and
// mantissa bits under bf16's (subnormals included) and multiplying by 2^120.
//
// K stays, Q streams: an item is (request, kv head, 128 positions). Its codes
// arrive by TMA, are converted once and written to TMEM as the A operand (64
// columns of bf16 pairs for dim 128, two buffers); the query rows that see the
// tile come in steps of 128 through a ring in shared memory, and S has two
// buffers of 128 columns, so that the product of one step runs under the
// exponentials of the last. With one token a request an item is one step, and the
// bound is HBM, dim bytes a position and head; with prompts it is the tensor
// core (2 dim flops a position and row) and the exponentials next to it.
//
// Work split: a persistent grid, each CTA a run of items of equal cost (steps,
// and a constant for the conversion). A request's tiles are taken from both ends
// in turn, since the last ones are seen by fewer rows.
//
// Per CTA: warps 0-7 convert and sum (warps w and w + 4 take half of the dims and
// half of the columns each), warp 8 brings K, warp 9 issues the products, warps
// 10-13 bring Q and lse.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv8_common.cuh"

namespace dsmla {

namespace {

constexpr int kTile = 128;                 // positions of an item
constexpr int kStep = 128;                 // query rows of a step
constexpr int kSumWarps = 8, kSum = 32 * kSumWarps;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kQWarp = 10, kQWarps = 4;
constexpr int kThreads = 32 * (kQWarp + kQWarps);
constexpr int kMetaSlots = 8;
constexpr int kItemCost = 3;               // of the conversion, in steps
constexpr int kErrPage = DS_DEVERR_PAGE, kErrTimeout = DS_DEVERR_TIMEOUT;

template <int DIM>
struct Layout {
  static constexpr int kKBytes = kTile * DIM;
  static constexpr int kQBytes = kStep * DIM * 2;
  static constexpr int kNK = DIM == 128 ? 4 : 6;    // stages (at most kMetaSlots - 2)
  static constexpr int kNQ = DIM == 128 ? 3 : 4;
  static constexpr int kK = 0;
  static constexpr int kQ = kK + kNK * kKBytes;
  static constexpr int kLse = kQ + kNQ * kQBytes;             // per stage: 128 lse, 128 visible
  static constexpr int kBars = kLse + kNQ * kStep * 8;
  static constexpr int kMeta = kBars + 64 * 8;                // kMetaSlots x float4
  static constexpr int kOther = kMeta + kMetaSlots * 16;      // sums of warps 4-7, two slots
  static constexpr int kMisc = kOther + 2 * kTile * 4;        // tmem slot, start of work, scan
  static constexpr int kEnd = kMisc + 32 + 8 * (kThreads / 32);
  static constexpr int kSmem = kEnd + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  // TMEM columns: S0, S1, then A0, A1.
  static constexpr int kA = 2 * kStep;
  static constexpr int kACols = DIM / 2;
  static constexpr uint32_t kCols = 512;
  static_assert(kA + 2 * kACols <= 512, "TMEM columns");
};

enum Bar {
  kKFull = 0,       // K landed (<= 6)
  kKEmpty = 8,      // K converted
  kQFull = 16,      // Q landed (<= 4)
  kLFull = 20,      // lse written
  kQEmpty = 24,     // product done and lse read
  kAFull = 28,      // 2: A written
  kSFull = 30,      // 2: S ready
  kSFree = 32,      // 2: S read
  kXFull = 34,      // 2: the other half's sums written
  kXFree = 36,      // 2: read
  kDrain = 38,
  kNumBars = 39
};

struct Params {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const float* lse;
  const int32_t* starts;
  int64_t tokens;
  int heads, group;
  int step_heads, step_tokens;     // the rows of a pass of copies: heads, and tokens
  int all_heads, all_tokens;       // the rows of a step
  float scale_log2;
  float* mass;
  int64_t mass_stride;
  Kv8Cache c;
};

// One request, and the CTA's place in it.
struct Walk {
  int64_t at, end;       // cost before the present item; end of the CTA's share
  int r, item_r;         // request; of the item before
  int raw, len, n;       // lens[r], clamped, new tokens
  int64_t t0;            // first token
  int tiles, cost;       // cost of an item
  int i, items;          // present item, items of the request
  int kvh, tile;         // of the present item
  int row_lo;            // first row that sees the tile
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
  w.items = w.tiles * p.c.kv_heads;
  w.cost = kItemCost + (w.n * p.group + kStep - 1) / kStep;   // (rows are below 2^31 - 256)
}

__device__ __forceinline__ void tile_of(const Walk& w, int i, int* kvh, int* tile) {
  *kvh = i / w.tiles;
  const int j = i % w.tiles;
  *tile = j & 1 ? w.tiles - 1 - (j >> 1) : j >> 1;
}

__device__ __forceinline__ void load_item(const Params& p, Walk& w) {
  const int kvh = w.kvh, row_lo = w.row_lo, r = w.item_r;
  const bool one = w.steps == 1;
  tile_of(w, w.i, &w.kvh, &w.tile);
  // Token i sees position p if p <= base + i.
  const int64_t first = (int64_t)w.tile * kTile - ((int64_t)w.raw - w.n);
  w.row_lo = first > 0 ? (int)first * p.group : 0;
  w.steps = (w.n * p.group - w.row_lo + kStep - 1) / kStep;
  w.same = one && w.steps == 1 && r == w.r && kvh == w.kvh && row_lo == w.row_lo;
  w.item_r = w.r;
}

// The next item from w.i on, in later requests where need be.
__device__ __forceinline__ bool walk_settle(const Params& p, Walk& w) {
  while (w.i >= w.items) {
    if (++w.r >= p.c.requests) return false;
    load_request(p, w.r, w);
    w.i = 0;
  }
  if (w.at >= w.end) return false;
  load_item(p, w);
  return true;
}
__device__ __forceinline__ bool walk_next(const Params& p, Walk& w, int items = 1) {
  w.at += (int64_t)items * w.cost;
  w.i += items;
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

template <int DIM>
__global__ void __launch_bounds__(kThreads, 1) kv8_mass_kernel(
    const __grid_constant__ CUtensorMap map, const Params p) {
  using LY = Layout<DIM>;
  constexpr int NK = LY::kNK, NQ = LY::kNQ;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + LY::kBars);
  float4* meta = reinterpret_cast<float4*>(smem + LY::kMeta);
  float* other = reinterpret_cast<float*>(smem + LY::kOther);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + LY::kMisc);
  int64_t* start_s = reinterpret_cast<int64_t*>(smem + LY::kMisc + 8);   // request, cost before it
  int64_t* scan_s = reinterpret_cast<int64_t*>(smem + LY::kMisc + 32);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t n = 1;
      if ((i >= kKEmpty && i < kKEmpty + NK) || (i >= kAFull && i < kAFull + 2)) n = kSum;
      if (i >= kQFull && i < kLFull + NQ) n = 32 * kQWarps;
      if (i >= kQEmpty && i < kQEmpty + NQ) n = 1 + kSumWarps;
      if (i >= kSFree && i < kSFree + 2) n = kSumWarps;
      if (i >= kXFull && i < kXFree + 2) n = kSum / 2;
      mbar_init(&bars[i], n);
    }
    mbar_fence_init();
    start_s[0] = -1;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, LY::kCols);
    tmem_relinquish();
  }
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
    some = walk_settle(p, w);
  }

  bool failed = false;
  if (warp == kProducerWarp) {
    // ---------------------------------------------------------- K producer
    const int none = (int)(p.c.num_pages * 2 * p.c.kv_heads * kPage);   // a row past the pool: zeros
    int err_bits = 0;
    uint32_t g = 0, issued = 0;
    // Lanes 2 e and 2 e + 1 look up the pages of the e-th item from w.i on, 16
    // items of a request at once, and the next 16 while these are issued.
    struct Lookup {
      int count, y;
      float ks;
    };
    auto look = [&](const Walk& v) {
      Lookup k;
      const int64_t left = (v.end - v.at + v.cost - 1) / v.cost;
      k.count = v.items - v.i < 16 ? v.items - v.i : 16;
      if (left < k.count) k.count = (int)left;
      k.y = none;
      k.ks = 0.0f;
      if (lane / 2 < k.count) {
        int kvh, tile;
        tile_of(v, v.i + lane / 2, &kvh, &tile);
        const int b = 2 * tile + (lane & 1);
        if ((int64_t)b * kPage < v.len) {
          const int64_t page = p.c.block_table[(int64_t)v.r * p.c.bt_stride + b];
          if (page >= 0 && page < p.c.num_pages) {
            const int64_t part = page * 2 * p.c.kv_heads + kvh;
            k.y = (int)(part * kPage);
            k.ks = p.c.scales[part] * p.scale_log2;
          } else {
            err_bits |= kErrPage;
          }
        }
      }
      return k;
    };
    Lookup next;
    if (some) next = look(w);
    while (some && !failed) {
      const Lookup now = next;
      some = walk_next(p, w, now.count);
      if (some) next = look(w);
      for (int e = 0; e < now.count; ++e, ++g) {
        const int y0 = __shfl_sync(0xffffffffu, now.y, 2 * e);
        const int y1 = __shfl_sync(0xffffffffu, now.y, 2 * e + 1);
        const float k0 = __shfl_sync(0xffffffffu, now.ks, 2 * e);
        const float k1 = __shfl_sync(0xffffffffu, now.ks, 2 * e + 1);
        bool ok = true;
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
        if (!__all_sync(0xffffffffu, ok)) {
          failed = true;
          break;
        }
      }
    }
    if (lane == 0)   // every copy has landed before the CTA can exit
      for (uint32_t i = issued > NK ? issued - NK : 0; i < issued; ++i)
        if (!mbar_wait_long(&bars[kKFull + i % NK], (uint32_t)((i / NK) & 1))) failed = true;
    if (err_bits && p.c.err != nullptr) atomicOr(p.c.err, err_bits);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer
    const uint64_t q_desc = make_sw128_desc(sbase + LY::kQ, 16, 1024);
    const bool leader = elect_one();
    // Steps (of S buffers) and loads of Q so far: an item of one step may use the
    // load of the one before it, which is let go when the next comes.
    uint32_t item = 0, g = 0, ql = 0;
    bool held = false;
    while (some && !failed) {
      const int rows = w.n * p.group - w.row_lo;
      bool ok = mbar_wait_long(&bars[kAFull + (item & 1)], (item >> 1) & 1u);
      if (held && !w.same) {
        if (leader) mma_commit(&bars[kQEmpty + (ql - 1) % NQ]);
        __syncwarp();
        held = false;
      }
      for (int s = 0; s < w.steps; ++s, ++g) {
        const uint32_t buf = g & 1;
        if (!w.same) ++ql;
        const uint32_t st = (ql - 1) % NQ;
        ok = ok && (w.same || mbar_wait_long(&bars[kQFull + st], ((ql - 1) / NQ) & 1u)) &&
             (g < 2 || mbar_wait_long(&bars[kSFree + buf], ((g >> 1) - 1) & 1u));
        if (!__all_sync(0xffffffffu, ok)) {
          failed = true;
          break;
        }
        fence_proxy_async_smem();   // Q landed through cp.async
        tc_fence_after();
        const int left = rows - s * kStep;
        const int n = left >= kStep ? kStep : (left + 15) & ~15;
        if (leader) {
          const uint32_t idesc = make_idesc_bf16(kTile, n, 0, 0);
          const uint64_t b = q_desc + (uint64_t)((st * LY::kQBytes) >> 4);
#pragma unroll
          for (int k = 0; k < DIM / 16; ++k)
            mma_f16_ts(tmem + buf * kStep, tmem + LY::kA + (item & 1) * LY::kACols + 8 * k,
                       b + (((k >> 2) * (kStep * 128) + (k & 3) * 32) >> 4), idesc, k > 0 ? 1u : 0u);
          if (w.steps > 1) mma_commit(&bars[kQEmpty + st]);
          mma_commit(&bars[kSFull + buf]);
        }
        __syncwarp();
      }
      held = w.steps == 1;
      ++item;
      if (!failed) some = walk_next(p, w);
    }
    if (leader) mma_commit(&bars[kDrain]);
    __syncwarp();
    if (!mbar_wait_long(&bars[kDrain], 0)) failed = true;
    __syncwarp();
  } else if (warp >= kQWarp) {
    // -------------------------------------------------------- Q and lse
    constexpr int L = DIM / 8;                 // lanes of a row (16 bytes each)
    constexpr int ROWS = 32 * kQWarps / L;     // rows of a pass
    const int t = tid - 32 * kQWarp, col = t % L;
    uint32_t g = 0;
    while (some && !failed) {
      if (w.same) {
        some = walk_next(p, w);
        continue;
      }
      const int rows = w.n * p.group - w.row_lo;      // of the item
      const int seen = w.raw - w.n + 1;               // by token 0
      const __nv_bfloat16* q0 = p.q + w.t0 * p.q_stride + (int64_t)w.kvh * p.group * DIM + col * 8;
      const float* lse0 = p.lse + w.t0 * p.heads + w.kvh * p.group;
      // (token, head) of this thread's next row to copy, and of its row of lse,
      // which is read a step ahead.
      int token = (w.row_lo + t / L) / p.group, h = (w.row_lo + t / L) % p.group;
      int l_token = (w.row_lo + t) / p.group, l_h = (w.row_lo + t) % p.group;
      float l_next = t < rows ? lse0[(int64_t)l_token * p.heads + l_h] : INFINITY;
      for (int s = 0; s < w.steps; ++s, ++g) {
        const uint32_t st = g % NQ;
        const int left = rows - s * kStep;
        if (!__all_sync(0xffffffffu, g < NQ || mbar_wait_long(&bars[kQEmpty + st],
                                                              (g / NQ - 1) & 1u))) {
          failed = true;
          break;
        }
        const uint32_t dst = sbase + LY::kQ + st * LY::kQBytes;
        const int upto = left < kStep ? (left + 15) & ~15 : kStep;
#pragma unroll 4
        for (int r = t / L; r < upto; r += ROWS) {
          const bool in = r < left;
          const __nv_bfloat16* src = in ? q0 + token * p.q_stride + h * DIM : p.q;
          cp_async_16(dst + (col >> 3) * (kStep * 128) + r * 128 + (((col & 7) ^ (r & 7)) << 4), src,
                      in ? 16u : 0u);
          token += p.step_tokens;
          h += p.step_heads;
          if (h >= p.group) {
            h -= p.group;
            ++token;
          }
        }
        cp_async_mbar_arrive_noinc(&bars[kQFull + st]);
        // A row that sees nothing adds nothing, nor does one behind the last.
        const float l = l_next;
        const int vis = t < left ? seen + l_token : 0;
        l_token += p.all_tokens;
        l_h += p.all_heads;
        if (l_h >= p.group) {
          l_h -= p.group;
          ++l_token;
        }
        l_next = t < left - kStep ? lse0[(int64_t)l_token * p.heads + l_h] : INFINITY;
        float* ls = reinterpret_cast<float*>(smem + LY::kLse + st * (kStep * 8));
        ls[t] = t >= left || l == -INFINITY ? -INFINITY : -l * kLog2e;
        reinterpret_cast<int*>(ls)[kStep + t] = vis;
        mbar_arrive(&bars[kLFull + st]);
      }
      if (!failed) some = walk_next(p, w);
    }
    cp_async_wait_all();
  } else {
    // --------------------------------------------------- convert and sum
    const int quad = warp & 3, half = warp >> 2;
    const int tok = quad * 32 + lane;          // position of the tile (TMEM lane)
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    uint32_t item = 0, g = 0, ql = 0;
    bool held = false;
    // K of the item-th item to bf16, this thread's half of the dims; returns
    // (scale, page there, a NaN among them).
    auto convert = [&](uint32_t it, float* ks, bool* there, bool* nan) {
      const int st = (int)(it % NK);
      if (!__all_sync(0xffffffffu, mbar_wait_long(&bars[kKFull + st], (it / NK) & 1u))) return false;
      const float4 m = meta[it & (kMetaSlots - 1)];
      *ks = tok < kPage ? m.x : m.z;
      *there = (tok < kPage ? m.y : m.w) != 0.0f;
      const uint8_t* src = smem + LY::kK + st * LY::kKBytes;
      uint32_t bad = 0;
      const uint32_t t_a = tmem + lane_base + LY::kA + (it & 1) * LY::kACols + half * (DIM / 4);
      tc_fence_after();
#pragma unroll
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
      *nan = (bad & 0x80808080u) != 0u;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars[kKEmpty + st]);
      mbar_arrive(&bars[kAFull + (it & 1)]);
      return true;
    };
    float ks = 0.0f, ks_next = 0.0f;
    bool there = false, there_next = false, nan = false, nan_next = false;
    if (some && !convert(0, &ks, &there, &nan)) failed = true;
    while (some && !failed) {
      const int rows_all = w.n * p.group - w.row_lo;
      const int base = w.raw - w.n;
      const int pos0 = w.tile * kTile, pos = pos0 + tok;
      const bool edge = pos0 + kTile - 1 > base;   // some row does not see all of the tile
      const int steps = w.steps;
      const bool same = w.same;
      if (held && !same && lane == 0) mbar_arrive(&bars[kQEmpty + (ql - 1) % NQ]);
      held = steps == 1;
      float* at = p.mass + ((int64_t)w.r * p.c.kv_heads + w.kvh) * p.mass_stride + pos;
      const bool in = pos < w.len;
      float old = 0.0f;
      if (half == 0 && in && pos < base) old = *at;
      // The next item's K, while the products of this one run.
      some = walk_next(p, w);
      if (some && !convert(item + 1, &ks_next, &there_next, &nan_next)) {
        failed = true;
        break;
      }
      const float2 k2 = make_float2(ks, ks);
      float total = 0.0f;
      for (int s = 0; s < steps; ++s, ++g) {
        if (!same) ++ql;
        const uint32_t st = (ql - 1) % NQ, buf = g & 1;
        const int left = rows_all - s * kStep;
        const float* ls = reinterpret_cast<const float*>(smem + LY::kLse + st * (kStep * 8));
        const int* vs = reinterpret_cast<const int*>(ls) + kStep;
        const bool ok = (same || mbar_wait_long(&bars[kLFull + st], ((ql - 1) / NQ) & 1u)) &&
                        mbar_wait_long(&bars[kSFull + buf], (g >> 1) & 1u);
        if (!__all_sync(0xffffffffu, ok)) {
          failed = true;
          break;
        }
        tc_fence_after();
        const uint32_t t_s = tmem + lane_base + buf * kStep + half * 8;
        const float* lh = ls + half * 8;
        const int* vh = vs + half * 8;
        // Columns of 8, warps w and w + 4 in turn. ls holds minus the lse.
        float2 acc0 = make_float2(0.0f, 0.0f), acc1 = acc0;
        const bool masked = edge && vs[0] < pos0 + kTile;
        auto add8 = [&](const float* x, int c) {
          const float4 l0 = *reinterpret_cast<const float4*>(lh + c);
          const float4 l1 = *reinterpret_cast<const float4*>(lh + c + 4);
          float2 a = fma2(make_float2(x[0], x[1]), k2, make_float2(l0.x, l0.y));
          float2 b = fma2(make_float2(x[2], x[3]), k2, make_float2(l0.z, l0.w));
          float2 d = fma2(make_float2(x[4], x[5]), k2, make_float2(l1.x, l1.y));
          float2 e = fma2(make_float2(x[6], x[7]), k2, make_float2(l1.z, l1.w));
          if (masked) {
            const int4 v0 = *reinterpret_cast<const int4*>(vh + c);
            const int4 v1 = *reinterpret_cast<const int4*>(vh + c + 4);
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
        if (left >= kStep) {
          float x[64];
#pragma unroll
          for (int c = 0; c < 8; ++c) tmem_ld<8>(t_s + 16 * c, x + 8 * c);
          tmem_fence<64>(x);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kSFree + buf]);
#pragma unroll
          for (int c = 0; c < 8; ++c) add8(x + 8 * c, 16 * c);
        } else {
          for (int c = 0; c + half * 8 < left; c += 16) {
            float x[8];
            tmem_ld<8>(t_s + c, x);
            tmem_fence<8>(x);
            add8(x, c);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kSFree + buf]);
        }
        if (steps > 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kQEmpty + st]);
        }
        total += (acc0.x + acc1.x) + (acc0.y + acc1.y);
      }
      if (failed) break;
      // Both halves together; a page outside the pool adds nothing, and a NaN key
      // makes its position NaN.
      if (nan) total = NAN;
      const uint32_t slot = item & 1;
      if (half == 1) {
        if (!__all_sync(0xffffffffu, item < 2 || mbar_wait_long(&bars[kXFree + slot],
                                                                ((item >> 1) - 1) & 1u))) {
          failed = true;
          break;
        }
        other[slot * kTile + tok] = total;
        mbar_arrive(&bars[kXFull + slot]);
      } else {
        if (!__all_sync(0xffffffffu, mbar_wait_long(&bars[kXFull + slot], (item >> 1) & 1u))) {
          failed = true;
          break;
        }
        total += other[slot * kTile + tok];
        mbar_arrive(&bars[kXFree + slot]);
        if (in && (there || pos >= base)) *at = old + (there ? total : 0.0f);
      }
      ++item;
      ks = ks_next;
      there = there_next;
      nan = nan_next;
    }
  }
  if (failed && p.c.err != nullptr) atomicOr(p.c.err, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, LY::kCols);
}

template <int DIM>
cudaError_t launch_dim(const CUtensorMap& map, const Params& p, int dev, cudaStream_t stream) {
  static PerDeviceOnce once;
  auto kern = kv8_mass_kernel<DIM>;
  const cudaError_t e = set_max_dynamic_smem(once, dev, kern, Layout<DIM>::kSmem);
  if (e != cudaSuccess) return e;
  // At most one CTA per item.
  const int64_t items = p.c.requests * p.c.kv_heads * ((p.c.bt_stride + 1) / 2);
  const int64_t sms = kv8_sm_count(dev);
  return launch_pdl(kern, dim3((unsigned)(items < sms ? items : sms)), dim3(kThreads),
                    Layout<DIM>::kSmem, stream, 1u, map, p);
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
  const int rows = 32 * kQWarps / (dim / 8);
  p.step_tokens = rows / p.group;
  p.step_heads = rows % p.group;
  p.all_tokens = kStep / p.group;
  p.all_heads = kStep % p.group;
  p.scale_log2 = a.scale * kLog2e;
  p.mass = a.mass;
  p.mass_stride = a.mass_stride;
  p.c = a.c;
  return dim == 128 ? launch_dim<128>(map, p, dev, stream) : launch_dim<64>(map, p, dev, stream);
}

}  // namespace dsmla
