// Decode attention over the block-scaled 8-bit cache: keys are multiplied on the
// 8-bit tensor cores as they lie in the cache, values in f16.
//
// Mathematics. With codes K, V (E4M3) and page scales a, b, position i of a
// page gives s_i = scale * a * (q . K_i) and out = sum_i 2^(s_i - M) b V_i / L.
//
// S^T = K Q^T runs on the 8-bit tensor cores with the cache's key bytes as
// they lie there. They take 8-bit operands on both sides, so q is written as
// two E4M3 pieces, each a column of its own with its own power of two:
//   q = 2^-k (q0 + q1 / 32): |q| 2^k is at most 256, q0 = E4M3(q 2^k), q1 the
//   rounded remainder times 32. A bf16 number has 8 significant bits and two
//   pieces hold 2 x 4, so this is exact down to 2^-14 of the row's largest
//   |q| and off by up to 2^-22 of that below, which moves a score by at most
//   scale * a * 448 * the sum of what is lost. Where that passes 2^-14 (an
//   element of q hundreds of times the others; its keys may well be 0) the
//   softmax threads add the lost part's product with the keys: a decision of
//   the row and the page, so that bits depend on nothing else.
//
// O^T = V^T P^T runs in f16: E4M3 to f16 is exact and one instruction for two
// values, and a weight p b, kept as 2^3 p b <= 2^15 in f16, has 11 significant
// bits down to p b = 2^-17 and at least 8 down to 2^-20.
// (Weights as three E4M3 pieces, with V as it lies, were built first: the
// pieces cost more instructions per row than converting V costs per tile, and
// allow a factor of 4 between a weight and the maximum instead of 2^8, so that
// most tiles rescaled: 32 x 5 tokens of 64/8 heads took 1462 us.)
//
// The reference m of a row is the largest s_i + log2 b_i of its first tile and
// moves only when a tile passes it by more than 2^12 (so p b <= 2^12 whatever
// the page scales are). 8 p b is one exponential, of S g + (log2 8b - m), so
// that no large b meets a p below the smallest float; l = sum 2^(s_i - m) is
// kept in fp32 of the unrounded weights, each times 1 / 8b.
//
// Work split. A row's context is cut into spans of 1024 to 4096 positions, the
// power of two that gives at most 32 spans up to 131072 positions: a
// function of the request's length alone, so a request's bits do not depend
// on the batch. (64 / 8 heads x 128, one token of one request on 4096 / 16384
// positions: 14 / 16 us; with spans of 2048 at least 21 / 21 us, of 4096 31 / 34
// us. Large batches pay for it: 32 x 5 tokens on 4096 to 32768 positions 20 us of
// 318, as the spans' partial outputs are written and read once more.)
// A persistent grid takes the (request, kv head, row group, span) items in
// order, each CTA an equal share of the 128-position tiles; a second kernel
// joins the spans in order. Rows with one span are finished by the first kernel.
//
// Per CTA: warps 0-7 softmax (TMEM lane = position; warps w and w + 4 take one
// half of the rows each; they also convert V), warp 8 TMA producer over a ring
// of K and a ring of V tiles (128 positions), warp 9 MMA issuer. The rings
// and barriers run on across items, so the next item's pages stream in while
// the last one is finished. The bound is HBM, 2 * dim bytes a position, with
// one token a request (16 requests on 8192 to 131072 positions, 128 / 8 heads:
// 344 us, 5.74 TB/s), and the softmax threads' work with many rows a kv head (32
// x 5 tokens, 64 / 8 heads: 40 rows a tile, 314 us, 3.74 TB/s, issue slots 46 %
// busy, DRAM 56 %).

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kv8_common.cuh"

namespace dsmla {

namespace {

constexpr int kTile = 128;                 // positions per tile (two pages)
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmax = 32 * kSoftmaxWarps;
constexpr int kProducerWarp = kSoftmaxWarps, kMmaWarp = kSoftmaxWarps + 1;
constexpr int kThreads = kSoftmax + 64;
constexpr int kMaxRows = 40;               // query rows of one row group
constexpr int kMetaSlots = 8;
constexpr float kTau = 12.0f;              // log2: p b may reach 2^kTau
constexpr float kPScale = 8.0f;            // 2^(15 - kTau): stored weights stay <= 2^15
constexpr float kLog2PScale = 3.0f;
constexpr int kErrPage = DS_DEVERR_PAGE, kErrTimeout = DS_DEVERR_TIMEOUT;
constexpr int kMinSpan = 1024, kMaxSpan = 4096;
constexpr float kOnlyLow = -0x1p30f;        // reference of a span's row that only has lower scores
constexpr float kLostMax = 0x1p-14f;       // log2: what two pieces of q may lose of a score

__host__ __device__ inline int span_of(int64_t len) {
  int s = kMinSpan;
  while (s < kMaxSpan && (int64_t)s * 32 < len) s *= 2;
  return s;
}

// Most spans a row of at most `len` positions can have.
int64_t max_spans(int64_t len) {
  const int64_t a = (len + kMinSpan - 1) / kMinSpan, b = (len + kMaxSpan - 1) / kMaxSpan;
  return a < 32 ? a : (b > 32 ? b : 32);
}

struct Shape {
  int rows;     // per row group
  int groups;   // row groups of a kv head
};

Shape shape_of(int next_n, int group) {
  const int total = next_n * group;
  Shape s;
  s.groups = (total + kMaxRows - 1) / kMaxRows;
  s.rows = (total + s.groups - 1) / s.groups;
  return s;
}

template <int R8, int DIM>
struct Layout {
  static constexpr int kNP = (R8 + 15) / 16 * 16;           // columns of P and O
  static constexpr int kUnit = kTile * DIM;                 // K or V codes of one tile
  static constexpr int kQBytes = (2 * R8 * DIM + 1023) / 1024 * 1024;
  // P^T [position][row] in f16: rows of 32, 64 or 128 bytes, swizzled to match.
  static constexpr int kPRow = kNP <= 16 ? 32 : (kNP <= 32 ? 64 : 128);
  static constexpr int kPBytes = kTile * kPRow;
  static constexpr int kRest = 2 * kUnit + kQBytes + kPBytes + 2048 + 1024;
  // CTAs per SM: three where their registers and shared memory allow it (dim 64
  // and up to 16 rows, 64 requests on 4k to 32k positions: 260 us instead of 281
  // with two, 170 instead of 183 with 8 rows; dim 128 is slower with three).
  static constexpr int kCtas = DIM == 64 && R8 <= 16 ? 3 : 2;
  static constexpr int kBudget = 228 * 1024 / kCtas - 1024;   // (1 KB a CTA is the system's)
  static constexpr int kFit = (kBudget - kRest) / kUnit;
  static constexpr int kUnits = kFit > 8 ? 8 : kFit;
  static constexpr int kNK = (kUnits + 1) / 2, kNV = kUnits / 2;   // stages of the two rings
  static_assert(kNK >= 1 && kNV >= 1, "a tile fits");
  static constexpr int kK = 0;
  static constexpr int kV = kK + kNK * kUnit;
  static constexpr int kV16 = kV + kNV * kUnit;             // V of the present tile in f16
  static constexpr int kP = kV16 + 2 * kUnit;
  static constexpr int kQ = kP + kPBytes;
  static constexpr int kBars = kQ + kQBytes;
  static constexpr int kMeta = kBars + 32 * 8;              // kMetaSlots x 2 float4
  static constexpr int kF = kMeta + kMetaSlots * 32;        // per row: factor, minus the reference, alpha
  static constexpr int kM = kF + R8 * 4;
  static constexpr int kAlpha = kM + R8 * 4;
  static constexpr int kWarpMax = kAlpha + R8 * 4;          // 4 x R8 floats
  static constexpr int kVis = kWarpMax + 4 * R8 * 4;        // positions each row sees
  static constexpr int kBy = kVis + R8 * 4;                 // by how much a reference moved
  static constexpr int kSet = kBy + R8 * 4;                 // 1: row has one; 2: only low scores
  static constexpr int kLost = kSet + R8 * 4;               // what a score may lose at key scale 1
  static constexpr int kMisc = kLost + R8 * 4;              // tmem slot, abort, start of work
  static constexpr int kEnd = kMisc + 64;
  static constexpr int kSmem = kEnd + 1024;
  static_assert(kSmem <= kBudget, "shared memory of an SM");
  static constexpr uint32_t kCols = 2 * R8 + kNP <= 32 ? 32u : (2 * R8 + kNP <= 64 ? 64u : 128u);
  static_assert(2 * R8 + kNP <= 128 && kCtas * kCols <= 512, "TMEM columns");
};

enum Bar {
  kKFull = 0,       // <= 4: K landed
  kKEmpty = 4,      // <= 4: its MMAs done
  kVFull = 8,       // <= 4: V landed
  kVEmpty = 12,     // <= 4: V read by the softmax threads
  kSFull = 16,      // S ready
  kSFree = 17,      // S read by the softmax threads
  kPFull = 18,      // P and the f16 V written
  kPvDone = 19,     // PV done (P and f16 V free, O holds the tile)
  kQReady = 20,     // Q pieces written
  kVote = 21,       // every softmax warp has said whether a reference moves
  kDrain = 22,
  kNumBars = 23
};

struct Params {
  const __nv_bfloat16* q;
  int64_t q_stride;
  int next_n, heads, group, rows, row_groups;
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  float* part_o;
  float2* part_ml;
  int64_t spans;         // slots per (request, kv head, row group)
  Kv8Cache c;
};

// The items of one CTA, in order. Every role walks the same sequence.
struct Walk {
  int64_t at, end;       // tile numbers: start of the present item, end of the CTA's share
  int r;                 // request
  int len;               // its positions (at most 2^30)
  int raw;               // lens[r] as it is
  int tiles, span_tiles, spans;
  int hg, s;             // kv head * row_groups + row group; span
  int kvh, rg;           // the two parts of hg
};

__device__ __forceinline__ int clamp_len(const Params& p, int len) {
  const int most = (int)(p.c.bt_stride * kPage);
  return len < 0 ? 0 : (len > most ? most : len);
}
__device__ __forceinline__ int row_len(const Params& p, int64_t r) {
  return clamp_len(p, p.c.lens[r]);
}

__device__ __forceinline__ void walk_load(const Params& p, Walk& w) {
  w.raw = p.c.lens[w.r];
  w.len = clamp_len(p, w.raw);
  w.tiles = (int)((w.len + kTile - 1) / kTile);
  const int span = span_of(w.len);
  w.span_tiles = span / kTile;
  w.spans = (int)((w.len + span - 1) / span);
}

// Moves to the first item at or behind tile offset x of request w.r (whose
// first tile is number `base`), then to later requests while empty.
__device__ __forceinline__ bool walk_settle(const Params& p, Walk& w) {
  const int hgs = p.c.kv_heads * p.row_groups;
  while (true) {
    if (w.s >= w.spans) {   // also a request without positions
      w.s = 0;
      ++w.hg;
      if (++w.rg == p.row_groups) {
        w.rg = 0;
        ++w.kvh;
      }
    }
    if (w.spans == 0 || w.hg >= hgs) {
      w.hg = w.kvh = w.rg = 0;
      w.s = 0;
      if (++w.r >= p.c.requests) return false;
      walk_load(p, w);
      if (w.spans == 0) {
        w.s = 0;
        continue;
      }
    }
    return w.at < w.end;
  }
}

__device__ __forceinline__ int item_tiles(const Walk& w) {
  const int left = w.tiles - w.s * w.span_tiles;
  return left < w.span_tiles ? left : w.span_tiles;
}

__device__ __forceinline__ bool walk_next(const Params& p, Walk& w) {
  w.at += item_tiles(w);
  ++w.s;
  if (w.at >= w.end) return false;
  return walk_settle(p, w);
}

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t b) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)b, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
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
// Two values as two pieces each, and (exactly) what they leave out.
struct Pieces {
  uint32_t b0, b1;
  float lost0, lost1;
};
__device__ __forceinline__ Pieces q_pieces(float u0, float u1) {
  Pieces x;
  x.b0 = to_e4m3x2(u0, u1);
  const float2 h = from_e4m3x2(x.b0);
  const float r0 = (u0 - h.x) * 32.0f, r1 = (u1 - h.y) * 32.0f;
  x.b1 = to_e4m3x2(r0, r1);
  const float2 t = from_e4m3x2(x.b1);
  x.lost0 = (r0 - t.x) * 0.03125f;
  x.lost1 = (r1 - t.y) * 0.03125f;
  return x;
}

__device__ __forceinline__ float warp_top(float a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// Adds to two TMEM columns of the warp's lanes.
__device__ __forceinline__ void tmem_add2(uint32_t taddr, float a, float b) {
  float v[2];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];"
               : "=f"(v[0]), "=f"(v[1])
               : "r"(taddr)
               : "memory");
  tmem_fence<2>(v);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(taddr),
               "f"(v[0] + a), "f"(v[1] + b)
               : "memory");
}

// Lane l's dims (DIM / 32 from l * DIM / 32 on) of a query row.
template <int DIM>
__device__ __forceinline__ void load_q(const __nv_bfloat16* row, int lane, float* x) {
  constexpr int E = DIM / 32;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const uint32_t v = reinterpret_cast<const uint32_t*>(row + lane * E)[e / 2];
    x[e] = __uint_as_float(v << 16);
    x[e + 1] = __uint_as_float(v & 0xFFFF0000u);
  }
}

// Adds what the pieces of up to eight query rows lose to S of the warp's 32
// positions: the lost part times 2^29 (at most 2^14, 8 significant bits) and the
// codes are exact in f16, and the product is summed in fp32. `row` is query row
// lane / 4 of them or nullptr, `keys` the first position's codes, `there` how
// many of them are in the context, `taddr` S of the first row. By mma.sync from
// global memory, as there is no room in shared memory for two more pieces of q.
// 32 x 5 tokens of 64 / 8 heads x 128 on 16384 positions: 268 us, 2055 us where
// every row needs this.
template <int DIM>
__device__ __noinline__ void add_lost(const __nv_bfloat16* row, const uint8_t* keys, int there,
                                      uint32_t taddr, int rows) {
  // Lane 4 g + c holds dims [c, c + 1) * DIM / 4 of row g, and of positions g + 8 i;
  // four of the dims a step. (Kept small: its registers are taken from those of
  // the tiles that need none of this.)
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  auto q4 = [&](int s) {
    return row ? reinterpret_cast<const uint2*>(row + c * (DIM / 4))[s] : make_uint2(0u, 0u);
  };
  float up = 0.0f;
#pragma unroll 1
  for (int s = 0; s < DIM / 16; ++s) {
    const uint2 w = q4(s);
    up = fmaxf(fmaxf(up, fabsf(__uint_as_float(w.x << 16))),
               fmaxf(fabsf(__uint_as_float(w.x & 0xFFFF0000u)),
                     fmaxf(fabsf(__uint_as_float(w.y << 16)),
                           fabsf(__uint_as_float(w.y & 0xFFFF0000u)))));
  }
  up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 1));
  up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 2));
  up = pow2f(q_exponent(up));
  auto lost = [&](uint32_t w) {
    const Pieces z =
        q_pieces(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
    const __half2 h = __floats2half2_rn(z.lost0 * 0x1p29f, z.lost1 * 0x1p29f);
    return *reinterpret_cast<const uint32_t*>(&h);
  };
  float d[2][4] = {};
  keys += g * DIM + c * (DIM / 4);
#pragma unroll 1
  for (int s = 0; s < DIM / 16; ++s) {
    const uint2 w = q4(s);
    const uint32_t b0 = lost(w.x), b1 = lost(w.y);
    auto codes = [&](int i) {
      const uint32_t k =
          8 * i + g < there ? reinterpret_cast<const uint32_t*>(keys + 8 * i * DIM)[s] : 0u;
      return codes_to_f16(k);
    };
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint2 lo = codes(2 * m), hi = codes(2 * m + 1);
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
          "{%8,%9}, {%0,%1,%2,%3};"
          : "+f"(d[m][0]), "+f"(d[m][1]), "+f"(d[m][2]), "+f"(d[m][3])
          : "r"(lo.x), "r"(hi.x), "r"(lo.y), "r"(hi.y), "r"(b0), "r"(b1));
    }
  }
  // Position `lane` of row j lies in d[lane / 16][2 (lane / 8 % 2) + j % 2] of
  // lane 4 (lane % 8) + j / 2.
#pragma unroll 1
  for (int j = 0; j < 8; j += 2) {
    float x[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = __shfl_sync(0xffffffffu, d[i / 2][2 * (i % 2) + u], (lane & 7) * 4 + j / 2);
        if (lane / 8 == i) x[u] = v;
      }
    }
    if (j < rows) tmem_add2(taddr + j, x[0] * 0x1p-29f, x[1] * 0x1p-29f);
  }
  tmem_wait_st();
}

// Sums over the warp of four values a lane: lane l returns the sum of value
// 2 * bit4(l) + bit3(l).
__device__ __forceinline__ float warp_sum4(const float* v, int lane) {
  float a[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 16;
    a[i] = (up ? v[2 + i] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[2 + i], 16);
  }
  const bool up = lane & 8;
  float c = (up ? a[1] : a[0]) + __shfl_xor_sync(0xffffffffu, up ? a[0] : a[1], 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
  return c;
}

// Maxima the same way (a REDUX per row instead is several times slower: 7 us
// a move of 40 rows, measured).
__device__ __forceinline__ float warp_max4(const float* v, int lane) {
  float a[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 16;
    a[i] = fmaxf(up ? v[2 + i] : v[i], __shfl_xor_sync(0xffffffffu, up ? v[i] : v[2 + i], 16));
  }
  const bool up = lane & 8;
  float c = fmaxf(up ? a[1] : a[0], __shfl_xor_sync(0xffffffffu, up ? a[0] : a[1], 8));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, o));
  return c;
}

template <int DIM>
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
  if constexpr (DIM == 128)
    return make_sw128_desc(addr, 16, 1024);
  else
    return make_sw64_desc(addr, 16, 512);
}

template <int R8, int DIM>
__global__ void __launch_bounds__(kThreads, Layout<R8, DIM>::kCtas) kv8_decode_kernel(
    const __grid_constant__ CUtensorMap map, const Params p) {
  using LY = Layout<R8, DIM>;
  constexpr int NP = LY::kNP, NK = LY::kNK, NV = LY::kNV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + LY::kBars);
  float4* meta = reinterpret_cast<float4*>(smem + LY::kMeta);
  float* f_s = reinterpret_cast<float*>(smem + LY::kF);
  float* m_s = reinterpret_cast<float*>(smem + LY::kM);
  float* alpha_s = reinterpret_cast<float*>(smem + LY::kAlpha);
  float* wmax_s = reinterpret_cast<float*>(smem + LY::kWarpMax);
  int* vis_s = reinterpret_cast<int*>(smem + LY::kVis);
  float* by_s = reinterpret_cast<float*>(smem + LY::kBy);
  int* set_s = reinterpret_cast<int*>(smem + LY::kSet);
  float* lost_s = reinterpret_cast<float*>(smem + LY::kLost);
  volatile int* lossy_s = reinterpret_cast<volatile int*>(smem + LY::kMisc + 48);   // a Q's number
  volatile int* move_s = reinterpret_cast<volatile int*>(smem + LY::kMisc + 32);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + LY::kMisc);
  volatile int* abort_s = reinterpret_cast<volatile int*>(smem + LY::kMisc + 40);
  int64_t* start_s = reinterpret_cast<int64_t*>(smem + LY::kMisc + 8);   // request, its first tile
  int64_t* scan_s = reinterpret_cast<int64_t*>(smem + LY::kWarpMax);     // before the loop only
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      const bool all = i == kSFree || i == kPFull || i == kQReady ||
                       (i >= kVEmpty && i < kVEmpty + NV);
      mbar_init(&bars[i], all ? (uint32_t)kSoftmax : (i == kVote ? (uint32_t)kSoftmaxWarps : 1u));
    }
    mbar_fence_init();
    abort_s[0] = abort_s[1] = 0;
    move_s[0] = move_s[1] = *lossy_s = 0;
    for (int r = 0; r < R8; ++r) set_s[r] = 0;
    start_s[0] = -1;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, LY::kCols);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's share: tiles of all requests in a row, an equal part each.
  // Thread t sums a run of requests; a scan over the block finds the run that
  // holds the first tile of the share.
  const int hgs = p.c.kv_heads * p.row_groups;
  const int64_t per = (p.c.requests + kThreads - 1) / kThreads;
  int64_t sum = 0;
  for (int64_t r = tid * per; r < p.c.requests && r < (tid + 1) * per; ++r)
    sum += (row_len(p, r) + kTile - 1) / kTile * (int64_t)hgs;
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
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scan_s[w];
    total += scan_s[w];
  }
  const int64_t lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
  if (lo < hi && lo >= before && lo < before + sum) {
    int64_t base = before;
    for (int64_t r = tid * per; r < p.c.requests; ++r) {
      const int64_t n = (row_len(p, r) + kTile - 1) / kTile * (int64_t)hgs;
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
  Walk w;
  w.r = (int)start_s[0];
  w.end = hi;
  bool some = w.r >= 0;
  if (some) {
    walk_load(p, w);
    const int64_t x = lo - start_s[1];
    w.hg = (int)(x / w.tiles);
    w.kvh = w.hg / p.row_groups;
    w.rg = w.hg % p.row_groups;
    const int tt = (int)(x % w.tiles);
    w.s = (tt + w.span_tiles - 1) / w.span_tiles;
    // The item's first tile (also where s is one past the last span).
    const int st = w.s * w.span_tiles < w.tiles ? w.s * w.span_tiles : w.tiles;
    w.at = lo + (st - tt);
    some = w.at < w.end && walk_settle(p, w);
  }

  bool failed = false;
  if (warp == kProducerWarp) {
    // ---------------------------------------------------------- producer
    uint32_t g = 0;         // tiles issued
    uint32_t k_issued = 0, v_issued = 0;
    int err_bits = 0;
    const int none = (int)(p.c.num_pages * 2 * p.c.kv_heads * kPage);   // a row past the pool: zeros
    // Lane l looks up pages l and l + 32 of a span (and their scales), all at
    // once; the next item's while this item's tiles are issued, since a lookup
    // takes two trips to memory and the rings hold less than that.
    struct Lookup {
      int y[2];
      float ks[2], vs[2];
    };
    auto look = [&](const Walk& i) {
      Lookup k;
      const int kvh = i.kvh, n = 2 * item_tiles(i);
      const int block0 = i.s * i.span_tiles * 2;
      const int blocks = (i.len + kPage - 1) / kPage;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int b = block0 + lane + 32 * e;
        k.y[e] = none;
        k.ks[e] = 0.0f;
        k.vs[e] = 1.0f;
        if (lane + 32 * e < n && b < blocks) {
          const int64_t page = p.c.block_table[(int64_t)i.r * p.c.bt_stride + b];
          if (page >= 0 && page < p.c.num_pages) {
            const int64_t part = page * 2 * p.c.kv_heads + kvh;
            k.y[e] = (int)(part * kPage);
            k.ks[e] = p.c.scales[part];
            k.vs[e] = p.c.scales[part + p.c.kv_heads];
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
      const int nt = item_tiles(w);
      const Lookup now = next;
      const int* y = now.y;
      const float *ks = now.ks, *vs = now.vs;
      some = walk_next(p, w);
      if (some) next = look(w);
      for (int t = 0; t < nt; ++t, ++g) {
        int yy[2];
        float kk[2], vv[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int src = (2 * t + h) & 31, hi2 = (2 * t + h) >> 5;
          yy[h] = __shfl_sync(0xffffffffu, hi2 ? y[1] : y[0], src);
          kk[h] = __shfl_sync(0xffffffffu, hi2 ? ks[1] : ks[0], src);
          vv[h] = __shfl_sync(0xffffffffu, hi2 ? vs[1] : vs[0], src);
        }
        bool ok = true;
        if (lane == 0) {
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            const int n = side ? NV : NK;
            const int st = (int)(g % n);
            uint64_t* full = &bars[(side ? kVFull : kKFull) + st];
            if (g >= n && !mbar_wait_long(&bars[(side ? kVEmpty : kKEmpty) + st],
                                     (uint32_t)((g / n - 1) & 1))) {
              ok = false;
              break;
            }
            if (side == 0) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
                meta[(g & (kMetaSlots - 1)) * 2 + h] =
                    make_float4(kk[h], log2f(vv[h]) + kLog2PScale,
                                __fdiv_rn(1.0f / kPScale, vv[h]), yy[h] == none ? 0.0f : 1.0f);
            }
            mbar_arrive_expect_tx(full, LY::kUnit);
            const uint32_t dst = sbase + (side ? LY::kV : LY::kK) + st * LY::kUnit;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int row = yy[h] == none ? none : yy[h] + side * p.c.kv_heads * kPage;
              tma_load_box(dst + h * (kPage * DIM), &map, 0, row, full);
            }
            if (side == 0)
              k_issued = g + 1;
            else
              v_issued = g + 1;
          }
        }
        if (!__all_sync(0xffffffffu, ok)) {
          failed = true;
          break;
        }
      }
    }
    if (lane == 0) {
      // Every copy has landed before the CTA can exit.
      for (uint32_t i = k_issued > NK ? k_issued - NK : 0; i < k_issued; ++i)
        if (!mbar_wait_long(&bars[kKFull + i % NK], (uint32_t)((i / NK) & 1))) failed = true;
      for (uint32_t i = v_issued > NV ? v_issued - NV : 0; i < v_issued; ++i)
        if (!mbar_wait_long(&bars[kVFull + i % NV], (uint32_t)((i / NV) & 1))) failed = true;
    }
    if (err_bits && p.c.err != nullptr) atomicOr(p.c.err, err_bits);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // -------------------------------------------------------- MMA issuer
    // (the whole warp; one lane issues)
    constexpr uint32_t idesc_s = make_idesc_e4m3(kTile, 2 * R8, 0, 0);
    constexpr uint32_t idesc_o = make_idesc_f16(DIM, NP, 1, 1);
    const uint64_t q_desc = tile_desc<DIM>(sbase + LY::kQ);
    const uint64_t k_desc = tile_desc<DIM>(sbase + LY::kK);
    // f16 V: 64-dim column blocks of 128 rows x 128 bytes.
    const uint64_t v_desc = make_sw128_desc(sbase + LY::kV16, kTile * 128, 1024);
    // P^T: 8 positions x kPRow bytes an atom.
    const uint64_t p_desc = LY::kPRow == 128 ? make_sw128_desc(sbase + LY::kP, 16, 1024)
                            : LY::kPRow == 64 ? make_sw64_desc(sbase + LY::kP, 16, 512)
                                              : make_sw32_desc(sbase + LY::kP, 16, 256);
    const bool leader = elect_one();
    uint32_t g = 0;         // tiles whose S was issued
    uint32_t pv = 0;        // tiles whose PV was issued
    uint32_t queries = 0;
    int64_t last_q = -1;
    auto issue_pv = [&](bool first) {
      // O^T (+)= V^T P^T of tile pv.
      if (!__all_sync(0xffffffffu, mbar_wait_long(&bars[kPFull], pv & 1u))) return false;
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_bf16_ss(tmem + 2 * R8, v_desc + ((k * 16 * 128) >> 4),
                      p_desc + ((k * 16 * LY::kPRow) >> 4), idesc_o,
                      k > 0 ? 1u : (first ? 0u : 1u));
        mma_commit(&bars[kPvDone]);
      }
      __syncwarp();
      ++pv;
      return true;
    };
    while (some && !failed) {
      const int nt = item_tiles(w);
      const int64_t qid = (int64_t)w.r * hgs + w.hg;
      for (int t = 0; t < nt && !failed; ++t) {
        const int st = (int)(g % NK);
        // New Q pieces (written after the last S of the old ones was read); S is
        // free again once tile g - 1 was read.
        bool ok = true;
        if (qid != last_q) {
          last_q = qid;
          ok = mbar_wait_long(&bars[kQReady], queries & 1u);
          ++queries;
        }
        ok = ok && (g == 0 || mbar_wait_long(&bars[kSFree], (g - 1) & 1u)) &&
             mbar_wait_long(&bars[kKFull + st], (g / NK) & 1u);
        if (!__all_sync(0xffffffffu, ok)) {
          failed = true;
          break;
        }
        tc_fence_after();
        if (leader) {
          const uint64_t a = k_desc + (uint64_t)((st * LY::kUnit) >> 4);
#pragma unroll
          for (int k = 0; k < DIM / 32; ++k)
            mma_f8_ss(tmem, a + ((k * 32) >> 4), q_desc + ((k * 32) >> 4), idesc_s,
                      k > 0 ? 1u : 0u);
          mma_commit(&bars[kKEmpty + st]);
          mma_commit(&bars[kSFull]);
        }
        __syncwarp();
        ++g;
        if (t > 0 && !issue_pv(t == 1)) failed = true;
      }
      if (failed) break;
      if (!issue_pv(nt == 1)) failed = true;
      if (!failed) some = walk_next(p, w);
    }
    if (leader) mma_commit(&bars[kDrain]);
    __syncwarp();
    if (!mbar_wait_long(&bars[kDrain], 0)) failed = true;
    __syncwarp();
  } else {
    // ----------------------------------------------------------- softmax
    constexpr int RH = R8 / 2;             // rows of this warp: half * RH ...
    const int quad = warp & 3, half = warp >> 2;
    const int tok = quad * 32 + lane;      // position of the tile (TMEM lane)
    const int rh = half * RH;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    constexpr int PH = NP / 2;             // P and O columns of a half: rows, then padding
    const uint32_t t_s = tmem + lane_base + rh, t_o = tmem + lane_base + 2 * R8 + half * PH;
    const int dim0 = DIM == 128 ? tok : quad * 16 + lane;   // this lane's O row
    const bool has_dim = DIM == 128 || lane < 16;
    // 16-byte chunk c (eight columns) of this thread's position in P^T.
    auto p_chunk = [&](int c) {
      constexpr int W = LY::kPRow;
      const int x = W == 128 ? (tok & 7) : (W == 64 ? (tok >> 1) & 3 : (tok >> 2) & 1);
      return reinterpret_cast<uint4*>(smem + LY::kP + tok * W + ((c ^ x) << 4));
    };
    float l[RH];
    uint32_t g = 0;
    // A wait that gave up ends the loop at the next vote, for every warp alike:
    // it is noted under that vote's tile, before this warp votes there.
    auto give_up = [&] { abort_s[(g + 1) & 1] = (int)(g + 2); };
    int64_t last_q = -1;       // (request, hg) whose Q is in shared memory
    int token = 0;             // of row tid
    int queries = 0;           // Qs so far
    // Requests without positions are no items: their outputs here.
    for (int64_t r = blockIdx.x; r < p.c.requests; r += gridDim.x) {
      if (row_len(p, r) > 0) continue;
      const int64_t n = (int64_t)p.next_n * p.heads;
      uint4* out = reinterpret_cast<uint4*>(p.out + r * n * DIM);
      for (int64_t i = tid; i < n * DIM / 8; i += kSoftmax) out[i] = make_uint4(0u, 0u, 0u, 0u);
      for (int64_t i = tid; i < n; i += kSoftmax) p.lse[r * n + i] = -INFINITY;
    }
    while (some && !failed) {
      const int nt = item_tiles(w);
      const int kvh = w.kvh, row0 = w.rg * p.rows;
      const int rows = min(p.rows, p.next_n * p.group - row0);
      const int64_t qid = (int64_t)w.r * hgs + w.hg;
      auto q_row = [&](int row) {
        return p.q + ((int64_t)w.r * p.next_n + row / p.group) * p.q_stride +
               ((int64_t)kvh * p.group + row % p.group) * DIM;
      };
      // The Q pieces: warp w takes rows w, w + 8, ...; a row's largest |q| sets
      // its power of two. (All S that read the last Q are complete: their
      // results were read.)
      if (qid != last_q) {
        last_q = qid;
        token = (row0 + tid) / p.group;
        ++queries;
        constexpr int E = DIM / 32, NR = R8 / 8;
        float x[NR][E];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int r = warp + 8 * i;
#pragma unroll
          for (int e = 0; e < E; ++e) x[i][e] = 0.0f;
          if (r < rows) load_q<DIM>(q_row(row0 + r), lane, x[i]);
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int r = warp + 8 * i;
          float a = 0.0f;
          bool nan = false;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            a = fmaxf(a, fabsf(x[i][e]));
            nan |= x[i][e] != x[i][e];
          }
          a = warp_top(a);
          nan = __any_sync(0xffffffffu, nan) || a == INFINITY;
          const int k = q_exponent(a);
          const float up = pow2f(k);
          bool tiny = false;     // some element is too small for two pieces
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float u0 = x[i][e] * up, u1 = x[i][e + 1] * up;
            const Pieces z = q_pieces(u0, u1);
            tiny |= (fabsf(u0) < 0x1p-7f && u0 != 0.0f) || (fabsf(u1) < 0x1p-7f && u1 != 0.0f);
            uint8_t* q0 = smem + LY::kQ;
            *reinterpret_cast<uint16_t*>(q0 + swz<DIM>(r, lane * E + e)) = (uint16_t)z.b0;
            *reinterpret_cast<uint16_t*>(q0 + swz<DIM>(R8 + r, lane * E + e)) = (uint16_t)z.b1;
          }
          float lost = 0.0f;     // (a NaN row's scores are NaN whatever it loses)
          if (!nan && __any_sync(0xffffffffu, tiny)) {
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              const Pieces z = q_pieces(x[i][e] * up, x[i][e + 1] * up);
              lost += fabsf(z.lost0) + fabsf(z.lost1);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) lost += __shfl_xor_sync(0xffffffffu, lost, o);
            if (lane == 0) *lossy_s = queries;
          }
          const float f = pow2f(-k) * p.scale_log2;
          if (lane == 0) {
            f_s[r] = nan ? NAN : f;
            lost_s[r] = 448.0f * lost * fabsf(f);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&bars[kQReady]);   // (f_s is read behind the barrier below)
      }
      // Row r's token j sees len - next_n + 1 + j positions (clamped).
      if (tid < R8) {
        const int64_t v = (int64_t)w.raw - p.next_n + 1 + token;
        m_s[tid] = 0.0f;
        vis_s[tid] = (int)(v < 0 ? 0 : (v > w.len ? w.len : v));
      }
#pragma unroll
      for (int i = 0; i < RH; ++i) l[i] = 0.0f;
      uint32_t nan_rows = 0;    // rows that see a NaN value in this lane's dim
      named_bar_sync(1, kSoftmax);   // f_s, m_s, vis_s, lost_s, lossy_s
      float lost_top = 0.0f;    // most that a row of this warp may lose at key scale 1
      if (*lossy_s == queries)
        for (int i = 0; i < RH; ++i) lost_top = fmaxf(lost_top, lost_s[rh + i]);
      const int min_vis = vis_s[0];
      bool unset = true;        // some row has no reference yet

      for (int t = 0; t < nt; ++t, ++g) {
        const int pos0 = (w.s * w.span_tiles + t) * kTile;
        const int pos = pos0 + tok;
        if (!mbar_wait_long(&bars[kSFull], (uint32_t)(g & 1))) abort_s[g & 1] = (int)(g + 1);
        tc_fence_after();
        // (key scale, log2 of 8 times the value scale, its reciprocal, valid)
        const float4 mt = meta[(g & (kMetaSlots - 1)) * 2 + (tok >> 6)];
        if (lost_top * mt.x > kLostMax) {
          // What q's pieces lose goes to S where it lies. (The page is there, and
          // the warp's positions share it.)
          const int first = pos0 + quad * 32;
          const int64_t page = p.c.block_table[(int64_t)w.r * p.c.bt_stride + first / kPage];
          const uint8_t* keys =
              p.c.pages + ((page * 2 * p.c.kv_heads + kvh) * kPage + first % kPage) * DIM;
#pragma unroll 1
          for (int i = 0; i < RH; i += 8) {
            const int r = i + lane / 4;
            const bool lossy = r < RH && lost_s[rh + r] * mt.x > kLostMax;
            if (__any_sync(0xffffffffu, lossy))
              add_lost<DIM>(lossy ? q_row(row0 + rh + r) : nullptr, keys, w.len - first, t_s + i,
                            RH - i);
          }
        }
        float s[RH];
        {
          float lo[RH];
          tmem_ld<RH>(t_s, s);
          tmem_ld<RH>(t_s + R8, lo);
          tmem_fence<RH>(s);
          tmem_fence<RH>(lo);
          const float2 w = make_float2(0.03125f, 0.03125f);
#pragma unroll
          for (int i = 0; i < RH; i += 2) {
            const float2 x = fma2(make_float2(lo[i], lo[i + 1]), w, make_float2(s[i], s[i + 1]));
            s[i] = x.x;
            s[i + 1] = x.y;
          }
        }
        tc_fence_before();
        mbar_arrive(&bars[kSFree]);
        const bool edge = pos0 + kTile > min_vis;   // some row's context ends in the tile
        // s becomes log2 of the stored weight: the exponent relative to the row's
        // reference, and 8 b.
        const float2 ks = make_float2(mt.x, mt.x), vs = make_float2(mt.y, mt.y);
#pragma unroll
        for (int i = 0; i < RH; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(f_s + rh + i);
          const float4 m = *reinterpret_cast<const float4*>(m_s + rh + i);   // minus the reference
          const float2 g0 = mul2(make_float2(f.x, f.y), ks), g1 = mul2(make_float2(f.z, f.w), ks);
          const float2 c0 = add2(make_float2(m.x, m.y), vs), c1 = add2(make_float2(m.z, m.w), vs);
          const float2 x = fma2(make_float2(s[i], s[i + 1]), g0, c0);
          const float2 y = fma2(make_float2(s[i + 2], s[i + 3]), g1, c1);
          s[i] = x.x;
          s[i + 1] = x.y;
          s[i + 2] = y.x;
          s[i + 3] = y.y;
        }
        if (edge || mt.w == 0.0f) {
          const bool here = mt.w != 0.0f && pos < w.len;
#pragma unroll
          for (int i = 0; i < RH; ++i)
            if (!here || pos >= vis_s[rh + i]) s[i] = -INFINITY;
        }
        bool above = unset;
#pragma unroll
        for (int i = 0; i < RH; ++i) above |= s[i] > kTau + kLog2PScale;
        // Does some row's reference move? Each warp says so and goes on to V; the
        // answer is there when it is needed. (Slot g & 1 holds the last tile,
        // plus 1, that moved one; a warp is at most one tile ahead.)
        if (__any_sync(0xffffffffu, above) && lane == 0) move_s[g & 1] = (int)(g + 1);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kVote]);
        // P and the f16 V are free once PV of the last tile is done.
        if (g > 0 && !mbar_wait_long(&bars[kPvDone], (uint32_t)((g - 1) & 1))) give_up();
        // V to f16: half a position's dims per thread.
        {
          const int st = (int)(g % NV);
          if (!mbar_wait_long(&bars[kVFull + st], (uint32_t)((g / NV) & 1))) give_up();
          const uint8_t* src = smem + LY::kV + st * LY::kUnit;
          uint8_t* dst = smem + LY::kV16 + tok * 128;
          constexpr int NC = DIM / 32;         // 16-code chunks of this thread
          bool nan = false;
          auto convert = [&](int c, uint4 v) {
            const uint2 a = codes_to_f16(v.x), b = codes_to_f16(v.y), d = codes_to_f16(v.z),
                        e = codes_to_f16(v.w);
            const int cc = half * NC + c;
            uint8_t* at = dst + (cc >> 2) * (kTile * 128);
            const int ch = (cc & 3) * 2;
            *reinterpret_cast<uint4*>(at + ((ch ^ (tok & 7)) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
            *reinterpret_cast<uint4*>(at + (((ch + 1) ^ (tok & 7)) << 4)) =
                make_uint4(d.x, d.y, e.x, e.y);
          };
          auto codes = [&](int c) {
            return *reinterpret_cast<const uint4*>(src + swz<DIM>(tok, (half * NC + c) * 16));
          };
          if (!edge) {
#pragma unroll
            for (int c0 = 0; c0 < NC; c0 += 2) {
              const uint4 v0 = codes(c0), v1 = codes(c0 + 1);
              convert(c0, v0);
              convert(c0 + 1, v1);
            }
          } else {
            // What lies behind the context is anything, and a weight of 0 times NaN
            // is NaN: it becomes 0.
#pragma unroll 1
            for (int c = 0; c < NC; ++c) {
              uint4 v = codes(c);
              if (pos >= w.len) v = make_uint4(0u, 0u, 0u, 0u);
              nan |= has_nan_code(v);
              convert(c, v);
            }
          }
          mbar_arrive(&bars[kVEmpty + st]);
          // Where the rows of the group see different lengths, a NaN value that
          // only some of them see becomes 0 and is remembered for those (each
          // warp for its own rows; warps of the first half clear it).
          if (edge && named_bar_or(2, kSoftmax, nan && pos >= min_vis)) {
            for (int pass = 0; pass < 2; ++pass) {
              if (has_dim && (pass == 0 || half == 0)) {
                for (int i = 0; i < kTile; ++i) {
                  const int ps = pos0 + i;
                  if (ps < min_vis || ps >= w.len) continue;
                  uint16_t* at = reinterpret_cast<uint16_t*>(
                      smem + LY::kV16 + (dim0 >> 6) * (kTile * 128) + swz<128>(i, (dim0 & 63) * 2));
                  if ((*at & 0x7FFFu) <= 0x7C00u) continue;
                  if (pass == 1) *at = 0;
                  for (int r = 0; r < RH; ++r)
                    if (ps < vis_s[rh + r]) nan_rows |= 1u << r;
                }
              }
              named_bar_sync(1, kSoftmax);
            }
          }
        }
        if (!mbar_wait_long(&bars[kVote], g & 1u)) give_up();
        if (abort_s[g & 1] == (int)(g + 1)) {
          failed = true;
          break;
        }
        if (move_s[g & 1] == (int)(g + 1)) {
          // Rows without a reference take the largest s + log2 b of the tile;
          // rows that pass theirs by more than 2^kTau move it there, and
          // their sums and outputs so far are rescaled. Each row by its own
          // values alone.
#pragma unroll
          for (int i = 0; i < RH; i += 4) {
            const float top = warp_max4(s + i, lane);
            const int r = ((lane >> 4) & 1) * 2 + ((lane >> 3) & 1);
            if ((lane & 7) == 0) wmax_s[quad * R8 + rh + i + r] = top;
          }
          named_bar_sync(1, kSoftmax);
          bool open = false;
          if (tid < R8) {
            float top = wmax_s[tid];
#pragma unroll
            for (int v = 1; v < 4; ++v) top = fmaxf(top, wmax_s[v * R8 + tid]);
            const int vis = vis_s[tid];
            const bool first = set_s[tid] != 1;
            float by = 0.0f, al = 1.0f;
            if (top > (first ? kLowest : kTau + kLog2PScale)) {
              // (By what the reference moves once rounded.)
              const float m = m_s[tid] - reference_step(m_s[tid], top);
              by = m_s[tid] - m;
              al = first ? 0.0f : ex2(-by);
              m_s[tid] = m;
              set_s[tid] = 1;
            } else if (first) {
              if (top > -INFINITY) set_s[tid] = 2;
              open = vis > pos0 + kTile;   // it may see something later
              // (Where no join follows, the row's last tile makes its sum NaN.)
              if (!open && w.spans == 1 && set_s[tid] == 2) by = NAN;
            }
            alpha_s[tid] = al;
            by_s[tid] = by;
          }
          unset = named_bar_or(1, kSoftmax, open);
#pragma unroll
          for (int i = 0; i < RH; i += 4) {
            const float4 al = *reinterpret_cast<const float4*>(alpha_s + rh + i);
            const float4 by = *reinterpret_cast<const float4*>(by_s + rh + i);
            l[i] *= al.x;
            l[i + 1] *= al.y;
            l[i + 2] *= al.z;
            l[i + 3] *= al.w;
            s[i] -= by.x;
            s[i + 1] -= by.y;
            s[i + 2] -= by.z;
            s[i + 3] -= by.w;
          }
          if (t > 0) {
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < RH; i += 4) {
              const float4 al = *reinterpret_cast<const float4*>(alpha_s + rh + i);
              if (al.x != 1.0f || al.y != 1.0f || al.z != 1.0f || al.w != 1.0f) {
                float o[4];
                tmem_ld<4>(t_o + i, o);
                tmem_fence<4>(o);
                o[0] *= al.x;
                o[1] *= al.y;
                o[2] *= al.z;
                o[3] *= al.w;
                tmem_st4(t_o + i, o);
              }
            }
            tmem_wait_st();
          }
        }
        // The weights, their sum, and P.
        const float2 rv = make_float2(mt.z, mt.z);
#pragma unroll
        for (int i = 0; i < RH; i += 2) {
          const float2 e = make_float2(ex2(s[i]), ex2(s[i + 1]));
          const float2 sum = fma2(e, rv, make_float2(l[i], l[i + 1]));
          l[i] = sum.x;
          l[i + 1] = sum.y;
          s[i] = e.x;
          s[i + 1] = e.y;
        }
#pragma unroll
        for (int c = 0; c < (RH + 7) / 8; ++c) {
          uint32_t b[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 8 * c + 2 * e;
            const __half2 h = i < RH ? __floats2half2_rn(s[i < RH ? i : 0], s[i < RH ? i + 1 : 0])
                                     : __floats2half2_rn(0.0f, 0.0f);
            b[e] = *reinterpret_cast<const uint32_t*>(&h);
          }
          *p_chunk(half * (PH / 8) + c) = make_uint4(b[0], b[1], b[2], b[3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&bars[kPFull]);
      }

      // ------------------------------------------------ end of the item
#pragma unroll
      for (int i = 0; i < RH; i += 4) {
        const float v = warp_sum4(l + i, lane);
        const int r = ((lane >> 4) & 1) * 2 + ((lane >> 3) & 1);
        if ((lane & 7) == 0) wmax_s[quad * R8 + rh + i + r] = v;
      }
      if (!mbar_wait_long(&bars[kPvDone], (uint32_t)((g - 1) & 1))) abort_s[g & 1] = (int)(g + 1);
      tc_fence_after();
      float o[RH];
      tmem_ld<RH>(t_o, o);
      tmem_fence<RH>(o);
      named_bar_sync(1, kSoftmax);
      if (nan_rows != 0) {
#pragma unroll
        for (int i = 0; i < RH; ++i)
          if ((nan_rows >> i) & 1) o[i] = NAN;
      }
      auto sum_of = [&](int r) {
        return (wmax_s[r] + wmax_s[R8 + r]) + (wmax_s[2 * R8 + r] + wmax_s[3 * R8 + r]);
      };
      if (w.spans == 1) {
        // The row is complete.
#pragma unroll
        for (int i = 0; i < RH; ++i) {
          const int r = rh + i;
          if (r < rows) {
            const int64_t token = (int64_t)w.r * p.next_n + (row0 + r) / p.group;
            const int64_t h = token * p.heads + kvh * p.group + (row0 + r) % p.group;
            const float ls = sum_of(r);
            const float x = ls == 0.0f ? 0.0f : __fdiv_rn(o[i] * (1.0f / kPScale), ls);
            if (has_dim) p.out[h * DIM + dim0] = __float2bfloat16(x);
            if (tok == 0) p.lse[h] = ls == 0.0f ? -INFINITY : (log2f(ls) - m_s[r]) * kLn2;
          }
        }
      } else {
        const int64_t slot = (qid * p.spans + w.s) * p.rows;
        float* at = p.part_o + (slot + rh) * DIM + dim0;
#pragma unroll
        for (int i = 0; i < RH; ++i)
          if (has_dim && rh + i < rows) at[i * DIM] = o[i] * (1.0f / kPScale);
        if (tid < rows)
          p.part_ml[slot + tid] = make_float2(
              set_s[tid] == 1 ? -m_s[tid] : (set_s[tid] == 2 ? kOnlyLow : -INFINITY), sum_of(tid));
      }
      if (tid < R8) set_s[tid] = 0;
      named_bar_sync(1, kSoftmax);   // m_s and wmax_s are read before the next item writes them
      some = walk_next(p, w);
    }
    failed |= (abort_s[0] | abort_s[1]) != 0;
  }
  if (failed && p.c.err != nullptr) atomicOr(p.c.err, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, LY::kCols);
}

// Joins the spans of a row, in order: one warp per (request, token, head).
// Requests with one span (or none) are complete already.
template <int DIM>
__global__ void __launch_bounds__(256) kv8_decode_join_kernel(const Params p) {
  constexpr int E = DIM / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  if (w >= p.c.requests * p.next_n * p.heads) return;
  const int64_t token = w / p.heads;
  const int h = (int)(w % p.heads);
  const int64_t r = token / p.next_n;
  const int len = row_len(p, r);
  const int span = span_of(len);
  const int spans = (len + span - 1) / span;
  if (spans <= 1) return;
  const int kvh = h / p.group;
  const int row = (int)(token % p.next_n) * p.group + h % p.group;
  const int rg = row / p.rows, rr = row % p.rows;
  const int64_t slot0 =
      ((r * p.c.kv_heads + kvh) * p.row_groups + rg) * p.spans * p.rows + rr;
  float M = -INFINITY;
  for (int s = lane; s < spans; s += 32) M = fmaxf(M, p.part_ml[slot0 + s * p.rows].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float m0 = M == -INFINITY ? 0.0f : M;
  float L = 0.0f, acc[E];
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] = 0.0f;
#pragma unroll 4
  for (int s = 0; s < spans; ++s) {
    const float2 ml = p.part_ml[slot0 + s * p.rows];
    const float wt = ex2(ml.x - m0);
    L = __fmaf_rn(wt, ml.y, L);
    const float* o = p.part_o + (slot0 + s * p.rows) * DIM + lane * E;
    if constexpr (E == 4) {
      const float4 v = *reinterpret_cast<const float4*>(o);
      acc[0] = __fmaf_rn(wt, v.x, acc[0]);
      acc[1] = __fmaf_rn(wt, v.y, acc[1]);
      acc[2] = __fmaf_rn(wt, v.z, acc[2]);
      acc[3] = __fmaf_rn(wt, v.w, acc[3]);
    } else {
      const float2 v = *reinterpret_cast<const float2*>(o);
      acc[0] = __fmaf_rn(wt, v.x, acc[0]);
      acc[1] = __fmaf_rn(wt, v.y, acc[1]);
    }
  }
  if (M == kOnlyLow) L = NAN;
  const float inv = L == 0.0f ? 0.0f : __fdiv_rn(1.0f, L);
  uint32_t b[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    b[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  __nv_bfloat16* out = p.out + w * DIM + lane * E;
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(out) = make_uint2(b[0], b[1]);
  else
    *reinterpret_cast<uint32_t*>(out) = b[0];
  if (lane == 0) p.lse[w] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
}

template <int R8, int DIM>
cudaError_t launch_main(const CUtensorMap& map, const Params& p, int dev, int64_t items,
                        cudaStream_t stream) {
  using LY = Layout<R8, DIM>;
  static PerDeviceOnce once;
  auto kern = kv8_decode_kernel<R8, DIM>;
  const cudaError_t e = set_max_dynamic_smem(once, dev, kern, LY::kSmem);
  if (e != cudaSuccess) return e;
  // At most one CTA per item.
  const int64_t most = LY::kCtas * (int64_t)kv8_sm_count(dev);
  return launch_pdl(kern, dim3((unsigned)(items < most ? items : most)), dim3(kThreads), LY::kSmem,
                    stream, 1u, map, p);
}

template <int DIM>
cudaError_t launch_dim(const CUtensorMap& map, const Params& p, int dev, cudaStream_t stream) {
  const int64_t items = p.c.requests * p.c.kv_heads * p.row_groups * p.spans;
  cudaError_t e;
  switch ((p.rows + 7) / 8) {
    case 1: e = launch_main<8, DIM>(map, p, dev, items, stream); break;
    case 2: e = launch_main<16, DIM>(map, p, dev, items, stream); break;
    case 3: e = launch_main<24, DIM>(map, p, dev, items, stream); break;
    case 4: e = launch_main<32, DIM>(map, p, dev, items, stream); break;
    default: e = launch_main<40, DIM>(map, p, dev, items, stream); break;
  }
  if (e != cudaSuccess || p.spans == 1) return e;   // no table holds a row of two spans
  const int64_t rows = p.c.requests * p.next_n * p.heads;
  return launch_pdl(kv8_decode_join_kernel<DIM>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0,
                    stream, 1u, p);
}

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

int kv8_sm_count(int dev) {
  static std::atomic<int> cached[PerDeviceOnce::kMaxDevices];
  const bool tracked = dev >= 0 && dev < PerDeviceOnce::kMaxDevices;
  int n = tracked ? cached[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      return 152;
    }
    if (tracked) cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

size_t kv8_decode_workspace_bytes(int64_t requests, int next_n, int heads, int kv_heads, int dim,
                                  int64_t bt_stride) {
  const Shape s = shape_of(next_n, heads / kv_heads);
  const int64_t rows = requests * kv_heads * s.groups * max_spans(bt_stride * kPage) * s.rows;
  return 256 + pad256((size_t)rows * dim * 4) + (size_t)rows * 8;
}

cudaError_t launch_kv8_decode(const Kv8AttnArgs& a, cudaStream_t stream) {
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
  cudaError_t e = stream_device(stream, &dev);
  if (e != cudaSuccess) return e;
  Params p;
  const Shape s = shape_of(a.next_n, a.heads / a.c.kv_heads);
  p.q = reinterpret_cast<const __nv_bfloat16*>(a.q);
  p.q_stride = a.q_stride;
  p.next_n = a.next_n;
  p.heads = a.heads;
  p.group = a.heads / a.c.kv_heads;
  p.rows = s.rows;
  p.row_groups = s.groups;
  p.scale_log2 = a.scale * kLog2e;
  p.out = reinterpret_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.spans = max_spans(a.c.bt_stride * kPage);
  const int64_t slots = a.c.requests * a.c.kv_heads * s.groups * p.spans * s.rows;
  p.part_o = reinterpret_cast<float*>(a.workspace);
  p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(a.workspace) +
                                        pad256((size_t)slots * dim * 4));
  p.c = a.c;
  return dim == 128 ? launch_dim<128>(map, p, dev, stream) : launch_dim<64>(map, p, dev, stream);
}

}  // namespace dsmla
