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
// in order, so that a K/V tile serves the whole group; a CTA owns 256 rows in
// two row tiles of 128, one kv head, and all positions they see.
//   warps 0-3, 4-7   softmax of row tile 0 and 1 (thread = row = TMEM lane);
//   warps 8-11       codes from global memory, through registers, to f16 tiles
//                    of K and V in shared memory (two buffers each): the copy
//                    engine cannot widen them, and staging the codes in shared
//                    memory first would cost 64 KB of its bandwidth a tile;
//   warp 12          MMA issuer: S = Q K^T (M 128, N 128), O += P V with P from
//                    TMEM, where it lies over S. The two row tiles alternate,
//                    so that one's products run under the other's softmax.
// The bound is the tensor pipe and shared-memory bandwidth behind it: an M 128
// x N 128 x K 16 product reads 8 KB in the 64 cycles it takes.

#include <cuda_runtime.h>
#include <stdint.h>

#include "kv8_common.cuh"

namespace dsmla {

namespace {

constexpr int kTile = 128;               // positions per K/V tile (two pages)
constexpr int kRows = 256;               // query rows per CTA
constexpr int kThreads = 512;
constexpr int kLoaderWarp = 8, kMmaWarp = 12;
constexpr int kErrPage = DS_DEVERR_PAGE, kErrTimeout = DS_DEVERR_TIMEOUT;
// Registers: 512 threads launch with 128 each; 256 * 176 + 128 * 112 +
// 128 * 48 = 65536 = 512 * 128.
constexpr int kRegsSoftmax = 176, kRegsLoader = 112, kRegsMma = 48;

template <int DIM>
struct Layout {
  static constexpr int kBlock = kTile * 128;              // 64 dims of 128 rows in f16
  static constexpr int kTileBytes = DIM / 64 * kBlock;
  static constexpr int kQ = 0;                            // two row tiles
  static constexpr int kK = kQ + 2 * kTileBytes;          // two buffers
  static constexpr int kV = kK + 2 * kTileBytes;          // two buffers
  static constexpr int kBars = kV + 2 * kTileBytes;
  static constexpr int kMeta = kBars + 32 * 8;            // 4 tiles x 2 pages x float4
  static constexpr int kNanMap = kMeta + 4 * 32;          // 2 x [128][DIM / 16] u16
  static constexpr int kNanMapBytes = kTile * (DIM / 16) * 2;
  static constexpr int kRowNan = kNanMap + 2 * kNanMapBytes;   // [256][DIM / 16] u16
  static constexpr int kMisc = kRowNan + kRows * (DIM / 16) * 2;
  static constexpr int kEnd = kMisc + 64;
  static constexpr int kSmem = kEnd + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // TMEM: S (P over its first half) and O of both row tiles.
  static constexpr uint32_t kS = 0, kO = 2 * kTile;
  static constexpr uint32_t kCols = 2 * kTile + 2 * DIM <= 256 ? 256u : 512u;
};

enum Bar {
  kQFull = 0,       // the softmax threads of the row tiles
  kKFull = 1,       // 2: the 128 loader threads
  kKEmpty = 3,      // 2: commit
  kVFull = 5,       // 2: the 128 loader threads
  kVEmpty = 7,      // 2: commit
  kSFull = 9,       // 2 (row tile): commit
  kPFull = 11,      // 2: the row tile's 128 softmax threads
  kPvDone = 13,     // 2: commit
  kDrain = 15,
  kNumBars = 16
};

struct Params {
  const __nv_bfloat16* q;
  int64_t q_stride;
  int64_t tokens;
  const int32_t* starts;
  int heads, group;
  int64_t units;         // row tiles pairs of one kv head, an upper bound
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  Kv8Cache c;
};

template <int DIM>
__global__ void __launch_bounds__(kThreads, 1) kv8_prefill_kernel(const Params p) {
  using LY = Layout<DIM>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + LY::kBars);
  float4* meta = reinterpret_cast<float4*>(smem + LY::kMeta);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + LY::kMisc);
  volatile int* nan_tag = reinterpret_cast<volatile int*>(smem + LY::kMisc + 8);   // 2
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();

  // ---- which rows: n tokens of request r are n * group rows, and the row
  // tile pairs of request r are numbered from floor(starts[r] * group / 256) +
  // r (at least as many as it has). The last ones, which see most, go first.
  const int64_t unit = p.units - 1 - blockIdx.x % p.units;
  const int kvh = (int)(blockIdx.x / p.units);
  auto start_of = [&](int64_t r) {
    const int64_t s = p.starts[r];
    return s < 0 ? 0 : (s > p.tokens ? p.tokens : s);
  };
  int64_t lo = 0, hi = p.c.requests - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (start_of(mid) * p.group / kRows + mid <= unit)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int64_t r = lo, t0 = start_of(r);
  const int64_t n = start_of(r + 1) - t0;
  const int64_t row0 = (unit - (t0 * p.group / kRows + r)) * kRows;
  if (n <= 0 || row0 < 0 || row0 >= n * p.group) return;   // the whole CTA
  const int raw_len = p.c.lens[r];
  const int most = (int)(p.c.bt_stride * kPage);
  auto clamp_pos = [&](int64_t v) { return (int)(v < 0 ? 0 : (v > most ? most : v)); };
  const int len = clamp_pos(raw_len);
  auto visible = [&](int64_t row) { return clamp_pos(raw_len - n + 1 + row / p.group); };
  const int64_t last_row = row0 + kRows <= n * p.group ? row0 + kRows - 1 : n * p.group - 1;
  const int mts = last_row - row0 >= kTile ? 2 : 1;         // row tiles with rows
  const int min_vis = visible(row0);
  const int nt = (visible(last_row) + kTile - 1) / kTile;   // tiles

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t count = 1u;
      if (i == kQFull) count = 128u * mts;
      if ((i >= kKFull && i < kKFull + 2) || (i >= kVFull && i < kVFull + 2) ||
          (i >= kPFull && i < kPFull + 2))
        count = 128u;
      mbar_init(&bars[i], count);
    }
    mbar_fence_init();
    nan_tag[0] = nan_tag[1] = 0;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, LY::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  bool failed = false;
  if (warp < kLoaderWarp) {
    // ----------------------------------------------------------- softmax
    regs_inc<kRegsSoftmax>();
    const int m = warp >> 2;                         // row tile
    const int tiles = m < mts ? nt : 0;
    const int row = (warp & 3) * 32 + lane;          // TMEM lane
    const int64_t grow = row0 + m * kTile + row;     // row of the request
    const bool active = grow < n * p.group;
    const int64_t token = t0 + grow / p.group;
    const int head = kvh * p.group + (int)(grow % p.group);
    const int vis = active ? visible(grow) : 0;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_base + LY::kS + m * kTile;
    const uint32_t t_o = tmem + lane_base + LY::kO + m * DIM;
    float f;
    {
      // The row's q times a power of two, in f16.
      uint4 x[DIM / 8];
      const uint4* src = reinterpret_cast<const uint4*>(p.q + token * p.q_stride + head * DIM);
#pragma unroll
      for (int i = 0; i < DIM / 8; ++i) x[i] = active ? src[i] : make_uint4(0u, 0u, 0u, 0u);
      uint32_t top = 0u;   // largest magnitude bits (NaN above infinity)
#pragma unroll
      for (int i = 0; i < DIM / 8; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int u = 0; u < 4; ++u)
          top = max(top, max((w[u] << 16) & 0x7FFFFFFFu, w[u] & 0x7FFF0000u));
      }
      // Largest |q| 2^k in [2^14, 2^15); 2^k stays a normal float.
      int k = top > 0u ? 14 - ((int)(top >> 23) - 127) : 0;
      k = k > 120 ? 120 : (k < -120 ? -120 : k);
      const float up = __uint_as_float((uint32_t)(k + 127) << 23);
      f = top >= 0x7F800000u ? NAN
                             : __uint_as_float((uint32_t)(127 - k) << 23) * p.scale_log2;
      uint8_t* dst = smem + LY::kQ + m * LY::kTileBytes;
#pragma unroll
      for (int i = 0; i < DIM / 8; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t h[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const __half2 v = __floats2half2_rn(__uint_as_float(w[u] << 16) * up,
                                              __uint_as_float(w[u] & 0xFFFF0000u) * up);
          h[u] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(dst + (i >> 3) * LY::kBlock + swz<128>(row, (i & 7) * 16)) =
            make_uint4(h[0], h[1], h[2], h[3]);
      }
      fence_proxy_async_smem();
      if (m < mts) mbar_arrive(&bars[kQFull]);
    }
    float ref = 0.0f, l = 0.0f;
    bool unset = true, row_nan = false;
    for (int j = 0; j < tiles; ++j) {
      const int pos0 = j * kTile;
      if (!__all_sync(0xffffffffu, mbar_wait_long(&bars[kSFull + m], j & 1))) {
        failed = true;
        break;
      }
      tc_fence_after();
      float s[kTile];
#pragma unroll
      for (int c = 0; c < kTile; c += 32) tmem_ld32(t_s + c, s + c);
      const float4 mt0 = meta[(j & 3) * 2], mt1 = meta[(j & 3) * 2 + 1];
      tmem_fence<kTile>(s);
      // (key scale, log2 of 8 times the value scale, its reciprocal, valid)
      const float g0 = f * mt0.x, g1 = f * mt1.x;
      const float c0 = mt0.y - ref, c1 = mt1.y - ref;
#pragma unroll
      for (int i = 0; i < 64; ++i) s[i] = __fmaf_rn(s[i], g0, c0);
#pragma unroll
      for (int i = 64; i < 128; ++i) s[i] = __fmaf_rn(s[i], g1, c1);
      if (pos0 + kTile > vis || mt0.w == 0.0f || mt1.w == 0.0f) {
        const int end0 = mt0.w != 0.0f ? vis - pos0 : 0, end1 = mt1.w != 0.0f ? vis - pos0 : 0;
#pragma unroll
        for (int i = 0; i < 64; ++i) s[i] = i < end0 ? s[i] : -INFINITY;
#pragma unroll
        for (int i = 64; i < 128; ++i) s[i] = i < end1 ? s[i] : -INFINITY;
      }
      float top[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) top[u] = fmaxf(s[u], s[4 + u]);
#pragma unroll
      for (int i = 8; i < kTile; i += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u) top[u] = fmaxf(top[u], fmaxf(s[i + u], s[i + 4 + u]));
      const float ymax = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      const bool move = unset ? ymax > -INFINITY : ymax > 15.0f;
      if (__any_sync(0xffffffffu, move)) {
        const float by = move ? ymax - 3.0f : 0.0f;
        const float al = move ? (unset ? 0.0f : ex2(-by)) : 1.0f;
        if (move) {
          ref += by;
          l *= al;
          unset = false;
#pragma unroll
          for (int i = 0; i < kTile; ++i) s[i] -= by;
        }
        // (S of tile j was issued behind the end of PV of tile j - 1.)
        if (j > 0 && __any_sync(0xffffffffu, al != 1.0f)) {
#pragma unroll 1
          for (int c = 0; c < DIM; c += 16) {
            float o[16];
            tmem_ld<16>(t_o + c, o);
            tmem_fence<16>(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= al;
#pragma unroll
            for (int i = 0; i < 16; i += 4) tmem_st4(t_o + c + i, o + i);
          }
        }
      }
      float sum0[2] = {0.0f, 0.0f}, sum1[2] = {0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < kTile; c += 32) {
        uint32_t h[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float a = ex2(s[c + 2 * i]), b = ex2(s[c + 2 * i + 1]);
          if (c < 64) {
            sum0[0] += a;
            sum0[1] += b;
          } else {
            sum1[0] += a;
            sum1[1] += b;
          }
          const __half2 v = __floats2half2_rn(a, b);
          h[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        tmem_st16u(t_s + c / 2, h);
      }
      l = __fmaf_rn(sum0[0] + sum0[1], mt0.z, l);
      l = __fmaf_rn(sum1[0] + sum1[1], mt1.z, l);
      // Where rows see different lengths, NaN values were taken out of the tile
      // and listed: the rows that see one get a NaN in that dim.
      if (pos0 + kTile > min_vis) {
        if (!__all_sync(0xffffffffu, mbar_wait_long(&bars[kVFull + (j & 1)], (j >> 1) & 1))) {
          failed = true;
          break;
        }
        if (nan_tag[j & 1] == j + 1) {
          const uint16_t* map =
              reinterpret_cast<const uint16_t*>(smem + LY::kNanMap + (j & 1) * LY::kNanMapBytes);
          uint16_t* mine =
              reinterpret_cast<uint16_t*>(smem + LY::kRowNan) + (m * kTile + row) * (DIM / 16);
          if (!row_nan)
            for (int c = 0; c < DIM / 16; ++c) mine[c] = 0;
          row_nan = true;
          for (int i = 0; i < kTile && pos0 + i < vis; ++i)
            for (int c = 0; c < DIM / 16; ++c) mine[c] |= map[i * (DIM / 16) + c];
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars[kPFull + m]);
    }
    if (!failed && tiles > 0 &&
        !__all_sync(0xffffffffu, mbar_wait_long(&bars[kPvDone + m], (tiles - 1) & 1)))
      failed = true;
    tc_fence_after();
    if (!failed) {
      const float inv = l == 0.0f ? 0.0f : __fdiv_rn(0.125f, l);
      __nv_bfloat16* dst = p.out + (token * p.heads + head) * DIM;
      const uint16_t* mine =
          reinterpret_cast<const uint16_t*>(smem + LY::kRowNan) + (m * kTile + row) * (DIM / 16);
#pragma unroll
      for (int c = 0; c < DIM; c += 32) {
        float o[32];
        if (tiles > 0) {
          tmem_ld32(t_o + c, o);
          tmem_fence<32>(o);
        }
        uint32_t h[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float a = l == 0.0f ? 0.0f : o[2 * i] * inv, b = l == 0.0f ? 0.0f : o[2 * i + 1] * inv;
          if (row_nan) {
            const int d = c + 2 * i;
            if ((mine[d >> 4] >> (d & 15)) & 1) a = NAN;
            if ((mine[d >> 4] >> ((d & 15) + 1)) & 1) b = NAN;
          }
          const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
          h[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        if (active) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            reinterpret_cast<uint4*>(dst + c)[i] =
                make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
        }
      }
      if (active)
        p.lse[token * p.heads + head] = l == 0.0f ? -INFINITY : (ref + log2f(l)) * kLn2;
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------ loader
    regs_dec<kRegsLoader>();
    constexpr int NC = kTile * DIM / 16 / 128;     // 16-code chunks per thread and tile
    constexpr int RC = DIM / 16;                   // chunks per position
    const int lt = tid - kLoaderWarp * 32;
    const int32_t* table = p.c.block_table + r * p.c.bt_stride;
    const int64_t side = (int64_t)p.c.kv_heads * kPage * DIM;
    int err_bits = 0;
    // The pages of tile j (-1: none, or outside the pool).
    auto pages_of = [&](int j, int64_t* pg) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        pg[h] = -1;
        const int b = j * 2 + h;
        if (j < nt && b * kPage < len) {
          const int64_t v = table[b];
          if (v >= 0 && v < p.c.num_pages)
            pg[h] = v;
          else
            err_bits |= kErrPage;
        }
      }
    };
    // Chunk e of this thread: position lt / RC + e * 128 / RC of the tile.
    auto load = [&](const int64_t* pg, int64_t off, uint4* x) {
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        const int64_t page = pg[e / (NC / 2)];
        x[e] = make_uint4(0u, 0u, 0u, 0u);
        if (page >= 0)
          x[e] = __ldg(reinterpret_cast<const uint4*>(
                           p.c.pages + ((page * 2) * p.c.kv_heads + kvh) * (int64_t)(kPage * DIM) +
                           off) +
                       lt + (e % (NC / 2)) * 128);
      }
    };
    auto store = [&](uint8_t* dst, const uint4* x) {
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        const int row = lt / RC + e * (128 / RC), c = lt % RC;
        const uint2 a = codes_to_f16(x[e].x), b = codes_to_f16(x[e].y),
                    d = codes_to_f16(x[e].z), g = codes_to_f16(x[e].w);
        uint8_t* at = dst + (c >> 2) * LY::kBlock;
        const int ch = (c & 3) * 2;
        *reinterpret_cast<uint4*>(at + row * 128 + ((ch ^ (row & 7)) << 4)) =
            make_uint4(a.x, a.y, b.x, b.y);
        *reinterpret_cast<uint4*>(at + row * 128 + (((ch + 1) ^ (row & 7)) << 4)) =
            make_uint4(d.x, d.y, g.x, g.y);
      }
    };
    uint4 kx[NC], vx[NC];
    int64_t now[2], next[2];
    float ks = 0.0f, vs = 1.0f;      // scales of page lt of the tile (threads 0 and 1)
    auto scales_of = [&](const int64_t* pg) {
      ks = 0.0f;
      vs = 1.0f;
      const int64_t page = lt == 0 ? pg[0] : pg[1];
      if (lt < 2 && page >= 0) {
        const int64_t part = page * 2 * p.c.kv_heads + kvh;
        ks = p.c.scales[part];
        vs = p.c.scales[part + p.c.kv_heads];
      }
    };
    pages_of(0, now);
    pages_of(1, next);
    load(now, 0, kx);
    load(now, side, vx);
    scales_of(now);
    for (int j = 0; j < nt; ++j) {
      const int st = j & 1;
      if (!__all_sync(0xffffffffu,
                      j < 2 || mbar_wait_long(&bars[kKEmpty + st], ((j >> 1) - 1) & 1))) {
        failed = true;
        break;
      }
      store(smem + LY::kK + st * LY::kTileBytes, kx);
      if (lt < 2)
        meta[(j & 3) * 2 + lt] =
            make_float4(ks, log2f(vs) + 3.0f, __fdiv_rn(0.125f, vs),
                        (lt == 0 ? now[0] : now[1]) >= 0 ? 1.0f : 0.0f);
      fence_proxy_async_smem();
      mbar_arrive(&bars[kKFull + st]);
      load(next, 0, kx);
      scales_of(next);
      if (!__all_sync(0xffffffffu,
                      j < 2 || mbar_wait_long(&bars[kVEmpty + st], ((j >> 1) - 1) & 1))) {
        failed = true;
        break;
      }
      // Positions behind the context hold anything: zeros in their place (a
      // weight of 0 times NaN is NaN). Where the CTA's rows see different
      // lengths, NaN codes become 0 too, and are listed.
      if ((j + 1) * kTile > min_vis) {
#pragma unroll
        for (int e = 0; e < NC; ++e) {
          const int row = lt / RC + e * (128 / RC), pos = j * kTile + row;
          uint32_t bits = 0u;
          if (pos >= len) {
            vx[e] = make_uint4(0u, 0u, 0u, 0u);
          } else if (pos >= min_vis && has_nan_code(vx[e])) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&vx[e]);
#pragma unroll
            for (int u = 0; u < 16; ++u)
              if (((w[u >> 2] >> (8 * (u & 3))) & 0x7Fu) == 0x7Fu) {
                bits |= 1u << u;
                w[u >> 2] &= ~(0xFFu << (8 * (u & 3)));
              }
            nan_tag[st] = j + 1;
          }
          reinterpret_cast<uint16_t*>(smem + LY::kNanMap + st * LY::kNanMapBytes)[row * RC + lt % RC] =
              (uint16_t)bits;
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
    if (err_bits && lt == 0 && p.c.err != nullptr) atomicOr(p.c.err, err_bits);
  } else {
    regs_dec<kRegsMma>();
    if (warp == kMmaWarp && nt > 0) {
      // -------------------------------------------------------- MMA issuer
      // (the whole warp; one lane issues)
      constexpr uint32_t idesc_s = make_idesc_f16(128, kTile, 0, 0);
      constexpr uint32_t idesc_o = make_idesc_f16(128, DIM, 0, 1);
      const uint64_t q_desc = make_sw128_desc(sbase + LY::kQ, 16, 1024);
      const uint64_t k_desc = make_sw128_desc(sbase + LY::kK, 16, 1024);
      const uint64_t v_desc = make_sw128_desc(sbase + LY::kV, LY::kBlock, 1024);
      const bool leader = elect_one();
      auto issue_s = [&](int m, uint64_t kd, uint64_t* k_empty) {
        if (leader) {
#pragma unroll
          for (int k = 0; k < DIM / 16; ++k) {
            const uint32_t off = (uint32_t)((k >> 2) * LY::kBlock + (k & 3) * 32);
            mma_bf16_ss(tmem + LY::kS + m * kTile, q_desc + ((m * LY::kTileBytes + off) >> 4),
                        kd + (off >> 4), idesc_s, k > 0 ? 1u : 0u);
          }
          mma_commit(&bars[kSFull + m]);
          if (m == mts - 1) mma_commit(k_empty);
        }
        __syncwarp();
      };
      auto issue_o = [&](int m, uint64_t vd, uint64_t* v_empty, bool first) {
        if (leader) {
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_f16_ts(tmem + LY::kO + m * DIM, tmem + LY::kS + m * kTile + k * 8,
                       vd + ((k * 16 * 128) >> 4), idesc_o, k > 0 ? 1u : (first ? 0u : 1u));
          mma_commit(&bars[kPvDone + m]);
          if (m == mts - 1) mma_commit(v_empty);
        }
        __syncwarp();
      };
      failed = !mbar_wait_long(&bars[kQFull], 0) || !mbar_wait_long(&bars[kKFull], 0);
      failed = __any_sync(0xffffffffu, failed);
      if (!failed) {
        tc_fence_after();
        issue_s(0, k_desc, &bars[kKEmpty]);
        if (mts == 2) issue_s(1, k_desc, &bars[kKEmpty]);
      }
      for (int j = 0; j < nt && !failed; ++j) {
        const int st = j & 1, sn = st ^ 1;
        const uint64_t vd = v_desc + (uint64_t)((st * LY::kTileBytes) >> 4);
        const uint64_t kd = k_desc + (uint64_t)((sn * LY::kTileBytes) >> 4);
        bool ok = mbar_wait_long(&bars[kVFull + st], (j >> 1) & 1);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (m >= mts) break;
          ok = ok && mbar_wait_long(&bars[kPFull + m], j & 1);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc_fence_after();
          issue_o(m, vd, &bars[kVEmpty + st], j == 0);
          if (j + 1 < nt) {
            // The next S overwrites this P: only once PV has ended.
            if (m == 0) ok = mbar_wait_long(&bars[kKFull + sn], ((j + 1) >> 1) & 1);
            ok = ok && mbar_wait_long(&bars[kPvDone + m], j & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            issue_s(m, kd, &bars[kKEmpty + sn]);
          }
        }
        failed = !__all_sync(0xffffffffu, ok);
      }
      if (leader) mma_commit(&bars[kDrain]);
      __syncwarp();
      if (!mbar_wait_long(&bars[kDrain], 0)) failed = true;
    }
    __syncwarp();
  }
  if (failed && p.c.err != nullptr) atomicOr(p.c.err, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, LY::kCols);
}

template <int DIM>
cudaError_t launch(const Params& p, int dev, cudaStream_t stream) {
  static PerDeviceOnce once;
  auto kern = kv8_prefill_kernel<DIM>;
  const cudaError_t e = set_max_dynamic_smem(once, dev, kern, Layout<DIM>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)(p.units * p.c.kv_heads)), dim3(kThreads),
                    Layout<DIM>::kSmem, stream, 1u, p);
}

}  // namespace

int64_t kv8_prefill_units(int64_t tokens, int64_t requests, int group) {
  return tokens * group / kRows + requests;
}

size_t kv8_prefill_workspace_bytes(int64_t, int64_t, int, int, int) { return 0; }

cudaError_t launch_kv8_prefill(const Kv8AttnArgs& a, cudaStream_t stream) {
  int dev = 0;
  const cudaError_t e = stream_device(stream, &dev);
  if (e != cudaSuccess) return e;
  Params p;
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
  return a.c.dim == 128 ? launch<128>(p, dev, stream) : launch<64>(p, dev, stream);
}

}  // namespace dsmla
