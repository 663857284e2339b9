// Norms of queries and keys per head, with the position rotation, in one pass.
//
// Mathematics. A head's row x of D values becomes
//   y_d = x_d * r * w_d for d < norm_dim, r = 1 / sqrt(mean_{d < norm_dim} x_d^2 + eps),
//   y_d = x_d behind,
// and with angles a_i = position * inv_freq_i the pairs (u, v) of the rotated dims
//   (u cos a_i - v sin a_i, v cos a_i + u sin a_i),
// all in fp32 and rounded to bf16 once. The angle is taken in turns: the position in two
// floats times the frequency in three, whole turns dropped from each product exactly, so
// that a position of 2^31 loses no more than one of 10 (with frequencies up to 1024 the
// angle is off by 2^-23 turns; with the frequency in two floats it was 2^-18.5).
//
// Layout. A row is cut into units of two 16-byte chunks so that a unit holds
// both halves of the pairs it rotates (dims i and i + rot / 2 are 8 chunks apart
// with rot 128): no exchange between lanes but the sum of squares. LANES lanes
// hold a row (8 for D = 128), UNITS units each. A warp takes a token (or, of few
// tokens, some of a token's heads): what all heads share, the weights and the sines
// and cosines, it has in registers (or, with several units a lane, in shared memory)
// and works out once. A row is then about 100 instructions for 32 / LANES of them.
//
// The bound is HBM, 4 bytes an element: 16384 tokens of 72 heads x 128, all normed
// and turned, 110 us (5.5 TB/s, 81 % of a plain copy; a CTA for some rows with the
// angles worked out per CTA and a barrier took 144), 4095 tokens of 129 latent rows of
// 576 dims 206 us (5.9 TB/s; 217). Two tokens: 5 us, the launch and two dependent reads.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv8_common.cuh"
#include "norm_rope.h"

namespace dsmla {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Side {
  const __nv_bfloat16* x;
  int64_t x_stride;
  __nv_bfloat16* out;
  int64_t out_stride;
  const __nv_bfloat16* weight;
  int heads;
};

struct Params {
  Side q, k;
  int64_t tokens;
  int splits, part;            // warps of a token, and the heads of each
  int units;                   // of a row
  int norm_dim, rot_chunk, rot_chunks;   // first rotated chunk, number of them
  const int32_t* positions;
  const float* inv_freq;
  float eps, inv_norm;
};

// cos and sin of pos * freq.
__device__ __forceinline__ float2 rotation(int pos, float freq) {
  // 1 / (2 pi) in three floats.
  constexpr float kHi = 0x1.45f306p-3f, kLo = 0x1.b93910p-28f, kRest = 0x1.529fc2p-54f;
  // The frequency in turns, fh + fl + fr: fl is (what fh leaves) + freq * kLo, fr what the
  // rounding of that sum leaves (Knuth's sum) and the last term. (No product below is
  // contracted with a sum: its own rounding error is what the next term holds.)
  const float fh = __fmul_rn(freq, kHi), r = __fmaf_rn(freq, kHi, -fh);
  const float p = __fmul_rn(freq, kLo), pl = __fmaf_rn(freq, kLo, -p);
  const float fl = __fadd_rn(r, p), y = __fsub_rn(fl, r);
  const float left = __fadd_rn(__fsub_rn(r, __fsub_rn(fl, y)), __fsub_rn(p, y));
  const float fr = __fadd_rn(left, __fmaf_rn(freq, kRest, pl));
  // The position as a multiple of 4096 and a rest, both exact in a float. Near 2^31
  // the products of a have whole turns down to that with fl.
  const float a = (float)(pos & ~4095), b = (float)(pos & 4095);
  const float ah = __fmul_rn(a, fh), al = __fmaf_rn(a, fh, -ah);
  const float am = __fmul_rn(a, fl), ar = __fmaf_rn(a, fl, -am);
  const float bh = __fmul_rn(b, fh), bl = __fmaf_rn(b, fh, -bh);
  float t = (ah - rintf(ah)) + (bh - rintf(bh));
  t += ((al - rintf(al)) + (am - rintf(am))) + (__fmaf_rn(a, fr, ar) + __fmaf_rn(b, fl, bl));
  float2 cs;
  sincospif(2.0f * t, &cs.y, &cs.x);
  return cs;
}

__device__ __forceinline__ void unpack(uint4 v, float2* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack(const float2* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[i].x, x[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// What turns a float2 of values. Halves: two pairs (u from one chunk, v from the
// other); u' = u c + v ns, v' = v c + u s. Neighbours: one pair (u, v); with c twice
// and (-s, s), the pair times c plus the swapped pair times that.
struct Turn {
  float2 c, s, ns;
};

template <int LANES, int UNITS, bool PAIRS>
__global__ void __launch_bounds__(kThreads, UNITS == 1 ? 3 : (UNITS < 4 ? 2 : 1)) norm_rope_kernel(const Params p) {
  constexpr int kRows = 32 / LANES;            // rows of a warp at a time
  extern __shared__ float2 tables[];
  const int lane32 = threadIdx.x & 31, lane = lane32 % LANES, group = lane32 / LANES;
  const int64_t job = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t token = job / p.splits;
  const int head0 = (int)(job % p.splits) * p.part;
  pdl_wait();
  pdl_trigger();
  if (token >= p.tokens) return;

  // The token's angles.
  const int half = p.rot_chunks * 4;
  float2* cs = tables + (threadIdx.x >> 5) * half;
  if (half > 0) {
    const int pos = p.positions[token];
    for (int i = lane32; i < half; i += 32) cs[i] = rotation(pos, p.inv_freq[i]);
    __syncwarp();
  }

  // The two chunks of unit i of this lane, and whether they are turned. Rotated by
  // halves: chunk u of the first half and of the second; all others two neighbours in
  // what is left.
  struct Place {
    int c0, c1;
    bool in, turn0, turn1;
  };
  auto place = [&](int i) {
    const int u = lane + i * LANES;
    Place x;
    x.in = u < p.units;
    if constexpr (PAIRS) {
      x.c0 = 2 * u;
      x.c1 = 2 * u + 1;
      x.turn0 = x.in && (unsigned)(x.c0 - p.rot_chunk) < (unsigned)p.rot_chunks;
      x.turn1 = x.in && (unsigned)(x.c1 - p.rot_chunk) < (unsigned)p.rot_chunks;
    } else {
      const int hc = p.rot_chunks / 2;
      x.turn0 = x.turn1 = u < hc;
      if (u < hc) {
        x.c0 = p.rot_chunk + u;
        x.c1 = p.rot_chunk + hc + u;
      } else {
        const int v = 2 * (u - hc);
        x.c0 = v < p.rot_chunk ? v : v + p.rot_chunks;
        x.c1 = v + 1 < p.rot_chunk ? v + 1 : v + 1 + p.rot_chunks;
      }
    }
    return x;
  };
  // The turns of a unit: [0..3] for the first chunk's float2s, [4..7] the second's
  // (halves: the same four for both).
  auto turn_of = [&](const Place& x, int e) {
    Turn t;
    if constexpr (PAIRS) {
      const float2 a = cs[((e < 4 ? x.c0 : x.c1) - p.rot_chunk) * 4 + (e & 3)];
      t.c = make_float2(a.x, a.x);
      t.s = t.ns = make_float2(-a.y, a.y);
    } else {
      const float4 a =
          *reinterpret_cast<const float4*>(cs + (x.c0 - p.rot_chunk) * 8 + 2 * (e & 3));
      t.c = make_float2(a.x, a.z);
      t.s = make_float2(a.y, a.w);
      t.ns = make_float2(-a.y, -a.w);
    }
    return t;
  };
  constexpr int kTurns = PAIRS ? 8 : 4;
  constexpr bool kKeep = UNITS == 1;           // weights and turns in registers
  const Place only = place(0);
  Turn turns[kKeep ? kTurns : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int e = 0; e < kTurns; ++e)
      if (e < 4 ? only.turn0 : only.turn1) turns[e] = turn_of(only, e);
  }

  // Some heads of one side.
  auto side = [&](const Side& sd, int lo, int hi) {
    if (lo >= hi) return;
    const bool norm = sd.weight != nullptr;
    const uint4* w4 = reinterpret_cast<const uint4*>(sd.weight);
    float2 weight[kKeep ? 8 : 1];
    if constexpr (kKeep) {
#pragma unroll
      for (int e = 0; e < 8; ++e) weight[e] = make_float2(1.0f, 1.0f);
      if (norm && only.in && 8 * only.c0 < p.norm_dim) unpack(w4[only.c0], weight);
      if (norm && only.in && 8 * only.c1 < p.norm_dim) unpack(w4[only.c1], weight + 4);
    }
    const uint4* from = reinterpret_cast<const uint4*>(sd.x + token * sd.x_stride);
    uint4* to = reinterpret_cast<uint4*>(sd.out + token * sd.out_stride);
    const int row_chunks = 2 * p.units;
    uint4 raw[UNITS][2];
    auto load = [&](int h) {
      if (h >= hi) return;
#pragma unroll
      for (int i = 0; i < UNITS; ++i) {
        const Place x = UNITS == 1 ? only : place(i);
        if (x.in) {
          raw[i][0] = from[(int64_t)h * row_chunks + x.c0];
          raw[i][1] = from[(int64_t)h * row_chunks + x.c1];
        }
      }
    };
    load(lo + group);
    // (Whole warps stay together: a group behind the last head works on nothing.)
    for (int base = lo; base < hi; base += kRows) {
      const int h = base + group;
      const bool on = h < hi;
      float2 x[UNITS][8];
#pragma unroll
      for (int i = 0; i < UNITS; ++i) {
        const Place c = UNITS == 1 ? only : place(i);
        if (on && c.in) {
          unpack(raw[i][0], x[i]);
          unpack(raw[i][1], x[i] + 4);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[i][e] = make_float2(0.0f, 0.0f);
        }
      }
      load(h + kRows);   // the next row's, while this one is worked on
      if (norm) {
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
          const Place c = UNITS == 1 ? only : place(i);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (8 * (e < 4 ? c.c0 : c.c1) < p.norm_dim) sum = fma2(x[i][e], x[i][e], sum);
        }
        float total = sum.x + sum.y;
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        const float r = rsqrtf(__fmaf_rn(total, p.inv_norm, p.eps));
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
          const Place c = UNITS == 1 ? only : place(i);
          float2 g[8];
          if constexpr (!kKeep) {
            if (c.in && 8 * c.c0 < p.norm_dim) unpack(w4[c.c0], g);
            if (c.in && 8 * c.c1 < p.norm_dim) unpack(w4[c.c1], g + 4);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (8 * (e < 4 ? c.c0 : c.c1) < p.norm_dim)
              x[i][e] = mul2(mul2(x[i][e], r2), kKeep ? weight[e] : g[e]);
        }
      }
#pragma unroll
      for (int i = 0; i < UNITS; ++i) {
        const Place c = UNITS == 1 ? only : place(i);
        if constexpr (PAIRS) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (!(e < 4 ? c.turn0 : c.turn1)) continue;
            const Turn t = kKeep ? turns[e] : turn_of(c, e);
            const float2 v = x[i][e];
            x[i][e] = fma2(v, t.c, mul2(make_float2(v.y, v.x), t.s));
          }
        } else if (c.turn0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const Turn t = kKeep ? turns[e] : turn_of(c, e);
            const float2 u = x[i][e], v = x[i][4 + e];
            x[i][e] = fma2(u, t.c, mul2(v, t.ns));
            x[i][4 + e] = fma2(v, t.c, mul2(u, t.s));
          }
        }
        if (on && c.in) {
          to[(int64_t)h * row_chunks + c.c0] = pack(x[i]);
          to[(int64_t)h * row_chunks + c.c1] = pack(x[i] + 4);
        }
      }
    }
  };
  const int end = head0 + p.part;
  side(p.q, head0, end < p.q.heads ? end : p.q.heads);
  const int k0 = head0 - p.q.heads, k1 = end - p.q.heads;
  side(p.k, k0 > 0 ? k0 : 0, k1 < p.k.heads ? k1 : p.k.heads);
}

template <int LANES, int UNITS>
cudaError_t launch_shape(const NormRopeArgs& a, cudaStream_t stream) {
  constexpr int kRows = 32 / LANES;
  int dev = 0;
  const cudaError_t e = stream_device(stream, &dev);
  if (e != cudaSuccess) return e;
  Params p;
  auto side = [](const NormRopeSide& s) {
    return Side{static_cast<const __nv_bfloat16*>(s.x), s.x_stride,
                static_cast<__nv_bfloat16*>(s.out), s.out_stride,
                static_cast<const __nv_bfloat16*>(s.weight), s.heads};
  };
  p.q = side(a.q);
  p.k = side(a.k);
  p.tokens = a.tokens;
  p.units = a.dim / 16;
  p.norm_dim = a.norm_dim;
  p.rot_chunk = a.rot_start / 8;
  p.rot_chunks = a.rot_dim / 8;
  p.positions = a.positions;
  p.inv_freq = a.inv_freq;
  p.eps = a.eps;
  p.inv_norm = a.norm_dim > 0 ? 1.0f / (float)a.norm_dim : 0.0f;
  // A warp a token where that fills the GPU (32 warps an SM), else as many as it has
  // turns of kRows heads.
  const int heads = a.q.heads + a.k.heads, most = (heads + kRows - 1) / kRows;
  const int64_t want = (kv8_sm_count(dev) * 32 + a.tokens - 1) / a.tokens;
  p.splits = want < most ? (int)want : most;
  const int turns = (most + p.splits - 1) / p.splits;
  p.part = turns * kRows;
  p.splits = (most + turns - 1) / turns;
  const int64_t jobs = a.tokens * p.splits;
  const dim3 grid((unsigned)((jobs + kWarps - 1) / kWarps));
  const size_t smem = (size_t)kWarps * p.rot_chunks * 4 * sizeof(float2);
  return a.interleaved ? launch_pdl(norm_rope_kernel<LANES, UNITS, true>, grid, dim3(kThreads),
                                    smem, stream, 1u, p)
                       : launch_pdl(norm_rope_kernel<LANES, UNITS, false>, grid, dim3(kThreads),
                                    smem, stream, 1u, p);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  const int units = a.dim / 16;
  if (units <= 4) return launch_shape<4, 1>(a, stream);
  if (units <= 8) return launch_shape<8, 1>(a, stream);
  if (units <= 16) return launch_shape<16, 1>(a, stream);
  if (units <= 32) return launch_shape<16, 2>(a, stream);
  if (units <= 48) return launch_shape<16, 3>(a, stream);
  return launch_shape<16, 4>(a, stream);
}

}  // namespace dsmla
