// Norms of queries and keys per head, with the position rotation, in one pass.
//
// Mathematics. A head's row x of D values becomes
//   y_d = x_d * r * w_d for d < norm_dim, r = 1 / sqrt(mean_{d < norm_dim} x_d^2 + eps),
//   y_d = x_d behind,
// and with angles a_i = position * inv_freq_i the pairs (u, v) of the rotated dims
//   (u cos a_i - v sin a_i, v cos a_i + u sin a_i),
// all in fp32 and rounded to bf16 once. The angle is taken in turns: position and
// frequency are multiplied in two floats each, whole turns are dropped from the
// high part exactly, so that a position of 10^6 loses no more than one of 10.
//
// Layout. A row is cut into units of two 16-byte chunks so that a unit holds
// both halves of the pairs it rotates (dims i and i + rot / 2 are 8 chunks apart
// with rot 128): no exchange between lanes but the sum of squares. LANES lanes
// hold a row (8 for D = 128), UNITS units each. A CTA takes TOK tokens and works
// out their sines and cosines once, in shared memory, for all heads of both sides.
//
// The bound is HBM, 4 bytes an element.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "norm_rope.h"

namespace dsmla {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxAngles = 1024;   // of one CTA

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
  int per_cta;                 // tokens of a CTA
  int row_step;                // rows of a CTA's tokens that the CTAs of grid.y share: stride
  int units;                   // of a row
  int norm_dim, rot_chunk, rot_chunks;   // first rotated chunk, number of them
  const int32_t* positions;
  const float* inv_freq;
  float eps, inv_norm;
};

// cos and sin of pos * freq.
__device__ __forceinline__ float2 rotation(int pos, float freq) {
  // 1 / (2 pi) in two floats; the frequency in turns, in two floats.
  constexpr double kInv2Pi = 0.15915494309189533576888;
  constexpr float kHi = (float)kInv2Pi, kLo = (float)(kInv2Pi - (double)kHi);
  const float fh = freq * kHi;
  const float fl = __fmaf_rn(freq, kLo, __fmaf_rn(freq, kHi, -fh));
  // The position as a multiple of 4096 and a rest, both exact in a float.
  const float a = (float)(pos & ~4095), b = (float)(pos & 4095);
  const float ah = a * fh, al = __fmaf_rn(a, fh, -ah);
  const float bh = b * fh, bl = __fmaf_rn(b, fh, -bh);
  float t = (ah - rintf(ah)) + (bh - rintf(bh));
  t += (al - rintf(al)) + (bl + __fmaf_rn(a, fl, b * fl));
  float2 cs;
  sincospif(2.0f * t, &cs.y, &cs.x);
  return cs;
}

__device__ __forceinline__ void unpack(uint4 v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int LANES, int UNITS, bool PAIRS>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const Params p) {
  constexpr int kRows = kThreads / LANES;      // rows at a time
  __shared__ float2 cs[kMaxAngles];
  const int tid = threadIdx.x, lane = tid % LANES, group = tid / LANES;
  const int heads = p.q.heads + p.k.heads;
  const int64_t token0 = (int64_t)blockIdx.x * p.per_cta;
  const int here = p.tokens - token0 < p.per_cta ? (int)(p.tokens - token0) : p.per_cta;
  const int rows = here * heads;
  const int half = p.rot_chunks * 4;           // angles of a token
  pdl_wait();
  pdl_trigger();

  // The two chunks of unit u. Rotated by halves: chunk i of the first half and of
  // the second; all others two neighbours in what is left.
  auto chunks = [&](int u, int* c0, int* c1, bool* turn0, bool* turn1) {
    if constexpr (PAIRS) {
      *c0 = 2 * u;
      *c1 = 2 * u + 1;
      *turn0 = (unsigned)(*c0 - p.rot_chunk) < (unsigned)p.rot_chunks;
      *turn1 = (unsigned)(*c1 - p.rot_chunk) < (unsigned)p.rot_chunks;
    } else {
      const int hc = p.rot_chunks / 2;
      *turn0 = *turn1 = u < hc;
      if (u < hc) {
        *c0 = p.rot_chunk + u;
        *c1 = p.rot_chunk + hc + u;
      } else {
        const int v = 2 * (u - hc);
        *c0 = v < p.rot_chunk ? v : v + p.rot_chunks;
        *c1 = v + 1 < p.rot_chunk ? v + 1 : v + 1 + p.rot_chunks;
      }
    }
  };
  auto row_at = [&](int row, const Side** side, int64_t* token, int* head) {
    *token = token0 + row / heads;
    const int h = row % heads;
    *side = h < p.q.heads ? &p.q : &p.k;
    *head = h < p.q.heads ? h : h - p.q.heads;
  };

  uint4 raw[UNITS][2];
  auto load = [&](int row) {
    if (row >= rows) return;
    const Side* side;
    int64_t token;
    int head;
    row_at(row, &side, &token, &head);
    const uint4* x = reinterpret_cast<const uint4*>(side->x + token * side->x_stride) +
                     (int64_t)head * (2 * p.units);
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int u = lane + i * LANES;
      if (u < p.units) {
        int c0, c1;
        bool t0, t1;
        chunks(u, &c0, &c1, &t0, &t1);
        raw[i][0] = x[c0];
        raw[i][1] = x[c1];
      }
    }
  };
  int row = blockIdx.y * kRows + group;
  load(row);
  for (int i = tid; i < here * half; i += kThreads)
    cs[i] = rotation(p.positions[token0 + i / half], p.inv_freq[i % half]);
  __syncthreads();

  // Every lane of a row's group runs the same turns, and whole warps stay
  // together: rows past the end are skipped inside.
  for (int base = blockIdx.y * kRows; base < rows; base += p.row_step, row += p.row_step) {
    const bool on = row < rows;
    float x[UNITS][16];
    const Side* side = &p.q;
    int64_t token = token0;
    int head = 0;
    if (on) row_at(row, &side, &token, &head);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int u = lane + i * LANES;
      if (on && u < p.units) {
        unpack(raw[i][0], x[i]);
        unpack(raw[i][1], x[i] + 8);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[i][e] = 0.0f;
      }
    }
    load(row + p.row_step);   // the next row's, while this one is worked on
    if (p.norm_dim > 0) {
#pragma unroll
      for (int i = 0; i < UNITS; ++i) {
        int c0, c1;
        bool t0, t1;
        chunks(lane + i * LANES, &c0, &c1, &t0, &t1);
        if (8 * c0 < p.norm_dim) {
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = __fmaf_rn(x[i][e], x[i][e], sum);
        }
        if (8 * c1 < p.norm_dim) {
#pragma unroll
          for (int e = 8; e < 16; ++e) sum = __fmaf_rn(x[i][e], x[i][e], sum);
        }
      }
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (!on) continue;
    const __nv_bfloat16* w = side->weight;
    const float r = w != nullptr ? rsqrtf(__fmaf_rn(sum, p.inv_norm, p.eps)) : 1.0f;
    const float2* turn = cs + (row / heads) * half;
    uint4* out = reinterpret_cast<uint4*>(side->out + token * side->out_stride) +
                 (int64_t)head * (2 * p.units);
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int u = lane + i * LANES;
      if (u >= p.units) continue;
      int c[2];
      bool t[2];
      chunks(u, &c[0], &c[1], &t[0], &t[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (w != nullptr && 8 * c[h] < p.norm_dim) {
          float g[8];
          unpack(reinterpret_cast<const uint4*>(w)[c[h]], g);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[i][8 * h + e] *= r * g[e];
        }
      }
      if constexpr (PAIRS) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!t[h]) continue;
          const float2* a = turn + (c[h] - p.rot_chunk) * 4;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* y = x[i] + 8 * h + 2 * e;
            const float y0 = y[0], y1 = y[1];
            y[0] = y0 * a[e].x - y1 * a[e].y;
            y[1] = y1 * a[e].x + y0 * a[e].y;
          }
        }
      } else if (t[0]) {
        const float2* a = turn + u * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y0 = x[i][e], y1 = x[i][8 + e];
          x[i][e] = y0 * a[e].x - y1 * a[e].y;
          x[i][8 + e] = y1 * a[e].x + y0 * a[e].y;
        }
      }
      out[c[0]] = pack(x[i]);
      out[c[1]] = pack(x[i] + 8);
    }
  }
}

template <int LANES, int UNITS>
cudaError_t launch_shape(const NormRopeArgs& a, cudaStream_t stream) {
  constexpr int kRows = kThreads / LANES;
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
  p.norm_dim = a.q.weight != nullptr || a.k.weight != nullptr ? a.norm_dim : 0;
  p.rot_chunk = a.rot_start / 8;
  p.rot_chunks = a.rot_dim / 8;
  p.positions = a.positions;
  p.inv_freq = a.inv_freq;
  p.eps = a.eps;
  p.inv_norm = a.norm_dim > 0 ? 1.0f / (float)a.norm_dim : 0.0f;
  const int heads = a.q.heads + a.k.heads, half = a.rot_dim / 2;
  // Few heads: several tokens a CTA, so that it has about four turns.
  int per = 4 * kRows / heads;
  if (half > 0 && per > kMaxAngles / half) per = kMaxAngles / half;
  if (per < 1) per = 1;
  // Fewer where that leaves SMs without work.
  while (per > 1 && (a.tokens + per - 1) / per < 608) per /= 2;
  p.per_cta = per;
  const int64_t blocks = (a.tokens + per - 1) / per;
  // A small call's rows are shared by several CTAs, one turn each.
  int split = (per * heads + kRows - 1) / kRows;
  if (blocks >= 152) split = 1;
  if (split > 64) split = 64;
  p.row_step = split * kRows;
  const dim3 grid((unsigned)blocks, (unsigned)split);
  return a.interleaved
             ? launch_pdl(norm_rope_kernel<LANES, UNITS, true>, grid, dim3(kThreads), 0, stream, 1u, p)
             : launch_pdl(norm_rope_kernel<LANES, UNITS, false>, grid, dim3(kThreads), 0, stream, 1u,
                          p);
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
