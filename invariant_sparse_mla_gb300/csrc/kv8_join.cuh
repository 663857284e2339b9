// Contexts cut into spans, and the kernel that joins what the spans of a row gave.
// (The trees by tiles of 256 rows have spans of their own length and keep their
// partial outputs in another order, which their own kernel joins.)
#pragma once

#include "kv8_common.cuh"

namespace dsmla {

// Spans of MIN to MAX positions, the power of two that gives at most MOST of them
// where MAX allows it: a function of the request's length alone.
template <int MIN, int MAX, int MOST>
struct SpanRule {
  static constexpr int kMost = MOST;
  __host__ __device__ static int of(int64_t len) {
    int s = MIN;
    while (s < MAX && (int64_t)s * MOST < len) s *= 2;
    return s;
  }
  // Most spans a row of at most `len` positions can have.
  static int64_t most(int64_t len) {
    const int64_t a = (len + MIN - 1) / MIN, b = (len + MAX - 1) / MAX;
    return a < MOST ? a : (b > MOST ? b : MOST);
  }
};

// Reference of a span's row that only has scores too low for one.
constexpr float kOnlyLow = -0x1p30f;

// Slot ((request, kv head, row group) * spans + span) * rows + row of the partial
// outputs [.., dim] and (reference, sum).
struct JoinArgs {
  const float* part_o;
  const float2* part_ml;
  __nv_bfloat16* out;
  float* lse;
  Kv8Cache c;
  int next_n, heads, group, rows, row_groups;
  int64_t spans;
};

// Joins the spans of a row, in order: one warp per (request, token, head).
// Requests with one span (or none) are complete already.
template <int DIM, class Spans>
__global__ void __launch_bounds__(256) kv8_join_kernel(const JoinArgs p) {
  constexpr int E = DIM / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  if (w >= p.c.requests * p.next_n * p.heads) return;
  const int64_t token = w / p.heads;
  const int h = (int)(w % p.heads);
  const int64_t r = token / p.next_n;
  const int64_t most = p.c.bt_stride * kPage, raw = p.c.lens[r];
  const int len = (int)(raw < 0 ? 0 : (raw > most ? most : raw));
  const int span = Spans::of(len);
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

}  // namespace dsmla
