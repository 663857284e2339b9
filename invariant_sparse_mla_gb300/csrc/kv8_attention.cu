// Attention over the block-scaled 8-bit cache, the plain kernel: one warp
// per (token, query head), online softmax in fp32, four positions at a time
// (each lane holds dim / 32 of a row's codes, a dot product is a five-step
// warp sum). Right for every shape; its bound is the warp sums.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv8.h"

namespace dsmla {

namespace {

constexpr int kWarps = 8;
constexpr int kErrPage = DS_DEVERR_PAGE;

struct Params {
  const __nv_bfloat16* q;
  int64_t q_stride;
  int64_t tokens;
  const int32_t* starts;
  int heads, group;
  float scale;
  __nv_bfloat16* out;
  float* lse;
  Kv8Cache c;
};

template <int N>
__device__ __forceinline__ void load_codes(const uint8_t* p, float* f) {
  uint32_t w;
  if constexpr (N == 4)
    w = *reinterpret_cast<const uint32_t*>(p);
  else
    w = *reinterpret_cast<const uint16_t*>(p);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)((w >> (16 * i)) & 0xFFFFu), __NV_E4M3);
    const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[2 * i] = g.x;
    f[2 * i + 1] = g.y;
  }
}

template <int DIM>
__global__ void __launch_bounds__(32 * kWarps) kv8_attention_kernel(const Params p) {
  constexpr int N = DIM / 32;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (w >= p.tokens * p.heads) return;
  const int64_t t = w / p.heads;
  const int h = (int)(w % p.heads), g = h / p.group;
  int64_t r, seen;
  {
    auto start_of = [&](int64_t i) {
      const int64_t s = p.starts[i];
      return s < 0 ? 0 : (s > p.tokens ? p.tokens : s);
    };
    int64_t lo = 0, hi = p.c.requests - 1;
    while (lo < hi) {
      const int64_t mid = (lo + hi + 1) >> 1;
      if (start_of(mid) <= t)
        lo = mid;
      else
        hi = mid - 1;
    }
    r = lo;
    const int64_t t0 = start_of(r), t1 = start_of(r + 1);
    if (t < t0 || t >= t1) return;   // no request's row
    seen = (int64_t)p.c.lens[r] - (t1 - t0) + 1 + (t - t0);
  }
  if (seen < 0) seen = 0;
  if (seen > p.c.bt_stride * kPage) seen = p.c.bt_stride * kPage;

  float q[N], o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = __bfloat162float(p.q[t * p.q_stride + h * DIM + lane * N + i]) *
           (p.scale * 1.44269504088896340736f);
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t b = 0; b * kPage < seen; ++b) {
    const int64_t page = p.c.block_table[r * p.c.bt_stride + b];
    if (page < 0 || page >= p.c.num_pages) {
      if (lane == 0 && p.c.err != nullptr) atomicOr(p.c.err, kErrPage);
      continue;
    }
    const int64_t part = page * 2 * p.c.kv_heads + g;
    const float ks = p.c.scales[part], vs = p.c.scales[part + p.c.kv_heads];
    const uint8_t* kp = p.c.pages + part * (kPage * DIM) + lane * N;
    const uint8_t* vp = kp + (int64_t)p.c.kv_heads * kPage * DIM;
    const int n = seen - b * kPage < kPage ? (int)(seen - b * kPage) : kPage;
    for (int s0 = 0; s0 < n; s0 += 4) {
      float s[4], mt = m;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float kf[N], d = 0.0f;
        load_codes<N>(kp + (s0 + u) * DIM, kf);
#pragma unroll
        for (int i = 0; i < N; ++i) d = __fmaf_rn(q[i], kf[i], d);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
        s[u] = s0 + u < n ? d * ks : -INFINITY;
        mt = fmaxf(mt, s[u]);
      }
      if (mt == -INFINITY) continue;
      const float al = exp2f(m - mt);
      l *= al;
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] *= al;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (s0 + u >= n) continue;
        const float e = exp2f(s[u] - mt);
        float vf[N];
        load_codes<N>(vp + (s0 + u) * DIM, vf);
        l += e;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = __fmaf_rn(e * vs, vf[i], o[i]);
      }
      m = mt;
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
  for (int i = 0; i < N; ++i)
    p.out[(t * p.heads + h) * DIM + lane * N + i] = __float2bfloat16(o[i] * inv);
  if (lane == 0)
    p.lse[t * p.heads + h] =
        l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

cudaError_t launch(const Kv8AttnArgs& a, cudaStream_t stream) {
  Params p{reinterpret_cast<const __nv_bfloat16*>(a.q), a.q_stride, a.tokens, a.starts,
           a.heads, a.heads / a.c.kv_heads, a.scale, reinterpret_cast<__nv_bfloat16*>(a.out),
           a.lse, a.c};
  const dim3 grid((unsigned)((a.tokens * a.heads + kWarps - 1) / kWarps));
  if (a.c.dim == 128)
    return launch_pdl(kv8_attention_kernel<128>, grid, dim3(32 * kWarps), 0, stream, 1u, p);
  return launch_pdl(kv8_attention_kernel<64>, grid, dim3(32 * kWarps), 0, stream, 1u, p);
}

}  // namespace

cudaError_t launch_kv8_prefill(const Kv8AttnArgs& a, cudaStream_t stream) {
  return launch(a, stream);
}

size_t kv8_prefill_workspace_bytes(int64_t, int64_t, int, int, int) { return 0; }

}  // namespace dsmla
