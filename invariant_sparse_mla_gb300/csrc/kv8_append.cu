// Append to the block-scaled 8-bit cache: new tokens' keys and values become
// E4M3 codes under one power-of-two scale per page, side and head.
//
// For a touched (page, side, head): a = max |x| over the new tokens in it,
// need = the smallest 2^e with a <= 448 * 2^e (E4M3's largest value is 448 =
// 1.75 * 2^8, so with a = m * 2^x, 1 <= m < 2: e = x - 8, one more if m >
// 1.75), scale = max(old, need). A power of two costs no precision (E4M3's
// rounding is relative), and a page whose scale grows while a request is
// written token by token keeps its earlier values exactly, but for codes that
// fall below the normal range.
//
// One CTA of 128 threads owns one (page of a request, side, head): nothing
// is shared between CTAs, so there is no atomic and no second pass. The
// tokens stay in registers between the maximum and the rounding: thread i
// holds 16-byte chunks i, i + 128, ... of the page's [64, dim] block. The
// bound is HBM: 2 bytes read and 1 written per element.
//
// The grid covers an upper bound of the touched pages: n consecutive
// positions touch at most floor(n / 64) + 2 pages, so request r's pages are
// numbered from floor(starts[r] / 64) + 2 r and a binary search finds r.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv8.h"

namespace dsmla {

namespace {

constexpr int kThreads = 128;
constexpr int kErrPage = DS_DEVERR_PAGE, kErrLen = DS_DEVERR_LEN;

// Smallest power of two s with a <= 448 s, exponent limited to [-60, 120].
__device__ __forceinline__ float need_scale(float a) {
  if (!(a > 0.0f)) return 0.0f;
  const uint32_t b = __float_as_uint(a);
  int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < -60 ? -60 : (e > 120 ? 120 : e);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

struct Params {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t k_stride, v_stride;
  int64_t tokens;
  const int32_t* starts;
  Kv8Cache c;
};

template <int DIM>
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(const Params p) {
  constexpr int kRowChunks = DIM / 8;                     // 16-byte chunks of a token's head
  constexpr int kSteps = kPage * kRowChunks / kThreads;   // chunks per thread
  __shared__ float warp_max[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int head = blockIdx.y >> 1, side = blockIdx.y & 1;
  const int64_t unit = blockIdx.x;
  // The last request whose first unit is not past this one.
  int64_t lo = 0, hi = p.c.requests - 1;
  auto start_of = [&](int64_t r) {
    const int64_t s = p.starts[r];
    return s < 0 ? 0 : (s > p.tokens ? p.tokens : s);
  };
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if ((start_of(mid) >> 6) + 2 * mid <= unit)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int64_t r = lo;
  const int64_t t0 = start_of(r), n = start_of(r + 1) - t0;
  if (n <= 0) return;
  const int64_t len = p.c.lens[r], first = len - n;
  const int64_t j = unit - ((t0 >> 6) + 2 * r);   // page of this request's touched ones
  if (first < 0) {
    if (j == 0 && blockIdx.y == 0 && tid == 0 && p.c.err != nullptr)
      atomicOr(p.c.err, kErrLen);
    return;
  }
  const int64_t block = (first >> 6) + j;
  if (j < 0 || (block << 6) >= len) return;
  int64_t page = -1;
  if (block < p.c.bt_stride) page = p.c.block_table[r * p.c.bt_stride + block];
  if (page < 0 || page >= p.c.num_pages) {
    if (blockIdx.y == 0 && tid == 0 && p.c.err != nullptr) atomicOr(p.c.err, kErrPage);
    return;
  }
  const int64_t pos0 = block << 6;
  const int had = first > pos0 ? (int)(first - pos0) : 0;             // earlier positions
  const int upto = len - pos0 < kPage ? (int)(len - pos0) : kPage;    // new: [had, upto)
  const int64_t part = (page * 2 + side) * p.c.kv_heads + head;
  float* scale_at = p.c.scales + part;
  const float old = had > 0 ? *scale_at : 0.0f;

  const __nv_bfloat16* src = side ? p.v : p.k;
  const int64_t stride = side ? p.v_stride : p.k_stride;
  uint4 x[kSteps];
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int c = tid + i * kThreads, slot = c / kRowChunks, ch = c % kRowChunks;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (slot >= had && slot < upto) {
      const int64_t t = t0 + (pos0 + slot - first);
      x[i] = *reinterpret_cast<const uint4*>(src + t * stride + head * DIM + ch * 8);
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int u = 0; u < 4; ++u)
      a = fmaxf(a, fmaxf(fabsf(__uint_as_float(w[u] << 16)),
                         fabsf(__uint_as_float(w[u] & 0xFFFF0000u))));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((tid & 31) == 0) warp_max[tid >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) a = fmaxf(a, warp_max[w]);
  float s = fmaxf(old, need_scale(a));
  if (!(s > 0.0f)) s = __uint_as_float((uint32_t)(127 - 60) << 23);

  uint8_t* dst = p.c.pages + part * (int64_t)(kPage * DIM);
  if (had > 0 && s != old) {
    // Earlier codes at the grown scale.
    const float f = __fdiv_rn(old, s);
    for (int c = tid; c < had * DIM / 4; c += kThreads) {
      uint32_t* at = reinterpret_cast<uint32_t*>(dst) + c;
      const uint32_t w = *at;
      uint32_t r2 = 0u;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((w >> (16 * u)) & 0xFFFFu), __NV_E4M3);
        const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&h));
        r2 |= e4m3x2(g.x * f, g.y * f) << (16 * u);
      }
      *at = r2;
    }
  }
  // Dividing by a power of two is multiplying by its reciprocal, exactly; a
  // scale that a caller set to something else takes the division.
  const uint32_t sb = __float_as_uint(s);
  const bool pow2 = (sb & 0x7FFFFFu) == 0u && sb >= (67u << 23) && sb <= (247u << 23);
  const float inv = pow2 ? __uint_as_float((254u << 23) - sb) : 0.0f;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int c = tid + i * kThreads, slot = c / kRowChunks;
    if (slot < had || slot >= upto) continue;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t o[2] = {0u, 0u};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float f0 = __uint_as_float(w[u] << 16), f1 = __uint_as_float(w[u] & 0xFFFF0000u);
      const uint32_t b = pow2 ? e4m3x2(f0 * inv, f1 * inv)
                              : e4m3x2(__fdiv_rn(f0, s), __fdiv_rn(f1, s));
      o[u >> 1] |= b << (16 * (u & 1));
    }
    reinterpret_cast<uint2*>(dst)[c] = make_uint2(o[0], o[1]);
  }
  if (tid == 0) *scale_at = s;
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t stream) {
  Params p{reinterpret_cast<const __nv_bfloat16*>(a.k), reinterpret_cast<const __nv_bfloat16*>(a.v),
           a.k_stride, a.v_stride, a.tokens, a.starts, a.c};
  const dim3 grid((unsigned)(a.tokens / kPage + 2 * a.c.requests), (unsigned)(2 * a.c.kv_heads));
  if (a.c.dim == 128)
    return launch_pdl(kv8_append_kernel<128>, grid, dim3(kThreads), 0, stream, 1u, p);
  return launch_pdl(kv8_append_kernel<64>, grid, dim3(kThreads), 0, stream, 1u, p);
}

}  // namespace dsmla
