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
// A CTA takes a (page of a request, side) and some heads, one after the other,
// or, where requests bring few tokens, a warp takes a (page, side, head):
// nothing is shared between them, so there is no atomic and no second pass. The
// tokens stay in registers between the maximum and the rounding. The bound is
// HBM, 2 bytes read and 1 written per element, and for few tokens the chain of
// lookups (request, length, page, scale).
//
// The grid covers an upper bound of the touched pages: n consecutive
// positions touch at most floor(n / 64) + 2 pages, so request r's pages are
// numbered from floor(starts[r] / 64) + 2 r and a search by 32 finds r.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv8.h"
#include "ptx.cuh"

namespace dsmla {

namespace {

constexpr int kThreads = 256;
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

// One touched page: where its new tokens come from and go to.
struct Unit {
  int64_t token0;     // token at slot 0 of the page (may be before the first)
  int64_t page;
  int had, upto;      // earlier positions; new ones are slots [had, upto)
};

// The page that unit number `unit` stands for; false if none. Called by whole
// warps: the request is found by probing 32 of them at a time.
__device__ __forceinline__ bool find_unit(const Params& p, int64_t unit, bool report, Unit* u) {
  const int lane = threadIdx.x & 31;
  auto start_of = [&](int64_t r) {
    const int64_t s = p.starts[r];
    return s < 0 ? 0 : (s > p.tokens ? p.tokens : s);
  };
  // The last request whose first unit is not past this one lies in
  // [lo, lo + size).
  int64_t lo = 0, size = p.c.requests;
  while (size > 1) {
    const int64_t step = (size + 31) / 32;
    const int64_t r = lo + lane * step;
    const bool at = r < lo + size && (start_of(r) >> 6) + 2 * r <= unit;
    const int n = __popc(__ballot_sync(0xffffffffu, at));   // monotone: the first n lanes
    const int64_t end = lo + size;
    lo += (n > 0 ? n - 1 : 0) * step;
    size = end - lo < step ? end - lo : step;
  }
  const int64_t t0 = start_of(lo), n = start_of(lo + 1) - t0;
  if (n <= 0) return false;
  const int64_t len = p.c.lens[lo], first = len - n;
  const int64_t j = unit - ((t0 >> 6) + 2 * lo);   // page of this request's touched ones
  if (first < 0) {
    if (j == 0 && report && p.c.err != nullptr) atomicOr(p.c.err, kErrLen);
    return false;
  }
  const int64_t block = (first >> 6) + j;
  if (j < 0 || (block << 6) >= len) return false;
  u->page = -1;
  if (block < p.c.bt_stride) u->page = p.c.block_table[lo * p.c.bt_stride + block];
  if (u->page < 0 || u->page >= p.c.num_pages) {
    if (report && p.c.err != nullptr) atomicOr(p.c.err, kErrPage);
    return false;
  }
  const int64_t pos0 = block << 6;
  u->token0 = t0 + (pos0 - first);
  u->had = first > pos0 ? (int)(first - pos0) : 0;
  u->upto = len - pos0 < kPage ? (int)(len - pos0) : kPage;
  return true;
}

__device__ __forceinline__ __nv_bfloat162 pair(uint32_t w) {
  return *reinterpret_cast<const __nv_bfloat162*>(&w);
}

// Largest magnitudes, two at a time (a NaN loses against any number).
struct Amax {
  __nv_bfloat162 m = pair(0u);
  __device__ __forceinline__ void add(uint4 x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) m = __hmax2(m, __habs2(pair(w[u])));
  }
  __device__ __forceinline__ float value() const {
    return fmaxf(__low2float(m), __high2float(m));
  }
};

__device__ __forceinline__ float warp_max(float a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

__device__ __forceinline__ float new_scale(float old, float a) {
  const float s = fmaxf(old, need_scale(a));
  return s > 0.0f ? s : __uint_as_float((uint32_t)(127 - 60) << 23);
}

// Eight values over the scale. Dividing by a power of two is multiplying by
// its reciprocal, exactly, also in bf16 (what falls below bf16's normal range
// rounds to a code of 0); a scale that a caller set to something else takes the
// division.
struct Quantizer {
  float s;
  __nv_bfloat162 inv;
  bool pow2;
  __device__ __forceinline__ explicit Quantizer(float scale) : s(scale) {
    const uint32_t b = __float_as_uint(scale);
    pow2 = (b & 0x7FFFFFu) == 0u && b >= (67u << 23) && b <= (247u << 23);
    const uint32_t h = ((254u << 23) - b) >> 16;
    inv = pair(pow2 ? h | (h << 16) : 0u);
  }
  __device__ __forceinline__ uint2 operator()(uint4 x) const {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (pow2) {
        const __nv_bfloat162 y = __hmul2(pair(w[u]), inv);
        b[u] = e4m3x2(__low2float(y), __high2float(y));
      } else {
        b[u] = e4m3x2(__fdiv_rn(__uint_as_float(w[u] << 16), s),
                      __fdiv_rn(__uint_as_float(w[u] & 0xFFFF0000u), s));
      }
    }
    return make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
  }
};

// Four earlier codes at a grown scale, f = old / new.
__device__ __forceinline__ uint32_t again(uint32_t w, float f) {
  uint32_t r = 0u;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((w >> (16 * u)) & 0xFFFFu), __NV_E4M3);
    const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&h));
    r |= e4m3x2(g.x * f, g.y * f) << (16 * u);
  }
  return r;
}

// One CTA per touched page, side and run of heads. A thread's 16-byte copies
// land in shared memory (two heads ahead, without holding registers) and are
// read back by the same thread, so only the maximum crosses threads. 8 prompts
// of 700 to 4001 tokens, 8 heads x 128: 23 us, 4.6 TB/s of 105 MB, issue slots
// 62 % busy. (A CTA per head with the loads in registers spent most of its time
// on the lookups: 30 us.)
template <int DIM>
__global__ void __launch_bounds__(kThreads) kv8_append_page_kernel(const Params p,
                                                                  const int heads_per_cta) {
  constexpr int kRowChunks = DIM / 8;                     // 16-byte chunks of a token's head
  constexpr int kSteps = kPage * kRowChunks / kThreads;   // chunks per thread
  constexpr int kStages = 3;
  extern __shared__ uint4 staged[];                       // [kStages][kSteps][kThreads]
  __shared__ float warp_top[2][kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int runs = (p.c.kv_heads + heads_per_cta - 1) / heads_per_cta;
  const int side = blockIdx.x & 1, run = (int)(blockIdx.x >> 1) % runs;
  const int64_t unit = (blockIdx.x >> 1) / runs;
  Unit u;
  if (!find_unit(p, unit, tid == 0 && side == 0 && run == 0, &u)) return;
  const int h0 = run * heads_per_cta, h1 = min(h0 + heads_per_cta, p.c.kv_heads);
  const int64_t part0 = (u.page * 2 + side) * p.c.kv_heads;
  const int64_t stride = side ? p.v_stride : p.k_stride;
  const __nv_bfloat16* src = (side ? p.v : p.k) + u.token0 * stride;
  auto fetch = [&](int h) {
    if (h < h1) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int c = tid + i * kThreads, slot = c / kRowChunks, ch = c % kRowChunks;
        if (slot >= u.had && slot < u.upto)
          cp_async_16(smem_u32(&staged[((h - h0) % kStages * kSteps + i) * kThreads + tid]),
                      src + slot * stride + h * DIM + ch * 8, 16);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(h0 + s);
  for (int h = h0; h < h1; ++h) {
    float* scale_at = p.c.scales + part0 + h;
    const float old = u.had > 0 ? *scale_at : 0.0f;
    fetch(h + kStages - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    uint4 x[kSteps];
    Amax amax;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int slot = (tid + i * kThreads) / kRowChunks;
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (slot >= u.had && slot < u.upto)
        x[i] = staged[((h - h0) % kStages * kSteps + i) * kThreads + tid];
      amax.add(x[i]);
    }
    float a = warp_max(amax.value());
    float* top = warp_top[h & 1];   // the last head's is still read by others
    if ((tid & 31) == 0) top[tid >> 5] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) a = fmaxf(a, top[w]);
    const float s = new_scale(old, a);
    uint8_t* dst = p.c.pages + (part0 + h) * (int64_t)(kPage * DIM);
    if (u.had > 0 && s != old) {
      const float f = __fdiv_rn(old, s);
      for (int c = tid; c < u.had * DIM / 4; c += kThreads) {
        uint32_t* at = reinterpret_cast<uint32_t*>(dst) + c;
        *at = again(*at, f);
      }
    }
    const Quantizer quant(s);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int c = tid + i * kThreads, slot = c / kRowChunks;
      if (slot >= u.had && slot < u.upto) reinterpret_cast<uint2*>(dst)[c] = quant(x[i]);
    }
    if (tid == 0) *scale_at = s;
  }
  cp_async_wait_all();
}

// The same with one warp per (page, side, head), for calls with few tokens a
// request: a CTA then finds its page once for eight of them, and there are an
// eighth of the CTAs.
template <int DIM>
__global__ void __launch_bounds__(256) kv8_append_few_kernel(const Params p) {
  constexpr int kRowChunks = DIM / 8;
  constexpr int kHeld = 4;            // chunks a lane keeps in registers
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int parts = 2 * p.c.kv_heads, per_unit = (parts + 7) / 8;
  const int64_t unit = blockIdx.x / per_unit;
  const int ph = (int)(blockIdx.x % per_unit) * 8 + (threadIdx.x >> 5);   // side, head
  if (ph >= parts) return;
  Unit u;
  if (!find_unit(p, unit, lane == 0 && ph == 0, &u)) return;
  const int side = ph / p.c.kv_heads, head = ph % p.c.kv_heads;
  const int64_t part = (u.page * 2 + side) * p.c.kv_heads + head;
  float* scale_at = p.c.scales + part;
  const float old = u.had > 0 ? *scale_at : 0.0f;
  const int64_t stride = side ? p.v_stride : p.k_stride;
  const __nv_bfloat16* src = (side ? p.v : p.k) + u.token0 * stride + head * DIM;
  const int c0 = u.had * kRowChunks, c1 = u.upto * kRowChunks;
  auto at = [&](int c) {
    return *reinterpret_cast<const uint4*>(src + (c / kRowChunks) * stride + (c % kRowChunks) * 8);
  };
  uint4 x[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = c0 + lane + 32 * i;
    x[i] = c < c1 ? at(c) : make_uint4(0u, 0u, 0u, 0u);
  }
  Amax amax;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) amax.add(x[i]);
  for (int c = c0 + lane + 32 * kHeld; c < c1; c += 32) amax.add(at(c));
  const float s = new_scale(old, warp_max(amax.value()));
  uint8_t* dst = p.c.pages + part * (int64_t)(kPage * DIM);
  if (u.had > 0 && s != old) {
    const float f = __fdiv_rn(old, s);
    for (int c = lane; c < u.had * DIM / 4; c += 32) {
      uint32_t* w = reinterpret_cast<uint32_t*>(dst) + c;
      *w = again(*w, f);
    }
  }
  const Quantizer quant(s);
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = c0 + lane + 32 * i;
    if (c < c1) reinterpret_cast<uint2*>(dst)[c] = quant(x[i]);
  }
  for (int c = c0 + lane + 32 * kHeld; c < c1; c += 32) reinterpret_cast<uint2*>(dst)[c] = quant(at(c));
  __syncwarp();   // every lane has read the old scale
  if (lane == 0) *scale_at = s;
}

template <int DIM>
cudaError_t launch_pages(const Params& p, dim3 grid, int heads_per_cta, cudaStream_t stream) {
  constexpr int kSmem = 3 * kPage * DIM * 2;
  static PerDeviceOnce once;
  int dev = 0;
  cudaError_t e = stream_device(stream, &dev);
  if (e == cudaSuccess) e = set_max_dynamic_smem(once, dev, kv8_append_page_kernel<DIM>, kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv8_append_page_kernel<DIM>, grid, dim3(kThreads), kSmem, stream, 1u, p,
                    heads_per_cta);
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t stream) {
  Params p{reinterpret_cast<const __nv_bfloat16*>(a.k), reinterpret_cast<const __nv_bfloat16*>(a.v),
           a.k_stride, a.v_stride, a.tokens, a.starts, a.c};
  // Few tokens a request (on average): a warp per (page, side, head). us of this
  // kernel against the other one:
  //   requests x tokens   128 x 5   128 x 32   128 x 64   16 x 8   16 x 24
  //   8 heads x 128       4.5 12.5  10.8 15.2  18.2 17.9  3.1 3.9  5.2 4.1
  //   8 heads x 64        4.2 11.3  6.8 14.6   11.1 15.9  2.8 4.4  3.8 4.4
  //   4 heads x 128       3.4 7.7   9.1 9.4    15.9 10.9  3.0 2.8  5.6 3.0
  //   1 head x 128        3.1 4.2   6.6 4.9    10.1 5.9   2.8 2.7  4.7 2.8
  // so up to 40 tokens, or 16 where few CTAs of the other one wait for a place. (At
  // the limits the slower side may be taken: 128 x 40 of 4 heads x 128 11.3 for
  // 9.8, 16 x 16 of 1 head 3.8 for 2.8. One long prompt among many short ones goes
  // with them, since the lengths are on the device.)
  const int64_t units = a.tokens / kPage + 2 * a.c.requests;
  if (a.tokens <= (a.c.requests * a.c.kv_heads >= 512 ? 40 : 16) * a.c.requests) {
    const dim3 grid((unsigned)(units * ((2 * a.c.kv_heads + 7) / 8)));
    if (a.c.dim == 128)
      return launch_pdl(kv8_append_few_kernel<128>, grid, dim3(256), 0, stream, 1u, p);
    return launch_pdl(kv8_append_few_kernel<64>, grid, dim3(256), 0, stream, 1u, p);
  }
  // Heads per CTA: all CTAs resident at once, four per SM, where that is less
  // than all heads.
  const int64_t items = units * 2 * a.c.kv_heads;
  int64_t per = (items + 152 * 4 - 1) / (152 * 4);
  if (per > a.c.kv_heads) per = a.c.kv_heads;
  const int64_t runs = (a.c.kv_heads + per - 1) / per;
  const dim3 grid((unsigned)(units * 2 * runs));
  return a.c.dim == 128 ? launch_pages<128>(p, grid, (int)per, stream)
                        : launch_pages<64>(p, grid, (int)per, stream);
}

}  // namespace dsmla
