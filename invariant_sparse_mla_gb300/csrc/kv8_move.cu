// Positions of a request moved to the front of its pages: the accepted ones of a
// tree of drafts (kv8_accept) and those that an eviction keeps (kv8_evict).
//
// A page that gets positions from several pages takes the largest of their
// scales, so that no code leaves the range; a code whose page had a smaller one
// becomes E4M3(code * (old / scale)), all others are copied as they are.
//
// Moving in place is safe without a second copy of the cache because kept
// positions keep their order: the i-th of them comes from position i or behind.
// What is written in one go (a chunk of rows in accept, a round of pages in
// evict) is read before that, and nothing that is read later lies in front of it.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv8.h"
#include "kv8_common.cuh"

namespace dsmla {

namespace {

constexpr int kErrIdx = DS_DEVERR_IDX, kErrPage = DS_DEVERR_PAGE, kErrLen = DS_DEVERR_LEN,
              kErrShared = DS_DEVERR_SHARED;

__device__ __forceinline__ void raise(int32_t* err, int bit) {
  if (err != nullptr) atomicOr(err, bit);
}

// Four codes under a scale 1 / ratio times their own.
__device__ __forceinline__ uint32_t requantise4(uint32_t w, float ratio) {
  const uint2 h = codes_to_f16(w);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h.y));
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a.x * ratio, a.y * ratio),
                                               __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(b.x * ratio, b.y * ratio),
                                               __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ uint4 requantise(uint4 v, float ratio) {
  if (ratio == 1.0f) return v;
  return make_uint4(requantise4(v.x, ratio), requantise4(v.y, ratio), requantise4(v.z, ratio),
                    requantise4(v.w, ratio));
}

// What codes under scale s are times under `top`. (Equal scales change nothing,
// whatever they are: 0 or an infinity has no quotient.)
__device__ __forceinline__ float ratio_of(float s, float top) {
  return s == top ? 1.0f : __fdiv_rn(s, top);
}

// ------------------------------------------------------------------ accept
constexpr int kAcceptWarps = 8;
constexpr int kFewLayers = 16;

template <int MAX>
struct Layers {
  int n;
  uint8_t* pages[MAX];
  float* scales[MAX];
};

// A warp per (request, layer, side, head): all of them read the request's list
// and come to the same decision, and nothing is shared between them. Bound by its
// dependent reads (list, table, scales, codes): 4.7 us for 4 requests of 2 layers, 12
// for 128 requests x 6 layers x 8 heads x 128 with up to 16 drafts accepted of 64 (10 MB).
template <int DIM, int MAX>
__global__ void __launch_bounds__(32 * kAcceptWarps) kv8_accept_kernel(
    const __grid_constant__ Layers<MAX> layers, const Kv8AcceptArgs a) {
  constexpr int L = DIM / 16;          // lanes of a row
  constexpr int ROWS = 32 / L;         // rows a warp takes at a time
  constexpr int CHUNK = 16;            // rows read before any is written
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kAcceptWarps + (threadIdx.x >> 5);
  const int per = layers.n * 2 * a.c.kv_heads;
  const int64_t r = unit / per;
  pdl_wait();
  pdl_trigger();
  if (r >= a.c.requests) return;
  const int part = (int)(unit % per);
  const bool first_part = part == 0;
  const int len = a.c.lens[r];
  // The list, two entries a lane: ascending node numbers, -1 behind them.
  const int32_t* list = a.accepted + r * a.width;
  const int n0 = lane < a.width ? list[lane] : -1;
  const int n1 = lane + 32 < a.width ? list[lane + 32] : -1;
  const uint32_t in0 = __ballot_sync(0xffffffffu, n0 >= 0);
  const uint32_t in1 = __ballot_sync(0xffffffffu, n1 >= 0);
  const uint64_t in = (uint64_t)in1 << 32 | in0;
  const int count = in == ~0ull ? 64 : __ffsll((long long)~in) - 1;
  auto node = [&](int j) {             // (all lanes call it)
    const int x = __shfl_sync(0xffffffffu, n0, j & 31), y = __shfl_sync(0xffffffffu, n1, j & 31);
    return j < 32 ? x : y;
  };
  if (len <= 0) {                      // a padded request holds nothing
    if (first_part && lane == 0) a.new_lens[r] = len;
    return;
  }
  const int64_t base = (int64_t)len - a.next_n;
  int bad = 0;
  if (base < 0 || len > a.c.bt_stride * kPage) bad = kErrLen;
  // Ascending, within the drafts, and nothing behind the first -1.
  const int p0 = __shfl_up_sync(0xffffffffu, n0, 1), p1 = __shfl_up_sync(0xffffffffu, n1, 1);
  const int last0 = __shfl_sync(0xffffffffu, n0, 31);
  bool wrong = n0 >= a.next_n || n1 >= a.next_n || (count < 64 && (in >> count) != 0);
  if (lane > 0 && lane < count && n0 <= p0) wrong = true;
  if (lane + 32 < count && n1 <= (lane > 0 ? p1 : last0)) wrong = true;
  if (__any_sync(0xffffffffu, wrong)) bad |= kErrIdx;
  const int64_t block = base >> 6;
  const int off = (int)(base & 63);
  int64_t page[2] = {0, 0};
  const int last = count > 0 ? node(count - 1) : 0;
  const bool second = count > 0 && off + last >= kPage;
  if (bad == 0 && count > 0) {
    page[0] = a.c.block_table[r * a.c.bt_stride + block];
    page[1] = second ? a.c.block_table[r * a.c.bt_stride + block + 1] : page[0];
    for (int i = 0; i < 2; ++i)
      if (page[i] < 0 || page[i] >= a.c.num_pages) bad = kErrPage;
  }
  if (first_part && lane == 0) {
    a.new_lens[r] = bad ? len : (int)(base + count);
    if (bad) raise(a.c.err, bad);
  }
  if (bad || count == 0) return;

  const int layer = part / (2 * a.c.kv_heads);
  const int sh = part % (2 * a.c.kv_heads);          // side * heads + head
  const int64_t t0 = page[0] * 2 * a.c.kv_heads + sh, t1 = page[1] * 2 * a.c.kv_heads + sh;
  float* scales = layers.scales[layer];
  uint8_t* const at0 = layers.pages[layer] + t0 * (kPage * DIM);
  uint8_t* const at1 = layers.pages[layer] + t1 * (kPage * DIM);
  const float s0 = scales[t0], s1 = scales[t1];
  // Scales of both pages afterwards: that of the second one stays, as what
  // comes to it was there.
  auto low = [&](int j, int n) { return off + j < kPage && off + n < kPage; };
  const bool from0 = __any_sync(0xffffffffu, (lane < count && low(lane, n0)) ||
                                                 (lane + 32 < count && low(lane + 32, n1)));
  auto cross = [&](int j, int n) { return off + j < kPage && off + n >= kPage; };
  const bool from1 = __any_sync(0xffffffffu, (lane < count && cross(lane, n0)) ||
                                                 (lane + 32 < count && cross(lane + 32, n1)));
  float top = off > 0 || from0 ? s0 : s1;
  if (from1) top = fmaxf(top, s1);
  const float ratio0 = ratio_of(s0, top), ratio1 = ratio_of(s1, top);
  const int col = lane % L;
  for (int j0 = 0; j0 < count; j0 += CHUNK) {
    uint4 v[CHUNK / ROWS];
#pragma unroll
    for (int i = 0; i < CHUNK / ROWS; ++i) {
      const int j = j0 + i * ROWS + lane / L;
      const int n = node(j & 63);
      if (j < count && (n != j || (off + n < kPage && ratio0 != 1.0f))) {
        const int s = off + n;
        v[i] = reinterpret_cast<const uint4*>((s < kPage ? at0 : at1) + (s & 63) * DIM)[col];
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < CHUNK / ROWS; ++i) {
      const int j = j0 + i * ROWS + lane / L;
      const int n = node(j & 63);
      if (j < count && (n != j || (off + n < kPage && ratio0 != 1.0f))) {
        const int s = off + n, d = off + j;
        if (d < kPage) v[i] = requantise(v[i], s < kPage ? ratio0 : ratio1);
        reinterpret_cast<uint4*>((d < kPage ? at0 : at1) + (d & 63) * DIM)[col] = v[i];
      }
    }
    __syncwarp();
  }
  if (top != s0) {
    // The page's earlier positions under the new scale.
    if (ratio0 != 1.0f)
      for (int i = lane; i < off * L; i += 32) {
        uint4* x = reinterpret_cast<uint4*>(at0) + i;
        *x = requantise(*x, ratio0);
      }
    if (lane == 0) scales[t0] = top;
  }
}

// ------------------------------------------------------------------- evict
constexpr int kPlanThreads = 256;
constexpr int kMoveThreads = 256;
constexpr int kCluster = 8;            // CTAs of one (request, head, side)
constexpr int kRound = 4;              // pages that a CTA reads before it writes any
constexpr int kBlock = 8;              // pages that it looks up at once

// Which requests are cut, their new lengths, and the range that is ranked.
__global__ void __launch_bounds__(kPlanThreads) kv8_evict_plan_kernel(const Kv8EvictArgs a) {
  const int64_t r = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  const int len = a.c.lens[r];
  int bad = 0;
  if (len > a.budget) {
    if (len > a.c.bt_stride * kPage || len > a.mass_stride) {
      bad = kErrLen;
    } else {
      const int blocks = (len + kPage - 1) / kPage, written = (a.budget + kPage - 1) / kPage;
      for (int b = threadIdx.x; b < blocks; b += kPlanThreads) {
        const int64_t page = a.c.block_table[r * a.c.bt_stride + b];
        if (page < 0 || page >= a.c.num_pages)
          bad |= kErrPage;
        else if (a.refcounts != nullptr && b < written && a.refcounts[page] > 1)
          bad |= kErrShared;
      }
    }
  }
  const bool any_page = __syncthreads_or(bad & kErrPage);
  const bool any_shared = __syncthreads_or(bad & kErrShared);
  const bool cut = len > a.budget && !any_page && !any_shared && bad == 0;
  if (threadIdx.x == 0) {
    const int bits = (any_page ? kErrPage : 0) | (any_shared ? kErrShared : 0) | (bad & kErrLen);
    if (bits) raise(a.c.err, bits);
    a.new_lens[r] = cut ? a.budget : len;
  }
  for (int g = threadIdx.x; g < a.c.kv_heads; g += kPlanThreads) {
    a.starts[r * a.c.kv_heads + g] = cut ? a.first : 0;
    a.ends[r * a.c.kv_heads + g] = cut ? len - a.recent : 0;
  }
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// A cluster per (request, head, side) takes the pages of the budget in turn, a block
// of kCluster * kBlock at a time: where the positions come from, their scales and
// masses are looked up first (three dependent loads, once for the block), then
// the codes follow in rounds: all CTAs read what goes to their pages of the round, wait
// for one another, and write. 32 requests of 4096 to 32768 positions, 8 heads x 128,
// held to 4096: 135 us in all (561 MB; 83 at the rate of a plain copy), of which the
// moves take about 100, the ranking 27 and the plan 6.5. With one page a round and its
// lookups each time it was 196: rows of 128 bytes scattered over the pool come at
// about 5 TB/s, and a round waits for the slowest CTA of eight. The same requests with
// 1, 64 or 512 positions past the budget take 118, 128 or 132 us: all that lies behind the
// first dropped position moves up (20 us where nothing is past it).
template <int DIM>
__global__ void __launch_bounds__(kMoveThreads) kv8_evict_move_kernel(const Kv8EvictArgs a) {
  constexpr int L = DIM / 16;                     // lanes of a row
  constexpr int ROWS = kMoveThreads / L;          // rows of a pass
  constexpr int PASSES = kPage / ROWS;            // of a page
  constexpr int E = kBlock * kPage / kMoveThreads;   // places a thread looks up
  __shared__ int from[kBlock * kPage];            // row of the pool's codes, or -1
  __shared__ float scale[kBlock * kPage];
  __shared__ float weight[kBlock * kPage];        // side 0: mass
  __shared__ float warp_top[kBlock * 2];          // largest scale of half a page
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = blockIdx.x % kCluster;
  const int64_t unit = blockIdx.x / kCluster;
  const int side = (int)(unit & 1);
  const int64_t rg = unit >> 1, r = rg / a.c.kv_heads;
  const int g = (int)(rg % a.c.kv_heads);
  pdl_wait();
  pdl_trigger();
  const int len = a.c.lens[r];
  if (len <= a.budget || a.new_lens[r] != a.budget) return;   // the whole cluster
  const int k = a.budget - a.first - a.recent;
  const int32_t* top_idx = a.top + rg * k;
  const int32_t* table = a.c.block_table + r * a.c.bt_stride;
  float* mass = a.mass + rg * a.mass_stride;
  const int blocks = (a.budget + kPage - 1) / kPage;
  // The position that comes to place j.
  auto source = [&](int j) {
    if (j < a.first) return j;
    if (j >= a.first + k) return len - a.budget + j;
    return a.first + top_idx[j - a.first];
  };
  auto part = [&](int64_t page) { return (page * 2 + side) * a.c.kv_heads + g; };
  const int col = tid % L, row0 = tid / L;
  for (int b0 = 0; b0 < blocks; b0 += kCluster * kBlock) {
    // Page i of the block that this CTA writes is b0 + i * kCluster + rank.
    __syncthreads();               // the block before is written
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int at = tid + e * kMoveThreads;
      const int j = (b0 + at / kPage * kCluster + rank) * kPage + at % kPage;
      int row = -1;
      float s = 0.0f;
      if (j < a.budget) {
        const int p = source(j);
        const int64_t t = part(table[p >> 6]);
        row = (int)t * kPage + (p & 63);   // (below 2^31: the pool's rows are)
        s = a.c.scales[t];
        if (side == 0) weight[at] = mass[p];
      }
      from[at] = row;
      scale[at] = s;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, o));
      if (lane == 0) warp_top[at / 32] = s;
    }
    __syncthreads();
#pragma unroll 1
    for (int i0 = 0; i0 < kBlock; i0 += kRound) {
      // (The same for all CTAs of the cluster.)
      if (b0 + i0 * kCluster >= blocks) break;
      uint4 v[kRound][PASSES];
#pragma unroll
      for (int i = 0; i < kRound; ++i)
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
          const int row = from[(i0 + i) * kPage + q * ROWS + row0];
          if (row >= 0) v[i][q] = reinterpret_cast<const uint4*>(a.c.pages + (int64_t)row * DIM)[col];
        }
      cluster_arrive();
      cluster_wait();
#pragma unroll
      for (int i = 0; i < kRound; ++i) {
        const int b = b0 + (i0 + i) * kCluster + rank;
        if (b >= blocks) continue;
        const float top = fmaxf(warp_top[2 * (i0 + i)], warp_top[2 * (i0 + i) + 1]);
        const int64_t t = part(table[b]);
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
          const int slot = q * ROWS + row0, at = (i0 + i) * kPage + slot;
          const int to = (int)t * kPage + slot;
          if (from[at] < 0) continue;
          const float ratio = ratio_of(scale[at], top);
          if (from[at] != to || ratio != 1.0f)
            reinterpret_cast<uint4*>(a.c.pages + (int64_t)to * DIM)[col] = requantise(v[i][q], ratio);
          if (side == 0 && col == 0 && from[at] != to) mass[b * kPage + slot] = weight[at];
        }
        if (tid == 0) a.c.scales[t] = top;
      }
    }
  }
}

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

template <int MAX>
cudaError_t run_accept(const ds_kv8_layer* layers, int n, const Kv8AcceptArgs& a,
                       cudaStream_t stream) {
  Layers<MAX> l;
  l.n = n;
  for (int i = 0; i < n; ++i) {
    l.pages[i] = static_cast<uint8_t*>(layers[i].kv_pages);
    l.scales[i] = layers[i].kv_scales;
  }
  const int64_t units = a.c.requests * n * 2 * a.c.kv_heads;
  const dim3 grid((unsigned)((units + kAcceptWarps - 1) / kAcceptWarps));
  return a.c.dim == 128 ? launch_pdl(kv8_accept_kernel<128, MAX>, grid, dim3(32 * kAcceptWarps), 0,
                                     stream, 1u, l, a)
                        : launch_pdl(kv8_accept_kernel<64, MAX>, grid, dim3(32 * kAcceptWarps), 0,
                                     stream, 1u, l, a);
}

struct EvictWorkspace {
  int32_t *starts, *ends, *top;
  size_t bytes;
};

EvictWorkspace carve(void* base, int64_t rows, int k) {
  EvictWorkspace w;
  uint8_t* p = static_cast<uint8_t*>(base);
  size_t at = 0;
  auto take = [&](size_t n) {
    uint8_t* x = p ? p + at : nullptr;
    at += pad256(n);
    return x;
  };
  w.starts = reinterpret_cast<int32_t*>(take((size_t)rows * 4));
  w.ends = reinterpret_cast<int32_t*>(take((size_t)rows * 4));
  w.top = reinterpret_cast<int32_t*>(take((size_t)rows * k * 4));
  w.bytes = at + 256;
  return w;
}

}  // namespace

cudaError_t launch_kv8_accept(const ds_kv8_layer* layers, int n, const Kv8AcceptArgs& a,
                              cudaStream_t stream) {
  return n <= kFewLayers ? run_accept<kFewLayers>(layers, n, a, stream)
                         : run_accept<DS_MAX_KV8_LAYERS>(layers, n, a, stream);
}

size_t kv8_evict_workspace_bytes(int64_t requests, int kv_heads, int k) {
  return carve(nullptr, requests * kv_heads, k).bytes;
}

cudaError_t launch_kv8_evict(Kv8EvictArgs a, void* workspace, cudaStream_t stream) {
  const int64_t rows = a.c.requests * a.c.kv_heads;
  const int k = a.budget - a.first - a.recent;
  const EvictWorkspace w = carve(workspace, rows, k);
  a.starts = w.starts;
  a.ends = w.ends;
  a.top = w.top;
  cudaError_t e = launch_pdl(kv8_evict_plan_kernel, dim3((unsigned)a.c.requests),
                             dim3(kPlanThreads), 0, stream, 1u, a);
  if (e != cudaSuccess) return e;
  if (k > 0) {
    // Without the grid kernel's workspace: over rows of mass it took 19 us where the
    // cluster kernel takes 7 (8 rows of 2048), 41 and 15 (8 of 131072), 60 and 45 (64 of
    // 131072), and 70 and 80 with 128 rows, for 143 MB of it.
    e = launch_topk(a.mass, a.mass_stride, rows, w.starts, w.ends, k, w.top, nullptr, 0, stream);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((unsigned)(rows * 2 * kCluster));
  return a.c.dim == 128
             ? launch_pdl(kv8_evict_move_kernel<128>, grid, dim3(kMoveThreads), 0, stream,
                          (unsigned)kCluster, a)
             : launch_pdl(kv8_evict_move_kernel<64>, grid, dim3(kMoveThreads), 0, stream,
                          (unsigned)kCluster, a);
}

}  // namespace dsmla
