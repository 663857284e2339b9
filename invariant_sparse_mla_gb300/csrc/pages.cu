// Pages of a paged cache: copying, forking, freeing, extending, compacting.
//
// A page is free when its reference count is not positive, and free pages are
// handed out lowest number first: what a call does follows from the state
// before it alone, with no free list whose order would depend on the order
// of atomics. (Counts change by integer atomics, whose order does not show.)
//
// To find the i-th free page without a serial scan, one launch writes a
// bitmap of the live pages and the number of free ones in each segment of
// 1024 pages; the next launch locates rank i by a prefix over the segment
// counts and a walk over the segment's 32 words. The bitmap is a snapshot:
// the second launch changes counts while it reads the bitmap, so no CTA sees
// another's half-done work.
//
// The table work is a few thousand integers, bound by launches and memory
// latency; page payloads are bound by HBM (each byte read and written once)
// and are cut into 16 KB pieces so that every SM takes part however few pages
// move. Copying 366 MB takes 56.0 us and compacting a pool by moving 3 GB 473
// us (6.5 and 6.4 TB/s counting reads and writes); freeing, forking and
// extending 96 of 256 rows, 98 MB copied, takes 40 us (the forking kernel 21 of
// them, five launches most of the rest). Fork and extend look for an entry's
// rank and page in every CTA and for repeats in every entry: made for lists of
// dozens or hundreds, right for 65535 (extending as many rows takes 1.7 ms,
// forking them 2.6).

#include <cuda_runtime.h>
#include <stdint.h>

#include "kv8.h"

namespace dsmla {

namespace {

constexpr int kSeg = 1024;            // pages per segment
constexpr int kSegWords = kSeg / 32;
constexpr int kMaxSegs = 4096;        // 2^22 pages
constexpr int kThreads = 256;
constexpr int kPiece = 16384;         // payload bytes per CTA
constexpr int kErrPage = DS_DEVERR_PAGE, kErrRow = DS_DEVERR_ROWREQ,
              kErrNoPage = DS_DEVERR_NOPAGE, kErrLen = DS_DEVERR_LEN;

// Passed by value: a call with few pools (up to 16) launches with a tenth of
// the parameter bytes of one with many (a fork and a free, 2 pools: 19.4 us on
// the host, 20.2 with the many's parameters).
constexpr int kFewPools = 16;
template <int MAX>
struct Pools {
  int n;
  int pieces;                         // over all pools, for one page
  uint8_t* data[MAX];
  int64_t bytes[MAX];                 // of a page
  int first[MAX + 1];                 // first piece of each pool
};

template <int MAX>
Pools<MAX> make_pools(const ds_page_pool* pools, int n) {
  Pools<MAX> r;
  r.n = n;
  r.first[0] = 0;
  for (int i = 0; i < n; ++i) {
    r.data[i] = static_cast<uint8_t*>(pools[i].data);
    r.bytes[i] = pools[i].page_bytes;
    r.first[i + 1] = r.first[i] + (int)((pools[i].page_bytes + kPiece - 1) / kPiece);
  }
  r.pieces = r.first[n];
  return r;
}

// Workspace: the live bitmap, free pages per segment, then (fork, extend) two
// ints per list entry or (compact) the live rank at each word, and the lists
// of holes and of moved pages.
struct Workspace {
  uint32_t* live;        // [segs * 32]
  int32_t* seg_free;     // [segs]
  int32_t* need;         // [n]
  int32_t* aux;          // [n]
  int32_t* word_rank;    // [segs * 32] live pages before the word
  int32_t* holes;        // [num_pages / 2 + 1]
  int32_t* moved;        // [num_pages / 2 + 1]
  int32_t* totals;       // {num_live, number moved}
};

int num_segs(int64_t pages) { return (int)((pages + kSeg - 1) / kSeg); }

size_t carve(Workspace* w, void* base, int64_t pages, int64_t n) {
  size_t at = 0;
  const int segs = num_segs(pages);
  auto take = [&](size_t count) {
    int32_t* p = base ? reinterpret_cast<int32_t*>(static_cast<uint8_t*>(base) + at) : nullptr;
    at += (count * 4 + 255) / 256 * 256;
    return p;
  };
  Workspace r;
  r.live = reinterpret_cast<uint32_t*>(take((size_t)segs * kSegWords));
  r.seg_free = take(segs);
  r.need = take(n);
  r.aux = take(n);
  r.word_rank = take((size_t)segs * kSegWords);
  r.holes = take(pages / 2 + 1);
  r.moved = take(pages / 2 + 1);
  r.totals = take(2);
  if (w) *w = r;
  return at;
}

__device__ __forceinline__ void raise(int32_t* err, int bit) {
  if (err != nullptr) atomicOr(err, bit);
}

__device__ __forceinline__ int64_t clamp_len(int64_t len, int64_t bt_stride) {
  return len < 0 ? 0 : (len > bt_stride * kPage ? bt_stride * kPage : len);
}

// Sum over the block (all threads get it). `sh` holds kThreads / 32 values.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  T s = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += sh[i];
  return s;
}

// Piece `piece` of one page's payload, from page src to page dst. 16-byte
// vectors where the pool's base and page size allow it, else 4-byte words.
template <int MAX>
__device__ __forceinline__ void copy_piece(const Pools<MAX>& pools, int piece, int64_t src,
                                           int64_t dst) {
  int lo = 0, hi = pools.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pools.first[mid] <= piece)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int64_t bytes = pools.bytes[lo];
  const int64_t off = (int64_t)(piece - pools.first[lo]) * kPiece;
  const int n = bytes - off < kPiece ? (int)(bytes - off) : kPiece;
  const uint8_t* s = pools.data[lo] + src * bytes + off;
  uint8_t* d = pools.data[lo] + dst * bytes + off;
  if (((reinterpret_cast<uintptr_t>(pools.data[lo]) | (uintptr_t)bytes) & 15u) == 0u) {
    // 16384 / 16 / 256 = 4 vectors per thread, all loads before the stores.
    uint4 v[kPiece / 16 / kThreads];
#pragma unroll
    for (int i = 0; i < kPiece / 16 / kThreads; ++i) {
      const int c = threadIdx.x + i * kThreads;
      if (c < n / 16) v[i] = reinterpret_cast<const uint4*>(s)[c];
    }
#pragma unroll
    for (int i = 0; i < kPiece / 16 / kThreads; ++i) {
      const int c = threadIdx.x + i * kThreads;
      if (c < n / 16) reinterpret_cast<uint4*>(d)[c] = v[i];
    }
  } else {
    for (int c = threadIdx.x; c < n / 4; c += kThreads)
      reinterpret_cast<uint32_t*>(d)[c] = reinterpret_cast<const uint32_t*>(s)[c];
  }
}

// ------------------------------------------------------------------- copy
template <int MAX>
__global__ void __launch_bounds__(kThreads) pages_copy_kernel(
    const __grid_constant__ Pools<MAX> pools, int64_t num_pages, const int32_t* __restrict__ src,
    const int32_t* __restrict__ dst, int32_t* err) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = blockIdx.x / pools.pieces;
  const int piece = (int)(blockIdx.x % pools.pieces);
  const int64_t s = src[i], d = dst[i];
  if (s < 0 || d < 0) return;
  if (s >= num_pages || d >= num_pages) {
    if (piece == 0 && threadIdx.x == 0) raise(err, kErrPage);
    return;
  }
  copy_piece(pools, piece, s, d);
}

// ------------------------------------------------------------------- free
__global__ void __launch_bounds__(kThreads) pages_free_kernel(const PageState s,
                                                             const int32_t* __restrict__ rows) {
  pdl_wait();
  pdl_trigger();
  const int64_t r = rows[blockIdx.x];
  if (r < 0) return;
  if (r >= s.num_rows) {
    if (threadIdx.x == 0) raise(s.err, kErrRow);
    return;
  }
  const int64_t held = (clamp_len(s.lens[r], s.bt_stride) + kPage - 1) / kPage;
  __syncthreads();   // every thread has read the length
  // An exchange takes each entry once, also when the row is listed twice.
  for (int64_t j = threadIdx.x; j < held; j += kThreads) {
    const int page = atomicExch(&s.table[r * s.bt_stride + j], -1);
    if (page == -1) continue;
    if (page < 0 || page >= s.num_pages) {
      raise(s.err, kErrPage);
      continue;
    }
    if (atomicSub(&s.refs[page], 1) <= 0) {
      atomicAdd(&s.refs[page], 1);
      raise(s.err, kErrPage);
    }
  }
  if (threadIdx.x == 0) s.lens[r] = 0;
}

// ---------------------------------------------------- snapshot (all others)
// Block b < segs: the live bitmap and the free count of segment b.
__device__ __forceinline__ void snapshot_segment(const PageState& s, const Workspace& w, int seg,
                                                 int* sh) {
  const int tid = threadIdx.x;
  int free_here = 0;
#pragma unroll
  for (int i = 0; i < kSeg / kThreads; ++i) {
    const int64_t page = (int64_t)seg * kSeg + i * kThreads + tid;
    const bool in = page < s.num_pages;
    const bool live = in && s.refs[page] > 0;
    const uint32_t b = __ballot_sync(0xffffffffu, live || !in);   // past the pool: never free
    const uint32_t lv = __ballot_sync(0xffffffffu, live);
    if ((tid & 31) == 0) {
      w.live[seg * kSegWords + i * (kThreads / 32) + (tid >> 5)] = lv;
      free_here += 32 - __popc(b);
    }
  }
  const int total = block_sum(free_here, sh);
  if (tid == 0) w.seg_free[seg] = total;
}

// Free ranks over the segments: sh[i] = free pages before segment i.
__device__ __forceinline__ int scan_segments(const Workspace& w, int segs, int* sh, int* tmp) {
  // Each thread sums a run of segments, then the runs are scanned.
  const int tid = threadIdx.x;
  const int per = (segs + kThreads - 1) / kThreads;
  __syncthreads();   // tmp may still be read
  int sum = 0;
  for (int i = tid * per; i < segs && i < (tid + 1) * per; ++i) sum += w.seg_free[i];
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if ((tid & 31) >= o) inc += v;
  }
  if ((tid & 31) == 31) tmp[tid >> 5] = inc;
  __syncthreads();
  int before = inc - sum, total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < (tid >> 5)) before += tmp[i];
    total += tmp[i];
  }
  for (int i = tid * per; i < segs && i < (tid + 1) * per; ++i) {
    sh[i] = before;
    before += w.seg_free[i];
  }
  __syncthreads();
  return total;
}

// The page with free rank `rank` (< total), from sh as scan_segments left it.
__device__ __forceinline__ int select_free(const Workspace& w, int64_t num_pages, int segs,
                                           const int* sh, int rank) {
  int lo = 0, hi = segs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sh[mid] <= rank)
      lo = mid;
    else
      hi = mid - 1;
  }
  int left = rank - sh[lo];
  for (int i = 0; i < kSegWords; ++i) {
    const int64_t base = (int64_t)lo * kSeg + i * 32;
    uint32_t f = ~w.live[lo * kSegWords + i];
    if (base + 32 > num_pages) f &= base >= num_pages ? 0u : (1u << (num_pages - base)) - 1u;
    const int c = __popc(f);
    if (left < c) {
      for (; left > 0; --left) f &= f - 1;
      return (int)base + __ffs(f) - 1;
    }
    left -= c;
  }
  return -1;   // not reached: rank < total
}

// Sum of need[0 .. i): 64 bits, since a list may ask for more than there is.
__device__ __forceinline__ int64_t need_before(const Workspace& w, int64_t i) {
  __shared__ long long tmp[kThreads / 32];
  long long v = 0;
  for (int64_t j = threadIdx.x; j < i; j += kThreads) v += w.need[j];
  return block_sum(v, tmp);
}

// Fork: need = 1 where a partly filled page is copied (one outside the pool is
// not), aux = the parent's length, -1 for an entry that is skipped. Extend: need
// = pages to add, aux = the present length or -1. Everything is read before
// anything is written.
template <bool FORK>
__global__ void __launch_bounds__(kThreads) pages_plan_kernel(
    const PageState s, const Workspace w, int segs, const int32_t* __restrict__ a,
    const int32_t* __restrict__ b, int64_t n) {
  __shared__ int tmp[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x < segs) {
    snapshot_segment(s, w, blockIdx.x, tmp);
    return;
  }
  const int64_t i = (int64_t)(blockIdx.x - segs) * kThreads + threadIdx.x;
  if (i >= n) return;
  int need = 0;
  int64_t aux = -1;
  const int32_t* rows = FORK ? b : a;   // the rows that change
  const int64_t row = rows[i];
  bool ok = row >= 0 && (!FORK || a[i] >= 0);
  if (ok && (row >= s.num_rows || (FORK && a[i] >= s.num_rows))) {
    raise(s.err, kErrRow);
    ok = false;
  }
  if (ok) {
    bool again = false;
    for (int64_t j = 0; j < i; ++j) again |= rows[j] == (int32_t)row && (!FORK || a[j] >= 0);
    if (again || (FORK && s.lens[row] > 0)) {
      raise(s.err, kErrRow);
      ok = false;
    }
  }
  if (ok && FORK) {
    aux = clamp_len(s.lens[a[i]], s.bt_stride);
    if (aux % kPage != 0) {
      const int64_t page = s.table[a[i] * s.bt_stride + aux / kPage];
      need = page >= 0 && page < s.num_pages;
    }
  }
  if (ok && !FORK) {
    const int64_t len = clamp_len(s.lens[row], s.bt_stride), want = b[i];
    if (want < len || want > s.bt_stride * kPage) {
      raise(s.err, kErrLen);
    } else {
      aux = len;
      need = (int)((want + kPage - 1) / kPage - (len + kPage - 1) / kPage);
    }
  }
  w.need[i] = need;
  w.aux[i] = (int32_t)aux;
}

template <int MAX>
__global__ void __launch_bounds__(kThreads) pages_fork_kernel(
    const __grid_constant__ Pools<MAX> pools, const PageState s, const Workspace w, int segs,
    const int32_t* __restrict__ parents, const int32_t* __restrict__ children) {
  extern __shared__ int seg_at[];
  __shared__ int tmp[kThreads / 32];
  __shared__ int new_page;
  pdl_wait();
  pdl_trigger();
  const int per = pools.pieces > 0 ? pools.pieces : 1;
  const int64_t i = blockIdx.x / per;
  const int piece = (int)(blockIdx.x % per);
  const int64_t len = w.aux[i];
  if (len < 0) return;
  const int64_t parent = parents[i], child = children[i];
  const int64_t full = len / kPage;
  const int32_t* from = s.table + parent * s.bt_stride;
  int32_t* to = s.table + child * s.bt_stride;
  if (w.need[i]) {
    const int64_t rank = need_before(w, i);
    const int total = scan_segments(w, segs, seg_at, tmp);
    if (rank >= total) {
      if (piece == 0 && threadIdx.x == 0) raise(s.err, kErrNoPage);
      return;
    }
    if (threadIdx.x == 0) new_page = select_free(w, s.num_pages, segs, seg_at, (int)rank);
    __syncthreads();
    if (piece == 0 && threadIdx.x == 0) {
      to[full] = new_page;
      s.refs[new_page] = 1;
    }
    if (pools.pieces > 0) copy_piece(pools, piece, (int64_t)from[full], (int64_t)new_page);
  }
  if (piece != 0) return;
  if (!w.need[i] && len % kPage != 0 && threadIdx.x == 0) {
    to[full] = from[full];
    raise(s.err, kErrPage);
  }
  for (int64_t j = threadIdx.x; j < full; j += kThreads) {
    const int page = from[j];
    to[j] = page;
    if (page >= 0 && page < s.num_pages)
      atomicAdd(&s.refs[page], 1);
    else
      raise(s.err, kErrPage);
  }
  if (threadIdx.x == 0) s.lens[child] = (int32_t)len;
}

__global__ void __launch_bounds__(kThreads) pages_extend_kernel(
    const PageState s, const Workspace w, int segs, const int32_t* __restrict__ rows,
    const int32_t* __restrict__ new_lens) {
  extern __shared__ int seg_at[];
  __shared__ int tmp[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int64_t i = blockIdx.x;
  const int64_t len = w.aux[i];
  if (len < 0) return;
  const int need = w.need[i];
  const int64_t row = rows[i];
  if (need > 0) {
    const int64_t rank = need_before(w, i);
    const int total = scan_segments(w, segs, seg_at, tmp);
    if (rank + need > total) {
      if (threadIdx.x == 0) raise(s.err, kErrNoPage);
      return;
    }
    int32_t* to = s.table + row * s.bt_stride + (len + kPage - 1) / kPage;
    for (int j = threadIdx.x; j < need; j += kThreads) {
      const int page = select_free(w, s.num_pages, segs, seg_at, (int)rank + j);
      to[j] = page;
      s.refs[page] = 1;
    }
  }
  if (threadIdx.x == 0) s.lens[row] = new_lens[i];
}

// ---------------------------------------------------------------- compact
__global__ void __launch_bounds__(kThreads) pages_snapshot_kernel(const PageState s,
                                                                 const Workspace w) {
  __shared__ int tmp[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  snapshot_segment(s, w, blockIdx.x, tmp);
}

// Per segment: the live rank at each word, and the segment's share of the
// holes (free pages below num_live, ascending: free rank = index) and of the
// moved pages (live pages from num_live on, ascending).
__global__ void __launch_bounds__(kThreads) pages_lists_kernel(const PageState s, const Workspace w,
                                                              int segs, int32_t* num_live_out) {
  __shared__ int tmp[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, seg = blockIdx.x;
  int all = 0, before = 0;
  for (int i = tid; i < segs; i += kThreads) {
    const int f = w.seg_free[i];
    all += f;
    if (i < seg) before += f;
  }
  const int total_free = block_sum(all, tmp);
  const int free_before = block_sum(before, tmp);
  const int num_live = (int)s.num_pages - total_free;
  // Free pages below num_live = number of holes = number of moved pages.
  const int cut = num_live / kSeg;
  int below = 0;
  for (int i = tid; i < cut; i += kThreads) below += w.seg_free[i];
  if (cut < segs && tid < kSegWords) {
    const int64_t base = (int64_t)cut * kSeg + tid * 32;
    if (base < num_live) {
      uint32_t f = ~w.live[cut * kSegWords + tid];
      if (base + 32 > num_live) f &= (1u << (num_live - base)) - 1u;
      below += __popc(f);
    }
  }
  const int moved = block_sum(below, tmp);
  if (seg == 0 && tid == 0) {
    w.totals[0] = num_live;
    w.totals[1] = moved;
    *num_live_out = num_live;
  }
  if (tid >= 32) return;
  // One warp: lane l has word l of the segment.
  const int64_t base = (int64_t)seg * kSeg + tid * 32;
  const uint32_t live = w.live[seg * kSegWords + tid];
  const int64_t left = s.num_pages - base;
  uint32_t open = ~live;
  if (left < 32) open &= left <= 0 ? 0u : (1u << left) - 1u;
  int lr = __popc(live), fr = __popc(open);
  const int lc = lr, fc = fr;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, lr, o), b = __shfl_up_sync(0xffffffffu, fr, o);
    if (tid >= o) {
      lr += a;
      fr += b;
    }
  }
  lr += seg * kSeg - free_before - lc;   // live pages before this word
  fr += free_before - fc;                // free pages before this word
  w.word_rank[seg * kSegWords + tid] = lr;
  const int live_below = num_live - moved;   // live pages that stay
  for (uint32_t f = open; f != 0u; f &= f - 1) {
    const int page = (int)base + __ffs(f) - 1;
    if (page < num_live) w.holes[fr] = page;
    ++fr;
  }
  for (uint32_t f = live; f != 0u; f &= f - 1) {
    const int page = (int)base + __ffs(f) - 1;
    if (page >= num_live) w.moved[lr - live_below] = page;
    ++lr;
  }
}

// Where a live page goes.
__device__ __forceinline__ int new_page_of(const Workspace& w, int page, int num_live, int moved) {
  if (page < num_live) return page;
  const uint32_t bits = w.live[page >> 5] & ((1u << (page & 31)) - 1u);
  return w.holes[w.word_rank[page >> 5] + __popc(bits) - (num_live - moved)];
}

// Block ranges: reference counts, block-table rows, payload.
template <int MAX>
__global__ void __launch_bounds__(kThreads) pages_apply_kernel(
    const __grid_constant__ Pools<MAX> pools, const PageState s, const Workspace w, int ref_blocks,
    int64_t row_blocks, int32_t* refs_out, int32_t* table_out) {
  pdl_wait();
  pdl_trigger();
  const int num_live = w.totals[0], moved = w.totals[1];
  int64_t b = blockIdx.x;
  if (b < ref_blocks) {
    const int64_t page = b * kThreads + threadIdx.x;
    if (page >= s.num_pages) return;
    const bool live = (w.live[page >> 5] >> (page & 31)) & 1u;
    if (live) {
      const int to = new_page_of(w, (int)page, num_live, moved);
      refs_out[to] = s.refs[page];
    }
    if (page >= num_live) refs_out[page] = 0;   // read above, by this thread alone
    return;
  }
  b -= ref_blocks;
  if (b < row_blocks) {
    const int64_t held = (clamp_len(s.lens[b], s.bt_stride) + kPage - 1) / kPage;
    const int32_t* from = s.table + b * s.bt_stride;
    int32_t* to = table_out + b * s.bt_stride;
    for (int64_t j = threadIdx.x; j < s.bt_stride; j += kThreads) {
      int page = from[j];
      if (j < held) {
        if (page >= 0 && page < s.num_pages && ((w.live[page >> 5] >> (page & 31)) & 1u))
          page = new_page_of(w, page, num_live, moved);
        else
          raise(s.err, kErrPage);
      }
      to[j] = page;
    }
    return;
  }
  b -= row_blocks;
  const int64_t workers = gridDim.x - ref_blocks - row_blocks;
  for (int64_t i = b; i < (int64_t)moved * pools.pieces; i += workers)
    copy_piece(pools, (int)(i % pools.pieces), w.moved[i / pools.pieces],
               w.holes[i / pools.pieces]);
}

template <int MAX>
cudaError_t run_copy(const ds_page_pool* pools, int num_pools, int64_t num_pages,
                     const int32_t* src, const int32_t* dst, int64_t n, int32_t* err,
                     cudaStream_t stream) {
  const Pools<MAX> p = make_pools<MAX>(pools, num_pools);
  return launch_pdl(pages_copy_kernel<MAX>, dim3((unsigned)(n * p.pieces)), dim3(kThreads), 0,
                    stream, 1u, p, num_pages, src, dst, err);
}

template <int MAX>
cudaError_t run_fork(const ds_page_pool* pools, int num_pools, const PageState& s,
                     const Workspace& w, int segs, const int32_t* parents,
                     const int32_t* children, int64_t n, cudaStream_t stream) {
  const Pools<MAX> p = make_pools<MAX>(pools, num_pools);
  const int64_t per = p.pieces > 0 ? p.pieces : 1;
  return launch_pdl(pages_fork_kernel<MAX>, dim3((unsigned)(n * per)), dim3(kThreads), segs * 4,
                    stream, 1u, p, s, w, segs, parents, children);
}

template <int MAX>
cudaError_t run_apply(const ds_page_pool* pools, int num_pools, const PageState& s,
                      const Workspace& w, int32_t* refs_out, int32_t* table_out,
                      cudaStream_t stream) {
  const Pools<MAX> p = make_pools<MAX>(pools, num_pools);
  const int ref_blocks = (int)((s.num_pages + kThreads - 1) / kThreads);
  const int64_t copy_blocks = p.pieces > 0 ? 152 * 8 : 0;
  return launch_pdl(pages_apply_kernel<MAX>,
                    dim3((unsigned)(ref_blocks + s.num_rows + copy_blocks)), dim3(kThreads), 0,
                    stream, 1u, p, s, w, ref_blocks, s.num_rows, refs_out, table_out);
}

}  // namespace

size_t pages_workspace_bytes(int64_t num_pages, int64_t n) {
  return carve(nullptr, nullptr, num_pages, n);
}

cudaError_t launch_pages_copy(const ds_page_pool* pools, int num_pools, int64_t num_pages,
                              const int32_t* src, const int32_t* dst, int64_t n, int32_t* err,
                              cudaStream_t stream) {
  return num_pools <= kFewPools
             ? run_copy<kFewPools>(pools, num_pools, num_pages, src, dst, n, err, stream)
             : run_copy<DS_MAX_POOLS>(pools, num_pools, num_pages, src, dst, n, err, stream);
}

cudaError_t launch_pages_free(const PageState& s, const int32_t* rows, int64_t n,
                              cudaStream_t stream) {
  return launch_pdl(pages_free_kernel, dim3((unsigned)n), dim3(kThreads), 0, stream, 1u, s, rows);
}

cudaError_t launch_pages_fork(const ds_page_pool* pools, int num_pools, const PageState& s,
                              const int32_t* parents, const int32_t* children, int64_t n,
                              void* workspace, cudaStream_t stream) {
  Workspace w;
  carve(&w, workspace, s.num_pages, n);
  const int segs = num_segs(s.num_pages);
  const cudaError_t e = launch_pdl(pages_plan_kernel<true>,
                                   dim3((unsigned)(segs + (n + kThreads - 1) / kThreads)),
                                   dim3(kThreads), 0, stream, 1u, s, w, segs, parents, children, n);
  if (e != cudaSuccess) return e;
  return num_pools <= kFewPools
             ? run_fork<kFewPools>(pools, num_pools, s, w, segs, parents, children, n, stream)
             : run_fork<DS_MAX_POOLS>(pools, num_pools, s, w, segs, parents, children, n, stream);
}

cudaError_t launch_pages_extend(const PageState& s, const int32_t* rows, const int32_t* new_lens,
                                int64_t n, void* workspace, cudaStream_t stream) {
  Workspace w;
  carve(&w, workspace, s.num_pages, n);
  const int segs = num_segs(s.num_pages);
  cudaError_t e = launch_pdl(pages_plan_kernel<false>,
                             dim3((unsigned)(segs + (n + kThreads - 1) / kThreads)),
                             dim3(kThreads), 0, stream, 1u, s, w, segs, rows, new_lens, n);
  if (e != cudaSuccess) return e;
  return launch_pdl(pages_extend_kernel, dim3((unsigned)n), dim3(kThreads), segs * 4, stream, 1u, s,
                    w, segs, rows, new_lens);
}

cudaError_t launch_pages_compact(const ds_page_pool* pools, int num_pools, const PageState& s,
                                 int32_t* refs_out, int32_t* table_out, int32_t* num_live_out,
                                 void* workspace, cudaStream_t stream) {
  Workspace w;
  carve(&w, workspace, s.num_pages, 0);
  const int segs = num_segs(s.num_pages);
  cudaError_t e = launch_pdl(pages_snapshot_kernel, dim3((unsigned)segs), dim3(kThreads), 0, stream,
                             1u, s, w);
  if (e != cudaSuccess) return e;
  e = launch_pdl(pages_lists_kernel, dim3((unsigned)segs), dim3(kThreads), 0, stream, 1u, s, w,
                 segs, num_live_out);
  if (e != cudaSuccess) return e;
  return num_pools <= kFewPools
             ? run_apply<kFewPools>(pools, num_pools, s, w, refs_out, table_out, stream)
             : run_apply<DS_MAX_POOLS>(pools, num_pools, s, w, refs_out, table_out, stream);
}

static_assert(kMaxSegs * 4 <= 48 * 1024 - 256, "segment counts fit the default shared memory");

}  // namespace dsmla
