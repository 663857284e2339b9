// Host side of the block-scaled 8-bit cache and of the page operations:
// argument validation before any launch, with messages that name the
// parameter, and the workspace sizes.

#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "ds_sparse_mla.h"
#include "internal.h"
#include "kv8.h"

namespace {

using dsmla::report_error;
using dsmla::report_ok;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Ptr {
  const void* p;
  const char* name;
  int align;
  bool optional = false;
};

template <int N>
int check_ptrs(const char* fn, const Ptr (&ptrs)[N]) {
  for (const Ptr& x : ptrs) {
    if (x.p == nullptr) {
      if (x.optional) continue;
      return report_error(DS_ERR_NULL, "%s: %s is NULL", fn, x.name);
    }
    if (!aligned(x.p, x.align))
      return report_error(DS_ERR_ALIGN, "%s: %s must be %d-byte aligned", fn, x.name, x.align);
  }
  return DS_OK;
}

int check_cache(const char* fn, const dsmla::Kv8Cache& c) {
  if (c.dim != 64 && c.dim != 128)
    return report_error(DS_ERR_UNSUPPORTED, "%s: head_dim=%d is not supported; available: 64, 128",
                        fn, c.dim);
  if (c.kv_heads < 1 || c.kv_heads > 1024)
    return report_error(DS_ERR_UNSUPPORTED,
                        "%s: num_kv_heads=%d is not supported; available: 1 .. 1024", fn,
                        c.kv_heads);
  if (c.num_pages < 1)
    return report_error(DS_ERR_SHAPE, "%s: num_pages=%lld must be >= 1", fn,
                        (long long)c.num_pages);
  const int64_t most = ((int64_t)1 << 31) / (2 * dsmla::kPage * (int64_t)c.kv_heads);
  if (c.num_pages >= most)
    return report_error(DS_ERR_UNSUPPORTED,
                        "%s: num_pages=%lld is too large (below %lld with %d kv heads)", fn,
                        (long long)c.num_pages, (long long)most, c.kv_heads);
  if (c.bt_stride < 1)
    return report_error(DS_ERR_SHAPE, "%s: bt_stride=%lld must be >= 1", fn,
                        (long long)c.bt_stride);
  if (c.bt_stride > (1 << 24))
    return report_error(DS_ERR_UNSUPPORTED, "%s: bt_stride=%lld exceeds 2^24", fn,
                        (long long)c.bt_stride);
  if (c.requests < 0)
    return report_error(DS_ERR_SHAPE, "%s: num_requests=%lld is negative", fn,
                        (long long)c.requests);
  if (c.requests > (1 << 20))
    return report_error(DS_ERR_UNSUPPORTED, "%s: num_requests=%lld exceeds 2^20", fn,
                        (long long)c.requests);
  return DS_OK;
}

int check_heads(const char* fn, int heads, int kv_heads, int64_t q_stride, int dim, float scale) {
  if (heads < 1 || heads > 1024 || heads % kv_heads != 0)
    return report_error(DS_ERR_UNSUPPORTED,
                        "%s: num_heads=%d is not supported; available: multiples of "
                        "num_kv_heads=%d up to 1024",
                        fn, heads, kv_heads);
  if (q_stride < (int64_t)heads * dim || q_stride % 8 != 0)
    return report_error(DS_ERR_SHAPE,
                        "%s: q_stride=%lld must be a multiple of 8 and at least num_heads * "
                        "head_dim = %lld",
                        fn, (long long)q_stride, (long long)heads * dim);
  if (!std::isfinite(scale)) return report_error(DS_ERR_SHAPE, "%s: scale must be finite", fn);
  return DS_OK;
}

int check_tokens(const char* fn, int64_t tokens) {
  if (tokens < 0)
    return report_error(DS_ERR_SHAPE, "%s: num_tokens=%lld is negative", fn, (long long)tokens);
  if (tokens > (1 << 24))
    return report_error(DS_ERR_UNSUPPORTED, "%s: num_tokens=%lld exceeds 2^24", fn,
                        (long long)tokens);
  return DS_OK;
}

int launched(const char* fn, cudaError_t e) {
  if (e != cudaSuccess)
    return report_error(DS_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return report_ok();
}

cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

int ds_kv8_append(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                  int64_t num_tokens, const int32_t* token_starts, int64_t num_requests,
                  const int32_t* block_table, int64_t bt_stride, const int32_t* lens,
                  int num_kv_heads, int head_dim, void* kv_pages, float* kv_scales,
                  int64_t num_pages, int32_t* err_flag, void* stream) {
  const char* fn = "ds_kv8_append";
  dsmla::Kv8AppendArgs a{{static_cast<uint8_t*>(kv_pages), kv_scales, num_pages, block_table,
                          bt_stride, lens, num_requests, num_kv_heads, head_dim, err_flag},
                         k, v, k_stride, v_stride, num_tokens, token_starts};
  int st = check_cache(fn, a.c);
  if (st == DS_OK) st = check_tokens(fn, num_tokens);
  if (st != DS_OK) return st;
  const int64_t row = (int64_t)num_kv_heads * head_dim;
  if (k_stride < row || k_stride % 8 != 0 || v_stride < row || v_stride % 8 != 0)
    return report_error(DS_ERR_SHAPE,
                        "%s: k_stride=%lld and v_stride=%lld must be multiples of 8 and at least "
                        "num_kv_heads * head_dim = %lld",
                        fn, (long long)k_stride, (long long)v_stride, (long long)row);
  if (num_tokens == 0 || num_requests == 0) return report_ok();
  if (num_tokens / dsmla::kPage + 2 * num_requests > (int64_t)INT32_MAX / (2 * num_kv_heads))
    return report_error(DS_ERR_UNSUPPORTED, "%s: num_tokens=%lld and num_requests=%lld are too "
                        "large for one launch", fn, (long long)num_tokens, (long long)num_requests);
  st = check_ptrs(fn, {{k, "k", 16},
                       {v, "v", 16},
                       {token_starts, "token_starts", 4},
                       {block_table, "block_table", 4},
                       {lens, "lens", 4},
                       {kv_pages, "kv_pages", 16},
                       {kv_scales, "kv_scales", 4},
                       {err_flag, "err_flag", 4, true}});
  if (st != DS_OK) return st;
  return launched(fn, dsmla::launch_kv8_append(a, as_stream(stream)));
}

size_t ds_kv8_decode_workspace_size(int64_t num_requests, int next_n, int num_heads,
                                    int num_kv_heads, int head_dim, int64_t bt_stride) {
  const char* fn = "ds_kv8_decode_workspace_size";
  dsmla::Kv8Cache c{};
  c.num_pages = 1;
  c.bt_stride = bt_stride;
  c.requests = num_requests;
  c.kv_heads = num_kv_heads;
  c.dim = head_dim;
  if (check_cache(fn, c) != DS_OK ||
      check_heads(fn, num_heads, num_kv_heads, (int64_t)num_heads * head_dim, head_dim, 1.0f) !=
          DS_OK)
    return 0;
  if (next_n < 1 || next_n > 64) {
    report_error(DS_ERR_UNSUPPORTED, "%s: next_n=%d is not supported; available: 1 .. 64", fn,
                 next_n);
    return 0;
  }
  return dsmla::kv8_decode_workspace_bytes(num_requests, next_n, num_heads, num_kv_heads, head_dim,
                                           bt_stride);
}

int ds_kv8_decode(const void* q, int64_t q_stride, const void* kv_pages, const float* kv_scales,
                  int64_t num_pages, const int32_t* block_table, int64_t bt_stride,
                  const int32_t* lens, int64_t num_requests, int next_n, int num_heads,
                  int num_kv_heads, int head_dim, float scale, void* out, float* lse,
                  void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream) {
  const char* fn = "ds_kv8_decode";
  dsmla::Kv8AttnArgs a{};
  a.c = {const_cast<uint8_t*>(static_cast<const uint8_t*>(kv_pages)),
         const_cast<float*>(kv_scales), num_pages, block_table, bt_stride, lens, num_requests,
         num_kv_heads, head_dim, err_flag};
  int st = check_cache(fn, a.c);
  if (st == DS_OK) st = check_heads(fn, num_heads, num_kv_heads, q_stride, head_dim, scale);
  if (st != DS_OK) return st;
  if (next_n < 1 || next_n > 64)
    return report_error(DS_ERR_UNSUPPORTED, "%s: next_n=%d is not supported; available: 1 .. 64",
                        fn, next_n);
  if (num_requests * next_n > (int64_t)INT32_MAX / num_heads)
    return report_error(DS_ERR_UNSUPPORTED,
                        "%s: num_requests=%lld is too large with next_n=%d and num_heads=%d "
                        "(below 2^31 rows)", fn, (long long)num_requests, next_n, num_heads);
  if (num_requests == 0) return report_ok();
  st = check_ptrs(fn, {{q, "q", 16},
                       {kv_pages, "kv_pages", 16},
                       {kv_scales, "kv_scales", 4},
                       {block_table, "block_table", 4},
                       {lens, "lens", 4},
                       {out, "out", 16},
                       {lse, "lse", 4},
                       {workspace, "workspace", 256},
                       {err_flag, "err_flag", 4, true}});
  if (st != DS_OK) return st;
  const size_t need = dsmla::kv8_decode_workspace_bytes(num_requests, next_n, num_heads,
                                                        num_kv_heads, head_dim, bt_stride);
  if (workspace_bytes < need)
    return report_error(DS_ERR_WORKSPACE,
                        "%s: workspace_bytes=%zu is smaller than the %zu bytes needed", fn,
                        workspace_bytes, need);
  a.q = q;
  a.q_stride = q_stride;
  a.tokens = num_requests * next_n;
  a.next_n = next_n;
  a.heads = num_heads;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  return launched(fn, dsmla::launch_kv8_decode(a, as_stream(stream)));
}

size_t ds_kv8_prefill_workspace_size(int64_t num_tokens, int64_t num_requests, int num_heads,
                                     int num_kv_heads, int head_dim) {
  const char* fn = "ds_kv8_prefill_workspace_size";
  dsmla::Kv8Cache c{};
  c.num_pages = 1;
  c.bt_stride = 1;
  c.requests = num_requests;
  c.kv_heads = num_kv_heads;
  c.dim = head_dim;
  if (check_cache(fn, c) != DS_OK || check_tokens(fn, num_tokens) != DS_OK ||
      check_heads(fn, num_heads, num_kv_heads, (int64_t)num_heads * head_dim, head_dim, 1.0f) !=
          DS_OK)
    return 0;
  return dsmla::kv8_prefill_workspace_bytes(num_tokens, num_requests, num_heads, num_kv_heads,
                                            head_dim);
}

int ds_kv8_prefill(const void* q, int64_t q_stride, int64_t num_tokens,
                   const int32_t* token_starts, int64_t num_requests, const void* kv_pages,
                   const float* kv_scales, int64_t num_pages, const int32_t* block_table,
                   int64_t bt_stride, const int32_t* lens, int num_heads, int num_kv_heads,
                   int head_dim, float scale, void* out, float* lse, void* workspace,
                   size_t workspace_bytes, int32_t* err_flag, void* stream) {
  const char* fn = "ds_kv8_prefill";
  dsmla::Kv8AttnArgs a{};
  a.c = {const_cast<uint8_t*>(static_cast<const uint8_t*>(kv_pages)),
         const_cast<float*>(kv_scales), num_pages, block_table, bt_stride, lens, num_requests,
         num_kv_heads, head_dim, err_flag};
  int st = check_cache(fn, a.c);
  if (st == DS_OK) st = check_heads(fn, num_heads, num_kv_heads, q_stride, head_dim, scale);
  if (st == DS_OK) st = check_tokens(fn, num_tokens);
  if (st != DS_OK) return st;
  if (bt_stride > (1 << 20))
    return report_error(DS_ERR_UNSUPPORTED, "%s: bt_stride=%lld exceeds 2^20", fn,
                        (long long)bt_stride);
  if (num_tokens == 0 || num_requests == 0) return report_ok();
  if (num_tokens > (int64_t)INT32_MAX / (num_heads / num_kv_heads) - 256)
    return report_error(DS_ERR_UNSUPPORTED, "%s: num_tokens=%lld is too large with %d query heads "
                        "a kv head (below 2^31 rows)", fn, (long long)num_tokens,
                        num_heads / num_kv_heads);
  const size_t need = dsmla::kv8_prefill_workspace_bytes(num_tokens, num_requests, num_heads,
                                                         num_kv_heads, head_dim);
  st = check_ptrs(fn, {{q, "q", 16},
                       {token_starts, "token_starts", 4},
                       {kv_pages, "kv_pages", 16},
                       {kv_scales, "kv_scales", 4},
                       {block_table, "block_table", 4},
                       {lens, "lens", 4},
                       {out, "out", 16},
                       {lse, "lse", 4},
                       {workspace, "workspace", 256, need == 0},
                       {err_flag, "err_flag", 4, true}});
  if (st != DS_OK) return st;
  if (workspace_bytes < need)
    return report_error(DS_ERR_WORKSPACE,
                        "%s: workspace_bytes=%zu is smaller than the %zu bytes needed", fn,
                        workspace_bytes, need);
  a.q = q;
  a.q_stride = q_stride;
  a.tokens = num_tokens;
  a.starts = token_starts;
  a.heads = num_heads;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  return launched(fn, dsmla::launch_kv8_prefill(a, as_stream(stream)));
}

}  // extern "C"

// ------------------------------------------------------------------- pages
namespace {

constexpr int64_t kMaxPages = (int64_t)1 << 22;
constexpr int64_t kMaxList = 65535;

int check_pools(const char* fn, const ds_page_pool* pools, int num_pools) {
  if (num_pools < 0 || num_pools > DS_MAX_POOLS)
    return report_error(DS_ERR_UNSUPPORTED, "%s: num_pools=%d must be in [0, %d]", fn, num_pools,
                        DS_MAX_POOLS);
  if (num_pools > 0 && pools == nullptr) return report_error(DS_ERR_NULL, "%s: pools is NULL", fn);
  int64_t bytes = 0;
  for (int i = 0; i < num_pools; ++i) {
    if (pools[i].data == nullptr)
      return report_error(DS_ERR_NULL, "%s: pools[%d].data is NULL", fn, i);
    if (!aligned(pools[i].data, 4))
      return report_error(DS_ERR_ALIGN, "%s: pools[%d].data must be 4-byte aligned", fn, i);
    if (pools[i].page_bytes < 4 || pools[i].page_bytes % 4 != 0 ||
        pools[i].page_bytes > ((int64_t)1 << 28))
      return report_error(DS_ERR_SHAPE,
                          "%s: pools[%d].page_bytes=%lld must be a positive multiple of 4 up to "
                          "2^28",
                          fn, i, (long long)pools[i].page_bytes);
    bytes += pools[i].page_bytes;
  }
  if (bytes > ((int64_t)1 << 28))
    return report_error(DS_ERR_UNSUPPORTED,
                        "%s: the pools' page_bytes sum to %lld; available: up to 2^28", fn,
                        (long long)bytes);
  return DS_OK;
}

int check_list(const char* fn, int64_t n) {
  if (n < 0) return report_error(DS_ERR_SHAPE, "%s: n=%lld is negative", fn, (long long)n);
  if (n > kMaxList)
    return report_error(DS_ERR_UNSUPPORTED, "%s: n=%lld exceeds %lld", fn, (long long)n,
                        (long long)kMaxList);
  return DS_OK;
}

int check_num_pages(const char* fn, int64_t num_pages) {
  if (num_pages < 1)
    return report_error(DS_ERR_SHAPE, "%s: num_pages=%lld must be >= 1", fn, (long long)num_pages);
  if (num_pages > kMaxPages)
    return report_error(DS_ERR_UNSUPPORTED, "%s: num_pages=%lld exceeds 2^22", fn,
                        (long long)num_pages);
  return DS_OK;
}

int check_state(const char* fn, const dsmla::PageState& s) {
  int st = check_num_pages(fn, s.num_pages);
  if (st != DS_OK) return st;
  if (s.bt_stride < 1 || s.bt_stride > (int64_t)INT32_MAX / dsmla::kPage)
    return report_error(DS_ERR_SHAPE, "%s: bt_stride=%lld must be in [1, %lld]", fn,
                        (long long)s.bt_stride, (long long)(INT32_MAX / dsmla::kPage));
  if (s.num_rows < 1 || s.num_rows > (1 << 24))
    return report_error(DS_ERR_SHAPE, "%s: num_rows=%lld must be in [1, 2^24]", fn,
                        (long long)s.num_rows);
  return check_ptrs(fn, {{s.refs, "refcounts", 4},
                         {s.table, "block_table", 4},
                         {s.lens, "lens", 4},
                         {s.err, "err_flag", 4, true}});
}

int check_workspace(const char* fn, const void* ws, size_t bytes, int64_t num_pages, int64_t n) {
  const int st = check_ptrs(fn, {{ws, "workspace", 256}});
  if (st != DS_OK) return st;
  const size_t need = dsmla::pages_workspace_bytes(num_pages, n);
  if (bytes < need)
    return report_error(DS_ERR_WORKSPACE,
                        "%s: workspace_bytes=%zu is smaller than the %zu bytes needed", fn, bytes,
                        need);
  return DS_OK;
}

}  // namespace

extern "C" {

size_t ds_pages_workspace_size(int64_t num_pages, int64_t n) {
  const char* fn = "ds_pages_workspace_size";
  if (check_num_pages(fn, num_pages) != DS_OK || check_list(fn, n) != DS_OK) return 0;
  return dsmla::pages_workspace_bytes(num_pages, n);
}

int ds_pages_copy(const ds_page_pool* pools, int num_pools, int64_t num_pages, const int32_t* src,
                  const int32_t* dst, int64_t n, int32_t* err_flag, void* stream) {
  const char* fn = "ds_pages_copy";
  int st = check_pools(fn, pools, num_pools);
  if (st == DS_OK) st = check_num_pages(fn, num_pages);
  if (st == DS_OK) st = check_list(fn, n);
  if (st != DS_OK) return st;
  if (n == 0 || num_pools == 0) return report_ok();
  st = check_ptrs(fn, {{src, "src", 4}, {dst, "dst", 4}, {err_flag, "err_flag", 4, true}});
  if (st != DS_OK) return st;
  return launched(fn, dsmla::launch_pages_copy(pools, num_pools, num_pages, src, dst, n, err_flag,
                                               as_stream(stream)));
}

int ds_pages_free(int32_t* refcounts, int64_t num_pages, int32_t* block_table, int64_t bt_stride,
                  int32_t* lens, int64_t num_rows, const int32_t* rows, int64_t n,
                  int32_t* err_flag, void* stream) {
  const char* fn = "ds_pages_free";
  const dsmla::PageState s{refcounts, num_pages, block_table, bt_stride, lens, num_rows, err_flag};
  int st = check_state(fn, s);
  if (st == DS_OK) st = check_list(fn, n);
  if (st != DS_OK) return st;
  if (n == 0) return report_ok();
  st = check_ptrs(fn, {{rows, "rows", 4}});
  if (st != DS_OK) return st;
  return launched(fn, dsmla::launch_pages_free(s, rows, n, as_stream(stream)));
}

int ds_pages_fork(const ds_page_pool* pools, int num_pools, int32_t* refcounts, int64_t num_pages,
                  int32_t* block_table, int64_t bt_stride, int32_t* lens, int64_t num_rows,
                  const int32_t* parents, const int32_t* children, int64_t n, void* workspace,
                  size_t workspace_bytes, int32_t* err_flag, void* stream) {
  const char* fn = "ds_pages_fork";
  const dsmla::PageState s{refcounts, num_pages, block_table, bt_stride, lens, num_rows, err_flag};
  int st = check_pools(fn, pools, num_pools);
  if (st == DS_OK) st = check_state(fn, s);
  if (st == DS_OK) st = check_list(fn, n);
  if (st != DS_OK) return st;
  if (n == 0) return report_ok();
  st = check_ptrs(fn, {{parents, "parents", 4}, {children, "children", 4}});
  if (st == DS_OK) st = check_workspace(fn, workspace, workspace_bytes, num_pages, n);
  if (st != DS_OK) return st;
  return launched(fn, dsmla::launch_pages_fork(pools, num_pools, s, parents, children, n,
                                               workspace, as_stream(stream)));
}

int ds_pages_extend(int32_t* refcounts, int64_t num_pages, int32_t* block_table,
                    int64_t bt_stride, int32_t* lens, int64_t num_rows, const int32_t* rows,
                    const int32_t* new_lens, int64_t n, void* workspace, size_t workspace_bytes,
                    int32_t* err_flag, void* stream) {
  const char* fn = "ds_pages_extend";
  const dsmla::PageState s{refcounts, num_pages, block_table, bt_stride, lens, num_rows, err_flag};
  int st = check_state(fn, s);
  if (st == DS_OK) st = check_list(fn, n);
  if (st != DS_OK) return st;
  if (n == 0) return report_ok();
  st = check_ptrs(fn, {{rows, "rows", 4}, {new_lens, "new_lens", 4}});
  if (st == DS_OK) st = check_workspace(fn, workspace, workspace_bytes, num_pages, n);
  if (st != DS_OK) return st;
  return launched(fn, dsmla::launch_pages_extend(s, rows, new_lens, n, workspace,
                                                 as_stream(stream)));
}

int ds_pages_compact(const ds_page_pool* pools, int num_pools, const int32_t* refcounts,
                     int64_t num_pages, const int32_t* block_table, int64_t bt_stride,
                     const int32_t* lens, int64_t num_rows, int32_t* refcounts_out,
                     int32_t* block_table_out, int32_t* num_live_out, void* workspace,
                     size_t workspace_bytes, int32_t* err_flag, void* stream) {
  const char* fn = "ds_pages_compact";
  const dsmla::PageState s{const_cast<int32_t*>(refcounts), num_pages,
                           const_cast<int32_t*>(block_table), bt_stride,
                           const_cast<int32_t*>(lens), num_rows, err_flag};
  int st = check_pools(fn, pools, num_pools);
  if (st == DS_OK) st = check_state(fn, s);
  if (st == DS_OK)
    st = check_ptrs(fn, {{refcounts_out, "refcounts_out", 4},
                         {block_table_out, "block_table_out", 4},
                         {num_live_out, "num_live_out", 4}});
  if (st == DS_OK) st = check_workspace(fn, workspace, workspace_bytes, num_pages, 0);
  if (st != DS_OK) return st;
  return launched(fn, dsmla::launch_pages_compact(pools, num_pools, s, refcounts_out,
                                                  block_table_out, num_live_out, workspace,
                                                  as_stream(stream)));
}

}  // extern "C"
