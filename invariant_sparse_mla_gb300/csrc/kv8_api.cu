// Host side of the block-scaled 8-bit cache, of the norm with rotation in front
// of it and of the page operations:
// argument validation before any launch, with messages that name the
// parameter, and the workspace sizes.

#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "ds_sparse_mla.h"
#include "internal.h"
#include "kv8.h"
#include "norm_rope.h"

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

int check_budget(const char* fn, int budget, int first, int recent, int64_t mass_stride) {
  if (mass_stride < 4 || mass_stride % 4 != 0 || mass_stride > ((int64_t)1 << 28))
    return report_error(DS_ERR_SHAPE,
                        "%s: mass_stride=%lld must be a positive multiple of 4 up to 2^28", fn,
                        (long long)mass_stride);
  if (budget < 1 || first < 0 || recent < 0 || first > budget || recent > budget - first)
    return report_error(DS_ERR_SHAPE,
                        "%s: budget=%d must be positive and at least first=%d + recent=%d, neither "
                        "of them negative",
                        fn, budget, first, recent);
  if (budget - first - recent > 16384)
    return report_error(DS_ERR_UNSUPPORTED,
                        "%s: budget - first - recent = %d is not supported; available: up to 16384",
                        fn, budget - first - recent);
  return DS_OK;
}

int launched(const char* fn, cudaError_t e) {
  if (e != cudaSuccess)
    return report_error(DS_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return report_ok();
}

cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

bool check_decode_shape(const char* fn, int64_t num_requests, int next_n, int num_heads,
                        int num_kv_heads, int head_dim, int64_t bt_stride) {
  dsmla::Kv8Cache c{};
  c.num_pages = 1;
  c.bt_stride = bt_stride;
  c.requests = num_requests;
  c.kv_heads = num_kv_heads;
  c.dim = head_dim;
  if (check_cache(fn, c) != DS_OK ||
      check_heads(fn, num_heads, num_kv_heads, (int64_t)num_heads * head_dim, head_dim, 1.0f) !=
          DS_OK)
    return false;
  if (next_n < 1 || next_n > 64) {
    report_error(DS_ERR_UNSUPPORTED, "%s: next_n=%d is not supported; available: 1 .. 64", fn,
                 next_n);
    return false;
  }
  return true;
}

// Decode attention, causal or (tree) by masks.
int decode(const char* fn, const void* q, int64_t q_stride, bool tree, const uint64_t* masks,
           const void* kv_pages, const float* kv_scales, int64_t num_pages,
           const int32_t* block_table, int64_t bt_stride, const int32_t* lens,
           int64_t num_requests, int next_n, int num_heads, int num_kv_heads, int head_dim,
           float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
           int32_t* err_flag, void* stream) {
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
  if (tree && bt_stride > (1 << 20))
    return report_error(DS_ERR_UNSUPPORTED, "%s: bt_stride=%lld exceeds 2^20", fn,
                        (long long)bt_stride);
  if (num_requests * next_n > (int64_t)INT32_MAX / num_heads)
    return report_error(DS_ERR_UNSUPPORTED,
                        "%s: num_requests=%lld is too large with next_n=%d and num_heads=%d "
                        "(below 2^31 rows)", fn, (long long)num_requests, next_n, num_heads);
  if (num_requests == 0) return report_ok();
  st = check_ptrs(fn, {{q, "q", 16},
                       {masks, "masks", 8, !tree},
                       {kv_pages, "kv_pages", 16},
                       {kv_scales, "kv_scales", 4},
                       {block_table, "block_table", 4},
                       {lens, "lens", 4},
                       {out, "out", 16},
                       {lse, "lse", 4},
                       {workspace, "workspace", 256},
                       {err_flag, "err_flag", 4, true}});
  if (st != DS_OK) return st;
  const bool tiles = tree && dsmla::kv8_tree_tiles(next_n, num_heads / num_kv_heads);
  const size_t need = (tiles ? dsmla::kv8_tree_workspace_bytes : dsmla::kv8_decode_workspace_bytes)(
      num_requests, next_n, num_heads, num_kv_heads, head_dim, bt_stride);
  if (workspace_bytes < need)
    return report_error(DS_ERR_WORKSPACE,
                        "%s: workspace_bytes=%zu is smaller than the %zu bytes needed", fn,
                        workspace_bytes, need);
  a.q = q;
  a.q_stride = q_stride;
  a.tokens = num_requests * next_n;
  a.next_n = next_n;
  a.masks = masks;
  a.heads = num_heads;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  return launched(fn, tiles ? dsmla::launch_kv8_tree(a, as_stream(stream))
                            : dsmla::launch_kv8_decode(a, as_stream(stream)));
}

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
  if (!check_decode_shape("ds_kv8_decode_workspace_size", num_requests, next_n, num_heads,
                          num_kv_heads, head_dim, bt_stride))
    return 0;
  return dsmla::kv8_decode_workspace_bytes(num_requests, next_n, num_heads, num_kv_heads, head_dim,
                                           bt_stride);
}

size_t ds_kv8_tree_decode_workspace_size(int64_t num_requests, int next_n, int num_heads,
                                         int num_kv_heads, int head_dim, int64_t bt_stride) {
  if (!check_decode_shape("ds_kv8_tree_decode_workspace_size", num_requests, next_n, num_heads,
                          num_kv_heads, head_dim, bt_stride))
    return 0;
  const bool tiles = dsmla::kv8_tree_tiles(next_n, num_heads / num_kv_heads);
  return (tiles ? dsmla::kv8_tree_workspace_bytes : dsmla::kv8_decode_workspace_bytes)(
      num_requests, next_n, num_heads, num_kv_heads, head_dim, bt_stride);
}

int ds_kv8_decode(const void* q, int64_t q_stride, const void* kv_pages, const float* kv_scales,
                  int64_t num_pages, const int32_t* block_table, int64_t bt_stride,
                  const int32_t* lens, int64_t num_requests, int next_n, int num_heads,
                  int num_kv_heads, int head_dim, float scale, void* out, float* lse,
                  void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream) {
  return decode("ds_kv8_decode", q, q_stride, false, nullptr, kv_pages, kv_scales, num_pages,
                block_table, bt_stride, lens, num_requests, next_n, num_heads, num_kv_heads,
                head_dim, scale, out, lse, workspace, workspace_bytes, err_flag, stream);
}

int ds_kv8_tree_decode(const void* q, int64_t q_stride, const uint64_t* masks,
                       const void* kv_pages, const float* kv_scales, int64_t num_pages,
                       const int32_t* block_table, int64_t bt_stride, const int32_t* lens,
                       int64_t num_requests, int next_n, int num_heads, int num_kv_heads,
                       int head_dim, float scale, void* out, float* lse, void* workspace,
                       size_t workspace_bytes, int32_t* err_flag, void* stream) {
  return decode("ds_kv8_tree_decode", q, q_stride, true, masks, kv_pages, kv_scales, num_pages,
                block_table, bt_stride, lens, num_requests, next_n, num_heads, num_kv_heads,
                head_dim, scale, out, lse, workspace, workspace_bytes, err_flag, stream);
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

int ds_kv8_mass(const void* q, int64_t q_stride, const float* lse, int64_t num_tokens,
                const int32_t* token_starts, int64_t num_requests, const void* kv_pages,
                const float* kv_scales, int64_t num_pages, const int32_t* block_table,
                int64_t bt_stride, const int32_t* lens, int num_heads, int num_kv_heads,
                int head_dim, float scale, float* mass, int64_t mass_stride, int32_t* err_flag,
                void* stream) {
  const char* fn = "ds_kv8_mass";
  dsmla::Kv8MassArgs a{};
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
  if (mass_stride < bt_stride * dsmla::kPage)
    return report_error(DS_ERR_SHAPE,
                        "%s: mass_stride=%lld must be at least 64 * bt_stride = %lld", fn,
                        (long long)mass_stride, (long long)bt_stride * dsmla::kPage);
  if (num_tokens == 0 || num_requests == 0) return report_ok();
  if (num_tokens > (int64_t)INT32_MAX / (num_heads / num_kv_heads) - 256)
    return report_error(DS_ERR_UNSUPPORTED, "%s: num_tokens=%lld is too large with %d query heads "
                        "a kv head (below 2^31 rows)", fn, (long long)num_tokens,
                        num_heads / num_kv_heads);
  st = check_ptrs(fn, {{q, "q", 16},
                       {lse, "lse", 4},
                       {token_starts, "token_starts", 4},
                       {kv_pages, "kv_pages", 16},
                       {kv_scales, "kv_scales", 4},
                       {block_table, "block_table", 4},
                       {lens, "lens", 4},
                       {mass, "mass", 4},
                       {err_flag, "err_flag", 4, true}});
  if (st != DS_OK) return st;
  a.q = q;
  a.q_stride = q_stride;
  a.lse = lse;
  a.tokens = num_tokens;
  a.starts = token_starts;
  a.heads = num_heads;
  a.scale = scale;
  a.mass = mass;
  a.mass_stride = mass_stride;
  return launched(fn, dsmla::launch_kv8_mass(a, as_stream(stream)));
}

size_t ds_kv8_evict_workspace_size(int64_t num_requests, int num_kv_heads, int64_t mass_stride,
                                   int budget, int first, int recent) {
  const char* fn = "ds_kv8_evict_workspace_size";
  dsmla::Kv8Cache c{};
  c.num_pages = 1;
  c.bt_stride = 1;
  c.requests = num_requests;
  c.kv_heads = num_kv_heads;
  c.dim = 64;
  if (check_cache(fn, c) != DS_OK || check_budget(fn, budget, first, recent, mass_stride) != DS_OK)
    return 0;
  return dsmla::kv8_evict_workspace_bytes(num_requests, num_kv_heads, budget - first - recent);
}

int ds_kv8_evict(float* mass, int64_t mass_stride, int budget, int first, int recent,
                 void* kv_pages, float* kv_scales, int64_t num_pages, const int32_t* refcounts,
                 const int32_t* block_table, int64_t bt_stride, const int32_t* lens,
                 int64_t num_requests, int num_kv_heads, int head_dim, int32_t* new_lens,
                 void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream) {
  const char* fn = "ds_kv8_evict";
  dsmla::Kv8EvictArgs a{};
  a.c = {static_cast<uint8_t*>(kv_pages), kv_scales, num_pages, block_table, bt_stride, lens,
         num_requests, num_kv_heads, head_dim, err_flag};
  int st = check_cache(fn, a.c);
  if (st == DS_OK) st = check_budget(fn, budget, first, recent, mass_stride);
  if (st != DS_OK) return st;
  if (num_requests * num_kv_heads > (int64_t)1 << 26)
    return report_error(DS_ERR_UNSUPPORTED,
                        "%s: num_requests=%lld with %d kv heads is too large (2^26 rows)", fn,
                        (long long)num_requests, num_kv_heads);
  if (num_requests == 0) return report_ok();
  st = check_ptrs(fn, {{mass, "mass", 16},
                       {kv_pages, "kv_pages", 16},
                       {kv_scales, "kv_scales", 4},
                       {refcounts, "refcounts", 4, true},
                       {block_table, "block_table", 4},
                       {lens, "lens", 4},
                       {new_lens, "new_lens", 4},
                       {workspace, "workspace", 256},
                       {err_flag, "err_flag", 4, true}});
  if (st != DS_OK) return st;
  if (new_lens == lens)
    return report_error(DS_ERR_SHAPE, "%s: new_lens must not be lens", fn);
  const size_t need =
      dsmla::kv8_evict_workspace_bytes(num_requests, num_kv_heads, budget - first - recent);
  if (workspace_bytes < need)
    return report_error(DS_ERR_WORKSPACE,
                        "%s: workspace_bytes=%zu is smaller than the %zu bytes needed", fn,
                        workspace_bytes, need);
  a.mass = mass;
  a.mass_stride = mass_stride;
  a.budget = budget;
  a.first = first;
  a.recent = recent;
  a.refcounts = refcounts;
  a.new_lens = new_lens;
  return launched(fn, dsmla::launch_kv8_evict(a, workspace, as_stream(stream)));
}

int ds_kv8_accept(const ds_kv8_layer* layers, int num_layers, int64_t num_pages,
                  const int32_t* block_table, int64_t bt_stride, const int32_t* lens,
                  int64_t num_requests, int num_kv_heads, int head_dim, int next_n,
                  const int32_t* accepted, int width, int32_t* new_lens, int32_t* err_flag,
                  void* stream) {
  const char* fn = "ds_kv8_accept";
  dsmla::Kv8AcceptArgs a{};
  a.c = {nullptr, nullptr, num_pages, block_table, bt_stride, lens, num_requests, num_kv_heads,
         head_dim, err_flag};
  int st = check_cache(fn, a.c);
  if (st != DS_OK) return st;
  if (num_layers < 1 || num_layers > DS_MAX_KV8_LAYERS)
    return report_error(DS_ERR_UNSUPPORTED, "%s: num_layers=%d must be in [1, %d]", fn, num_layers,
                        DS_MAX_KV8_LAYERS);
  if (next_n < 1 || next_n > 64)
    return report_error(DS_ERR_UNSUPPORTED, "%s: next_n=%d is not supported; available: 1 .. 64",
                        fn, next_n);
  if (width < 1 || width > next_n)
    return report_error(DS_ERR_SHAPE, "%s: width=%d must be in [1, next_n=%d]", fn, width, next_n);
  if (num_requests > (int64_t)INT32_MAX / (2 * num_layers * (int64_t)num_kv_heads))
    return report_error(DS_ERR_UNSUPPORTED,
                        "%s: num_requests=%lld is too large with num_layers=%d and %d kv heads", fn,
                        (long long)num_requests, num_layers, num_kv_heads);
  if (num_requests == 0) return report_ok();
  if (layers == nullptr) return report_error(DS_ERR_NULL, "%s: layers is NULL", fn);
  for (int i = 0; i < num_layers; ++i) {
    if (layers[i].kv_pages == nullptr || layers[i].kv_scales == nullptr)
      return report_error(DS_ERR_NULL, "%s: layers[%d].%s is NULL", fn, i,
                          layers[i].kv_pages == nullptr ? "kv_pages" : "kv_scales");
    if (!aligned(layers[i].kv_pages, 16) || !aligned(layers[i].kv_scales, 4))
      return report_error(DS_ERR_ALIGN,
                          "%s: layers[%d]: kv_pages must be 16-byte and kv_scales 4-byte aligned",
                          fn, i);
    for (int j = 0; j < i; ++j)
      if (layers[j].kv_pages == layers[i].kv_pages || layers[j].kv_scales == layers[i].kv_scales)
        return report_error(DS_ERR_SHAPE, "%s: layers[%d] and layers[%d] are the same cache", fn, j,
                            i);
  }
  st = check_ptrs(fn, {{block_table, "block_table", 4},
                       {lens, "lens", 4},
                       {accepted, "accepted", 4},
                       {new_lens, "new_lens", 4},
                       {err_flag, "err_flag", 4, true}});
  if (st != DS_OK) return st;
  if (new_lens == lens)
    return report_error(DS_ERR_SHAPE, "%s: new_lens must not be lens", fn);
  a.accepted = accepted;
  a.width = width;
  a.next_n = next_n;
  a.new_lens = new_lens;
  return launched(fn, dsmla::launch_kv8_accept(layers, num_layers, a, as_stream(stream)));
}

// ------------------------------------------------------ norm with rotation
int ds_qk_norm_rope(const void* q, int64_t q_stride, int num_q_heads, const void* q_weight,
                    const void* k, int64_t k_stride, int num_k_heads, const void* k_weight,
                    int64_t num_tokens, int head_dim, int norm_dim, float eps,
                    const int32_t* positions, const float* inv_freq, int rot_start, int rot_dim,
                    int interleaved, void* q_out, int64_t q_out_stride, void* k_out,
                    int64_t k_out_stride, void* stream) {
  const char* fn = "ds_qk_norm_rope";
  if (head_dim < 16 || head_dim > 1024 || head_dim % 16 != 0)
    return report_error(DS_ERR_UNSUPPORTED,
                        "%s: head_dim=%d is not supported; available: multiples of 16 up to 1024",
                        fn, head_dim);
  if (num_q_heads < 1 || num_q_heads > 1024)
    return report_error(DS_ERR_UNSUPPORTED,
                        "%s: num_q_heads=%d is not supported; available: 1 .. 1024", fn,
                        num_q_heads);
  if (num_k_heads < 0 || num_k_heads > 1024)
    return report_error(DS_ERR_UNSUPPORTED,
                        "%s: num_k_heads=%d is not supported; available: 0 .. 1024", fn,
                        num_k_heads);
  int st = check_tokens(fn, num_tokens);
  if (st != DS_OK) return st;
  if (norm_dim < 0 || norm_dim > head_dim || norm_dim % 8 != 0)
    return report_error(DS_ERR_SHAPE,
                        "%s: norm_dim=%d must be a multiple of 8 in [0, head_dim=%d]", fn, norm_dim,
                        head_dim);
  if (norm_dim == 0 && (q_weight != nullptr || k_weight != nullptr))
    return report_error(DS_ERR_SHAPE, "%s: norm_dim=0 takes no q_weight or k_weight", fn);
  if (rot_dim < 0 || rot_dim % 16 != 0 || rot_start < 0 || rot_start % 8 != 0 ||
      rot_dim > head_dim || rot_start > head_dim - rot_dim)
    return report_error(DS_ERR_SHAPE,
                        "%s: rot_dim=%d must be a multiple of 16 and rot_start=%d one of 8, inside "
                        "head_dim=%d",
                        fn, rot_dim, rot_start, head_dim);
  if (!(eps >= 0.0f) || !std::isfinite(eps))
    return report_error(DS_ERR_SHAPE, "%s: eps must be finite and not negative", fn);
  const struct {
    const char* name;
    int64_t stride;
    int heads;
  } strides[] = {{"q_stride", q_stride, num_q_heads},
                 {"k_stride", k_stride, num_k_heads},
                 {"q_out_stride", q_out_stride, num_q_heads},
                 {"k_out_stride", k_out_stride, num_k_heads}};
  for (const auto& s : strides)
    if (s.heads > 0 && (s.stride < (int64_t)s.heads * head_dim || s.stride % 8 != 0))
      return report_error(DS_ERR_SHAPE,
                          "%s: %s=%lld must be a multiple of 8 and at least heads * head_dim = %lld",
                          fn, s.name, (long long)s.stride, (long long)s.heads * head_dim);
  if (num_tokens == 0) return report_ok();
  const bool no_k = num_k_heads == 0;
  st = check_ptrs(fn, {{q, "q", 16},
                       {k, "k", 16, no_k},
                       {q_weight, "q_weight", 16, true},
                       {k_weight, "k_weight", 16, true},
                       {positions, "positions", 4, rot_dim == 0},
                       {inv_freq, "inv_freq", 4, rot_dim == 0},
                       {q_out, "q_out", 16},
                       {k_out, "k_out", 16, no_k}});
  if (st != DS_OK) return st;
  dsmla::NormRopeArgs a{};
  a.q = {q, q_stride, q_out, q_out_stride, q_weight, num_q_heads};
  a.k = {k, k_stride, k_out, k_out_stride, k_weight, num_k_heads};
  a.tokens = num_tokens;
  a.dim = head_dim;
  a.norm_dim = norm_dim;
  a.rot_start = rot_start;
  a.rot_dim = rot_dim;
  a.interleaved = interleaved != 0;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.eps = eps;
  return launched(fn, dsmla::launch_norm_rope(a, as_stream(stream)));
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

int ds_pages_shrink(int32_t* refcounts, int64_t num_pages, int32_t* block_table,
                    int64_t bt_stride, int32_t* lens, int64_t num_rows, const int32_t* rows,
                    const int32_t* new_lens, int64_t n, int32_t* err_flag, void* stream) {
  const char* fn = "ds_pages_shrink";
  const dsmla::PageState s{refcounts, num_pages, block_table, bt_stride, lens, num_rows, err_flag};
  int st = check_state(fn, s);
  if (st == DS_OK) st = check_list(fn, n);
  if (st != DS_OK) return st;
  if (n == 0) return report_ok();
  st = check_ptrs(fn, {{rows, "rows", 4}, {new_lens, "new_lens", 4}});
  if (st != DS_OK) return st;
  return launched(fn, dsmla::launch_pages_shrink(s, rows, new_lens, n, as_stream(stream)));
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
