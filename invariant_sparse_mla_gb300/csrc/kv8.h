// Declarations shared by the block-scaled 8-bit cache (kv8_*.cu) and the page
// operations (pages.cu).
#pragma once

#include <stdint.h>
#include <cuda_runtime.h>

#include "ds_sparse_mla.h"
#include "internal.h"

namespace dsmla {

constexpr int kPage = DS_PAGE_BLOCK_SIZE;

// One layer's kv8 cache and the block table that indexes it.
struct Kv8Cache {
  uint8_t* pages;             // [num_pages, 2, kv_heads, 64, dim]
  float* scales;              // [num_pages, 2, kv_heads]
  int64_t num_pages;
  const int32_t* block_table; // [requests, bt_stride]
  int64_t bt_stride;
  const int32_t* lens;        // [requests]
  int64_t requests;
  int kv_heads;
  int dim;
  int32_t* err;               // may be nullptr
};

struct Kv8AppendArgs {
  Kv8Cache c;
  const void* k;
  const void* v;
  int64_t k_stride, v_stride;  // elements
  int64_t tokens;
  const int32_t* starts;       // [requests + 1]
};

struct Kv8AttnArgs {
  Kv8Cache c;
  const void* q;
  int64_t q_stride;            // elements between tokens
  int64_t tokens;              // rows of q: requests * next_n, or num_tokens
  const int32_t* starts;       // prefill: [requests + 1]; decode: nullptr
  int next_n;                  // decode; 0 for prefill
  int heads;
  float scale;
  void* out;
  float* lse;
  void* workspace;
};

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t stream);
cudaError_t launch_kv8_decode(const Kv8AttnArgs& a, cudaStream_t stream);
cudaError_t launch_kv8_prefill(const Kv8AttnArgs& a, cudaStream_t stream);
size_t kv8_decode_workspace_bytes(int64_t requests, int next_n, int heads, int kv_heads, int dim,
                                  int64_t bt_stride);
size_t kv8_prefill_workspace_bytes(int64_t tokens, int64_t requests, int heads, int kv_heads,
                                   int dim);

// SMs of a device (looked up once).
int kv8_sm_count(int dev);
// Items (256 query rows) of a prefill call per kv head, an upper bound.
int64_t kv8_prefill_units(int64_t tokens, int64_t requests, int group);

// ---- pages
struct PageState {
  int32_t* refs;
  int64_t num_pages;
  int32_t* table;
  int64_t bt_stride;
  int32_t* lens;
  int64_t num_rows;
  int32_t* err;
};

cudaError_t launch_pages_copy(const ds_page_pool* pools, int num_pools, int64_t num_pages,
                              const int32_t* src, const int32_t* dst, int64_t n, int32_t* err,
                              cudaStream_t stream);
cudaError_t launch_pages_free(const PageState& s, const int32_t* rows, int64_t n,
                              cudaStream_t stream);
cudaError_t launch_pages_fork(const ds_page_pool* pools, int num_pools, const PageState& s,
                              const int32_t* parents, const int32_t* children, int64_t n,
                              void* workspace, cudaStream_t stream);
cudaError_t launch_pages_extend(const PageState& s, const int32_t* rows, const int32_t* new_lens,
                                int64_t n, void* workspace, cudaStream_t stream);
cudaError_t launch_pages_compact(const ds_page_pool* pools, int num_pools, const PageState& s,
                                 int32_t* refs_out, int32_t* table_out, int32_t* num_live_out,
                                 void* workspace, cudaStream_t stream);
size_t pages_workspace_bytes(int64_t num_pages, int64_t n);

}  // namespace dsmla
