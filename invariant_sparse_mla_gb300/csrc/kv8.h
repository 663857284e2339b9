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
  const uint64_t* masks;       // decode of a tree: [requests, next_n]; nullptr: causal
  int heads;
  float scale;
  void* out;
  float* lse;
  void* workspace;
};

// Accepted drafts (layers give the pages and scales; c.pages is not used).
struct Kv8AcceptArgs {
  Kv8Cache c;
  const int32_t* accepted;     // [requests, width]
  int width;
  int next_n;
  int32_t* new_lens;           // [requests]
};

struct Kv8EvictArgs {
  Kv8Cache c;
  float* mass;                 // [requests, kv_heads, mass_stride]
  int64_t mass_stride;
  int budget, first, recent;
  const int32_t* refcounts;    // [num_pages] or nullptr
  int32_t* new_lens;           // [requests]
  int32_t *starts, *ends, *top;   // workspace: [requests * kv_heads], and [.., ranked]
};

struct Kv8MassArgs {
  Kv8Cache c;
  const void* q;
  int64_t q_stride;            // elements between tokens
  const float* lse;            // [tokens, heads]
  int64_t tokens;
  const int32_t* starts;       // [requests + 1]
  int heads;
  float scale;
  float* mass;                 // [requests, kv_heads, mass_stride]
  int64_t mass_stride;
};

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t stream);
cudaError_t launch_kv8_decode(const Kv8AttnArgs& a, cudaStream_t stream);
cudaError_t launch_kv8_prefill(const Kv8AttnArgs& a, cudaStream_t stream);
// A tree of drafts (masks) by tiles of 256 rows instead of 40.
cudaError_t launch_kv8_tree(const Kv8AttnArgs& a, cudaStream_t stream);
size_t kv8_tree_workspace_bytes(int64_t requests, int next_n, int heads, int kv_heads, int dim,
                                int64_t bt_stride);
// Whether a tree takes that form, by its rows (nodes * heads of a kv head): from
// three row groups of decode on. us by decode / by tiles, 8 kv heads, one build, inputs not
// in L2:
//   rows                                  64      80      88      96     128     192     256
//   x 128, 16 requests on 4k to 32k    326/390 408/452 470/416 417/363 522/344 816/438 889/369
//          one on 32768                 61/103  68/109  81/111  81/104  97/104 123/116 151/118
//          16 on 512 to 1024            53/51   62/51   62/59   59/54   72/45   99/54  119/56
//          one on 1000                  30/43   35/44   32/45   34/45   33/43   37/47   38/48
//   x 64,  16 requests on 4k to 32k    249/280 326/329 321/290 342/276 452/248 675/325 971/308
//          one on 32768                 52/78   63/88   65/91   66/81   77/75  110/93  128/88
// The limit is that of batches, which have most to lose; a lone request would like 128 to
// 192 rows (up to 30 us), but what a request gets may not depend on the batch.
inline bool kv8_tree_tiles(int next_n, int group) { return next_n * group > 80; }
cudaError_t launch_kv8_mass(const Kv8MassArgs& a, cudaStream_t stream);
cudaError_t launch_kv8_accept(const ds_kv8_layer* layers, int num_layers, const Kv8AcceptArgs& a,
                              cudaStream_t stream);
cudaError_t launch_kv8_evict(Kv8EvictArgs a, void* workspace, cudaStream_t stream);
size_t kv8_evict_workspace_bytes(int64_t requests, int kv_heads, int ranked);
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
cudaError_t launch_pages_shrink(const PageState& s, const int32_t* rows, const int32_t* new_lens,
                                int64_t n, cudaStream_t stream);
cudaError_t launch_pages_compact(const ds_page_pool* pools, int num_pools, const PageState& s,
                                 int32_t* refs_out, int32_t* table_out, int32_t* num_live_out,
                                 void* workspace, cudaStream_t stream);
size_t pages_workspace_bytes(int64_t num_pages, int64_t n);

}  // namespace dsmla
