// Arguments of the norm of queries and keys with the position rotation.
#pragma once

#include <stdint.h>
#include <cuda_runtime.h>

#include "ds_sparse_mla.h"
#include "internal.h"

namespace dsmla {

// One side (queries or keys) of the call.
struct NormRopeSide {
  const void* x;
  int64_t x_stride;            // elements between tokens
  void* out;
  int64_t out_stride;
  const void* weight;          // bf16 [norm_dim] or nullptr: no norm
  int heads;
};

struct NormRopeArgs {
  NormRopeSide q, k;
  int64_t tokens;
  int dim, norm_dim, rot_start, rot_dim;
  bool interleaved;
  const int32_t* positions;    // [tokens]
  const float* inv_freq;       // [rot_dim / 2]
  float eps;
};

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream);

}  // namespace dsmla
