// Rotary positions (rope.cu): launch interface of the C ABI (api_diff.cu).
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "fbd.h"

namespace fbd {

struct RopeTensor {
  const void* x;
  void* y;
  int heads;
  int64_t xs[3], ys[3];  // strides of (batch, head, position), in elements
};
struct RopeArgs {
  RopeTensor t[ATTN_ROPE_MAX_TENSORS];
  int64_t B, N;
  int64_t pos_axis, pos_batch;  // strides of pos, in elements
  int d, axes, heads;           // heads: of all tensors together
  int per_thread;               // heads per thread (set by the launcher)
  bool inverse;
};
cudaError_t rope(const RopeArgs& a, int dtype, bool half, const int* pos, const float* freq, const int* axis,
                 cudaStream_t st);

}  // namespace fbd
