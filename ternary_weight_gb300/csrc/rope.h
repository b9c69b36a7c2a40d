// rope.h -- rotary positions (rope.cu): what a call has, and the launch.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace bitnet {

// One operand (queries or keys): rows of `heads` heads, in and out (the same memory, or apart).
struct RopeRows {
  const void* in;
  void* out;
  int64_t in_stride, out_stride;
  int heads;
};
struct Rope {
  const uint64_t* turns;  // dims / 2
  const int32_t* positions;
  RopeRows q, k;          // k.heads may be 0
  int64_t rows;
  int head_dim, dims;
  float magnitude;
  bool interleaved;
};
cudaError_t launch_rope(const Rope& r, bool bf16, int num_sms, cudaStream_t stream);

}  // namespace bitnet
