// w4.h -- 4-bit weights with group scales (w4_matmul.cu, w4_quant.cu): what a call has, and the launches.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace bitnet {

struct W4 {
  const uint8_t* codes;    // N x K / 2
  const uint16_t* scales;  // N x K / group, fp16
  const uint8_t* zeros;    // N x K / group, or null (8)
  int N, K, group;
};
constexpr int64_t kW4MaxK = 1 << 15;
cudaError_t launch_w4_matmul(const W4& w, const void* x, bool bf16, int64_t M, float* out, int num_sms, cudaStream_t stream);
cudaError_t launch_w4_quant(const void* w, bool bf16, int64_t N, int64_t K, int group, uint8_t* codes, uint16_t* scales,
                            uint8_t* zeros, cudaStream_t stream);
cudaError_t read_clear_device_error_w4_quant(int* value);

}  // namespace bitnet
