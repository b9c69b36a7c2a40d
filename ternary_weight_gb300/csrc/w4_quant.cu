// w4_quant.cu -- weights to 4-bit codes with a scale (and a zero point) for each group.
//
// Off the timed path (once a model). A warp takes 128 weights of a row, four a lane; a group's extremes
// are joined over its 8, 16 or 32 lanes. Bound by reading the weights.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bitnet_dev.cuh"
#include "w4.h"

namespace bitnet {
namespace {

constexpr int THREADS = 256;
constexpr int kErrRange = -6;  // BITNET_ERANGE

__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
}

template <typename T>
__global__ void __launch_bounds__(THREADS) w4_quant_kernel(const T* __restrict__ w, int64_t chunks, int group,
                                                           uint8_t* __restrict__ codes, uint16_t* __restrict__ scales,
                                                           uint8_t* __restrict__ zeros) {
  const int lane = threadIdx.x % 32, lanes = group / 4;
  const int64_t step = (int64_t)gridDim.x * (THREADS / 32);
  bool bad = false;
  for (int64_t i = (int64_t)blockIdx.x * (THREADS / 32) + threadIdx.x / 32; i < chunks; i += step) {
    float x[4];
    load4(w + i * 128 + lane * 4, x);
    float lo = 0.0f, hi = 0.0f;  // zero is always among what the codes can say
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bad |= !(fabsf(x[j]) < __int_as_float(0x7f800000));
      lo = fminf(lo, x[j]);
      hi = fmaxf(hi, x[j]);
    }
    for (int o = lanes / 2; o >= 1; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const float range = zeros ? __fsub_rn(hi, lo) : fmaxf(hi, -lo);
    const __half h = __float2half_rn(__fdiv_rn(range, zeros ? 15.0f : 7.0f));
    const float s = __half2float(h);
    bad |= !(s < __int_as_float(0x7f800000));
    float zero = 8.0f;
    if (zeros) zero = s > 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f) : 0.0f;
    uint32_t c = 0;
#pragma unroll
    for (int j = 3; j >= 0; --j) {
      const float q = s > 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(x[j], s)), -16.0f), 16.0f) : 0.0f;  // 16: beyond every code
      c = c << 4 | (uint32_t)fminf(fmaxf(q + zero, 0.0f), 15.0f);
    }
    *reinterpret_cast<uint16_t*>(codes + i * 64 + lane * 2) = (uint16_t)c;
    if (lane % lanes == 0) {
      const int64_t g = i * (128 / group) + lane / lanes;
      scales[g] = __half_as_ushort(h);
      if (zeros) zeros[g] = (uint8_t)zero;
    }
  }
  if (bad) record_device_error(kErrRange);
}

}  // namespace

cudaError_t launch_w4_quant(const void* w, bool bf16, int64_t N, int64_t K, int group, uint8_t* codes, uint16_t* scales,
                            uint8_t* zeros, cudaStream_t st) {
  const int64_t chunks = N * (K / 128), blocks = (chunks + THREADS / 32 - 1) / (THREADS / 32);
  const unsigned grid = (unsigned)(blocks < 152 * 64 ? blocks : 152 * 64);
  if (bf16)
    w4_quant_kernel<<<grid, THREADS, 0, st>>>(static_cast<const __nv_bfloat16*>(w), chunks, group, codes, scales, zeros);
  else
    w4_quant_kernel<<<grid, THREADS, 0, st>>>(static_cast<const float*>(w), chunks, group, codes, scales, zeros);
  return cudaGetLastError();
}

cudaError_t read_clear_device_error_w4_quant(int* value) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, g_device_error, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
}

}  // namespace bitnet
