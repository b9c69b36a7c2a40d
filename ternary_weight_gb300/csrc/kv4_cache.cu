// kv4_cache.cu -- writing the 4-bit key/value cache and reading it back.
//
// Both kernels move each vector once: W = D / 8 neighbouring lanes hold one vector, lane w the
// word w (dimensions w + W n, n = 0..7), so a nibble is one load or store of W neighbouring
// elements. Work items are numbered (row, head, key or value) over the packed rows, so the grid
// holds no idle blocks for short sequences of a ragged batch.
//
// Quantisation is exact: the code is the correctly rounded quotient (x - base) / step although only
// fp32 is used. t = (x - base) * (1 / step) is within 3 roundings, 16 * 3 * 2^-24 < 2^-18, of the
// quotient where it matters (below 16); unless t lies within 2^-17 of a half integer its rounding
// is the quotient's. Near one, x is compared with the border step * (n + 1/2) + base itself: the
// product is exact in fp32 (5 + 11 bits), and the sum's rounding error is known exactly.
#include "kv4.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace bitnet {
namespace {

constexpr int THREADS = 256;
constexpr float kKvMax = 61440.0f;
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: x + kMagic holds rne(x) in its low bits

// NaN-keeping minimum and maximum (fminf and fmaxf drop a NaN)
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// rne((x - base) / step) where the quotient lies next to n + 1/2
__device__ __noinline__ float border_code(float x, float base, float step, float n) {
  const float m = __fmul_rn(n + 0.5f, step);  // exact
  const float s = __fadd_rn(m, base);
  const float bb = __fsub_rn(s, m);  // the sum's error, exactly: m + base = s + err
  const float err = __fadd_rn(__fsub_rn(m, __fsub_rn(s, bb)), __fsub_rn(base, bb));
  bool above = x > s, tie = false;
  if (x == s) above = err < 0.0f, tie = err == 0.0f;
  if (tie) above = ((int)n & 1) != 0;
  return above ? n + 1.0f : n;
}

// Where a work item's vector lies: row, head and kind of the packed arrays, sequence and position in
// the cache. pos < 0: the item has no place (past the end, or a token that the cache cannot hold).
struct Place {
  int64_t row;
  int b, pos, h, is_v;
  bool bad;
};
__device__ __forceinline__ Place place_of(const Kv4& c, int64_t item) {
  const uint32_t per = 2 * c.kv_heads;
  Place p{0, 0, -1, 0, 0, false};
  if (item >= (int64_t)c.total_q * per) return p;
  p.row = item / per;
  const uint32_t hv = (uint32_t)(item - p.row * per);
  p.h = hv >> 1;
  p.is_v = hv & 1;
  p.b = kv4_find(c, (int)p.row);
  if (p.b < 0) return p;
  const Kv4Seq s = kv4_sequence(c, p.b, &p.bad);
  const int i = (int)p.row - s.q0;
  p.pos = i < s.n ? s.len - s.n + i : -1;
  p.bad |= p.pos < 0;
  return p;
}

template <typename T>
__device__ __forceinline__ float load1(const T* p);
template <>
__device__ __forceinline__ float load1<float>(const float* p) { return __ldg(p); }
template <>
__device__ __forceinline__ float load1<__nv_bfloat16>(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16);
}

template <int D, typename T>
__global__ void __launch_bounds__(THREADS) kv4_append_kernel(Kv4 c, const T* __restrict__ k, const T* __restrict__ v,
                                                             int64_t k_stride, int64_t v_stride) {
  constexpr int W = D / 8, VPB = THREADS / W;
  const int w = threadIdx.x % W;
  const Place p = place_of(c, (int64_t)blockIdx.x * VPB + threadIdx.x / W);  // the same for a vector's W lanes
  bool bad = p.bad;
  float x[8];
  if (p.pos >= 0) {
    const T* row = (p.is_v ? v + p.row * v_stride : k + p.row * k_stride) + (int64_t)p.h * D + w;
#pragma unroll
    for (int n = 0; n < 8; ++n) x[n] = load1(row + W * n);
  } else {
#pragma unroll
    for (int n = 0; n < 8; ++n) x[n] = 0.0f;
  }
  float lo = kKvMax, hi = -kKvMax;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    x[n] = max_nan(min_nan(x[n], kKvMax), -kKvMax);
    lo = min_nan(lo, x[n]);
    hi = max_nan(hi, x[n]);
  }
#pragma unroll
  for (int o = W / 2; o >= 1; o >>= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const __half base_h = __float2half_rn(lo), step_h = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
  const float base = __half2float(base_h), step = __half2float(step_h);
  uint32_t word = 0;
  if (step > 0.0f) {
    const float inv = __frcp_rn(step);
    float t[8];
    bool near = false;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      t[n] = fminf(fmaxf(__fmul_rn(__fsub_rn(x[n], base), inv), 0.0f), 15.0f);
      const float m = __fadd_rn(t[n], kMagic);
      near |= fabsf(t[n] - __fsub_rn(m, kMagic)) > 0.5f - 7.62939453125e-6f;
      word |= (__float_as_uint(m) & 15u) << (4 * n);
    }
    if (near) {
      word = 0;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        float r = __fsub_rn(__fadd_rn(t[n], kMagic), kMagic);
        if (fabsf(t[n] - r) > 0.5f - 7.62939453125e-6f)
          r = border_code(x[n], base, step, fminf(floorf(t[n]), 14.0f));
        word |= (uint32_t)r << (4 * n);
      }
    }
  }
  if (p.pos >= 0) {
    const int t = p.pos % kKvPage;
    uint8_t* blk = kv4_block(c, p.b, p.pos / kKvPage, p.h, kv4_block_bytes(D), &bad);
    if (!bad) {
      uint32_t* rows = reinterpret_cast<uint32_t*>(blk);
      if (p.is_v)
        rows[(kKvPage + t) * W + (D == 128 && (t & 2) ? w ^ (W / 2) : w)] = word;
      else
        rows[kv4_rho(t) * W + w] = word;
      if (w == 0)
        reinterpret_cast<__half2*>(blk + kKvPage * D)[2 * kv4_rho(t) + p.is_v] = __halves2half2(step_h, base_h);
    }
  }
  if (bad) record_device_error(kErrRange);
}

__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <int D, typename T>
__global__ void __launch_bounds__(THREADS) kv4_read_kernel(Kv4 c, T* __restrict__ k, T* __restrict__ v,
                                                           int64_t k_stride, int64_t v_stride) {
  constexpr int W = D / 8, VPB = THREADS / W;
  const int w = threadIdx.x % W;
  const Place p = place_of(c, (int64_t)blockIdx.x * VPB + threadIdx.x / W);
  bool bad = p.bad;
  if (p.pos >= 0) {
    const int t = p.pos % kKvPage;
    const uint8_t* blk = kv4_block(c, p.b, p.pos / kKvPage, p.h, kv4_block_bytes(D), &bad);
    const uint32_t* rows = reinterpret_cast<const uint32_t*>(blk);
    const uint32_t word = p.is_v ? rows[(kKvPage + t) * W + (D == 128 && (t & 2) ? w ^ (W / 2) : w)]
                                 : rows[kv4_rho(t) * W + w];
    const __half2 par = reinterpret_cast<const __half2*>(blk + kKvPage * D)[2 * kv4_rho(t) + p.is_v];
    const float step = __low2float(par), base = __high2float(par);
    T* row = (p.is_v ? v + p.row * v_stride : k + p.row * k_stride) + (int64_t)p.h * D + w;
#pragma unroll
    for (int n = 0; n < 8; ++n) store1(row + W * n, __fmaf_rn(step, (float)((word >> (4 * n)) & 15u), base));
  }
  if (bad) record_device_error(kErrRange);
}

template <int D>
int64_t blocks_of(const Kv4& c) {
  constexpr int VPB = THREADS / (D / 8);
  return ((int64_t)c.total_q * 2 * c.kv_heads + VPB - 1) / VPB;
}

template <int D, typename T>
cudaError_t append(const Kv4& c, const void* k, const void* v, int64_t k_stride, int64_t v_stride, cudaStream_t st) {
  kv4_append_kernel<D, T><<<(unsigned)blocks_of<D>(c), THREADS, 0, st>>>(
      c, static_cast<const T*>(k), static_cast<const T*>(v), k_stride, v_stride);
  return cudaGetLastError();
}
template <int D, typename T>
cudaError_t read(const Kv4& c, void* k, void* v, int64_t k_stride, int64_t v_stride, cudaStream_t st) {
  kv4_read_kernel<D, T><<<(unsigned)blocks_of<D>(c), THREADS, 0, st>>>(c, static_cast<T*>(k), static_cast<T*>(v),
                                                                      k_stride, v_stride);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4& c, int dim, const void* k, const void* v, bool bf16, int64_t k_stride,
                              int64_t v_stride, cudaStream_t st) {
  if (dim == 128)
    return bf16 ? append<128, __nv_bfloat16>(c, k, v, k_stride, v_stride, st)
                : append<128, float>(c, k, v, k_stride, v_stride, st);
  return bf16 ? append<64, __nv_bfloat16>(c, k, v, k_stride, v_stride, st)
              : append<64, float>(c, k, v, k_stride, v_stride, st);
}
cudaError_t launch_kv4_read(const Kv4& c, int dim, void* k, void* v, bool bf16, int64_t k_stride, int64_t v_stride,
                            cudaStream_t st) {
  if (dim == 128)
    return bf16 ? read<128, __nv_bfloat16>(c, k, v, k_stride, v_stride, st)
                : read<128, float>(c, k, v, k_stride, v_stride, st);
  return bf16 ? read<64, __nv_bfloat16>(c, k, v, k_stride, v_stride, st)
              : read<64, float>(c, k, v, k_stride, v_stride, st);
}

cudaError_t read_clear_device_error_kv4_cache(int* value) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, g_device_error, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
}

}  // namespace bitnet
