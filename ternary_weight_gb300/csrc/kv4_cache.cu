// kv4_cache.cu -- writing the 4-bit key/value cache and reading it back.
//
// Both kernels move each vector once and are bound by bytes.
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

// A block takes `rows` consecutive packed rows, all heads. The rows' places (page id and place in it,
// negative where a row has none) are looked up once, a thread a row; then W lanes take a vector, four
// vectors in flight. Lane w of a vector loads or stores dimensions 8 w .. 8 w + 7 in 16-byte pieces;
// between that and its words (dimensions w + W n) lies a transpose of 8 x 8 nibbles over 8 lanes.
constexpr int MAX_ROWS = 32, BATCH = 4;

__device__ __forceinline__ void row_places(const Kv4& c, int row0, int rows, int2* place, bool* bad) {
  const int i = threadIdx.x;
  if (i >= rows) return;
  int2 p = make_int2(-1, 0);
  const int b = kv4_find(c, row0 + i);
  if (b >= 0) {
    bool wrong = false;
    const Kv4Seq s = kv4_sequence(c, b, &wrong);
    const int k = row0 + i - s.q0, pos = k < s.n ? s.len - s.n + k : -1;
    if (pos >= 0 && !wrong) {
      p.x = c.page_table[(int64_t)b * c.max_pages + pos / kKvPage];
      p.y = pos % kKvPage;
    }
    if (p.x < 0 || p.x >= c.n_pages) *bad = true, p.x = -1;
  }
  place[i] = p;
}
// nibble j of lane i of each group of 8 lanes <-> nibble i of lane j; lanes i and i ^ 1 are `gap` apart
__device__ __forceinline__ uint32_t transpose_nibbles(uint32_t x, int lane, int gap) {
  const int i = lane / gap;
  uint32_t y = __shfl_xor_sync(0xffffffffu, x, 4 * gap);
  x = i & 4 ? (x & 0xffff0000u) | (y >> 16) : (x & 0xffffu) | (y << 16);
  y = __shfl_xor_sync(0xffffffffu, x, 2 * gap);
  x = i & 2 ? (x & 0xff00ff00u) | ((y >> 8) & 0x00ff00ffu) : (x & 0x00ff00ffu) | ((y << 8) & 0xff00ff00u);
  y = __shfl_xor_sync(0xffffffffu, x, gap);
  return i & 1 ? (x & 0xf0f0f0f0u) | ((y >> 4) & 0x0f0f0f0fu) : (x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u);
}
// Lane w has the codes of dimensions 8 w + k in nibble k; the word that it then holds. D = 128: lanes of
// like parity hold nibbles n = w / 2 of words 8 (w & 1) + k, so lane w gets word 8 (w & 1) + w / 2.
template <int D>
__device__ __forceinline__ int word_of(int w) {
  return D == 128 ? 8 * (w & 1) + (w >> 1) : w;
}
template <int D>
__device__ __forceinline__ uint32_t exchange(uint32_t x, int lane) {
  return transpose_nibbles(x, D == 128 ? lane & 15 : lane & 7, D == 128 ? 2 : 1);
}

template <typename T>
struct Eight {  // 8 numbers as they are loaded
  uint4 a;
  __device__ __forceinline__ void load(const T* p) { a = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[2 * k] = __uint_as_float(u[k] << 16), x[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(T* p, const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
      u[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// vector e of a block: row, head, key or value (e < 2^16, m = ceil(2^32 / per))
struct Vec {
  int row, h, is_v;
};
__device__ __forceinline__ Vec vec_of(uint32_t e, uint32_t per, uint32_t m) {
  const uint32_t r = per == 1 ? e : __umulhi(e, m), hv = e - r * per;
  return Vec{(int)r, (int)(hv >> 1), (int)(hv & 1)};
}
template <int D>
__device__ __forceinline__ uint32_t* word_at(uint8_t* blk, int t, int is_v, int word) {
  uint32_t* rows = reinterpret_cast<uint32_t*>(blk);
  constexpr int W = D / 8;
  return rows + (is_v ? (kKvPage + t) * W + (D == 128 && (t & 2) ? word ^ (W / 2) : word) : kv4_rho(t) * W + word);
}

template <int D, typename T>
__global__ void __launch_bounds__(THREADS) kv4_append_kernel(Kv4 c, const T* __restrict__ k, const T* __restrict__ v,
                                                             int64_t k_stride, int64_t v_stride, int max_rows, uint32_t m) {
  constexpr int W = D / 8, WORKERS = THREADS / W;
  __shared__ int2 place[MAX_ROWS];
  const int w = threadIdx.x % W, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * max_rows, rows = min(max_rows, c.total_q - row0);
  const uint32_t per = 2 * c.kv_heads, count = rows * per;
  bool bad = false;
  for (uint32_t e0 = 0; e0 < count; e0 += WORKERS * BATCH) {  // the same for the whole block
    Eight<T> in[BATCH];
    const uint32_t first = e0 + threadIdx.x / W;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const Vec q = vec_of(min(first + i * WORKERS, count - 1), per, m);
      in[i].load((q.is_v ? v + (row0 + q.row) * v_stride : k + (row0 + q.row) * k_stride) + (int64_t)q.h * D + 8 * w);
    }
    if (e0 == 0) {  // the numbers are on their way
      row_places(c, row0, rows, place, &bad);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const uint32_t e = first + i * WORKERS;
      if (e0 + i * WORKERS >= count) break;  // the whole block
      float x[8];
      in[i].get(x);
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
          const float r = __fadd_rn(t[n], kMagic);
          near |= fabsf(t[n] - __fsub_rn(r, kMagic)) > 0.5f - 7.62939453125e-6f;
          word |= (__float_as_uint(r) & 15u) << (4 * n);
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
      word = exchange<D>(word, lane);
      if (e < count) {
        const Vec q = vec_of(e, per, m);
        const int2 p = place[q.row];
        if (p.x >= 0) {
          uint8_t* blk = c.pages + ((int64_t)p.x * c.kv_heads + q.h) * kv4_block_bytes(D);
          *word_at<D>(blk, p.y, q.is_v, word_of<D>(w)) = word;
          if (w == 0)
            reinterpret_cast<__half2*>(blk + kKvPage * D)[2 * kv4_rho(p.y) + q.is_v] = __halves2half2(step_h, base_h);
        }
      }
    }
  }
  if (bad) record_device_error(kErrRange);
}

template <int D, typename T>
__global__ void __launch_bounds__(THREADS) kv4_read_kernel(Kv4 c, T* __restrict__ k, T* __restrict__ v,
                                                           int64_t k_stride, int64_t v_stride, int max_rows, uint32_t m) {
  constexpr int W = D / 8, WORKERS = THREADS / W;
  __shared__ int2 place[MAX_ROWS];
  const int w = threadIdx.x % W, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * max_rows, rows = min(max_rows, c.total_q - row0);
  const uint32_t per = 2 * c.kv_heads, count = rows * per;
  bool bad = false;
  row_places(c, row0, rows, place, &bad);
  __syncthreads();
  for (uint32_t e0 = 0; e0 < count; e0 += WORKERS * BATCH) {
    uint32_t word[BATCH];
    __half2 par[BATCH];
    const uint32_t first = e0 + threadIdx.x / W;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const Vec q = vec_of(min(first + i * WORKERS, count - 1), per, m);
      const int2 p = place[q.row];
      uint8_t* blk = c.pages + ((int64_t)max(p.x, 0) * c.kv_heads + q.h) * kv4_block_bytes(D);
      word[i] = *word_at<D>(blk, p.y, q.is_v, word_of<D>(w));
      par[i] = reinterpret_cast<const __half2*>(blk + kKvPage * D)[2 * kv4_rho(p.y) + q.is_v];
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const uint32_t e = first + i * WORKERS;
      if (e0 + i * WORKERS >= count) break;
      const uint32_t x = exchange<D>(word[i], lane);
      const float step = __low2float(par[i]), base = __high2float(par[i]);
      float y[8];
#pragma unroll
      for (int n = 0; n < 8; ++n) y[n] = __fmaf_rn(step, (float)((x >> (4 * n)) & 15u), base);
      if (e < count) {
        const Vec q = vec_of(e, per, m);
        if (place[q.row].x >= 0)
          Eight<T>::store((q.is_v ? v + (row0 + q.row) * v_stride : k + (row0 + q.row) * k_stride) + (int64_t)q.h * D + 8 * w, y);
      }
    }
  }
  if (bad) record_device_error(kErrRange);
}

// rows of a block: few enough that all SMs have several blocks
int block_rows(const Kv4& c) {
  const int r = c.total_q / 608;
  return r < 1 ? 1 : r > MAX_ROWS ? MAX_ROWS : r;
}
uint32_t per_magic(const Kv4& c) { return (uint32_t)(((uint64_t(1) << 32) + 2 * c.kv_heads - 1) / (2 * c.kv_heads)); }

template <int D, typename T>
cudaError_t append(const Kv4& c, const void* k, const void* v, int64_t k_stride, int64_t v_stride, cudaStream_t st) {
  const int rows = block_rows(c);
  kv4_append_kernel<D, T><<<(unsigned)((c.total_q + (int64_t)rows - 1) / rows), THREADS, 0, st>>>(
      c, static_cast<const T*>(k), static_cast<const T*>(v), k_stride, v_stride, rows, per_magic(c));
  return cudaGetLastError();
}
template <int D, typename T>
cudaError_t read(const Kv4& c, void* k, void* v, int64_t k_stride, int64_t v_stride, cudaStream_t st) {
  const int rows = block_rows(c);
  kv4_read_kernel<D, T><<<(unsigned)((c.total_q + (int64_t)rows - 1) / rows), THREADS, 0, st>>>(
      c, static_cast<T*>(k), static_cast<T*>(v), k_stride, v_stride, rows, per_magic(c));
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
