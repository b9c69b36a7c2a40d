// rope.cu -- rotary positions: pairs of numbers of queries and keys, turned by position * frequency.
//
// Angles. A pair's frequency comes as a 64-bit fixed-point fraction of a turn a position, so that
// position * frequency modulo a turn is one wrapping 64-bit product: exact range reduction whatever the
// position (in fp32 the product alone is off by 0.004 rad at position 131072). The top 32 bits, rounded, go to
// sincospi: the angle is off by 2^-24 half turns at most, as much as an fp32 sine is anyway.
//
// Bound by bytes: every number is read once and written once. A thread takes four pairs of one row
// and keeps their sines and cosines for a run of heads, so that they cost little beside the numbers. Measured: 16001
// rows of 20 and 5 heads x 128, fp32, 70.9 us (410 MB, 5.8 TB/s of the measured 6.8), bf16 53 us (8 bytes a load: 3.9 TB/s); one row 2.2 us.
#include "rope.h"

#include <cuda_bf16.h>

#include "bitnet_dev.cuh"

namespace bitnet {
namespace {

constexpr int THREADS = 256;
constexpr int UNIT = 8;  // numbers of a unit: four pairs, or eight numbers that stay

template <typename T>
struct Four;
template <>
struct Four<float> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = v; }
  __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
  __device__ __forceinline__ void set(const float (&x)[4]) { v = make_float4(x[0], x[1], x[2], x[3]); }
};
template <>
struct Four<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = v; }
  __device__ __forceinline__ void get(float (&x)[4]) const {
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
  }
  __device__ __forceinline__ void set(const float (&x)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    v = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};

// cosine and sine of position * frequency, times the magnitude
__device__ __forceinline__ void turn(uint64_t freq, int position, float magnitude, float* c, float* s) {
  const uint64_t phase = (uint64_t)(int64_t)position * freq;  // modulo a turn
  const float half_turns = (float)(int32_t)((phase + 0x80000000u) >> 32) * 4.656612873077393e-10f;  // 2^-31
  sincospif(half_turns, s, c);
  *c *= magnitude;
  *s *= magnitude;
}

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) rope_kernel(Rope r, int units, int groups, int run) {
  const int64_t all = r.rows * groups * units;
  const int half = r.dims / 2, heads = r.q.heads + r.k.heads;
  for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < all; i += (int64_t)gridDim.x * THREADS) {
    const int64_t rest = i / units;
    const int u = (int)(i - rest * units);
    const int64_t row = rest / groups;
    const int h0 = (int)(rest - row * groups) * run, h1 = min(h0 + run, heads);
    const bool turns = u * UNIT < r.dims;
    // the unit's numbers: x[0..3] and x[4..7] at these places of a head
    const int at0 = turns && !INTERLEAVED ? u * 4 : u * UNIT, at1 = turns && !INTERLEAVED ? half + u * 4 : u * UNIT + 4;
    float c[4], s[4];
    if (turns) {
      const int p = r.positions[row];
#pragma unroll
      for (int j = 0; j < 4; ++j) turn(r.turns[u * 4 + j], p, r.magnitude, &c[j], &s[j]);
    }
    for (int h = h0; h < h1; ++h) {
      const bool is_q = h < r.q.heads;
      const RopeRows& o = is_q ? r.q : r.k;
      const int hh = is_q ? h : h - r.q.heads;
      const T* in = static_cast<const T*>(o.in) + row * o.in_stride + (int64_t)hh * r.head_dim;
      T* out = static_cast<T*>(o.out) + row * o.out_stride + (int64_t)hh * r.head_dim;
      if (!turns) {
        if (in == out) continue;
        Four<T> a, b;
        a.load(in + at0), b.load(in + at1);
        a.store(out + at0), b.store(out + at1);
        continue;
      }
      Four<T> a, b;
      a.load(in + at0), b.load(in + at1);
      float x[4], y[4], p[4], q[4];
      a.get(x), b.get(y);
      if (INTERLEAVED) {  // x: pairs 0 and 1, y: pairs 2 and 3
        p[0] = fmaf(x[0], c[0], -(x[1] * s[0])), p[1] = fmaf(x[1], c[0], x[0] * s[0]);
        p[2] = fmaf(x[2], c[1], -(x[3] * s[1])), p[3] = fmaf(x[3], c[1], x[2] * s[1]);
        q[0] = fmaf(y[0], c[2], -(y[1] * s[2])), q[1] = fmaf(y[1], c[2], y[0] * s[2]);
        q[2] = fmaf(y[2], c[3], -(y[3] * s[3])), q[3] = fmaf(y[3], c[3], y[2] * s[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = fmaf(x[j], c[j], -(y[j] * s[j])), q[j] = fmaf(y[j], c[j], x[j] * s[j]);
      }
      a.set(p), b.set(q);
      a.store(out + at0), b.store(out + at1);
    }
  }
}

template <typename T>
cudaError_t launch(const Rope& r, int num_sms, cudaStream_t st) {
  const int units = r.head_dim / UNIT, heads = r.q.heads + r.k.heads;
  const int64_t full = (int64_t)num_sms * 2048;  // threads that the GPU holds
  // heads that share a thread's angles: as many as leave the GPU full
  int64_t run = r.rows * units * heads / full;
  run = run < 1 ? 1 : run > 8 ? 8 : run;
  const int groups = (heads + (int)run - 1) / (int)run;
  const int64_t need = (r.rows * groups * units + THREADS - 1) / THREADS;
  const unsigned grid = (unsigned)(need < (1 << 30) ? need : (1 << 30));
  if (r.interleaved)
    rope_kernel<T, true><<<grid, THREADS, 0, st>>>(r, units, groups, (int)run);
  else
    rope_kernel<T, false><<<grid, THREADS, 0, st>>>(r, units, groups, (int)run);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const Rope& r, bool bf16, int num_sms, cudaStream_t st) {
  return bf16 ? launch<__nv_bfloat16>(r, num_sms, st) : launch<float>(r, num_sms, st);
}

}  // namespace bitnet
