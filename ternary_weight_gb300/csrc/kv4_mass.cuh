// kv4_mass.cuh -- what the kernels of the gathered attention weight share (kv4_mass.cu, kv4_mass_tc.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4.cuh"

namespace bitnet {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// A unit's rows: which vote, and where they stand.
struct Rows {
  int b, h;
  Kv4Seq s;
  int votes;
  __device__ __forceinline__ int position(int i) const { return s.len - votes + i; }  // of voting row i
};
__device__ __forceinline__ Rows rows_of(const Kv4& c, int unit, int voters, bool* bad) {
  Rows r;
  r.b = unit / c.kv_heads;
  r.h = unit - r.b * c.kv_heads;
  bool wrong = false;
  r.s = kv4_sequence(c, r.b, &wrong);
  if (wrong && c.cu_q[r.b] != c.cu_q[r.b + 1]) *bad = true;
  r.votes = min(r.s.n, voters);
  return r;
}
__device__ __forceinline__ float2 params(uint32_t p) { return __half22float2(*reinterpret_cast<const __half2*>(&p)); }
__device__ __forceinline__ bool visible(const Kv4Attn& a, int p, int j) {
  return j <= p && (j > (int64_t)p - a.window || j < a.sinks);
}
// The same with the window's beginning worked out: a row at p sees j where j <= p and (j >= lo or j < sinks).
__device__ __forceinline__ int window_from(const Kv4Attn& a, int p) { return (int)max((int64_t)0, (int64_t)p - a.window + 1); }
__device__ __forceinline__ bool visible(const Kv4Attn& a, int p, int lo, int j) { return j <= p && (j >= lo || j < a.sinks); }
// what rows at positions first .. last see of tokens [j0, j0 + n): 0 nothing, 1 some, 2 all
__device__ __forceinline__ int seen(const Kv4Attn& a, int first, int last, int j0, int n) {
  if (j0 > last || ((int64_t)j0 + n - 1 <= (int64_t)first - a.window && j0 >= a.sinks)) return 0;
  return j0 + n - 1 <= first && (j0 > (int64_t)last - a.window || j0 + n - 1 < a.sinks) ? 2 : 1;
}
// The sum of a row's numbers at its power of two, from that of the bare ones (over the row's W lanes): where it might overflow they
// are added up anew.
template <int W>
__device__ __forceinline__ float row_sum(const float (&x)[8], float sum, float up, uint32_t top) {
  if (!__any_sync(0xffffffffu, top >= 0x7b800000u)) return sum * up;  // none of 2^120 or more
  sum = 0.0f;
#pragma unroll
  for (int n = 0; n < 8; ++n) sum += x[n] * up;
#pragma unroll
  for (int o = W / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}
// A row's constant b, NaN where its largest magnitude (as bits) is none: an infinity's scores may all be -inf, which is what
// tokens have that the row does not see.
__device__ __forceinline__ float or_nan(float b, uint32_t top) { return top < 0x7f800000u ? b : __int_as_float(0x7fffffff); }
constexpr float kLeastA = 7.888609052210118e-31f, kMostA = 3.4028234663852886e38f;  // 2^-100, the greatest
__device__ __forceinline__ uint64_t f2pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f2unpack(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// A kernel that is launched behind another one of the call may start once all blocks of that one have; what it reads of it, it
// reads after the wait, which all its blocks come to.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), unsigned grid, int threads, int smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// joins (m, l) with (m2, l2), maxima of u
__device__ __forceinline__ void join_u(float a, float& m, float& l, float m2, float l2) {
  const float top = fmaxf(m, m2), from = top == kNegInf ? 0.0f : top;
  l = fmaf(l, exp2_approx(a * (m - from)), l2 * exp2_approx(a * (m2 - from)));
  m = top;
}

}  // namespace

// Many rows of a unit (that vote x heads that share a key/value head): kv4_mass_tc.cu. Measured, us, 5 prompts of 1000 to 9000
// tokens, 20 and 5 heads x 128, m16n8k16 and tcgen05: bf16 queries 64 rows 29.9, 49.5; 96 rows 45.4, 50.4; 128 rows 53.3, 51.6;
// 256 rows 87.3, 61.9; fp32 queries 64 rows 49.0, 61.2; 80 rows 58.7, 62.4; 96 rows 63.2, 62.5; 256 rows 133, 94.4. (Other shapes
// go by the same rule; it was not measured for them.)
inline bool mass_on_tc(int64_t rows, bool f32) { return rows > (f32 ? 80 : 96); }
int64_t kv4_mass_tc_ws_bytes(const Kv4& c, int dim, int share, int64_t rows, bool f32);
cudaError_t launch_kv4_mass_tc(const Kv4& c, int dim, const Kv4Attn& a, const Kv4Mass& m, int64_t rows, void* ws, cudaStream_t stream);

}  // namespace bitnet
