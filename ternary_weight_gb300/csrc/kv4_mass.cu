// kv4_mass.cu -- the attention weight that cached tokens gather from a call's queries.
//
// Simple form: a warp for each voting row and head finds the maximum and the sum of its softmax; then a
// block for each page and head adds up its tokens' weights. fp32 throughout.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4.cuh"

namespace bitnet {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float q_number(const Kv4Attn& a, int64_t row, int head, int dim, int d) {
  const int64_t at = row * a.q_stride + (int64_t)head * dim + d;
  return a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at]) : static_cast<const float*>(a.q)[at];
}
__device__ __forceinline__ bool visible(const Kv4Attn& a, int p, int j) {
  return j <= p && ((int64_t)j > (int64_t)p - a.window || j < a.sinks);
}
// scale log2 e (q . k) of the token in place t of a block
template <int D>
__device__ __forceinline__ float score(const uint8_t* blk, int t, const float* q, float qsum, float scale) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(blk) + kv4_rho(t) * (D / 8);
  const __half2 sb = *reinterpret_cast<const __half2*>(blk + kKvPage * D + kv4_rho(t) * 8);
  float s = 0.0f;
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int n = 0; n < 8; ++n) s = fmaf((float)((w[i] >> (4 * n)) & 15u), q[i + D / 8 * n], s);
  // no multiply-add with what follows: both kernels get the same bits
  return __fmul_rn(__fmul_rn(scale, kLog2e), __fmaf_rn(__low2float(sb), s, __fmul_rn(__high2float(sb), qsum)));
}

template <int D>
__global__ void __launch_bounds__(32) kv4_mass_rows(Kv4 c, Kv4Attn a, int voters, float2* stats) {
  __shared__ float q[D];
  const int row = blockIdx.x, head = blockIdx.y, lane = threadIdx.x;
  const int b = kv4_find(c, row);
  if (b < 0) return;
  bool bad = false;
  const Kv4Seq s = kv4_sequence(c, b, &bad);
  const int i = row - s.q0, p = s.len - s.n + i;
  if (i >= s.n || i < s.n - voters) return;
  float sum = 0.0f;
  for (int d = lane; d < D; d += 32) sum += q[d] = q_number(a, row, head, D, d);
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncwarp();
  float m = kNegInf, l = 0.0f;
  for (int j = lane; j <= p; j += 32) {
    if (!visible(a, p, j)) continue;
    const uint8_t* blk = kv4_block(c, b, j / kKvPage, head / a.share, kv4_block_bytes(D), &bad);
    const float x = score<D>(blk, j % kKvPage, q, sum, a.scale);
    const float top = fmaxf(m, x), from = top == kNegInf ? 0.0f : top;  // a NaN is no maximum, but stays in the sum
    l = l * exp2f(m - from) + exp2f(x - from);
    m = top;
  }
  for (int o = 16; o >= 1; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
    const float top = fmaxf(m, m2), from = top == kNegInf ? 0.0f : top;
    l = l * exp2f(m - from) + l2 * exp2f(m2 - from);
    m = top;
  }
  if (lane == 0) stats[(int64_t)row * a.q_heads + head] = make_float2(m, l);
  if (bad) record_device_error(kErrRange);
}

template <int D>
__global__ void __launch_bounds__(64) kv4_mass_pages(Kv4 c, Kv4Attn a, Kv4Mass m, const float2* stats) {
  __shared__ float q[D];
  const int page = blockIdx.x, h = blockIdx.y, b = blockIdx.z, t = threadIdx.x;
  bool bad = false;
  const Kv4Seq s = kv4_sequence(c, b, &bad);
  bad = bad && c.cu_q[b] != c.cu_q[b + 1];
  if (s.n == 0 || page * kKvPage >= s.len) {
    if (bad && page == 0 && h == 0 && t == 0) record_device_error(kErrRange);
    return;
  }
  bool wrong = false;
  const uint8_t* blk = kv4_block(c, b, page, h, kv4_block_bytes(D), &wrong);
  const int j = page * kKvPage + t;
  float votes = 0.0f;
  for (int i = max(0, s.n - m.voters); i < s.n; ++i) {
    const int p = s.len - s.n + i;
    for (int head = h * a.share; head < (h + 1) * a.share; ++head) {
      __syncthreads();
      for (int d = t; d < D; d += 64) q[d] = q_number(a, s.q0 + i, head, D, d);
      __syncthreads();
      if (j >= s.len || !visible(a, p, j)) continue;
      float lanes[32] = {};  // as the first kernel adds them up
      for (int d = 0; d < D; ++d) lanes[d % 32] += q[d];
      for (int o = 16; o >= 1; o >>= 1)
        for (int l = 0; l < o; ++l) lanes[l] += lanes[l + o];
      const float sum = lanes[0];
      const float2 st = stats[(int64_t)(s.q0 + i) * a.q_heads + head];
      votes += exp2f(score<D>(blk, t, q, sum, a.scale) - st.x) / st.y;
    }
  }
  if (j < s.len && !wrong) {
    const int64_t at = ((int64_t)c.page_table[(int64_t)b * c.max_pages + page] * c.kv_heads + h) * kKvPage + t;
    m.out[at] = j < s.len - s.n ? fmaf(m.decay, m.in[at], votes) : votes;
  }
  if (bad || wrong) record_device_error(kErrRange);
}

template <int D>
cudaError_t launch(const Kv4& c, const Kv4Attn& a, const Kv4Mass& m, void* ws, cudaStream_t st) {
  float2* stats = static_cast<float2*>(ws);
  kv4_mass_rows<D><<<dim3(c.total_q, a.q_heads), 32, 0, st>>>(c, a, m.voters, stats);
  if (cudaError_t e = cudaGetLastError()) return e;
  const unsigned pages = (unsigned)((c.max_kv + kKvPage - 1) / kKvPage);
  if (pages == 0) return cudaSuccess;
  kv4_mass_pages<D><<<dim3(pages, c.kv_heads, c.batch), 64, 0, st>>>(c, a, m, stats);
  return cudaGetLastError();
}

}  // namespace

int64_t kv4_mass_ws_bytes(const Kv4& c, int dim, int q_heads, int voters) {
  return ((int64_t)c.total_q * q_heads * 8 + 255) / 256 * 256;
}
cudaError_t launch_kv4_mass(const Kv4& c, int dim, const Kv4Attn& a, const Kv4Mass& m, void* ws, int num_sms, cudaStream_t st) {
  return dim == 128 ? launch<128>(c, a, m, ws, st) : launch<64>(c, a, m, ws, st);
}

cudaError_t read_clear_device_error_kv4_mass(int* value) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, g_device_error, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
}

}  // namespace bitnet
