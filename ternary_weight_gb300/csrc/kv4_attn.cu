// kv4_attn.cu -- attention over the 4-bit key/value cache: one warp for each query row and head.
#include "kv4.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace bitnet {
namespace {

constexpr int WARPS = 4;

template <int D, bool BF16>
__global__ void __launch_bounds__(32 * WARPS) kv4_attn_simple_kernel(Kv4 c, Kv4Attn a, int done_rows) {
  constexpr int W = D / 8;
  __shared__ float qs[WARPS][D];
  __shared__ float ps[WARPS][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * WARPS + warp;
  if (item >= (int64_t)c.total_q * a.q_heads) return;
  const int64_t row = item / a.q_heads;
  const int hq = (int)(item % a.q_heads), h = hq / a.share;
  bool bad = false;
  const int b = kv4_find(c, (int)row);
  if (b < 0) return;
  const Kv4Seq s = kv4_sequence(c, b, &bad);
  if ((int64_t)s.n * a.share <= done_rows) return;
  const int i = (int)row - s.q0;
  const int p = i < s.n ? s.len - s.n + i : -1;
  for (int d = lane; d < D; d += 32) {
    const int64_t at = row * a.q_stride + (int64_t)hq * D + d;
    const float x = BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at]) : static_cast<const float*>(a.q)[at];
    qs[warp][d] = x * a.scale;
  }
  __syncwarp();
  float m = -INFINITY, l = 0.0f, base_sum = 0.0f, acc[D / 32];
  for (int e = 0; e < D / 32; ++e) acc[e] = 0.0f;
  const int low = max((int64_t)0, (int64_t)p - a.window + 1), sink = min(a.sinks, low);
  for (int j0 = 0; j0 <= p; j0 += 32) {
    if (j0 >= sink && j0 + 32 <= low) continue;
    const int j = j0 + lane;
    const bool sees = j <= p && (j >= low || j < sink);
    float sc = -INFINITY, vs = 0.0f, vbase = 0.0f;
    const uint8_t* blk = kv4_block(c, b, j0 / kKvPage, h, kv4_block_bytes(D), &bad);
    if (sees) {
      const int t = j % kKvPage, r = kv4_rho(t);
      const __half2* par = reinterpret_cast<const __half2*>(blk + kKvPage * D) + 2 * r;
      const float ks = __low2float(par[0]), kb = __high2float(par[0]);
      vs = __low2float(par[1]);
      vbase = __high2float(par[1]);
      sc = 0.0f;
      for (int w = 0; w < W; ++w) {
        const uint32_t word = reinterpret_cast<const uint32_t*>(blk)[r * W + w];
        for (int n = 0; n < 8; ++n) sc += qs[warp][w + W * n] * (ks * (float)((word >> (4 * n)) & 15u) + kb);
      }
    }
    float mx = sc;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.0f : mn;
    const float f = expf(m - ref), pr = sees ? expf(sc - ref) : 0.0f;
    m = mn;
    l = l * f + pr;
    base_sum = base_sum * f + (sees ? pr * vbase : 0.0f);
    __syncwarp();
    ps[warp][lane] = sees ? pr * vs : 0.0f;
    __syncwarp();
    for (int e = 0; e < D / 32; ++e) {
      const int d = lane + 32 * e, w = d % W, n = d / W;
      float t = 0.0f;
      for (int jj = 0; jj < 32; ++jj) {
        const int tt = (j0 + jj) % kKvPage;
        const uint32_t word = reinterpret_cast<const uint32_t*>(blk)[(kKvPage + tt) * W + (D == 128 && (tt & 2) ? w ^ (W / 2) : w)];
        t += ps[warp][jj] * (float)((word >> (4 * n)) & 15u);
      }
      acc[e] = acc[e] * f + t;
    }
  }
  for (int o = 16; o; o >>= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, o);
    base_sum += __shfl_xor_sync(0xffffffffu, base_sum, o);
  }
  const bool none = m == -INFINITY && l == 0.0f;
  for (int e = 0; e < D / 32; ++e)
    reinterpret_cast<__nv_bfloat16*>(a.out)[row * a.out_stride + (int64_t)hq * D + lane + 32 * e] =
        __float2bfloat16_rn(none ? 0.0f : (acc[e] + base_sum) / l);
  if (bad) record_device_error(kErrRange);
}

}  // namespace

// The rows that the few-row kernel takes of a sequence, 0 if it is not needed: it is where a sequence
// may have so few; a batch of equal, longer sequences has none.
static int decode_rows(const Kv4& c, int share) {
  const int64_t all = (int64_t)c.max_q * share;
  if (all > kKvDecodeRows && (c.batch == 1 || (int64_t)c.batch * c.max_q == c.total_q)) return 0;
  const int64_t rows = all <= kKvDecodeRows ? all : share;  // with longer sequences beside: single tokens
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= kKvDecodeRows ? kKvDecodeRows : 0;
}

int64_t kv4_attention_ws_bytes(const Kv4& c, int dim, int q_heads) {
  const int rows = decode_rows(c, q_heads / c.kv_heads);
  return rows ? kv4_decode_ws_bytes(c, dim, rows) : 0;
}

cudaError_t launch_kv4_attention(const Kv4& c, int dim, const Kv4Attn& a, void* workspace, int num_sms,
                                 cudaStream_t st) {
  const int rows = decode_rows(c, a.share);
  if (rows) {
    if (cudaError_t e = launch_kv4_decode(c, dim, a, rows, workspace, num_sms, st)) return e;
    if ((int64_t)c.max_q * a.share <= rows) return cudaSuccess;
  }
  const unsigned grid = (unsigned)(((int64_t)c.total_q * a.q_heads + WARPS - 1) / WARPS);
  if (dim == 128)
    a.bf16 ? kv4_attn_simple_kernel<128, true><<<grid, 32 * WARPS, 0, st>>>(c, a, rows)
         : kv4_attn_simple_kernel<128, false><<<grid, 32 * WARPS, 0, st>>>(c, a, rows);
  else
    a.bf16 ? kv4_attn_simple_kernel<64, true><<<grid, 32 * WARPS, 0, st>>>(c, a, rows)
         : kv4_attn_simple_kernel<64, false><<<grid, 32 * WARPS, 0, st>>>(c, a, rows);
  return cudaGetLastError();
}

cudaError_t read_clear_device_error_kv4_attn(int* value) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, g_device_error, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
}

}  // namespace bitnet
