// capi.cu -- the extern "C" boundary of libbitnet_gb300 (declared in include/bitnet.h).
//
// Every entry point validates its arguments on the host before anything is launched and
// returns a status code; no C++ exception crosses the ABI. Device-side state: one error word
// per kernel translation unit (written by bounded waits), the 64 MiB scratch array of
// noalloc.cu (part of the device image, resident on every GPU that loads the library), and
// the device table of each sweep plan, the one cudaMalloc the library makes (in
// bitnet_sweep_plan_create, freed by bitnet_sweep_plan_destroy).
#include "bitnet.h"
#include "bitnet_dev.cuh"
#include "gemm_pair.h"
#include "kv4.cuh"
#include "rope.h"
#include "w4.h"

#include <cmath>
#include <new>
#include <vector>

#include <atomic>
#include <cstdint>

namespace bitnet {
namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxK = 1 << 16;          // staged activation rows must fit shared memory
constexpr int64_t kMaxKTensorCore = 1 << 15; // exact fp32 accumulation bound of the GEMM
// auto dispatch: the few-token tensor-core kernel from this many rows on. The dp4a GEMV's cost
// grows with the rows (every weight word is decoded once per row); the tensor-core kernel's is
// flat up to 16 rows. Measured (N x K = 6912 x 2560, 2560 x 6912, 2560 x 2560, 28672 x 8192):
// the persistent few-row GEMV (K <= 10240) wins up to 4 rows (4 rows: 6.2 against 7.6 us at
// 6912 x 2560) and loses from 5 (9.2 against 7.6 us; 9 rows 16.9 against 7.6). Past K = 10240
// the plain GEMV takes over and loses from 3 rows (8192 x 28672: 48.4 against 39.5 us).
constexpr int64_t kSmallmMinM = 5;           // K <= 10240
constexpr int64_t kSmallmMinMLongK = 3;      // K > 10240
// auto dispatch: the CTA-pair prompt-length kernel beyond one 64-token chunk of the few-token
// kernel. Measured per call, us (N x K = 6912 x 2560 / 2560 x 6912; few-token chunks, one-CTA
// prompt-length kernel, CTA-pair kernel): M = 64: 11.1 / 12.0, 13.6 / 16.4, 12.7 / 13.6;
// M = 96: 14.3 / 14.9, 13.7 / 16.5, 12.7 / 13.6; M = 128: 14.5 / 15.0, 14.0 / 16.7, 12.8 / 13.7;
// M = 192: 27.9 / 18.7, 19.0 / 18.7, 15.9 / 17.2; M = 512: 43.2 / 56.3, 25.2 / 25.8, 21.1 / 21.7;
// M = 4096: 329 / 256, 151 / 164, 127 / 130. The one-CTA kernel stays available when forced.
constexpr int64_t kPairMinM = 65;

// per-device: 0 = unchecked, 1 = sm_103 ok, -1 = unsupported; and SM count
std::atomic<int> g_dev_state[kMaxDevices];
std::atomic<int> g_dev_sms[kMaxDevices];

int check_device(int* num_sms) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return BITNET_EUNSUPPORTED;
  }
  int st = g_dev_state[dev].load(std::memory_order_acquire);
  if (st == 0) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return BITNET_EUNSUPPORTED;
    }
    st = (major == 10 && minor == 3) ? 1 : -1;
    g_dev_sms[dev].store(sms, std::memory_order_relaxed);
    g_dev_state[dev].store(st, std::memory_order_release);
  }
  if (st != 1) return BITNET_EUNSUPPORTED;
  if (num_sms) *num_sms = g_dev_sms[dev].load(std::memory_order_relaxed);
  return BITNET_OK;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int status_of(cudaError_t e) { return e == cudaSuccess ? BITNET_OK : BITNET_ECUDA; }

bool valid_k(int64_t K) { return K >= 128 && K % 128 == 0 && K <= kMaxK; }

}  // namespace
}  // namespace bitnet

using namespace bitnet;

extern "C" {

BITNET_API int bitnet_version(void) { return 100; }

BITNET_API const char* bitnet_strerror(int status) {
  switch (status) {
    case BITNET_OK: return "ok";
    case BITNET_EINVAL: return "invalid argument (null pointer, size out of range, K not a multiple of 128, bad enum)";
    case BITNET_EALIGN: return "misaligned pointer (16-byte alignment required)";
    case BITNET_ECUDA: return "CUDA runtime error or kernel launch failure";
    case BITNET_EUNSUPPORTED: return "unsupported device (an sm_103 / GB300 GPU is required)";
    case BITNET_ETIMEOUT: return "a device-side bounded wait timed out; results are invalid";
    case BITNET_ERANGE: return "an input value outside the operation's supported range (found on the device)";
    default: return "unknown status";
  }
}

BITNET_API int bitnet_pack_i2s(const int8_t* w, uint8_t* wp, int64_t N, int64_t K, int32_t* invalid_count,
                               void* stream) {
  if (!w || !wp || N < 1 || N > INT32_MAX || !valid_k(K)) return BITNET_EINVAL;
  if (!aligned(w, 16) || !aligned(wp, 16) || (invalid_count && !aligned(invalid_count, 4))) return BITNET_EALIGN;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  return status_of(launch_pack_i2s(w, wp, N, K, invalid_count, static_cast<cudaStream_t>(stream)));
}

BITNET_API int bitnet_quant_act(const void* x, int dtype, int64_t M, int64_t K, int8_t* xq, float* act_scale,
                                int32_t* rowsum, void* stream) {
  if (!x || !xq || !act_scale || !rowsum) return BITNET_EINVAL;
  if (dtype != BITNET_F32 && dtype != BITNET_BF16) return BITNET_EINVAL;
  if (M < 1 || M > INT32_MAX || !valid_k(K)) return BITNET_EINVAL;
  if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(act_scale, 4) || !aligned(rowsum, 4)) return BITNET_EALIGN;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  return status_of(launch_quant_act(x, dtype, M, K, xq, act_scale, rowsum, static_cast<cudaStream_t>(stream)));
}

BITNET_API int bitnet_quant_weight(const void* w, int dtype, int mode, int64_t N, int64_t K, uint8_t* wp,
                                   float* w_scale, void* stream) {
  if (!w || !wp || !w_scale) return BITNET_EINVAL;
  if (dtype != BITNET_F32 && dtype != BITNET_BF16) return BITNET_EINVAL;
  if (mode != BITNET_QW_ABSMEAN && mode != BITNET_QW_SIGN) return BITNET_EINVAL;
  if (N < 1 || !valid_k(K) || N > (int64_t(1) << 40) / K) return BITNET_EINVAL;
  if (!aligned(w, 16) || !aligned(wp, 16) || !aligned(w_scale, 4)) return BITNET_EALIGN;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  return status_of(launch_quant_weight(w, dtype == BITNET_BF16, N, K, mode, wp, w_scale, sms,
                                       static_cast<cudaStream_t>(stream)));
}

BITNET_API int bitnet_i2s_matmul_algo(const int8_t* xq, const float* act_scale, const int32_t* rowsum,
                                      const uint8_t* wp, float w_scale, float* out, int32_t* acc_out, int64_t M,
                                      int64_t N, int64_t K, int algo, void* stream) {
  if (!xq || !act_scale || !rowsum || !wp || !out) return BITNET_EINVAL;
  if (M < 1 || M > INT32_MAX || N < 1 || N > INT32_MAX || !valid_k(K)) return BITNET_EINVAL;
  if (algo < BITNET_ALGO_AUTO || algo > BITNET_ALGO_PREFILL_PAIR) return BITNET_EINVAL;
  if (!aligned(xq, 16) || !aligned(wp, 16) || !aligned(act_scale, 4) || !aligned(rowsum, 4) || !aligned(out, 4) ||
      (acc_out && !aligned(acc_out, 4)))
    return BITNET_EALIGN;
  if (algo == BITNET_ALGO_AUTO) {
    // dp4a GEMV for a few tokens (it decodes each weight word once per token row, cheap while
    // the rows are few); from 5 rows (3 past K = 10240) the few-token tensor-core kernel, which
    // decodes each weight once for up to 64 rows; beyond 64 rows the CTA-pair prompt-length
    // kernel (256 weight rows x 128 or 256 tokens per pair of CTAs). The one-CTA prompt-length
    // kernel and the in-kernel-expansion tile GEMM stay available when forced.
    const int64_t smallm_from = K > 10240 ? kSmallmMinMLongK : kSmallmMinM;
    if (K > kMaxKTensorCore || M < smallm_from)
      algo = BITNET_ALGO_GEMV;
    else if (M >= kPairMinM && gemm_pair_supported(M, N, K))
      algo = BITNET_ALGO_PREFILL_PAIR;
    else
      algo = BITNET_ALGO_SMALLM;
  }
  if (algo == BITNET_ALGO_GEMM && (K > kMaxKTensorCore || M > 65535LL * 128)) return BITNET_EINVAL;
  if (algo == BITNET_ALGO_GEMV && M > 65535LL * 8) return BITNET_EINVAL;
  if (algo == BITNET_ALGO_SMALLM && !gemm_smallm_supported(M, K)) return BITNET_EINVAL;
  if (algo == BITNET_ALGO_PREFILL && !gemm_prefill_supported(M, N, K)) return BITNET_EINVAL;
  if (algo == BITNET_ALGO_PREFILL_PAIR && !gemm_pair_supported(M, N, K)) return BITNET_EINVAL;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (algo) {
    case BITNET_ALGO_GEMV:
      e = launch_gemv_i2s(xq, act_scale, rowsum, wp, w_scale, out, acc_out, M, N, K, sms, s);
      break;
    case BITNET_ALGO_SMALLM:
      e = launch_gemm_smallm(xq, act_scale, rowsum, wp, w_scale, out, acc_out, M, N, K, sms, s);
      break;
    case BITNET_ALGO_PREFILL:
      e = launch_gemm_prefill(xq, act_scale, rowsum, wp, w_scale, out, acc_out, M, N, K, sms, s);
      break;
    case BITNET_ALGO_PREFILL_PAIR:
      e = launch_gemm_pair(xq, act_scale, rowsum, wp, w_scale, out, acc_out, M, N, K, sms, s);
      break;
    default:
      e = launch_gemm_i2s_tc(xq, act_scale, rowsum, wp, w_scale, out, acc_out, M, N, K, sms, s);
  }
  return status_of(e);
}

BITNET_API int64_t bitnet_i2s_matmul_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || M > INT32_MAX || N < 1 || N > INT32_MAX || !valid_k(K) || K > kMaxKTensorCore) return BITNET_EINVAL;
  return gemm_ws_bytes(M, N, K);
}

BITNET_API int bitnet_i2s_matmul_ws(const int8_t* xq, const float* act_scale, const int32_t* rowsum, const uint8_t* wp,
                                    float w_scale, float* out, int32_t* acc_out, int64_t M, int64_t N, int64_t K,
                                    void* workspace, int64_t workspace_bytes, void* stream) {
  if (!xq || !act_scale || !rowsum || !wp || !out || !workspace) return BITNET_EINVAL;
  if (M < 1 || M > INT32_MAX || N < 1 || N > INT32_MAX || !valid_k(K) || K > kMaxKTensorCore) return BITNET_EINVAL;
  if (workspace_bytes < gemm_ws_bytes(M, N, K)) return BITNET_EINVAL;
  if (!aligned(xq, 16) || !aligned(wp, 16) || !aligned(act_scale, 4) || !aligned(rowsum, 4) || !aligned(out, 4) ||
      (acc_out && !aligned(acc_out, 4)) || !aligned(workspace, 256))
    return BITNET_EALIGN;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  return status_of(launch_gemm_tc_ws(xq, act_scale, rowsum, wp, w_scale, out, acc_out, M, N, K, workspace, sms,
                                     static_cast<cudaStream_t>(stream)));
}

BITNET_API int bitnet_i2s_matmul(const int8_t* xq, const float* act_scale, const int32_t* rowsum,
                                 const uint8_t* wp, float w_scale, float* out, int32_t* acc_out, int64_t M,
                                 int64_t N, int64_t K, void* stream) {
  return bitnet_i2s_matmul_algo(xq, act_scale, rowsum, wp, w_scale, out, acc_out, M, N, K, BITNET_ALGO_AUTO,
                                stream);
}

BITNET_API int bitnet_w2a8_linear_group_ex(const void* x, int dtype, int64_t M, int64_t K, int count,
                                           const uint8_t* const* wp, const float* w_scale, const int64_t* N,
                                           float* const* out, int32_t* const* acc_out, int8_t* xq, float* act_scale,
                                           int32_t* rowsum, int prefetch_count, const void* const* prefetch_ptr,
                                           const int64_t* prefetch_bytes, void* stream) {
  if (!x || !wp || !w_scale || !N || !out) return BITNET_EINVAL;
  if (dtype != BITNET_F32 && dtype != BITNET_BF16) return BITNET_EINVAL;
  if (count < 1 || count > kMaxGroupLinears) return BITNET_EINVAL;
  if (M < 1 || M > INT32_MAX || !valid_k(K)) return BITNET_EINVAL;
  if (prefetch_count < 0 || prefetch_count > kMaxPrefetch) return BITNET_EINVAL;
  if (prefetch_count > 0 && (!prefetch_ptr || !prefetch_bytes)) return BITNET_EINVAL;
  if (!aligned(x, 16)) return BITNET_EALIGN;
  for (int l = 0; l < count; ++l) {
    if (!wp[l] || !out[l] || N[l] < 1 || N[l] > INT32_MAX) return BITNET_EINVAL;
    if (!aligned(wp[l], 16) || !aligned(out[l], 4) || (acc_out && acc_out[l] && !aligned(acc_out[l], 4)))
      return BITNET_EALIGN;
  }
  Prefetch pf{};
  for (int p = 0; p < prefetch_count; ++p) {
    if (!prefetch_ptr[p] || prefetch_bytes[p] < 0) return BITNET_EINVAL;
    if (!aligned(prefetch_ptr[p], 16)) return BITNET_EALIGN;
    pf.ptr[p] = prefetch_ptr[p];
    pf.bytes[p] = prefetch_bytes[p];
  }
  pf.count = prefetch_count;
  int64_t total_rows = 0;
  for (int l = 0; l < count; ++l) total_rows += N[l];
  const bool single_launch = (M == 1 && gemv_group_supported(K) && total_rows <= INT32_MAX);
  if (!single_launch && (!xq || !act_scale || !rowsum)) return BITNET_EINVAL;
  if ((xq && !aligned(xq, 16)) || (act_scale && !aligned(act_scale, 4)) || (rowsum && !aligned(rowsum, 4)))
    return BITNET_EALIGN;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (single_launch) {
    LinearSet set{};
    for (int l = 0; l < count; ++l) {
      set.wp[l] = wp[l];
      set.out[l] = out[l];
      set.acc[l] = acc_out ? acc_out[l] : nullptr;
      set.w_scale[l] = w_scale[l];
      set.N[l] = (int)N[l];
    }
    set.count = count;
    return status_of(launch_gemv_group(x, dtype == BITNET_BF16, set, QuantOut{xq, act_scale, rowsum}, pf, K, sms, s));
  }
  if (cudaError_t e = launch_quant_act(x, dtype, M, K, xq, act_scale, rowsum, s)) return status_of(e);
  for (int l = 0; l < count; ++l) {
    int st = bitnet_i2s_matmul_algo(xq, act_scale, rowsum, wp[l], w_scale[l], out[l], acc_out ? acc_out[l] : nullptr,
                                    M, N[l], K, BITNET_ALGO_AUTO, stream);
    if (st != BITNET_OK) return st;
  }
  return BITNET_OK;
}

BITNET_API int bitnet_w2a8_linear_group(const void* x, int dtype, int64_t M, int64_t K, int count,
                                        const uint8_t* const* wp, const float* w_scale, const int64_t* N,
                                        float* const* out, int32_t* const* acc_out, int8_t* xq, float* act_scale,
                                        int32_t* rowsum, void* stream) {
  return bitnet_w2a8_linear_group_ex(x, dtype, M, K, count, wp, w_scale, N, out, acc_out, xq, act_scale, rowsum, 0,
                                     nullptr, nullptr, stream);
}

BITNET_API int bitnet_w2a8_linear(const void* x, int dtype, int64_t M, int64_t K, const uint8_t* wp, float w_scale,
                                  int64_t N, float* out, int32_t* acc_out, int8_t* xq, float* act_scale,
                                  int32_t* rowsum, void* stream) {
  int32_t* accs[1] = {acc_out};
  return bitnet_w2a8_linear_group(x, dtype, M, K, 1, &wp, &w_scale, &N, &out, accs, xq, act_scale, rowsum, stream);
}

BITNET_API int bitnet_ffn_act_quant(const float* gate, const float* up, const float* gamma, float eps, int64_t M,
                                    int64_t F, int8_t* xq, float* act_scale, int32_t* rowsum, float* inner_out,
                                    void* stream) {
  if (!gate || !up || !gamma || !xq || !act_scale || !rowsum) return BITNET_EINVAL;
  if (M < 1 || M > INT32_MAX || !valid_k(F) || F > kFfnMaxF) return BITNET_EINVAL;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return BITNET_EINVAL;
  if (!aligned(gate, 16) || !aligned(up, 16) || !aligned(gamma, 16) || !aligned(xq, 16) || !aligned(act_scale, 4) ||
      !aligned(rowsum, 4) || (inner_out && !aligned(inner_out, 16)))
    return BITNET_EALIGN;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  return status_of(launch_ffn_act_quant(FfnIn{gate, up, gamma, eps}, M, F, xq, act_scale, rowsum, inner_out,
                                        static_cast<cudaStream_t>(stream)));
}

namespace {
bool valid_ffn_shape(int64_t M, int64_t K, int64_t F) {
  return M >= 1 && M <= INT32_MAX && valid_k(K) && valid_k(F) && F <= kFfnMaxF;
}
// Workspace the FFN block uses: none. Its projections take the workspace-free kernels of auto
// dispatch at every M: the CTA-pair prompt-length kernel measured faster than the expand-once
// workspace path at every size tried (per projection, N x K = 6912 x 2560 / 2560 x 6912: M = 1024
// 41.7 / 44.0 against 52.6 / 58.0 us, M = 2048 63.9 / 86.0 against 82.9 / 94.5, M = 4096 127 /
// 130 against 145 / 151, M = 8192 252 / 218 against 269 / 272).
int64_t ffn_ws_bytes(int64_t, int64_t, int64_t) { return 0; }
}  // namespace

BITNET_API int64_t bitnet_w2a8_ffn_workspace_size(int64_t M, int64_t K, int64_t F) {
  if (!valid_ffn_shape(M, K, F)) return BITNET_EINVAL;
  return ffn_ws_bytes(M, K, F);
}

BITNET_API int bitnet_w2a8_ffn(const void* x, int dtype, int64_t M, int64_t K, int64_t F, const uint8_t* wp_gate,
                               float a_gate, const uint8_t* wp_up, float a_up, const uint8_t* wp_down, float a_down,
                               const float* gamma, float eps, float* gate_out, float* up_out, float* out, int8_t* xq,
                               float* act_scale, int32_t* rowsum, void* workspace, int64_t workspace_bytes,
                               void* stream) {
  if (!x || !wp_gate || !wp_up || !wp_down || !gamma || !gate_out || !up_out || !out) return BITNET_EINVAL;
  if (dtype != BITNET_F32 && dtype != BITNET_BF16) return BITNET_EINVAL;
  if (!valid_ffn_shape(M, K, F)) return BITNET_EINVAL;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return BITNET_EINVAL;
  const bool single = M == 1 && gemv_group_supported(K) && gemv_group_supported(F);
  if (!single && (!xq || !act_scale || !rowsum)) return BITNET_EINVAL;
  const int64_t ws_need = ffn_ws_bytes(M, K, F);
  if (workspace && workspace_bytes < ws_need) return BITNET_EINVAL;
  if (!aligned(x, 16) || !aligned(wp_gate, 16) || !aligned(wp_up, 16) || !aligned(wp_down, 16) ||
      !aligned(gamma, 16) || !aligned(gate_out, 16) || !aligned(up_out, 16) || !aligned(out, 4))
    return BITNET_EALIGN;
  if ((xq && !aligned(xq, 16)) || (act_scale && !aligned(act_scale, 4)) || (rowsum && !aligned(rowsum, 4)) ||
      (workspace && !aligned(workspace, 256)))
    return BITNET_EALIGN;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const FfnIn ffn{gate_out, up_out, gamma, eps};
  if (single) {
    // two launches: the gate/up group (quantising x), then the down projection whose input
    // row is the sub-normed, quantised inner activation computed in its own prologue
    LinearSet gu{};
    gu.wp[0] = wp_gate, gu.wp[1] = wp_up;
    gu.out[0] = gate_out, gu.out[1] = up_out;
    gu.w_scale[0] = a_gate, gu.w_scale[1] = a_up;
    gu.N[0] = gu.N[1] = (int)F;
    gu.count = 2;
    if (cudaError_t e = launch_gemv_group(x, dtype == BITNET_BF16, gu, QuantOut{}, Prefetch{}, K, sms, s))
      return status_of(e);
    LinearSet dn{};
    dn.wp[0] = wp_down;
    dn.out[0] = out;
    dn.w_scale[0] = a_down;
    dn.N[0] = (int)K;
    dn.count = 1;
    return status_of(launch_gemv_group_ffn(ffn, dn, QuantOut{xq, act_scale, rowsum}, Prefetch{}, F, sms, s));
  }
  auto matmul = [&](const uint8_t* wp, float a, float* o, int64_t N, int64_t Kd) -> int {
    return bitnet_i2s_matmul_algo(xq, act_scale, rowsum, wp, a, o, nullptr, M, N, Kd, BITNET_ALGO_AUTO, stream);
  };
  if (cudaError_t e = launch_quant_act(x, dtype, M, K, xq, act_scale, rowsum, s)) return status_of(e);
  if (int st = matmul(wp_gate, a_gate, gate_out, F, K)) return st;
  if (int st = matmul(wp_up, a_up, up_out, F, K)) return st;
  if (cudaError_t e = launch_ffn_act_quant(ffn, M, F, xq, act_scale, rowsum, nullptr, s)) return status_of(e);
  return matmul(wp_down, a_down, out, K, F);
}

// ---- the persistent sweep: a plan owns device copies of the group table and of the per-CTA
// slices (built once on the host) ----
struct bitnet_sweep_plan_s {
  bitnet::SweepGroup* table;   // device, n_groups entries
  bitnet::SweepSlice* slices;  // device, n_slices entries (one per CTA)
  int n_groups;
  int n_slices;
  int dtype;
  int device;
};

BITNET_API int bitnet_sweep_plan_create(const bitnet_linear_group* groups, int n_groups, int dtype,
                                        bitnet_sweep_plan* plan) {
  if (!plan) return BITNET_EINVAL;
  *plan = nullptr;
  if (!groups || n_groups < 1 || n_groups > (1 << 20)) return BITNET_EINVAL;
  if (dtype != BITNET_F32 && dtype != BITNET_BF16) return BITNET_EINVAL;
  std::vector<SweepGroup> host((size_t)n_groups);
  int64_t rows = 0, bytes = 0;
  for (int g = 0; g < n_groups; ++g) {
    const bitnet_linear_group& in = groups[g];
    if (!in.x || in.count < 1 || in.count > kMaxGroupLinears) return BITNET_EINVAL;
    if (!valid_k(in.K) || !gemv_sweep_supported(in.K)) return BITNET_EINVAL;
    if (!aligned(in.x, 16)) return BITNET_EALIGN;
    SweepGroup& out = host[(size_t)g];
    out = SweepGroup{};
    out.x = in.x;
    out.K = (int)in.K;
    out.count = in.count;
    out.row0 = (int)rows;
    out.byte0 = bytes;
    for (int l = 0; l < in.count; ++l) {
      if (!in.wp[l] || !in.out[l] || in.N[l] < 1 || in.N[l] > INT32_MAX) return BITNET_EINVAL;
      if (!aligned(in.wp[l], 16) || !aligned(in.out[l], 4)) return BITNET_EALIGN;
      out.wp[l] = in.wp[l];
      out.out[l] = in.out[l];
      out.w_scale[l] = in.w_scale[l];
      out.N[l] = (int)in.N[l];
      rows += in.N[l];
      if (rows > INT32_MAX) return BITNET_EINVAL;
    }
    out.rows = (int)(rows - out.row0);
    bytes += (int64_t)out.rows * (in.K / 4);
    sweep_fill_layout(out);
  }
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  // one CTA per SM (fewer if there are fewer rows), each with a byte-balanced slice
  const int n_slices = (int)(rows < sms ? rows : sms);
  std::vector<SweepSlice> slices((size_t)n_slices);
  sweep_slices(host.data(), n_groups, (int)rows, bytes, n_slices, slices.data());
  auto* p = new (std::nothrow) bitnet_sweep_plan_s{};
  if (!p) return BITNET_ECUDA;
  const size_t tb = sizeof(SweepGroup) * (size_t)n_groups, sb = sizeof(SweepSlice) * (size_t)n_slices;
  const bool ok = cudaGetDevice(&p->device) == cudaSuccess &&
                  cudaMalloc(reinterpret_cast<void**>(&p->table), tb) == cudaSuccess &&
                  cudaMalloc(reinterpret_cast<void**>(&p->slices), sb) == cudaSuccess &&
                  cudaMemcpy(p->table, host.data(), tb, cudaMemcpyHostToDevice) == cudaSuccess &&
                  cudaMemcpy(p->slices, slices.data(), sb, cudaMemcpyHostToDevice) == cudaSuccess;
  if (!ok) {
    cudaFree(p->table);
    cudaFree(p->slices);
    delete p;
    return BITNET_ECUDA;
  }
  p->n_groups = n_groups;
  p->n_slices = n_slices;
  p->dtype = dtype;
  *plan = p;
  return BITNET_OK;
}

BITNET_API int bitnet_sweep_plan_run(bitnet_sweep_plan plan, void* stream) {
  if (!plan) return BITNET_EINVAL;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BITNET_ECUDA;
  if (dev != plan->device) return BITNET_EINVAL;
  return status_of(launch_gemv_sweep(plan->table, plan->n_groups, plan->slices, plan->n_slices,
                                     plan->dtype == BITNET_BF16, static_cast<cudaStream_t>(stream)));
}

BITNET_API int bitnet_sweep_plan_destroy(bitnet_sweep_plan plan) {
  if (!plan) return BITNET_OK;
  const cudaError_t e1 = cudaFree(plan->table);
  const cudaError_t e2 = cudaFree(plan->slices);
  delete plan;
  return e1 == cudaSuccess && e2 == cudaSuccess ? BITNET_OK : BITNET_ECUDA;
}

// ---- the 4-bit key/value cache ----
namespace {
constexpr int64_t kKvMaxHeads = 1024, kKvMaxBatch = 65535, kKvMaxPages = 1 << 24, kKvMaxShare = 128;

bool valid_kv4_sizes(int64_t n_pages, int64_t kv_heads, int64_t head_dim) {
  return n_pages >= 1 && n_pages <= INT32_MAX && kv_heads >= 1 && kv_heads <= kKvMaxHeads &&
         (head_dim == 64 || head_dim == 128);
}
// the checks that every call makes of its cache and batch; fills *out
int check_kv4(const bitnet_kv4_cache* cache, const bitnet_kv4_batch* b, Kv4* out) {
  if (!cache || !b || !cache->pages || !b->cu_q || !b->kv_len || !b->page_table) return BITNET_EINVAL;
  if (!valid_kv4_sizes(cache->n_pages, cache->kv_heads, cache->head_dim)) return BITNET_EINVAL;
  if (b->batch < 1 || b->batch > kKvMaxBatch || b->max_pages < 1 || b->max_pages > kKvMaxPages || b->total_q < 0 ||
      b->total_q > INT32_MAX || b->max_q < 1 || b->max_q > INT32_MAX || b->max_kv < 0 ||
      b->max_kv > b->max_pages * kKvPage)
    return BITNET_EINVAL;
  // rows x heads of a call fit the grids (2^31 blocks of at least 16 vectors)
  if (b->total_q > (int64_t(1) << 33) / cache->kv_heads) return BITNET_EINVAL;
  // and a warp's share of the pages its counters
  if ((b->max_kv + kKvPage - 1) / kKvPage > (int64_t(1) << 40) / (b->batch * cache->kv_heads)) return BITNET_EINVAL;
  if (!aligned(cache->pages, 16) || !aligned(b->cu_q, 4) || !aligned(b->kv_len, 4) || !aligned(b->page_table, 4))
    return BITNET_EALIGN;
  *out = Kv4{static_cast<uint8_t*>(cache->pages), (int)cache->n_pages, cache->kv_heads, b->cu_q, b->kv_len,
             b->page_table, b->max_pages, (int)b->batch, (int)b->total_q, (int)b->max_q, (int)b->max_kv};
  return BITNET_OK;
}
// a row stride in elements: at least `least`, at most 2^26 (16 rows' offsets are 32-bit), and a multiple
// of 16 bytes
int check_stride(int64_t stride, int64_t least, int64_t elem_bytes) {
  if (stride < least || stride > (int64_t(1) << 26)) return BITNET_EINVAL;
  return stride * elem_bytes % 16 == 0 ? BITNET_OK : BITNET_EALIGN;
}
int check_kv4_rows(const Kv4& c, int dim, const void* k, const void* v, int dtype, int64_t k_stride, int64_t v_stride) {
  if (!k || !v || (dtype != BITNET_F32 && dtype != BITNET_BF16)) return BITNET_EINVAL;
  const int64_t eb = dtype == BITNET_BF16 ? 2 : 4;
  if (int st = check_stride(k_stride, (int64_t)c.kv_heads * dim, eb)) return st;
  if (int st = check_stride(v_stride, (int64_t)c.kv_heads * dim, eb)) return st;
  return aligned(k, 16) && aligned(v, 16) ? BITNET_OK : BITNET_EALIGN;
}
bool valid_q_heads(int64_t q_heads, int64_t kv_heads) {
  return q_heads >= kv_heads && q_heads % kv_heads == 0 && q_heads / kv_heads <= kKvMaxShare;
}
// rows of a key/value head are counted in 32 bits
bool valid_q_rows(const Kv4& c, int64_t q_heads) {
  return (int64_t)c.total_q * (q_heads / c.kv_heads) <= INT32_MAX - 4096;
}
}  // namespace

BITNET_API int64_t bitnet_kv4_cache_bytes(int64_t n_pages, int64_t kv_heads, int64_t head_dim) {
  if (!valid_kv4_sizes(n_pages, kv_heads, head_dim)) return BITNET_EINVAL;
  return n_pages * kv_heads * kv4_block_bytes((int)head_dim);
}

BITNET_API int bitnet_kv4_append(const bitnet_kv4_cache* cache, const bitnet_kv4_batch* batch, const void* k,
                                 const void* v, int dtype, int64_t k_stride, int64_t v_stride, void* stream) {
  Kv4 c{};
  if (int st = check_kv4(cache, batch, &c)) return st;
  if (int st = check_kv4_rows(c, cache->head_dim, k, v, dtype, k_stride, v_stride)) return st;
  if (c.total_q == 0) return BITNET_OK;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  return status_of(launch_kv4_append(c, cache->head_dim, k, v, dtype == BITNET_BF16, k_stride, v_stride,
                                     static_cast<cudaStream_t>(stream)));
}

BITNET_API int bitnet_kv4_read(const bitnet_kv4_cache* cache, const bitnet_kv4_batch* batch, void* k, void* v,
                               int dtype, int64_t k_stride, int64_t v_stride, void* stream) {
  Kv4 c{};
  if (int st = check_kv4(cache, batch, &c)) return st;
  if (int st = check_kv4_rows(c, cache->head_dim, k, v, dtype, k_stride, v_stride)) return st;
  if (c.total_q == 0) return BITNET_OK;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  return status_of(launch_kv4_read(c, cache->head_dim, k, v, dtype == BITNET_BF16, k_stride, v_stride,
                                   static_cast<cudaStream_t>(stream)));
}

BITNET_API int64_t bitnet_kv4_attention_workspace_size(const bitnet_kv4_cache* cache, const bitnet_kv4_batch* batch,
                                                       int64_t q_heads) {
  Kv4 c{};
  if (int st = check_kv4(cache, batch, &c)) return st;
  if (!valid_q_heads(q_heads, c.kv_heads) || !valid_q_rows(c, q_heads)) return BITNET_EINVAL;
  return kv4_attention_ws_bytes(c, cache->head_dim, (int)q_heads);
}

BITNET_API int bitnet_kv4_attention(const bitnet_kv4_cache* cache, const bitnet_kv4_batch* batch, const void* q,
                                    int dtype, int64_t q_heads, int64_t q_stride, float scale, int64_t window,
                                    int64_t sinks, void* out, int64_t out_stride, void* workspace,
                                    int64_t workspace_bytes, void* stream) {
  Kv4 c{};
  if (int st = check_kv4(cache, batch, &c)) return st;
  if (!q || !out || (dtype != BITNET_F32 && dtype != BITNET_BF16)) return BITNET_EINVAL;
  if (!valid_q_heads(q_heads, c.kv_heads) || !std::isfinite(scale)) return BITNET_EINVAL;
  if (window < 0 || window > INT32_MAX || sinks < 0 || sinks > INT32_MAX) return BITNET_EINVAL;
  const int64_t row = q_heads * cache->head_dim;
  if (int st = check_stride(q_stride, row, dtype == BITNET_BF16 ? 2 : 4)) return st;
  if (int st = check_stride(out_stride, row, 2)) return st;
  if (!valid_q_rows(c, q_heads)) return BITNET_EINVAL;
  const int64_t need = kv4_attention_ws_bytes(c, cache->head_dim, (int)q_heads);
  if (need > 0 && (!workspace || workspace_bytes < need)) return BITNET_EINVAL;
  if (!aligned(q, 16) || !aligned(out, 16) || (workspace && !aligned(workspace, 256))) return BITNET_EALIGN;
  if (c.total_q == 0) return BITNET_OK;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  const Kv4Attn a{q, static_cast<uint16_t*>(out), q_stride, out_stride, (int)q_heads, (int)(q_heads / c.kv_heads),
                  scale, window ? (int)window : INT32_MAX, window ? (int)sinks : 0, dtype == BITNET_BF16};
  return status_of(launch_kv4_attention(c, cache->head_dim, a, workspace, sms,
                                        static_cast<cudaStream_t>(stream)));
}

namespace {
// what attention and the weights that it gathers have in common; fills *out
int check_kv4_queries(const Kv4& c, int dim, const void* q, int dtype, int64_t q_heads, int64_t q_stride, float scale,
                      int64_t window, int64_t sinks, Kv4Attn* out) {
  if (!q || (dtype != BITNET_F32 && dtype != BITNET_BF16)) return BITNET_EINVAL;
  if (!valid_q_heads(q_heads, c.kv_heads) || !std::isfinite(scale)) return BITNET_EINVAL;
  if (window < 0 || window > INT32_MAX || sinks < 0 || sinks > INT32_MAX) return BITNET_EINVAL;
  if (int st = check_stride(q_stride, q_heads * dim, dtype == BITNET_BF16 ? 2 : 4)) return st;
  if (!valid_q_rows(c, q_heads)) return BITNET_EINVAL;
  *out = Kv4Attn{q, nullptr, q_stride, 0, (int)q_heads, (int)(q_heads / c.kv_heads), scale,
                 window ? (int)window : INT32_MAX, window ? (int)sinks : 0, dtype == BITNET_BF16};
  return aligned(q, 16) ? BITNET_OK : BITNET_EALIGN;
}
// columns (two a row of fp32) are counted in 32 bits
bool valid_mass_rows(const Kv4& c, int64_t q_heads) { return (int64_t)c.total_q * (q_heads / c.kv_heads) <= (1 << 30) - 64; }
int voters_of(int64_t voters) { return voters ? (int)voters : INT32_MAX; }
}  // namespace

BITNET_API int64_t bitnet_kv4_mass_bytes(int64_t n_pages, int64_t kv_heads) {
  if (!valid_kv4_sizes(n_pages, kv_heads, 64)) return BITNET_EINVAL;
  return n_pages * kv_heads * kKvPage * 4;
}

BITNET_API int64_t bitnet_kv4_attention_mass_workspace_size(const bitnet_kv4_cache* cache, const bitnet_kv4_batch* batch,
                                                            int64_t q_heads, int64_t voters) {
  Kv4 c{};
  if (int st = check_kv4(cache, batch, &c)) return st;
  if (!valid_q_heads(q_heads, c.kv_heads) || !valid_mass_rows(c, q_heads)) return BITNET_EINVAL;
  if (voters < 0 || voters > INT32_MAX) return BITNET_EINVAL;
  return kv4_mass_ws_bytes(c, cache->head_dim, (int)q_heads, voters_of(voters));
}

BITNET_API int bitnet_kv4_attention_mass(const bitnet_kv4_cache* cache, const bitnet_kv4_batch* batch, const void* q,
                                         int dtype, int64_t q_heads, int64_t q_stride, float scale, int64_t window,
                                         int64_t sinks, int64_t voters, float decay, const float* mass,
                                         float* mass_out, void* workspace, int64_t workspace_bytes, void* stream) {
  Kv4 c{};
  Kv4Attn a{};
  if (int st = check_kv4(cache, batch, &c)) return st;
  if (!mass || !mass_out || !std::isfinite(decay) || voters < 0 || voters > INT32_MAX) return BITNET_EINVAL;
  if (int st = check_kv4_queries(c, cache->head_dim, q, dtype, q_heads, q_stride, scale, window, sinks, &a)) return st;
  if (!valid_mass_rows(c, q_heads)) return BITNET_EINVAL;
  const int64_t need = kv4_mass_ws_bytes(c, cache->head_dim, (int)q_heads, voters_of(voters));
  if (need > 0 && (!workspace || workspace_bytes < need)) return BITNET_EINVAL;
  const uintptr_t from = reinterpret_cast<uintptr_t>(mass), to = reinterpret_cast<uintptr_t>(mass_out);
  const uintptr_t bytes = (uintptr_t)bitnet_kv4_mass_bytes(c.n_pages, c.kv_heads);
  if (from != to && from < to + bytes && to < from + bytes) return BITNET_EINVAL;  // they overlap
  if (!aligned(mass, 16) || !aligned(mass_out, 16) || (workspace && !aligned(workspace, 256))) return BITNET_EALIGN;
  if (c.total_q == 0) return BITNET_OK;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  return status_of(launch_kv4_mass(c, cache->head_dim, a, Kv4Mass{mass, mass_out, decay, voters_of(voters)}, workspace,
                                   sms, static_cast<cudaStream_t>(stream)));
}

BITNET_API int64_t bitnet_kv4_evict_workspace_size(const bitnet_kv4_cache* cache, const bitnet_kv4_batch* batch,
                                                   int64_t budget) {
  Kv4 c{};
  if (int st = check_kv4(cache, batch, &c)) return st;
  if (budget < 1 || budget > INT32_MAX) return BITNET_EINVAL;
  return kv4_evict_ws_bytes(c, (int)budget);
}

BITNET_API int bitnet_kv4_evict(const bitnet_kv4_cache* cache, const bitnet_kv4_batch* batch, float* mass,
                                int64_t budget, int64_t limit, int64_t sinks, int64_t recent, const int32_t* into,
                                int64_t into_pages, int32_t* new_len, void* workspace, int64_t workspace_bytes,
                                void* stream) {
  Kv4 c{};
  if (int st = check_kv4(cache, batch, &c)) return st;
  if (!mass || budget < 1 || limit < budget || limit > INT32_MAX) return BITNET_EINVAL;
  if (sinks < 0 || sinks > budget || recent < 0 || recent > budget - sinks) return BITNET_EINVAL;
  if (into && (into_pages < 1 || into_pages > kKvMaxPages || into_pages * kKvPage < budget)) return BITNET_EINVAL;
  if (!aligned(new_len, 4)) return BITNET_EALIGN;
  // lengths that are written over those of other sequences: the blocks of a cluster would read different ones
  const uintptr_t from = reinterpret_cast<uintptr_t>(c.kv_len), to = reinterpret_cast<uintptr_t>(new_len), bytes = (uintptr_t)c.batch * 4;
  if (new_len && from != to && from < to + bytes && to < from + bytes) return BITNET_EINVAL;
  const int64_t need = kv4_evict_ws_bytes(c, (int)budget);
  if (!workspace || workspace_bytes < need) return BITNET_EINVAL;
  if (!aligned(mass, 16) || !aligned(workspace, 256) || !aligned(into, 4)) return BITNET_EALIGN;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  const Kv4Evict e{mass, into, into_pages, new_len, (int)budget, (int)limit, (int)sinks, (int)recent};
  return status_of(launch_kv4_evict(c, cache->head_dim, e, workspace, sms, static_cast<cudaStream_t>(stream)));
}

// ---- rotary positions ----
namespace {
constexpr int64_t kRopeMaxDim = 1024, kRopeMaxHeads = 1 << 17;
constexpr double kTwoPi = 6.283185307179586476925;

// one operand's checks; `out` is its input or apart from it
int check_rope_rows(const void* in, int64_t in_stride, const void* out, int64_t out_stride, int64_t least, int64_t eb) {
  if (!in || !out) return BITNET_EINVAL;
  if (int st = check_stride(in_stride, least, eb)) return st;
  if (int st = check_stride(out_stride, least, eb)) return st;
  if (in == out && in_stride != out_stride) return BITNET_EINVAL;
  return aligned(in, 16) && aligned(out, 16) ? BITNET_OK : BITNET_EALIGN;
}
// Whether two operands' rows share bytes. Rows of one stride may lie between each other's (slices of a fused row); those of two
// strides have to lie apart as a whole.
bool rows_overlap(const void* a, int64_t a_stride, int64_t a_bytes, const void* b, int64_t b_stride, int64_t b_bytes, int64_t rows) {
  const int64_t d = (int64_t)(reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a));
  if (d >= (rows - 1) * a_stride + a_bytes || -d >= (rows - 1) * b_stride + b_bytes) return false;
  if (rows == 1 || a_stride != b_stride) return true;
  // row i of b begins d - k stride beyond row i + k of a
  const int64_t k = d >= 0 ? d / a_stride : -((-d + a_stride - 1) / a_stride), beyond = d - k * a_stride;
  return (k > -rows && k < rows && beyond < a_bytes) || (k + 1 > -rows && k + 1 < rows && a_stride - beyond < b_bytes);
}
}  // namespace

BITNET_API int bitnet_rope_turns(int64_t dims, double base, int scaling, double factor, double original, double low,
                                 double high, uint64_t* turns, float* magnitude) {
  if (!turns || !magnitude || dims < 2 || dims > kRopeMaxDim || dims % 2) return BITNET_EINVAL;
  if (scaling < BITNET_ROPE_NONE || scaling > BITNET_ROPE_BY_WAVELENGTH) return BITNET_EINVAL;
  if (!std::isfinite(base) || !(base > 1.0)) return BITNET_EINVAL;
  if (scaling != BITNET_ROPE_NONE && (!std::isfinite(factor) || !(factor >= 1.0))) return BITNET_EINVAL;
  const bool ends = scaling == BITNET_ROPE_BY_PARTS || scaling == BITNET_ROPE_BY_WAVELENGTH;
  if (ends && (!std::isfinite(original) || !std::isfinite(low) || !std::isfinite(high) || !(original > 0.0) ||
               !(low > 0.0) || !(high > low)))
    return BITNET_EINVAL;
  if (scaling == BITNET_ROPE_NTK) {
    if (dims == 2) return BITNET_EINVAL;
    base *= std::pow(factor, (double)dims / (double)(dims - 2));
    if (!std::isfinite(base)) return BITNET_EINVAL;
  }
  const auto at = [&](double n) { return dims / 2 * std::log(original / (kTwoPi * n)) / std::log(base); };
  double a = 0.0, b = 0.0;
  if (scaling == BITNET_ROPE_BY_PARTS) {
    a = std::fmax(std::floor(at(high)), 0.0);
    b = std::fmin(std::ceil(at(low)), (double)(dims - 1));
  }
  for (int64_t i = 0; i < dims / 2; ++i) {
    double f = std::pow(base, -2.0 * (double)i / (double)dims);
    if (scaling == BITNET_ROPE_LINEAR) f /= factor;
    if (scaling == BITNET_ROPE_BY_PARTS) {
      const double r = std::fmin(std::fmax(((double)i - a) / std::fmax(b - a, 0.001), 0.0), 1.0);
      f = f * (1.0 - r) + f / factor * r;
    }
    if (scaling == BITNET_ROPE_BY_WAVELENGTH) {
      const double t = std::fmin(std::fmax((original * f / kTwoPi - low) / (high - low), 0.0), 1.0);
      f *= t + (1.0 - t) / factor;
    }
    // f <= 1: less than a turn, and the product below 2^62
    turns[i] = (uint64_t)std::llrint(f / kTwoPi * 18446744073709551616.0);
  }
  *magnitude = scaling == BITNET_ROPE_BY_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return BITNET_OK;
}

BITNET_API int bitnet_rope(const bitnet_rope_table* table, const int32_t* positions, int64_t rows, const void* q,
                           int64_t q_heads, int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k,
                           int64_t kv_heads, int64_t k_stride, void* k_out, int64_t k_out_stride, int64_t head_dim,
                           int dtype, void* stream) {
  if (!table || !table->turns || !positions || rows < 0 || rows > INT32_MAX) return BITNET_EINVAL;
  if (dtype != BITNET_F32 && dtype != BITNET_BF16) return BITNET_EINVAL;
  if (head_dim < 8 || head_dim > kRopeMaxDim || head_dim % 8) return BITNET_EINVAL;
  if (table->dims < 8 || table->dims > head_dim || table->dims % 8 || !std::isfinite(table->magnitude))
    return BITNET_EINVAL;
  if (table->layout != BITNET_ROPE_HALF && table->layout != BITNET_ROPE_INTERLEAVED) return BITNET_EINVAL;
  if (q_heads < 1 || q_heads > kRopeMaxHeads || kv_heads < 0 || kv_heads > kRopeMaxHeads) return BITNET_EINVAL;
  const int64_t eb = dtype == BITNET_BF16 ? 2 : 4;
  if (int st = check_rope_rows(q, q_stride, q_out, q_out_stride, q_heads * head_dim, eb)) return st;
  if (kv_heads)
    if (int st = check_rope_rows(k, k_stride, k_out, k_out_stride, kv_heads * head_dim, eb)) return st;
  if (rows > 0) {  // what is written over another operand, other than in place
    const int64_t qb = q_heads * head_dim * eb, kb = kv_heads * head_dim * eb;
    const auto over = [&](const void* a, int64_t as, int64_t ab, const void* b, int64_t bs, int64_t bb) {
      return rows_overlap(a, as * eb, ab, b, bs * eb, bb, rows);
    };
    if (q_out != q && over(q_out, q_out_stride, qb, q, q_stride, qb)) return BITNET_EINVAL;
    if (kv_heads && ((k_out != k && over(k_out, k_out_stride, kb, k, k_stride, kb)) || over(q_out, q_out_stride, qb, k, k_stride, kb) ||
                     over(k_out, k_out_stride, kb, q, q_stride, qb) || over(q_out, q_out_stride, qb, k_out, k_out_stride, kb)))
      return BITNET_EINVAL;
  }
  if (!aligned(table->turns, 8) || !aligned(positions, 4)) return BITNET_EALIGN;
  if (rows == 0) return BITNET_OK;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  const Rope r{table->turns, positions, {q, q_out, q_stride, q_out_stride, (int)q_heads},
               {k, k_out, k_stride, k_out_stride, (int)kv_heads}, rows, (int)head_dim, table->dims, table->magnitude,
               table->layout == BITNET_ROPE_INTERLEAVED};
  return status_of(launch_rope(r, dtype == BITNET_BF16, sms, static_cast<cudaStream_t>(stream)));
}

// ---- 4-bit weights ----
namespace {
int check_w4(const void* rows, int dtype, int64_t N, int64_t K, int64_t group, const uint8_t* codes,
             const uint16_t* scales, const uint8_t* zeros) {
  if (!rows || !codes || !scales || (dtype != BITNET_F32 && dtype != BITNET_BF16)) return BITNET_EINVAL;
  if (N < 1 || N > INT32_MAX || !valid_k(K) || K > kW4MaxK) return BITNET_EINVAL;
  if (group != 32 && group != 64 && group != 128) return BITNET_EINVAL;
  return aligned(rows, 16) && aligned(codes, 16) && aligned(scales, 16) && aligned(zeros, 16) ? BITNET_OK : BITNET_EALIGN;
}
}  // namespace

BITNET_API int bitnet_w4_quant_weight(const void* w, int dtype, int64_t N, int64_t K, int64_t group, uint8_t* codes,
                                      uint16_t* scales, uint8_t* zeros, void* stream) {
  if (int st = check_w4(w, dtype, N, K, group, codes, scales, zeros)) return st;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  return status_of(launch_w4_quant(w, dtype == BITNET_BF16, N, K, (int)group, codes, scales, zeros,
                                   static_cast<cudaStream_t>(stream)));
}

BITNET_API int bitnet_w4_matmul(const void* x, int dtype, int64_t M, int64_t K, const uint8_t* codes,
                                const uint16_t* scales, const uint8_t* zeros, int64_t N, int64_t group, float* out,
                                void* stream) {
  if (!out || M < 1 || M > INT32_MAX) return BITNET_EINVAL;
  if (int st = check_w4(x, dtype, N, K, group, codes, scales, zeros)) return st;
  if (!aligned(out, 4)) return BITNET_EALIGN;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  const W4 w4{codes, scales, zeros, (int)N, (int)K, (int)group};
  return status_of(launch_w4_matmul(w4, x, dtype == BITNET_BF16, M, out, sms, static_cast<cudaStream_t>(stream)));
}

BITNET_API int bitnet_selftest_wait_timeout(const void* src, int64_t bytes, int32_t max_polls, uint32_t* report,
                                            void* stream) {
  if (!src || !report || !selftest_bytes_ok(bytes) || max_polls < 1 || max_polls > (1 << 20)) return BITNET_EINVAL;
  if (!aligned(src, 16) || !aligned(report, 4)) return BITNET_EALIGN;
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  return status_of(launch_wait_timeout_selftest(src, bytes, (uint32_t)max_polls, report,
                                                static_cast<cudaStream_t>(stream)));
}

BITNET_API int bitnet_last_device_error(void) {
  int sms = 0;
  if (int st = check_device(&sms)) return st;
  if (cudaDeviceSynchronize() != cudaSuccess) return BITNET_ECUDA;
  int status = BITNET_OK;
  cudaError_t (*readers[])(int*) = {read_clear_device_error_gemm, read_clear_device_error_gemm_ws,
                                    read_clear_device_error_gemv_group, read_clear_device_error_smallm,
                                    read_clear_device_error_quant_weight, read_clear_device_error_sweep,
                                    read_clear_device_error_gemv_ring, read_clear_device_error_selftest,
                                    read_clear_device_error_prefill, read_clear_device_error_pair,
                                    read_clear_device_error_kv4_cache, read_clear_device_error_kv4_decode,
                                    read_clear_device_error_kv4_prompt, read_clear_device_error_w4_quant,
                                    read_clear_device_error_kv4_mass, read_clear_device_error_kv4_mass_tc,
                                    read_clear_device_error_kv4_evict};
  for (auto rd : readers) {
    int v = 0;
    if (rd(&v) != cudaSuccess) return BITNET_ECUDA;
    if (v != 0 && status == BITNET_OK) status = v;
  }
  return status;
}

}  // extern "C"
