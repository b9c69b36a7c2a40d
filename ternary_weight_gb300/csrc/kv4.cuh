// kv4.cuh -- the 4-bit key/value cache as the kernels see it: page format, batch, and the launch
// declarations that the C-ABI translation unit calls. The format is stated in include/bitnet.h.
//
// Why this format. One block per page and head holds everything that a warp needs of 64 tokens in
// one contiguous, 16-byte aligned piece (8704 bytes at D = 128), which a single bulk copy fetches.
// One step and base per vector let both products run on the bare codes: q.k = step (q.code) +
// base sum(q), and step folds into the softmax weight of a value. Nibble n of word w is dimension
// w + W n, so masking a word with 0x000f000f (and its shifts) gives pairs of codes as they enter
// 16-bit matrix operands, and W lanes that take one nibble each store W neighbouring dimensions.
// The row orders (rho for keys, exchanged halves for wide values) make the matrix-fragment loads
// of kv4_decode.cu free of shared-memory bank conflicts.
#pragma once

#include "bitnet_dev.cuh"

namespace bitnet {

constexpr int kKvPage = 64;      // tokens of a page
constexpr int kErrRange = -6;    // BITNET_ERANGE

__host__ __device__ constexpr int64_t kv4_block_bytes(int dim) { return (int64_t)kKvPage * dim + kKvPage * 8; }
// row of token t (of its page) among the key rows and the parameters
__host__ __device__ __forceinline__ int kv4_rho(int t) { return (t & ~7) | ((t & 3) << 1) | ((t >> 2) & 1); }
// its inverse: the token in row r
__host__ __device__ __forceinline__ int kv4_rho_inv(int r) { return (r & ~7) | ((r >> 1) & 3) | ((r & 1) << 2); }

// cache and batch, passed to kernels by value (checked on the host)
struct Kv4 {
  uint8_t* pages;
  int n_pages, kv_heads;
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* page_table;
  int64_t max_pages;
  int batch, total_q, max_q, max_kv;
};

// One sequence of a batch: its first packed row, its new tokens and its cached tokens.
struct Kv4Seq {
  int q0, n, len;
};

// Reads a sequence's entries and keeps them within the batch's bounds, so that nothing outside the
// arrays is touched whatever they hold; *bad tells that something had to be changed.
__device__ __forceinline__ Kv4Seq kv4_sequence(const Kv4& c, int b, bool* bad) {
  const int a0 = c.cu_q[b], a1 = c.cu_q[b + 1], l = c.kv_len[b];
  Kv4Seq s;
  s.q0 = min(max(a0, 0), c.total_q);
  const int q1 = min(max(a1, s.q0), c.total_q);
  s.n = min(q1 - s.q0, c.max_q);
  s.len = min(max(l, 0), c.max_kv);
  *bad = s.q0 != a0 || s.q0 + s.n != a1 || s.len != l;
  return s;
}

// The sequence that packed row `row` (< total_q) belongs to; -1 if cu_q gives it to none. The first
// guess holds for batches of equal sequences (a decode step), so they search nothing.
__device__ __forceinline__ int kv4_find(const Kv4& c, int row) {
  int lo = min(row / c.max_q, c.batch - 1);
  if (c.cu_q[lo] <= row && row < c.cu_q[lo + 1]) return lo;
  lo = 0;
  int hi = c.batch;  // the last b with cu_q[b] <= row lies in [lo, hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (c.cu_q[mid] <= row)
      lo = mid;
    else
      hi = mid;
  }
  return c.cu_q[lo] <= row && row < c.cu_q[lo + 1] ? lo : -1;
}

// The block of page number `page` (of sequence b, < max_pages) and head h. An id outside the pool
// reads as page 0, and *bad is set.
__device__ __forceinline__ uint8_t* kv4_block(const Kv4& c, int b, int page, int h, int64_t block_bytes, bool* bad) {
  int id = c.page_table[(int64_t)b * c.max_pages + page];
  if (id < 0 || id >= c.n_pages) {
    *bad = true;
    id = 0;
  }
  return c.pages + ((int64_t)id * c.kv_heads + h) * block_bytes;
}

// Softmax weights 2^(c u + off) = 2^(c1 (u - m)) of scores c1 u, m their maximum, in one multiply-add. Its
// rounding, and that of off, is one of 2^-24 of |c1 m|: a common factor of a row's weights while that is small, but one
// that takes them all out of range where |c1 m| passes 2^28. Beyond 2^top c is a power of two below
// c1 with |c m| in [2^(top - 1), 2^top), for which off is exact: scores that far from 0 are apart by units where they
// differ in fp32 at all, and what little they are brought closer is within the error of their sums. The weights are
// 2^lift (a whole number) times what they stand for.
struct Kv4Weight {
  float c, off;
};
__device__ __forceinline__ Kv4Weight kv4_weight(float c1, float m, int top, float lift = 0.0f) {
  if (m == -__builtin_huge_valf()) return {c1, 0.0f};
  Kv4Weight w{c1, fmaf(-c1, m, lift)};
  if (fabsf(w.off) > __int_as_float((127 + top) << 23)) {
    w.c = __int_as_float((253 + top - (int)((__float_as_uint(m) >> 23) & 255u)) << 23);
    w.off = fmaf(-w.c, m, lift);
  }
  return w;
}

cudaError_t launch_kv4_append(const Kv4& c, int dim, const void* k, const void* v, bool bf16, int64_t k_stride,
                              int64_t v_stride, cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4& c, int dim, void* k, void* v, bool bf16, int64_t k_stride, int64_t v_stride,
                            cudaStream_t stream);
cudaError_t read_clear_device_error_kv4_cache(int* value);

// What an attention call has besides the cache and the batch.
struct Kv4Attn {
  const void* q;
  uint16_t* out;  // bf16
  int64_t q_stride, out_stride;
  int q_heads, share;  // share = q_heads / kv_heads
  float scale;
  int window, sinks;   // window 0x7fffffff: all positions
  bool bf16;           // of q
};
int64_t kv4_attention_ws_bytes(const Kv4& c, int dim, int q_heads);
cudaError_t launch_kv4_attention(const Kv4& c, int dim, const Kv4Attn& a, void* workspace, int num_sms,
                                 cudaStream_t stream);

// A few rows a sequence (kv4_decode.cu): sequences with n * share <= rows, rows = 8, 16 or 32. (With 16 it would
// take up to 32: 16 is for batches without longer sequences.)
constexpr int kKvDecodeRows = 32;
int64_t kv4_decode_ws_bytes(const Kv4& c, int dim, int rows);
cudaError_t launch_kv4_decode(const Kv4& c, int dim, const Kv4Attn& a, int rows, void* ws, int num_sms,
                              cudaStream_t stream);
cudaError_t read_clear_device_error_kv4_decode(int* value);
// Many rows (kv4_prompt.cu): sequences with n * share > done_rows.
int64_t kv4_prompt_ws_bytes(const Kv4& c, int dim, int share);
cudaError_t launch_kv4_prompt(const Kv4& c, int dim, const Kv4Attn& a, int done_rows, void* ws, cudaStream_t stream);
cudaError_t read_clear_device_error_kv4_prompt(int* value);

// Attention weight that cached tokens gather (kv4_mass.cu): one fp32 number for each page, head and place.
struct Kv4Mass {
  const float* in;  // n_pages x kv_heads x 64
  float* out;       // the same memory, or apart
  float decay;
  int voters;       // the last rows of a sequence that vote
};
int64_t kv4_mass_ws_bytes(const Kv4& c, int dim, int q_heads, int voters);
cudaError_t launch_kv4_mass(const Kv4& c, int dim, const Kv4Attn& a, const Kv4Mass& m, void* ws, int num_sms, cudaStream_t stream);
cudaError_t read_clear_device_error_kv4_mass(int* value);
cudaError_t read_clear_device_error_kv4_mass_tc(int* value);

// Eviction (kv4_evict.cu).
struct Kv4Evict {
  float* mass;
  const int32_t* into;  // batch x into_pages, or null: in place
  int64_t into_pages;
  int32_t* new_len;     // batch, or null
  int budget, limit, sinks, recent;
};
int64_t kv4_evict_ws_bytes(const Kv4& c, int budget);
cudaError_t launch_kv4_evict(const Kv4& c, int dim, const Kv4Evict& e, void* ws, int num_sms, cudaStream_t stream);
cudaError_t read_clear_device_error_kv4_evict(int* value);

}  // namespace bitnet
