// kv4_evict.cu -- eviction: long sequences keep the tokens that gathered most attention weight.
//
// Two kernels, a block for each sequence and head in both. The first finds the least mass that is kept, by
// three passes over the masses that count their digits (11, 11 and 10 bits, from the top), and lists the
// kept tokens in order. The second moves them: their codes, parameters and mass, as they are. In
// place a token only moves to an earlier slot, and a chunk of tokens is read whole before any of it
// is written, so that nothing is overwritten before it has been read.
#include "kv4.cuh"

namespace bitnet {
namespace {

constexpr int THREADS = 1024, WARPS = THREADS / 32;
constexpr int BINS = 2048;

// Masses as whole numbers in the same order; a NaN above all, both zeros alike.
__device__ __forceinline__ uint32_t rank_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Sizes {
  int len;    // cached tokens, -1 where the sequence's entry is out of bounds
  int keeps;  // of them kept
};
__device__ __forceinline__ Sizes sizes_of(const Kv4& c, const Kv4Evict& e, int b) {
  const int l = c.kv_len[b];
  if (l < 0 || l > c.max_kv) return {-1, 0};
  return {l, l > e.limit ? e.budget : l};
}
__device__ __forceinline__ float* mass_of(const Kv4& c, const Kv4Evict& e, int b, int h, int j, bool* bad) {
  int id = c.page_table[(int64_t)b * c.max_pages + j / kKvPage];
  if (id < 0 || id >= c.n_pages) *bad = true, id = 0;
  return e.mass + ((int64_t)id * c.kv_heads + h) * kKvPage + j % kKvPage;
}

__global__ void __launch_bounds__(THREADS) kv4_select_kernel(Kv4 c, Kv4Evict e, int32_t* lens, int32_t* kept, int cap) {
  __shared__ uint32_t bins[BINS];
  __shared__ uint32_t warp_sum[WARPS];
  __shared__ int2 warp_count[WARPS];
  __shared__ uint32_t found[2];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const Sizes s = sizes_of(c, e, b);
  if (h == 0 && tid == 0) lens[b] = s.len;
  if (s.len < 0) {
    if (tid == 0) record_device_error(kErrRange);
    return;
  }
  if (s.len <= e.limit) return;
  bool bad = false;
  const int lo = e.sinks, hi = s.len - e.recent;  // the tokens that are chosen from
  uint32_t want = (uint32_t)(e.budget - e.sinks - e.recent);  // how many of them
  uint32_t least = 0, mask = 0;  // the digits found so far
  if (want == 0) least = 0xffffffffu, mask = 0xffffffffu;
  for (int pass = 0; want > 0 && pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 10 : 11;
    for (int i = tid; i < BINS; i += THREADS) bins[i] = 0;
    __syncthreads();
    for (int j = lo + tid; j < hi; j += THREADS) {
      const uint32_t r = rank_of(*mass_of(c, e, b, h, j, &bad));
      if ((r & mask) == least) atomicAdd(&bins[(r >> shift) & ((1u << width) - 1)], 1u);
    }
    __syncthreads();
    // the digit from which on `want` tokens are counted, from above: threads take two bins each, the highest first
    const uint32_t b1 = bins[BINS - 1 - 2 * tid], b0 = bins[BINS - 2 - 2 * tid];
    uint32_t sum = b1 + b0;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    const uint32_t above = before + sum - b1 - b0;  // tokens of higher digits than this thread's
    if (above < want && want <= above + b1) found[0] = BINS - 1 - 2 * tid, found[1] = want - above;
    if (above + b1 < want && want <= above + b1 + b0) found[0] = BINS - 2 - 2 * tid, found[1] = want - above - b1;
    __syncthreads();
    least |= found[0] << shift;
    mask |= ((1u << width) - 1) << shift;
    want = found[1];
    __syncthreads();
  }
  // `want` is now how many of the tokens at `least` are kept. Each warp takes a run of tokens: it counts, then lists.
  const int per = ((s.len + WARPS - 1) / WARPS + 31) / 32 * 32, j0 = min(warp * per, s.len), j1 = min(j0 + per, s.len);
  const bool none = e.budget == e.sinks + e.recent;
  const auto kind = [&](int j, bool* sure, bool* level) {
    const uint32_t r = j < j1 && j >= lo && j < hi && !none ? rank_of(*mass_of(c, e, b, h, j, &bad)) : 0;
    const bool middle = j >= lo && j < hi;
    *sure = j < j1 && (!middle || (!none && r > least));
    *level = j < j1 && middle && !none && r == least;
  };
  int sures = 0, levels = 0;
  for (int j = j0 + lane; j - lane < j1; j += 32) {
    bool sure, level;
    kind(j, &sure, &level);
    sures += __popc(__ballot_sync(0xffffffffu, sure));
    levels += __popc(__ballot_sync(0xffffffffu, level));
  }
  if (lane == 0) warp_count[warp] = make_int2(sures, levels);
  __syncthreads();
  sures = levels = 0;
  for (int w = 0; w < warp; ++w) sures += warp_count[w].x, levels += warp_count[w].y;
  int32_t* list = kept + ((int64_t)b * c.kv_heads + h) * cap;
  for (int j = j0 + lane; j - lane < j1; j += 32) {
    bool sure, level;
    kind(j, &sure, &level);
    const uint32_t sm = __ballot_sync(0xffffffffu, sure), lm = __ballot_sync(0xffffffffu, level), below = (1u << lane) - 1;
    const int ls = levels + __popc(lm & below), at = sures + __popc(sm & below) + min(ls, (int)want);
    if ((sure || (level && ls < (int)want)) && at < cap) list[at] = j;
    sures += __popc(sm);
    levels += __popc(lm);
  }
  if (bad) record_device_error(kErrRange);
}

// A token's data: lanes take 16 bytes of its key or value row each, the first its parameters and mass too.
template <int D>
__global__ void __launch_bounds__(THREADS) kv4_move_kernel(Kv4 c, Kv4Evict e, const int32_t* lens, const int32_t* kept, int cap) {
  constexpr int BLK = (int)kv4_block_bytes(D), LANES = D / 16, PIECES = LANES / 2, TOKENS = THREADS / LANES, BATCH = 4;
  const int h = blockIdx.x, b = blockIdx.y, part = threadIdx.x % LANES, worker = threadIdx.x / LANES;
  const int len = lens[b];
  if (len < 0) {
    if (h == 0 && threadIdx.x == 0 && e.new_len) e.new_len[b] = c.kv_len[b];
    return;
  }
  const bool cut = len > e.limit;
  const int keeps = cut ? e.budget : len;
  if (h == 0 && threadIdx.x == 0 && e.new_len) e.new_len[b] = keeps;
  if (!cut && !e.into) return;
  if (e.into && keeps > e.into_pages * kKvPage) {  // not one that is cut
    if (threadIdx.x == 0) record_device_error(kErrRange);
    return;
  }
  const int32_t* list = kept + ((int64_t)b * c.kv_heads + h) * cap;
  const int32_t* from = c.page_table + (int64_t)b * c.max_pages;
  const int32_t* to = e.into ? e.into + (int64_t)b * e.into_pages : from;
  bool bad = false;
  for (int r0 = 0; r0 < keeps; r0 += TOKENS * BATCH) {
    uint4 data[BATCH];
    uint2 par[BATCH];
    float mass[BATCH];
    int src[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int r = r0 + i * TOKENS + worker;
      src[i] = -1;
      if (r >= keeps) continue;
      const int j = cut ? list[r] : r;
      if (!e.into && j == r) continue;
      const int id = from[j / kKvPage], t = j % kKvPage;
      if (id < 0 || id >= c.n_pages) {
        bad = true;
        continue;
      }
      src[i] = j;
      const uint8_t* blk = c.pages + ((int64_t)id * c.kv_heads + h) * BLK;
      const int row = part < PIECES ? kv4_rho(t) : kKvPage + t;
      data[i] = *reinterpret_cast<const uint4*>(blk + row * (D / 2) + part % PIECES * 16);
      if (part == 0) par[i] = *reinterpret_cast<const uint2*>(blk + kKvPage * D + kv4_rho(t) * 8);
      if (part == 1) mass[i] = e.mass[((int64_t)id * c.kv_heads + h) * kKvPage + t];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int r = r0 + i * TOKENS + worker;
      if (src[i] < 0) continue;
      const int id = to[r / kKvPage], t = r % kKvPage;
      if (id < 0 || id >= c.n_pages) {
        bad = true;
        continue;
      }
      uint8_t* blk = c.pages + ((int64_t)id * c.kv_heads + h) * BLK;
      const int row = part < PIECES ? kv4_rho(t) : kKvPage + t;
      int piece = part % PIECES;
      if (D == 128 && part >= PIECES && ((src[i] ^ r) & 2)) piece ^= 2;  // the halves of a wide value row
      *reinterpret_cast<uint4*>(blk + row * (D / 2) + piece * 16) = data[i];
      if (part == 0) *reinterpret_cast<uint2*>(blk + kKvPage * D + kv4_rho(t) * 8) = par[i];
      if (part == 1) e.mass[((int64_t)id * c.kv_heads + h) * kKvPage + t] = mass[i];
    }
    __syncthreads();
  }
  if (bad) record_device_error(kErrRange);
}

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }
int cap_of(const Kv4& c, int budget) { return budget < c.max_kv ? budget : c.max_kv; }

}  // namespace

int64_t kv4_evict_ws_bytes(const Kv4& c, int budget) {
  return align256((int64_t)c.batch * 4) + align256((int64_t)c.batch * c.kv_heads * cap_of(c, budget) * 4);
}
cudaError_t launch_kv4_evict(const Kv4& c, int dim, const Kv4Evict& e, void* ws, int num_sms, cudaStream_t st) {
  int32_t* lens = static_cast<int32_t*>(ws);
  int32_t* kept = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + align256((int64_t)c.batch * 4));
  const dim3 grid(c.kv_heads, c.batch);
  kv4_select_kernel<<<grid, THREADS, 0, st>>>(c, e, lens, kept, cap_of(c, e.budget));
  if (cudaError_t err = cudaGetLastError()) return err;
  if (dim == 128)
    kv4_move_kernel<128><<<grid, THREADS, 0, st>>>(c, e, lens, kept, cap_of(c, e.budget));
  else
    kv4_move_kernel<64><<<grid, THREADS, 0, st>>>(c, e, lens, kept, cap_of(c, e.budget));
  return cudaGetLastError();
}

cudaError_t read_clear_device_error_kv4_evict(int* value) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, g_device_error, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
}

}  // namespace bitnet
