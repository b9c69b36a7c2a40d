// kv4_cache.cu -- writing the 4-bit key/value cache and reading it back.
//
// Both kernels move each vector once, and nothing else: bound by bytes, with issue slots next (2.5 of 4 an
// SM and cycle). Why this layout: W lanes share the key and the value of a token and head, so that each
// lane's loads and stores of numbers are 16 bytes and its codes one word after an exchange of nibbles;
// a ninth warp hides the look-up of the places (three dependent loads a row) behind the last chunk's
// work; four blocks an SM cover the latency of the rest. Measured (5 heads x 128, bf16): 73 000 tokens of 6 sequences
// read back in 46.8 us (237 MB, 5.1 TB/s of the measured 6.7; with two blocks an SM 50 us, with a look-up
// by every worker 62 us); 23 165 tokens of 5 prompts written in 32.6 us (75 MB, 2.3 TB/s: the quantisation
// takes the issue slots) and read back in 19.3; one token, or 96, written in 5 us and read in 3.6, the time
// of a launch and a chain of loads.
//
// Quantisation is exact: the code is the correctly rounded quotient (x - base) / step although only
// fp32 is used. An approximate quotient decides unless it lies near a half integer (within several times
// its error); there x is compared with the border step * (n + 1/2) + base itself: the product is exact
// in fp32 (5 + 11 bits), and the sum's rounding error is known exactly.
#include "kv4.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace bitnet {
namespace {

constexpr int WORK = 256, THREADS = WORK + 32;
constexpr float kKvMax = 61440.0f;
constexpr float kNear = 0.5f - 7.62939453125e-6f;       // 2^-17 below a half
constexpr float kNearPlain = 0.5f - 1.52587890625e-5f;  // 2^-16
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
__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// two fp32 lanes an instruction
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

// A block takes chunks of `rows` consecutive packed rows, all heads, one after another. Eight warps move
// the vectors: W lanes take the key and the value of one row and head, lane w dimensions 8 w .. 8 w + 7
// in 16-byte pieces; between that and the words (dimensions w + W n) lies a transpose of 8 x 8 nibbles
// over 8 lanes. A ninth warp looks up the next chunk's places meanwhile (page id, and place in the page;
// negative where a row has none): three dependent loads a row.
constexpr int MAX_ROWS = 16, BATCH = 2, READ_BATCH = 4;

// Where a row's vectors lie: its page (null where it has no place) and its token there.
struct Place {
  uint8_t* page;
  int t, unused;
};
template <int D>
__device__ __forceinline__ void row_places(const Kv4& c, int row0, int max_rows, Place* place, bool* bad) {
  const int i = threadIdx.x - WORK;
  if (i < 0 || i >= max_rows || row0 + i >= c.total_q) return;
  Place p{nullptr, 0, 0};
  const int b = kv4_find(c, row0 + i);
  if (b >= 0) {
    bool wrong = false;
    const Kv4Seq s = kv4_sequence(c, b, &wrong);
    const int k = row0 + i - s.q0, pos = k < s.n ? s.len - s.n + k : -1;
    if (pos >= 0 && !wrong) {
      wrong = true;
      const int id = c.page_table[(int64_t)b * c.max_pages + pos / kKvPage];
      if (id >= 0 && id < c.n_pages) {
        wrong = false;
        p.page = c.pages + (int64_t)id * c.kv_heads * kv4_block_bytes(D);
        p.t = pos % kKvPage;
      }
    }
    if (p.page == nullptr) *bad = true;
  }
  place[i] = p;
}
// The pairs (row, head) of a worker: `WORKERS` pairs on is dr rows and dh heads.
struct Pair {
  int row, h;
  __device__ __forceinline__ void next(int dr, int dh, int heads) {
    row += dr;
    h += dh;
    if (h >= heads) h -= heads, ++row;
  }
};
struct Steps {
  int dr, dh;      // WORKERS / heads, WORKERS % heads
  uint32_t magic;  // worker / heads = umulhi(worker, magic)
};
// The transpose: nibble j of lane i of 8 lanes <-> nibble i of lane j, lanes i and i ^ 1 `gap` apart, in
// three exchanges (halves, bytes, nibbles). Lane w has the codes of dimensions 8 w + k in nibble k. With
// D = 128 lanes of like parity hold nibbles n = w / 2 of words 8 (w & 1) + k, so gap is 2 and lane w ends
// with word 8 (w & 1) + w / 2; with D = 64 gap is 1 and lane w ends with word w.
template <int D>
struct Exchange {
  uint32_t halves, bytes, shift, keep;  // byte selectors, rotation and mask of the lane
  __device__ __forceinline__ explicit Exchange(int w) {
    const int i = D == 128 ? w >> 1 : w;
    halves = i & 4 ? 0x3276 : 0x5410;
    bytes = i & 2 ? 0x3715 : 0x6240;
    shift = i & 1 ? 28 : 4;
    keep = i & 1 ? 0xf0f0f0f0u : 0x0f0f0f0fu;
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t x) const {
    constexpr int gap = D == 128 ? 2 : 1;
    x = __byte_perm(x, __shfl_xor_sync(0xffffffffu, x, 4 * gap), halves);
    x = __byte_perm(x, __shfl_xor_sync(0xffffffffu, x, 2 * gap), bytes);
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, gap);
    return (x & keep) | (__funnelshift_l(y, y, shift) & ~keep);
  }
};
template <int D>
__device__ __forceinline__ int word_of(int w) {
  return D == 128 ? 8 * (w & 1) + (w >> 1) : w;
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

template <int D>
__device__ __forceinline__ uint32_t* key_word(uint8_t* blk, int t, int word) {
  return reinterpret_cast<uint32_t*>(blk) + kv4_rho(t) * (D / 8) + word;
}
template <int D>
__device__ __forceinline__ uint32_t* value_word(uint8_t* blk, int t, int word) {
  constexpr int W = D / 8;
  return reinterpret_cast<uint32_t*>(blk) + (kKvPage + t) * W + (D == 128 && (t & 2) ? word ^ (W / 2) : word);
}
// step and base of token t: keys', then values'
template <int D>
__device__ __forceinline__ uint2* params(uint8_t* blk, int t) {
  return reinterpret_cast<uint2*>(blk + kKvPage * D) + kv4_rho(t);
}

// The codes one by one, with every care: the clamps, and the borders. The numbers are clamped as lo and hi
// are: where lo lies just below 61440, base = fp16(lo) may be 61440 itself, and a number beyond it would
// take a code above the clamped number's.
__device__ __noinline__ uint32_t careful_codes(const float (&x)[8], float base, float step) {
  const float inv = __frcp_rn(step);
  uint32_t word = 0;
#pragma unroll 1
  for (int n = 7; n >= 0; --n) {
    const float y = fminf(fmaxf(x[n], -kKvMax), kKvMax);
    const float t = fminf(fmaxf(__fmul_rn(__fsub_rn(y, base), inv), 0.0f), 15.0f);
    float r = __fsub_rn(__fadd_rn(t, kMagic), kMagic);
    if (fabsf(t - r) > kNear) r = border_code(y, base, step, floorf(t));
    word = word << 4 | (uint32_t)r;
  }
  return word;
}

// Quantises a vector, 8 numbers a lane of W: the lane's codes (number k in nibble k) and the parameters.
template <int W>
__device__ __forceinline__ uint32_t quantise(const float (&x)[8], uint32_t* par) {
  float lo = min_nan(min3_nan(x[0], x[1], x[2]), min3_nan(x[3], x[4], min3_nan(x[5], x[6], x[7])));
  float hi = max_nan(max3_nan(x[0], x[1], x[2]), max3_nan(x[3], x[4], max3_nan(x[5], x[6], x[7])));
#pragma unroll
  for (int o = W / 2; o >= 1; o >>= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float range = __fsub_rn(max_nan(min_nan(hi, kKvMax), -kKvMax), max_nan(min_nan(lo, kKvMax), -kKvMax));
  // range / 15, correctly rounded: one correction by the exact remainder (Markstein)
  float q = __fmul_rn(range, 1.0f / 15.0f);
  q = __fmaf_rn(__fmaf_rn(q, -15.0f, range), 1.0f / 15.0f, q);
  const __half2 sb = __halves2half2(__float2half_rn(q), __float2half_rn(max_nan(min_nan(lo, kKvMax), -kKvMax)));
  const float step = __low2float(sb), base = __high2float(sb);
  *par = *reinterpret_cast<const uint32_t*>(&sb);
  // t = x inv - base inv: within 2^-23 (2 |x inv| + 2 |base inv|) < 2^-16 of the quotient where the base
  // is less than 16 steps off zero; else, and where a quotient may need the clamp or lies near a border,
  // the careful way
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(step));
  const float off = -base * inv;
  float near = 0.0f;  // the largest distance from an integer
  uint32_t word = 0;
  const uint64_t inv2 = f2pack(inv, inv), off2 = f2pack(off, off), magic2 = f2pack(kMagic, kMagic),
                 minus2 = f2pack(-kMagic, -kMagic), neg2 = f2pack(-1.0f, -1.0f);
#pragma unroll
  for (int n = 6; n >= 0; n -= 2) {
    const uint64_t t = fma2(f2pack(x[n], x[n + 1]), inv2, off2), r = add2(t, magic2);
    const float2 d = f2unpack(fma2(add2(r, minus2), neg2, t)), c = f2unpack(r);
    near = fmaxf(near, fmaxf(fabsf(d.x), fabsf(d.y)));
    word = (word * 16u + __float_as_uint(c.y)) * 16u + __float_as_uint(c.x);
  }
  word -= 0x4b400000u * 0x11111111u;  // the eight kMagic
  const bool plain = near < kNearPlain && fabsf(off) < 16.0f && fmaf(lo, inv, off) > -0.49f && fmaf(hi, inv, off) < 15.49f;
  if (!plain) word = step > 0.0f ? careful_codes(x, base, step) : 0;
  return word;
}

template <int D, typename T>
__global__ void __launch_bounds__(THREADS, 4) kv4_append_kernel(Kv4 c, const T* __restrict__ k, const T* __restrict__ v,
                                                                int64_t k_stride, int64_t v_stride, int max_rows,
                                                                Steps steps) {
  constexpr int W = D / 8, WORKERS = WORK / W, BLK = (int)kv4_block_bytes(D);
  __shared__ Place place[2][MAX_ROWS];
  const int w = threadIdx.x % W, worker = threadIdx.x / W;
  const Exchange<D> ex(w);
  const int stride = gridDim.x * max_rows, heads = c.kv_heads;
  Pair first;
  first.row = heads == 1 ? worker : (int)__umulhi((uint32_t)worker, steps.magic);
  first.h = worker - first.row * heads;
  bool bad = false;
  int buf = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * max_rows; row0 < c.total_q; row0 += stride, buf ^= 1) {
    const int rows = (int)min((int64_t)max_rows, c.total_q - row0);
    const T *const kc = k + row0 * k_stride + 8 * w, *const vc = v + row0 * v_stride + 8 * w;
    Eight<T> in[BATCH][2];
    Pair at[BATCH], p = first;
    const auto load = [&]() {
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        at[i] = p;
        p.next(steps.dr, steps.dh, heads);
        if (at[i].row < rows) {
          in[i][0].load(kc + (at[i].row * (int)k_stride + at[i].h * D));
          in[i][1].load(vc + (at[i].row * (int)v_stride + at[i].h * D));
        }
      }
    };
    if (threadIdx.x < WORK) load();  // on their way while the places are looked up
    if (row0 == (int64_t)blockIdx.x * max_rows) row_places<D>(c, (int)row0, max_rows, place[0], &bad);
    __syncthreads();
    if (threadIdx.x >= WORK) {
      if (row0 + stride < c.total_q) row_places<D>(c, (int)(row0 + stride), max_rows, place[buf ^ 1], &bad);
      continue;
    }
    for (int e = 0; e < rows * heads; e += WORKERS * BATCH) {
      if (e) load();
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        if (e + i * WORKERS >= rows * heads) break;
        const bool there = at[i].row < rows;
        float x[8];
        uint2 par;
        in[i][0].get(x);
        const uint32_t kw = ex(quantise<W>(x, &par.x));
        in[i][1].get(x);
        const uint32_t vw = ex(quantise<W>(x, &par.y));
        const Place pl = place[buf][there ? at[i].row : 0];
        if (there && pl.page) {
          uint8_t* blk = pl.page + at[i].h * BLK;
          *key_word<D>(blk, pl.t, word_of<D>(w)) = kw;
          *value_word<D>(blk, pl.t, word_of<D>(w)) = vw;
          if (w == 0) *params<D>(blk, pl.t) = par;
        }
      }
    }
  }
  if (bad) record_device_error(kErrRange);
}

template <int D, typename T>
__global__ void __launch_bounds__(THREADS, 4) kv4_read_kernel(Kv4 c, T* __restrict__ k, T* __restrict__ v,
                                                              int64_t k_stride, int64_t v_stride, int max_rows,
                                                              Steps steps) {
  constexpr int W = D / 8, WORKERS = WORK / W, BLK = (int)kv4_block_bytes(D);
  __shared__ Place place[2][MAX_ROWS];
  const int w = threadIdx.x % W, worker = threadIdx.x / W;
  const Exchange<D> ex(w);
  const int stride = gridDim.x * max_rows, heads = c.kv_heads;
  Pair first;
  first.row = heads == 1 ? worker : (int)__umulhi((uint32_t)worker, steps.magic);
  first.h = worker - first.row * heads;
  bool bad = false;
  int buf = 0;
  row_places<D>(c, blockIdx.x * max_rows, max_rows, place[0], &bad);
  for (int64_t row0 = (int64_t)blockIdx.x * max_rows; row0 < c.total_q; row0 += stride, buf ^= 1) {
    const int rows = (int)min((int64_t)max_rows, c.total_q - row0);
    __syncthreads();
    if (threadIdx.x >= WORK) {
      if (row0 + stride < c.total_q) row_places<D>(c, (int)(row0 + stride), max_rows, place[buf ^ 1], &bad);
      continue;
    }
    T *const kc = k + row0 * k_stride + 8 * w, *const vc = v + row0 * v_stride + 8 * w;
    Pair p = first;
    for (int e = 0; e < rows * heads; e += WORKERS * READ_BATCH) {
      uint32_t kw[READ_BATCH], vw[READ_BATCH];
      uint2 par[READ_BATCH];
      Pair at[READ_BATCH];
#pragma unroll
      for (int i = 0; i < READ_BATCH; ++i) {
        at[i] = p;
        p.next(steps.dr, steps.dh, heads);
        kw[i] = vw[i] = 0;
        par[i] = make_uint2(0, 0);
        if (at[i].row >= rows) continue;
        const Place pl = place[buf][at[i].row];
        if (pl.page) {
          uint8_t* blk = pl.page + at[i].h * BLK;
          kw[i] = *key_word<D>(blk, pl.t, word_of<D>(w));
          vw[i] = *value_word<D>(blk, pl.t, word_of<D>(w));
          par[i] = *params<D>(blk, pl.t);
        } else {
          at[i].row = rows;  // nothing is written
        }
      }
#pragma unroll
      for (int i = 0; i < READ_BATCH; ++i) {
        if (e + i * WORKERS >= rows * heads) break;
        const bool there = at[i].row < rows;
        const auto give = [&](uint32_t word, uint32_t pr, T* to) {
          const uint32_t x = ex(word), even = x & 0x0f0f0f0fu, odd = (x >> 4) & 0x0f0f0f0fu;
          const float2 sb = __half22float2(*reinterpret_cast<const __half2*>(&pr));
          float y[8];
#pragma unroll
          for (int n = 0; n < 8; n += 2) {  // 2^23 + code, exactly
            const uint32_t c0 = __byte_perm(even, 0x4b000000u, 0x7650 | (n >> 1)), c1 = __byte_perm(odd, 0x4b000000u, 0x7650 | (n >> 1));
            const uint64_t code = add2(f2pack(__uint_as_float(c0), __uint_as_float(c1)), f2pack(-8388608.0f, -8388608.0f));
            const float2 t = f2unpack(fma2(code, f2pack(sb.x, sb.x), f2pack(sb.y, sb.y)));
            y[n] = t.x;
            y[n + 1] = t.y;
          }
          if (there) Eight<T>::store(to, y);
        };
        give(kw[i], par[i].x, kc + (at[i].row * (int)k_stride + at[i].h * D));
        give(vw[i], par[i].y, vc + (at[i].row * (int)v_stride + at[i].h * D));
      }
    }
  }
  if (bad) record_device_error(kErrRange);
}

// rows of a chunk: few enough that all SMs have several blocks
int chunk_rows(const Kv4& c) {
  const int r = c.total_q / (4 * 152);
  return r < 1 ? 1 : r > MAX_ROWS ? MAX_ROWS : r;
}
// blocks: four an SM (what fits), each with as many chunks as the next
unsigned blocks(const Kv4& c, int rows) {
  const int64_t chunks = (c.total_q + (int64_t)rows - 1) / rows;
  return (unsigned)(chunks < 4 * 152 ? chunks : 4 * 152);
}
template <int D>
Steps steps_of(const Kv4& c) {
  constexpr int workers = WORK / (D / 8);
  return Steps{workers / c.kv_heads, workers % c.kv_heads,
               (uint32_t)(((uint64_t(1) << 32) + c.kv_heads - 1) / c.kv_heads)};
}

template <int D, typename T>
cudaError_t append(const Kv4& c, const void* k, const void* v, int64_t k_stride, int64_t v_stride, cudaStream_t st) {
  const int rows = chunk_rows(c);
  kv4_append_kernel<D, T><<<blocks(c, rows), THREADS, 0, st>>>(c, static_cast<const T*>(k), static_cast<const T*>(v),
                                                               k_stride, v_stride, rows, steps_of<D>(c));
  return cudaGetLastError();
}
template <int D, typename T>
cudaError_t read(const Kv4& c, void* k, void* v, int64_t k_stride, int64_t v_stride, cudaStream_t st) {
  const int rows = chunk_rows(c);
  kv4_read_kernel<D, T><<<blocks(c, rows), THREADS, 0, st>>>(c, static_cast<T*>(k), static_cast<T*>(v), k_stride,
                                                             v_stride, rows, steps_of<D>(c));
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
