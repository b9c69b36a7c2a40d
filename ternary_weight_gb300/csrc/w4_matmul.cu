// w4_matmul.cu -- out = x w^T for a few rows x and 4-bit weights w = scale (code - zero), scales for
// groups of 32, 64 or 128 along K.
//
// Bound by the bytes of the codes. Per group:  out += scale (sum (code - zero) x') / up, where
// x' = up x is the row at a power of two of its own, as fp16: bf16 rows keep their bits, fp32 rows
// enter as two fp16 parts (22 bits), each a column of its own. A nibble masked out of its word and
// set into the bits of 1024 is 1024 + code as fp16 (1024 + 16 code for the nibble above, not shifted); one
// subtraction (or multiply-add by 1/16) leaves code - zero exactly. So a word of 8 codes costs 9 instructions
// and is multiplied with 8 columns by m16n8k16 whatever the number of rows. (Codes as fp16 subnormals, with the
// zero point's share of the sum taken off behind it, cost 5, but sums of codes that are not centred cancel:
// 3e-6 of the result where one number of the row is great.)
//
// A warp takes 16 weight rows and a part of K, and streams 16 x 128 codes at a time through a ring of
// its own in shared memory (cp.async), the next tile's behind this one's. The block keeps the rows x'
// in shared memory in the order of the B fragments. Where tiles are few, several warps share one along K and their sums are added in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bitnet_dev.cuh"
#include "w4.h"

namespace bitnet {
namespace {

constexpr int ROWS = 16;               // weight rows of a tile
constexpr int STAGE = ROWS * 64 + ROWS * 8 + ROWS * 4;  // codes, scales, zero points of 16 x 128 weights
constexpr int MAX_SMEM = 227 * 1024;

struct Call {
  W4 w;
  const void* x;
  float* out;
  int m;        // rows of this launch
  int cols;     // m, or 2 m where fp32 rows enter as two parts
  int splits;   // warps that share a tile
  int stages;
  bool bf16;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_bits(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }
// The pairs (0, 4), (1, 5), (2, 6), (3, 7) of a word's codes less their zero point, as fp16; z: 1024 + zero, twice.
__device__ __forceinline__ void centred(uint32_t w, uint32_t z, uint32_t (&p)[4]) {
  const uint32_t w8 = w >> 8, one16 = 0x2c002c00u;  // 1/16, twice
  // 64 + zero: 1024 + zero has steps of 1, 64 + zero of 1/16
  const uint32_t z64 = 0xd400d400u | (z & 0x000f000fu) << 4;  // negative
  p[0] = as_bits(__hsub2(as_half2((w & 0x000f000fu) | 0x64006400u), as_half2(z)));
  p[1] = as_bits(__hfma2(as_half2((w & 0x00f000f0u) | 0x64006400u), as_half2(one16), as_half2(z64)));
  p[2] = as_bits(__hsub2(as_half2((w8 & 0x000f000fu) | 0x64006400u), as_half2(z)));
  p[3] = as_bits(__hfma2(as_half2((w8 & 0x00f000f0u) | 0x64006400u), as_half2(one16), as_half2(z64)));
}

// Shared memory: row factors (2 floats a row), fragments, then the warps' rings.
__host__ __device__ __forceinline__ int frag_bytes(int K, int cols) { return K * cols * 2; }
__host__ __device__ __forceinline__ int align16(int x) { return (x + 15) & ~15; }
__host__ __device__ __forceinline__ int rows_bytes(int K, int m, int cols) { return align16(m * 8) + frag_bytes(K, cols); }

// where word i of lane quad t of a 128-block begins in K: a lane's words of one matrix step stay in one group
template <int G>
__device__ __forceinline__ int word_k(int i, int t) {
  return G == 128 ? t * 32 + i * 8 : G == 64 ? (i >> 1) * 64 + t * 16 + (i & 1) * 8 : i * 32 + t * 8;
}
// pieces of 16 bytes of row r of a stage are exchanged so that reads of 4 and 8 bytes a lane meet no bank twice
__device__ __forceinline__ int swizzle(int r) { return ((r >> 1) & 1) * 2 + ((r >> 2) & 1); }

// The rows as fragments. xf[(block * 4 + word) * cols + col][t]: the 8 numbers that word meets, as
// (0, 4), (1, 5), (2, 6), (3, 7).
template <int G>
__device__ __forceinline__ void load_rows(const Call& c, uint8_t* smem) {
  const int K = c.w.K, tid = threadIdx.x, threads = blockDim.x, lane = tid % 32, warp = tid / 32, warps = threads / 32;
  float2* factor = reinterpret_cast<float2*>(smem);
  uint4* xf = reinterpret_cast<uint4*>(smem + align16(c.m * 8));
  const int parts = c.bf16 ? 1 : 2;
  const auto eight = [&](int m, int k, float (&x)[8]) {
    if (c.bf16) {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(c.x) + (int64_t)m * K + k);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) x[2 * j] = __uint_as_float(u[j] << 16), x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    } else {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(c.x) + (int64_t)m * K + k);
      const float4 a = p[0], b = p[1];
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
  };
  // a row's power of two: its largest number comes to [2^14, 2^15)
  for (int m = warp; m < c.m; m += warps) {
    uint32_t top = 0;
    for (int k = lane * 8; k < K; k += 256) {
      float x[8];
      eight(m, k, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) {
      int e = top == 0 ? 0 : 14 - ((int)(top >> 23) - 127);  // up = 2^e
      e = e > 127 ? 127 : e < -113 ? -113 : e;
      const int half = -e / 2;  // 2^-e in two factors: it may pass the range of one
      factor[m] = make_float2(__int_as_float((half + 127) << 23), __int_as_float((-e - half + 127) << 23));
    }
  }
  __syncthreads();
  const int octets = K / 8;
  for (int i = tid; i < c.m * octets; i += threads) {
    const int m = i / octets, o = i - m * octets, k = o * 8;
    float x[8];
    eight(m, k, x);
    const float2 f = factor[m];
    // up = 1 / (f.x f.y): its exponent from theirs
    const int e = -((int)(__float_as_uint(f.x) >> 23) - 127) - ((int)(__float_as_uint(f.y) >> 23) - 127);
    const float up = __int_as_float((e + 127) << 23);
    const int block = k >> 7, in = k & 127;
    const int t = G == 128 ? in >> 5 : G == 64 ? (in >> 4) & 3 : (in >> 3) & 3;
    const int word = G == 128 ? (in >> 3) & 3 : G == 64 ? (in >> 6) * 2 + ((in >> 3) & 1) : in >> 5;
    float hi[8], lo[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      hi[j] = x[j] * up;
      lo[j] = hi[j] - __half2float(__float2half_rn(hi[j]));
    }
    uint4* to = xf + ((block * 4 + word) * c.cols + m * parts) * 4 + t;
    *to = make_uint4(pack_half2(hi[0], hi[4]), pack_half2(hi[1], hi[5]), pack_half2(hi[2], hi[6]), pack_half2(hi[3], hi[7]));
    if (parts == 2)
      to[4] = make_uint4(pack_half2(lo[0], lo[4]), pack_half2(lo[1], lo[5]), pack_half2(lo[2], lo[6]), pack_half2(lo[3], lo[7]));
  }
  __syncthreads();
}

// NT: eights of columns
template <int G, bool ZEROS, int NT>
__global__ void __launch_bounds__(NT <= 2 ? 256 : 512) w4_matmul_kernel(Call c) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int PER = 128 / G;  // groups of a 128-block
  const int K = c.w.K, N = c.w.N, lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  const int g = lane >> 2, t = lane & 3;
  load_rows<G>(c, smem);
  const float2* factor = reinterpret_cast<const float2*>(smem);
  const uint4* xf = reinterpret_cast<const uint4*>(smem + align16(c.m * 8));
  uint8_t* ring = smem + rows_bytes(K, c.m, c.cols) + warp * c.stages * STAGE;
  float* share = reinterpret_cast<float*>(smem + rows_bytes(K, c.m, c.cols) + warps * c.stages * STAGE);

  const int tiles = (N + ROWS - 1) / ROWS, per_pass = warps / c.splits, split = warp % c.splits;
  const int blocks = K / 128, kb0 = blocks * split / c.splits, kb1 = blocks * (split + 1) / c.splits;
  const int64_t groups = K / G, last_group = (int64_t)N * groups;
  const int first = (int)blockIdx.x * per_pass + warp / c.splits, stride = (int)gridDim.x * per_pass;

  // asks for the block (tile, kb) of weights
  const auto ask = [&](int tile, int kb, int stage) {
    const uint32_t to = smem_u32(ring + stage * STAGE);
    if (tile < tiles) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = g + 8 * h, row = min(tile * ROWS + r, N - 1);
        cp_async_16(to + r * 64 + (t ^ swizzle(r)) * 16, c.w.codes + (int64_t)row * (K / 2) + kb * 64 + t * 16, 16);
      }
      const int r = lane & 15, row = min(tile * ROWS + r, N - 1);
      const int64_t at = row * groups + (int64_t)kb * PER;  // the row's first group in this block
      if (lane < 16) {
        if (PER == 4) {
          cp_async_8(to + 1024 + r * 8, c.w.scales + at);
        } else {  // the aligned word that holds it
          const int64_t even = at & ~1;
          cp_async_4(to + 1024 + r * 8, c.w.scales + even, even + 1 < last_group ? 4 : 2);
        }
      } else if (ZEROS) {
        const int64_t four = at & ~3;
        cp_async_4(to + 1152 + r * 4, c.w.zeros + four, (uint32_t)min((int64_t)4, last_group - four));
      }
    }
    cp_async_commit();
  };

  int ask_tile = first, ask_kb = kb0, ask_stage = 0;
  const auto ask_next = [&]() {
    ask(ask_tile, ask_kb, ask_stage);
    if (++ask_kb >= kb1) ask_kb = kb0, ask_tile += stride;
    if (++ask_stage == c.stages) ask_stage = 0;
  };
  if (kb0 < kb1)
    for (int i = 0; i < c.stages - 1; ++i) ask_next();

  int stage = 0;
  // every warp of the block makes the same number of passes
  for (int tile = first; tile - warp / c.splits < tiles; tile += stride) {
    float tot[NT][4] = {};
    for (int kb = kb0; kb < kb1; ++kb) {
      if (c.stages == 8) cp_async_wait<6>();
      else if (c.stages == 6) cp_async_wait<4>();
      else cp_async_wait<2>();
      __syncwarp();  // the other lanes' copies are in, and they have read the stage that is asked for next
      ask_next();
      const uint8_t* st = ring + stage * STAGE;
      if (++stage == c.stages) stage = 0;
      float scale[2][PER];
      uint32_t zero[2][PER];  // 1024 + zero as two fp16
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = g + 8 * h, row = min(tile * ROWS + r, N - 1);
        const int64_t at = row * groups + (int64_t)kb * PER;
        const uint32_t* sp = reinterpret_cast<const uint32_t*>(st + 1024 + r * 8);
        if (PER == 4) {
          const uint2 v = *reinterpret_cast<const uint2*>(sp);
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
          scale[h][0] = a.x, scale[h][1 % PER] = a.y, scale[h][2 % PER] = b.x, scale[h][3 % PER] = b.y;
        } else {
          const uint32_t v = *sp;
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v));
          if (PER == 2) scale[h][0] = a.x, scale[h][1 % PER] = a.y;
          else scale[h][0] = at & 1 ? a.y : a.x;
        }
        if (ZEROS) {
          const uint32_t v = *reinterpret_cast<const uint32_t*>(st + 1152 + r * 4) >> (8 * (int)(at & 3));
#pragma unroll
          for (int p = 0; p < PER; ++p) zero[h][p] = __byte_perm(v, 0x64646464u, 0x4040 | p | p << 8);
        }
      }
      uint32_t wa[4], wb[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = g + 8 * h, sw = swizzle(r);
        uint32_t(&w)[4] = h ? wb : wa;
        const uint8_t* row = st + r * 64;
        if (G == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(row + (t ^ sw) * 16);
          w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else if (G == 64) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint2 v = *reinterpret_cast<const uint2*>(row + ((2 * p + (t >> 1)) ^ sw) * 16 + (t & 1) * 8);
            w[2 * p] = v.x, w[2 * p + 1] = v.y;
          }
        } else {
#pragma unroll
          for (int p = 0; p < 4; ++p) w[p] = *reinterpret_cast<const uint32_t*>(row + (p ^ sw) * 16 + t * 4);
        }
      }
      float acc[NT][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        constexpr int STEP = 4 / PER;  // words of a group
        if (i % STEP == 0) {
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
        }
        const uint32_t z0 = ZEROS ? zero[0][i / STEP] : 0x64086408u, z1 = ZEROS ? zero[1][i / STEP] : 0x64086408u;
        uint32_t a[4], b[4];
        centred(wa[i], z0, a);
        centred(wb[i], z1, b);
        const uint4* f = xf + (kb * 4 + i) * c.cols * 4 + t;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int col = n * 8 + g;
          const uint4 v = f[(col < c.cols ? col : 0) * 4];
          mma16816(acc[n], a[0], b[0], a[1], b[1], v.x, v.y);
          mma16816(acc[n], a[2], b[2], a[3], b[3], v.z, v.w);
        }
        if (i % STEP == STEP - 1) {
          const int p = i / STEP;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            tot[n][0] = fmaf(scale[0][p], acc[n][0], tot[n][0]);
            tot[n][1] = fmaf(scale[0][p], acc[n][1], tot[n][1]);
            tot[n][2] = fmaf(scale[1][p], acc[n][2], tot[n][2]);
            tot[n][3] = fmaf(scale[1][p], acc[n][3], tot[n][3]);
          }
        }
      }
    }
    if (c.splits > 1) {  // the first warp of a tile adds the others' sums, in order
      float* mine = share + (warp * 32 + lane) * (NT * 4);
      if (split) {
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<float4*>(mine + 4 * n) = make_float4(tot[n][0], tot[n][1], tot[n][2], tot[n][3]);
      }
      __syncthreads();
      if (split == 0) {
        for (int s = 1; s < c.splits; ++s) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float4 v = *reinterpret_cast<const float4*>(mine + s * 32 * (NT * 4) + 4 * n);
            tot[n][0] += v.x, tot[n][1] += v.y, tot[n][2] += v.z, tot[n][3] += v.w;
          }
        }
      }
      __syncthreads();
    }
    if (split == 0 && tile < tiles) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = tile * ROWS + g + 8 * h;
          if (row >= N) continue;
          if (c.bf16) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int m = n * 8 + 2 * t + j;
              if (m < c.m) c.out[(int64_t)m * N + row] = tot[n][2 * h + j] * factor[m].x * factor[m].y;
            }
          } else {
            const int m = n * 4 + t;
            if (m < c.m) c.out[(int64_t)m * N + row] = (tot[n][2 * h] + tot[n][2 * h + 1]) * factor[m].x * factor[m].y;
          }
        }
      }
    }
  }
}

template <int G, bool ZEROS, int NT>
cudaError_t launch(Call c, int num_sms, cudaStream_t st) {
  const int threads = NT <= 2 ? 256 : 512, warps = threads / 32;
  const int rows = rows_bytes(c.w.K, c.m, c.cols);
  c.stages = 8;
  int smem = 0;
  const auto total = [&]() { return rows + warps * c.stages * STAGE + (c.splits > 1 ? warps * 32 * NT * 16 : 0); };
  const int tiles = (c.w.N + ROWS - 1) / ROWS, blocks = c.w.K / 128;
  // warps along K: where tiles would not occupy 16 warps an SM
  c.splits = 1;
  while (c.splits < 8 && (int64_t)tiles * c.splits < (int64_t)num_sms * 16 && blocks >= 2 * c.splits) c.splits *= 2;
  for (c.stages = 8; c.stages > 4 && total() > MAX_SMEM; c.stages -= 2) {
  }
  smem = total();
  if (smem > MAX_SMEM) return cudaErrorInvalidValue;
  auto kernel = w4_matmul_kernel<G, ZEROS, NT>;
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return e;
  int per_sm = 0;
  if (cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem)) return e;
  const int passes = (tiles + warps / c.splits - 1) / (warps / c.splits);
  const int grid = passes < num_sms * per_sm ? passes : num_sms * per_sm;
  kernel<<<grid, threads, smem, st>>>(c);
  return cudaGetLastError();
}

template <int G, bool ZEROS>
cudaError_t by_columns(const Call& c, int num_sms, cudaStream_t st) {
  if (c.cols <= 8) return launch<G, ZEROS, 1>(c, num_sms, st);
  if (c.cols <= 16) return launch<G, ZEROS, 2>(c, num_sms, st);
  if (c.cols <= 32) return launch<G, ZEROS, 4>(c, num_sms, st);
  return launch<G, ZEROS, 8>(c, num_sms, st);
}
template <int G>
cudaError_t by_zeros(const Call& c, int num_sms, cudaStream_t st) {
  return c.w.zeros ? by_columns<G, true>(c, num_sms, st) : by_columns<G, false>(c, num_sms, st);
}

}  // namespace

cudaError_t launch_w4_matmul(const W4& w, const void* x, bool bf16, int64_t M, float* out, int num_sms, cudaStream_t st) {
  const int parts = bf16 ? 1 : 2;
  // rows of a launch: at most 64 columns, and what leaves the rings their place beside the fragments
  int most = 64 / parts;
  const auto fits = [&](int m) {
    const int cols = m * parts, nt = cols <= 8 ? 1 : cols <= 16 ? 2 : cols <= 32 ? 4 : 8, warps = nt <= 2 ? 8 : 16;
    return rows_bytes(w.K, m, cols) + warps * 4 * STAGE + warps * 32 * nt * 16 <= MAX_SMEM;
  };
  while (most > 1 && !fits(most)) --most;
  for (int64_t m0 = 0; m0 < M; m0 += most) {
    const int m = (int)(M - m0 < most ? M - m0 : most);
    Call c{w, nullptr, out + m0 * w.N, m, m * parts, 1, 8, bf16};
    c.x = bf16 ? static_cast<const void*>(static_cast<const __nv_bfloat16*>(x) + m0 * w.K)
               : static_cast<const void*>(static_cast<const float*>(x) + m0 * w.K);
    const cudaError_t e = w.group == 128 ? by_zeros<128>(c, num_sms, st)
                          : w.group == 64 ? by_zeros<64>(c, num_sms, st) : by_zeros<32>(c, num_sms, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace bitnet
