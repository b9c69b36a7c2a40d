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
// A block keeps the rows x' in shared memory in the order of the B fragments, and takes a run of tiles of 16
// weight rows; its warps cut the run's 16 x 128-code pieces into equal parts. A warp loads its pieces straight into the
// registers that the A fragments are made from, AHEAD pieces before they are used, and writes the tiles that it has whole; the
// tiles that it shares are added up at the end, in order.
//
// Measured, 131072 x 2560: one row 39 us (groups of 128; 174 MB, 4.4 TB/s of the measured 6.8, further rows of weights at 5.4),
// 44.4 us (groups of 64, zero points), 51.9 us (32); 9 to 16 rows 50 to 51.5 us; 32 rows (bf16) 78 us, bound by issue slots and m16n8k16.
// 2560 x 6912, one row: 7.4 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bitnet_dev.cuh"
#include "smem_limit.h"
#include "w4.h"

namespace bitnet {
namespace {

constexpr int ROWS = 16;  // weight rows of a tile
constexpr int MAX_SMEM = 227 * 1024;

struct Call {
  W4 w;
  const void* x;
  float* out;
  int m;     // rows of this launch
  int cols;  // m, or 2 m where fp32 rows enter as two parts
  bool bf16;
};

// ZERO: the sum begins at 0 (d is not read)
template <bool ZERO>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (ZERO)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_bits(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }
// (w & mask) | magic in one instruction: magic is in a register
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "n"(MASK), "r"(magic));
  return r;
}
// The pairs (0, 4), (1, 5), (2, 6), (3, 7) of a word's codes less their zero point, as fp16; z: 1024 + zero, twice;
// magic: 1024, twice.
__device__ __forceinline__ void centred(uint32_t w, uint32_t z, uint32_t magic, uint32_t (&p)[4]) {
  const uint32_t w8 = w >> 8, one16 = 0x2c002c00u;  // 1/16, twice
  // 64 + zero: 1024 + zero has steps of 1, 64 + zero of 1/16
  const uint32_t z64 = 0xd400d400u | (z & 0x000f000fu) << 4;  // negative
  p[0] = as_bits(__hsub2(as_half2(and_or<0x000f000fu>(w, magic)), as_half2(z)));
  p[1] = as_bits(__hfma2(as_half2(and_or<0x00f000f0u>(w, magic)), as_half2(one16), as_half2(z64)));
  p[2] = as_bits(__hsub2(as_half2(and_or<0x000f000fu>(w8, magic)), as_half2(z)));
  p[3] = as_bits(__hfma2(as_half2(and_or<0x00f000f0u>(w8, magic)), as_half2(one16), as_half2(z64)));
}

// Shared memory: row factors (2 floats a row), fragments, then the warps' shares of tiles.
__host__ __device__ __forceinline__ int frag_bytes(int K, int cols) { return K * cols * 2; }
__host__ __device__ __forceinline__ int align16(int x) { return (x + 15) & ~15; }
__host__ __device__ __forceinline__ int rows_bytes(int K, int m, int cols) { return align16(m * 8) + frag_bytes(K, cols); }

// The rows as fragments. xf[(block * 4 + word) * cols + col][t]: the 8 numbers that word meets, as
// (0, 4), (1, 5), (2, 6), (3, 7).
template <int G>
__device__ __forceinline__ void load_rows(const Call& c, uint8_t* smem) {
  const int K = c.w.K, tid = threadIdx.x, threads = blockDim.x, lane = tid % 32;
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
  // A row's power of two: its largest number comes to [2^14, 2^15). Warps share rows where there are more of them; the
  // loads of a step do not wait for each other.
  constexpr int STEP = 4;
  const int octets = K / 8, warp = tid / 32, warps = threads / 32;
  int per_row = 1;
  while (per_row * 2 * c.m <= warps) per_row *= 2;
  const int first = warp / per_row, rows_a_step = warps / per_row, o0 = (warp % per_row) * 32 + lane, stride = per_row * 32;
  uint32_t* tops = reinterpret_cast<uint32_t*>(xf);
  for (int m = tid; m < c.m; m += threads) tops[m] = 0;
  __syncthreads();
  for (int m = first; m < c.m; m += rows_a_step) {
    uint32_t top = 0;
    for (int o = o0; o - lane < octets; o += STEP * stride) {
      float x[STEP][8];
#pragma unroll
      for (int i = 0; i < STEP; ++i)
        if (o + i * stride < octets) eight(m, (o + i * stride) * 8, x[i]);
#pragma unroll
      for (int i = 0; i < STEP; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (o + i * stride < octets) top = max(top, __float_as_uint(x[i][j]) & 0x7fffffffu);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) atomicMax(&tops[m], top);
  }
  __syncthreads();
  for (int m = tid; m < c.m; m += threads) {
    const uint32_t top = tops[m];
    int e = top == 0 ? 0 : 14 - ((int)(top >> 23) - 127);  // up = 2^e
    e = e > 127 ? 127 : e < -113 ? -113 : e;
    const int half = -e / 2;  // 2^-e in two factors: it may pass the range of one
    factor[m] = make_float2(__int_as_float((half + 127) << 23), __int_as_float((-e - half + 127) << 23));
  }
  __syncthreads();
  for (int m = first; m < c.m; m += rows_a_step) {
    const float2 f = factor[m];
    // up = 1 / (f.x f.y): its exponent from theirs
    const int e = -((int)(__float_as_uint(f.x) >> 23) - 127) - ((int)(__float_as_uint(f.y) >> 23) - 127);
    const float up = __int_as_float((e + 127) << 23);
    for (int o = o0; o < octets; o += STEP * stride) {
      float x[STEP][8];
#pragma unroll
      for (int i = 0; i < STEP; ++i)
        if (o + i * stride < octets) eight(m, (o + i * stride) * 8, x[i]);
#pragma unroll
      for (int i = 0; i < STEP; ++i) {
        if (o + i * stride >= octets) break;
        const int k = (o + i * stride) * 8, block = k >> 7, in = k & 127;
        const int t = G == 128 ? in >> 5 : G == 64 ? (in >> 4) & 3 : (in >> 3) & 3;
        const int word = G == 128 ? (in >> 3) & 3 : G == 64 ? (in >> 6) * 2 + ((in >> 3) & 1) : in >> 5;
        float hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          hi[j] = x[i][j] * up;
          lo[j] = hi[j] - __half2float(__float2half_rn(hi[j]));
        }
        uint4* to = xf + ((block * 4 + word) * c.cols + m * parts) * 4 + t;
        *to = make_uint4(pack_half2(hi[0], hi[4]), pack_half2(hi[1], hi[5]), pack_half2(hi[2], hi[6]), pack_half2(hi[3], hi[7]));
        if (parts == 2)
          to[4] = make_uint4(pack_half2(lo[0], lo[4]), pack_half2(lo[1], lo[5]), pack_half2(lo[2], lo[6]), pack_half2(lo[3], lo[7]));
      }
    }
  }
  __syncthreads();
}

// A piece of weights as a lane loads it: 16 bytes of rows g and g + 8, and their scales and zero points. The words of a
// matrix step have to be of one group over the four lanes of a row: with groups of 128 each lane's own 16 bytes are; with
// groups of 64 a lane loads twice 8 bytes; with 32 the row's 64 bytes are dealt out anew through shared memory, since
// every load touches a line for each row (one row x 131072 x 2560: groups of 32 by loads of 4 bytes 59.5 us, dealt
// out 51.6; groups of 64 by loads of 8 bytes 44.3, dealt out 45.6).
template <int G, bool ZEROS>
struct Piece {
  static constexpr int PER = 128 / G;  // groups
  uint32_t w[2][4];
  uint32_t s[2][PER == 4 ? 2 : 1];  // fp16 scales
  uint32_t z[2];
  // codes, scales, zeros: of this lane's row and quad place, at the piece
  __device__ __forceinline__ void load(int h, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros) {
    if (G == 64) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(codes + p * 32));
        w[h][2 * p] = v.x, w[h][2 * p + 1] = v.y;
      }
    } else {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(codes));
      w[h][0] = v.x, w[h][1] = v.y, w[h][2] = v.z, w[h][3] = v.w;
    }
    if (G == 128) {
      s[h][0] = __ldg(scales);
      if (ZEROS) z[h] = __ldg(zeros);
    } else if (G == 64) {
      s[h][0] = __ldg(reinterpret_cast<const uint32_t*>(scales));
      if (ZEROS) z[h] = __ldg(reinterpret_cast<const uint16_t*>(zeros));
    } else {
      const uint2 sc = __ldg(reinterpret_cast<const uint2*>(scales));
      s[h][0] = sc.x, s[h][PER == 4 ? 1 : 0] = sc.y;
      if (ZEROS) z[h] = __ldg(reinterpret_cast<const uint32_t*>(zeros));
    }
  }
  // The words in the order of the fragments. buf: 1 KB of this warp's; pieces of 16 bytes of row r are exchanged so that
  // neither stores nor loads meet a bank twice.
  __device__ __forceinline__ void deal(uint8_t* buf, int g, int t) {
    if (G != 32) return;
    const auto sw = [](int r) { return ((r >> 1) & 1) * 2 + ((r >> 2) & 1); };
#pragma unroll
    for (int h = 0; h < 2; ++h) *reinterpret_cast<uint4*>(buf + (g + 8 * h) * 64 + (t ^ sw(g)) * 16) = make_uint4(w[h][0], w[h][1], w[h][2], w[h][3]);
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t* row = buf + (g + 8 * h) * 64;
#pragma unroll
      for (int p = 0; p < 4; ++p) w[h][p] = *reinterpret_cast<const uint32_t*>(row + (p ^ sw(g)) * 16 + t * 4);
    }
  }
  __device__ __forceinline__ float scale(int h, int p) const {
    const float2 f = __half22float2(as_half2(s[h][PER == 4 ? p >> 1 : 0]));
    return p & 1 ? f.y : f.x;
  }
  // 1024 + zero as two fp16
  __device__ __forceinline__ uint32_t zero(int h, int p) const {
    return ZEROS ? __byte_perm(z[h], 0x64646464u, 0x4040 | p | p << 8) : 0x64086408u;
  }
};

// NT: eights of columns
template <int NT>
struct Shape {
  static constexpr int WARPS = 16, THREADS = WARPS * 32;  // one block an SM
  static constexpr int AHEAD = NT == 1 ? 6 : NT == 2 ? 4 : 2;  // pieces on their way
  static constexpr int EARLY = NT == 1 ? 3 : AHEAD;            // of them asked for before the rows are made ready
  static constexpr int SHARE = 32 * NT * 16;                   // bytes of a warp's share of a tile
};

template <int G, bool ZEROS, int NT>
__global__ void __launch_bounds__(Shape<NT>::THREADS, 1) w4_matmul_kernel(Call c) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int PER = 128 / G, WARPS = Shape<NT>::WARPS, AHEAD = Shape<NT>::AHEAD;
  const int K = c.w.K, N = c.w.N, lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);  // known to be the same for all lanes
  const int tiles = (N - 1) / ROWS + 1, blocks = K / 128, groups = K / G;
  const int tile0 = (int)((int64_t)tiles * blockIdx.x / gridDim.x), tile1 = (int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x);
  const int64_t all = (int64_t)(tile1 - tile0) * blocks;
  const int64_t p0 = all * warp / WARPS, p1 = all * (warp + 1) / WARPS;  // this warp's pieces

  // where the next piece to load lies: its tile's places (the same for the warp) and the lane's in a tile
  int in_tile = tile0 + (int)(p0 / blocks), in_block = (int)(p0 % blocks), left_in = (int)(p1 - p0);
  const uint8_t *codes, *zeros;
  const uint16_t* scales;
  int code_at[2], scale_at[2];
  const auto place = [&]() {
    const int64_t row = (int64_t)in_tile * ROWS;
    codes = c.w.codes + row * (K / 2) + in_block * 64;
    scales = c.w.scales + row * groups + in_block * PER;
    if (ZEROS) zeros = c.w.zeros + row * groups + in_block * PER;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int in = min(g + 8 * h, N - 1 - in_tile * ROWS);  // rows beyond the last: the last
      code_at[h] = in * (K / 2) + t * (G == 64 ? 8 : 16);
      scale_at[h] = in * groups;
    }
  };
  const auto load = [&](Piece<G, ZEROS>& p) {
    if (left_in <= 0) return;
    --left_in;
#pragma unroll
    for (int h = 0; h < 2; ++h) p.load(h, codes + code_at[h], scales + scale_at[h], ZEROS ? zeros + scale_at[h] : nullptr);
    if (++in_block == blocks) {
      in_block = 0, ++in_tile;
      if (left_in > 0) place();
    } else {
      codes += 64, scales += PER;
      if (ZEROS) zeros += PER;
    }
  };
  Piece<G, ZEROS> ring[AHEAD];
  if (left_in > 0) place();
#pragma unroll
  for (int u = 0; u < Shape<NT>::EARLY; ++u) load(ring[u]);  // on their way while the rows are made ready

  load_rows<G>(c, smem);
#pragma unroll
  for (int u = Shape<NT>::EARLY; u < AHEAD; ++u) load(ring[u]);
  const float2* factor = reinterpret_cast<const float2*>(smem);
  const uint4* xf = reinterpret_cast<const uint4*>(smem + align16(c.m * 8));
  float* share = reinterpret_cast<float*>(smem + rows_bytes(K, c.m, c.cols));
  uint8_t* deals = smem + rows_bytes(K, c.m, c.cols) + WARPS * Shape<NT>::SHARE + warp * 2048;
  __shared__ int share_tile[WARPS];
  if (lane == 0) share_tile[warp] = -1;

  const auto write = [&](int tile, const float (&tot)[NT][4]) {
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
  };

  int tile = tile0 + (int)(p0 / blocks), block = (int)(p0 % blocks), left = (int)(p1 - p0);
  bool begun = block == 0;  // this warp has the tile from its first piece
  float tot[NT][4] = {};
  uint32_t magic;
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));  // kept in a register
  const uint4* f = xf + block * 16 * c.cols + t;
  int col[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) col[n] = (n * 8 + g < c.cols ? n * 8 + g : 0) * 4;
  while (left > 0) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (left <= 0) break;
      --left;
      Piece<G, ZEROS>& p = ring[u];
      p.deal(deals + (u & 1) * 1024, g, t);  // two places in turn: one barrier each
      float acc[NT][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        constexpr int STEP = 4 / PER;  // words of a group
        uint32_t a[4], b[4];
        centred(p.w[0][i], p.zero(0, i / STEP), magic, a);
        centred(p.w[1][i], p.zero(1, i / STEP), magic, b);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 v = f[i * 4 * c.cols + col[n]];
          if (i % STEP == 0) mma16816<true>(acc[n], a[0], b[0], a[1], b[1], v.x, v.y);
          else mma16816<false>(acc[n], a[0], b[0], a[1], b[1], v.x, v.y);
          mma16816<false>(acc[n], a[2], b[2], a[3], b[3], v.z, v.w);
        }
        if (i % STEP == STEP - 1) {
          const float s0 = p.scale(0, i / STEP), s1 = p.scale(1, i / STEP);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            tot[n][0] = fmaf(s0, acc[n][0], tot[n][0]);
            tot[n][1] = fmaf(s0, acc[n][1], tot[n][1]);
            tot[n][2] = fmaf(s1, acc[n][2], tot[n][2]);
            tot[n][3] = fmaf(s1, acc[n][3], tot[n][3]);
          }
        }
      }
      load(ring[u]);
      f += 16 * c.cols;
      if (++block == blocks) {
        if (begun) {
          write(tile, tot);
        } else {  // its first pieces are another warp's
          float* mine = share + (warp * 32 + lane) * (NT * 4);
#pragma unroll
          for (int n = 0; n < NT; ++n) *reinterpret_cast<float4*>(mine + 4 * n) = make_float4(tot[n][0], tot[n][1], tot[n][2], tot[n][3]);
          if (lane == 0) share_tile[warp] = tile;
        }
        block = 0, ++tile, begun = true, f = xf + t;
#pragma unroll
        for (int n = 0; n < NT; ++n) tot[n][0] = tot[n][1] = tot[n][2] = tot[n][3] = 0.0f;
      }
    }
  }
  // the last tile, where it is not whole: its first warp adds the others' shares
  const bool open = block != 0 && p1 > p0;
  if (open && !begun) {
    float* mine = share + (warp * 32 + lane) * (NT * 4);
#pragma unroll
    for (int n = 0; n < NT; ++n) *reinterpret_cast<float4*>(mine + 4 * n) = make_float4(tot[n][0], tot[n][1], tot[n][2], tot[n][3]);
    if (lane == 0) share_tile[warp] = tile;
  }
  __syncthreads();
  if (open && begun) {
    for (int w = warp + 1; w < WARPS; ++w) {
      if (share_tile[w] != tile) continue;
      const float* other = share + (w * 32 + lane) * (NT * 4);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float4 v = *reinterpret_cast<const float4*>(other + 4 * n);
        tot[n][0] += v.x, tot[n][1] += v.y, tot[n][2] += v.z, tot[n][3] += v.w;
      }
    }
    write(tile, tot);
  }
}

template <int NT>
int smem_of(int group, int K, int m, int cols) {
  return rows_bytes(K, m, cols) + Shape<NT>::WARPS * (Shape<NT>::SHARE + (group == 32 ? 2048 : 0));
}

template <int G, bool ZEROS, int NT>
cudaError_t launch(const Call& c, int num_sms, cudaStream_t st) {
  const int smem = smem_of<NT>(G, c.w.K, c.m, c.cols);
  auto kernel = w4_matmul_kernel<G, ZEROS, NT>;
  static std::atomic<uint64_t> configured{0};
  if (cudaError_t e = allow_smem(configured, kernel, MAX_SMEM - 1024)) return e;
  const int tiles = (c.w.N - 1) / ROWS + 1;
  kernel<<<min(tiles, num_sms), Shape<NT>::THREADS, smem, st>>>(c);
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
    const int cols = m * parts;
    return (cols <= 8 ? smem_of<1>(w.group, w.K, m, cols) : cols <= 16 ? smem_of<2>(w.group, w.K, m, cols)
            : cols <= 32 ? smem_of<4>(w.group, w.K, m, cols) : smem_of<8>(w.group, w.K, m, cols)) <= MAX_SMEM - 1024;
  };
  while (most > 1 && !fits(most)) --most;
  if (M > most) {  // launches of like size: fewer columns each cost less
    const int64_t launches = (M + most - 1) / most;
    most = (int)((M + launches - 1) / launches);
  }
  for (int64_t m0 = 0; m0 < M; m0 += most) {
    const int m = (int)(M - m0 < most ? M - m0 : most);
    Call c{w, nullptr, out + m0 * w.N, m, m * parts, bf16};
    c.x = bf16 ? static_cast<const void*>(static_cast<const __nv_bfloat16*>(x) + m0 * w.K)
               : static_cast<const void*>(static_cast<const float*>(x) + m0 * w.K);
    const cudaError_t e = w.group == 128 ? by_zeros<128>(c, num_sms, st)
                          : w.group == 64 ? by_zeros<64>(c, num_sms, st) : by_zeros<32>(c, num_sms, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace bitnet
