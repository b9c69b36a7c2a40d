// kv4_mass.cu -- the attention weight that cached tokens gather from a call's queries.
//
// A sequence's voting rows times the query heads that share a key/value head are its columns (fp32
// queries: two columns each, the parts of their 22 bits). A tile is 32 tokens of one head; a block of columns
// against a tile is m16n8k16 with the codes as the A operand:
//   raw[t][r] = sum_d code[t][d] q'[r][d],   x = scale log2 e (step raw / up + base sum(q))
// The weight of a token needs its row's maximum M and sum L over all tokens first: the first kernel finds (M, L) of
// each column over each chunk of tiles, the second joins them and adds up
//   votes[t] = sum_r 2^(x - M) / L
// The scores of both are the same bits (kept, or made by the same instructions), so that each row's votes add up to 1 however
// large they are.
// There are no atomics: results do not depend on timing.
//
// A code enters as the fp16 subnormal c 2^-24 (its nibble masked out of the word) or c 2^-20 (the nibble above, not
// shifted; q' carries the 2^-4): 5 instructions for a word of 8 codes, sums exact in fp32. Lane t of four takes 16
// bytes of a key row (8 with D = 64), so a warp's loads of a tile are contiguous, straight from the cache.
//
// Few columns (16 at most): of short sequences, and of many whose scores fit the shared memory of a cluster of up to eight
// blocks, one kernel does it all: scores once, (M, L) exchanged between the blocks, votes from the kept scores. Else the first
// kernel leaves the scores in the workspace and the second starts behind it; where that would take more than 256 MB, the second
// makes them again. Bound by latency (chains of loads and products), at half of the issue slots: a tile takes 445 instructions in
// the one kernel and 363 and 197 in the two, of which 80 unpack its codes. Measured (20 and 5 heads x 128): one query over 77 tokens
// 4.9 us, 64 over 87 to 8086 43.9 us (fp32 queries), one over 131007 19.6 us (25.4 where the scores are made again).
//
// More columns, up to 96 rows (kv4_mass_tc.cu has the others): blocks of 64 whose fragments the first kernel leaves in the
// workspace; the second kernel's blocks keep their tiles' codes and go through a share of the columns, and where these are more
// than one a third adds up the shares. Bound by the products' latency and issue slots (tensor pipe 38% busy): 64 rows of 5 prompts of
// 1000 to 9000 tokens each 29.9 us.
#include <type_traits>

#include "kv4_mass.cuh"
#include "smem_limit.h"

namespace bitnet {
namespace {

constexpr int WARPS = 8, THREADS = WARPS * 32;
constexpr int TILE = 32;  // tokens of a tile: half a page
constexpr int MAX_CHUNK = 32 * WARPS;  // tiles of a chunk: a warp keeps the page ids of its own, one a lane
struct Plan {
  int parts;    // columns of a row: 1, or 2 for fp32 queries
  int votes;    // rows of a sequence that vote, at most
  int nt;       // eights of columns of a block
  int blocks;   // blocks of columns of a unit (a sequence's head), at most
  int tiles;    // tiles of a unit, at most
  int chunk;    // of them in a chunk
  int chunks;
  int shares;   // of the columns, in the second kernel; 0: few columns
  int groups;   // runs of WARPS tiles (many columns)
};
struct Stats {
  float2* part;  // unit, block, chunk, column: (M, L)
  float* votes;  // unit, group, share, WARPS x TILE (more than one share)
  uint8_t* slabs;  // unit, block
  float* scores;   // few columns: unit, row, token; null where they are not kept
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the first of a chain of products: the sum begins at 0
__device__ __forceinline__ void mma_first(float (&d)[4], uint4 a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.0f));
}
// What a column needs besides its fragments.
// step a raw and base b stay below 2^116 in size. Where a is cut, scores that differ at all are infinitely far apart either way:
// they are 2^-72 or more apart before the factor.
constexpr float kMostFew = 1.2676506002282294e30f;  // 2^100
struct Column {
  float a, b;  // x = step (a raw) + base b
  int p;       // the row's position
};
template <int D, int NT>
struct __align__(16) Shared {
  uint4 frag[NT][D / 32][32];  // eight, word, lane: its column's numbers for that word's codes
  Column col[NT * 8];
  float2 part[WARPS][NT * 8];
};

// The fragments and constants of columns [col0, col0 + 8 NT): D / 8 lanes a row, 8 numbers each.
template <int D, int NT, bool F32>
__device__ __forceinline__ void load_columns(const Kv4Attn& a, const Rows& r, int col0, Shared<D, NT>& sh) {
  constexpr int W = D / 8, PARTS = F32 ? 2 : 1, ROWS = NT * 8 / PARTS, PER = THREADS / W;
  const int w = threadIdx.x % W, rows = r.votes * a.share;
  for (int k = threadIdx.x / W; k < ROWS; k += PER) {
    const int row = col0 / PARTS + k, i = row / a.share;
    const bool there = row < rows;
    float x[8];  // number n: dimension w + W n, the nibbles of word w
    float sum = 0.0f;
    uint32_t top = 0;
    const int64_t at = there ? (int64_t)(r.s.q0 + r.s.n - r.votes + i) * a.q_stride + (int64_t)(r.h * a.share + row - i * a.share) * D : 0;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      x[n] = 0.0f;
      if (there)
        x[n] = F32 ? static_cast<const float*>(a.q)[at + w + W * n]
                   : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at + w + W * n]);
      sum += x[n];
      top = max(top, __float_as_uint(x[n]) & 0x7fffffffu);
    }
#pragma unroll
    for (int o = W / 2; o >= 1; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    // the row's power of two: its largest number comes to [2^14, 2^15)
    int e = top == 0 ? 0 : 14 - ((int)(top >> 23) - 127);
    e = e > 127 ? 127 : e < -113 ? -113 : e;
    const float up = __int_as_float((e + 127) << 23);
    sum = row_sum<W>(x, sum, up, top);
    // words of lane quad t: W / 4 of them
    constexpr int WORDS = W / 4;
    const int t = w / WORDS, word = w % WORDS;
    float hi[8], lo[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      hi[n] = x[n] * up * (n & 1 ? 0.0625f : 1.0f);
      lo[n] = hi[n] - __half2float(__float2half_rn(hi[n]));
    }
    const int col = k * PARTS;
    sh.frag[col >> 3][word][(col & 7) * 4 + t] =
        make_uint4(pack_half2(hi[0], hi[4]), pack_half2(hi[1], hi[5]), pack_half2(hi[2], hi[6]), pack_half2(hi[3], hi[7]));
    if (F32)
      sh.frag[col >> 3][word][((col & 7) + 1) * 4 + t] =
          make_uint4(pack_half2(lo[0], lo[4]), pack_half2(lo[1], lo[5]), pack_half2(lo[2], lo[6]), pack_half2(lo[3], lo[7]));
    if (w == 0) {
      const float c1 = __fmul_rn(a.scale, kLog2e);
      // c1 2^(24 - e) in two steps: the power may pass fp32's range
      const int f = 24 - e, half = f / 2;
      const float ca = __fmul_rn(__fmul_rn(c1, __int_as_float((half + 127) << 23)), __int_as_float((f - half + 127) << 23));
      Column c;
      c.a = copysignf(fminf(fabsf(ca), kMostFew), ca);
      c.b = or_nan(__fmul_rn(c.a, __fmul_rn(sum, 5.9604644775390625e-8f)), top);  // 2^-24
      c.p = there ? r.position(i) : -1;
      sh.col[col] = c;
      if (F32) sh.col[col + 1] = c;
    }
  }
}

// A tile's codes and parameters as they lie in the cache: rows mt * 16 + g and + 8.
template <int D>
struct Codes {
  static constexpr int WORDS = D / 32;  // words of a lane and row
  uint32_t w[2][2][WORDS];
  uint32_t par[2][2];
  __device__ __forceinline__ void load(const uint8_t* blk, int tile, int g, int t) {
    const int row0 = (tile & 1) * TILE;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = row0 + mt * 16 + h * 8 + g;
        const uint8_t* p = blk + row * (D / 2) + t * (WORDS * 4);
        if (D == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(p);
          w[mt][h][0] = v.x, w[mt][h][1] = v.y, w[mt][h][2 % WORDS] = v.z, w[mt][h][3 % WORDS] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          w[mt][h][0] = v.x, w[mt][h][1] = v.y;
        }
        par[mt][h] = *reinterpret_cast<const uint32_t*>(blk + kKvPage * D + row * 8);
      }
  }
};
// the token (of its page half) in row `row` of a tile
__device__ __forceinline__ int token_of(int row) { return kv4_rho_inv(row); }

// Products of a tile's two m16 x n8: the lane has rows mt * 16 + g and + 8, columns 2 t and 2 t + 1 (fp32 queries: one
// row's parts).
template <int D, int NT>
__device__ __forceinline__ void products(const Codes<D>& k, const Shared<D, NT>& sh, int n, int lane, float (&d)[2][4]) {
#pragma unroll
  for (int i = 0; i < Codes<D>::WORDS; ++i) {
    const uint4 f = sh.frag[n][i][lane];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const uint32_t a = k.w[mt][0][i], b = k.w[mt][1][i], a8 = a >> 8, b8 = b >> 8;
      if (i == 0) mma_first(d[mt], make_uint4(a & 0x000f000fu, b & 0x000f000fu, a & 0x00f000f0u, b & 0x00f000f0u), f.x, f.y);
      else mma16816(d[mt], a & 0x000f000fu, b & 0x000f000fu, a & 0x00f000f0u, b & 0x00f000f0u, f.x, f.y);
      mma16816(d[mt], a8 & 0x000f000fu, b8 & 0x000f000fu, a8 & 0x00f000f0u, b8 & 0x00f000f0u, f.z, f.w);
    }
  }
}
__device__ __forceinline__ float score(float raw, const Column& c, float2 par) {
  return __fmaf_rn(par.x, __fmul_rn(c.a, raw), __fmul_rn(par.y, c.b));
}
// joins (m, l) with (m2, l2); a NaN is no maximum, but stays in the sum
__device__ __forceinline__ void join(float& m, float& l, float m2, float l2) {
  const float top = fmaxf(m, m2), from = top == kNegInf ? 0.0f : top;
  l = l * exp2_approx(m - from) + l2 * exp2_approx(m2 - from);
  m = top;
}

// ------------------------------------------------------------- first kernel: maxima and sums
template <int D, int NT, bool F32>
__global__ void __launch_bounds__(THREADS, NT == 1 ? 3 : 2) kv4_mass_rows(Kv4 c, Kv4Attn a, int voters, Plan pl, Stats st) {
  __shared__ Shared<D, NT> sh;
  constexpr int COLS = NT * 8, PARTS = F32 ? 2 : 1, BLK = (int)kv4_block_bytes(D);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
  bool bad = false;
  pdl_launch_dependents();
  const int64_t items = (int64_t)c.batch * c.kv_heads * pl.chunks;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int unit = (int)(item / pl.chunks), chunk = (int)(item - (int64_t)unit * pl.chunks);
    const Rows r = rows_of(c, unit, voters, &bad);
    const int rows = r.votes * a.share, kept = st.scores ? rows : 0;
    if (rows == 0) continue;
    const int tile0 = chunk * pl.chunk, tile1 = min(tile0 + pl.chunk, (r.s.len + TILE - 1) / TILE);
    const int first = r.position(0), last = r.position(r.votes - 1);
    float2* out = st.part + item * COLS;
    if (tile0 >= tile1 || seen(a, first, last, tile0 * TILE, (tile1 - tile0) * TILE) == 0) {
      for (int i = threadIdx.x; i < COLS; i += THREADS) out[i] = make_float2(kNegInf, 0.0f);
      continue;
    }
    // the blocks of this warp's tiles, one a lane, and which tiles the rows see any and all of
    uint32_t id = r.h;
    const int mine = tile0 + warp + lane * WARPS, what = mine < tile1 ? seen(a, first, last, mine * TILE, TILE) : 0;
    const uint32_t any = __ballot_sync(0xffffffffu, what > 0), whole = __ballot_sync(0xffffffffu, what == 2);
    if (mine < tile1) {
      const int page = c.page_table[(int64_t)r.b * c.max_pages + mine / 2];
      if (page < 0 || page >= c.n_pages) bad = true;
      else id = (uint32_t)page * c.kv_heads + r.h;
    }
    load_columns<D, NT, F32>(a, r, 0, sh);
    __syncthreads();
    const int eights = min(NT, (rows * PARTS + 7) / 8);
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = kNegInf, l[n][0] = l[n][1] = 0.0f;
    Codes<D> cur;
    const auto load = [&](int k) {
      const uint32_t from = __shfl_sync(0xffffffffu, id, k);
      const int tile = tile0 + warp + k * WARPS;
      if (tile < tile1) cur.load(c.pages + (uint64_t)from * BLK, tile, g, t);
    };
    load(0);
    for (int k = 0, tile = tile0 + warp; tile < tile1; ++k, tile += WARPS) {
      const int j0 = tile * TILE;
      const bool sees = any >> k & 1, masked = !(whole >> k & 1);
      float* to = st.scores + ((int64_t)unit * pl.votes * a.share * pl.tiles + tile) * TILE;
      const float2 par[4] = {params(cur.par[0][0]), params(cur.par[0][1]), params(cur.par[1][0]), params(cur.par[1][1])};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float d[2][4];
        if (n < eights) products<D, NT>(cur, sh, n, lane, d);
        if (n == NT - 1 && k < 31) load(k + 1);  // the codes' registers are free
        if (n >= eights || !sees) continue;
#pragma unroll
        for (int e = 0; e < (F32 ? 1 : 2); ++e) {
          const Column& col = sh.col[n * 8 + 2 * t + e];
          const int row = (n * 8 + 2 * t + e) / PARTS;
          float x[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int mt = v >> 1, h = v & 1, in = token_of(mt * 16 + h * 8 + g);
            x[v] = score(F32 ? d[mt][2 * h] + d[mt][2 * h + 1] : d[mt][2 * h + e], col, par[v]);
            if (masked && !visible(a, col.p, j0 + in)) x[v] = kNegInf;
            if (row < kept) to[(int64_t)row * pl.tiles * TILE + in] = x[v];
          }
          const float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), m[n][e]), from = top == kNegInf ? 0.0f : top;
          l[n][e] = l[n][e] * exp2_approx(m[n][e] - from) + ((exp2_approx(x[0] - from) + exp2_approx(x[1] - from)) + (exp2_approx(x[2] - from) + exp2_approx(x[3] - from)));
          m[n][e] = top;
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1)
          join(m[n][e], l[n][e], __shfl_xor_sync(0xffffffffu, m[n][e], o), __shfl_xor_sync(0xffffffffu, l[n][e], o));
        if (g == 0) sh.part[warp][n * 8 + 2 * t + e] = make_float2(m[n][e], l[n][e]);
      }
    __syncthreads();
    for (int i = threadIdx.x; i < COLS; i += THREADS) {
      float2 v = sh.part[0][i];
      for (int w = 1; w < WARPS; ++w) join(v.x, v.y, sh.part[w][i].x, sh.part[w][i].y);
      out[i] = v;
    }
    __syncthreads();  // the next item's columns
  }
  if (bad) record_device_error(kErrRange);
}

// ------------------------------------------------------------- second kernel, few columns
// The rows' M and 1 / L from the (M, L) of the chunks, a warp each.
template <int NT, bool F32>
__device__ __forceinline__ void join_chunks(const Plan& pl, const Stats& st, int unit, int chunks, int rows, float2* ml) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int row = warp; row < rows; row += WARPS) {
    float m = kNegInf, l = 0.0f;
    for (int k = lane; k < chunks; k += 32) {
      const float2 v = st.part[((int64_t)unit * pl.chunks + k) * (NT * 8) + row * (F32 ? 2 : 1)];
      join(m, l, v.x, v.y);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) join(m, l, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, l, o));
    if (lane == 0) ml[row] = make_float2(m == kNegInf ? 0.0f : m, l == 0.0f ? 0.0f : __frcp_rn(l));
  }
}
// A thread a token; the scores are the first kernel's.
template <int NT, bool F32>
__global__ void __launch_bounds__(THREADS) kv4_mass_votes(Kv4 c, Kv4Attn a, Kv4Mass ms, Plan pl, Stats st) {
  __shared__ float2 ml[NT * 8];  // of the rows: M and 1 / L
  constexpr int AHEAD = 4, QUAD = 4;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  bool bad = false;
  const int64_t items = (int64_t)c.batch * c.kv_heads * pl.chunks;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int unit = (int)(item / pl.chunks), chunk = (int)(item - (int64_t)unit * pl.chunks);
    const Rows r = rows_of(c, unit, ms.voters, &bad);
    const int rows = r.votes * a.share, all = (r.s.len + TILE - 1) / TILE;
    const int tile0 = chunk * pl.chunk, tile1 = min(tile0 + pl.chunk, all);
    if (rows == 0 || tile0 >= tile1) continue;
    const int first = r.position(0), last = r.position(r.votes - 1), old = r.s.len - r.s.n, chunks = (all + pl.chunk - 1) / pl.chunk;
    const int32_t* table = c.page_table + (int64_t)r.b * c.max_pages;
    const float* scores = st.scores + (int64_t)unit * pl.votes * a.share * pl.tiles * TILE + lane;
    // four tiles of the warp at a time: their tokens' places and old masses, which wait for nothing, then four rows' scores
    float before[AHEAD], votes[AHEAD], x[QUAD][AHEAD];
    int64_t at[AHEAD];
    bool write[AHEAD], any[AHEAD];
    const auto places = [&](int tile) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int now = tile + i * WARPS, j = now * TILE + lane;
        any[i] = now < tile1 && seen(a, first, last, now * TILE, TILE) != 0;
        write[i] = now < tile1 && j < r.s.len && (ms.decay != 1.0f || ms.in != ms.out || j >= old || any[i]);
        int id = 0;
        if (write[i]) id = table[now / 2];
        if (id < 0 || id >= c.n_pages) bad = true, write[i] = false, id = 0;
        at[i] = ((int64_t)id * c.kv_heads + r.h) * kKvPage + j % kKvPage;
        before[i] = write[i] && j < old ? ms.in[at[i]] : 0.0f;
        votes[i] = 0.0f;
      }
    };
    const auto load = [&](int tile, int row0) {
#pragma unroll
      for (int q = 0; q < QUAD; ++q)
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          x[q][i] = any[i] && row0 + q < rows ? scores[((int64_t)(row0 + q) * pl.tiles + tile + i * WARPS) * TILE] : kNegInf;
    };
    places(tile0 + warp);
    pdl_wait();
    load(tile0 + warp, 0);
    join_chunks<NT, F32>(pl, st, unit, chunks, rows, ml);
    __syncthreads();
#pragma unroll 1
    for (int tile = tile0 + warp; tile < tile1;) {
#pragma unroll 1
      for (int row0 = 0; row0 < rows; row0 += QUAD) {
        if (row0) load(tile, row0);
        // a masked score is -inf; it takes no part, whatever the row's sum is
#pragma unroll
        for (int q = 0; q < QUAD; ++q) {
          const float2 v = ml[min(row0 + q, rows - 1)];
#pragma unroll
          for (int i = 0; i < AHEAD; ++i)
            if (x[q][i] != kNegInf) votes[i] = fmaf(exp2_approx(x[q][i] - v.x), v.y, votes[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (write[i]) ms.out[at[i]] = (tile + i * WARPS) * TILE + lane < old ? fmaf(ms.decay, before[i], votes[i]) : votes[i];
      tile += AHEAD * WARPS;
      if (tile < tile1) places(tile), load(tile, 0);
    }
    __syncthreads();
  }
  pdl_wait();
  if (bad) record_device_error(kErrRange);
}

// The same where the scores are not kept: made again by the first kernel's instructions, a warp a tile.
template <int D, int NT, bool F32>
__global__ void __launch_bounds__(THREADS, NT == 1 ? 3 : 2) kv4_mass_again(Kv4 c, Kv4Attn a, Kv4Mass ms, Plan pl, Stats st) {
  __shared__ Shared<D, NT> sh;
  __shared__ float2 ml[NT * 8];
  constexpr int PARTS = F32 ? 2 : 1, BLK = (int)kv4_block_bytes(D);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
  const int own = token_of((t >> 1) * 16 + (t & 1) * 8 + g);  // the token (of a tile) whose votes end up in this lane
  bool bad = false;
  const int64_t items = (int64_t)c.batch * c.kv_heads * pl.chunks;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int unit = (int)(item / pl.chunks), chunk = (int)(item - (int64_t)unit * pl.chunks);
    const Rows r = rows_of(c, unit, ms.voters, &bad);
    const int rows = r.votes * a.share, all = (r.s.len + TILE - 1) / TILE;
    const int tile0 = chunk * pl.chunk, tile1 = min(tile0 + pl.chunk, all);
    if (rows == 0 || tile0 >= tile1) continue;
    const int first = r.position(0), last = r.position(r.votes - 1), old = r.s.len - r.s.n;
    // the blocks of this warp's tiles, one a lane (-1: not in the pool), and which of them the rows see any and all of
    int id = -1, what = 0;
    const int mine = tile0 + warp + lane * WARPS;
    if (mine < tile1) {
      const int page = c.page_table[(int64_t)r.b * c.max_pages + mine / 2];
      if (page < 0 || page >= c.n_pages) bad = true;
      else id = page * c.kv_heads + r.h, what = seen(a, first, last, mine * TILE, TILE);
    }
    const uint32_t any = __ballot_sync(0xffffffffu, what > 0), whole = __ballot_sync(0xffffffffu, what == 2);
    Codes<D> cur;
    const auto load = [&](int k) {
      const int from = __shfl_sync(0xffffffffu, id, k);
      if (from >= 0) cur.load(c.pages + (int64_t)from * BLK, tile0 + warp + k * WARPS, g, t);
    };
    load(0);
    load_columns<D, NT, F32>(a, r, 0, sh);
    pdl_wait();
    join_chunks<NT, F32>(pl, st, unit, (all + pl.chunk - 1) / pl.chunk, rows, ml);
    __syncthreads();
    const int eights = min(NT, (rows * PARTS + 7) / 8);
    for (int k = 0, tile = tile0 + warp; tile < tile1; ++k, tile += WARPS) {
      const int from = __shfl_sync(0xffffffffu, id, k), j0 = tile * TILE, j = j0 + own;
      const bool sees = any >> k & 1, masked = !(whole >> k & 1);
      const bool write = from >= 0 && j < r.s.len && (ms.decay != 1.0f || ms.in != ms.out || j >= old || sees);
      const int64_t at = (int64_t)from * kKvPage + j % kKvPage;
      const float before = write && j < old ? ms.in[at] : 0.0f;
      const float2 par[4] = {params(cur.par[0][0]), params(cur.par[0][1]), params(cur.par[1][0]), params(cur.par[1][1])};
      float votes[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float d[2][4];
        if (n < eights) products<D, NT>(cur, sh, n, lane, d);
        if (n == NT - 1 && k < 31) load(k + 1);  // the codes' registers are free
        if (n >= eights || !sees) continue;
#pragma unroll
        for (int e = 0; e < (F32 ? 1 : 2); ++e) {
          const Column& col = sh.col[n * 8 + 2 * t + e];
          if (col.p < 0) continue;  // no row, or one that sees nothing
          const float2 of = ml[(n * 8 + 2 * t + e) / PARTS];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int mt = v >> 1, h = v & 1;
            const float x = score(F32 ? d[mt][2 * h] + d[mt][2 * h + 1] : d[mt][2 * h + e], col, par[v]);
            if (!masked || visible(a, col.p, j0 + token_of(mt * 16 + h * 8 + g))) votes[v] = fmaf(exp2_approx(x - of.x), of.y, votes[v]);
          }
        }
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        votes[v] += __shfl_xor_sync(0xffffffffu, votes[v], 1);
        votes[v] += __shfl_xor_sync(0xffffffffu, votes[v], 2);
      }
      const float got = t == 0 ? votes[0] : t == 1 ? votes[1] : t == 2 ? votes[2] : votes[3];
      if (write) ms.out[at] = j < old ? fmaf(ms.decay, before, got) : got;
    }
    __syncthreads();  // the next item's columns
  }
  pdl_wait();
  if (bad) record_device_error(kErrRange);
}

// ------------------------------------------------------------- few columns, short enough: one kernel
// A cluster of one to eight blocks takes a unit; its blocks keep the scores of their tiles in shared memory, exchange
// their (M, L) through distributed shared memory, and add up the votes from the scores: a thread a token.
constexpr int kScoreBytes = 64 * 1024;  // of a block: three blocks an SM
struct Cluster {
  int blocks;   // of a cluster
  int tiles;    // of a block, at most
  int rows;     // of scores a token
};
template <int D, int NT, bool F32>
__global__ void __launch_bounds__(THREADS, NT == 1 ? 3 : 2) kv4_mass_cluster(Kv4 c, Kv4Attn a, Kv4Mass ms, Cluster cl) {
  extern __shared__ __align__(16) float kept[];  // token, row
  __shared__ Shared<D, NT> sh;
  __shared__ float2 mine[NT * 8];  // this block's (M, L) of each column
  constexpr int COLS = NT * 8, PARTS = F32 ? 2 : 1, BLK = (int)kv4_block_bytes(D);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
  const int unit = blockIdx.x / cl.blocks, me = cl.blocks > 1 ? (int)cluster_ctarank() : 0;
  bool bad = false;
  const Rows r = rows_of(c, unit, ms.voters, &bad);
  const int rows = r.votes * a.share, all = (r.s.len + TILE - 1) / TILE, per = (all + cl.blocks - 1) / cl.blocks;
  if (rows == 0 || all == 0) {
    if (bad && threadIdx.x == 0) record_device_error(kErrRange);
    return;
  }
  const int tile0 = min(me * per, all), tile1 = min(tile0 + per, all), first = r.position(0), last = r.position(r.votes - 1);
  // the blocks (below 2^30) of this warp's next 32 tiles, one a lane (-1: not in the pool), and which of them the rows see any and all of
  uint32_t any = 0, whole = 0;
  const int32_t* table = c.page_table + (int64_t)r.b * c.max_pages;
  const auto ids_of = [&](int k) {
    const int tile = tile0 + warp + (k + lane) * WARPS;
    int id = -1, what = 0;
    if (tile < tile1) {
      const int page = table[tile / 2];
      if (page < 0 || page >= c.n_pages) bad = true;
      else id = page * c.kv_heads + r.h, what = seen(a, first, last, tile * TILE, TILE);
    }
    any = __ballot_sync(0xffffffffu, what > 0), whole = __ballot_sync(0xffffffffu, what == 2);
    return id;
  };
  int ids = ids_of(0);
  load_columns<D, NT, F32>(a, r, 0, sh);
  __syncthreads();
  const int eights = min(NT, (rows * PARTS + 7) / 8);
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = kNegInf, l[n][0] = l[n][1] = 0.0f;
  Codes<D> cur;
  const auto load = [&](int k) {
    const int id = __shfl_sync(0xffffffffu, ids, k & 31);
    if (id >= 0) cur.load(c.pages + (int64_t)id * BLK, tile0 + warp + k * WARPS, g, t);
  };
  load(0);
#pragma unroll 1
  for (int k = 0, tile = tile0 + warp; tile < tile1; ++k, tile += WARPS) {
    const int j0 = tile * TILE;
    const bool sees = any >> (k & 31) & 1, masked = !(whole >> (k & 31) & 1);
    float* to = kept + (int64_t)(tile - tile0) * TILE * cl.rows;
    const float2 par[4] = {params(cur.par[0][0]), params(cur.par[0][1]), params(cur.par[1][0]), params(cur.par[1][1])};
    if ((k & 31) == 31) ids = ids_of(k + 1);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float d[2][4];
      if (n < eights) products<D, NT>(cur, sh, n, lane, d);
      if (n == NT - 1) load(k + 1);  // the codes' registers are free
      if (n >= eights || !sees) continue;
#pragma unroll
      for (int e = 0; e < (F32 ? 1 : 2); ++e) {
        const Column& col = sh.col[n * 8 + 2 * t + e];
        const int row = (n * 8 + 2 * t + e) / PARTS;
        float x[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int mt = v >> 1, h = v & 1, in = token_of(mt * 16 + h * 8 + g);
          x[v] = score(F32 ? d[mt][2 * h] + d[mt][2 * h + 1] : d[mt][2 * h + e], col, par[v]);
          if (masked && !visible(a, col.p, j0 + in)) x[v] = kNegInf;
          if (row < cl.rows) to[in * cl.rows + row] = x[v];
        }
        const float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), m[n][e]), from = top == kNegInf ? 0.0f : top;
        l[n][e] = fmaf(l[n][e], exp2_approx(m[n][e] - from), (exp2_approx(x[0] - from) + exp2_approx(x[1] - from)) + (exp2_approx(x[2] - from) + exp2_approx(x[3] - from)));
        m[n][e] = top;
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1)
        join(m[n][e], l[n][e], __shfl_xor_sync(0xffffffffu, m[n][e], o), __shfl_xor_sync(0xffffffffu, l[n][e], o));
      if (g == 0) sh.part[warp][n * 8 + 2 * t + e] = make_float2(m[n][e], l[n][e]);
    }
  __syncthreads();
  if (threadIdx.x < COLS) {
    float2 v = sh.part[0][threadIdx.x];
#pragma unroll 1
    for (int w = 1; w < WARPS; ++w) join(v.x, v.y, sh.part[w][threadIdx.x].x, sh.part[w][threadIdx.x].y);
    mine[threadIdx.x] = v;
  }
  if (cl.blocks > 1) cluster_sync_all();
  else __syncthreads();
  if (threadIdx.x < COLS) {  // all blocks' in the same order
    float top = kNegInf, sum = 0.0f;
    const uint32_t at = smem_u32(&mine[threadIdx.x]);
#pragma unroll 1
    for (int k = 0; k < cl.blocks; ++k) join(top, sum, ld_cluster_f32(map_to_rank(at, k)), ld_cluster_f32(map_to_rank(at, k) + 4));
    sh.part[0][threadIdx.x] = make_float2(top == kNegInf ? 0.0f : top, sum == 0.0f ? 0.0f : __frcp_rn(sum));
  }
  if (cl.blocks > 1) cluster_sync_all();  // no block leaves while another reads its sums
  else __syncthreads();
  // the votes: a lane a token of the warp's tiles, the masses of four tiles on their way at once
  const int old = r.s.len - r.s.n;
  ids = ids_of(0);
#pragma unroll 1
  for (int k = 0; tile0 + warp + k * WARPS < tile1; k += 4) {
    if (k && (k & 31) == 0) ids = ids_of(k);
    float before[4];
    uint32_t writes = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = __shfl_sync(0xffffffffu, ids, (k + i) & 31), j = (tile0 + warp + (k + i) * WARPS) * TILE + lane;
      const bool write = id >= 0 && j < r.s.len && (ms.decay != 1.0f || ms.in != ms.out || j >= old || (any >> ((k + i) & 31) & 1));
      before[i] = write && j < old ? ms.in[(int64_t)id * kKvPage + j % kKvPage] : 0.0f;
      writes |= write << i;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = __shfl_sync(0xffffffffu, ids, (k + i) & 31), tile = tile0 + warp + (k + i) * WARPS, j = tile * TILE + lane;
      if (!(writes >> i & 1)) continue;
      float votes = 0.0f;
      if (any >> ((k + i) & 31) & 1) {
        const float* x = kept + (int64_t)((tile - tile0) * TILE + lane) * cl.rows;
#pragma unroll 1
        for (int row = 0; row < rows; ++row) {
          const float2 ml = sh.part[0][row * PARTS];
          // a masked score is -inf; it takes no part, whatever the row's sum is
          if (x[row] != kNegInf) votes = fmaf(exp2_approx(x[row] - ml.x), ml.y, votes);
        }
      }
      ms.out[(int64_t)id * kKvPage + j % kKvPage] = j < old ? fmaf(ms.decay, before[i], votes) : votes;
    }
  }
  if (bad) record_device_error(kErrRange);
}

// ------------------------------------------------------------- many columns
// what the second kernel needs of a row: -M (0 where it sees nothing) and 1 / L, twice
__device__ __forceinline__ float4 finished(float m, float l) {
  const float minus = m == kNegInf ? 0.0f : -m, inv = l == 0.0f ? 0.0f : __frcp_rn(l);
  return make_float4(minus, minus, inv, inv);
}
// Here the columns are the rows of m16n8k16 and the tokens its columns: a lane's accumulators are pairs of tokens of one
// column (paired fp32 operations), and four chains of products run side by side. Scores stay in units of their
// column: x = a u, u = step raw + base b, so that max and difference are those of u; a is positive (a negative scale turns the
// query's sign), and large or tiny enough ones are clamped, where every weight is 0 or 1 anyway.
//
// A block of 64 columns as the first kernel leaves it for the second: fragments and constants, copied as they are.
constexpr int COLS = 64, SIXTEENS = COLS / 16;
template <int D>
struct __align__(16) Slab {
  uint4 frag[SIXTEENS][D / 16][32];  // columns g and g + 8 (fp32 queries: the parts of row g), by k step
  float4 ab[COLS];                   // a, a, b, b
  float4 ml[COLS];                   // -M, -M, 1 / L, 1 / L
  int p[COLS];                       // the row's position
};
// A tile's codes as B fragments of four eights of tokens, and its parameters: rows 2 t and 2 t + 1 of each.
template <int D>
struct Tile {
  uint32_t w[4][D / 32];
  uint4 par[4];
  __device__ __forceinline__ void load(const uint8_t* blk, int tile, int g, int t) {
    constexpr int WORDS = D / 32;
    const int row0 = (tile & 1) * TILE;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint8_t* p = blk + (row0 + e * 8 + g) * (D / 2) + t * (WORDS * 4);
      if (D == 128) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[e][0] = v.x, w[e][1] = v.y, w[e][2 % WORDS] = v.z, w[e][3 % WORDS] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[e][0] = v.x, w[e][1] = v.y;
      }
      par[e] = *reinterpret_cast<const uint4*>(blk + kKvPage * D + (row0 + e * 8 + 2 * t) * 8);
    }
  }
};
template <int D>
struct Unpacked {
  uint32_t u[4][D / 32][4];   // word: the two registers of each of its two products
  uint64_t step[4], base[4];  // of tokens 2 t and 2 t + 1
  __device__ __forceinline__ explicit Unpacked(const Tile<D>& k) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t a = k.w[e][i], a8 = a >> 8;
        u[e][i][0] = a & 0x000f000fu, u[e][i][1] = a & 0x00f000f0u, u[e][i][2] = a8 & 0x000f000fu, u[e][i][3] = a8 & 0x00f000f0u;
      }
      const float2 even = params(k.par[e].x), odd = params(k.par[e].z);
      step[e] = f2pack(even.x, odd.x), base[e] = f2pack(even.y, odd.y);
    }
  }
};
// the token (of its tile) of the lane's place j (0, 1) in eight e
__device__ __forceinline__ int token_at(int e, int t, int j) { return kv4_rho_inv(e * 8 + 2 * t + j); }

// u of sixteen columns against a tile: u[h][e] has column g + 8 h (fp32 queries: row g, h = 0 alone), tokens 2 t and 2 t + 1 of eight e.
template <int D, bool F32>
__device__ __forceinline__ void scores(const Unpacked<D>& k, const Slab<D>& sl, int j, int lane, const float4 (&ab)[2], uint64_t (&u)[2][4]) {
  float d[4][4];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const uint4 f = sl.frag[j][2 * i][lane], f2 = sl.frag[j][2 * i + 1][lane];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (i == 0) mma_first(d[e], f, k.u[e][0][0], k.u[e][0][1]);
      else mma16816(d[e], f.x, f.y, f.z, f.w, k.u[e][i][0], k.u[e][i][1]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) mma16816(d[e], f2.x, f2.y, f2.z, f2.w, k.u[e][i][2], k.u[e][i][3]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (F32) {
      u[0][e] = fma2(k.step[e], add2(f2pack(d[e][0], d[e][1]), f2pack(d[e][2], d[e][3])), mul2(k.base[e], f2pack(ab[0].z, ab[0].w)));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        u[h][e] = fma2(k.step[e], f2pack(d[e][2 * h], d[e][2 * h + 1]), mul2(k.base[e], f2pack(ab[h].z, ab[h].w)));
    }
  }
}

// The fragments and constants of columns [col0, col0 + 64): D / 8 lanes a row, 8 numbers each, all loads first.
template <int D, bool F32>
__device__ __forceinline__ void load_slab(const Kv4Attn& a, const Rows& r, int64_t col0, Slab<D>& sl) {
  constexpr int W = D / 8, PARTS = F32 ? 2 : 1, ROWS = COLS / PARTS, PER = THREADS / W, TIMES = ROWS / PER;
  static_assert(ROWS % PER == 0, "every thread takes as many rows");
  const int w = threadIdx.x % W, k0 = threadIdx.x / W, rows = r.votes * a.share, row0 = (int)(col0 / PARTS);
  float x[TIMES][8];
#pragma unroll
  for (int k = 0; k < TIMES; ++k) {
    const int row = row0 + k0 + k * PER, i = row / a.share;
    const bool there = row < rows;
    const int64_t at = there ? (int64_t)(r.s.q0 + r.s.n - r.votes + i) * a.q_stride + (int64_t)(r.h * a.share + row - i * a.share) * D + w : 0;
#pragma unroll
    for (int n = 0; n < 8; ++n)
      x[k][n] = !there ? 0.0f
                : F32  ? static_cast<const float*>(a.q)[at + W * n]
                       : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at + W * n]);
  }
#pragma unroll
  for (int k = 0; k < TIMES; ++k) {
    const int row = row0 + k0 + k * PER;
    float sum = 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int n = 0; n < 8; ++n) sum += x[k][n], top = max(top, __float_as_uint(x[k][n]) & 0x7fffffffu);
#pragma unroll
    for (int o = W / 2; o >= 1; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    int e = top == 0 ? 0 : 14 - ((int)(top >> 23) - 127);
    e = e > 127 ? 127 : e < -113 ? -113 : e;
    const float up = copysignf(__int_as_float((e + 127) << 23), a.scale);
    sum = row_sum<W>(x[k], sum, up, top);
    constexpr int WORDS = W / 4;
    // where the row's numbers stand: fp32 queries have 8 rows in sixteen columns, their parts 8 apart
    const int t = w / WORDS, word = w % WORDS, at = k0 + k * PER, j = at / (16 / PARTS), in = at % (16 / PARTS);
    const int col = j * 16 + in;
    float hi[8], lo[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      hi[n] = x[k][n] * up * (n & 1 ? 0.0625f : 1.0f);
      lo[n] = hi[n] - __half2float(__float2half_rn(hi[n]));
    }
    uint32_t* to = reinterpret_cast<uint32_t*>(&sl.frag[j][2 * word][(in & 7) * 4 + t]) + (F32 ? 0 : in >> 3);
    constexpr int NEXT = 32 * 4;  // words to the next k step
    to[0] = pack_half2(hi[0], hi[4]), to[2] = pack_half2(hi[1], hi[5]);
    to[NEXT] = pack_half2(hi[2], hi[6]), to[NEXT + 2] = pack_half2(hi[3], hi[7]);
    if (F32) {
      to[1] = pack_half2(lo[0], lo[4]), to[3] = pack_half2(lo[1], lo[5]);
      to[NEXT + 1] = pack_half2(lo[2], lo[6]), to[NEXT + 3] = pack_half2(lo[3], lo[7]);
    }
    if (w == 0) {
      const float c1 = __fmul_rn(fabsf(a.scale), kLog2e);
      const int f = 24 - e, half = f / 2;
      const float ca = __fmul_rn(__fmul_rn(c1, __int_as_float((half + 127) << 23)), __int_as_float((f - half + 127) << 23));
      const float aa = fminf(fmaxf(ca, kLeastA), kMostA), bb = __fmul_rn(sum, 5.9604644775390625e-8f);  // 2^-24
      sl.ab[col] = make_float4(aa, aa, or_nan(bb, top), or_nan(bb, top));
      sl.p[col] = row < rows ? r.position(row / a.share) : -1;
    }
  }
}
// First kernel: each column's maximum and sum over a chunk of tiles. A warp's running ones lie in shared memory.
template <int D>
struct __align__(16) RowsShared {
  Slab<D> sl;
  float4 run[WARPS][SIXTEENS][32];
  float2 part[WARPS][COLS];
};
template <int D, bool F32>
__global__ void __launch_bounds__(THREADS, 2) kv4_mass_rows_many(Kv4 c, Kv4Attn a, int voters, Plan pl, Stats st) {
  extern __shared__ __align__(16) uint8_t smem[];
  RowsShared<D>& sh = *reinterpret_cast<RowsShared<D>*>(smem);
  constexpr int PARTS = F32 ? 2 : 1, BLK = (int)kv4_block_bytes(D), HALVES = F32 ? 1 : 2;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
  bool bad = false;
  pdl_launch_dependents();
  const int64_t items = (int64_t)c.batch * c.kv_heads * pl.blocks * pl.chunks;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t rest = item / pl.chunks;
    const int chunk = (int)(item - rest * pl.chunks), unit = (int)(rest / pl.blocks), block = (int)(rest - (int64_t)unit * pl.blocks);
    const Rows r = rows_of(c, unit, voters, &bad);
    const int64_t rows = (int64_t)r.votes * a.share, col0 = (int64_t)block * COLS;
    if (col0 >= rows * PARTS) continue;
    const int tile0 = chunk * pl.chunk, tile1 = min(tile0 + pl.chunk, (r.s.len + TILE - 1) / TILE);
    const int first = r.position((int)(col0 / PARTS) / a.share), last = r.position((int)((min((col0 + COLS) / PARTS, rows) - 1) / a.share));
    const bool some = tile0 < tile1 && seen(a, first, last, tile0 * TILE, (tile1 - tile0) * TILE) != 0;
    if (!some && chunk) {
      for (int i = threadIdx.x; i < COLS; i += THREADS) st.part[item * COLS + i] = make_float2(kNegInf, 0.0f);
      continue;
    }
    int id = 0;
    const int mine = tile0 + warp + lane * WARPS;
    if (mine < tile1) {
      id = c.page_table[(int64_t)r.b * c.max_pages + mine / 2];
      if (id < 0 || id >= c.n_pages) bad = true, id = 0;
    }
    Tile<D> cur;
    const auto load = [&](int k) {
      const int from = __shfl_sync(0xffffffffu, id, k);
      const int tile = tile0 + warp + k * WARPS;
      if (tile < tile1) cur.load(c.pages + ((int64_t)from * c.kv_heads + r.h) * BLK, tile, g, t);
    };
    load_slab<D, F32>(a, r, col0, sh.sl);
    load(0);
#pragma unroll
    for (int j = 0; j < SIXTEENS; ++j) sh.run[warp][j][lane] = make_float4(kNegInf, 0.0f, kNegInf, 0.0f);
    __syncthreads();
    const int sixteens = (int)min((int64_t)SIXTEENS, (rows * PARTS - col0 + 15) / 16);
    for (int k = 0, tile = tile0 + warp; some && tile < tile1; ++k, tile += WARPS) {
      const Unpacked<D> now(cur);
      if (k < 31) load(k + 1);
      const int j0 = tile * TILE, sees = seen(a, first, last, j0, TILE);
      if (sees == 0) continue;
      // (masked tiles are few: their loop is apart from the other's)
      const auto columns = [&](auto masked) {
        constexpr bool MASKED = decltype(masked)::value;
#pragma unroll 1
        for (int j = 0; j < sixteens; ++j) {
          uint64_t u[2][4];
          const float4 ab[2] = {sh.sl.ab[j * 16 + g], sh.sl.ab[j * 16 + g + 8]};
          scores<D, F32>(now, sh.sl, j, lane, ab, u);
          float4 run = sh.run[warp][j][lane];
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            float2 x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = f2unpack(u[h][e]);
            if (MASKED) {
              const int p = sh.sl.p[j * 16 + g + 8 * h];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (!visible(a, p, j0 + token_at(e, t, 0))) x[e].x = kNegInf;
                if (!visible(a, p, j0 + token_at(e, t, 1))) x[e].y = kNegInf;
              }
            }
            float &m = h ? run.z : run.x, &l = h ? run.w : run.y;
            const float top = max3(max3(max3(x[0].x, x[0].y, x[1].x), x[1].y, x[2].x), max3(x[2].y, x[3].x, x[3].y), m);
            const float from = top == kNegInf ? 0.0f : top, aa = ab[h].x;
            const uint64_t a2 = f2pack(aa, aa), minus = f2pack(-from, -from);
            float s[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 y = f2unpack(mul2(a2, add2(f2pack(x[e].x, x[e].y), minus)));
              s[e] = exp2_approx(y.x) + exp2_approx(y.y);
            }
            l = fmaf(l, exp2_approx(aa * (m - from)), (s[0] + s[1]) + (s[2] + s[3]));
            m = top;
          }
          sh.run[warp][j][lane] = run;
        }
      };
      if (sees == 2) columns(std::false_type{});
      else columns(std::true_type{});
    }
#pragma unroll 1
    for (int j = 0; j < SIXTEENS; ++j) {
      const float4 run = sh.run[warp][j][lane];
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        float m = h ? run.z : run.x, l = h ? run.w : run.y;
        const float aa = sh.sl.ab[j * 16 + g + 8 * h].x;
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) join_u(aa, m, l, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, l, o));
        if (t == 0) sh.part[warp][j * 16 + g + 8 * h] = make_float2(m, l);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < COLS; i += THREADS) {
      if (F32 && (i & 8)) continue;
      float2 v = sh.part[0][i];
      for (int w = 1; w < WARPS; ++w) join_u(sh.sl.ab[i].x, v.x, v.y, sh.part[w][i].x, sh.part[w][i].y);
      st.part[item * COLS + i] = v;
      sh.sl.ml[i] = finished(v.x, v.y);  // what the second kernel needs where there is one chunk
    }
    __syncthreads();
    if (chunk == 0) {
      uint4* to = reinterpret_cast<uint4*>(st.slabs + rest * (int64_t)sizeof(Slab<D>));
      for (int i = threadIdx.x; i < (int)(sizeof(Slab<D>) / 16); i += THREADS) to[i] = reinterpret_cast<const uint4*>(&sh.sl)[i];
    }
    __syncthreads();  // the next item's columns
  }
  if (bad) record_device_error(kErrRange);
}

// Joins the chunks' maxima and sums of each block of columns (more than one chunk).
template <int D>
__global__ void __launch_bounds__(COLS) kv4_mass_sums(Kv4 c, Kv4Attn a, int voters, Plan pl, Stats st) {
  const int64_t items = (int64_t)c.batch * c.kv_heads * pl.blocks;
  pdl_launch_dependents();
  pdl_wait();
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int unit = (int)(item / pl.blocks), block = (int)(item - (int64_t)unit * pl.blocks);
    bool bad = false;
    const Rows r = rows_of(c, unit, voters, &bad);
    if ((int64_t)block * COLS >= (int64_t)r.votes * a.share * pl.parts || (pl.parts == 2 && (threadIdx.x & 8))) continue;
    Slab<D>& sl = *reinterpret_cast<Slab<D>*>(st.slabs + item * (int64_t)sizeof(Slab<D>));
    const int chunks = ((r.s.len + TILE - 1) / TILE + pl.chunk - 1) / pl.chunk;
    const float aa = sl.ab[threadIdx.x].x;
    float m = kNegInf, l = 0.0f;
    for (int k = 0; k < chunks; ++k) {
      const float2 v = st.part[(item * pl.chunks + k) * COLS + threadIdx.x];
      join_u(aa, m, l, v.x, v.y);
    }
    sl.ml[threadIdx.x] = finished(m, l);
  }
}

// Second kernel: a warp keeps its tile's codes and goes through a share of the blocks of columns, the next one's copy under
// way while it computes.
template <int D, bool F32>
__global__ void __launch_bounds__(THREADS, 2) kv4_mass_shares(Kv4 c, Kv4Attn a, Kv4Mass ms, Plan pl, Stats st) {
  extern __shared__ __align__(16) uint8_t smem[];
  Slab<D>* const slabs = reinterpret_cast<Slab<D>*>(smem);
  constexpr int PARTS = F32 ? 2 : 1, BLK = (int)kv4_block_bytes(D), PIECES = (int)(sizeof(Slab<D>) / 16);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
  bool bad = false;
  pdl_launch_dependents();
  // the groups of tiles outermost: with a causal mask the first ones have most to do
  const int units = c.batch * c.kv_heads;
  const int64_t items = (int64_t)units * pl.groups * pl.shares;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t rest = item / pl.shares;
    const int share = (int)(item - rest * pl.shares), group = (int)(rest / units), unit = (int)(rest - (int64_t)group * units);
    const Rows r = rows_of(c, unit, ms.voters, &bad);
    const int64_t rows = (int64_t)r.votes * a.share;
    const int all = (r.s.len + TILE - 1) / TILE, tile = group * WARPS + warp;
    if (rows == 0 || group * WARPS >= all) continue;
    const int blocks = (int)((rows * PARTS + COLS - 1) / COLS);
    const auto ends = [&](int block, int* first, int* last) {
      const int64_t col0 = (int64_t)block * COLS;
      *first = r.position((int)(col0 / PARTS) / a.share);
      *last = r.position((int)((min((col0 + COLS) / PARTS, rows) - 1) / a.share));
    };
    // the next block of this share from `block` on that sees any of the tiles
    const auto next = [&](int block) {
      for (; block < blocks; block += pl.shares) {
        int first, last;
        ends(block, &first, &last);
        if (seen(a, first, last, group * WARPS * TILE, WARPS * TILE)) break;
      }
      return block;
    };
    const auto copy = [&](int block, int buf) {
      if (block < blocks) {
        const uint8_t* from = st.slabs + ((int64_t)unit * pl.blocks + block) * (int64_t)sizeof(Slab<D>);
        const uint32_t to = smem_u32(&slabs[buf]);
        for (int i = threadIdx.x; i < PIECES; i += THREADS) cp_async_16(to + i * 16, from + i * 16, 16);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int block = next(share), buf = 0;
    Tile<D> k{};
    bool there = tile < all;
    int id = 0;
    if (there) {
      id = c.page_table[(int64_t)r.b * c.max_pages + tile / 2];
      if (id < 0 || id >= c.n_pages) bad = true, there = false;
      else k.load(c.pages + ((int64_t)id * c.kv_heads + r.h) * BLK, tile, g, t);
    }
    pdl_wait();
    copy(block, 0);
    const Unpacked<D> now(k);
    uint64_t votes[4] = {0, 0, 0, 0};  // of tokens 2 t and 2 t + 1 of the eights
    while (block < blocks) {
      const int then = next(block + pl.shares);
      copy(then, buf ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      int first, last;
      ends(block, &first, &last);
      const int j0 = tile * TILE, sees = there ? seen(a, first, last, j0, TILE) : 0;
      const Slab<D>& sl = slabs[buf];
      const int sixteens = (int)min((int64_t)SIXTEENS, (rows * PARTS - (int64_t)block * COLS + 15) / 16);
      const auto columns = [&](auto masked) {
        constexpr bool MASKED = decltype(masked)::value;
#pragma unroll 1
        for (int j = 0; j < sixteens; ++j) {
          uint64_t u[2][4];
          const float4 ab[2] = {sl.ab[j * 16 + g], sl.ab[j * 16 + g + 8]};
          scores<D, F32>(now, sl, j, lane, ab, u);
#pragma unroll
          for (int h = 0; h < (F32 ? 1 : 2); ++h) {
            const int p = sl.p[j * 16 + g + 8 * h];
            float4 ml = sl.ml[j * 16 + g + 8 * h];
            if (p < 0) ml.z = ml.w = 0.0f;  // no row, or one that sees nothing
            const uint64_t a2 = f2pack(ab[h].x, ab[h].y), minus = f2pack(ml.x, ml.y), inv = f2pack(ml.z, ml.w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 y = f2unpack(mul2(a2, add2(u[h][e], minus)));
              const uint64_t more = fma2(f2pack(exp2_approx(y.x), exp2_approx(y.y)), inv, votes[e]);
              if (MASKED) {
                const float2 v = f2unpack(votes[e]), w = f2unpack(more);
                votes[e] = f2pack(visible(a, p, j0 + token_at(e, t, 0)) ? w.x : v.x, visible(a, p, j0 + token_at(e, t, 1)) ? w.y : v.y);
              } else {
                votes[e] = more;
              }
            }
          }
        }
      };
      if (sees == 2) columns(std::false_type{});
      else if (sees) columns(std::true_type{});
      __syncthreads();  // the buffer is copied into again
      block = then, buf ^= 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // over the eight lanes that share tokens; lane g = 2 e + j writes place j of eight e
    float mine = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float2 v = f2unpack(votes[e]);
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) v.x += __shfl_xor_sync(0xffffffffu, v.x, o), v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      if (g >> 1 == e) mine = g & 1 ? v.y : v.x;
    }
    const int in = token_at(g >> 1, t, g & 1), j = tile * TILE + in;
    if (pl.shares > 1) {
      st.votes[((((int64_t)unit * pl.groups + group) * pl.shares + share) * WARPS + warp) * TILE + in] = mine;
    } else if (there && j < r.s.len) {
      const int64_t at = ((int64_t)id * c.kv_heads + r.h) * kKvPage + j % kKvPage;
      ms.out[at] = j < r.s.len - r.s.n ? fmaf(ms.decay, ms.in[at], mine) : mine;
    }
    __syncthreads();
  }
  pdl_wait();
  if (bad) record_device_error(kErrRange);
}

__global__ void __launch_bounds__(THREADS) kv4_mass_join(Kv4 c, Kv4Mass ms, Plan pl, Stats st) {
  const int64_t items = (int64_t)c.batch * c.kv_heads * pl.groups;
  pdl_wait();
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int unit = (int)(item / pl.groups), group = (int)(item - (int64_t)unit * pl.groups);
    bool bad = false;
    const Rows r = rows_of(c, unit, ms.voters, &bad);
    const int j = group * (WARPS * TILE) + threadIdx.x;
    if (r.votes == 0 || j >= r.s.len) continue;
    const int id = c.page_table[(int64_t)r.b * c.max_pages + j / kKvPage];
    if (id < 0 || id >= c.n_pages) continue;
    float got = 0.0f;
    for (int s = 0; s < pl.shares; ++s) got += st.votes[(item * pl.shares + s) * (WARPS * TILE) + threadIdx.x];
    const int64_t at = ((int64_t)id * c.kv_heads + r.h) * kKvPage + j % kKvPage;
    ms.out[at] = j < r.s.len - r.s.n ? fmaf(ms.decay, ms.in[at], got) : got;
  }
}

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }
unsigned grid_of(int64_t items) { return (unsigned)(items < (1 << 20) ? items : (1 << 20)); }

// rows of a unit, at most
int64_t rows_of_plan(const Kv4& c, int share, int voters) {
  int votes = voters < c.max_q ? voters : c.max_q;
  votes = votes < c.total_q ? votes : c.total_q;
  return (int64_t)votes * share;
}
Plan plan_of(const Kv4& c, int share, int voters, bool f32, int num_sms) {
  Plan p{};
  p.parts = f32 ? 2 : 1;
  p.votes = voters < c.max_q ? voters : c.max_q;
  p.votes = p.votes < c.total_q ? p.votes : c.total_q;
  const int64_t cols = (int64_t)p.votes * share * p.parts, units = (int64_t)c.batch * c.kv_heads;
  p.nt = cols <= 8 ? 1 : cols <= 16 ? 2 : COLS / 8;
  p.blocks = (int)((cols + p.nt * 8 - 1) / (p.nt * 8));
  p.tiles = (c.max_kv + TILE - 1) / TILE;
  // a chunk: as many tiles as leave each SM several blocks
  const int64_t slots = (int64_t)num_sms * (p.nt == 1 ? 3 : p.nt == 2 ? 2 : 4) * WARPS;
  int64_t per = (units * p.blocks * p.tiles + slots - 1) / slots;
  per = per < 1 ? 1 : per > MAX_CHUNK / WARPS ? MAX_CHUNK / WARPS : per;
  p.chunk = (int)per * WARPS;
  p.chunks = (p.tiles + p.chunk - 1) / p.chunk;
  if (p.nt == COLS / 8) {
    p.groups = (p.tiles + WARPS - 1) / WARPS;
    const int64_t all = units * (p.groups > 0 ? p.groups : 1);
    const int64_t s = ((int64_t)num_sms * 4 + all - 1) / all;
    p.shares = (int)(s < 1 ? 1 : s > p.blocks ? p.blocks : s);
  }
  return p;
}
int64_t part_bytes(const Kv4& c, const Plan& p) { return align256((int64_t)c.batch * c.kv_heads * p.blocks * p.chunks * p.nt * 8 * 8); }
int64_t votes_bytes(const Kv4& c, const Plan& p) {
  return p.shares > 1 ? align256((int64_t)c.batch * c.kv_heads * p.groups * p.shares * WARPS * TILE * 4) : 0;
}
// Scores are kept while the batch's sizes leave room for no more than this: a pool of caches should not need a call's workspace of
// its own size. Beyond it they are made again. Measured, us, kept and made again (5 heads x 128): 4 rows, 2 x 131007 tokens (21
// MB) 33.6, 44.8; 16 x 131007 (168 MB) 218, 298; 64 x 131007 (671 MB) 810, 1087; 64 x 1000 with room for 131072 (671 MB) 32.0,
// 38.7; 16 rows, 16 x 131007 (671 MB) 448, 536.
constexpr int64_t kScoresMost = 256 << 20;
int64_t scores_bytes(const Kv4& c, const Plan& p, int share) {
  const int64_t bytes = p.shares ? 0 : align256((int64_t)c.batch * c.kv_heads * p.votes * share * p.tiles * TILE * 4);
  return bytes > kScoresMost ? 0 : bytes;
}
int64_t slabs_bytes(const Kv4& c, const Plan& p, int dim) {
  return p.shares ? align256((int64_t)c.batch * c.kv_heads * p.blocks * (int64_t)(dim == 128 ? sizeof(Slab<128>) : sizeof(Slab<64>))) : 0;
}

// The clusters that take the units, if their blocks' scores fit: no more blocks than that needs. For sequences of up to 256
// tokens, and where the units fill the GPU by themselves; else two kernels. Measured, us (5 heads x 128, one token of each sequence),
// one kernel (there with clusters that fill the GPU) and two: 250 tokens 5.1, 5.6; 300 6.1, 5.5; 25000 21.3, 8.2; 32 sequences of
// 1000 9.8, 8.9; 48 of 1000 10.5, 13.4; 64 of 17 to 8175 45.7, 53.5.
Cluster cluster_of(const Kv4& c, const Plan& p, int share, int num_sms) {
  Cluster k{1, 0, p.votes * share};
  const int64_t units = (int64_t)c.batch * c.kv_heads, row_bytes = (int64_t)k.rows * 4 * TILE;
  if (p.tiles > WARPS && units * 2 <= num_sms * 3) return k;
  const auto bytes = [&](int n) { return (p.tiles + n - 1) / n * row_bytes; };
  while (k.blocks < 8 && bytes(k.blocks) > kScoreBytes) k.blocks *= 2;
  k.tiles = bytes(k.blocks) > kScoreBytes ? 0 : (p.tiles + k.blocks - 1) / k.blocks;
  return k;
}
template <int D, int NT, bool F32>
cudaError_t launch_cluster(const Kv4& c, const Kv4Attn& a, const Kv4Mass& m, const Cluster& k, cudaStream_t st) {
  auto kernel = kv4_mass_cluster<D, NT, F32>;
  static std::atomic<uint64_t> configured{0};
  if (cudaError_t e = allow_smem(configured, kernel, kScoreBytes)) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = k.blocks, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(c.batch * c.kv_heads * k.blocks));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = (size_t)k.tiles * TILE * k.rows * 4;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, c, a, m, k);
}

template <int D, int NT, bool F32>
cudaError_t launch_few(const Kv4& c, const Kv4Attn& a, const Kv4Mass& m, const Plan& p, const Stats& s, cudaStream_t st) {
  const Cluster k = cluster_of(c, p, a.share, 152);
  if (k.tiles) return launch_cluster<D, NT, F32>(c, a, m, k, st);
  const int64_t units = (int64_t)c.batch * c.kv_heads;
  kv4_mass_rows<D, NT, F32><<<grid_of(units * p.chunks), THREADS, 0, st>>>(c, a, m.voters, p, s);
  if (cudaError_t e = cudaGetLastError()) return e;
  if (!s.scores) return launch_behind(kv4_mass_again<D, NT, F32>, grid_of(units * p.chunks), THREADS, 0, st, c, a, m, p, s);
  return launch_behind(kv4_mass_votes<NT, F32>, grid_of(units * p.chunks), THREADS, 0, st, c, a, m, p, s);
}
template <int D, bool F32>
cudaError_t launch_many(const Kv4& c, const Kv4Attn& a, const Kv4Mass& m, const Plan& p, const Stats& s, cudaStream_t st) {
  const int64_t units = (int64_t)c.batch * c.kv_heads;
  const int rows_smem = (int)sizeof(RowsShared<D>), shares_smem = 2 * (int)sizeof(Slab<D>);
  static std::atomic<uint64_t> configured[2];
  if (cudaError_t e = allow_smem(configured[0], kv4_mass_rows_many<D, F32>, rows_smem)) return e;
  if (cudaError_t e = allow_smem(configured[1], kv4_mass_shares<D, F32>, shares_smem)) return e;
  kv4_mass_rows_many<D, F32><<<grid_of(units * p.blocks * p.chunks), THREADS, rows_smem, st>>>(c, a, m.voters, p, s);
  if (cudaError_t e = cudaGetLastError()) return e;
  if (p.chunks > 1)
    if (cudaError_t e = launch_behind(kv4_mass_sums<D>, grid_of(units * p.blocks), COLS, 0, st, c, a, m.voters, p, s)) return e;
  if (cudaError_t e = launch_behind(kv4_mass_shares<D, F32>, grid_of(units * p.groups * p.shares), THREADS, shares_smem, st, c, a, m, p, s)) return e;
  return p.shares > 1 ? launch_behind(kv4_mass_join, grid_of(units * p.groups), THREADS, 0, st, c, m, p, s) : cudaSuccess;
}
template <int D, bool F32>
cudaError_t by_columns(const Kv4& c, const Kv4Attn& a, const Kv4Mass& m, const Plan& p, const Stats& s, cudaStream_t st) {
  if (p.tiles == 0) return cudaSuccess;
  if (p.nt == 1) return launch_few<D, 1, F32>(c, a, m, p, s, st);
  if (p.nt == 2) return launch_few<D, 2, F32>(c, a, m, p, s, st);
  return launch_many<D, F32>(c, a, m, p, s, st);
}

}  // namespace

int64_t kv4_mass_ws_bytes(const Kv4& c, int dim, int q_heads, int voters) {
  int64_t most = 0;  // whatever the queries' type
  for (int f32 = 0; f32 < 2; ++f32) {
    const int64_t rows = rows_of_plan(c, q_heads / c.kv_heads, voters);
    if (mass_on_tc(rows, f32 != 0)) {
      const int64_t n = kv4_mass_tc_ws_bytes(c, dim, q_heads / c.kv_heads, rows, f32 != 0);
      most = n > most ? n : most;
      continue;
    }
    const Plan p = plan_of(c, q_heads / c.kv_heads, voters, f32, 152);
    if (p.tiles == 0 || (p.nt <= 2 && cluster_of(c, p, q_heads / c.kv_heads, 152).tiles)) continue;
    const int64_t n = part_bytes(c, p) + votes_bytes(c, p) + slabs_bytes(c, p, dim) + scores_bytes(c, p, q_heads / c.kv_heads);
    most = n > most ? n : most;
  }
  return most;
}
cudaError_t launch_kv4_mass(const Kv4& c, int dim, const Kv4Attn& a, const Kv4Mass& m, void* ws, int num_sms, cudaStream_t st) {
  const int64_t rows = rows_of_plan(c, a.share, m.voters);
  if (mass_on_tc(rows, !a.bf16)) return launch_kv4_mass_tc(c, dim, a, m, rows, ws, st);
  const Plan p = plan_of(c, a.share, m.voters, !a.bf16, 152);
  uint8_t* at = static_cast<uint8_t*>(ws);
  const Stats s{reinterpret_cast<float2*>(at), reinterpret_cast<float*>(at + part_bytes(c, p)), at + part_bytes(c, p) + votes_bytes(c, p),
                scores_bytes(c, p, a.share) ? reinterpret_cast<float*>(at + part_bytes(c, p)) : nullptr};
  if (dim == 128) return a.bf16 ? by_columns<128, false>(c, a, m, p, s, st) : by_columns<128, true>(c, a, m, p, s, st);
  return a.bf16 ? by_columns<64, false>(c, a, m, p, s, st) : by_columns<64, true>(c, a, m, p, s, st);
}

cudaError_t read_clear_device_error_kv4_mass(int* value) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, g_device_error, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
}

}  // namespace bitnet
