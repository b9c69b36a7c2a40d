// kv4_mass_tc.cu -- the attention weight that cached tokens gather from many rows, on the 5th-generation tensor cores.
//
// A unit's rows (of a sequence: voting tokens x heads that share a key/value head) go in blocks of 128, its tokens in tiles of
// 128 (two pages). Scores of a block and a tile are one 128 x 128 product with K = D in tensor memory, codes as exact
// fp16 subnormals c 2^-24 (c 2^-20 for every second one; q' carries the 2^-4), fp32 queries as two parts with
// a product each. As for few rows (kv4_mass.cu), x = a u, u = step raw + base b; the first kernel finds each row's maximum M
// of u and its sum L, the second adds up 2^(a (u - M)) / L.
//
// First kernel: rows are the lanes of the accumulator, so that a thread has its row's constants, maximum and sum in registers
// and a token's parameters come from shared memory, a pair of tokens at a time. Second kernel: tokens are the lanes, so that a
// thread adds up its token's votes and a pair of rows' constants comes from shared memory. In both the products of one
// tile (block) run while the last one's scores are worked off; two blocks an SM cover what is left.
//
// Bound by the latency of a tile, of which a block has up to 16 in turn, with 41 to 46% of the issue slots used (some 720 instructions
// for a warp's 64 x 32 scores, 320 of them their arithmetic). Measured (20 and 5 heads x 128): 2048 tokens that all vote 67.1 us (21
// GFLOP in the two passes; fp32 queries 98.4), 4096 179 us, the last 64 of 5 prompts of 1000 to 9000 tokens 61.4 us (94.5); on
// m16n8k16 the first and last took 114.5 and 87.
#include <type_traits>

#include "kv4_mass.cuh"
#include "smem_limit.h"

namespace bitnet {
namespace {

constexpr int THREADS = 256;
constexpr int TOK = 128, ROWS = 128;

struct Plan {
  int blocks, tiles, chunk, chunks, shares;
  int64_t room;  // places for a head's blocks of rows, all sequences' together; 0: a place for each unit and block
};
// Where a block of rows lies in the workspace. Sequences that have far fewer rows than the longest lie one behind another: those of the
// packed rows [q0, q0 + n) take ceil(n share / ROWS) places at most, from floor(q0 share / ROWS) + b on, which is up to where the
// next one's begin.
__device__ __forceinline__ int64_t place_of(const Plan& pl, const Rows& r, int unit, int share, int block) {
  return (pl.room ? r.h * pl.room + (int64_t)r.s.q0 * share / ROWS + r.b : (int64_t)unit * pl.blocks) + block;
}
// What the second kernel needs of a block's rows, in pairs.
struct Constants {
  float4 ab[ROWS / 2];  // a0, a1, b0, b1
  float4 ml[ROWS / 2];  // -M0, -M1, 1 / L0, 1 / L1
  int2 seen[ROWS];      // the row's position (-1: no row), and where its window begins
};
template <int D, bool F32>
struct Shape {
  static constexpr int PARTS = F32 ? 2 : 1;
  static constexpr int IMAGE = 128 * D * 2;               // an operand: D / 64 atoms of 128 rows x 128 bytes
  static constexpr int BLOCK = IMAGE * PARTS + (int)sizeof(Constants);  // as the first kernel leaves it
  static constexpr int CON = 3 * 1024;                    // place of the constants in shared memory
  static constexpr int ROWS_SMEM = IMAGE * PARTS + CON + 2 * IMAGE + 3 * 1024 + 1024;
  static constexpr int VOTES_SMEM = IMAGE + 2 * IMAGE * PARTS + 3 * CON + 1024;
  static constexpr int BLOCKS = F32 && D == 128 ? 1 : 2;  // resident on an SM
};
static_assert(sizeof(Constants) <= 3 * 1024 && sizeof(Constants) % 16 == 0, "");

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// byte offset of 16-byte chunk c of row r in an operand of 64-column atoms, K-major, 128-byte swizzle
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return (uint32_t)((c >> 3) * (128 * 128) + (r >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r != 0;
}
// the token (of its half of a tile) in row r of the half: pages keep keys in the order rho
__device__ __forceinline__ int token_of(int r) { return kv4_rho_inv(r); }

// D[tmem] = A B^T over both parts of the operand that has two (PA parts of A, PB of B), by one lane
template <int D, int PA, int PB>
__device__ __forceinline__ void issue(uint32_t d_tmem, uint32_t a_smem, uint32_t b_smem, uint64_t* bar) {
  constexpr int IMAGE = 128 * D * 2;
#pragma unroll
  for (int p = 0; p < PA * PB; ++p) {
    const uint64_t ad = make_sw128_kmajor_desc(a_smem + (PA > 1 ? p * IMAGE : 0)), bd = make_sw128_kmajor_desc(b_smem + (PB > 1 ? p * IMAGE : 0));
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const uint64_t o = (uint64_t)((s >> 2) * ((128 * 128) >> 4) + (s & 3) * 2);
      mma_f16_ss(d_tmem, ad + o, bd + o, make_idesc_f16_f32(128, 128), p > 0 || s > 0);
    }
  }
  mma_commit(bar);
}

// A thread's part of a tile: half a key row, as codes.
template <int D>
struct Half {
  static constexpr int WORDS = D / 16;
  uint32_t w[WORDS], par;
  // id: of the page that has the row; -1 for none
  __device__ __forceinline__ void load(const Kv4& c, int id, int h, int row, int half) {
    if (id < 0) {
#pragma unroll
      for (int i = 0; i < WORDS; ++i) w[i] = 0;
      par = 0;
      return;
    }
    const uint8_t* blk = c.pages + ((int64_t)id * c.kv_heads + h) * kv4_block_bytes(D);
#pragma unroll
    for (int i = 0; i < WORDS; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(blk + row * (D / 2) + half * (D / 4) + i * 4);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
    par = *reinterpret_cast<const uint32_t*>(blk + kKvPage * D + row * 8);
  }
  __device__ __forceinline__ void store(uint32_t image, int row, int half) const {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      const uint32_t a = w[i], a8 = a >> 8;
      sts128(image + chunk_at(row, half * WORDS + i), a & 0x000f000fu, a & 0x00f000f0u, a8 & 0x000f000fu, a8 & 0x00f000f0u);
    }
  }
};

// The queries of rows row0 .. row0 + 127 of a unit as an operand, and their constants: W = D / 8 lanes a row. Lane w
// loads numbers 8 w .. 8 w + 7, which are nibble n = w / (W / 8) of eight words; nibbles n and n + 4 of a word lie side by side
// in the operand, so half of a lane's numbers go to the lane that has the other nibble, and half of that one's come here.
template <int D, bool F32>
__device__ __forceinline__ void load_block(const Kv4Attn& a, const Rows& r, int row0, uint32_t image, Constants& con) {
  constexpr int W = D / 8, PER = THREADS / W, BATCH = 4, IMAGE = 128 * D * 2;
  const int w = threadIdx.x % W, rows = r.votes * a.share, n = w / (W / 8);
  const bool high = n >= 4;
  const int word0 = 8 * w % W + (high ? 4 : 0);  // of the four words that the lane stores
  const float odd = n & 1 ? 0.0625f : 1.0f;
  // voting row and head of row row0 + k: x / share for x < 256 and share <= 128 by a product
  const int first = row0 / a.share, rest = row0 - first * a.share, by = 65536 / a.share + 1;
  const int64_t from = (int64_t)(r.s.q0 + r.s.n - r.votes + first) * a.q_stride + (int64_t)r.h * a.share * D + 8 * w;
#pragma unroll 1
  for (int k0 = threadIdx.x / W; k0 < ROWS; k0 += PER * BATCH) {
    float x[BATCH][8];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int in = k0 + k * PER, i = (rest + in) * by >> 16;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[k][j] = 0.0f;
      if (row0 + in >= rows) continue;
      const int64_t at = from + i * a.q_stride + (rest + in - i * a.share) * D;
      if (F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
        const float4 u = __ldg(p), v = __ldg(p + 1);
        x[k][0] = u.x, x[k][1] = u.y, x[k][2] = u.z, x[k][3] = u.w, x[k][4] = v.x, x[k][5] = v.y, x[k][6] = v.z, x[k][7] = v.w;
      } else {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at));
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) x[k][2 * j] = __uint_as_float(u[j] << 16), x[k][2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int in = k0 + k * PER;
      float sum = ((x[k][0] + x[k][1]) + (x[k][2] + x[k][3])) + ((x[k][4] + x[k][5]) + (x[k][6] + x[k][7]));
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[k][j]) & 0x7fffffffu);
#pragma unroll
      for (int o = W / 2; o >= 1; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      // the row's power of two: its largest number comes to [2^14, 2^15)
      int e = top == 0 ? 0 : 14 - ((int)(top >> 23) - 127);
      e = e > 127 ? 127 : e < -113 ? -113 : e;
      const float up = copysignf(__int_as_float((e + 127) << 23), a.scale);
      sum = row_sum<W>(x[k], sum, up, top);
#pragma unroll
      for (int part = 0; part < (F32 ? 2 : 1); ++part) {
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float y0 = x[k][2 * j] * up * odd, y1 = x[k][2 * j + 1] * up * odd;
          h[j] = pack_half2(y0, y1);
          if (part) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
            h[j] = pack_half2(y0 - f.x, y1 - f.y);
          }
        }
        const uint32_t to = image + part * IMAGE + 4 * (n & 3);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? h[j] : h[2 + j], W / 2), own = high ? h[2 + j] : h[j];
          const uint32_t lo = high ? got : own, hi = high ? own : got;
          st_shared_u32(to + chunk_at(in, word0 + 2 * j), __byte_perm(lo, hi, 0x5410));
          st_shared_u32(to + chunk_at(in, word0 + 2 * j + 1), __byte_perm(lo, hi, 0x7632));
        }
      }
      if (w == 0) {  // the row's constants begin with these
        float* ab = reinterpret_cast<float*>(&con.ab[in >> 1]) + (in & 1);
        ab[0] = __int_as_float(e);
        ab[2] = or_nan(sum, top);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < ROWS) {
    const int in = threadIdx.x;
    float* ab = reinterpret_cast<float*>(&con.ab[in >> 1]) + (in & 1);
    const float c1 = __fmul_rn(fabsf(a.scale), kLog2e);
    const int f = 24 - __float_as_int(ab[0]), half = f / 2;
    const float ca = __fmul_rn(__fmul_rn(c1, __int_as_float((half + 127) << 23)), __int_as_float((f - half + 127) << 23));
    ab[0] = fminf(fmaxf(ca, kLeastA), kMostA);
    ab[2] = __fmul_rn(ab[2], 5.9604644775390625e-8f);  // 2^-24
    const int p = row0 + in < rows ? r.position(first + ((rest + in) * by >> 16)) : -1;
    con.seen[in] = make_int2(p, window_from(a, p));
  }
}

// Goes through steps (tiles, blocks) that have anything to do. What 32 of them see is found by the 32 lanes at once: asked
// again for each step it cost 3 to 7% of the time (2048 voting tokens 72 us, 4096 201; so 69.7 and 187). All lanes hold the same.
struct Walk {
  int first = 0, end = 0;  // the steps that `any` and `all` tell of
  uint32_t any = 0, all = 0;
  // the next step from k on, `last` if there is none; sees(k): 0 nothing, 1 some, 2 all
  template <class Sees>
  __device__ __forceinline__ int next(int k, int last, bool* whole, Sees sees) {
    while (k < last) {
      if (k >= end) {
        const int at = k + (int)(threadIdx.x % 32), v = at < last ? sees(at) : 0;
        first = k, end = k + 32;
        any = __ballot_sync(0xffffffffu, v > 0), all = __ballot_sync(0xffffffffu, v == 2);
      }
      const uint32_t left = any >> (k - first);
      if (left) {
        k += __ffs(left) - 1;
        *whole = all >> (k - first) & 1;
        return k;
      }
      k = end;
    }
    return last;
  }
};

// The lowest n bits.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }

// The first and last position of a block's rows.
__device__ __forceinline__ void ends_of(const Kv4Attn& a, const Rows& r, int row0, int* first, int* last) {
  *first = r.position(row0 / a.share);
  *last = r.position((min(row0 + ROWS, r.votes * a.share) - 1) / a.share);
}

template <int D, bool F32>
__global__ void __launch_bounds__(THREADS, Shape<D, F32>::BLOCKS) kv4_mass_tc_rows(Kv4 c, Kv4Attn a, int voters, Plan pl, uint8_t* blocks, float2* part) {
  using S = Shape<D, F32>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t done[2], all_done;
  __shared__ uint32_t tmem_slot;
  __shared__ float2 halves[ROWS];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  Constants& con = *reinterpret_cast<Constants*>(smem + S::IMAGE * S::PARTS);
  constexpr int KEYS = S::IMAGE * S::PARTS + S::CON, TABLE = KEYS + 2 * S::IMAGE;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, half = warp >> 2, row = (warp & 3) * 32 + lane;
  if (threadIdx.x == 0) {
    mbar_init(&done[0], 1), mbar_init(&done[1], 1), mbar_init(&all_done, 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_launch_dependents();  // not before: the next kernel's blocks take tensor memory and then wait for all of these
  bool bad = false, abort = false;
  uint32_t issued = 0;  // products so far: buffer issued & 1
  // the last blocks of rows outermost: with a causal mask they have most to do
  const int units = c.batch * c.kv_heads;
  const int64_t items = (int64_t)units * pl.blocks * pl.chunks;
  for (int64_t at = blockIdx.x; at < items; at += gridDim.x) {
    const int64_t rest = at / pl.chunks;
    const int chunk = (int)(at - rest * pl.chunks), behind = (int)(rest / units), unit = (int)(rest - (int64_t)behind * units);
    const int block = pl.blocks - 1 - behind;
    const Rows r = rows_of(c, unit, voters, &bad);
    const int rows = r.votes * a.share, row0 = block * ROWS;
    if (row0 >= rows) continue;
    const int64_t place = place_of(pl, r, unit, a.share, block), item = place * pl.chunks + chunk;
    const int t0 = chunk * pl.chunk, t1 = min(t0 + pl.chunk, (r.s.len + TOK - 1) / TOK), pages = (r.s.len + kKvPage - 1) / kKvPage;
    int first, last;
    ends_of(a, r, row0, &first, &last);
    Walk walk;
    const auto next = [&](int t, bool* whole) { return walk.next(t, t1, whole, [&](int k) { return seen(a, first, last, k * TOK, TOK); }); };
    bool t_whole = false, then_whole = false, after_whole = false, before_whole = false;
    int t = next(t0, &t_whole);
    if (t >= t1 && chunk) {
      for (int i = threadIdx.x; i < ROWS; i += THREADS) part[item * ROWS + i] = make_float2(kNegInf, 0.0f);
      continue;
    }
    const int krow = threadIdx.x >> 1, khalf = threadIdx.x & 1;
    // ids are asked for a tile before they are used, and looked at then
    constexpr int NONE = INT32_MIN;
    const auto page_id = [&](int tile) {
      const int page = tile * 2 + (krow >> 6);
      return tile < t1 && page < pages ? c.page_table[(int64_t)r.b * c.max_pages + page] : NONE;
    };
    const auto checked = [&](int id) {
      if (id >= 0 && id < c.n_pages) return id;
      bad |= id != NONE;
      return -1;
    };
    Half<D> codes;
    codes.load(c, checked(page_id(t)), r.h, krow & 63, khalf);
    int then = t < t1 ? next(t + 1, &then_whole) : t1, id_then = page_id(then);
    load_block<D, F32>(a, r, row0, base, con);
    __syncthreads();
    const float4 ab4 = con.ab[row >> 1];
    const float aa = row & 1 ? ab4.y : ab4.x, bb = row & 1 ? ab4.w : ab4.z;
    const uint64_t a2 = f2pack(aa, aa), b2 = f2pack(bb, bb);
    const int p = con.seen[row].x, lo = con.seen[row].y;
    float m = kNegInf, l = 0.0f;
    int before = -1;  // the tile whose scores are to be worked off
    while (t < t1 || before >= 0) {
      const uint32_t buf = issued & 1;
      if (t < t1) {
        codes.store(base + KEYS + buf * S::IMAGE, krow, khalf);
        if (khalf == 0) {
          const float2 sb = params(codes.par);
          // (three tables: a warp may still read the one before the last)
          float* tab = reinterpret_cast<float*>(smem + TABLE + (issued % 3) * 1024 + (krow >> 1) * 16) + (krow & 1);
          tab[0] = sb.x, tab[2] = sb.y;
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
      if (t < t1 && warp == 0) {
        if (elect_one()) issue<D, S::PARTS, 1>(tmem + buf * 128, base, base + KEYS + buf * S::IMAGE, &done[buf]);
        __syncwarp();
      }
      if (then < t1) codes.load(c, checked(id_then), r.h, krow & 63, khalf);
      const int after = then < t1 ? next(then + 1, &after_whole) : t1, id_after = page_id(after);
      if (before >= 0) {
        const uint32_t was = issued - 1, at = was & 1;
        mbar_wait_warp(&done[at], (was >> 1) & 1, &abort);
        tc_fence_after();
        const int j0 = before * TOK + half * 64;
        const uint32_t ts = tmem + ((uint32_t)((warp & 3) * 32) << 16) + at * 128 + half * 64;
        const float4* tab = reinterpret_cast<const float4*>(smem + TABLE + (was % 3) * 1024) + half * 32;
        const auto work = [&](auto masked) {
          constexpr bool MASKED = decltype(masked)::value;
#pragma unroll 1
          for (int k = 0; k < 2; ++k) {
            uint32_t s[32];
            tmem_ld_32x32b_x32(ts + k * 32, s);
            // which of the 32 tokens the row sees, in the order of their positions
            const int j = j0 + k * 32;
            const uint32_t sees = MASKED ? below(p + 1 - j) & (~below(lo - j) | below(a.sinks - j)) : 0;
            tmem_ld_wait();
            uint64_t u[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float4 sb = tab[k * 16 + i];
              u[i] = fma2(f2pack(sb.x, sb.y), f2pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), mul2(f2pack(sb.z, sb.w), b2));
              if (MASKED) {
                float2 v = f2unpack(u[i]);
                if (!(sees & 1u << token_of(2 * i))) v.x = kNegInf;
                if (!(sees & 1u << token_of(2 * i + 1))) v.y = kNegInf;
                u[i] = f2pack(v.x, v.y);
              }
            }
            float top[4] = {m, m, m, m};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 v = f2unpack(u[i]);
              top[i & 3] = max3(top[i & 3], v.x, v.y);
            }
            const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), from = now == kNegInf ? 0.0f : now;
            const uint64_t minus = f2pack(-from, -from);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 y = f2unpack(mul2(a2, add2(u[i], minus)));
              sum[i & 1] = add2(sum[i & 1], f2pack(exp2_approx(y.x), exp2_approx(y.y)));
            }
            const float2 e = f2unpack(add2(sum[0], sum[1]));
            l = fmaf(l, exp2_approx(aa * (m - from)), e.x + e.y);
            m = now;
          }
        };
        if (before_whole) work(std::false_type{});
        else work(std::true_type{});
      }
      before = -1;
      if (t < t1) before = t, before_whole = t_whole, ++issued;
      t = then, t_whole = then_whole, then = after, then_whole = after_whole, id_then = id_after;
    }
    if (half) halves[row] = make_float2(m, l);
    __syncthreads();
    if (!half) {
      join_u(aa, m, l, halves[row].x, halves[row].y);
      part[item * ROWS + row] = make_float2(m, l);
      // what the second kernel needs where there is one chunk
      float* ml = reinterpret_cast<float*>(&con.ml[row >> 1]) + (row & 1);
      const bool none = p < 0 || m == kNegInf;
      ml[0] = none ? 0.0f : -m;
      ml[2] = p < 0 || l == 0.0f ? 0.0f : __frcp_rn(l);
    }
    __syncthreads();
    if (chunk == 0) {
      uint4* to = reinterpret_cast<uint4*>(blocks + place * (int64_t)S::BLOCK);
      for (int i = threadIdx.x; i < S::BLOCK / 16; i += THREADS) to[i] = reinterpret_cast<const uint4*>(smem)[i];
    }
    __syncthreads();  // the next item's queries
  }
  // what was issued ends before the tensor memory is given back, whichever wait gave up
  if (warp == 0) {
    if (elect_one()) mma_commit(&all_done);
    __syncwarp();
    abort = false;
    mbar_wait_warp(&all_done, 0, &abort);
  }
  if (bad) record_device_error(kErrRange);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 256);
}

// Joins the chunks' maxima and sums of each block of rows (more than one chunk).
template <int D, bool F32>
__global__ void __launch_bounds__(ROWS) kv4_mass_tc_sums(Kv4 c, Kv4Attn a, int voters, Plan pl, uint8_t* blocks, const float2* part) {
  using S = Shape<D, F32>;
  const int64_t items = (int64_t)c.batch * c.kv_heads * pl.blocks;
  pdl_launch_dependents();
  pdl_wait();
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int unit = (int)(item / pl.blocks), block = (int)(item - (int64_t)unit * pl.blocks), row = threadIdx.x;
    bool bad = false;
    const Rows r = rows_of(c, unit, voters, &bad);
    if (block * ROWS >= r.votes * a.share) continue;
    const int64_t place = place_of(pl, r, unit, a.share, block);
    Constants& con = *reinterpret_cast<Constants*>(blocks + place * (int64_t)S::BLOCK + S::IMAGE * S::PARTS);
    const int chunks = ((r.s.len + TOK - 1) / TOK + pl.chunk - 1) / pl.chunk;
    const float aa = reinterpret_cast<const float*>(&con.ab[row >> 1])[row & 1];
    float m = kNegInf, l = 0.0f;
    for (int k = 0; k < chunks; ++k) {
      const float2 v = part[(place * pl.chunks + k) * ROWS + row];
      join_u(aa, m, l, v.x, v.y);
    }
    const bool none = con.seen[row].x < 0 || m == kNegInf;
    float* ml = reinterpret_cast<float*>(&con.ml[row >> 1]) + (row & 1);
    ml[0] = none ? 0.0f : -m;
    ml[2] = con.seen[row].x < 0 || l == 0.0f ? 0.0f : __frcp_rn(l);
  }
}

template <int D, bool F32>
__global__ void __launch_bounds__(THREADS, Shape<D, F32>::BLOCKS) kv4_mass_tc_votes(Kv4 c, Kv4Attn a, Kv4Mass ms, Plan pl, const uint8_t* blocks, float* shares) {
  using S = Shape<D, F32>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[2], done[2], all_done;
  __shared__ uint32_t tmem_slot;
  __shared__ float halves[TOK];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  constexpr int QUERIES = S::IMAGE, CONS = QUERIES + 2 * S::IMAGE * S::PARTS;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, half = warp >> 2, row = (warp & 3) * 32 + lane;
  if (pl.shares > 1) pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(&full[i], 1), mbar_init(&done[i], 1);
    mbar_init(&all_done, 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  bool bad = false, abort = false;
  uint32_t issued = 0, copied = 0;
  // the groups of tokens outermost: with a causal mask the first ones have most to do
  const int units = c.batch * c.kv_heads;
  const int64_t items = (int64_t)units * pl.tiles * pl.shares;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t rest = item / pl.shares;
    const int share = (int)(item - rest * pl.shares), tile = (int)(rest / units), unit = (int)(rest - (int64_t)tile * units);
    const Rows r = rows_of(c, unit, ms.voters, &bad);
    const int rows = r.votes * a.share, pages = (r.s.len + kKvPage - 1) / kKvPage;
    if (rows == 0 || tile * TOK >= r.s.len) continue;
    const int n_blocks = (rows + ROWS - 1) / ROWS;
    // the share's k-th block is share + k pl.shares
    const int steps = n_blocks > share ? (n_blocks - share + pl.shares - 1) / pl.shares : 0;
    Walk walk;
    const auto next = [&](int k, bool* whole) {
      return walk.next(k, steps, whole, [&](int i) {
        int first, last;
        ends_of(a, r, (share + i * pl.shares) * ROWS, &first, &last);
        return seen(a, first, last, tile * TOK, TOK);
      });
    };
    const int64_t place0 = place_of(pl, r, unit, a.share, share);
    // a block's copy: its queries to buffer copied & 1, its constants to place copied % 3
    const auto copy = [&](int k) {
      if (threadIdx.x == 0 && !abort) {  // after a wait that gave up the last ones may still be under way
        const uint8_t* from = blocks + (place0 + k * pl.shares) * (int64_t)S::BLOCK;
        uint64_t* bar = &full[copied & 1];
        mbar_arrive_expect_tx(bar, S::BLOCK);
        bulk_copy_g2s(smem + QUERIES + (copied & 1) * S::IMAGE * S::PARTS, from, S::IMAGE * S::PARTS, bar);
        bulk_copy_g2s(smem + CONS + (copied % 3) * S::CON, from + S::IMAGE * S::PARTS, (uint32_t)sizeof(Constants), bar);
      }
      copied += !abort;
    };
    const auto page_of = [&](int in) {
      const int page = tile * 2 + (in >> 6);
      if (page >= pages) return -1;
      const int id = c.page_table[(int64_t)r.b * c.max_pages + page];
      if (id >= 0 && id < c.n_pages) return id;
      bad = true;
      return -1;
    };
    bool k_whole = false, then_whole = false, before_whole = false;
    int k = next(0, &k_whole);
    const int krow = threadIdx.x >> 1, khalf = threadIdx.x & 1;
    Half<D> codes;
    codes.load(c, page_of(krow), r.h, krow & 63, khalf);
    pdl_wait();
    if (k < steps) copy(k);
    codes.store(base, krow, khalf);
    fence_proxy_async_smem();
    const int mine = page_of(row);
    float2 sb = make_float2(0.0f, 0.0f);
    if (mine >= 0) sb = params(*reinterpret_cast<const uint32_t*>(c.pages + ((int64_t)mine * c.kv_heads + r.h) * kv4_block_bytes(D) + kKvPage * D + (row & 63) * 8));
    const uint64_t step2 = f2pack(sb.x, sb.x), base2 = f2pack(sb.y, sb.y);
    const int in = (row & 64) + token_of(row & 63), j = tile * TOK + in;  // this thread's token
    // the rows that see it: from row_from on, before row_to
    const int64_t p0 = r.position(0), last = j < a.sinks ? r.s.len : (int64_t)j + a.window;
    const int row_from = (int)min(max(j - p0, (int64_t)0), (int64_t)r.votes) * a.share;
    const int row_to = (int)min(max(last - p0, (int64_t)0), (int64_t)r.votes) * a.share;
    uint64_t votes[2] = {0, 0};
    int before = -1;
    while (k < steps || before >= 0) {
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
      const uint32_t buf = issued & 1;
      if (k < steps) {
        mbar_wait_warp(&full[buf], (issued >> 1) & 1, &abort);
        if (warp == 0) {
          if (elect_one()) issue<D, 1, S::PARTS>(tmem + buf * 128, base, base + QUERIES + buf * S::IMAGE * S::PARTS, &done[buf]);
          __syncwarp();
        }
      }
      const uint32_t was = issued - 1;
      if (before >= 0) {
        mbar_wait_warp(&done[was & 1], (was >> 1) & 1, &abort);
        tc_fence_after();
      }
      // the buffer of the last products is free now
      const int then = k < steps ? next(k + 1, &then_whole) : steps;
      if (then < steps) copy(then);
      if (before >= 0) {
        const int row0 = (share + before * pl.shares) * ROWS + half * 64, left = rows - row0;
        const uint32_t ts = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (was & 1) * 128 + half * 64;
        const Constants& con = *reinterpret_cast<const Constants*>(smem + CONS + (was % 3) * S::CON);
        const auto work = [&](auto masked) {
          constexpr bool MASKED = decltype(masked)::value;
#pragma unroll 1
          for (int q = 0; q < 2 && q * 32 < left; ++q) {
            uint32_t s[32];
            tmem_ld_32x32b_x32(ts + q * 32, s);
            const uint32_t sees = MASKED ? below(row_to - row0 - q * 32) & ~below(row_from - row0 - q * 32) : 0;
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float4 ab = con.ab[half * 32 + q * 16 + i], ml = con.ml[half * 32 + q * 16 + i];
              const uint64_t u = fma2(step2, f2pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), mul2(base2, f2pack(ab.z, ab.w)));
              const float2 y = f2unpack(mul2(f2pack(ab.x, ab.y), add2(u, f2pack(ml.x, ml.y))));
              const uint64_t more = fma2(f2pack(exp2_approx(y.x), exp2_approx(y.y)), f2pack(ml.z, ml.w), votes[i & 1]);
              if (MASKED) {
                const float2 v = f2unpack(votes[i & 1]), w = f2unpack(more);
                votes[i & 1] = f2pack(sees & 1u << 2 * i ? w.x : v.x, sees & 2u << 2 * i ? w.y : v.y);
              } else {
                votes[i & 1] = more;
              }
            }
          }
        };
        if (before_whole) work(std::false_type{});
        else work(std::true_type{});
      }
      before = -1;
      if (k < steps) before = k, before_whole = k_whole, ++issued;
      k = then, k_whole = then_whole;
    }
    const float2 v = f2unpack(add2(votes[0], votes[1]));
    if (half) halves[row] = v.x + v.y;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!half) {
      const float got = (v.x + v.y) + halves[row];
      if (pl.shares > 1) {
        shares[(((int64_t)unit * pl.tiles + tile) * pl.shares + share) * TOK + in] = got;
      } else if (j < r.s.len && mine >= 0) {
        const int64_t at = ((int64_t)mine * c.kv_heads + r.h) * kKvPage + j % kKvPage;
        ms.out[at] = j < r.s.len - r.s.n ? fmaf(ms.decay, ms.in[at], got) : got;
      }
    }
    __syncthreads();  // the next item's codes
  }
  pdl_wait();
  if (warp == 0) {
    if (abort) {  // a wait gave up: the copies that it may have left under way end before the shared memory is given back
      for (uint32_t i = 0; i < 2; ++i) {
        const uint32_t to = (copied + 1 - i) >> 1;  // copies to buffer i
        bool late = false;
        if (to) mbar_wait_warp(&full[i], (to - 1) & 1, &late);
      }
    }
    if (elect_one()) mma_commit(&all_done);
    __syncwarp();
    abort = false;
    mbar_wait_warp(&all_done, 0, &abort);
  }
  if (bad) record_device_error(kErrRange);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 256);
}

// Adds up the shares' votes.
__global__ void __launch_bounds__(TOK) kv4_mass_tc_join(Kv4 c, Kv4Mass ms, Plan pl, const float* shares) {
  pdl_wait();
  const int64_t items = (int64_t)c.batch * c.kv_heads * pl.tiles;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int unit = (int)(item / pl.tiles), tile = (int)(item - (int64_t)unit * pl.tiles), j = tile * TOK + threadIdx.x;
    bool bad = false;
    const Rows r = rows_of(c, unit, ms.voters, &bad);
    if (r.votes == 0 || j >= r.s.len) continue;
    const int id = c.page_table[(int64_t)r.b * c.max_pages + j / kKvPage];
    if (id < 0 || id >= c.n_pages) continue;
    float got = 0.0f;
    for (int s = 0; s < pl.shares; ++s) got += shares[(item * pl.shares + s) * TOK + threadIdx.x];
    const int64_t at = ((int64_t)id * c.kv_heads + r.h) * kKvPage + j % kKvPage;
    ms.out[at] = j < r.s.len - r.s.n ? fmaf(ms.decay, ms.in[at], got) : got;
  }
}

constexpr int kSms = 152;
int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }
unsigned grid_of(int64_t items, int64_t most) { return (unsigned)(items < most ? items : most); }

Plan plan_of(const Kv4& c, int share, int64_t rows) {
  Plan p{};
  const int64_t units = (int64_t)c.batch * c.kv_heads;
  p.blocks = (int)((rows + ROWS - 1) / ROWS);
  p.tiles = (c.max_kv + TOK - 1) / TOK;
  // tiles of a chunk: four blocks an SM, but enough that a block's queries are not made ready for little (which takes as long
  // as two tiles): 8, and 16 where the blocks of rows alone fill the GPU (2048 voting tokens: 71 us against 76; 64 of 5
  // prompts each, which do not: 77 against 62)
  int64_t per = (units * p.blocks * p.tiles + kSms * 4 - 1) / (kSms * 4);
  const int64_t least = units * p.blocks >= kSms * 2 ? 16 : 8;
  per = per < least ? least : per;
  p.chunk = (int)(per > p.tiles ? (p.tiles ? p.tiles : 1) : per);
  p.chunks = (p.tiles + p.chunk - 1) / p.chunk;
  const int64_t all = units * (p.tiles ? p.tiles : 1), s = (kSms * 4 + all - 1) / all;
  p.shares = (int)(s > p.blocks ? p.blocks : s);
  const int64_t room = (int64_t)c.total_q * share / ROWS + c.batch;
  p.room = room < (int64_t)c.batch * p.blocks ? room : 0;
  return p;
}
int64_t places(const Kv4& c, const Plan& p) { return p.room ? c.kv_heads * p.room : (int64_t)c.batch * c.kv_heads * p.blocks; }
int64_t block_bytes(int dim, bool f32) { return (int64_t)128 * dim * 2 * (f32 ? 2 : 1) + (int64_t)sizeof(Constants); }
int64_t blocks_bytes(const Kv4& c, const Plan& p, int dim, bool f32) { return align256(places(c, p) * block_bytes(dim, f32)); }
int64_t part_bytes(const Kv4& c, const Plan& p) { return align256(places(c, p) * p.chunks * ROWS * 8); }

template <int D, bool F32>
cudaError_t launch(const Kv4& c, const Kv4Attn& a, const Kv4Mass& m, const Plan& p, uint8_t* ws, cudaStream_t st) {
  using S = Shape<D, F32>;
  if (p.tiles == 0) return cudaSuccess;
  uint8_t* blocks = ws;
  float2* part = reinterpret_cast<float2*>(ws + blocks_bytes(c, p, D, F32));
  float* shares = reinterpret_cast<float*>(ws + blocks_bytes(c, p, D, F32) + part_bytes(c, p));
  const int64_t units = (int64_t)c.batch * c.kv_heads;
  static std::atomic<uint64_t> configured[2];
  if (cudaError_t e = allow_smem(configured[0], kv4_mass_tc_rows<D, F32>, S::ROWS_SMEM)) return e;
  if (cudaError_t e = allow_smem(configured[1], kv4_mass_tc_votes<D, F32>, S::VOTES_SMEM)) return e;
  kv4_mass_tc_rows<D, F32><<<grid_of(units * p.blocks * p.chunks, 1 << 20), THREADS, S::ROWS_SMEM, st>>>(c, a, m.voters, p, blocks, part);
  if (cudaError_t e = cudaGetLastError()) return e;
  if (p.chunks > 1)
    if (cudaError_t e = launch_behind(kv4_mass_tc_sums<D, F32>, grid_of(units * p.blocks, 1 << 20), ROWS, 0, st, c, a, m.voters, p, blocks, part)) return e;
  if (cudaError_t e = launch_behind(kv4_mass_tc_votes<D, F32>, grid_of(units * p.tiles * p.shares, 1 << 20), THREADS, S::VOTES_SMEM, st, c, a, m, p, blocks,
                                    shares))
    return e;
  return p.shares > 1 ? launch_behind(kv4_mass_tc_join, grid_of(units * p.tiles, 1 << 20), TOK, 0, st, c, m, p, shares) : cudaSuccess;
}

}  // namespace

int64_t kv4_mass_tc_ws_bytes(const Kv4& c, int dim, int share, int64_t rows, bool f32) {
  const Plan p = plan_of(c, share, rows);
  const int64_t shares = p.shares > 1 ? align256((int64_t)c.batch * c.kv_heads * p.tiles * p.shares * TOK * 4) : 0;
  return blocks_bytes(c, p, dim, f32) + part_bytes(c, p) + shares;
}
cudaError_t launch_kv4_mass_tc(const Kv4& c, int dim, const Kv4Attn& a, const Kv4Mass& m, int64_t rows, void* ws, cudaStream_t st) {
  const Plan p = plan_of(c, a.share, rows);
  uint8_t* at = static_cast<uint8_t*>(ws);
  if (dim == 128) return a.bf16 ? launch<128, false>(c, a, m, p, at, st) : launch<128, true>(c, a, m, p, at, st);
  return a.bf16 ? launch<64, false>(c, a, m, p, at, st) : launch<64, true>(c, a, m, p, at, st);
}

cudaError_t read_clear_device_error_kv4_mass_tc(int* value) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, g_device_error, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
}

}  // namespace bitnet
