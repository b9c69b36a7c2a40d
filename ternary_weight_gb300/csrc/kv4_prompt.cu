// kv4_prompt.cu -- attention over the 4-bit key/value cache for many query rows a sequence (prompts
// and their chunks), on the 5th-generation tensor cores.
//
// A block takes 256 query rows of one sequence and key/value head (tokens x shared heads, so that the
// heads that share keys and values share their expansion too) as two tiles of 128, and walks over the
// cache 128 tokens (two pages) at a time:
//   S_t = Q_t K^T     128 x 128, K = D: both operands in shared memory (128-byte swizzle, K-major)
//   P_t = 2^(c1 S - c1 m + 7)  in registers, written over S_t in tensor memory as fp16
//   O_t += P_t V      128 x D, K = 128: P from tensor memory, V^T in shared memory
// What bounds it: 4096 tokens (20 and 5 heads x 128) take 97.2 us, 884 TFLOP/s of the measured 1902, with the
// tensor cores 43% busy and 2.6 of 4 issue slots used; 4 chunks with a window of 1024 (32 and 8 heads x 64)
// 79.3 us, 365 TFLOP/s. A step of 2 x 128 x 128 scores takes 1.98 us (D = 128) or 1.53 us (D = 64): at D =
// 128 the products need 1.1 us of it, the exponentials 0.53, issue slots 1.3; the rest is the chain scores ->
// weights -> product -> scores of a tile, whose weights lie over its scores. A block has about 10 us besides
// its steps: 1.1 until it starts, 1.3 the search for its item, 4 to 5 queries and first codes (all blocks
// of a wave read at once, and one-time code misses the instruction cache), 1.1 the first weights, 1.9
// the last product and the rows' way out.
//
// Operands are fp16 and sums fp32: q at a power-of-two scale of its row, k and v as step * code + base
// rounded to fp16 (2^-11 of the number itself, less than the 4-bit step by far), p up to 2^15,
// a scale of 2^7 among that.
// The codes are expanded once for both tiles: a code masked into the mantissa of 1024.0 (or 16 of it)
// becomes an exact fp16 by one multiply-add, the number by another. Word w of a key goes to columns
// 8 w .. 8 w + 7 in nibble order 0 4 1 5 2 6 3 7; the queries are stored in the same order. Values are
// transposed on the way: a lane takes one word of 8 tokens, pairs them byte by byte, and stores 8
// tokens of a dimension as 16 bytes.
//
// Roles (24 warps): 0-7 and 8-15 softmax of the two tiles, half a row (one page's columns) a thread;
// 16-18 keys; 19-22 values; 23 issues the MMAs in the order  PV_A(j) S_A(j+1) PV_B(j) S_B(j+1): one tile's
// softmax has the time of the other's two products. The running maximum is moved (and O rescaled) only where
// a row's has grown by more than 2^8. What carried it, for the 4096 tokens: 16 softmax warps 244 -> 148 us,
// loops short enough for the instruction cache 148 -> 111, half a row a thread 111 -> 107, a converged MMA
// warp 107 -> 104, waits of few instructions and seven expanding warps 103 -> 96.
//
// With at most 128 rows both slots hold the same queries and take the steps in turn, so that the two
// chains still overlap; their results are joined at the end as those of two halves of the cache.
//
// Where the query tiles are fewer than the SMs, the cache positions are cut into `splits` parts whose
// results a second kernel joins in order.
#include "kv4.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace bitnet {
namespace {

constexpr int THREADS = 768;
constexpr int ROWS = 256;   // query rows of a block
constexpr int TOK = 128;    // cache tokens of a step
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kMostC1 = 1.2089258196146292e24f;  // 2^80
constexpr float kSlack = 8.0f;  // log2 of how far a weight may exceed that of the maximum in use before it is moved
// log2 of what all weights are scaled by (their sums too): up to 2^15 as fp16, so the small ones are rounded by 2^-32
// of the row's largest at most, where a first token takes most of the weight and the others' values are what counts
constexpr float kLift = 7.0f;

template <int D>
struct Prompt {
  static constexpr int W = D / 8;
  static constexpr int BLK = 64 * D + 512;
  static constexpr int Q_TILE = 128 * D * 2, K_STAGE = TOK * D * 2, V_STAGE = D * TOK * 2;
  static constexpr int SMEM = 2 * Q_TILE + 2 * K_STAGE + 2 * V_STAGE + 1024;
  static constexpr uint32_t IDESC_S = make_idesc_f16_f32(128, TOK), IDESC_O = make_idesc_f16_f32(128, D);
};
// Tensor memory columns of the two slots: scores (128 each), outputs (D each), weights (64 each). With
// D = 128 that is more than there is, and a half of the weights lies over the first half of its scores:
// the next scores then have to wait for the product that reads the weights. With D = 64 the weights have
// columns of their own, and the next scores only wait for the last ones to be read.
constexpr uint32_t TM_S = 0, TM_O = 256;
template <int D>
struct Weights {
  static constexpr bool APART = D == 64;
  static constexpr uint32_t AT = APART ? 384 : TM_S, SLOT = APART ? 64 : 128, HALF = APART ? 32 : 64;
};

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
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
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// the codes in nibbles 0 and 4 of x, or 1 and 5, as exact fp16
__device__ __forceinline__ uint32_t codes_even(uint32_t x) {
  return hsub2((x & 0x000f000fu) | 0x64006400u, 0x64006400u);  // 1024 + c
}
__device__ __forceinline__ uint32_t codes_odd(uint32_t x) {
  return hfma2((x & 0x00f000f0u) | 0x64006400u, 0x2c002c00u, 0xd400d400u);  // (1024 + 16 c) / 16 - 64
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// byte offset of 16-byte chunk c (0..7) of row r in a 128-byte-swizzled K-major tile
__device__ __forceinline__ uint32_t sw128(int r, int c) {
  return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}
// one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r != 0;
}
// descriptors by their low words: the high one is the same for every operand here
__device__ __forceinline__ void mma_f16_ss_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 ad, {%1, %3};\n\t"
      "mov.b64 bd, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %4, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 bd;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 bd, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %4, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Bounded waits of few instructions: the roles share their schedulers, so every instruction of a wait
// costs. One that gives up records it, and the later ones of the warp then poll once only; all roles keep
// going through their steps (their loops are bounded, what they touch stays in bounds, and the pairs'
// barriers match), with results that do not count.
struct Waits {
  uint32_t polls = kMaxPolls;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, 0;\n\t"
        "POLL:\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "add.u32 n, n, 1;\n\t"
        "setp.lt.u32 q, n, %3;\n\t"
        "@q bra POLL;\n\t"
        "DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(polls)
        : "memory");
    if (!ok) {
      if (polls > 1) record_device_error(kErrTimeout);
      polls = 1;
    }
  }
};

// x / d for x < 512, 1 <= d <= 128, with m = ceil(65536 / d)
__device__ __forceinline__ int small_div(int x, uint32_t m) { return (int)(((uint32_t)x * m) >> 16); }

// What a block works on: query rows row0 .. row0 + rows of one sequence and head, and the pages that
// any of them sees, page i being page i of the sequence, or i + skip from i = ns on.
struct Item {
  int b, h, row0, rows;
  int tok0, head0;  // token and shared head of row0
  int np, ns, skip;
  Kv4Seq s;
};
// a page's first position; past every query where there is no such page
__device__ __forceinline__ int page_first(const Item& it, int i) {
  return i >= it.np ? INT32_MAX - 2 * TOK : (i < it.ns ? i : i + it.skip) * kKvPage;
}

// Partials of a split call: for each item (tile x heads + head) and part ROWS x D sums, ROWS maxima (log2), ROWS sums; and
// for each item what it is.
struct Parts {
  float* sums;
  int4* info;  // first packed row of the sequence, first query row, query rows (0: none), head
  int splits;
};

// The queries of a warp's 16 rows of the item, scaled and in the operand's order: W lanes a row, 8 dimensions
// a lane (8 w .. 8 w + 7: nibble n = w / (W / 8) of words 8 w % W ..). q' = q 2^(13 - e), 2^e <= max |q| <
// 2^(e + 1), e not below -100, and 13 where there are infinities or NaN; 2^(e - 13) goes to row_f. The loads of
// all rows (bf16; fp32: of 4) are in flight together, and a pair of rows shares its exchanges: this stands
// at the head of every block, before the first product can begin.
template <int D, bool BF16>
__device__ __forceinline__ void store_queries(const Kv4Attn& a, const Item& it, uint32_t share_m, int warp, int lane,
                                              uint32_t q_s, float* row_f) {
  constexpr int W = D / 8, RPI = 32 / W, ALL = 16 / RPI, BATCH = BF16 ? ALL : 4, U = BF16 ? 4 : 8;
  static_assert(ALL % BATCH == 0 && (ALL == BATCH || BATCH * RPI % 8 == 0), "a batch begins at a row of eight");
  const int w = lane % W, n = w / (W / 8), sub = lane / W;
  const bool high = n >= 4;
  const uint32_t neg = a.scale < 0.0f ? 0x80008000u : 0u;
  // of row r, token t: base + t hop + r D
  const int64_t hop = a.q_stride - (int64_t)a.share * D;
  const int64_t base = (int64_t)(it.s.q0 + it.tok0) * a.q_stride + (int64_t)(it.h * a.share + it.head0) * D + 8 * w;
  uint32_t dst = q_s + (warp >> 3) * Prompt<D>::Q_TILE + (8 * w % W >> 3) * (128 * 128) +
                 ((warp & 7) * 16 + sub) * 128 + 4 * (n & 3);
  const uint32_t turn = ((high ? 4u : 0u) ^ (uint32_t)sub) << 4;
#pragma unroll 1
  for (int i0 = 0; i0 < ALL; i0 += BATCH, dst += BATCH * RPI * 128) {
    const int r0 = warp * 16 + i0 * RPI + sub;
    uint32_t u[BATCH][U];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {  // rows past the end read the last one
      const int r = min(r0 + i * RPI, it.rows - 1);
      const int64_t at = base + small_div(it.head0 + r, share_m) * hop + r * D;
      const uint4* src = BF16 ? reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at)
                              : reinterpret_cast<const uint4*>(static_cast<const float*>(a.q) + at);
#pragma unroll
      for (int k = 0; k < U / 4; ++k) {
        const uint4 x = __ldg(src + k);
        u[i][4 * k] = x.x, u[i][4 * k + 1] = x.y, u[i][4 * k + 2] = x.z, u[i][4 * k + 3] = x.w;
      }
    }
    // the upper 16 bits of the largest magnitudes of two rows: their exponents are all that counts
    uint32_t top[BATCH / 2];
#pragma unroll
    for (int i = 0; i < BATCH; i += 2) {
      uint32_t m[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        m[s] = 0;
#pragma unroll
        for (int k = 0; k < U; ++k)
          m[s] = BF16 ? __vmaxu2(m[s], u[i + s][k] & 0x7fff7fffu) : max(m[s], u[i + s][k] & 0x7fffffffu);
      }
      const uint32_t hi = __byte_perm(m[0], m[1], 0x7632);
      top[i / 2] = BF16 ? __vmaxu2(hi, __byte_perm(m[0], m[1], 0x5410)) : hi;
    }
#pragma unroll
    for (int o = W / 2; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < BATCH / 2; ++i) top[i] = __vmaxu2(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      uint32_t e = (top[i / 2] >> (i & 1 ? 23 : 7)) & 255u;  // e + 127
      e = e == 255u ? 140u : max(e, 27u);
      const float up = __uint_as_float((267u - e) << 23);
      if (w == 0) row_f[r0 + i * RPI] = __uint_as_float((e - 13u) << 23);
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = __uint_as_float(BF16 ? u[i][k % U] << 16 : u[i][2 * k % U]);
        const float y = __uint_as_float(BF16 ? u[i][k % U] & 0xffff0000u : u[i][(2 * k + 1) % U]);
        h[k] = pack_half2(x * up, y * up) ^ neg;
      }
      // nibbles n and n + 4 of a word lie side by side: half of the lane's numbers go to the lane that has the
      // other nibble, half of that one's come here
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? h[k] : h[2 + k], W / 2), own = high ? h[2 + k] : h[k];
        const uint32_t lo = high ? got : own, up2 = high ? own : got;
        st_shared_u32(dst + i * RPI * 128 + (turn ^ (((2 * k) ^ (i * RPI & 7)) << 4)), __byte_perm(lo, up2, 0x5410));
        st_shared_u32(dst + i * RPI * 128 + (turn ^ (((2 * k + 1) ^ (i * RPI & 7)) << 4)), __byte_perm(lo, up2, 0x7632));
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1) kv4_prompt_kernel(Kv4 c, Kv4Attn a, int done_rows, uint32_t share_m, Parts parts) {
  using P = Prompt<D>;
  constexpr int W = P::W;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  __shared__ __align__(8) uint64_t s_full[2], p_full[2], pv_done[2], q_full, all_done;
  __shared__ uint32_t tmem_slot;
  __shared__ int warp_sum[THREADS / 32];
  __shared__ Item item_s;
  __shared__ float row_c1[ROWS], row_x[2][2][ROWS];  // the halves' maxima (then sums), by step parity
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t q_s = base, k_s = q_s + 2 * P::Q_TILE, v_s = k_s + 2 * P::K_STAGE;
  bool bad = false;
  pdl_launch_dependents();

  // ---- which item: item x of a head is the x-th tile of all sequences, each one's last (longest) first
  const int x = blockIdx.x / c.kv_heads, split = blockIdx.y;
  const int64_t item_no = blockIdx.x;
  {
    const int per = (c.batch + THREADS - 1) / THREADS;
    const int b0 = min((int)threadIdx.x * per, c.batch), b1 = min(b0 + per, c.batch);
    const auto tiles_of = [&](const Kv4Seq& s) {
      const int64_t r = (int64_t)s.n * a.share;
      return r <= done_rows ? 0 : (int)((r + ROWS - 1) / ROWS);
    };
    int mine = 0;
    Kv4Seq s{};
    for (int b = b0; b < b1; ++b) mine += tiles_of(s = kv4_sequence(c, b, &bad));
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) warp_sum[warp] = upto;
    if (warp == 22 && lane == 0) {
      item_s.rows = 0;
      for (int i = 0; i < 2; ++i) {
        mbar_init(&k_full[i], 3);
        mbar_init(&v_full[i], 4);
        mbar_init(&k_empty[i], 1);
        mbar_init(&v_empty[i], 1);
        mbar_init(&s_full[i], 1);
        mbar_init(&p_full[i], 8);
        mbar_init(&pv_done[i], 1);
      }
      mbar_init(&q_full, 16);
      mbar_init(&all_done, 1);
      fence_mbar_init();
    }
    if (warp == 23) {
      tmem_alloc(&tmem_slot, 512);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int at0 = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0);
    int at = at0 + upto - mine;
    if (x >= at && x < at + mine) {
      for (int b = b0; b < b1; ++b) {
        if (per > 1) s = kv4_sequence(c, b, &bad);
        const int t = tiles_of(s);
        if (x < at + t) {
          Item it;
          it.b = b;
          it.h = blockIdx.x - x * c.kv_heads;
          it.s = s;
          it.row0 = (t - 1 - (x - at)) * ROWS;
          it.rows = min(ROWS, s.n * a.share - it.row0);
          it.tok0 = it.row0 / a.share;
          it.head0 = it.row0 - it.tok0 * a.share;
          const int pos0 = s.len - s.n + it.tok0, pos1 = pos0 + small_div(it.head0 + it.rows - 1, share_m);
          const int low = (int)max((int64_t)0, (int64_t)pos0 - a.window + 1);
          const int low_page = low / kKvPage, sink_pages = (min(a.sinks, low) + kKvPage - 1) / kKvPage;
          it.ns = min(sink_pages, low_page);
          it.skip = low_page - it.ns;
          it.np = pos1 < 0 ? 0 : it.ns + pos1 / kKvPage + 1 - low_page;
          item_s = it;
          break;
        }
        at += t;
      }
    }
  }
  __syncthreads();
  const Item it = item_s;
  if (parts.splits > 1 && split == 0 && threadIdx.x == 0)
    parts.info[item_no] = make_int4(it.s.q0, it.row0, it.rows, it.h);
  if (it.rows == 0) {  // fewer items than the grid was made for
    if (bad) record_device_error(kErrRange);
    if (warp == 23) tmem_dealloc(tmem_slot, 512);
    return;
  }
  const uint32_t tmem = tmem_slot;
  const int all = (it.np + 1) / 2;  // steps of the item, then of this part of it
  const int j0 = (int)((int64_t)all * split / parts.splits), j1 = (int)((int64_t)all * (split + 1) / parts.splits);
  const int steps = j1 - j0;
  const bool twin = it.rows <= 128;  // one tile of rows, in both slots
  Waits wait;

  if (warp < 16) {
    // ================================ softmax ================================
    const int tile = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
    // token (from the item's first) and head of a row of the item
    const auto token_of = [&](int r) { return small_div(it.head0 + r, share_m); };
    if (!twin || tile == 0) {
      if (a.bf16) store_queries<D, true>(a, it, share_m, warp, lane, q_s, row_c1);
      else store_queries<D, false>(a, it, share_m, warp, lane, q_s, row_c1);
      fence_proxy_async_smem();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_full);
    wait(&q_full, 0);
    __syncwarp();
    const int w0 = (twin ? 0 : tile * 128) + quarter * 32, r = w0 + lane;  // the warp's first row, the thread's row
    const int mine = twin ? (steps + 1 - tile) / 2 : steps;                // steps of this slot
    const bool there = r < it.rows;
    // a factor of 0 would make NaN of a masked score, and one of 2^80 already sets unlike scores (2^-48 apart at
    // least, 2^37 at most) infinitely far apart: from there on it would overflow
    const float c1 = fminf(fmaxf(fabsf(a.scale) * kLog2e * row_c1[r], 1.17549435e-38f), kMostC1);
    const int pos0 = it.s.len - it.s.n + it.tok0;
    // before position 0 nothing is seen, however far before: -1 keeps the mask's differences in 32 bits
    const int pos = there ? max(pos0 + token_of(r), -1) : -1;
    // of the warp's rows: the first position, and the last window's beginning (rows past the end follow the last)
    const int pos_first = pos0 + token_of(w0);
    const int low_last =
        (int)max((int64_t)0, (int64_t)pos0 + token_of(max(min(it.rows, w0 + 32) - 1, 0)) - a.window + 1);
    const uint32_t lane0 = (uint32_t)(quarter * 32) << 16;
    // this page's scores and weights
    using WT = Weights<D>;
    const uint32_t tp = tmem + lane0 + WT::AT + (uint32_t)tile * WT::SLOT + (uint32_t)half * WT::HALF;
    const uint32_t ts = tmem + lane0 + TM_S + (uint32_t)(tile * 128 + half * 64);
    const uint32_t to = tmem + lane0 + TM_O + (uint32_t)(tile * D + half * (D / 2));
    const int xr = tile * 128 + quarter * 32 + lane;  // the thread's place in row_x
    const int pair = 1 + tile * 4 + quarter;  // barrier of the two warps that share rows
    float m = kNegInf, l = 0.0f;
    for (int j = 0; j < mine; ++j) {
      const int first = page_first(it, 2 * (j0 + (twin ? 2 * j + tile : j)) + half);
      const bool whole = first + kKvPage - 1 <= pos_first && (first >= low_last || first + kKvPage <= a.sinks);
      wait(&s_full[tile], (uint32_t)j & 1u);
      __syncwarp();
      tc_fence_after();
      if (!whole) {  // what a row does not see becomes -inf in place, 32 columns at a time
        const int hi = pos - first;  // columns x <= hi with x >= lo or x < sk are seen
        const int lo = (int)max((int64_t)INT32_MIN, (int64_t)hi - a.window + 1), sk = max(a.sinks - first, 0);
#pragma unroll 1
        for (int ch = 0; ch < 2; ++ch) {
          const int h = hi - 32 * ch, b = max(lo, INT32_MIN + 64) - 32 * ch, k0 = sk - 32 * ch;
          const auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };  // bits 0 .. n - 1
          const uint32_t vis = below(h >= 31 ? 32 : h + 1) & (~below(b) | below(k0));
          uint32_t v[32];
          tmem_ld_32x32b_x32(ts + 32 * ch, v);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!((vis >> k) & 1u)) v[k] = __float_as_uint(kNegInf);
          tmem_st_x32(ts + 32 * ch, v);
        }
        tmem_st_wait();
      }
      // 16 columns at a time, the next ones on their way
      uint32_t v[2][16];
      float mx4[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
      tmem_ld_x16(ts, v[0]);
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        tmem_ld_wait();
        tmem_ld_x16(ts + 16 * ((ch + 1) & 3), v[(ch + 1) & 1]);  // at last the first ones again
#pragma unroll
        for (int k = 0; k < 16; ++k) mx4[k & 3] = fmaxf(mx4[k & 3], __uint_as_float(v[ch & 1][k]));
      }
      // the other page's maximum, from the other warp of these rows
      float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
      row_x[j & 1][half][xr] = mx;
      named_bar_sync(pair, 64);
      mx = fmaxf(m, fmaxf(mx, row_x[j & 1][half ^ 1][xr]));
      // a row's first scores, or scores far above the maximum in use: move it
      const bool far = mx > m && (m == kNegInf || c1 * (mx - m) > kSlack);
      if (__any_sync(0xffffffffu, far)) {
        const float f = m == kNegInf ? (mx == kNegInf ? 1.0f : 0.0f) : exp2_approx(c1 * (m - mx));
        m = mx;
        l *= f;
        if (j > 0) {  // after the last step's product with V
          if (WT::APART) {
            wait(&pv_done[tile], (uint32_t)(j - 1) & 1u);
            __syncwarp();
            tc_fence_after();
          }
#pragma unroll 1
          for (int ch = 0; ch < D / 64; ++ch) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(to + 32 * ch, v);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f);
            tmem_st_x32(to + 32 * ch, v);
          }
        }
      }
      if (WT::APART && j > 0) {  // its weights are read: the next ones may be stored over them
        wait(&pv_done[tile], (uint32_t)(j - 1) & 1u);
        __syncwarp();
        tc_fence_after();
      }
      const Kv4Weight wt = kv4_weight(c1, m, 22, kLift);
      const uint64_t c2 = f2pack(wt.c, wt.c), off2 = f2pack(wt.off, wt.off);
      uint64_t l2[2] = {0, 0};
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t w[8];
        tmem_ld_wait();
        if (ch < 3) tmem_ld_x16(ts + 16 * (ch + 1), v[(ch + 1) & 1]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t(&u)[16] = v[ch & 1];
          const float2 t = f2unpack(fma2(f2pack(__uint_as_float(u[2 * k]), __uint_as_float(u[2 * k + 1])), c2, off2));
          const float p0 = exp2_approx(t.x), p1 = exp2_approx(t.y);
          l2[k & 1] = add2(l2[k & 1], f2pack(p0, p1));
          w[k] = pack_half2(p0, p1);
        }
        tmem_st_x8(tp + 8 * ch, w);
      }
      const float2 la = f2unpack(add2(l2[0], l2[1]));
      l += la.x + la.y;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[tile]);
    }
    if (mine > 0) wait(&pv_done[tile], (uint32_t)(mine - 1) & 1u);
    __syncwarp();
    tc_fence_after();
    row_x[mine & 1][half][xr] = l;
    named_bar_sync(pair, 64);
    l = half ? row_x[mine & 1][0][xr] + l : l + row_x[mine & 1][1][xr];
    // twins: slot 1 leaves its sums where the keys were (128 rows x D fp32, 16-byte chunk c of row r at
    // c ^ (r & 7)) and its maximum and sum of weights in row_x; slot 0 takes them in
    float f0 = 1.0f, f1 = 0.0f;
    const uint32_t twin_s = k_s + (uint32_t)(quarter * 32 + lane) * (D * 4);
    if (twin) {
      named_bar_sync(9, 512);  // every product is done
      if (tile == 1) {
        if (half == 0) row_x[0][0][xr] = m, row_x[0][1][xr] = l;
#pragma unroll 1
        for (int ch = 0; ch < D / 64; ++ch) {
          uint32_t v[32];
          if (mine > 0) {
            tmem_ld_32x32b_x32(to + 32 * ch, v);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = 0;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            sts128(twin_s + (((half * (D / 8) + 8 * ch + k) ^ (lane & 7)) << 4), v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
      }
      named_bar_sync(9, 512);
      if (tile == 0) {
        const float m1 = row_x[0][0][xr + 128], l1 = row_x[0][1][xr + 128], mx = fmaxf(m, m1);
        const float ref = mx == kNegInf ? 0.0f : mx;
        f0 = exp2_approx(c1 * (m - ref));
        f1 = exp2_approx(c1 * (m1 - ref));
        m = mx;
        l = l * f0 + l1 * f1;
      }
    }
    const float norm = parts.splits > 1 ? 1.0f : (l == 0.0f ? 0.0f : 1.0f / l);
    float* part = parts.splits > 1 ? parts.sums + (item_no * parts.splits + split) * (ROWS * (D + 2)) : nullptr;
    // rows go out through this tile's query operand, which no product reads any more: 16-byte chunk c of
    // row r at (c ^ (r & 7)), so that a row leaves in one piece
    const uint32_t stage = q_s + tile * P::Q_TILE + quarter * (32 * D * 2);
    const bool gives = !twin || tile == 0;
#pragma unroll 1
    for (int ch = 0; ch < D / 64 && gives; ++ch) {
      uint32_t v[32];
      if (mine > 0) {
        tmem_ld_32x32b_x32(to + 32 * ch, v);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = 0;
      }
      if (twin) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint4 o = lds128(twin_s + (((half * (D / 8) + 8 * ch + k) ^ (lane & 7)) << 4));
          v[4 * k] = __float_as_uint(__uint_as_float(v[4 * k]) * f0 + __uint_as_float(o.x) * f1);
          v[4 * k + 1] = __float_as_uint(__uint_as_float(v[4 * k + 1]) * f0 + __uint_as_float(o.y) * f1);
          v[4 * k + 2] = __float_as_uint(__uint_as_float(v[4 * k + 2]) * f0 + __uint_as_float(o.z) * f1);
          v[4 * k + 3] = __float_as_uint(__uint_as_float(v[4 * k + 3]) * f0 + __uint_as_float(o.w) * f1);
        }
      }
      const int d = half * (D / 2) + 32 * ch;
      if (part) {
        if (there) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(part + r * D + d + 4 * k) = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(__uint_as_float(v[8 * k + 2 * i]) * norm,
                                                           __uint_as_float(v[8 * k + 2 * i + 1]) * norm);
            y[i] = *reinterpret_cast<const uint32_t*>(&t);
          }
          sts128(stage + lane * (D * 2) + (((d / 8 + k) ^ (lane & 7)) << 4), y[0], y[1], y[2], y[3]);
        }
      }
    }
    if (!gives) {
    } else if (part) {
      if (there && half == 0) {
        part[ROWS * D + r] = m * c1;
        part[ROWS * (D + 1) + r] = l;
      }
    } else {
      named_bar_sync(pair, 64);
      constexpr int C = D / 8, RPI = 32 / C;  // chunks of a row, rows at a time
      const int ck = lane % C;
#pragma unroll
      for (int i = 0; i < 16; i += RPI) {  // 16 of the rows each
        const int rr = half * 16 + i + lane / C, row = w0 + rr, t = token_of(row);
        if (row < it.rows)
          *reinterpret_cast<uint4*>(a.out + (int64_t)(it.s.q0 + it.tok0 + t) * a.out_stride +
                                    (int64_t)(it.h * a.share + it.head0 + row - t * a.share) * D + 8 * ck) =
              lds128(stage + rr * (D * 2) + ((ck ^ (rr & 7)) << 4));
      }
    }
    tc_fence_before();
  } else if (warp < 23) {
    // ================================ expansion ================================
    const int pages = 2 * steps;
    // a page's id (the last page's again where there is no such page), asked for ahead of its codes
    const auto page_id = [&](int i) {
      const int k = min(2 * j0 + i, it.np - 1);
      return __ldg(c.page_table + (int64_t)it.b * c.max_pages + (k < it.ns ? k : k + it.skip));
    };
    const auto block = [&](int id) -> const uint8_t* {
      if (id < 0 || id >= c.n_pages) bad = true, id = 0;
      return c.pages + ((int64_t)id * c.kv_heads + it.h) * P::BLK;
    };
    if (pages > 0 && warp < 19) {
      // keys: 8 rows of all chunks (D = 128), or 16 of both (D = 64), a unit; a page's units go to the three
      // warps in turn, which turn with the page. lane & 7 is the row of eight, so that 8 lanes store to 8 rows.
      constexpr int UPP = D == 128 ? 8 : 4, U = (UPP + 2) / 3, RPU = kKvPage / UPP;
      const int row8 = lane & 7, chunk = D == 128 ? lane >> 3 : (lane >> 3) & 1;
      const int row_in = D == 128 ? row8 : (lane >> 4) * 8 + row8;
      uint4 code[U], code_n[U];
      uint2 par[U], par_n[U];
      int turn = warp - 16;  // the page's first unit of this warp
      const auto load = [&](int id, int first, uint4(&cd)[U], uint2(&pr)[U]) {
        const uint8_t* p = block(id);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int row = min(first + 3 * i, UPP - 1) * RPU + row_in;
          cd[i] = __ldg(reinterpret_cast<const uint4*>(p + row * (D / 2) + 16 * chunk));
          pr[i] = __ldg(reinterpret_cast<const uint2*>(p + kKvPage * D + row * 8));
        }
      };
      const int id0 = page_id(0);
      int id = page_id(1), id_n = page_id(2);  // together: each would cost the block a memory latency
      load(id0, turn, code, par);
#pragma unroll 1
      for (int pg = 0; pg < pages; ++pg) {
        const int turn_n = turn == 0 ? 2 : turn - 1;
        load(id, turn_n, code_n, par_n);
        id = id_n;
        id_n = page_id(pg + 3);
        const int st = (pg >> 1) & 1;
        if (pg >= 4 && !(pg & 1)) wait(&k_empty[st], (uint32_t)((pg >> 2) - 1) & 1u);
        const uint32_t dst = k_s + st * P::K_STAGE;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          if (turn + 3 * i < UPP) {
            const int t = 64 * (pg & 1) + kv4_rho_inv((turn + 3 * i) * RPU + row_in);
            const uint32_t step = __byte_perm(par[i].x, 0, 0x1010);
            uint32_t bs = __byte_perm(par[i].x, 0, 0x3232);
            // a value vector of NaN acts through its key, so that a weight of 0 never meets a NaN
            const uint32_t z = hsub2(par[i].y, par[i].y);
            bs = hadd2(bs, hadd2(__byte_perm(z, 0, 0x1010), __byte_perm(z, 0, 0x3232)));
            const uint32_t wd[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t up = wd[k] >> 8;
              const int w = 4 * chunk + k;
              sts128(dst + (w >> 3) * (TOK * 128) + sw128(t, w & 7), hfma2(codes_even(wd[k]), step, bs),
                     hfma2(codes_odd(wd[k]), step, bs), hfma2(codes_even(up), step, bs), hfma2(codes_odd(up), step, bs));
            }
          }
          code[i] = code_n[i];
          par[i] = par_n[i];
        }
        turn = turn_n;
        if (pg & 1) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&k_full[st]);
        }
      }
    } else if (pages > 0) {
      // values: word w of 8 tokens a lane, 16 (D = 128) or 32 tokens a unit; the units of all pages go to
      // the four warps in turn
      constexpr int TPU = 8 * (32 / W), UPP = kKvPage / TPU;  // tokens of a unit, units of a page
      const int w = lane % W, grp = lane / W, units = UPP * pages;
      uint32_t code[8], par[8], code_n[8], par_n[8];
      const auto load = [&](int u, int id, uint32_t(&cd)[8], uint32_t(&pr)[8]) {
        const int t0 = (u % UPP) * TPU + 8 * grp;
        const uint8_t* p = block(id) + kKvPage * (D / 2) + t0 * (D / 2);
        const uint8_t* q = p + kKvPage * (D / 2) - t0 * (D / 2) + t0 * 8 + 4;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          cd[k] = __ldg(reinterpret_cast<const uint32_t*>(p + k * (D / 2)) + (D == 128 && (k & 2) ? w ^ (W / 2) : w));
          pr[k] = __ldg(reinterpret_cast<const uint32_t*>(q + kv4_rho(k) * 8));
        }
      };
      int u = warp - 19;
      const int id0 = page_id(u / UPP);
      int id = page_id((u + 4) / UPP), id_n = page_id((u + 8) / UPP);
      load(u, id0, code, par);
      int done = -1;  // the last step whose place was waited for
#pragma unroll 1
      for (; u < units; u += 4) {
        load(min(u + 4, units - 1), id, code_n, par_n);
        id = id_n;
        id_n = page_id((u + 12) / UPP);
        const int j = u / (2 * UPP), st = j & 1;
        if (j != done) {
          done = j;
          if (j >= 2) wait(&v_empty[st], (uint32_t)(j / 2 - 1) & 1u);
        }
        const uint32_t at = v_s + st * P::V_STAGE + ((u / UPP) & 1) * (D * 128);
        const int ch = ((u % UPP) * TPU >> 3) + grp;
        const int left = it.s.len - page_first(it, 2 * j0 + u / UPP) - ((u % UPP) * TPU + 8 * grp);
        uint32_t step[4], bs[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          step[k] = __byte_perm(par[2 * k], par[2 * k + 1], 0x5410);
          bs[k] = __byte_perm(par[2 * k], par[2 * k + 1], 0x7632);
          const uint32_t z = hadd2(hsub2(step[k], step[k]), hsub2(bs[k], bs[k]));
          uint32_t ok;  // all ones where finite
          asm("set.eq.u32.f16x2 %0, %1, %2;" : "=r"(ok) : "r"(z), "r"(0u));
          if (left < 2 * k + 2) ok &= left < 2 * k + 1 ? 0u : 0xffffu;  // no value where nothing is cached
          step[k] &= ok;
          bs[k] &= ok;
        }
#pragma unroll
        for (int by = 0; by < 4; ++by) {
          uint32_t e[4], o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t x = __byte_perm(code[2 * k], code[2 * k + 1], 0x4400 + 0x1111 * by);
            e[k] = hfma2(codes_even(x), step[k], bs[k]);
            o[k] = hfma2(codes_odd(x), step[k], bs[k]);
          }
          const int d = w + W * 2 * by;
          sts128(at + sw128(d, ch), e[0], e[1], e[2], e[3]);
          sts128(at + sw128(d + W, ch), o[0], o[1], o[2], o[3]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) code[k] = code_n[k], par[k] = par_n[k];
        if (u + 4 >= 2 * UPP * (j + 1)) {  // this warp's last unit of the step
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_full[st]);
        }
      }
    }
  } else if (steps > 0) {
    // ================================ MMA issue ================================
    // The whole warp goes through the waits, so that descriptors stay in uniform registers, and one
    // elected lane issues.
    const bool leader = elect_one();
    const uint64_t qd = make_sw128_kmajor_desc(q_s), kd = make_sw128_kmajor_desc(k_s), vd = make_sw128_kmajor_desc(v_s);
    const uint32_t hi = (uint32_t)(qd >> 32), q_lo = (uint32_t)qd, k_lo = (uint32_t)kd, v_lo = (uint32_t)vd;
    const auto scores = [&](int t, int j, bool frees) {
      const uint32_t ad = q_lo + (uint32_t)(twin ? 0 : t * (P::Q_TILE >> 4)), bd = k_lo + (uint32_t)((j & 1) * (P::K_STAGE >> 4));
      const uint32_t d = tmem + TM_S + (uint32_t)(t * 128);
      if (leader) {
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t o = (uint32_t)((s >> 2) * ((128 * 128) >> 4) + (s & 3) * 2);
          mma_f16_ss_lo(d, ad + o, bd + o, hi, P::IDESC_S, s > 0);
        }
        mma_commit(&s_full[t]);
        if (frees) mma_commit(&k_empty[j & 1]);
      }
      __syncwarp();
    };
    const auto values = [&](int t, int j, bool more, bool frees) {
      const uint32_t bd = v_lo + (uint32_t)((j & 1) * (P::V_STAGE >> 4));
      const uint32_t d = tmem + TM_O + (uint32_t)(t * D), p = tmem + Weights<D>::AT + (uint32_t)t * Weights<D>::SLOT;
      if (leader) {
#pragma unroll
        for (int s = 0; s < TOK / 16; ++s)
          mma_f16_ts_lo(d, p + (s >> 2) * Weights<D>::HALF + (s & 3) * 8, bd + (uint32_t)((s >> 2) * ((D * 128) >> 4) + (s & 3) * 2), hi,
                        P::IDESC_O, more || s > 0);
        mma_commit(&pv_done[t]);
        if (frees) mma_commit(&v_empty[j & 1]);
      }
      __syncwarp();
    };
    wait(&q_full, 0);
    wait(&k_full[0], 0);
    __syncwarp();
    tc_fence_after();
    scores(0, 0, twin);
    if (twin) {
      if (steps > 1) {
        wait(&k_full[1], 0);
        __syncwarp();
        tc_fence_after();
        scores(1, 1, true);
      }
      for (int j = 0; j < steps; ++j) {  // slot j & 1, its (j / 2)-th step
        const int t = j & 1;
        const uint32_t ph = (uint32_t)(j >> 1) & 1u;
        const bool next = j + 2 < steps;
        wait(&v_full[t], ph);
        wait(&p_full[t], ph);
        __syncwarp();
        tc_fence_after();
        if (!Weights<D>::APART) values(t, j, j > 1, true);
        if (next) {
          wait(&k_full[t], ph ^ 1u);
          if (!Weights<D>::APART) wait(&pv_done[t], ph);
          __syncwarp();
          tc_fence_after();
          scores(t, j + 2, true);
        }
        if (Weights<D>::APART) values(t, j, j > 1, true);
      }
    } else {
      scores(1, 0, true);
      for (int j = 0; j < steps; ++j) {
        const uint32_t ph = (uint32_t)j & 1u;
        const bool next = j + 1 < steps;
        wait(&v_full[j & 1], (uint32_t)(j >> 1) & 1u);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          wait(&p_full[t], ph);
          __syncwarp();
          tc_fence_after();
          if (!Weights<D>::APART) values(t, j, j > 0, t == 1);
          if (next) {
            if (t == 0) wait(&k_full[(j + 1) & 1], (uint32_t)((j + 1) >> 1) & 1u);
            if (!Weights<D>::APART) wait(&pv_done[t], ph);
            __syncwarp();
            tc_fence_after();
            scores(t, j + 1, t == 1);
          }
          if (Weights<D>::APART) values(t, j, j > 0, t == 1);
        }
      }
    }
    // what was issued ends before the tensor memory is given back, whichever warp's wait gave up before
    if (leader) mma_commit(&all_done);
    __syncwarp();
    wait.polls = kMaxPolls;
    wait(&all_done, 0);
  }
  if (bad) record_device_error(kErrRange);
  __syncwarp();
  __syncthreads();
  if (warp == 23) tmem_dealloc(tmem, 512);
}

// Joins the parts of a split item, a warp a row.
constexpr int JOIN_WARPS = 8;
template <int D>
__global__ void __launch_bounds__(32 * JOIN_WARPS) kv4_prompt_join_kernel(Kv4Attn a, Parts parts) {
  constexpr int E = D / 32;
  pdl_wait();
  const int4 info = parts.info[blockIdx.x];
  const int r = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= info.z) return;
  const float* part = parts.sums + (int64_t)blockIdx.x * parts.splits * (ROWS * (D + 2));
  float mx = kNegInf;
  for (int s = 0; s < parts.splits; ++s) mx = fmaxf(mx, part[(int64_t)s * (ROWS * (D + 2)) + ROWS * D + r]);
  if (mx == kNegInf) mx = 0.0f;
  float l = 0.0f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
  for (int s = 0; s < parts.splits; ++s) {
    const float* p = part + (int64_t)s * (ROWS * (D + 2));
    const float f = exp2_approx(p[ROWS * D + r] - mx);
    l = fmaf(p[ROWS * (D + 1) + r], f, l);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(p[r * D + E * lane + e], f, o[e]);
  }
  const float norm = l == 0.0f ? 0.0f : 1.0f / l;
  const int gr = info.y + r;
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + (int64_t)(info.x + gr / a.share) * a.out_stride +
                       (int64_t)(info.w * a.share + gr % a.share) * D;
#pragma unroll
  for (int e = 0; e < E; ++e) out[E * lane + e] = __float2bfloat16_rn(o[e] * norm);
}

// tiles of a call's sequences, at most
int64_t tiles_of(const Kv4& c, int share) {
  const int64_t rows = (int64_t)c.total_q * share;
  const int64_t tiles = rows / ROWS + c.batch;
  return c.batch == 1 ? (rows + ROWS - 1) / ROWS : tiles;
}
// Parts of an item: where there are fewer items than SMs, enough for two blocks each SM (the lengths
// differ), each of at least 4 steps.
int splits_of(const Kv4& c, int share) {
  const int64_t items = tiles_of(c, share) * c.kv_heads, steps = ((int64_t)c.max_kv + TOK - 1) / TOK;
  if (items >= 152) return 1;
  int64_t s = (2 * 152 + items - 1) / items;
  if (s > steps / 4) s = steps / 4;
  return s < 1 ? 1 : (int)s;
}

template <int D>
cudaError_t launch(const Kv4& c, const Kv4Attn& a, int done_rows, void* ws, cudaStream_t st) {
  using P = Prompt<D>;
  const int64_t items = tiles_of(c, a.share) * c.kv_heads;
  Parts parts{};
  parts.splits = splits_of(c, a.share);
  if (parts.splits > 1) {
    parts.info = static_cast<int4*>(ws);
    parts.sums = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + (items * 16 + 255) / 256 * 256);
  }
  cudaError_t e = cudaFuncSetAttribute(kv4_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::SMEM);
  if (e != cudaSuccess) return e;
  if (items > INT32_MAX) return cudaErrorInvalidValue;
  kv4_prompt_kernel<D><<<dim3((unsigned)items, (unsigned)parts.splits), THREADS, P::SMEM, st>>>(
      c, a, done_rows, (65536u + a.share - 1) / a.share, parts);
  if ((e = cudaGetLastError()) != cudaSuccess || parts.splits == 1) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)items, ROWS / JOIN_WARPS);
  cfg.blockDim = dim3(32 * JOIN_WARPS);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_prompt_join_kernel<D>, a, parts);
}

}  // namespace

int64_t kv4_prompt_ws_bytes(const Kv4& c, int dim, int share) {
  const int64_t items = tiles_of(c, share) * c.kv_heads;
  const int splits = splits_of(c, share);
  return splits == 1 ? 0 : (items * 16 + 255) / 256 * 256 + items * splits * ROWS * (dim + 2) * 4;
}

cudaError_t launch_kv4_prompt(const Kv4& c, int dim, const Kv4Attn& a, int done_rows, void* ws, cudaStream_t st) {
  return dim == 128 ? launch<128>(c, a, done_rows, ws, st) : launch<64>(c, a, done_rows, ws, st);
}

cudaError_t read_clear_device_error_kv4_prompt(int* value) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, g_device_error, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
}

}  // namespace bitnet
