// kv4_decode.cu -- attention over the 4-bit key/value cache for a few query rows a sequence: single
// tokens and drafted ones, n * share <= 32 rows (share = query heads of one key/value head).
//
// Bound by the bytes of the cache. Every warp is its own pipeline: it fetches whole page blocks (one
// head's 64 tokens, one bulk copy of 64 D + 512 contiguous bytes) into a ring of its own in shared
// memory and never waits for another warp.
//
// Arithmetic, for one block and the rows r of a sequence:
//   raw[t][r] = sum_d code_k[t][d] q'[r][d]     tokens x rows, m16n8k16 with the codes as the A operand
//   s = scale (step_k raw + base_k sum(q))      the raw dot and its correction, fp32
//   p = 2^(s log2 e - m), l = sum p             running maximum m and sum l, fp32
//   w[t][r] = up p step_v                       the weights of the codes, as fp16
//   O[d][r] += sum_t code_v[t][d] w[t][r]       dims x rows
//   bsum[r] += w base_v / step_v                out = (O + bsum) / (up l)
// A code enters as the fp16 subnormal c * 2^-24 (its nibble masked out of the word) or c * 2^-20 (the
// nibble above, not shifted): products and fp32 sums of subnormals are exact in the matrix unit, and
// the factors go into q' (whose dims of odd nibbles are scaled by 2^-4) and into the last scaling of
// O. So a word of 8 codes costs 5 instructions for keys; for values, pairs of tokens are joined byte
// by byte first (0.75 instructions a code). q' is q at a power-of-two scale of its own row, as fp16.
// up, a power of two of each row, puts the largest p step_v that the warp has met near 2^8 (and up to 2^15 before it
// is moved), whatever steps tokens without weight have: so a w is rounded by 2^-11 of itself, and the small ones by
// 2^-32 of the row's largest at most. The rounded w also takes the base, so that the two terms of a value
// do not part; where the base is more than 64 steps the unrounded one does, since the code's term is the small one.
// The scores' fragment (tokens x rows) becomes the second product's B fragment by an 8 x 8 transpose
// in registers.
//
// Split: the pages that the batch sees, in the order sequence, head, page, are cut into equal runs,
// one a warp, whatever the lengths are (a ragged batch keeps every SM busy to the end; 64 sequences
// of 87 to 8086 tokens). A (sequence, head) unit that lies in one run is finished by its warp; one
// that is cut leaves a partial (m, l, unscaled sum) for each run, and a second kernel joins them in
// order, so results do not depend on timing. Short caches are not cut (see cuts()).
//
// Measured (20 and 5 heads x 128, one query a sequence): 8 x 65536 tokens 68.2 us (357 MB, 5.2 TB/s of the
// measured 6.7), 1 x 131072 29.9 us, 64 of 87 to 8086 43.2 us (175 MB), 1 x 76 5.5 us. What is
// added by more pages comes at 6.5 TB/s; 13 to 16 us of a cut call are fixed: launch, the search for the
// runs (3 loads, one after another), the first pages' way, the last partials, the join. With 12 to 28
// rows (16 sequences of 1221 to 9955 tokens, 3 to 7 drafted ones each, 41.0 us) the products bind: two
// units read the same pages, and registers leave two blocks an SM.
// Tried and slower: 8 warps an SM for 12 (66 us for the 64 ragged ones against 51 at the time), e4m3 operands
// of m16n8k32 (72.9 against 48.9), weights as two fp16 parts (83.7 against 74.3 for the drafted tokens), 32
// rows in one unit (68 against 39.8). The scale of the weights costs 1 to 4%: the scale by the largest step met, which
// loses weights to steps without weight, took 41.8 us for the 64 and 40.2 for the drafted tokens; up as a factor
// of its own in place of the exponent 43.2 and 42.3; up moved by the exponents of the maxima alone, with an
// exact pass where a step is large, 45.7 and 42.8.
#include "kv4.cuh"
#include "kv4_join.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace bitnet {
namespace {

constexpr int WARPS = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kMostC1 = 1.2676506002282294e30f;  // 2^100
// operands of the values' product: where the largest of a row is put, how far one may grow before that is done
// again, the least that counts for it (2^-80), and the base, in steps, up to which the rounded one also takes the base
constexpr float kFull = 256.0f, kTop = 32768.0f, kLeast = 8.271806125530277e-25f, kFar = 64.0f;
constexpr float kFirstUp = kFull / kLeast;

template <int D, int NT>
struct Shape {
  static constexpr int W = D / 8;             // words of a vector
  static constexpr int KS = D / 16;           // k steps of the scores; m tiles of the values
  static constexpr int BLK = 64 * D + 512;    // bytes of a block
  static constexpr int ROWS = 8 * NT;         // rows of a unit
  static constexpr int GROUPS = NT == 1 ? 1 : 2;  // units of a head, at most
  static constexpr int BLOCKS = NT == 1 ? 3 : 2;  // resident blocks of an SM
  static constexpr int STAGES = BLOCKS == 3 ? 2 : 3;
  static constexpr int PBYTES = kKvPage * 16;  // the page's parameters as fp32
  static constexpr int WARP_BYTES = STAGES * BLK + PBYTES;
  static constexpr int SMEM = WARPS * WARP_BYTES;
  static constexpr int PART = ROWS * (D + 2);  // floats of a partial: ROWS x D sums, then m, then l
};

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }

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
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
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
// the least power of two that is not below x (x > 0); the inverse of a power of two, and its exponent
__device__ __forceinline__ float power_from(float x) { return __uint_as_float((__float_as_uint(x) + 0x007fffffu) & 0x7f800000u); }
__device__ __forceinline__ float inverse(float power) { return __uint_as_float(0x7f000000u - __float_as_uint(power)); }
__device__ __forceinline__ float exponent(float power) { return (float)((int)(__float_as_uint(power) >> 23) - 127); }
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// plain shared-memory loads: the compiler may move them past one another, not past the barriers
template <typename T>
__device__ __forceinline__ T lds(const uint8_t* p) {
  return *reinterpret_cast<const T*>(p);
}

// V consecutive numbers of the queries from element `at` on
template <int V>
__device__ __forceinline__ void load_q(const Kv4Attn& a, int64_t at, float* x) {
  if (a.bf16) {
    uint32_t u[V / 2];
    const uint16_t* p = static_cast<const uint16_t*>(a.q) + at;
    if constexpr (V == 4) {
      const uint2 t = *reinterpret_cast<const uint2*>(p);
      u[0] = t.x, u[1] = t.y;
    } else {
      u[0] = *reinterpret_cast<const uint32_t*>(p);
    }
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      x[2 * k] = __uint_as_float(u[k] << 16);
      x[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
    }
  } else {
    const float* p = static_cast<const float*>(a.q) + at;
    if constexpr (V == 4) {
      const float4 t = *reinterpret_cast<const float4*>(p);
      x[0] = t.x, x[1] = t.y, x[2] = t.z, x[3] = t.w;
    } else {
      const float2 t = *reinterpret_cast<const float2*>(p);
      x[0] = t.x, x[1] = t.y;
    }
  }
}

// The pages that the rows of a sequence see: page i of np is page i of the sequence, or i + skip from
// i = ns on (what lies between the sinks and the window of the first row). np = 0: no row of this
// kernel's, or nothing cached.
struct Span {
  int np, ns, skip;
};
__device__ __forceinline__ Span span_of(const Kv4& c, const Kv4Attn& a, const Kv4Seq& s, int max_rows) {
  Span p{0, 0, 0};
  if (s.n < 1 || (int64_t)s.n * a.share > max_rows || s.len < 1) return p;
  const int low = (int)max((int64_t)0, (int64_t)s.len - s.n - a.window + 1);
  const int low_page = low / kKvPage, sink_pages = (min(a.sinks, low) + kKvPage - 1) / kKvPage;
  p.ns = min(sink_pages, low_page);
  p.skip = low_page - p.ns;
  p.np = p.ns + (s.len + kKvPage - 1) / kKvPage - low_page;
  return p;
}

// where the runs' results go in the workspace: for each unit the first and the last run that hold a
// part of it, then two partials for each run (a run's first and last unit may be cut)
struct Work {
  int2* runs;     // batch x kv_heads x GROUPS
  float* parts;   // n_runs x 2 x PART
  int n_runs;     // of the grid: as many as are made, or more
};

// Rows beyond a unit's make another unit of the same head and pages (17 to 32 rows: registers hold the
// sums of 16).
__device__ __forceinline__ int groups_of(const Kv4Seq& s, const Kv4Attn& a, int rows) {
  return (s.n * a.share + rows - 1) / rows;
}
// A unit (sequence b, head h / groups, its rows from rows * (h % groups) on) and the pages [i, until) of it that a run holds; weight is what the run
// holds beyond them.
struct Unit {
  int b, h, i, until, weight, groups;  // groups: 1 or 2; MOST says where it is always 1
  template <int MOST>
  __device__ __forceinline__ int head() const {
    return MOST == 2 && groups == 2 ? h >> 1 : h;
  }
  template <int MOST>
  __device__ __forceinline__ int group() const {
    return MOST == 2 && groups == 2 ? h & 1 : 0;
  }
  Kv4Seq s;
  Span p;
};
// Beginning a unit costs about what a page does (its queries' latency, its results): it counts as
// kUnitCost pages when the runs are cut.
constexpr int kUnitCost = 2;

// the next unit of a run; false at the run's end
template <int ROWS, int GROUPS>
__device__ __forceinline__ bool next_unit(Unit& u, const Kv4& c, const Kv4Attn& a, bool* bad) {
  if (u.until < u.p.np || u.weight <= kUnitCost) return false;
  if (++u.h == c.kv_heads * (GROUPS == 1 ? 1 : u.groups)) {
    u.h = 0;
    do {
      if (++u.b >= c.batch) return false;
      u.s = kv4_sequence(c, u.b, bad);
      u.p = span_of(c, a, u.s, ROWS * GROUPS);
    } while (u.p.np == 0);
    u.groups = GROUPS == 1 ? 1 : groups_of(u.s, a, ROWS);
  }
  u.weight -= kUnitCost;
  u.i = 0;
  u.until = min(u.p.np, u.weight);
  u.weight -= u.until;
  return true;
}

// SPLIT: units are cut into runs of all warps of the grid, and what they leave is joined by a second
// kernel. Otherwise a block takes one unit, its warps a part each, and joins them itself.
template <int D, int NT, bool SPLIT>
__global__ void __launch_bounds__(32 * WARPS, Shape<D, NT>::BLOCKS) kv4_decode_kernel(Kv4 c, Kv4Attn a, Work ws) {
  using S = Shape<D, NT>;
  constexpr int W = S::W, KS = S::KS, BLK = S::BLK, STAGES = S::STAGES;
  constexpr int V = W / 4;  // consecutive words, so dimensions, of a lane's queries and keys
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[WARPS][STAGES];
  __shared__ int64_t scan[WARPS];
  __shared__ Unit starts[WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q4 = lane & 3;
  bool bad = false;
  if (SPLIT) pdl_launch_dependents();
  if (lane == 0)
    for (int i = 0; i < STAGES; ++i) mbar_init(&full[warp][i], 1);
  fence_mbar_init();

  Unit use;           // the unit being used
  bool inside;        // the block's warps join their partials in shared memory
  int64_t run = 0;
  if constexpr (SPLIT) {
    // weights of the sequences before each thread's share of them, then each run's start
    const int per = (c.batch + 32 * WARPS - 1) / (32 * WARPS);
    const int b0 = min((int)threadIdx.x * per, c.batch), b1 = min(b0 + per, c.batch);
    int64_t mine = 0;
    Kv4Seq s{0, 0, 0};
    Span p{0, 0, 0};
    for (int b = b0; b < b1; ++b) {
      s = kv4_sequence(c, b, &bad);
      p = span_of(c, a, s, S::ROWS * S::GROUPS);
      if (p.np) mine += (int64_t)(p.np + kUnitCost) * c.kv_heads * (S::GROUPS == 1 ? 1 : groups_of(s, a, S::ROWS));
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    int64_t before = upto - mine, total = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
      if (i < warp) before += scan[i];
      total += scan[i];
    }
    // run r begins at r * size + min(r, rest)
    const int64_t n_runs = min(total, (int64_t)gridDim.x * WARPS);
    const int64_t run0 = (int64_t)blockIdx.x * WARPS;
    if (run0 >= n_runs) {  // the whole block
      if (bad) record_device_error(kErrRange);
      return;
    }
    const int64_t size = total <= INT32_MAX ? (uint32_t)total / (uint32_t)n_runs : total / n_runs;
    const int64_t rest = total - size * n_runs;
    const auto begin = [&](int64_t r) { return r * size + min(r, rest); };
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
      const int64_t x = begin(run0 + i);
      if (run0 + i >= n_runs || x < before || x >= before + mine) continue;
      int64_t at = before;
      for (int b = b0; b < b1; ++b) {
        if (per > 1) {
          s = kv4_sequence(c, b, &bad);
          p = span_of(c, a, s, S::ROWS * S::GROUPS);
        }
        if (p.np == 0) continue;
        const int unit = p.np + kUnitCost;
        const int groups = S::GROUPS == 1 ? 1 : groups_of(s, a, S::ROWS);
        const int64_t here = (int64_t)unit * c.kv_heads * groups;
        if (x < at + here) {
          const int h = here <= INT32_MAX ? (uint32_t)(x - at) / (uint32_t)unit : (int)((x - at) / unit);
          starts[i] = Unit{b, h, (int)(x - at - (int64_t)h * unit), 0, (int)(begin(run0 + i + 1) - x), groups, s, p};
          break;
        }
        at += here;
      }
    }
    __syncthreads();
    run = run0 + warp;
    if (run >= n_runs) {
      if (bad) record_device_error(kErrRange);
      return;
    }
    use = starts[warp];
    // from a place in the unit's weight to its pages
    const int64_t unit_at = begin(run) - use.i;
    const int skip = max(0, kUnitCost - use.i);  // what the run pays of the unit's cost
    use.i = max(0, use.i - kUnitCost);
    use.weight -= skip;
    use.until = max(use.i, min(use.p.np, use.i + use.weight));
    use.weight -= use.until - use.i;
    inside = begin(run0) - unit_at > kUnitCost && begin(run0 + WARPS) - unit_at - kUnitCost < use.p.np;
    if (use.until == use.i) {  // it ends within the unit's cost
      if (bad) record_device_error(kErrRange);
      return;
    }
  } else {
    use.b = blockIdx.x / (c.kv_heads * S::GROUPS);
    use.h = blockIdx.x - use.b * c.kv_heads * S::GROUPS;
    use.s = kv4_sequence(c, use.b, &bad);
    use.p = span_of(c, a, use.s, S::ROWS * S::GROUPS);
    const bool few = (int64_t)use.s.n * a.share <= S::ROWS * S::GROUPS;
    use.groups = few ? groups_of(use.s, a, S::ROWS) : 0;
    if (use.h >= c.kv_heads * use.groups || use.p.np == 0) {
      if (use.h < c.kv_heads * use.groups)  // nothing cached: zeros
        for (int r = S::ROWS * use.template group<S::GROUPS>() + warp; r < min(use.s.n * a.share, S::ROWS * (use.template group<S::GROUPS>() + 1)); r += WARPS)
          for (int d = lane; d < D; d += 32)
            a.out[(int64_t)(use.s.q0 + r / a.share) * a.out_stride + (int64_t)(use.template head<S::GROUPS>() * a.share + r % a.share) * D + d] = 0;
      if (bad) record_device_error(kErrRange);
      return;
    }
    use.i = (int)((int64_t)use.p.np * warp / WARPS);
    use.until = (int)((int64_t)use.p.np * (warp + 1) / WARPS);
    use.weight = 0;
    inside = true;
  }
  // the first unit's rows: it is the only one where they are joined here
  const int rows0 = S::ROWS * use.template group<S::GROUPS>(), rows = min(S::ROWS, use.s.n * a.share - rows0);

  uint8_t* const ring = smem + warp * S::WARP_BYTES;
  float4* const par = reinterpret_cast<float4*>(ring + STAGES * BLK);
  Unit get = use;                    // the unit whose page is fetched next
  bool more = use.i < use.until;     // there is a page to fetch
  int ids = 0, ids_from = -64;       // page ids ids_from .. + 31 of the unit, one a lane
  int in_flight = 0;
  bool abort = false;

  auto fetch = [&](int stage) {
    if (!more) return;
    if (get.i < ids_from || get.i >= ids_from + 32) {
      ids_from = get.i;
      const int i = min(get.i + lane, get.p.np - 1);
      ids = c.page_table[(int64_t)get.b * c.max_pages + (i < get.p.ns ? i : i + get.p.skip)];
      if (ids < 0 || ids >= c.n_pages) bad = true, ids = 0;
    }
    const int id = __shfl_sync(0xffffffffu, ids, get.i - ids_from);
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[warp][stage], BLK);
      bulk_copy_g2s(ring + stage * BLK, c.pages + ((int64_t)id * c.kv_heads + get.template head<S::GROUPS>()) * BLK, BLK, &full[warp][stage]);
    }
    ++in_flight;
    if (++get.i == get.until) {
      const int b = get.b;
      more = next_unit<S::ROWS, S::GROUPS>(get, c, a, &bad);
      if (get.b != b) ids_from = -64;
      if (more) {  // its queries are wanted soon
        const int bytes = a.share * D * (a.bf16 ? 2 : 4);
        for (int i = 0; i < get.s.n; ++i) {
          const char* q = static_cast<const char*>(a.q) +
                          ((get.s.q0 + i) * a.q_stride + (int64_t)get.template head<S::GROUPS>() * a.share * D) * (a.bf16 ? 2 : 4);
          for (int o = 128 * lane; o < bytes; o += 128 * 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + o));
        }
      }
    }
  };

  uint32_t qf[NT][KS][2];
  // per row (column of the fragments): u = step raw + base qs is the score up to the factor c1 >= 0,
  // m its running maximum; weights, and so l, O and bs, are up times what they stand for, a power of two
  float c1[NT][2], qs2[NT][2], m[NT][2], up[NT][2];
  uint64_t l[NT], bs[NT];
  int pos[NT][2];
  float O[NT][KS][4];
  int stage = 0;
  uint32_t parity = 0;
  bool started = false;

  while (use.i < use.until) {
    const bool begun = use.i == 0;  // this run holds the unit's first page
    const int row0 = S::ROWS * use.template group<S::GROUPS>();
    {  // a new unit: its queries
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = row0 + 8 * nt + g, i = r / a.share;
        float x[D / 4];
        if (i < use.s.n) {
          const int64_t at = (int64_t)(use.s.q0 + i) * a.q_stride + (int64_t)(use.template head<S::GROUPS>() * a.share + r % a.share) * D + V * q4;
#pragma unroll
          for (int n = 0; n < 8; ++n) load_q<V>(a, at + W * n, &x[n * V]);
        } else {
#pragma unroll
          for (int e = 0; e < D / 4; ++e) x[e] = 0.0f;
        }
        if (!started) {  // behind the first queries: the copies fill the memory's queues
          started = true;
#pragma unroll
          for (int k = 0; k < STAGES; ++k) fetch(k);
        }
        float mx = 0.0f;
#pragma unroll
        for (int e = 0; e < D / 4; ++e) mx = fmaxf(mx, fabsf(x[e]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // q' = q 2^(13 - e), 2^e <= max |q| < 2^(e + 1): fp16 with 2^-28 of the maximum still a normal
        // number, also where it is scaled by 2^-4. Not below e = -100, and not for infinities.
        int e = (int)(__float_as_uint(mx) >> 23) - 127;
        e = e == 128 ? 13 : max(e, -100);
        const float grow = __int_as_float((13 - e + 127) << 23) * (a.scale < 0.0f ? -1.0f : 1.0f), down = __int_as_float((e - 13 + 127) << 23);
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < D / 4; ++k) {
          x[k] = __half2float(__float2half_rn(x[k] * grow));
          sum += x[k];
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int v = s >> 1, n = (s & 1) * 2;  // word v of the lane; nibbles n, n + 4 and n + 1, n + 5
          const uint32_t f0 = pack_half2(x[n * V + v], x[(n + 4) * V + v]);
          const uint32_t f1 = pack_half2(x[(n + 1) * V + v] * 0.0625f, x[(n + 5) * V + v] * 0.0625f);
          qf[nt][s][0] = f0, qf[nt][s][1] = f1;
        }
        // c1 of 0 would make NaN of a masked score, and c1 of 2^100 already sets unlike scores (2^-72 apart at
        // least, 2^14 at most) infinitely far apart: from there on it would overflow
        const float k1 = fminf(fmaxf(fabsf(a.scale) * kLog2e * down * 16777216.0f, 1.17549435e-38f), kMostC1);
        const float k0 = sum * 5.9604644775390625e-8f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = 2 * q4 + j;
          c1[nt][j] = __shfl_sync(0xffffffffu, k1, 4 * col);
          qs2[nt][j] = __shfl_sync(0xffffffffu, k0, 4 * col);
          pos[nt][j] = use.s.len - use.s.n + (row0 + 8 * nt + col) / a.share;
          m[nt][j] = kNegInf;
          up[nt][j] = kFirstUp;
        }
        l[nt] = bs[nt] = 0;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) O[nt][k][j] = 0.0f;
      }
      __syncwarp();
    }

    const int first_low = (int)max((int64_t)0, (int64_t)use.s.len - use.s.n - a.window + 1);
    const int last_low = (int)max((int64_t)0, (int64_t)use.s.len - a.window);
    for (; use.i < use.until; ++use.i) {
      if (__any_sync(0xffffffffu, !mbar_try_wait(smem_u32(&full[warp][stage]), parity)) &&
          !mbar_wait_warp(&full[warp][stage], parity, &abort))
        break;
      const uint8_t* const blk = ring + stage * BLK;
      const int first = (use.i < use.p.ns ? use.i : use.i + use.p.skip) * kKvPage;  // the page's first position
      // whether every row sees the whole page
      const bool whole = first + kKvPage <= use.s.len - use.s.n + 1 &&
                         (first >= last_low || first + kKvPage <= a.sinks);

      // the parameters of two tokens a lane, as fp32: key step and base, value step and base over step
      bool far = false;  // a base of many steps
      {
        float4 two[2];
        const uint4 u = lds<uint4>(blk + kKvPage * D + lane * 16);
        const uint32_t raw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 pk = __half22float2(*reinterpret_cast<const __half2*>(&raw[2 * e]));
          const float2 pv = __half22float2(*reinterpret_cast<const __half2*>(&raw[2 * e + 1]));
          // a value vector of NaN acts through its score, so that a weight of 0 never meets a NaN
          const float z = (pv.x - pv.x) + (pv.y - pv.y);
          bool none = z != 0.0f;
          if (!whole) {  // nor what lies where no row of the unit looks
            const int j = first + kv4_rho_inv(2 * lane + e);
            none |= j >= use.s.len || (j < first_low && j >= a.sinks);
          }
          // codes of a step of 0 are 0: any other step stands for the same value
          const float step = pv.x > 0.0f ? pv.x : fabsf(pv.y);
          two[e] = make_float4(pk.x, pk.y + z, none ? 0.0f : step, none || step == 0.0f ? 0.0f : __fdividef(pv.y, step));
          par[2 * lane + e] = two[e];
          far |= fabsf(two[e].w) > kFar;
        }
        far = __any_sync(0xffffffffu, far);
        __syncwarp();
      }

      // scores
      float s[NT][4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t k0[W / 4], k1[W / 4];  // rows g and g + 8 of the tile
        const uint8_t* const at = blk + (16 * i + g) * (D / 2) + q4 * W;
        if constexpr (D == 128) {
          const uint4 u = lds<uint4>(at), v = lds<uint4>(at + 8 * (D / 2));
          k0[0] = u.x, k0[1] = u.y, k0[2] = u.z, k0[3] = u.w;
          k1[0] = v.x, k1[1] = v.y, k1[2] = v.z, k1[3] = v.w;
        } else {
          const uint2 u = lds<uint2>(at), v = lds<uint2>(at + 8 * (D / 2));
          k0[0] = u.x, k0[1] = u.y;
          k1[0] = v.x, k1[1] = v.y;
        }
#pragma unroll
        for (int st = 0; st < KS; ++st) {
          const int v = st >> 1;
          const uint32_t x = st & 1 ? k0[v] >> 8 : k0[v], y = st & 1 ? k1[v] >> 8 : k1[v];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 f = make_uint2(qf[nt][st][0], qf[nt][st][1]);
            if (st == 0)
              mma16816<true>(s[nt][i], x & 0x000f000fu, y & 0x000f000fu, x & 0x00f000f0u, y & 0x00f000f0u, f.x, f.y);
            else
              mma16816<false>(s[nt][i], x & 0x000f000fu, y & 0x000f000fu, x & 0x00f000f0u, y & 0x00f000f0u, f.x, f.y);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // rows g and g + 8: the correction
          const float2 k = *reinterpret_cast<const float2*>(&par[16 * i + 8 * e + g]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              s[nt][i][2 * e + j] = fmaf(k.x, s[nt][i][2 * e + j], k.y * qs2[nt][j]);
        }
      }
      if (!whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = first + kv4_rho_inv(16 * i + 8 * e + g);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j2 = 0; j2 < 2; ++j2) {
                const int p = pos[nt][j2];
                if (j > p || (p - j >= a.window && j >= a.sinks)) s[nt][i][2 * e + j2] = kNegInf;
              }
          }
      }
      // running maxima
      float mn[NT][2], al[NT][2];  // al: what is left of the old weights
      bool moves = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v = m[nt][j];
#pragma unroll
          for (int i = 0; i < 4; ++i) v = fmaxf(v, fmaxf(s[nt][i][j], s[nt][i][2 + j]));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          mn[nt][j] = v;
          al[nt][j] = 1.0f;
          moves |= v > m[nt][j];
        }
      moves = __any_sync(0xffffffffu, moves);
      if (moves) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            al[nt][j] = mn[nt][j] == kNegInf ? 1.0f : exp2_approx(c1[nt][j] * (m[nt][j] - mn[nt][j]));
            m[nt][j] = mn[nt][j];
          }
          l[nt] = fma2(l[nt], f2pack(al[nt][0], al[nt][1]), 0);
        }
      }
      // weights times up in l; times steps, what a code adds to its row, in s
      float most[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const Kv4Weight w0 = kv4_weight(c1[nt][0], m[nt][0], 22), w1 = kv4_weight(c1[nt][1], m[nt][1], 22);
        const uint64_t c1p = f2pack(w0.c, w1.c), off = f2pack(w0.off + exponent(up[nt][0]), w1.off + exponent(up[nt][1]));
        most[nt][0] = most[nt][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float step = par[16 * i + 8 * e + g].z;
            const float2 t = f2unpack(fma2(f2pack(s[nt][i][2 * e], s[nt][i][2 * e + 1]), c1p, off));
            const uint64_t p = f2pack(exp2_approx(t.x), exp2_approx(t.y));
            l[nt] = add2(l[nt], p);
            const float2 y = f2unpack(mul2(p, f2pack(step, step)));
            s[nt][i][2 * e] = y.x, s[nt][i][2 * e + 1] = y.y;
          }
          most[nt][0] = max3(most[nt][0], s[nt][i][0], s[nt][i][2]);
          most[nt][1] = max3(most[nt][1], s[nt][i][1], s[nt][i][3]);
        }
        moves |= fmaxf(most[nt][0], most[nt][1]) > kTop;
      }
      // their scale follows the largest of them
      if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float f[2], more[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float v = most[nt][j];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            const float old = inverse(up[nt][j]);
            v = fmaxf(fmaxf(v, al[nt][j] * kFull) * old, kLeast);
            up[nt][j] = kFull * inverse(power_from(v));
            more[j] = up[nt][j] * old;
            f[j] = al[nt][j] * more[j];
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nt][i][j] *= more[j], s[nt][i][2 + j] *= more[j];
          }
          l[nt] = mul2(l[nt], f2pack(more[0], more[1]));
          bs[nt] = mul2(bs[nt], f2pack(f[0], f[1]));
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) O[nt][k][j] *= f[j & 1];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t wf[NT][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float ratio = par[16 * i + 8 * e + g].w;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t w = pack_half2(s[nt][i][2 * e], s[nt][i][2 * e + 1]);
            const float2 wr = __half22float2(*reinterpret_cast<const __half2*>(&w));
            bs[nt] = fma2(f2pack(wr.x, wr.y), f2pack(ratio, ratio), bs[nt]);
            wf[nt][e] = transpose8x8(w);
          }
        }
        // values: tokens 16 i + q4 (+ 4, + 8, + 12), the words of dimension rows g
        const uint8_t* const at = blk + kKvPage * (D / 2) + (16 * i + q4) * (D / 2);
        uint32_t v[4][W / 8];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          if constexpr (D == 128) {
            const uint2 u = lds<uint2>(at + t * 4 * (D / 2) + ((8 * g) ^ ((q4 & 2) << 4)));
            v[t][0] = u.x, v[t][1] = u.y;
          } else {
            v[t][0] = lds<uint32_t>(at + t * 4 * (D / 2) + 4 * g);
          }
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int x = k >> 2, by = k & 3;  // word, byte
          const uint32_t sel = 0x4400u + 0x1111u * by;
          const uint32_t a01 = __byte_perm(v[0][x], v[1][x], sel), a23 = __byte_perm(v[2][x], v[3][x], sel);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816<false>(O[nt][k], a01 & 0x000f000fu, a01 & 0x00f000f0u, a23 & 0x000f000fu, a23 & 0x00f000f0u,
                            wf[nt][0], wf[nt][1]);
        }
      }
      if (far) {  // a base of many steps takes what the rounding took
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float ratio = par[16 * i + 8 * e + g].w;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float y0 = s[nt][i][2 * e], y1 = s[nt][i][2 * e + 1];
              const float r = fabsf(ratio) > kFar ? ratio : 0.0f;
              const float d0 = y0 - __half2float(__float2half_rn(y0)), d1 = y1 - __half2float(__float2half_rn(y1));
              bs[nt] = fma2(f2pack(d0, d1), f2pack(r, r), bs[nt]);
            }
          }
      }
      __syncwarp();  // every lane has read the block: its place may be written again
      --in_flight;
      fetch(stage);
      if (++stage == STAGES) stage = 0, parity ^= 1u;
    }
    if (abort) break;

    {  // the unit ends, or this run's part of it
      const bool ends = use.i == use.p.np, alone = SPLIT && begun && ends;
      const int unit_rows = min(S::ROWS, use.s.n * a.share - row0);
      const int64_t unit = (int64_t)use.b * c.kv_heads * S::GROUPS + use.h;
      float* part = inside ? reinterpret_cast<float*>(ring) : ws.parts + (2 * run + (begun ? 1 : 0)) * S::PART;
      if (SPLIT && lane == 0) {
        if (begun) ws.runs[unit].x = (int)run;
        if (ends) ws.runs[unit].y = (int)run;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 ls = f2unpack(l[nt]), bsum = f2unpack(bs[nt]);
          float sl = j ? ls.y : ls.x, sb = j ? bsum.y : bsum.x;
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            sl += __shfl_xor_sync(0xffffffffu, sl, o);
            sb += __shfl_xor_sync(0xffffffffu, sb, o);
          }
          const int r = 8 * nt + 2 * q4 + j;
          if (r >= unit_rows) continue;
          const float norm = alone ? (sl == 0.0f ? 0.0f : 1.0f / sl) : inverse(up[nt][j]);
          uint16_t* out = a.out + (int64_t)(use.s.q0 + (row0 + r) / a.share) * a.out_stride +
                          (int64_t)(use.template head<S::GROUPS>() * a.share + (row0 + r) % a.share) * D;
#pragma unroll
          for (int n = 0; n < 8; ++n) {  // nibble n: dimension W n + word
            float y[W / 8];
#pragma unroll
            for (int x = 0; x < W / 8; ++x)
              y[x] = fmaf(O[nt][4 * x + (n >> 1)][(n & 1) * 2 + j], n & 1 ? 1048576.0f : 16777216.0f, sb) * norm;
            const int d = W * n + (W / 8) * g;
            if constexpr (D == 128) {
              if (alone)
                *reinterpret_cast<__nv_bfloat162*>(out + d) = __floats2bfloat162_rn(y[0], y[1]);
              else
                *reinterpret_cast<float2*>(part + r * D + d) = make_float2(y[0], y[1]);
            } else {
              if (alone)
                reinterpret_cast<__nv_bfloat16*>(out)[d] = __float2bfloat16_rn(y[0]);
              else
                part[r * D + d] = y[0];
            }
          }
          if (!alone && g == 0) {
            part[S::ROWS * D + r] = m[nt][j] * c1[nt][j];
            part[S::ROWS * (D + 1) + r] = sl * norm;
          }
        }
    }
    if (!next_unit<S::ROWS, S::GROUPS>(use, c, a, &bad)) break;
  }
  if (abort && lane == 0) {  // copies in flight land before the block ends
    bool given_up = false;
    for (; in_flight > 0; --in_flight) {
      mbar_wait(&full[warp][stage], parity, &given_up);
      if (++stage == STAGES) stage = 0, parity ^= 1u;
    }
  }
  if (inside) {
    __syncthreads();
    const auto parts = [&](int i) { return reinterpret_cast<const float*>(smem + i * S::WARP_BYTES); };
    float* part = SPLIT ? ws.parts + 2 * (int64_t)blockIdx.x * WARPS * S::PART : nullptr;
    for (int r = warp; r < rows; r += WARPS) {
      float mx = kNegInf, f[WARPS], sl = 0.0f;
      bool has[WARPS];  // a warp of a unit with fewer pages than warps has no part
#pragma unroll
      for (int i = 0; i < WARPS; ++i) {
        has[i] = SPLIT || (int64_t)use.p.np * (i + 1) / WARPS > (int64_t)use.p.np * i / WARPS;
        if (has[i]) mx = fmaxf(mx, parts(i)[S::ROWS * D + r]);
      }
      const float ref = mx == kNegInf ? 0.0f : mx;
#pragma unroll
      for (int i = 0; i < WARPS; ++i)
        if (has[i]) {
          f[i] = exp2_approx(parts(i)[S::ROWS * D + r] - ref);
          sl = fmaf(parts(i)[S::ROWS * (D + 1) + r], f[i], sl);
        }
      const float norm = sl == 0.0f ? 0.0f : 1.0f / sl;
      uint16_t* out = a.out + (int64_t)(use.s.q0 + (rows0 + r) / a.share) * a.out_stride +
                      (int64_t)(use.template head<S::GROUPS>() * a.share + (rows0 + r) % a.share) * D;
#pragma unroll
      for (int d = 0; d < D; d += 32) {
        float o = 0.0f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i)
          if (has[i]) o = fmaf(parts(i)[r * D + d + lane], f[i], o);
        if (SPLIT)
          part[r * D + d + lane] = o;
        else
          reinterpret_cast<__nv_bfloat16*>(out)[d + lane] = __float2bfloat16_rn(o * norm);
      }
      if (SPLIT && lane == 0) {
        part[S::ROWS * D + r] = mx;
        part[S::ROWS * (D + 1) + r] = sl;
      }
    }
  }
  if (bad) record_device_error(kErrRange);
}

// Joins the partials of one row of a unit, in the order of the runs; zeros for a row of a sequence
// that has nothing cached. A unit finished by one run is left alone.
constexpr int JOIN_WARPS = 16;  // at most
template <int D, int ROWS, int GROUPS>
__global__ void __launch_bounds__(32 * JOIN_WARPS) kv4_join_kernel(Kv4 c, Kv4Attn a, Work ws) {
  constexpr int PART = ROWS * (D + 2), E = D / 32;
  __shared__ float part_m[JOIN_WARPS], part_l[JOIN_WARPS], part_o[JOIN_WARPS][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int b = blockIdx.x / c.kv_heads, h = blockIdx.x - b * c.kv_heads, gr = blockIdx.y;  // row of the head
  bool bad = false;
  const Kv4Seq s = kv4_sequence(c, b, &bad);
  pdl_wait();
  const int64_t rows = (int64_t)s.n * a.share;
  if (rows > ROWS * GROUPS || gr >= rows) return;
  uint16_t* out = a.out + (int64_t)(s.q0 + gr / a.share) * a.out_stride + (int64_t)(h * a.share + gr % a.share) * D;
  if (s.len < 1) {
    for (int d = threadIdx.x; d < D; d += blockDim.x) out[d] = 0;
    if (bad && threadIdx.x == 0) record_device_error(kErrRange);
    return;
  }
  const int r = gr % ROWS, groups = groups_of(s, a, ROWS);
  const int2 runs = ws.runs[(int64_t)b * c.kv_heads * GROUPS + h * groups + gr / ROWS];
  const Kv4Join join = kv4_join(runs.x, runs.y, ws.n_runs, WARPS);
  if (join.count == 0) return;
  float m = kNegInf, l = 0.0f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll 4
  for (int k = warp; k < join.count; k += warps) {
    const int i = join.run(k);
    const float* part = ws.parts + (2 * (int64_t)i + (i == runs.x ? 1 : 0)) * PART;
    const float pm = part[ROWS * D + r], pl = part[ROWS * (D + 1) + r];
    float po[E];
#pragma unroll
    for (int e = 0; e < E; ++e) po[e] = part[r * D + E * lane + e];
    const float mn = fmaxf(m, pm), ref = mn == kNegInf ? 0.0f : mn;
    const float f = exp2_approx(m - ref), pf = exp2_approx(pm - ref);
    m = mn;
    l = l * f + pl * pf;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + po[e] * pf;
  }
  if (lane == 0) part_m[warp] = m, part_l[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) part_o[warp][E * lane + e] = o[e];
  __syncthreads();
  float mx = kNegInf;
  for (int i = 0; i < warps; ++i) mx = fmaxf(mx, part_m[i]);
  if (mx == kNegInf) mx = 0.0f;
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    float sl = 0.0f, so = 0.0f;
    for (int i = 0; i < warps; ++i) {
      const float f = exp2_approx(part_m[i] - mx);
      sl = fmaf(part_l[i], f, sl);
      so = fmaf(part_o[i][d], f, so);
    }
    reinterpret_cast<__nv_bfloat16*>(out)[d] = __float2bfloat16_rn(sl == 0.0f ? 0.0f : so / sl);
  }
}

// the most pages that a sequence can show the rows of a call, and units of a call
int64_t most_pages(const Kv4& c) { return ((int64_t)c.max_kv + kKvPage - 1) / kKvPage; }
int64_t units_of(const Kv4& c, int rows) { return (int64_t)c.batch * c.kv_heads * (rows > 16 ? 2 : 1); }
// runs of a call: a warp each of `resident` blocks, fewer where there are not as many pages to see
int64_t runs_of(const Kv4& c, int rows, int resident) {
  const int64_t weight = units_of(c, rows) * (most_pages(c) + kUnitCost);
  const int64_t blocks = (weight + WARPS - 1) / WARPS;
  return WARPS * (blocks < 1 ? 1 : blocks < resident ? blocks : resident);
}
int64_t runs_bytes(const Kv4& c, int rows) { return (units_of(c, rows) * (int64_t)sizeof(int2) + 255) / 256 * 256; }
// Warps that join a row: as many as its partials keep busy. Measured, us, with 16, 8 and 2 (20 and 5 heads x
// 128): 1 x 131072 tokens (365 runs a unit) 29.9, 32.5, 48.6; 16 x 4096 (23) 22.0, 21.9, 22.1; 8 x 65536 (46)
// 68.1, 68.3, 71.2; 64 x 4096 (6) 47.3, 44.2, 43.2; 256 x 8192 (1) 253, 240, 233.
unsigned join_warps(const Kv4& c, int rows, int resident) {
  const int64_t runs = runs_of(c, rows, resident), units = units_of(c, rows);
  return runs > 64 * units ? JOIN_WARPS : runs > 8 * units ? 8 : 2;
}
// Whether units are cut. A block for each unit needs no search for the runs and no second kernel, but
// lasts as long as the longest: measured, cut and uncut, us (20 and 5 heads x 128, one query a
// sequence): 1 x 512 tokens 9.7, 6.6; 1 x 1024 10.4, 9.4; 1 x 4096 10.9, 24.7; 64 x 1024 22.5, 17.4;
// 64 x 2048 29.7, 27.2; 64 x 4096 43.2, 46.0; 256 x 2048 76.0, 70.0. (Heads of 64 go by the same rule; their
// lengths were not swept.) A window bounds the pages too (for
// the workspace, whose size does not depend on it, it is taken for none).
bool cuts(const Kv4& c, int window, int sinks) {
  int64_t pages = most_pages(c);
  const int64_t seen = ((int64_t)window + c.max_q + 2 * kKvPage - 3) / kKvPage + ((int64_t)sinks + kKvPage - 1) / kKvPage;
  if (window != INT32_MAX && seen < pages) pages = seen;
  const int64_t uncut = 16 + (int64_t)c.batch * c.kv_heads / 10;
  return pages > (uncut < 64 ? uncut : 64);
}

// rows: 8, 16, or 32 (two units of 16 a head where a sequence has more than 16)
template <int D, int NT>
cudaError_t launch(const Kv4& c, const Kv4Attn& a, int rows, void* workspace, int num_sms, cudaStream_t st) {
  using S = Shape<D, NT>;
  Work ws{};
  cudaError_t e;
  if (!cuts(c, a.window, a.sinks)) {
    e = cudaFuncSetAttribute(kv4_decode_kernel<D, NT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    kv4_decode_kernel<D, NT, false><<<(unsigned)(c.batch * c.kv_heads * S::GROUPS), 32 * WARPS, S::SMEM, st>>>(c, a, ws);
    return cudaGetLastError();
  }
  ws.runs = static_cast<int2*>(workspace);
  ws.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + runs_bytes(c, S::ROWS * S::GROUPS));
  e = cudaFuncSetAttribute(kv4_decode_kernel<D, NT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
  if (e != cudaSuccess) return e;
  ws.n_runs = (int)runs_of(c, rows, S::BLOCKS * num_sms);
  kv4_decode_kernel<D, NT, true><<<(unsigned)(ws.n_runs / WARPS), 32 * WARPS, S::SMEM, st>>>(c, a, ws);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  const int64_t all = (int64_t)c.max_q * a.share;
  cfg.gridDim = dim3((unsigned)(c.batch * c.kv_heads), (unsigned)(all < rows ? all : rows));
  cfg.blockDim = dim3(32 * join_warps(c, rows, S::BLOCKS * num_sms));
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, S::ROWS, S::GROUPS>, c, a, ws);
}
template <int D>
cudaError_t launch_rows(const Kv4& c, const Kv4Attn& a, int rows, void* ws, int num_sms, cudaStream_t st) {
  return rows <= 8 ? launch<D, 1>(c, a, rows, ws, num_sms, st) : launch<D, 2>(c, a, rows, ws, num_sms, st);
}

}  // namespace

int64_t kv4_decode_ws_bytes(const Kv4& c, int dim, int rows) {
  if (!cuts(c, INT32_MAX, 0)) return 0;
  // as for the largest GPU of this kind (160 SMs), so that the size does not depend on the device
  const int unit_rows = rows <= 8 ? 8 : 16;
  return runs_bytes(c, rows <= 8 ? 8 : 32) + runs_of(c, rows, 3 * 160) * 2 * unit_rows * (dim + 2) * 4;
}

cudaError_t launch_kv4_decode(const Kv4& c, int dim, const Kv4Attn& a, int rows, void* ws, int num_sms,
                              cudaStream_t st) {
  if (num_sms > 160) num_sms = 160;
  return dim == 128 ? launch_rows<128>(c, a, rows, ws, num_sms, st) : launch_rows<64>(c, a, rows, ws, num_sms, st);
}

cudaError_t read_clear_device_error_kv4_decode(int* value) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, g_device_error, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
}

}  // namespace bitnet
