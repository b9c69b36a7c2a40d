// kv4_evict.cu -- eviction: long sequences keep the tokens that gathered most attention weight.
//
// One kernel; a cluster of one to sixteen blocks for each sequence and head. Its blocks take a run of tokens each and keep
// the ranks of their masses (whole numbers in the masses' order) in shared memory. The least rank that is kept is found by
// three passes that count digits (11, 11 and 10 bits, from the top; the first while the masses are read), added up over the cluster through distributed
// shared memory; then every warp counts and lists the kept tokens of its run, in order, and the cluster moves them: codes,
// parameters and mass, as they are. In place a token only moves to an earlier slot, and a chunk of tokens is read
// whole, by all blocks of the cluster, before any of it is written, so that nothing is overwritten before it has been read.
// New lengths that replace the old ones (which all clusters of a sequence read) are written by a second kernel.
//
// Bound by latency where sequences are few: loads that depend on each other (length, page, mass; kept token, page, data) and
// the cluster's barriers; by issue slots and the moved bytes where they are many. Measured (5 heads x 128, into other pages):
// 131007 tokens to 4096 24.3 us (in place 24.9), to 64 23; 16000 to 64 15.3; 48 sequences of 501 to 16001 to 2048 51.4 us (141 MB;
// in place 56.0), to 64 28.5; 300 to 200 8.7 us. Loops are kept short: unrolled ones cost the small cases half as much again, in
// instruction fetches.
#include "kv4.cuh"
#include "smem_limit.h"

namespace bitnet {
namespace {

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int BINS = 2048;
constexpr int MAX_CLUSTER = 16;
constexpr int MAX_RANKS = 20480;  // that a block keeps (80 KB, two blocks an SM); longer runs are read again each time

// Masses as whole numbers in the same order; a NaN above all, both zeros alike. Tokens that are kept in any case (the
// first and the last ones) rank above every mass.
constexpr uint32_t SURE = 0xffffffffu;
__device__ __forceinline__ uint32_t rank_of(float x) {
  if (x != x) return SURE - 1;
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
// The mass of token j. One whose page is not in the pool has none, whatever pass asks (and no other page's, which another
// cluster may be moving): all passes have to find the same tokens.
__device__ __forceinline__ float mass_of(const Kv4& c, const Kv4Evict& e, int b, int h, int j, bool* bad) {
  const int id = c.page_table[(int64_t)b * c.max_pages + j / kKvPage];
  if (id < 0 || id >= c.n_pages) {
    *bad = true;
    return 0.0f;
  }
  return e.mass[((int64_t)id * c.kv_heads + h) * kKvPage + j % kKvPage];
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint4 ld_cluster_u32x4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

template <int D>
__global__ void __launch_bounds__(THREADS, 2) kv4_evict_kernel(Kv4 c, Kv4Evict e, int32_t* kept, int cap, int cluster, int ranks_kept,
                                                               bool write_len) {
  extern __shared__ uint32_t ranks[];
  __shared__ __align__(16) uint32_t bins[BINS];
  __shared__ uint32_t warp_sum[WARPS];
  __shared__ int2 warp_count[WARPS], block_count;
  __shared__ uint32_t found[2], totals[MAX_CLUSTER];
  constexpr int BLK = (int)kv4_block_bytes(D);
  const int unit = blockIdx.x / cluster, me = cluster > 1 ? (int)cluster_ctarank() : 0, b = unit / c.kv_heads, h = unit - b * c.kv_heads;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const auto sync_all = [&]() {
    if (cluster > 1) cluster_sync_all();
    else __syncthreads();
  };
  const Sizes s = sizes_of(c, e, b);
  if (h == 0 && me == 0 && tid == 0 && write_len) e.new_len[b] = s.len < 0 ? c.kv_len[b] : s.keeps;
  const bool cut = s.len > e.limit;
  if (s.len < 0 || (e.into && s.keeps > e.into_pages * kKvPage)) {  // the second: not one that is cut
    if (tid == 0) record_device_error(kErrRange);
    return;
  }
  if (!cut && !e.into) return;
  bool bad = false;
  int32_t* list = kept + (int64_t)unit * cap;
  if (cut) {
    const int lo = e.sinks, hi = s.len - e.recent;  // the tokens that masses decide over
    uint32_t want = (uint32_t)e.budget;
    // this block's run of tokens, and its warps'
    const int per = ((s.len + cluster * WARPS - 1) / (cluster * WARPS) + 31) / 32 * 32;
    const int run0 = (int)min((int64_t)me * WARPS * per, (int64_t)s.len), j0 = (int)min(run0 + (int64_t)warp * per, (int64_t)s.len), j1 = (int)min(j0 + (int64_t)per, (int64_t)s.len);
    const bool keep = WARPS * per <= ranks_kept;
    const auto ranked = [&](int j, float mass) { return j < lo || j >= hi ? SURE : rank_of(mass); };
    // tokens without any mass may be many: a warp's are counted together, not one after another in one bin
    const uint32_t zero = 0x80000000u;
    uint32_t zeros = 0;
    if (keep) {
      for (int i = tid; i < BINS; i += THREADS) bins[i] = 0;
      __syncthreads();
      // the page ids of the next 32 pages, one a lane, then the masses of 8 x 32 tokens at a time
      for (int p0 = j0 / kKvPage; p0 * kKvPage < j1; p0 += 32) {
        int id = -1;  // not in the pool: its tokens have no mass
        if ((int64_t)(p0 + lane) * kKvPage < j1) {
          id = c.page_table[(int64_t)b * c.max_pages + p0 + lane];
          if (id < 0 || id >= c.n_pages) bad = true, id = -1;
        }
#pragma unroll 1
        for (int q = 0; q < 32 && (p0 + q) * kKvPage < j1; q += 4) {
          float m[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int from = __shfl_sync(0xffffffffu, id, q + (i >> 1)), j = (p0 + q) * kKvPage + i * 32 + lane;
            m[i] = 0.0f;
            if (j >= j0 && j < j1 && from >= 0) m[i] = e.mass[((int64_t)from * c.kv_heads + h) * kKvPage + (i & 1) * 32 + lane];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int j = (p0 + q) * kKvPage + i * 32 + lane;
            if (j < j0 || j >= j1) continue;
            const uint32_t r = ranked(j, m[i]);
            ranks[j - run0] = r;
            // the first pass's count
            if (r == zero) ++zeros;
            else atomicAdd(&bins[r >> 21], 1u);
          }
        }
      }
      __syncwarp();
    }
    // of token j of this warp's run; 0, which is no rank, past its end
    const auto rank = [&](int j) {
      if (j >= j1) return 0u;
      return keep ? ranks[j - run0] : ranked(j, mass_of(c, e, b, h, j, &bad));
    };
    uint32_t least = 0, mask = 0;  // the digits found so far
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 10 : 11;
      if (pass > 0 || !keep) {
        zeros = 0;
        for (int i = tid; i < BINS; i += THREADS) bins[i] = 0;
        __syncthreads();
        const uint32_t digits = (1u << width) - 1;
#pragma unroll 1
        for (int j = j0 + lane; j - lane < j1; j += 4 * 32) {
          uint32_t r[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) r[i] = rank(j + 32 * i);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (r[i] == zero) ++zeros;
            else if ((r[i] & mask) == least && r[i]) atomicAdd(&bins[(r[i] >> shift) & digits], 1u);
          }
        }
      }
      zeros = __reduce_add_sync(0xffffffffu, zeros);
      if (lane == 0 && zeros && (zero & mask) == least) atomicAdd(&bins[(zero >> shift) & ((1u << width) - 1)], zeros);
      sync_all();
      // The digit from which on `want` tokens are counted, from above. Each block adds up its slice of the bins over the
      // cluster, a slice's total goes to all blocks, and the block whose slice has the digit tells it.
      const int slice = BINS / cluster, mine = BINS - slice * (me + 1);  // the first block has the highest bins
      uint32_t n[4] = {0, 0, 0, 0}, sum = 0;
      if (4 * tid < slice) {
        const uint32_t at = smem_u32(&bins[mine + slice - 4 - 4 * tid]);
#pragma unroll 1
        for (int k = 0; k < cluster; k += 4) {
          uint4 v[4] = {};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (k + i < cluster) v[i] = ld_cluster_u32x4(map_to_rank(at, k + i));
#pragma unroll
          for (int i = 0; i < 4; ++i) n[0] += v[i].w, n[1] += v[i].z, n[2] += v[i].y, n[3] += v[i].x;
        }
        sum = n[0] + n[1] + n[2] + n[3];
      }
      const uint32_t own = sum;
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      if (lane == 31) warp_sum[warp] = sum;
      __syncthreads();
      uint32_t above = sum - own, total = 0;  // tokens of higher digits than this thread's in the slice; of the slice
      {
        const uint32_t x = lane < WARPS ? warp_sum[lane] : 0;
        total = __reduce_add_sync(0xffffffffu, x);
        above += __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
      }
      if (cluster > 1) {
        if (tid < cluster) st_cluster_u32(map_to_rank(smem_u32(&totals[me]), tid), total);
        cluster_sync_all();
        for (int k = 0; k < me; ++k) above += totals[k];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (4 * tid < slice && above < want && want <= above + n[i]) {
          const uint32_t digit = mine + slice - 1 - 4 * tid - i, rest = want - above;
#pragma unroll 1
          for (int k = 0; k < cluster; ++k) {
            st_cluster_u32(map_to_rank(smem_u32(&found[0]), k), digit);
            st_cluster_u32(map_to_rank(smem_u32(&found[1]), k), rest);
          }
        }
        above += n[i];
      }
      sync_all();  // `found` is written, and no block reads another's bins any more
      least |= found[0] << shift;
      mask |= ((1u << width) - 1) << shift;
      want = found[1];
    }
    // `want` is now how many of the tokens at `least` are kept. Each warp counts those of its run, then lists them.
    // (their ballots stay in the bins' place, where they fit)
    const bool fits = WARPS * per <= BINS / 2 * 32;
    uint2* masks = reinterpret_cast<uint2*>(bins) + warp * (per / 32);
    int sures = 0, levels = 0;
#pragma unroll 1
    for (int j = j0 + lane; j - lane < j1; j += 4 * 32) {
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = rank(j + 32 * i);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t sm = __ballot_sync(0xffffffffu, r[i] > least), lm = __ballot_sync(0xffffffffu, r[i] == least);
        sures += __popc(sm);
        levels += __popc(lm);
        if (fits && lane == 0 && j + 32 * i < j1) masks[(j - j0) / 32 + i] = make_uint2(sm, lm);
      }
    }
    if (lane == 0) warp_count[warp] = make_int2(sures, levels);
    __syncthreads();
    {
      const int2 x = lane < warp ? warp_count[lane] : make_int2(0, 0);
      sures = (int)__reduce_add_sync(0xffffffffu, (unsigned)x.x), levels = (int)__reduce_add_sync(0xffffffffu, (unsigned)x.y);
    }
    if (tid == THREADS - 1) block_count = make_int2(sures + warp_count[warp].x, levels + warp_count[warp].y);
    sync_all();
    const uint32_t count_at = smem_u32(&block_count);
    for (int k = 0; k < me; ++k) {
      sures += (int)ld_cluster_u32(map_to_rank(count_at, k));
      levels += (int)ld_cluster_u32(map_to_rank(count_at, k) + 4);
    }
    for (int j = j0 + lane; j - lane < j1; j += 32) {
      uint2 m;
      if (fits) {
        m = masks[(j - j0) / 32];
      } else {
        const uint32_t r = rank(j);
        m = make_uint2(__ballot_sync(0xffffffffu, r > least), __ballot_sync(0xffffffffu, r == least));
      }
      const uint32_t below = (1u << lane) - 1;
      const int ls = levels + __popc(m.y & below), at = sures + __popc(m.x & below) + min(ls, (int)want);
      const bool sure = m.x >> lane & 1, level = m.y >> lane & 1;
      if ((sure || (level && ls < (int)want)) && at < cap) list[at] = j;
      sures += __popc(m.x);
      levels += __popc(m.y);
    }
    sync_all();  // the list is written, and no block reads another's counts any more
  }

  // ---- the kept tokens move (all unsigned 32-bit: their indexes are below 2^30, and so are a pool's blocks)
  // A warp takes RUN tokens at a time. Lane l finds where token l comes from and goes to, and moves its parameters and mass; the
  // lanes move the rows in 16-byte pieces, LANES a token, by what that lane hands them.
  constexpr uint32_t LANES = D / 16, PIECES = LANES / 2, EACH = 32 / LANES, BATCH = 4, RUN = EACH * BATCH, PAGE = kKvPage;
  const uint32_t part = lane % LANES, keeps = s.keeps, piece = part % PIECES * 16;
  const bool is_key = part < PIECES;
  const uint32_t* from = reinterpret_cast<const uint32_t*>(c.page_table + (int64_t)b * c.max_pages);
  const uint32_t* to = e.into ? reinterpret_cast<const uint32_t*>(e.into + (int64_t)b * e.into_pages) : from;
  const uint32_t n_pages = c.n_pages, heads = c.kv_heads;
  // where the lane's 16 bytes and the parameters of place t lie in a head's block of a page
  const auto rho = [](uint32_t t) { return (t & ~7u) | (t & 3u) << 1 | (t >> 2 & 1u); };
  const auto data_at = [&](uint32_t t) { return (is_key ? rho(t) : PAGE + t) * (D / 2) + piece; };
  constexpr uint32_t NONE = 0xffffffffu;
  uint32_t from_blk = 0, to_blk = 0, places = NONE;  // the token's places in its pages, the old one and the new one << 8; NONE: it stays
  const auto look = [&](uint32_t first) {
    const uint32_t r = first + lane;
    places = NONE;
    if (lane >= RUN || r >= keeps) return;
    const uint32_t j = cut ? (uint32_t)list[r] : r;
    // A list is whole where the masses stood still. Where a table names pages of a sequence that another cluster moves they may
    // not have, and what the workspace held before is no token.
    if (j >= (uint32_t)s.len) {
      bad = true;
      return;
    }
    if (!e.into && j == r) return;
    const uint32_t x = from[j / PAGE], y = to[r / PAGE];
    if (x >= n_pages || y >= n_pages) {
      bad = true;
      return;
    }
    from_blk = x * heads + h, to_blk = y * heads + h, places = j % PAGE | (r % PAGE) << 8;
  };
  const uint32_t chunk = cluster * WARPS * RUN, mine = (me * WARPS + warp) * RUN;
  look(mine);
#pragma unroll 1
  for (uint32_t first = 0; first < keeps; first += chunk) {
    uint4 data[BATCH];
    uint2 par = make_uint2(0, 0);
    float mass = 0.0f;
    const uint32_t low = places & 63, high = places >> 8 & 63, blk = to_blk, both = places;
    if (both != NONE) {
      par = *reinterpret_cast<const uint2*>(c.pages + (uint64_t)from_blk * BLK + PAGE * D + rho(low) * 8);
      mass = e.mass[(uint64_t)from_blk * PAGE + low];
    }
#pragma unroll
    for (uint32_t i = 0; i < BATCH; ++i) {
      const uint32_t x = __shfl_sync(0xffffffffu, from_blk, i * EACH + lane / LANES), p = __shfl_sync(0xffffffffu, both, i * EACH + lane / LANES);
      if (p != NONE) data[i] = *reinterpret_cast<const uint4*>(c.pages + (uint64_t)x * BLK + data_at(p & 63));
    }
    look(first + chunk + mine);  // the next ones' places while these are on their way
    if (!e.into) sync_all();
#pragma unroll
    for (uint32_t i = 0; i < BATCH; ++i) {
      const uint32_t y = __shfl_sync(0xffffffffu, blk, i * EACH + lane / LANES), p = __shfl_sync(0xffffffffu, both, i * EACH + lane / LANES);
      // the halves of a wide value row are exchanged where bit 1 of the place is set
      const uint32_t turn = D == 128 && !is_key ? ((p ^ p >> 8) & 2) << 4 : 0;
      if (p != NONE) *reinterpret_cast<uint4*>(c.pages + (uint64_t)y * BLK + (data_at(p >> 8 & 63) ^ turn)) = data[i];
    }
    if (both != NONE) {
      *reinterpret_cast<uint2*>(c.pages + (uint64_t)blk * BLK + PAGE * D + rho(high) * 8) = par;
      e.mass[(uint64_t)blk * PAGE + high] = mass;
    }
    if (!e.into) sync_all();
  }
  if (bad) record_device_error(kErrRange);
}

// New lengths over the old ones, once no cluster reads them any more.
__global__ void kv4_evict_lengths(Kv4 c, Kv4Evict e) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= c.batch) return;
  const Sizes s = sizes_of(c, e, b);
  e.new_len[b] = s.len < 0 ? c.kv_len[b] : s.keeps;
}

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }
int cap_of(const Kv4& c, int budget) { return budget < c.max_kv ? budget : c.max_kv; }

template <int D>
cudaError_t launch(const cudaLaunchConfig_t& cfg, const Kv4& c, const Kv4Evict& e, int32_t* kept, int cluster, int ranks, bool write_len) {
  static std::atomic<uint64_t> configured{0};
  if (cudaError_t err = allow_smem(configured, kv4_evict_kernel<D>, MAX_RANKS * 4, true)) return err;
  return cudaLaunchKernelEx(&cfg, kv4_evict_kernel<D>, c, e, kept, cap_of(c, e.budget), cluster, ranks, write_len);
}

}  // namespace

int64_t kv4_evict_ws_bytes(const Kv4& c, int budget) { return align256((int64_t)c.batch * c.kv_heads * cap_of(c, budget) * 4); }
cudaError_t launch_kv4_evict(const Kv4& c, int dim, const Kv4Evict& e, void* ws, int num_sms, cudaStream_t st) {
  const int64_t units = (int64_t)c.batch * c.kv_heads;
  // blocks of a cluster: as many as two an SM leave room for, each with some thousand tokens (48 sequences of 501 to
  // 16001 tokens x 5 heads to 2048: a block each 59 us, two each, in two waves, 68; to 64: 31 and 39.7)
  int cluster = 1;
  while (cluster < 8 && units * cluster * 2 <= num_sms * 2 && c.max_kv > cluster * 1024) cluster *= 2;
  // sixteen: 131007 tokens x 5 heads 25.2 us, eight 33.4; 16000 tokens 17.6 and 15.4
  if (cluster == 8 && units * MAX_CLUSTER <= num_sms * 2 && c.max_kv > 48 * 1024) cluster = MAX_CLUSTER;
  int64_t per = ((c.max_kv + cluster * WARPS - 1) / (cluster * WARPS) + 31) / 32 * 32;
  const int ranks = (int)(per * WARPS < MAX_RANKS ? per * WARPS : MAX_RANKS);
  const bool over = e.new_len == c.kv_len;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(units * cluster));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = ranks * 4;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int32_t* kept = static_cast<int32_t*>(ws);
  if (cudaError_t err = dim == 128 ? launch<128>(cfg, c, e, kept, cluster, ranks, e.new_len && !over)
                                   : launch<64>(cfg, c, e, kept, cluster, ranks, e.new_len && !over))
    return err;
  if (!over) return cudaSuccess;
  kv4_evict_lengths<<<(c.batch + 127) / 128, 128, 0, st>>>(c, e);
  return cudaGetLastError();
}

cudaError_t read_clear_device_error_kv4_evict(int* value) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, g_device_error, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
}

}  // namespace bitnet
