// mxfp4_gemm.cu -- D = A * B^T of two MXFP4 operands (dense, contiguous and
// masked m-grouped), FP32 accumulation, BF16 out.
//
// D[i, j] = sum_g 2^(sa[i,g] + sb[j,g]) sum_{k < 32} A[i, 32g+k] B[j, 32g+k]:
// the tensor cores apply both scales (tcgen05.mma kind::mxf4 with one UE8M0
// scale per row and 32 K elements), so a tile accumulates in TMEM over all of
// K and is rounded once.
//
// The tile is D transposed: 128 rows of B (output columns) on the TMEM lanes
// and up to 256 rows of A (tokens) on its columns.  The MMA's N then follows
// the number of tokens (16 .. 256 in steps of 16, chosen per tile on the
// device), so a decode batch or an expert with few tokens does not pay for
// 128, and every weight row is read once per 256 tokens.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstdlib>

#include "dg.h"
#include "host.h"
#include "internal.h"
#include "mxfp4.cuh"
#include "ptx.cuh"

namespace dg {

namespace {

enum MxSched : int { kMxDense = 0, kMxContiguous = 1, kMxMasked = 2 };

constexpr int kTileN = 128;      // rows of B per tile (TMEM lanes)
constexpr int kMaxTokens = 256;  // rows of A per tile (TMEM columns)
constexpr int kStageK = 256;     // K elements per stage: a 128-byte row of codes
constexpr int kMmaK = 64;        // K elements per MMA
constexpr int kStageWords = kStageK / 128;
constexpr int kThreads = 384;    // producer, MMA, two set-up warps, 8 epilogue warps
constexpr int kEpiWarps = 8;
constexpr int kFirstEpiWarp = 4;
constexpr int kTurnBytes = 1024;  // per epilogue warp: 16 tokens x 32 columns of D
constexpr int kMaxStages = 12;
constexpr uint32_t kBBytes = kTileN * kStageK / 2;              // 16 KB
constexpr uint32_t kSfBBytes = kStageWords * kMxBlockBytes;     // one row block
// TMEM: two accumulators of up to 128 columns (one of 256), then scale slots of
// 32 columns: B's words at 0 and 4, A's word w of row block b at 8 + 8 w + 4 b.
constexpr uint32_t kSfSlotCols = 32;
constexpr int kSfSlots = 4;
// A CTA takes a whole SM (512 columns) or, with tiles of up to 64 tokens, half
// of one (256 columns, half the registers and shared memory): smem_apart.
constexpr int kHalfTokens = 64;

struct MxParams {
  uint16_t *d;
  const int32_t *m_indices, *masked_m;
  int *status;
  int rows;          // M, M_total or M_max
  int n, k;
  int groups;
  int tok_tile;      // tokens per tile: 16, 32, 64, 128 or 256
  int tok_tiles;     // dense: ceil(rows / tok_tile)
  int n_tiles;       // ceil(n / 128), for the pair form ceil(n / 256)
  int stages;
  int splits;        // CTAs of a cluster that split a tile's K (dense; 1: none)
  int starve;        // test hook: the stage whose loads CTA 0 leaves out (-1: none)
};

struct Tile {
  int n0;            // first row of B
  int tok0, tokens;  // first row of A within its slab, rows that are stored
  int slab, group;   // A / D slab (expert for masked), expert of B
  int k_begin, k_end;  // stages
};

// Contiguous layout: the expert of a 128-row block from its 128 indices, four per
// lane: the first non-negative one, -1 when the block is all padding or that
// index is out of range.  A block that mixes experts or names one out of range
// records DG_ERR_DEVICE_DATA (only the rows of the first expert are computed).
// Whole warp.
__device__ __forceinline__ int block_expert(const MxParams &p, const int4 &v) {
  const int vals[4] = {v.x, v.y, v.z, v.w};
  int first = -1;
#pragma unroll
  for (int i = 3; i >= 0; --i)
    if (vals[i] >= 0) first = vals[i];
  const unsigned any = __ballot_sync(0xffffffffu, first >= 0);
  if (!any) return -1;
  const int e = __shfl_sync(0xffffffffu, first, __ffs(any) - 1);
  bool bad = e >= p.groups;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= vals[i] >= 0 && vals[i] != e;
  if (bad) record_status(p.status, DG_ERR_DEVICE_DATA);
  return e < p.groups ? e : -1;
}

// What a launch's roles read about its tiles, in shared memory.  Masked:
// prefix[e] = tiles of the experts before e.  Contiguous: count tiles, tile i
// of list[i] = 2 * block + (two blocks ? 1 : 0), expert[block].
struct Tables {
  const int *prefix;
  const int *list, *expert;
  int count;
};

// Calls f(tile) for every tile of this CTA (or CTA pair), in order; f returns
// false to stop.  Every role walks the same list.
template <int SCHED, bool PAIR, typename F>
__device__ __forceinline__ void for_each_tile(const MxParams &p, const Tables &tab, F f) {
  const int k_stages = (p.k + kStageK - 1) / kStageK;
  Tile t;
  t.k_begin = 0;
  t.k_end = k_stages;
  t.slab = t.group = 0;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  if constexpr (SCHED == kMxMasked) {
    const int units = tab.prefix[p.groups];
    constexpr int kCtas = PAIR ? 2 : 1;
    for (int u = blockIdx.x / kCtas; u < units; u += gridDim.x / kCtas) {
      int lo = 0, hi = p.groups - 1;  // largest e with prefix[e] <= u
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.prefix[mid] <= u) lo = mid; else hi = mid - 1;
      }
      const int r = u - tab.prefix[lo];
      const int tt = (tab.prefix[lo + 1] - tab.prefix[lo]) / p.n_tiles;  // token tiles
      const int nt = r / tt;
      const int m = min(__ldcg(p.masked_m + lo), p.rows);
      t.slab = t.group = lo;
      t.n0 = (PAIR ? 2 * nt + rank : nt) * kTileN;
      t.tok0 = (r - nt * tt) * p.tok_tile;
      t.tokens = min(p.tok_tile, m - t.tok0);
      if (!f(t)) return;
    }
  } else {
    // a cluster's CTAs share a tile: a pair its rows of B, a split its K
    const int cluster = PAIR ? 2 : p.splits;
    const int tok_tiles = SCHED == kMxContiguous ? tab.count : p.tok_tiles;
    const int units = tok_tiles * p.n_tiles;
    const int first = blockIdx.x / cluster, stride = gridDim.x / cluster;
    if (SCHED == kMxDense && !PAIR && p.splits > 1) {
      const int s = blockIdx.x - first * p.splits;
      t.k_begin = k_stages * s / p.splits;
      t.k_end = k_stages * (s + 1) / p.splits;
    }
    // Dense: where half the CTAs or fewer would get a tile of 256 tokens in the last
    // wave, each gets one of 128 instead (4096 x 7168 x 16384, 448 tiles for 74
    // pairs: 160.4 -> 156.6 us; 2048 x 7168 x 4096: 26.8 -> 25.4 us).
    const int rest = units % stride;
    const bool halve =
        SCHED == kMxDense && p.tok_tile == 256 && units > stride && 2 * rest <= stride;
    const int whole = halve ? units - rest : units;
    for (int v = first; v < (halve ? units + rest : units); v += stride) {
      const int u = v < whole ? v : whole + (v - whole) / 2;
      // groups of kRaster token tiles, all rows of B for one after another:
      // a wave's tiles share both operands in L2
      constexpr int kRaster = 16;
      const int grp = u / (kRaster * p.n_tiles);
      const int in = u - grp * kRaster * p.n_tiles;
      const int across = min(kRaster, tok_tiles - grp * kRaster);
      const int nt = in / across;
      const int tt = grp * kRaster + in - nt * across;
      t.n0 = (PAIR ? 2 * nt + rank : nt) * kTileN;
      if constexpr (SCHED == kMxContiguous) {
        const int entry = tab.list[tt];
        t.tok0 = (entry >> 1) * 128;
        t.tokens = entry & 1 ? 256 : 128;
        t.group = tab.expert[entry >> 1];
      } else {
        t.tok0 = tt * p.tok_tile;
        t.tokens = min(p.tok_tile, p.rows - t.tok0);
        if (v >= whole) {
          if ((v - whole) % 2) {
            t.tok0 += 128;
            t.tokens -= 128;
            if (t.tokens <= 0) continue;
          } else {
            t.tokens = min(t.tokens, 128);
          }
        }
      }
      if (!f(t)) return;
    }
  }
}

// A role's place in the stage ring: the slot, and the parity of its use there.
// (Carried along: a division per stage by the run-time number of stages cost
// each role about a hundred cycles.)
struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void advance(int stages) {
    if (++slot == stages) {
      slot = 0;
      parity ^= 1;
    }
  }
};

// Rows of A (MMA columns) of a tile: a multiple of 16, of 32 for the pair,
// whose CTAs hold half of them each.
template <bool PAIR>
__device__ __forceinline__ int mma_n(const Tile &t) {
  return PAIR ? (t.tokens + 31) / 32 * 32 : (t.tokens + 15) / 16 * 16;
}

// PAIR: two CTAs of a cluster compute a tile of 256 rows of B with
// cta_group::2 MMAs issued by rank 0; each loads its 128 rows of B and half of
// the tokens, so an SM moves 32 KB per stage instead of 48 KB.
template <int SCHED, bool PAIR, bool HALF>
__global__ void __launch_bounds__(kThreads, HALF ? 2 : 1)
mxfp4_gemm_kernel(const __grid_constant__ CUtensorMap tmap_a,
                  const __grid_constant__ CUtensorMap tmap_b,
                  const __grid_constant__ CUtensorMap tmap_sfa,
                  const __grid_constant__ CUtensorMap tmap_sfb, const MxParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bars[2 * kMaxStages + 5];
  __shared__ uint32_t s_tmem;
  __shared__ int s_count;
  __shared__ volatile int s_abort;
  // 1024-byte aligned base of the stage ring (the 128-byte swizzle's atom)
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t a_bytes =
      static_cast<uint32_t>(PAIR ? p.tok_tile / 2 : p.tok_tile) * (kStageK / 2);
  const uint32_t stage_bytes = kBBytes + a_bytes;
  const uint32_t sf_stage = kSfBBytes + (p.tok_tile > 128 ? 2 * kSfBBytes : kSfBBytes);
  const uint32_t sf_base = base + static_cast<uint32_t>(p.stages) * stage_bytes;
  // the epilogue's turning area, then the tables
  const uint32_t turn_base = sf_base + static_cast<uint32_t>(p.stages) * sf_stage;
  int *s_table = reinterpret_cast<int *>(smem_raw + (turn_base - raw) + kEpiWarps * kTurnBytes);
  const uint32_t bars = smem_u32(s_bars);
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (kMaxStages + s); };
  auto tfull_bar = [&](int b) { return bars + 8u * (2 * kMaxStages + b); };
  auto tempty_bar = [&](int b) { return bars + 8u * (2 * kMaxStages + 2 + b); };
  const uint32_t drain_bar = bars + 8u * (2 * kMaxStages + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0;
  const int nbuf = p.tok_tile > 128 ? 1 : 2;
  const uint32_t buf_cols = HALF ? 64u : p.tok_tile > 128 ? 256u : 128u;
  constexpr uint32_t tmem_cols = HALF ? 256u : 512u, sf_col = tmem_cols / 2;
  constexpr int kChunks = (HALF ? kHalfTokens : kMaxTokens) / 32;  // 32 tokens each
  const int a_blocks = (p.rows + 127) / 128, b_blocks = (p.n + 127) / 128;  // per slab / expert
  const int blocks = p.rows / 128;  // contiguous
  Tables tab;
  tab.prefix = s_table;
  tab.expert = s_table;
  tab.list = s_table + blocks;
  tab.count = 0;

  grid_launch_dependents();
  if (SCHED == kMxDense && warp == 3) {
    // B's boxes of the first stages are asked into L2 before the set-up and the
    // dependency wait (a prefetch only fills L2, which the previous kernel's
    // writes go through as well), so HBM works meanwhile
    for_each_tile<SCHED, PAIR>(p, tab, [&](const Tile &t) {
      if (t.n0 < p.n && lane < p.stages && t.k_begin + lane < t.k_end)
        tma_prefetch_3d(&tmap_b, (t.k_begin + lane) * (kStageK / 2), t.n0, t.group);
      return false;
    });
  }
  if (threadIdx.x == 0) {
    prefetch_tmap(&tmap_a);
    prefetch_tmap(&tmap_b);
    prefetch_tmap(&tmap_sfa);
    prefetch_tmap(&tmap_sfb);
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), PAIR ? 2 * kEpiWarps : kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    s_abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(&s_tmem), tmem_cols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&s_tmem), tmem_cols);
      tmem_relinquish();
    }
  }
  grid_dependency_wait();
  if constexpr (SCHED == kMxMasked) {
    if (warp == 2) {
      int running = 0;
      for (int e0 = 0; e0 < p.groups; e0 += 32) {
        const int e = e0 + lane;
        int v = 0;
        if (e < p.groups) {
          const int m = __ldcg(p.masked_m + e);
          if (m < 0 || m > p.rows) record_status(p.status, DG_ERR_DEVICE_DATA);
          v = (min(max(m, 0), p.rows) + p.tok_tile - 1) / p.tok_tile * p.n_tiles;
        }
        int incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += t;
        }
        if (e < p.groups) s_table[e] = running + incl - v;
        running += __shfl_sync(0xffffffffu, incl, 31);
      }
      if (lane == 0) s_table[p.groups] = running;
    }
  }
  if constexpr (SCHED == kMxContiguous) {
    // (one round trip for four blocks of each warp)
    constexpr int kWarps = kThreads / 32, kAtOnce = 4;
    const int4 *idx = reinterpret_cast<const int4 *>(p.m_indices);
    for (int b0 = warp; b0 < blocks; b0 += kWarps * kAtOnce) {
      int4 v[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int b = b0 + j * kWarps;
        if (b < blocks) v[j] = __ldcg(idx + static_cast<int64_t>(b) * 32 + lane);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int b = b0 + j * kWarps;
        if (b < blocks) {
          const int e = block_expert(p, v[j]);
          if (lane == 0) s_table[b] = e;
        }
      }
    }
    __syncthreads();
    if (warp == 2) {
      // a tile starts at every other block (every one, for tiles of 128
      // tokens) of a run of blocks of one expert
      int *list = s_table + blocks;
      int count = 0, run = 0, before = -1;  // blocks of the run that ends before b0
      for (int b0 = 0; b0 < blocks; b0 += 32) {
        const int b = b0 + lane;
        const int e = b < blocks ? s_table[b] : -1;
        const int prev = __shfl_up_sync(0xffffffffu, e, 1);
        const bool starts = e != (lane ? prev : before);
        const unsigned st = __ballot_sync(0xffffffffu, starts);
        // the block's position in its run
        const unsigned upto = st & (0xFFFFFFFFu >> (31 - lane));
        const int pos = upto ? lane - (31 - __clz(upto)) : run + lane;
        const bool two = p.tok_tile > 128;
        const bool head = e >= 0 && (!two || pos % 2 == 0);
        const unsigned heads = __ballot_sync(0xffffffffu, head);
        if (head)
          list[count + __popc(heads & ((1u << lane) - 1u))] =
              2 * b + (two && b + 1 < blocks && s_table[b + 1] == e ? 1 : 0);
        count += __popc(heads);
        run = __shfl_sync(0xffffffffu, pos, 31) + 1;
        before = __shfl_sync(0xffffffffu, e, 31);
      }
      if (lane == 0) s_count = count;
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // both CTAs' barriers exist before any remote use
  tc_fence_after();
  if constexpr (SCHED == kMxContiguous) tab.count = s_count;
  const uint32_t tmem = s_tmem;
  volatile int *abort = &s_abort;

  if (warp == 0) {
    // ================================================================ producer
    // (one elected thread runs the role, and one the MMA issuer's: 0.21 us a stage
    // of a small tile; waiting with the whole warp and electing per stage, 0.24)
    if (elect_one()) {
      Ring ring;
      int issued = 0;  // stages, counted up to the ring's length
      int it = 0;
      const int starve = blockIdx.x == 0 ? p.starve : -1;
      for_each_tile<SCHED, PAIR>(p, tab, [&](const Tile &t) {
        const int b_block = t.group * b_blocks + t.n0 / 128;
        const int a_block = t.slab * a_blocks + t.tok0 / 128;
        const int a_row = t.tok0 + static_cast<int>(rank) * (mma_n<PAIR>(t) / 2);
        for (int ks = t.k_begin; ks < t.k_end; ++ks) {
          const int s = ring.slot;
          if (!mbar_wait(empty_bar(s), ring.parity ^ 1, abort, p.status)) return false;
          if (it != starve) {
            const uint32_t sb = base + static_cast<uint32_t>(s) * stage_bytes;
            const uint32_t sf = sf_base + static_cast<uint32_t>(s) * sf_stage;
            const int kc = ks * (kStageK / 2), wc = ks * kStageWords;
            if constexpr (PAIR) {
              // both CTAs' boxes complete on rank 0's barrier
              const uint32_t fb = mapa_shared(full_bar(s), 0);
              if (rank == 0) mbar_arrive_expect_tx(full_bar(s), 2 * (stage_bytes + sf_stage));
              tma_load_3d_pair(sb, &tmap_b, fb, kc, t.n0, t.group);
              tma_load_3d_pair(sb + kBBytes, &tmap_a, fb, kc, a_row, t.slab);
              tma_load_3d_pair(sf, &tmap_sfb, fb, 0, wc, b_block);
              tma_load_3d_pair(sf + kSfBBytes, &tmap_sfa, fb, 0, wc, a_block);
            } else {
              mbar_arrive_expect_tx(full_bar(s), stage_bytes + sf_stage);
              tma_load_3d(sb, &tmap_b, full_bar(s), kc, t.n0, t.group);
              tma_load_3d(sb + kBBytes, &tmap_a, full_bar(s), kc, a_row, t.slab);
              tma_load_3d(sf, &tmap_sfb, full_bar(s), 0, wc, b_block);
              tma_load_3d(sf + kSfBBytes, &tmap_sfa, full_bar(s), 0, wc, a_block);
            }
          }
          ring.advance(p.stages);
          if (issued < p.stages) ++issued;
          ++it;
        }
        return true;
      });
      // no copy may still be writing this CTA's shared memory when it exits: wait
      // for the last use of every stage that was armed (pair: rank 0's barriers
      // count both CTAs' bytes, and rank 1 leaves after rank 0 at the cluster
      // barrier)
      volatile int never = 0;
      if (rank == 0)
        for (int i = 0; i < issued; ++i) {
          // slots before the ring's place were used with its parity, the others
          // with the one before (a stage that was left out has no copies)
          if (starve < 0 || it <= starve || i != starve % p.stages)
            mbar_wait(full_bar(i), i < ring.slot ? ring.parity : ring.parity ^ 1, &never, p.status);
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    if (rank == 0 && elect_one()) {
      const int k_mmas = (p.k + kMmaK - 1) / kMmaK;
      const uint64_t bdesc0 = smem_desc_k128_sw128(base);
      const uint64_t sfdesc0 = smem_desc_rows16(sf_base);
      Ring ring;
      uint32_t it = 0;
      int tile_i = 0;
      for_each_tile<SCHED, PAIR>(p, tab, [&](const Tile &t) {
        const int buf = nbuf == 2 ? tile_i & 1 : 0;
        const uint32_t use = nbuf == 2 ? tile_i >> 1 : tile_i;
        if (!mbar_wait(tempty_bar(buf), (use & 1) ^ 1, abort, p.status)) return false;
        const uint32_t d = tmem + static_cast<uint32_t>(buf) * buf_cols;
        const uint32_t idesc = idesc_mxf4(PAIR ? 2 * kTileN : kTileN, mma_n<PAIR>(t));
        const bool second = t.tokens > 128;
        for (int ks = t.k_begin; ks < t.k_end; ++ks, ++it) {
          const int s = ring.slot;
          if (!mbar_wait(full_bar(s), ring.parity, abort, p.status)) return false;
          tc_fence_after();
          // (descriptor addresses are in units of 16 bytes, below 2^14: no carry)
          const uint64_t bdesc = bdesc0 + static_cast<uint32_t>(s) * (stage_bytes >> 4);
          const uint64_t adesc = bdesc + (kBBytes >> 4);
          const uint64_t sfdesc = sfdesc0 + static_cast<uint32_t>(s) * (sf_stage >> 4);
          const uint32_t slot = tmem + sf_col + (it % kSfSlots) * kSfSlotCols;
          const uint32_t first = ks == t.k_begin ? 1u : 0u;
          auto cp = [&](uint32_t to, uint32_t from) {
            if constexpr (PAIR) tmem_cp_32x128b_x4_pair(slot + to, sfdesc + (from >> 4));
            else tmem_cp_32x128b_x4(slot + to, sfdesc + (from >> 4));
          };
          auto scales = [&](int w) {
            cp(4 * w, kMxBlockBytes * w);
            cp(8 + 8 * w, kSfBBytes + kMxBlockBytes * w);
            if (second) cp(12 + 8 * w, 2 * kSfBBytes + kMxBlockBytes * w);
          };
          auto mma = [&](int j) {
            const uint32_t sfb = slot + 4 * (j >> 1), sfa = slot + 8 + 8 * (j >> 1);
            const uint32_t more = j > 0 ? 1u : first ^ 1u;
            if constexpr (PAIR)
              umma_mxf4_pair(d, bdesc + 2 * j, adesc + 2 * j, idesc, sfb, sfa, 2u * (j & 1),
                             more);
            else
              umma_mxf4(d, bdesc + 2 * j, adesc + 2 * j, idesc, sfb, sfa, 2u * (j & 1), more);
          };
          const int mmas = k_mmas - ks * (kStageK / kMmaK);
          scales(0);
          if (mmas >= kStageK / kMmaK) {
            scales(1);
#pragma unroll
            for (int j = 0; j < kStageK / kMmaK; ++j) mma(j);
          } else {
            // the last stage of a K off the 256 grid
            if (mmas > 2) scales(1);
            mma(0);
            if (mmas > 1) mma(1);
            if (mmas > 2) mma(2);
          }
          if constexpr (PAIR) {
            umma_commit_pair_both(empty_bar(s));
            if (ks + 1 == t.k_end) umma_commit_pair_both(tfull_bar(buf));
          } else {
            umma_commit(empty_bar(s));
            if (ks + 1 == t.k_end) umma_commit(tfull_bar(buf));
          }
          ring.advance(p.stages);
        }
        ++tile_i;
        return true;
      });
      // every MMA issued above completes before TMEM is freed
      if constexpr (PAIR) umma_commit_pair_own(drain_bar);
      else umma_commit(drain_bar);
      volatile int never = 0;
      mbar_wait(drain_bar, 0, &never, p.status);
    }
    __syncwarp();
  } else if (warp >= kFirstEpiWarp) {
    // ================================================================ epilogue
    // Warp w reads lanes 32 (w mod 4) .. and every other 16-column chunk; the
    // accumulator is handed back once it is in registers, as BF16 (a tile of 256
    // tokens has the only accumulator, so the MMAs of the next one wait).
    const int half = (warp - kFirstEpiWarp) >> 2;
    const int quarter = warp & 3;
    const uint32_t turn = turn_base + (warp - kFirstEpiWarp) * kTurnBytes;
    int tile_i = 0;
    for_each_tile<SCHED, PAIR>(p, tab, [&](const Tile &t) {
      const int buf = nbuf == 2 ? tile_i & 1 : 0;
      const uint32_t use = nbuf == 2 ? tile_i >> 1 : tile_i;
      // rows that are stored: bit l of live[i] is token 32 i + l
      uint32_t live[kChunks];
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        bool v = 32 * i + lane < t.tokens;
        if (SCHED == kMxContiguous && v)
          v = __ldcg(p.m_indices + t.tok0 + 32 * i + lane) == t.group;
        live[i] = __ballot_sync(0xffffffffu, v);
      }
      if (!mbar_wait(tfull_bar(buf), use & 1, abort, p.status)) return false;
      tc_fence_after();
      const uint32_t acc = tmem + static_cast<uint32_t>(buf) * buf_cols +
                           (static_cast<uint32_t>(quarter * 32) << 16);
      if (SCHED == kMxDense && !PAIR && p.splits > 1) {
        // this CTA's FP32 partial goes to its stage ring (drained: all its
        // MMAs are done), [token][128]
        for (int c0 = half * 16; c0 < t.tokens; c0 += 32) {
          uint32_t r[16];
          tmem_ld<16>(acc + c0, r);
          tmem_wait_ld();
          reg_barrier<16>(r);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(
                             base + static_cast<uint32_t>((c0 + i) * kTileN + quarter * 32 + lane) *
                                        4u),
                         "r"(r[i])
                         : "memory");
        }
        ++tile_i;
        return true;
      }
      // out[i]: 16 tokens of the warp's 32 columns, as 8 x 8 matrices: [4 h + m],
      // h the 16-lane half, m = 2 (token / 8) + (column / 8) within it
      uint32_t out[kChunks][8];
#pragma unroll
      for (int i = 0; i < kChunks; i += 2) {
        uint32_t r[2][16];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int c0 = (2 * (i + q) + half) * 16;
          if (c0 < t.tokens) {
            tmem_ld_16x256_x2(acc + c0, r[q]);
            tmem_ld_16x256_x2(acc + c0 + (16u << 16), r[q] + 8);
          }
        }
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          reg_barrier<16>(r[q]);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(r[q][2 * j]),
                                                           __uint_as_float(r[q][2 * j + 1]));
            out[i + q][j] = *reinterpret_cast<const uint32_t *>(&v);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster(mapa_shared(tempty_bar(buf), 0));
        else mbar_arrive(tempty_bar(buf));
      }
      // Turned to [token][column] in the warp's own kilobyte of shared memory (16
      // tokens of 64 bytes; 16-byte piece c of token t at c ^ (t / 2 mod 4):
      // no bank conflicts), then stored as 64 bytes of eight rows at a time.
      const uint32_t st_tok = (lane & 7) + 8 * (lane >> 4);
      const uint32_t st_piece = (lane >> 3) & 1;
      const uint32_t st_row = turn + st_tok * 64;
      const uint32_t st_a = st_row + ((st_piece ^ ((st_tok >> 1) & 3)) << 4);
      const uint32_t st_b = st_row + (((st_piece + 2) ^ ((st_tok >> 1) & 3)) << 4);
      const int tok = lane >> 2;
      const uint32_t ld = turn + tok * 64 + (((lane & 3) ^ ((tok >> 1) & 3)) << 4);
      const int n = t.n0 + quarter * 32 + 8 * (lane & 3);
      uint16_t *dst = p.d + (static_cast<int64_t>(t.slab) * p.rows + t.tok0 + tok) * p.n + n;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c0 = (2 * i + half) * 16;
        if (c0 < t.tokens) {
          stmatrix_x4_trans(st_a, out[i][0], out[i][1], out[i][2], out[i][3]);
          stmatrix_x4_trans(st_b, out[i][4], out[i][5], out[i][6], out[i][7]);
          __syncwarp();
          const uint4 v0 = ld_shared_v4(ld), v1 = ld_shared_v4(ld + 512);
          const uint32_t bits = live[i] >> (16 * half + tok);
          uint16_t *row = dst + static_cast<int64_t>(c0) * p.n;
          if (n < p.n) {  // (N % 8 == 0: eight columns or none)
            if (bits & 1u) *reinterpret_cast<uint4 *>(row) = v0;
            if (bits & 256u) *reinterpret_cast<uint4 *>(row + static_cast<int64_t>(8) * p.n) = v1;
          }
          __syncwarp();
        }
      }
      ++tile_i;
      return true;
    });
  }

  if (SCHED == kMxDense && !PAIR && p.splits > 1) {
    // ============================================================ K reduction
    // The CTAs of the cluster hold the partials of one tile: each sums a share
    // of the tokens over the cluster's shared memory, in split order.
    __syncwarp();
    cluster_sync();
    const int share = static_cast<int>(cluster_ctarank());
    for_each_tile<SCHED, PAIR>(p, tab, [&](const Tile &t) {
      const int n = t.n0 + 4 * lane;
      for (int c = share + p.splits * warp; c < t.tokens; c += p.splits * (kThreads / 32)) {
        const uint32_t at = base + static_cast<uint32_t>(c * kTileN + 4 * lane) * 4u;
        float4 v[8];
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s < p.splits) v[s] = ld_shared_cluster_v4(mapa_shared(at, s));
        float4 sum = v[0];
#pragma unroll
        for (int s = 1; s < 8; ++s)
          if (s < p.splits) {
            sum.x += v[s].x; sum.y += v[s].y; sum.z += v[s].z; sum.w += v[s].w;
          }
        if (n < p.n) {
          const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x, sum.y);
          const __nv_bfloat162 hi = __floats2bfloat162_rn(sum.z, sum.w);
          *reinterpret_cast<uint2 *>(p.d + static_cast<int64_t>(t.tok0 + c) * p.n + n) =
              make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                         *reinterpret_cast<const uint32_t *>(&hi));
        }
      }
      return true;
    });
    cluster_sync();  // no CTA leaves while its partial is being read
  }

  tc_fence_before();
  __syncthreads();
  // pair: neither CTA leaves or frees TMEM while rank 0's MMAs may still read
  // its shared memory or write its TMEM (rank 0 drained them)
  if constexpr (PAIR) cluster_sync();
  tc_fence_after();
  if (warp == 1) {
    if constexpr (PAIR) tmem_dealloc_pair(tmem, tmem_cols);
    else tmem_dealloc(tmem, tmem_cols);
  }
}

// ------------------------------------------------------------------ host side
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Codes [slabs][rows][K/2] as bytes, a box of `box` rows of 128 bytes.
int make_tmap(CUtensorMap *m, const void *ptr, int64_t k, int64_t rows, int64_t slabs, int box) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return DG_ERR_CUDA;
  const cuuint64_t bytes = static_cast<cuuint64_t>(k / 2);
  const cuuint64_t dims[3] = {bytes, static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(slabs)};
  const cuuint64_t strides[2] = {bytes, bytes * static_cast<cuuint64_t>(rows)};
  const cuuint32_t ext[3] = {kStageK / 2, static_cast<cuuint32_t>(box), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(ptr), dims,
                         strides, ext, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DG_OK : DG_ERR_CUDA;
}

// Scale words of `blocks` 128-row blocks: [blocks][ceil(K/128)][128], a box of two
// K words of `box` row blocks (zeros past K; past the last block, never used).
int make_scale_tmap(CUtensorMap *m, const void *ptr, int64_t k, int64_t blocks, int box) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return DG_ERR_CUDA;
  const cuuint64_t words = static_cast<cuuint64_t>(mx_k_words(k));
  const cuuint64_t dims[3] = {kMxBlockWords, words, static_cast<cuuint64_t>(blocks)};
  const cuuint64_t strides[2] = {kMxBlockBytes, kMxBlockBytes * words};
  const cuuint32_t ext[3] = {kMxBlockWords, kStageWords, static_cast<cuuint32_t>(box)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_INT32, 3, const_cast<void *>(ptr), dims,
                         strides, ext, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DG_OK : DG_ERR_CUDA;
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

constexpr int kMaxDevices = 64;
// Rows of one launch of the contiguous product (its table of blocks lives in
// shared memory, eight bytes a block); more rows are several launches.
constexpr int kMaxContiguousRows = 2048 * 128;

// Shared memory that an SM has for all its CTAs; 0 on a CUDA error.
int smem_per_sm(int dev) {
  static std::atomic<int> known[kMaxDevices];  // (any thread may be the first)
  int v = known[dev].load(std::memory_order_relaxed);
  if (v == 0 && cuda_status(cudaDeviceGetAttribute(
                    &v, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev)) == DG_OK)
    known[dev].store(v, std::memory_order_relaxed);
  return v;
}

template <int SCHED, bool PAIR, bool HALF>
int configure(int dev, int smem) {
  static std::atomic<bool> done[kMaxDevices];
  if (done[dev].load(std::memory_order_relaxed)) return DG_OK;
  const int rc = cuda_status(cudaFuncSetAttribute(
      mxfp4_gemm_kernel<SCHED, PAIR, HALF>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  if (!rc) done[dev].store(true, std::memory_order_relaxed);
  return rc;
}

// Most clusters of `size` CTAs (2 .. 8) with all shared memory that are resident
// at once; asked once per device, kernel and size.
template <int SCHED, bool PAIR, bool HALF>
int clusters_fit(int dev, int size, int smem) {
  static std::atomic<int> fit[kMaxDevices][9];  // count + 1; 0 = not asked yet
  int known = fit[dev][size].load(std::memory_order_relaxed);
  if (known == 0) {
    cudaLaunchConfig_t q = {};
    q.gridDim = dim3(size);
    q.blockDim = dim3(kThreads);
    q.dynamicSmemBytes = smem;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeClusterDimension;
    a[0].val.clusterDim.x = size;
    a[0].val.clusterDim.y = 1;
    a[0].val.clusterDim.z = 1;
    q.attrs = a;
    q.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, mxfp4_gemm_kernel<SCHED, PAIR, HALF>, &q) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    known = n + 1;
    fit[dev][size].store(known, std::memory_order_relaxed);
  }
  return known - 1;
}

// CTAs of a cluster that split K, for `tiles` tiles of one wave.
template <int SCHED, bool HALF>
int pick_splits(int dev, int tiles, int k_stages, int sms, int smem) {
  int s = sms / tiles;
  if (s > 8) s = 8;
  if (s > k_stages) s = k_stages;
  while (s > 1 && clusters_fit<SCHED, false, HALF>(dev, s, smem) < tiles) --s;
  return s;
}

// Whether tiles of `tok_tile` tokens run two CTAs per SM: where there are more
// than SMs, so that the tiles past one per SM start at once and each CTA's
// latencies overlap the other's (64 x 24576 x 4096, 192 tiles: 13.1 against
// 19.9 us; but 148 tiles, 64 x 18944 x 16384: 33.9 against 28.8 us, for half
// the stages each).  A cap on the SMs keeps one.
bool half_sms(int tok_tile, int64_t tiles, int sms, int all_sms) {
  return tok_tile <= kHalfTokens && tiles > sms && sms == all_sms;
}

struct Operands {
  const uint8_t *a, *b;
  const int32_t *sfa, *sfb;
};

// Dynamic shared memory that a CTA may take: all of an SM's, or half -- less the
// barriers (static) and, twice in a half, the kilobyte that the system takes per CTA.
struct Smem {
  int full, half, per_sm;
};
constexpr Smem smem_limits(int optin, int per_sm) {
  return {optin - 512, per_sm / 2 - 1024 - 512, per_sm};
}

// The ring of a form: the stages that fit beside `tables` bytes of tables, and
// the shared memory that they make.
struct RingSize {
  int stages, smem;
};
constexpr RingSize ring_of(bool pair, bool half, int tok_tile, int tables, const Smem &max) {
  const int stage = static_cast<int>(kBBytes) + (pair ? tok_tile / 2 : tok_tile) * (kStageK / 2) +
                    static_cast<int>(kSfBBytes) * (tok_tile > 128 ? 3 : 2);
  const int besides = 1024 + kEpiWarps * kTurnBytes + tables;
  const int fit = ((half ? max.half : max.full) - besides) / stage;
  const int stages = fit < kMaxStages ? fit : kMaxStages;
  return {stages, besides + stages * stage};
}

// TMEM is taken before the dependency wait, and the next launch starts before that:
// if CTAs that together want more than an SM's 512 columns met on one, one that
// waits for its columns (in a cluster, with its peers waiting for it) and one that
// holds them and waits for the launch before it would wait for each other.
// Shared memory keeps them apart: a whole SM's CTA takes more than two thirds of
// it, half an SM's more than a third, so a second one beside the first or a third
// beside two halves does not fit.  (The library's FP8 kernels, with 144 KB and more,
// do not fit beside the smallest half either, 87 KB of 228.)
constexpr bool smem_apart(bool half, int smem, int per_sm) {
  return 3 * smem > (half ? 1 : 2) * per_sm;
}
constexpr int kMaxGroups = 1024;  // of the masked form
constexpr bool all_apart(const Smem &max) {
  for (int tables : {0, (kMaxGroups + 1) * 4, kMaxContiguousRows / 128 * 8})
    for (int t = 16; t <= kMaxTokens; t *= 2) {
      if (!smem_apart(false, ring_of(false, false, t, tables, max).smem, max.per_sm)) return false;
      if (t == kMaxTokens &&
          !smem_apart(false, ring_of(true, false, t, tables, max).smem, max.per_sm))
        return false;
      if (t <= kHalfTokens && tables <= (kMaxGroups + 1) * 4 &&
          !smem_apart(true, ring_of(false, true, t, tables, max).smem, max.per_sm))
        return false;
    }
  return true;
}
static_assert(all_apart(smem_limits(227 * 1024, 228 * 1024)), "a B200's SM");

// Fills in the shapes that follow from p and launches `grid` CTAs.
template <int SCHED, bool PAIR, bool HALF>
int launch_form(const Operands &o, MxParams p, int grid, const Smem &max, cudaStream_t stream) {
  const int a_rows = PAIR ? p.tok_tile / 2 : p.tok_tile;
  const int tables = SCHED == kMxMasked       ? (p.groups + 1) * 4
                     : SCHED == kMxContiguous ? p.rows / 128 * 8
                                              : 0;
  const RingSize ring = ring_of(PAIR, HALF, p.tok_tile, tables, max);
  if (!smem_apart(HALF, ring.smem, max.per_sm)) return DG_ERR_UNSUPPORTED_ARCH;
  p.stages = ring.stages;
  CUtensorMap ta, tb, tsa, tsb;
  const int slabs = SCHED == kMxMasked ? p.groups : 1;
  int rc = make_tmap(&ta, o.a, p.k, p.rows, slabs, a_rows);
  if (!rc) rc = make_tmap(&tb, o.b, p.k, p.n, p.groups, kTileN);
  if (!rc) rc = make_scale_tmap(&tsa, o.sfa, p.k, slabs * mx_row_blocks(p.rows),
                                p.tok_tile > 128 ? 2 : 1);
  if (!rc) rc = make_scale_tmap(&tsb, o.sfb, p.k, p.groups * mx_row_blocks(p.n), 1);
  if (rc) return rc;
  const int cluster = PAIR ? 2 : p.splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = ring.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0] = pdl_attribute();
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cuda_status(
      cudaLaunchKernelEx(&cfg, mxfp4_gemm_kernel<SCHED, PAIR, HALF>, ta, tb, tsa, tsb, p));
}

template <int SCHED>
int launch_forms(const Operands &o, MxParams p, cudaStream_t stream) {
  const DeviceInfo *info = device_info();
  int dev = 0;
  if (!info || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
    return DG_ERR_CUDA;
  const int sms = effective_num_sms();
  const int per_sm = smem_per_sm(dev);
  if (per_sm <= 0) return DG_ERR_CUDA;
  const Smem max = smem_limits(info->max_smem_optin, per_sm);
  int rc = configure<SCHED, false, false>(dev, max.full);
  if (!rc && SCHED != kMxContiguous)
    rc = configure<SCHED, false, SCHED != kMxContiguous>(dev, max.half);
  if (!rc) rc = configure<SCHED, true, false>(dev, max.full);
  if (rc) return rc;
  const int k_stages = ceil_div(p.k, kStageK);
  // tokens per tile: the smallest power of two that holds all of them
  p.tok_tile = 16;
  while (p.tok_tile < kMaxTokens && p.tok_tile < p.rows) p.tok_tile *= 2;
  p.splits = 1;
  p.n_tiles = ceil_div(p.n, kTileN);
  // pairs that are resident at once
  int pairs = clusters_fit<SCHED, true, false>(dev, 2, max.full);
  if (pairs > sms / 2) pairs = sms / 2;
  if constexpr (SCHED == kMxMasked) {
    if (half_sms(p.tok_tile, static_cast<int64_t>(p.groups) * p.n_tiles, sms, info->num_sms))
      return launch_form<SCHED, false, true>(o, p, 2 * sms, max, stream);
    // (pairs: 32 experts of 7168 x 2048, 200 tokens each 66 -> 61 us, 8 of 4096 x
    // 7168, 700 tokens each 77 -> 67 us; no faster with tiles of 128 tokens)
    if (p.tok_tile == 256 && pairs > 0) {
      p.n_tiles = ceil_div(p.n, 2 * kTileN);
      return launch_form<SCHED, true, false>(o, p, 2 * pairs, max, stream);
    }
    return launch_form<SCHED, false, false>(o, p, sms, max, stream);
  } else {
    if constexpr (SCHED == kMxContiguous) {
      const int most = p.rows / 128;  // blocks that may hold an expert's rows
      const int n_pairs = ceil_div(p.n, 2 * kTileN);
      // Pairs for two tiles or more each, counted as if no run of an expert's blocks had
      // an odd length.  13 experts of 1448 x 1056: 42 to 72 tiles 10.1 to 11.9 us single
      // against 11.5 to 13.6, 156 tiles 19.9 against 17.5; 32 of 2048 x 1024: 128 tiles
      // 11.6 against 12.2, 184 tiles 15.2 against 16.9, 240 tiles 18.5 against 18.3; 8 of
      // 4096 x 7168: 64 tiles 25.9 against 26.3, 112 tiles 40.6 against 30.9, 528 tiles
      // 159 against 103.
      if (pairs > 0 && ceil_div(most, 2) * n_pairs >= 2 * pairs) {
        p.tok_tile = 256;
        p.n_tiles = n_pairs;
        return launch_form<SCHED, true, false>(o, p, 2 * pairs, max, stream);
      }
      // few tiles: 128 tokens each, for more of them
      p.tok_tile = 128;
      const int tiles = most * p.n_tiles;
      return launch_form<SCHED, false, false>(o, p, tiles < sms ? tiles : sms, max, stream);
    } else {
      p.tok_tiles = ceil_div(p.rows, p.tok_tile);
      const int tiles = p.tok_tiles * p.n_tiles;
      if (half_sms(p.tok_tile, tiles, sms, info->num_sms))
        return launch_form<SCHED, false, true>(o, p, tiles < 2 * sms ? tiles : 2 * sms, max,
                                               stream);
      // Pairs where there is a tile of 256 x 256 for each: 768 x 7168 x 7168, 84 of
      // them for 74 pairs, 21.6 us against 25.4 with single CTAs, 2048 x 7168 x 7168 39.8
      // against 45.8.  With fewer, single CTAs (K split where there are SMs for it) are
      // as often the faster: 2112 x 7168, 9 / 18 / 36 tiles, 14.3 / 12.5 / 13.6 us against
      // 17.4 / 14.3 / 13.9 with pairs; 4096 x 2048, 16 / 32 / 64 tiles, 9.9 / 10.2 / 8.1
      // against 8.0 / 8.4 / 9.3; 512 x 7168 x 7168, 56 tiles, 16.4 against 15.4.
      const int pair_tiles = p.tok_tiles * ceil_div(p.n, 2 * kTileN);
      if (p.tok_tile == 256 && pairs > 0 && pair_tiles >= pairs) {
        p.n_tiles = ceil_div(p.n, 2 * kTileN);
        return launch_form<SCHED, true, false>(o, p, 2 * pairs, max, stream);
      }
      if (tiles < sms) {
        p.splits = pick_splits<SCHED, false>(dev, tiles, k_stages, sms, max.full);
        return launch_form<SCHED, false, false>(o, p, tiles * p.splits, max, stream);
      }
      return launch_form<SCHED, false, false>(o, p, sms, max, stream);
    }
  }
}

// The limit of this file's bounded waits, from here on in stream order.
int set_wait_limit(unsigned long long limit_ns, cudaStream_t stream) {
  return cuda_status(cudaMemcpyToSymbolAsync(g_wait_limit_ns, &limit_ns, sizeof(limit_ns), 0,
                                             cudaMemcpyHostToDevice, stream));
}

// With the abort path's test knobs (gemm.cu's, both unset in normal use):
// DG_TEST_STARVE_LOAD=i makes CTA 0's producer leave out the loads of its i-th stage,
// DG_TEST_WAIT_LIMIT_US=t lowers the waits' limit to t microseconds for this call.
template <int SCHED>
int launch_mxfp4(const Operands &o, MxParams p, cudaStream_t stream) {
  const char *starve = getenv("DG_TEST_STARVE_LOAD"), *limit = getenv("DG_TEST_WAIT_LIMIT_US");
  p.starve = starve ? atoi(starve) : -1;
  if (!limit) return launch_forms<SCHED>(o, p, stream);
  int rc = set_wait_limit(strtoull(limit, nullptr, 10) * 1000ull, stream);
  if (rc) return rc;
  rc = launch_forms<SCHED>(o, p, stream);
  const int rc2 = set_wait_limit(kWaitLimitNs, stream);
  return rc ? rc : rc2;
}

int check_gemm(const void *A, const void *sfa, const void *B, const void *sfb, const void *D,
               int64_t rows, int64_t N, int64_t K, int64_t slabs, int64_t groups) {
  if (rows < 0 || N <= 0 || K <= 0 || K % kMxGroup != 0 || N % 8 != 0) return DG_ERR_INVALID_ARG;
  if (rows == 0) return DG_OK;
  if (!A || !sfa || !B || !sfb || !D) return DG_ERR_INVALID_ARG;
  // tile and block counts, and a grid's step past them, are 31-bit
  constexpr int64_t kMost = 0x7FFFF000;
  if (rows > kMost || N > kMost || K > kMost) return DG_ERR_INVALID_ARG;
  if (mx_row_blocks(rows) * mx_row_blocks(N) * slabs > kMost ||
      mx_row_blocks(N) * groups > kMost || mx_row_blocks(rows) * slabs > kMost)
    return DG_ERR_INVALID_ARG;
  if (!aligned16(A) || !aligned16(sfa) || !aligned16(B) || !aligned16(sfb) || !aligned16(D))
    return DG_ERR_ALIGNMENT;
  return DG_OK;
}

int usable_device() {
  const DeviceInfo *d = device_info();
  if (!d) return DG_ERR_CUDA;
  return d->ok ? DG_OK : DG_ERR_UNSUPPORTED_ARCH;
}

MxParams make_params(void *D, int64_t rows, int64_t N, int64_t K, int groups) {
  MxParams p{};
  p.d = static_cast<uint16_t *>(D);
  p.status = device_info()->status;
  p.rows = static_cast<int>(rows);
  p.n = static_cast<int>(N);
  p.k = static_cast<int>(K);
  p.groups = groups;
  return p;
}

}  // namespace

}  // namespace dg

extern "C" int dg_mxfp4_gemm_nt(const uint8_t *A, const int32_t *sfa, const uint8_t *B,
                                const int32_t *sfb, void *D, int64_t M, int64_t N, int64_t K,
                                dg_stream_t stream) {
  using namespace dg;
  int rc = check_gemm(A, sfa, B, sfb, D, M, N, K, 1, 1);
  if (rc) return rc;
  if (M == 0) return DG_OK;
  rc = usable_device();
  if (rc) return rc;
  return launch_mxfp4<kMxDense>({A, B, sfa, sfb}, make_params(D, M, N, K, 1),
                                reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int dg_m_grouped_mxfp4_gemm_nt_contiguous(const uint8_t *A, const int32_t *sfa,
                                                     const uint8_t *B, const int32_t *sfb,
                                                     void *D, const int32_t *m_indices,
                                                     int64_t M_total, int64_t N, int64_t K, int G,
                                                     dg_stream_t stream) {
  using namespace dg;
  if (G < 1) return DG_ERR_INVALID_ARG;
  int rc = check_gemm(A, sfa, B, sfb, D, M_total, N, K, 1, G);
  if (rc) return rc;
  if (M_total % 128 != 0) return DG_ERR_INVALID_ARG;
  if (M_total == 0) return DG_OK;
  if (!m_indices) return DG_ERR_INVALID_ARG;
  if (!aligned16(m_indices)) return DG_ERR_ALIGNMENT;
  rc = usable_device();
  if (rc) return rc;
  for (int64_t row = 0; row < M_total; row += kMaxContiguousRows) {
    const int64_t rows =
        M_total - row < kMaxContiguousRows ? M_total - row : kMaxContiguousRows;
    MxParams p = make_params(static_cast<uint16_t *>(D) + row * N, rows, N, K, G);
    p.m_indices = m_indices + row;
    rc = launch_mxfp4<kMxContiguous>(
        {A + row * (K / 2), B, sfa + row / 128 * mx_k_words(K) * kMxBlockWords, sfb}, p,
        reinterpret_cast<cudaStream_t>(stream));
    if (rc) return rc;
  }
  return DG_OK;
}

extern "C" int dg_m_grouped_mxfp4_gemm_nt_masked(const uint8_t *A, const int32_t *sfa,
                                                 const uint8_t *B, const int32_t *sfb, void *D,
                                                 const int32_t *masked_m, int G, int64_t M_max,
                                                 int64_t N, int64_t K, dg_stream_t stream) {
  using namespace dg;
  if (G < 1 || G > kMaxGroups || M_max < 1) return DG_ERR_INVALID_ARG;
  int rc = check_gemm(A, sfa, B, sfb, D, M_max, N, K, G, G);
  if (rc) return rc;
  if (!masked_m) return DG_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(masked_m) % 4 != 0) return DG_ERR_ALIGNMENT;
  rc = usable_device();
  if (rc) return rc;
  MxParams p = make_params(D, M_max, N, K, G);
  p.masked_m = masked_m;
  return launch_mxfp4<kMxMasked>({A, B, sfa, sfb}, p, reinterpret_cast<cudaStream_t>(stream));
}
