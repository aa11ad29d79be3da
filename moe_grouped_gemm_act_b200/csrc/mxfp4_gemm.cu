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

#include <cstdint>

#include "dg.h"
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
constexpr int kMaxStages = 12;
constexpr uint32_t kBBytes = kTileN * kStageK / 2;              // 16 KB
constexpr uint32_t kSfBBytes = kStageWords * kMxBlockBytes;     // one row block
// TMEM: 256 accumulator columns (two tiles of up to 128 tokens, or one of
// 256), then scale slots of 32 columns: B's words at 0 and 4, A's word w of
// row block b at 8 + 8 w + 4 b.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfCol = 256, kSfSlotCols = 32;
constexpr int kSfSlots = 4;
// Shared memory of a launch stays above half an SM's, so that no two CTAs
// that each want all TMEM columns sit on one SM (a CTA of a cluster waiting
// for TMEM there while its peers wait for it could deadlock two launches).
constexpr int kMinSmem = 120 * 1024;

struct MxParams {
  const uint8_t *sfa, *sfb;  // scale blocks
  uint16_t *d;
  const int32_t *m_indices, *masked_m;
  int *status;
  int rows;          // M, M_total or M_max
  int n, k;
  int groups;
  int tok_tile;      // tokens per tile: 16, 32, 64, 128 or 256
  int tok_tiles;     // dense, contiguous: ceil(rows / tok_tile)
  int n_tiles;       // ceil(n / 128)
  int stages;
  int splits;        // CTAs of a cluster that split a tile's K (dense; 1: none)
};

struct Tile {
  int n0;            // first row of B
  int tok0, tokens;  // first row of A within its slab, rows that are stored
  int slab, group;   // A / D slab (expert for masked), expert of B
  int k_begin, k_end;  // stages
};

// The expert of a 128-row block of the contiguous layout, -1 when it is all
// padding.  Whole warp.  With `check`, a block that mixes experts or holds an
// index >= groups records DG_ERR_DEVICE_DATA (the rows of other experts are
// then not written, and nothing is computed for an index out of range).
__device__ __forceinline__ int block_expert(const MxParams &p, int block, bool check) {
  const int lane = threadIdx.x & 31;
  const int4 v = __ldg(reinterpret_cast<const int4 *>(p.m_indices) + block * 32 + lane);
  const int vals[4] = {v.x, v.y, v.z, v.w};
  int first = -1;
#pragma unroll
  for (int i = 3; i >= 0; --i)
    if (vals[i] >= 0) first = vals[i];
  const unsigned any = __ballot_sync(0xffffffffu, first >= 0);
  if (!any) return -1;
  const int e = __shfl_sync(0xffffffffu, first, __ffs(any) - 1);
  if (check) {
    bool bad = e >= p.groups;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= vals[i] >= 0 && vals[i] != e;
    if (__any_sync(0xffffffffu, bad) && lane == 0) record_status(p.status, DG_ERR_DEVICE_DATA);
  }
  return e < p.groups ? e : -1;
}

// Calls f(tile) for every tile of this CTA, in order; f returns false to stop.
// Every role walks the same list.  Whole warp.
template <int SCHED, typename F>
__device__ __forceinline__ void for_each_tile(const MxParams &p, const int *s_prefix, bool check,
                                              F f) {
  const int k_stages = (p.k + kStageK - 1) / kStageK;
  Tile t;
  t.k_begin = 0;
  t.k_end = k_stages;
  t.slab = t.group = 0;
  if constexpr (SCHED == kMxMasked) {
    const int units = s_prefix[p.groups];
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      int lo = 0, hi = p.groups - 1;  // largest e with prefix[e] <= u
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_prefix[mid] <= u) lo = mid; else hi = mid - 1;
      }
      const int r = u - s_prefix[lo];
      const int tt = (s_prefix[lo + 1] - s_prefix[lo]) / p.n_tiles;  // token tiles
      const int nt = r / tt;
      const int m = min(__ldg(p.masked_m + lo), p.rows);
      t.slab = t.group = lo;
      t.n0 = nt * kTileN;
      t.tok0 = (r - nt * tt) * p.tok_tile;
      t.tokens = min(p.tok_tile, m - t.tok0);
      if (!f(t)) return;
    }
  } else {
    const int units = p.tok_tiles * p.n_tiles;
    // (a cluster's CTAs share one tile, each a part of its K)
    const int first = blockIdx.x / p.splits, stride = gridDim.x / p.splits;
    if (SCHED == kMxDense && p.splits > 1) {
      const int s = blockIdx.x - first * p.splits;
      t.k_begin = k_stages * s / p.splits;
      t.k_end = k_stages * (s + 1) / p.splits;
    }
    for (int u = first; u < units; u += stride) {
      // groups of kRaster token tiles, all rows of B for one after another:
      // a wave's tiles share both operands in L2
      constexpr int kRaster = 16;
      const int grp = u / (kRaster * p.n_tiles);
      const int in = u - grp * kRaster * p.n_tiles;
      const int width = min(kRaster, p.tok_tiles - grp * kRaster);
      const int nt = in / width;
      t.n0 = nt * kTileN;
      t.tok0 = (grp * kRaster + in - nt * width) * p.tok_tile;
      t.tokens = min(p.tok_tile, p.rows - t.tok0);
      if constexpr (SCHED == kMxContiguous) {
        // one tile for all blocks of one expert next to each other
        const int blocks = t.tokens / 128, tok0 = t.tok0;
        int e = block_expert(p, tok0 / 128, check);
        int from = 0;
        for (int b = 1; b <= blocks; ++b) {
          const int next = b < blocks ? block_expert(p, tok0 / 128 + b, check) : -1;
          if (next == e && b < blocks) continue;
          if (e >= 0) {
            t.tok0 = tok0 + from * 128;
            t.tokens = (b - from) * 128;
            t.group = e;
            if (!f(t)) return;
          }
          from = b;
          e = next;
        }
      } else {
        if (!f(t)) return;
      }
    }
  }
}

template <int SCHED>
__global__ void __launch_bounds__(kThreads, 1)
mxfp4_gemm_kernel(const __grid_constant__ CUtensorMap tmap_a,
                  const __grid_constant__ CUtensorMap tmap_b, const MxParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bars[2 * kMaxStages + 5];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  // 1024-byte aligned base of the stage ring (the 128-byte swizzle's atom)
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t a_bytes = static_cast<uint32_t>(p.tok_tile) * (kStageK / 2);
  const uint32_t stage_bytes = kBBytes + a_bytes;
  const uint32_t sf_a_bytes = p.tok_tile > 128 ? 2 * kSfBBytes : kSfBBytes;
  const uint32_t sf_stage = kSfBBytes + sf_a_bytes;
  const uint32_t sf_base = base + static_cast<uint32_t>(p.stages) * stage_bytes;
  int *s_prefix = reinterpret_cast<int *>(
      smem_raw + (sf_base - raw) + static_cast<uint32_t>(p.stages) * sf_stage);
  const uint32_t bars = smem_u32(s_bars);
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (kMaxStages + s); };
  auto tfull_bar = [&](int b) { return bars + 8u * (2 * kMaxStages + b); };
  auto tempty_bar = [&](int b) { return bars + 8u * (2 * kMaxStages + 2 + b); };
  const uint32_t drain_bar = bars + 8u * (2 * kMaxStages + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nbuf = p.tok_tile > 128 ? 1 : 2;
  const uint32_t buf_cols = p.tok_tile > 128 ? 256u : 128u;
  const int k_words = (p.k + 127) / 128;
  const int a_blocks = (p.rows + 127) / 128, b_blocks = (p.n + 127) / 128;  // per slab / expert

  grid_launch_dependents();
  if (threadIdx.x == 0) {
    prefetch_tmap(&tmap_a);
    prefetch_tmap(&tmap_b);
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    s_abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s_tmem), kTmemCols);
    tmem_relinquish();
  }
  grid_dependency_wait();
  if (SCHED == kMxMasked && warp == 2) {
    // prefix[e]: tiles of the experts before e
    int running = 0;
    for (int e0 = 0; e0 < p.groups; e0 += 32) {
      const int e = e0 + lane;
      int v = 0;
      if (e < p.groups) {
        const int m = __ldg(p.masked_m + e);
        if (m < 0 || m > p.rows) record_status(p.status, DG_ERR_DEVICE_DATA);
        v = (min(max(m, 0), p.rows) + p.tok_tile - 1) / p.tok_tile * p.n_tiles;
      }
      int incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      if (e < p.groups) s_prefix[e] = running + incl - v;
      running += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) s_prefix[p.groups] = running;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int *abort = &s_abort;

  if (warp == 0) {
    // ================================================================ producer
    int it = 0;
    for_each_tile<SCHED>(p, s_prefix, true, [&](const Tile &t) {
      const int b_block = t.group * b_blocks + t.n0 / 128;
      const int a_block = t.slab * a_blocks + t.tok0 / 128;
      // the second row block of a 256-token tile, where the tile reaches it
      const bool second = t.tokens > 128;
      for (int ks = t.k_begin; ks < t.k_end; ++ks, ++it) {
        const int s = it % p.stages;
        if (!mbar_wait(empty_bar(s), ((it / p.stages) & 1) ^ 1, abort, p.status)) return false;
        if (elect_one()) {
          const uint32_t sb = base + static_cast<uint32_t>(s) * stage_bytes;
          const uint32_t sf = sf_base + static_cast<uint32_t>(s) * sf_stage;
          const uint32_t sf_bytes = static_cast<uint32_t>(
              min(kStageWords, k_words - ks * kStageWords)) * kMxBlockBytes;
          mbar_arrive_expect_tx(full_bar(s), stage_bytes + sf_bytes * (second ? 3u : 2u));
          tma_load_3d(sb, &tmap_b, full_bar(s), ks * (kStageK / 2), t.n0, t.group);
          tma_load_3d(sb + kBBytes, &tmap_a, full_bar(s), ks * (kStageK / 2), t.tok0, t.slab);
          const int64_t w = static_cast<int64_t>(ks) * kStageWords;
          bulk_load(sf, p.sfb + (static_cast<int64_t>(b_block) * k_words + w) * kMxBlockBytes,
                    sf_bytes, full_bar(s));
          const uint8_t *src =
              p.sfa + (static_cast<int64_t>(a_block) * k_words + w) * kMxBlockBytes;
          bulk_load(sf + kSfBBytes, src, sf_bytes, full_bar(s));
          if (second)
            bulk_load(sf + 2 * kSfBBytes, src + static_cast<int64_t>(k_words) * kMxBlockBytes,
                      sf_bytes, full_bar(s));
        }
        __syncwarp();
      }
      return true;
    });
    // no copy may still be writing this CTA's shared memory when it exits
    volatile int never = 0;
    for (int i = max(0, it - p.stages); i < it; ++i)
      mbar_wait(full_bar(i % p.stages), (i / p.stages) & 1, &never, p.status);
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    const int k_mmas = (p.k + kMmaK - 1) / kMmaK;
    int it = 0, tile_i = 0;
    for_each_tile<SCHED>(p, s_prefix, false, [&](const Tile &t) {
      const int buf = tile_i % nbuf;
      if (!mbar_wait(tempty_bar(buf), ((tile_i / nbuf) & 1) ^ 1, abort, p.status)) return false;
      const uint32_t d = tmem + static_cast<uint32_t>(buf) * buf_cols;
      const uint32_t idesc = idesc_mxf4(kTileN, (t.tokens + 15) / 16 * 16);
      for (int ks = t.k_begin; ks < t.k_end; ++ks, ++it) {
        const int s = it % p.stages;
        if (!mbar_wait(full_bar(s), (it / p.stages) & 1, abort, p.status)) return false;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t sb = base + static_cast<uint32_t>(s) * stage_bytes;
          const uint32_t sf = sf_base + static_cast<uint32_t>(s) * sf_stage;
          const uint32_t slot = tmem + kSfCol + static_cast<uint32_t>(it % kSfSlots) * kSfSlotCols;
          const int words = min(kStageWords, k_words - ks * kStageWords);
          for (int w = 0; w < words; ++w) {
            tmem_cp_32x128b_x4(slot + 4 * w, smem_desc_rows16(sf + kMxBlockBytes * w));
            tmem_cp_32x128b_x4(slot + 8 + 8 * w,
                               smem_desc_rows16(sf + kSfBBytes + kMxBlockBytes * w));
            if (t.tokens > 128)
              tmem_cp_32x128b_x4(slot + 12 + 8 * w,
                                 smem_desc_rows16(sf + 2 * kSfBBytes + kMxBlockBytes * w));
          }
          const uint64_t bdesc = smem_desc_k128_sw128(sb);
          const uint64_t adesc = smem_desc_k128_sw128(sb + kBBytes);
          const int mmas = min(kStageK / kMmaK, k_mmas - ks * (kStageK / kMmaK));
#pragma unroll
          for (int j = 0; j < kStageK / kMmaK; ++j)
            if (j < mmas)
              umma_mxf4(d, bdesc + 2 * j, adesc + 2 * j, idesc, slot + 4 * (j >> 1),
                        slot + 8 + 8 * (j >> 1), 2u * (j & 1), ks > t.k_begin || j > 0 ? 1u : 0u);
          umma_commit(empty_bar(s));
          if (ks + 1 == t.k_end) umma_commit(tfull_bar(buf));
        }
        __syncwarp();
      }
      ++tile_i;
      return true;
    });
    // every MMA issued above completes before TMEM is freed
    if (elect_one()) umma_commit(drain_bar);
    __syncwarp();
    volatile int never = 0;
    mbar_wait(drain_bar, 0, &never, p.status);
  } else if (warp >= kFirstEpiWarp) {
    // ================================================================ epilogue
    // Warp w reads lanes 32 (w mod 4) .. and every other 16-column chunk; the
    // accumulator is handed back once it is in registers, as BF16.
    const int half = (warp - kFirstEpiWarp) >> 2;
    const int quarter = warp & 3;
    int tile_i = 0;
    for_each_tile<SCHED>(p, s_prefix, false, [&](const Tile &t) {
      const int buf = tile_i % nbuf;
      if (!mbar_wait(tfull_bar(buf), (tile_i / nbuf) & 1, abort, p.status)) return false;
      tc_fence_after();
      const uint32_t acc = tmem + static_cast<uint32_t>(buf) * buf_cols +
                           (static_cast<uint32_t>(quarter * 32) << 16);
      if (SCHED == kMxDense && p.splits > 1) {
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
      uint32_t out[8][8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c0 = (2 * i + half) * 16;
        if (c0 < t.tokens) {
          uint32_t r[16];
          tmem_ld<16>(acc + c0, r);
          tmem_wait_ld();
          reg_barrier<16>(r);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(r[2 * j]),
                                                           __uint_as_float(r[2 * j + 1]));
            out[i][j] = *reinterpret_cast<const uint32_t *>(&v);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty_bar(buf));
      // rows that are stored: bit l of live[i] is token 32 i + l
      uint32_t live[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        bool v = 32 * i + lane < t.tokens;
        if (SCHED == kMxContiguous && v)
          v = __ldg(p.m_indices + t.tok0 + 32 * i + lane) == t.group;
        live[i] = __ballot_sync(0xffffffffu, v);
      }
      // neighbouring lanes hold neighbouring columns of D: each pair of lanes
      // swaps halves so that the even lane stores two columns of one token,
      // the odd lane of the next (a warp's store: 64 bytes of two rows)
      const int odd = lane & 1;
      const int n = t.n0 + quarter * 32 + (lane & ~1);
      uint16_t *dst = p.d + (static_cast<int64_t>(t.slab) * p.rows + t.tok0) * p.n + n;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c0 = (2 * i + half) * 16;
        if (c0 < t.tokens) {
          const uint32_t bits = live[i] >> (16 * half + odd);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, out[i][j], 1);
            const uint32_t v = odd ? __byte_perm(other, out[i][j], 0x7632)
                                   : __byte_perm(out[i][j], other, 0x5410);
            if (((bits >> (2 * j)) & 1u) && n < p.n)
              *reinterpret_cast<uint32_t *>(dst + static_cast<int64_t>(c0 + 2 * j + odd) * p.n) =
                  v;
          }
        }
      }
      ++tile_i;
      return true;
    });
  }

  if (SCHED == kMxDense && p.splits > 1) {
    // ============================================================ K reduction
    // The CTAs of the cluster hold the partials of one tile: each sums a share
    // of the tokens over the cluster's shared memory, in split order.
    __syncwarp();
    cluster_sync();
    const int rank = static_cast<int>(cluster_ctarank());
    for_each_tile<SCHED>(p, s_prefix, false, [&](const Tile &t) {
      const int n = t.n0 + 4 * lane;
      for (int c = rank + p.splits * warp; c < t.tokens; c += p.splits * (kThreads / 32)) {
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
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
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

int ceil_div(int a, int b) { return (a + b - 1) / b; }

constexpr int kMaxDevices = 64;

// Most clusters of `size` CTAs (1 .. 8) with all shared memory that are
// resident at once; asked once per device and size.
int clusters_fit(int dev, int size, int smem) {
  static int fit[kMaxDevices][9] = {};  // count + 1; 0 = not asked yet
  if (fit[dev][size] == 0) {
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
    if (cudaOccupancyMaxActiveClusters(&n, mxfp4_gemm_kernel<kMxDense>, &q) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    fit[dev][size] = n + 1;
  }
  return fit[dev][size] - 1;
}

template <int SCHED>
int launch_mxfp4(const uint8_t *A, const uint8_t *B, MxParams p, cudaStream_t stream) {
  const DeviceInfo *info = device_info();
  int dev = 0;
  if (!info || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
    return DG_ERR_CUDA;
  const int sms = effective_num_sms();
  // tokens per tile: the smallest power of two that holds all of them
  p.tok_tile = 16;
  while (p.tok_tile < kMaxTokens && p.tok_tile < p.rows) p.tok_tile *= 2;
  p.tok_tiles = ceil_div(p.rows, p.tok_tile);
  p.n_tiles = ceil_div(p.n, kTileN);
  p.splits = 1;
  const int stage = static_cast<int>(kBBytes) + p.tok_tile * (kStageK / 2) +
                    static_cast<int>(kSfBBytes) * (p.tok_tile > 128 ? 3 : 2);
  const int tables = SCHED == kMxMasked ? (p.groups + 1) * 4 : 0;
  const int most = info->max_smem_optin - 2048;  // barriers and alignment
  p.stages = (most - tables) / stage;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  int smem = 1024 + p.stages * stage + tables;
  if (smem < kMinSmem) smem = kMinSmem;
  static bool configured[kMaxDevices] = {};
  if (!configured[dev]) {
    if (cudaFuncSetAttribute(mxfp4_gemm_kernel<SCHED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             info->max_smem_optin - 1024) != cudaSuccess)
      return DG_ERR_CUDA;
    configured[dev] = true;
  }
  int grid = sms;
  if (SCHED != kMxMasked) {
    const int tiles = p.tok_tiles * p.n_tiles;
    if (tiles < grid) grid = tiles;
    if (SCHED == kMxDense) {
      // fewer tiles than SMs: split K over the CTAs of a cluster
      const int k_stages = ceil_div(p.k, kStageK);
      int s = sms / tiles;
      if (s > 8) s = 8;
      if (s > k_stages) s = k_stages;
      while (s > 1 && clusters_fit(dev, s, info->max_smem_optin - 1024) < tiles) --s;
      if (s > 1) {
        p.splits = s;
        grid = tiles * s;
      }
    }
  }
  CUtensorMap ta, tb;
  const int slabs = SCHED == kMxMasked ? p.groups : 1;
  int rc = make_tmap(&ta, A, p.k, p.rows, slabs, p.tok_tile);
  if (!rc) rc = make_tmap(&tb, B, p.k, p.n, p.groups, kTileN);
  if (rc) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0] = pdl_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.splits > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, mxfp4_gemm_kernel<SCHED>, ta, tb, p) == cudaSuccess
             ? DG_OK
             : DG_ERR_CUDA;
}

int check_gemm(const void *A, const void *sfa, const void *B, const void *sfb, const void *D,
               int64_t rows, int64_t N, int64_t K, int64_t slabs, int64_t groups) {
  if (rows < 0 || N <= 0 || K <= 0 || K % kMxGroup != 0 || N % 8 != 0) return DG_ERR_INVALID_ARG;
  if (rows == 0) return DG_OK;
  if (!A || !sfa || !B || !sfb || !D) return DG_ERR_INVALID_ARG;
  // tile and block counts are 32-bit
  constexpr int64_t kMost = 0x7FFFFF00;
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

MxParams make_params(const int32_t *sfa, const int32_t *sfb, void *D, int64_t rows, int64_t N,
                     int64_t K, int groups) {
  MxParams p{};
  p.sfa = reinterpret_cast<const uint8_t *>(sfa);
  p.sfb = reinterpret_cast<const uint8_t *>(sfb);
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
  return launch_mxfp4<kMxDense>(A, B, make_params(sfa, sfb, D, M, N, K, 1),
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
  MxParams p = make_params(sfa, sfb, D, M_total, N, K, G);
  p.m_indices = m_indices;
  return launch_mxfp4<kMxContiguous>(A, B, p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int dg_m_grouped_mxfp4_gemm_nt_masked(const uint8_t *A, const int32_t *sfa,
                                                 const uint8_t *B, const int32_t *sfb, void *D,
                                                 const int32_t *masked_m, int G, int64_t M_max,
                                                 int64_t N, int64_t K, dg_stream_t stream) {
  using namespace dg;
  if (G < 1 || G > 1024 || M_max < 1) return DG_ERR_INVALID_ARG;
  int rc = check_gemm(A, sfa, B, sfb, D, M_max, N, K, G, G);
  if (rc) return rc;
  if (!masked_m) return DG_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(masked_m) % 4 != 0) return DG_ERR_ALIGNMENT;
  rc = usable_device();
  if (rc) return rc;
  MxParams p = make_params(sfa, sfb, D, M_max, N, K, G);
  p.masked_m = masked_m;
  return launch_mxfp4<kMxMasked>(A, B, p, reinterpret_cast<cudaStream_t>(stream));
}
