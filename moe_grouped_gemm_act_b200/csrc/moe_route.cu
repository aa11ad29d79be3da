// moe_route.cu -- routing of tokens to experts: softmax, top-k, per-expert
// counts and the balance loss, and the gradient of the logits.
//
// With p_t = softmax(logits_t) over the E experts and idx_t the k largest
// logits of a token (ties go to the lowest index):
//     w_tj     = p_t[idx_tj]            (normalized: divided by their sum)
//     counts_e = #{(t, j): idx_tj = e}
//     loss     = E / (k n^2) * sum_e counts_e * sum_t p_te
// where n counts the tokens that route at all.  The loss is E times the inner
// product of the experts' share of the choices and their mean probability;
// the counts are constants in its gradient.
//
// Gradient, c_e = dloss * E / (k n^2) * counts_e, <.,.> over a token's experts:
//     dlogits_e = p_e (c_e - <p, c>)
//               + [e = idx_j]  w_j (dw_j - <w, dw>)     (normalized)
//               + [e = idx_j]  w_j dw_j - p_e <w, dw>   (else)
//
// A warp takes a token, lane l the experts l V .. l V + V - 1, so that a token is
// read once, in contiguous 16-byte loads where its row allows them.  The top-k
// are k rounds of a warp maximum over order-preserving integer keys; the lowest
// lane that holds the maximum has the lowest index.  Sums over tokens are exact
// (counts) or taken in a fixed order (probabilities: per lane over a warp's
// tokens, over the warps of a block, over the blocks), so a repeated call gives
// the same bits.  Loads are coherent (no __ldg): the kernels start before the
// ones ahead of them on the stream have finished.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "dg.h"
#include "host.h"
#include "internal.h"
#include "ptx.cuh"

namespace dg {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;  // lane j keeps choice j
constexpr int kFinishCtas = 8;  // one cluster
// Up to this many tokens (two per warp of it) one cluster does everything in one
// launch; above it a second kernel joins the blocks' sums.  One cluster against the
// join, on the GPU: 32 experts, FP32, 128 / 256 / 512 tokens 3.8 / 5.3 / 8.0 against
// 4.9 / 5.2 / 5.2 us; 256 experts, BF16, 4.5 / 6.4 / 10.1 against 5.9 / 6.0 / 6.4 us;
// 1024 experts, FP32, 11.7 / 16.7 / 25.6 against 13.6 / 13.7 / 13.9 us.  So at 256
// tokens it loses up to 3 us there, and saves a launch and a workspace on the host.
constexpr int kClusterTokens = 2 * kWarps * kFinishCtas;

// Resident blocks per SM that an instance with V experts per lane is compiled
// for: a token is a chain of shuffles and warp maxima whose latency other warps
// hide, but with fewer registers than these leave it spills (V = 8 with three
// blocks: 26.8 us against 24.2 us for 32768 tokens of 256 experts; V = 2 with two:
// 27.9 against 17.7 us for 64 experts).  The one-cluster instances take the same
// figure, and with V = 1 and 2 spill 68 to 196 bytes; BF16 with V = 32 spills 12 to
// 16 bytes in both forms.
constexpr int resident(int v) { return v <= 2 ? 4 : v == 4 ? 3 : v == 8 ? 2 : 1; }

// Order-preserving key of an FP32 value that is not NaN; -0 and +0 are one key.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;  // order_key(-inf); 0: no candidate

// A word of the cluster's shared memory.
__device__ __forceinline__ uint32_t ld_shared_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void st_shared_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Experts l V .. l V + V - 1 of a row of E logits, -inf past E.  (Through L1: a lane's
// pieces share sectors.)  `vec`: rows start on a 16-byte boundary (or V elements, if
// that is less) and E % V == 0.
template <int V>
__device__ __forceinline__ void load_row(const float *row, int E, bool vec, float x[V]) {
  const int e0 = (threadIdx.x & 31) * V;
  if constexpr (V >= 2) {
    if (vec) {
      constexpr int S = V < 4 ? V : 4;
#pragma unroll
      for (int i = 0; i < V; i += S) {
        if constexpr (S == 4) {
          const float4 t = e0 < E ? *reinterpret_cast<const float4 *>(row + e0 + i)
                                  : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
          x[i] = t.x; x[i + 1] = t.y; x[i + 2] = t.z; x[i + 3] = t.w;
        } else {
          const float2 t = e0 < E ? *reinterpret_cast<const float2 *>(row + e0 + i)
                                  : make_float2(-INFINITY, -INFINITY);
          x[i] = t.x; x[i + 1] = t.y;
        }
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = e0 + i < E ? row[e0 + i] : -INFINITY;
}
__device__ __forceinline__ void unpack_bf16(uint32_t w, float &a, float &b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xFFFF0000u);
}
template <int V>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *row, int E, bool vec, float x[V]) {
  const int e0 = (threadIdx.x & 31) * V;
  constexpr uint32_t kNegInf2 = 0xFF80FF80u;
  if constexpr (V >= 2) {
    if (vec) {
      constexpr int S = V < 8 ? V : 8;
#pragma unroll
      for (int i = 0; i < V; i += S) {
        if constexpr (S == 8) {
          const uint4 t = e0 < E ? *reinterpret_cast<const uint4 *>(row + e0 + i)
                                 : make_uint4(kNegInf2, kNegInf2, kNegInf2, kNegInf2);
          unpack_bf16(t.x, x[i], x[i + 1]);
          unpack_bf16(t.y, x[i + 2], x[i + 3]);
          unpack_bf16(t.z, x[i + 4], x[i + 5]);
          unpack_bf16(t.w, x[i + 6], x[i + 7]);
        } else if constexpr (S == 4) {
          const uint2 t = e0 < E ? *reinterpret_cast<const uint2 *>(row + e0 + i)
                                 : make_uint2(kNegInf2, kNegInf2);
          unpack_bf16(t.x, x[i], x[i + 1]);
          unpack_bf16(t.y, x[i + 2], x[i + 3]);
        } else {
          const uint32_t t = e0 < E ? *reinterpret_cast<const uint32_t *>(row + e0 + i)
                                    : kNegInf2;
          unpack_bf16(t, x[i], x[i + 1]);
        }
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    x[i] = e0 + i < E
               ? __uint_as_float(
                     static_cast<uint32_t>(reinterpret_cast<const unsigned short *>(row)[e0 + i])
                     << 16)
               : -INFINITY;
}

struct RouteParams {
  const void *logits;
  int64_t tokens, ld;
  int experts, top_k, normalize, vec;
  const uint8_t *mask;  // token routes when nonzero (nullptr: all do)
  int32_t *idx;
  float *weights;
  int32_t *counts;
  float *loss;
  int32_t *num_tokens;
  // [blocks][E + 1]: an expert's probability sum (FP32 bits) and count; in
  // column E the block's routed tokens as a count
  int2 *part;
  int *status;
};

// A warp's row of shared memory: lane l's V words start at l row_step(V), whose
// multiples of 16 bytes are odd so that 16-byte accesses do not meet in a bank.
__host__ __device__ constexpr int row_step(int v) { return v >= 8 ? v + 4 : v; }
__host__ __device__ constexpr int row_words(int v) { return 32 * row_step(v); }

__device__ __forceinline__ float loss_of(const RouteParams &p, float total, int n) {
  const float nf = static_cast<float>(n);
  return n > 0 ? total * (static_cast<float>(p.experts) /
                          (static_cast<float>(p.top_k) * nf * nf))
               : 0.0f;
}

// The choice of the k largest, one per round; no open expert left ends it.  The
// first is the row's largest, which the softmax has found, and the last is not
// taken out (one round less of k: 32768 tokens of 256 experts, BF16, 24.8 -> 24.2
// us).
// (Compares, selects and integer maxima keep the ALU pipe at 57 %, so a round has
// few of them per expert: 32768 tokens of 256 experts take 19.0 us at k = 1 and 25.2
// at k = 8 in BF16, 18.9 and 28.3 in FP32.  The larger part of the time is what a
// token costs whatever k: its exponentials, divisions, warp sums and keys.)
//
// kRow: a lane keeps its largest key, the others wait in the warp's
// row of shared memory.  A round is a warp maximum; the lowest lane that holds
// it owns the lowest such expert, and the warp looks up the owner's V keys
// together, takes the chosen one out and finds the owner's next: some twenty
// instructions whatever V.
enum Form { kRow, kRegisters, kWords };
template <int V, int FORM>
struct TopK {
  uint32_t top, best;
  uint32_t *row;  // [row_words(V)]
  // Experts past E hold -inf, like closed ones.
  __device__ __forceinline__ void init(const float x[V], uint32_t *warp_row) {
    row = warp_row;
    uint32_t key[V];
    top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = order_key(x[i]);
      top = max(top, key[i]);
    }
    uint32_t *mine = row + (threadIdx.x & 31) * row_step(V);
    if constexpr (V >= 4) {
#pragma unroll
      for (int i = 0; i < V; i += 4)
        *reinterpret_cast<uint4 *>(mine + i) =
            make_uint4(key[i], key[i + 1], key[i + 2], key[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) mine[i] = key[i];
    }
  }
  // The row's largest logit (-inf: no expert is open).
  __device__ __forceinline__ float largest() {
    best = __reduce_max_sync(0xffffffffu, top);
    return key_value(best);
  }
  // The K largest, choice j to lane j: its expert (-1: none) and logit.
  __device__ __forceinline__ void choose(int K, int &expert, float &value) {
    const int lane = threadIdx.x & 31;
    uint32_t mine = kKeyNegInf;
    expert = -1;
    __syncwarp();  // the row is written
    for (int j = 0;;) {
      if (best <= kKeyNegInf) break;  // only closed experts are left
      const int owner = __ffs(__ballot_sync(0xffffffffu, top == best)) - 1;
      uint32_t *owned = row + owner * row_step(V);
      uint32_t key = lane < V ? owned[lane] : 0u;
      const int at = __ffs(__ballot_sync(0xffffffffu, key == best)) - 1;
      if (lane == j) {
        expert = owner * V + at;
        mine = best;
      }
      if (++j == K) break;
      if (lane == at) {
        key = 0;
        owned[at] = 0;
      }
      const uint32_t next = __reduce_max_sync(0xffffffffu, key);
      if (lane == owner) top = next;
      best = __reduce_max_sync(0xffffffffu, top);
      __syncwarp();
    }
    __syncwarp();  // the row is free
    value = key_value(mine);
  }
};
// Few experts per lane: the keys stay in registers, and every lane takes the
// choice out and finds its largest again (32 experts, FP32: 3.6 us a call of 64
// tokens against 4.4 us; from V = 4 on the form above is faster: 128 experts, 8
// choices 24.6 against 27.1 us for 32768 tokens, 1024 experts, 16 choices 28
// against 55 us for 8192).
template <int V>
struct TopK<V, kRegisters> {
  uint32_t key[V], top, best;
  int at;  // the lane's lowest expert with key == top
  __device__ __forceinline__ void find_top() {
    top = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = max(top, key[i]);
    at = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (key[i] == top) at = i;
    at += (threadIdx.x & 31) * V;
  }
  __device__ __forceinline__ void init(const float x[V], uint32_t *) {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = order_key(x[i]);
    find_top();
  }
  __device__ __forceinline__ float largest() {
    best = __reduce_max_sync(0xffffffffu, top);
    return key_value(best);
  }
  __device__ __forceinline__ void choose(int K, int &expert, float &value) {
    const int lane = threadIdx.x & 31;
    uint32_t mine = kKeyNegInf;
    expert = -1;
    for (int j = 0;;) {
      if (best <= kKeyNegInf) break;
      const int e = static_cast<int>(__reduce_min_sync(
          0xffffffffu, top == best ? static_cast<uint32_t>(at) : 0xFFFFFFFFu));
      if (lane == j) {
        expert = e;
        mine = best;
      }
      if (++j == K) break;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane * V + i == e) key[i] = 0;
      find_top();
      best = __reduce_max_sync(0xffffffffu, top);
    }
    value = key_value(mine);
  }
};
// BF16 logits: the 16-bit key and the expert (larger for lower experts) share a
// 26-bit word, so all words differ and a round is one warp maximum.  The words
// are kept relative to the last choice: chosen ones are zero or positive, the
// others negative, that is larger as unsigned numbers, so the unsigned maximum
// is the next choice and taking it out is one subtraction per word.
template <int V>
struct TopK<V, kWords> {
  uint32_t rel[V], top, best;
  __device__ __forceinline__ void find_top() {
    top = rel[0];
#pragma unroll
    for (int i = 1; i + 1 < V; i += 2) top = max(max(top, rel[i]), rel[i + 1]);
    if constexpr (V % 2 == 0) top = max(top, rel[V - 1]);
  }
  __device__ __forceinline__ void init(const float x[V], uint32_t *) {
    const uint32_t low = 1023u - (threadIdx.x & 31) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t u = __float_as_uint(x[i] + 0.0f);
      const uint32_t flip = (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) & 0x7FFF0000u) |
                            0x80000000u;
      rel[i] = ((u ^ flip) >> 6) + (low - i);
    }
    find_top();
  }
  static __device__ __forceinline__ float value_of(uint32_t word) {
    const uint32_t k = (word >> 10) << 16;
    return key_value((k & 0x80000000u) ? k : k | 0xFFFFu);
  }
  __device__ __forceinline__ float largest() {
    best = __reduce_max_sync(0xffffffffu, top);
    return value_of(best);
  }
  __device__ __forceinline__ void choose(int K, int &expert, float &value) {
    const int lane = threadIdx.x & 31;
    uint32_t mine = 0x7Fu << 10;  // -inf's key is 0x7F
    uint32_t base = best;
    for (int j = 0;;) {
      if (base < (0x80u << 10)) break;  // only closed experts are left
      if (lane == j) mine = base;
      if (++j == K) break;
#pragma unroll
      for (int i = 0; i < V; ++i) rel[i] -= best;
      find_top();
      best = __reduce_max_sync(0xffffffffu, top);
      base += best;
    }
    expert = mine < (0x80u << 10) ? -1 : 1023 - static_cast<int>(mine & 1023u);
    value = value_of(mine);
  }
};

// CLUSTER: the grid is one cluster of kFinishCtas CTAs, whose rank 0 joins the
// blocks' sums over the cluster's shared memory (one launch); else the sums go
// to the workspace.
template <typename T, int V, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, resident(V))
moe_route_kernel(const RouteParams p) {
  // [kWarps][row_words(V)], a warp's keys and then its probability sums; [E] counts
  extern __shared__ __align__(16) float s_mem[];
  constexpr int kStride = row_words(V);
  constexpr int kForm = sizeof(T) == 2 ? kWords : V <= 2 ? kRegisters : kRow;
  __shared__ float s_red[kWarps];
  __shared__ int32_t s_tokens;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.experts, K = p.top_k;
  float *s_psum = s_mem;
  int32_t *s_counts = reinterpret_cast<int32_t *>(s_mem + kWarps * kStride);
  grid_launch_dependents();
  for (int e = threadIdx.x; e < E; e += kThreads) s_counts[e] = 0;
  if (threadIdx.x == 0) s_tokens = 0;
  __syncthreads();
  grid_dependency_wait();

  float psum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) psum[i] = 0.0f;
  int routed = 0;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps;
  // (neighbouring tokens go to different blocks, so that few tokens spread)
  for (int64_t t = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x; t < p.tokens;
       t += stride) {
    float x[V];
    load_row<V>(static_cast<const T *>(p.logits) + t * p.ld, E, p.vec != 0, x);
    TopK<V, kForm> topk;
    topk.init(x, reinterpret_cast<uint32_t *>(s_psum + warp * kStride));
    const float xmax = topk.largest();
    // a NaN or +inf anywhere makes the sum NaN, and so does a row that is
    // closed altogether
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float e = expf(x[i] - xmax);
      sum += e;
      x[i] = e;
    }
    sum = warp_sum(sum);
    const bool masked = p.mask && !p.mask[t];
    int my_idx = -1;
    float my_w = 0.0f;
    if (!masked && sum == sum) {
      ++routed;
      // (a product with the reciprocal: one FP32 rounding more than a division for
      // each expert)
      const float inv = 1.0f / sum;
#pragma unroll
      for (int i = 0; i < V; ++i) psum[i] += x[i] * inv;
      float my_x;
      topk.choose(K, my_idx, my_x);
      my_w = expf(my_x - xmax) * inv;  // (0 in the lanes without a choice)
      if (p.normalize) my_w /= warp_sum(my_w);
      if (my_idx >= 0) atomicAdd(&s_counts[my_idx], 1);
    } else if (!masked) {
      // not routed: an error unless every logit is -inf
      bool bad = false;
      load_row<V>(static_cast<const T *>(p.logits) + t * p.ld, E, p.vec != 0, x);
#pragma unroll
      for (int i = 0; i < V; ++i) bad |= x[i] != -INFINITY;
      if (bad) record_status(p.status, DG_ERR_DEVICE_DATA);
    }
    if (lane < K) {
      p.idx[t * K + lane] = my_idx;
      p.weights[t * K + lane] = my_w;
    }
  }
  // A lane's sums lie where other lanes' keys were; after a last token that does not
  // route nothing else orders these writes behind those of init().
  __syncwarp();
#pragma unroll
  for (int i = 0; i < V; ++i)
    s_psum[warp * kStride + lane * V + i] = psum[i];
  if (lane == 0) atomicAdd(&s_tokens, routed);
  __syncthreads();
  // the block's sums, in the first row (a thread reads only its own columns)
  for (int e = threadIdx.x; e < E; e += kThreads) {
    float s = 0.0f;
#pragma unroll 4
    for (int w = 0; w < kWarps; ++w) s += s_psum[w * kStride + e];
    if constexpr (CLUSTER) {
      s_psum[e] = s;
    } else {
      p.part[static_cast<int64_t>(blockIdx.x) * (E + 1) + e] =
          make_int2(__float_as_int(s), s_counts[e]);
    }
  }
  if constexpr (CLUSTER) {
    __syncwarp();
    cluster_sync();
    if (blockIdx.x == 0) {
      float acc = 0.0f;
      for (int e = threadIdx.x; e < E; e += kThreads) {
        float s = 0.0f;
        int c = 0;
#pragma unroll
        for (int r = 0; r < kFinishCtas; ++r) {
          s += __uint_as_float(ld_shared_cluster(mapa_shared(smem_u32(s_psum + e), r)));
          c += static_cast<int>(ld_shared_cluster(mapa_shared(smem_u32(s_counts + e), r)));
        }
        p.counts[e] = c;
        acc += static_cast<float>(c) * s;
      }
      acc = warp_sum(acc);
      if (lane == 0) s_red[warp] = acc;
      __syncthreads();
      if (threadIdx.x == 0) {
        float total = 0.0f;
        for (int w = 0; w < kWarps; ++w) total += s_red[w];
        int n = 0;
#pragma unroll
        for (int r = 0; r < kFinishCtas; ++r)
          n += static_cast<int>(ld_shared_cluster(mapa_shared(smem_u32(&s_tokens), r)));
        *p.loss = loss_of(p, total, n);
        *p.num_tokens = n;
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while its sums are being read
  } else {
    if (threadIdx.x == 0)
      p.part[static_cast<int64_t>(blockIdx.x) * (E + 1) + E] = make_int2(0, s_tokens);
  }
}

// Joins the blocks' sums: a cluster of kFinishCtas CTAs, each with a share of the
// E + 1 columns.  A CTA's threads are `parts` rows of its columns, each summing
// every parts-th block with kBatch loads in flight (it is bound by latency: one
// round trip for most shapes); a warp adds a column's parts in a fixed order, and
// the CTAs' shares of the loss go to CTA 0.  (A share of the blocks for each CTA,
// all columns joined by CTA 0: 0.7 us more of 25 at 32768 tokens of 256 experts,
// 1.3 us more of 30 at 8192 tokens of 1024.)
constexpr int kFinishThreads = 1024;
__global__ void __launch_bounds__(kFinishThreads)
moe_route_finish_kernel(const RouteParams p, int blocks) {
  constexpr int kBatch = 12, kFinishWarps = kFinishThreads / 32;
  __shared__ float s_sum[kFinishThreads];
  __shared__ int32_t s_count[kFinishThreads];
  __shared__ float s_red[kFinishWarps];
  __shared__ uint32_t s_loss[kFinishCtas], s_tokens;  // CTA 0's are used
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cols = p.experts + 1;
  // (odd: a warp reads a column of s_sum without bank conflicts)
  const int share = ((cols + kFinishCtas - 1) / kFinishCtas) | 1;
  const int col0 = blockIdx.x * share;
  const int parts = kFinishThreads / share;
  const int part = tid / share, mine = tid - part * share;
  grid_launch_dependents();
  cluster_sync();  // all CTAs run before one writes into CTA 0's memory
  grid_dependency_wait();
  if (part < parts && col0 + mine < cols) {
    float s = 0.0f;
    int c = 0;
    for (int b0 = part; b0 < blocks; b0 += parts * kBatch) {
      int2 v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int b = b0 + j * parts;
        v[j] = b < blocks ? __ldcg(p.part + static_cast<int64_t>(b) * cols + col0 + mine)
                          : make_int2(0, 0);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        s += __int_as_float(v[j].x);
        c += v[j].y;
      }
    }
    s_sum[tid] = s;
    s_count[tid] = c;
  }
  __syncthreads();
  float acc = 0.0f;
  for (int i = warp; i < share && col0 + i < cols; i += kFinishWarps) {
    const int col = col0 + i;
    float s = 0.0f;
    int c = 0;
    for (int q = lane; q < parts; q += 32) {
      s += s_sum[q * share + i];
      c += s_count[q * share + i];
    }
    s = warp_sum(s);
    c = __reduce_add_sync(0xffffffffu, c);
    if (col < p.experts) {
      if (lane == 0) p.counts[col] = c;
      acc += static_cast<float>(c) * s;
    } else if (lane == 0) {  // the routed tokens
      st_shared_cluster(mapa_shared(smem_u32(&s_tokens), 0), static_cast<uint32_t>(c));
    }
  }
  if (lane == 0) s_red[warp] = acc;
  __syncthreads();
  if (warp == 0) {
    const float total = warp_sum(s_red[lane]);
    if (lane == 0)
      st_shared_cluster(mapa_shared(smem_u32(s_loss + blockIdx.x), 0), __float_as_uint(total));
  }
  __syncwarp();
  cluster_sync();
  if (blockIdx.x == 0 && tid == 0) {
    float total = 0.0f;
#pragma unroll
    for (int r = 0; r < kFinishCtas; ++r) total += __uint_as_float(s_loss[r]);
    const int n = static_cast<int>(s_tokens);
    *p.loss = loss_of(p, total, n);
    *p.num_tokens = n;
  }
}

// The gradient of the logits.  A token that did not route (idx[t][0] < 0) gets
// zeros; its logits are not used, so what they hold does not matter.  Probabilities
// are products with the reciprocal of their sum, as in the forward kernel.  A warp
// takes its tokens one after another and asks for a token's logits once its choices
// are there: two round trips each bound it (32768 tokens of 256 experts, BF16: ALU
// pipe 26 %, DRAM 12 %; 16 us, FP32 17 us).
struct RouteBackwardParams {
  const void *logits;
  int64_t tokens, ld;
  int experts, top_k, normalize, vec;
  const int32_t *idx;
  const float *weights;
  const int32_t *counts;
  const int32_t *num_tokens;
  const float *dweights;  // nullptr: zero
  const float *dloss;     // nullptr: zero
  void *dlogits;          // [tokens][experts]
};

// A lane's V consecutive gradients.  BF16 gradients of BF16 logits: the one
// rounding, to nearest even.
template <int V>
__device__ __forceinline__ void store_piece(float *row, int E, bool vec, const float g[V]) {
  const int e0 = (threadIdx.x & 31) * V;
  if constexpr (V >= 2) {
    if (vec) {
      if (e0 < E) {
        constexpr int S = V < 4 ? V : 4;
#pragma unroll
        for (int i = 0; i < V; i += S) {
          if constexpr (S == 4)
            *reinterpret_cast<float4 *>(row + e0 + i) =
                make_float4(g[i], g[i + 1], g[i + 2], g[i + 3]);
          else
            *reinterpret_cast<float2 *>(row + e0 + i) = make_float2(g[i], g[i + 1]);
        }
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (e0 + i < E) row[e0 + i] = g[i];
}
template <int V>
__device__ __forceinline__ void store_piece(__nv_bfloat16 *row, int E, bool vec, const float g[V]) {
  const int e0 = (threadIdx.x & 31) * V;
  if constexpr (V >= 2) {
    if (vec) {
      if (e0 < E) {
        uint32_t w[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          const __nv_bfloat162 t = __floats2bfloat162_rn(g[2 * i], g[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t *>(&t);
        }
        if constexpr (V >= 8) {
#pragma unroll
          for (int i = 0; i < V / 8; ++i)
            reinterpret_cast<uint4 *>(row + e0)[i] =
                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else if constexpr (V == 4) {
          *reinterpret_cast<uint2 *>(row + e0) = make_uint2(w[0], w[1]);
        } else {
          *reinterpret_cast<uint32_t *>(row + e0) = w[0];
        }
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (e0 + i < E) row[e0 + i] = __float2bfloat16_rn(g[i]);
}

__device__ __forceinline__ void store_one(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_one(__nv_bfloat16 *p, float v) {
  *p = __float2bfloat16_rn(v);
}
__device__ __forceinline__ void store_four(float *p, const float4 &v) {
  *reinterpret_cast<float4 *>(p) = v;
}
__device__ __forceinline__ void store_four(__nv_bfloat16 *p, const float4 &v) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                                             *reinterpret_cast<const uint32_t *>(&hi));
}
// A row of shared memory to E consecutive elements, neighbouring lanes to
// neighbouring addresses; `row` nullptr: zeros.
template <int V, typename T>
__device__ __forceinline__ void store_row(T *out, const float *row, int E, bool vec) {
  const int lane = threadIdx.x & 31;
  if (V >= 4 && vec) {
    for (int e = 4 * lane; e < E; e += 128)
      store_four(out + e, row ? *reinterpret_cast<const float4 *>(row + e / V * row_step(V) + e % V)
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f));
  } else {
    for (int e = lane; e < E; e += 32)
      store_one(out + e, row ? row[e / V * row_step(V) + e % V] : 0.0f);
  }
}

// Lane l's V words of a row of shared memory.
template <int V>
__device__ __forceinline__ void row_store(float *row, const float g[V]) {
  float *mine = row + (threadIdx.x & 31) * row_step(V);
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4 *>(mine + i) = make_float4(g[i], g[i + 1], g[i + 2], g[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) mine[i] = g[i];
  }
}

// Blocks per SM of the backward kernel.  From V = 16 on the experts' c are in
// shared memory, so that a lane only keeps its V gradients (BF16, 512 experts:
// 11.8 against 16.5 us for 16384 tokens); below, in registers (72 experts: 3.7
// against 4.3 us for 5001).
constexpr int resident_backward(int v) { return v == 16 ? 2 : resident(v); }

template <typename T, int V>
__global__ void __launch_bounds__(kThreads, resident_backward(V))
moe_route_backward_kernel(const RouteBackwardParams p) {
  // a row per warp for its gradients, to which the lanes of the chosen experts
  // add, then (V >= 16) the experts' c
  extern __shared__ __align__(16) float s_rows[];
  constexpr bool kShared = V >= 16;
  // Gradients leave from the row, neighbouring lanes to neighbouring addresses,
  // where a lane's own piece is 64 bytes or more (FP32, 1024 experts: 18.4
  // against 25.4 us for 8192 tokens); smaller pieces leave from the registers
  // (BF16, 256 experts: 13.0 against 15.4 us for 32768).
  constexpr bool kFromRow = V * sizeof(T) >= 64;
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int E = p.experts, K = p.top_k;
  float *row = s_rows + (threadIdx.x >> 5) * row_words(V);
  float *s_c = s_rows + kWarps * row_words(V);
  float c_own[kShared ? 1 : V];
  {
    const int n = *p.num_tokens;
    const float nf = static_cast<float>(n);
    const float f = p.dloss && n > 0
                        ? *p.dloss * (static_cast<float>(E) / (static_cast<float>(K) * nf * nf))
                        : 0.0f;
    if constexpr (kShared) {
      for (int e = threadIdx.x; e < 32 * V; e += kThreads)
        s_c[e / V * row_step(V) + e % V] = e < E ? f * static_cast<float>(p.counts[e]) : 0.0f;
      __syncthreads();
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        c_own[i] = lane * V + i < E ? f * static_cast<float>(p.counts[lane * V + i]) : 0.0f;
    }
  }
  auto c = [&](int i) -> float {
    if constexpr (kShared) return s_c[lane * row_step(V) + i];
    else return c_own[i];
  };
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); t < p.tokens;
       t += stride) {
    const int my_idx = lane < K ? p.idx[t * K + lane] : -1;
    T *out = static_cast<T *>(p.dlogits) + t * E;
    if (__shfl_sync(0xffffffffu, my_idx, 0) < 0) {
      if constexpr (kFromRow) {
        store_row<V>(out, nullptr, E, p.vec != 0);
      } else {
        float zero[V];
#pragma unroll
        for (int i = 0; i < V; ++i) zero[i] = 0.0f;
        store_piece<V>(out, E, p.vec != 0, zero);
      }
    } else {
      float g[V];
      const float w = my_idx >= 0 ? p.weights[t * K + lane] : 0.0f;
      const float dw = my_idx >= 0 && p.dweights ? p.dweights[t * K + lane] : 0.0f;
      load_row<V>(static_cast<const T *>(p.logits) + t * p.ld, E, p.vec != 0, g);
      float xmax = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) xmax = fmaxf(xmax, g[i]);
      xmax = key_value(__reduce_max_sync(0xffffffffu, order_key(xmax)));
      float sum = 0.0f, pc = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        g[i] = expf(g[i] - xmax);
        sum += g[i];
        pc += g[i] * c(i);
      }
      const float inv = 1.0f / warp_sum(sum);
      const float wdw = warp_sum(w * dw);
      // what every expert's probability is multiplied by, less its own c
      const float minus = warp_sum(pc) * inv + (p.normalize ? 0.0f : wdw);
      const float dv = p.normalize ? w * (dw - wdw) : w * dw;
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] = g[i] * inv * (c(i) - minus);
      // the chosen experts are distinct, so their lanes' additions do not meet
      row_store<V>(row, g);
      __syncwarp();
      if (my_idx >= 0 && my_idx < E) row[my_idx / V * row_step(V) + my_idx % V] += dv;
      __syncwarp();
      if constexpr (kFromRow) {
        store_row<V>(out, row, E, p.vec != 0);
      } else {
        const float *mine = row + lane * row_step(V);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = mine[i];
        store_piece<V>(out, E, p.vec != 0, g);
      }
      __syncwarp();  // the row is free for the next token
    }
  }
}

int check_device() {
  const DeviceInfo *d = device_info();
  if (!d) return DG_ERR_CUDA;
  return d->ok ? DG_OK : DG_ERR_UNSUPPORTED_ARCH;
}

// Experts per lane: the power of two that covers E with 32 lanes.
int per_lane(int experts) {
  int v = 1;
  while (32 * v < experts) v *= 2;
  return v;
}

// Blocks of a launch over `tokens`: all resident, a token per warp at least.
int token_blocks(int64_t tokens, int num_sms, int per_sm) {
  const int64_t want = (tokens + kWarps - 1) / kWarps;
  const int64_t most = static_cast<int64_t>(num_sms) * per_sm;
  return static_cast<int>(want < most ? want : most);
}

int route_blocks(int64_t tokens, int experts, int num_sms) {
  return tokens <= kClusterTokens ? kFinishCtas
                                  : token_blocks(tokens, num_sms, resident(per_lane(experts)));
}

// Scratch of a launch of `blocks`: RouteParams::part.
size_t part_bytes(int blocks, int experts) {
  return static_cast<size_t>(blocks) * (static_cast<size_t>(experts) + 1) * sizeof(int2);
}

// Whether a row's V-element pieces can be loaded whole: they start on a
// 16-byte boundary (their own size, if less) and none is cut by E.
int vector_rows(const void *a, const void *b, int64_t ld, int64_t ld_b, int experts, int esz) {
  const int v = per_lane(experts);
  const int64_t bytes = v * esz < 16 ? v * esz : 16;
  return v >= 2 && experts % v == 0 && (ld * esz) % bytes == 0 && (ld_b * esz) % bytes == 0 &&
         reinterpret_cast<uintptr_t>(a) % bytes == 0 && reinterpret_cast<uintptr_t>(b) % bytes == 0;
}

// `most`: the dynamic shared memory of the kernel's largest launch.
template <typename P>
int launch(void (*kern)(P), int blocks, int smem, int most, const P &p, cudaStream_t stream,
           int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0] = pdl_attribute();
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  // (a maximum of more than 48 KB has to be asked for, on each device; always the
  // same one, so that threads with launches of different sizes do not lower it for
  // each other)
  if (most > 48 * 1024) {
    const int rc = cuda_status(
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
    if (rc) return rc;
  }
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, p));
}

template <typename T, int V>
int route_instance(const RouteParams &p, int blocks, bool cluster, cudaStream_t stream) {
  const int rows = kWarps * row_words(V) * 4, smem = rows + p.experts * 4;
  const int most = rows + 32 * V * 4;
  return cluster ? launch(moe_route_kernel<T, V, true>, blocks, smem, most, p, stream, blocks)
                 : launch(moe_route_kernel<T, V, false>, blocks, smem, most, p, stream);
}

template <typename T>
int route_typed(const RouteParams &p, int blocks, bool cluster, cudaStream_t stream) {
  switch (per_lane(p.experts)) {
    case 1: return route_instance<T, 1>(p, blocks, cluster, stream);
    case 2: return route_instance<T, 2>(p, blocks, cluster, stream);
    case 4: return route_instance<T, 4>(p, blocks, cluster, stream);
    case 8: return route_instance<T, 8>(p, blocks, cluster, stream);
    case 16: return route_instance<T, 16>(p, blocks, cluster, stream);
    default: return route_instance<T, 32>(p, blocks, cluster, stream);
  }
}

template <typename T, int V>
int backward_instance(const RouteBackwardParams &p, int blocks, cudaStream_t stream) {
  const int smem = (1 + kWarps) * row_words(V) * 4;
  return launch(moe_route_backward_kernel<T, V>, blocks, smem, smem, p, stream);
}

template <typename T>
int backward_typed(const RouteBackwardParams &p, int blocks, cudaStream_t stream) {
  switch (per_lane(p.experts)) {
    case 1: return backward_instance<T, 1>(p, blocks, stream);
    case 2: return backward_instance<T, 2>(p, blocks, stream);
    case 4: return backward_instance<T, 4>(p, blocks, stream);
    case 8: return backward_instance<T, 8>(p, blocks, stream);
    case 16: return backward_instance<T, 16>(p, blocks, stream);
    default: return backward_instance<T, 32>(p, blocks, stream);
  }
}

int check_shape(int dtype, int64_t tokens, int experts, int64_t ld, int top_k, int normalize) {
  if (dtype != DG_DTYPE_F32 && dtype != DG_DTYPE_BF16) return DG_ERR_INVALID_ARG;
  if (normalize != 0 && normalize != 1) return DG_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > 0x7FFFFFFF || experts < 1 || experts > kMaxExperts)
    return DG_ERR_INVALID_ARG;
  if (top_k < 1 || top_k > kMaxTopK || top_k > experts) return DG_ERR_INVALID_ARG;
  if (ld < experts || ld > 0x7FFFFFFF) return DG_ERR_INVALID_ARG;
  return DG_OK;
}

bool aligned(const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

}  // namespace dg

extern "C" size_t dg_moe_route_workspace_size(int64_t T, int E) {
  using namespace dg;
  if (T <= kClusterTokens || E < 1 || E > kMaxExperts) return 0;
  // for all SMs, whatever the cap: another thread may raise it before the call
  const DeviceInfo *d = device_info();
  const int sms = d && d->num_sms > 0 ? d->num_sms : 148;  // (no device: a full B200's)
  return part_bytes(route_blocks(T, E, sms), E);
}

extern "C" int dg_moe_route(const void *logits, int dtype, int64_t T, int E, int64_t ld,
                            int top_k, int normalize, const uint8_t *token_mask, int32_t *idx,
                            float *weights, int32_t *counts, float *loss, int32_t *num_tokens,
                            void *workspace, size_t workspace_bytes, dg_stream_t stream) {
  using namespace dg;
  int rc = check_shape(dtype, T, E, ld, top_k, normalize);
  if (rc) return rc;
  if (!counts || !loss || !num_tokens) return DG_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !idx || !weights)) return DG_ERR_INVALID_ARG;
  if (!aligned(logits, dtype == DG_DTYPE_F32 ? 4 : 2) || !aligned(idx, 4) ||
      !aligned(weights, 4) || !aligned(counts, 4) || !aligned(loss, 4) ||
      !aligned(num_tokens, 4) || !aligned(workspace, 16))
    return DG_ERR_ALIGNMENT;
  rc = check_device();
  if (rc) return rc;
  // (the cap is read once: the workspace is checked for the blocks that are launched)
  const int blocks = route_blocks(T, E, effective_num_sms());
  const bool cluster = T <= kClusterTokens;
  if (!cluster && (!workspace || workspace_bytes < part_bytes(blocks, E)))
    return DG_ERR_WORKSPACE;
  RouteParams p{};
  p.logits = logits;
  p.tokens = T;
  p.ld = ld;
  p.experts = E;
  p.top_k = top_k;
  p.normalize = normalize;
  p.vec = vector_rows(logits, logits, ld, ld, E, dtype == DG_DTYPE_F32 ? 4 : 2);
  p.mask = token_mask;
  p.idx = idx;
  p.weights = weights;
  p.counts = counts;
  p.loss = loss;
  p.num_tokens = num_tokens;
  p.part = static_cast<int2 *>(workspace);
  p.status = device_info()->status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  rc = dtype == DG_DTYPE_F32 ? route_typed<float>(p, blocks, cluster, s)
                             : route_typed<__nv_bfloat16>(p, blocks, cluster, s);
  if (rc || cluster) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kFinishCtas);
  cfg.blockDim = dim3(kFinishThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0] = pdl_attribute();
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kFinishCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_status(cudaLaunchKernelEx(&cfg, moe_route_finish_kernel, p, blocks));
}

extern "C" int dg_moe_route_backward(const void *logits, int dtype, int64_t T, int E, int64_t ld,
                                     int top_k, int normalize, const int32_t *idx,
                                     const float *weights, const int32_t *counts,
                                     const int32_t *num_tokens, const float *dweights,
                                     const float *dloss, void *dlogits, dg_stream_t stream) {
  using namespace dg;
  int rc = check_shape(dtype, T, E, ld, top_k, normalize);
  if (rc) return rc;
  if (T == 0) return DG_OK;
  if (!logits || !idx || !weights || !counts || !num_tokens || !dlogits)
    return DG_ERR_INVALID_ARG;
  const int esz = dtype == DG_DTYPE_F32 ? 4 : 2;
  if (!aligned(logits, esz) || !aligned(dlogits, esz) || !aligned(idx, 4) ||
      !aligned(weights, 4) || !aligned(counts, 4) || !aligned(num_tokens, 4) ||
      !aligned(dweights, 4) || !aligned(dloss, 4))
    return DG_ERR_ALIGNMENT;
  rc = check_device();
  if (rc) return rc;
  RouteBackwardParams p{};
  p.logits = logits;
  p.tokens = T;
  p.ld = ld;
  p.experts = E;
  p.top_k = top_k;
  p.normalize = normalize;
  p.vec = vector_rows(logits, dlogits, ld, E, E, esz);
  p.idx = idx;
  p.weights = weights;
  p.counts = counts;
  p.num_tokens = num_tokens;
  p.dweights = dweights;
  p.dloss = dloss;
  p.dlogits = dlogits;
  const int blocks =
      token_blocks(T, effective_num_sms(), resident_backward(per_lane(E)));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == DG_DTYPE_F32 ? backward_typed<float>(p, blocks, s)
                               : backward_typed<__nv_bfloat16>(p, blocks, s);
}
