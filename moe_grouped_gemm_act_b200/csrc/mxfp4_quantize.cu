// mxfp4_quantize.cu -- MXFP4 quantizers (of the rows of a matrix, or of its
// columns) and the read-back of an MXFP4 operand, with their C entry points.
//
// Per group of 32:  amax = max |x|;  scale = the smallest 2^e with
// 6 * 2^e >= amax (the power-of-two rule of DG_SCALE_POW2, with E2M1's 6 in
// place of 448);  code = E2M1_RNE(x / scale), the quotient exact.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dg.h"
#include "internal.h"
#include "mxfp4.cuh"
#include "ptx.cuh"

namespace dg {

namespace {

constexpr int kThreads = 256;

// Eight consecutive elements (16-byte aligned) as FP32.
__device__ __forceinline__ void load8(const float *p, float v[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float v[8]) {
  const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// Rows: four lanes per group, eight elements per lane, so a warp takes 256
// consecutive elements of a row in one pass (contiguous 16-byte loads, one
// contiguous 128-byte code store) and two scale words.  An item is a row's
// chunk of kPasses passes, whose loads are all issued before the first use.
// Rows past M up to the end of the last 128-row block only get zero scales.
constexpr int kPasses = 4;

template <typename T>
__global__ void __launch_bounds__(kThreads)
quantize_mxfp4_rows_kernel(const T *__restrict__ x, int64_t batch, int64_t M, int64_t K,
                           int64_t ld_x, uint8_t *__restrict__ q, uint32_t *__restrict__ sf) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  const int64_t chunks = (K + 256 * kPasses - 1) / (256 * kPasses);
  const int64_t words = mx_k_words(K);
  const int64_t rows = mx_row_blocks(M) * 128;  // per batch, with the padding
  const int64_t slab_words = mx_row_blocks(M) * words * kMxBlockWords;
  const int64_t items = batch * rows * chunks;
  for (int64_t item = warp; item < items; item += nwarps) {
    const int64_t row = item / chunks, k0 = (item - row * chunks) * (256 * kPasses);
    const int64_t b = row / rows, r = row - b * rows;
    const bool live = r < M;
    const T *src = x + (b * M + r) * ld_x;
    float v[kPasses][8];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int64_t k = k0 + i * 256 + lane * 8;
      if (live && k < K) {
        load8(src + k, v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int64_t k = k0 + i * 256 + lane * 8;
      uint32_t a = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
      const uint32_t e = mx_scale_byte(a);
      const float inv = mx_inv_scale(e);
      if (live && k < K) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = e == 255u ? 0.0f : v[i][j] * inv;
        *reinterpret_cast<uint32_t *>(q + ((b * M + r) * K + k) / 2) = mx_encode8(v[i]);
      }
      // the four groups of a scale word sit in 16 lanes; groups past K and
      // rows past M are zero (their amax is)
      uint32_t w = e << (8 * ((lane >> 2) & 3));
      w |= __shfl_xor_sync(0xffffffffu, w, 4);
      w |= __shfl_xor_sync(0xffffffffu, w, 8);
      const int64_t p = (k0 + i * 256) / 128 + (lane >> 4);
      if ((lane & 15) == 0 && p < words)
        sf[b * slab_words + mx_word_index(r, p, words)] = w;
    }
  }
}

// Columns: x [K][M] (row stride ld_x), the operand's row m is column m of x.
// A block takes 64 columns x 256 K elements: each warp one group of 32 K
// rows, each thread two adjacent columns of it (a warp reads 64 consecutive
// columns of a row).  The codes are turned in shared memory, so that every
// operand row leaves as 128 contiguous bytes, and so are the scale bytes.
constexpr int kTCols = 64, kTK = 256;

template <typename T>
__device__ __forceinline__ void load_pair(const T *p, bool vec, bool c0, bool c1, float &a,
                                          float &b);
template <>
__device__ __forceinline__ void load_pair<float>(const float *p, bool vec, bool c0, bool c1,
                                                 float &a, float &b) {
  if (vec && c1) {
    const float2 t = __ldcs(reinterpret_cast<const float2 *>(p));
    a = t.x;
    b = t.y;
  } else {
    a = c0 ? __ldcs(p) : 0.0f;
    b = c1 ? __ldcs(p + 1) : 0.0f;
  }
}
template <>
__device__ __forceinline__ void load_pair<__nv_bfloat16>(const __nv_bfloat16 *p, bool vec,
                                                         bool c0, bool c1, float &a, float &b) {
  uint32_t t = 0;
  if (vec && c1) {
    t = __ldcs(reinterpret_cast<const uint32_t *>(p));
  } else {
    const unsigned short *s = reinterpret_cast<const unsigned short *>(p);
    if (c0) t = __ldcs(s);
    if (c1) t |= static_cast<uint32_t>(__ldcs(s + 1)) << 16;
  }
  a = __uint_as_float(t << 16);
  b = __uint_as_float(t & 0xFFFF0000u);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
quantize_mxfp4_cols_kernel(const T *__restrict__ x, int64_t M, int64_t K, int64_t ld_x,
                           uint8_t *__restrict__ q, uint32_t *__restrict__ sf, int vec) {
  __shared__ __align__(16) uint8_t s_codes[kTCols][kTK / 2 + 16];
  __shared__ __align__(4) uint8_t s_scale[kTCols][kTK / kMxGroup];
  grid_launch_dependents();
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t words = mx_k_words(K);
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kTCols;
  const int64_t m = m0 + 2 * lane;
  const bool c0 = m < M, c1 = m + 1 < M;
  for (int64_t kt = static_cast<int64_t>(blockIdx.y) * kTK; kt < K;
       kt += static_cast<int64_t>(gridDim.y) * kTK) {
    const int64_t k0 = kt + warp * kMxGroup;
    float v[2][kMxGroup];
    const bool live = k0 < K;  // K % 32 == 0: a whole group or none
#pragma unroll
    for (int i = 0; i < kMxGroup; ++i)
      load_pair<T>(x + (k0 + i) * ld_x + m, vec != 0, live && c0, live && c1, v[0][i], v[1][i]);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t a = 0;
#pragma unroll
      for (int i = 0; i < kMxGroup; ++i) a = max(a, __float_as_uint(v[c][i]) & 0x7FFFFFFFu);
      const uint32_t e = mx_scale_byte(a);
      const float inv = mx_inv_scale(e);
#pragma unroll
      for (int i = 0; i < kMxGroup; ++i) v[c][i] = e == 255u ? 0.0f : v[c][i] * inv;
      uint4 w;
      w.x = mx_encode8(v[c]);
      w.y = mx_encode8(v[c] + 8);
      w.z = mx_encode8(v[c] + 16);
      w.w = mx_encode8(v[c] + 24);
      *reinterpret_cast<uint4 *>(&s_codes[2 * lane + c][warp * 16]) = w;
      s_scale[2 * lane + c][warp] = static_cast<uint8_t>(e);
    }
    __syncthreads();
    // codes: 8 threads per operand row, 16 bytes (one group) each
    for (int i = threadIdx.x; i < kTCols * 8; i += kThreads) {
      const int row = i >> 3, g = i & 7;
      if (m0 + row < M && kt + g * kMxGroup < K)
        *reinterpret_cast<uint4 *>(q + ((m0 + row) * K + kt) / 2 + g * 16) =
            *reinterpret_cast<const uint4 *>(&s_codes[row][g * 16]);
    }
    // scale words, zero past M up to the end of the last 128-row block
    if (threadIdx.x < kTCols * 2) {
      const int row = threadIdx.x >> 1;
      const int64_t p = kt / 128 + (threadIdx.x & 1);
      if (p < words)
        sf[mx_word_index(m0 + row, p, words)] =
            *reinterpret_cast<const uint32_t *>(&s_scale[row][4 * (threadIdx.x & 1)]);
    }
    __syncthreads();
  }
}

// Read-back: eight codes per lane, a warp 256 consecutive elements of a row.
template <typename T>
__device__ __forceinline__ void store8(T *p, const float v[8]);
template <>
__device__ __forceinline__ void store8<float>(float *p, const float v[8]) {
  __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16 *p, const float v[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // exact: three significant bits (NaN stays NaN)
    const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&t);
  }
  __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
dequantize_mxfp4_kernel(const uint8_t *__restrict__ q, const uint32_t *__restrict__ sf,
                        int64_t batch, int64_t M, int64_t K, T *__restrict__ y, int64_t ld_y) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  const int64_t chunks = (K + 256 * kPasses - 1) / (256 * kPasses);
  const int64_t words = mx_k_words(K);
  const int64_t slab_words = mx_row_blocks(M) * words * kMxBlockWords;
  const int64_t items = batch * M * chunks;
  for (int64_t item = warp; item < items; item += nwarps) {
    const int64_t row = item / chunks, k0 = (item - row * chunks) * (256 * kPasses);
    const int64_t b = row / M, r = row - b * M;
    uint32_t code[kPasses], word[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int64_t k = k0 + i * 256 + lane * 8;
      code[i] = word[i] = 0;
      if (k < K) {
        code[i] = __ldcs(reinterpret_cast<const uint32_t *>(q + (row * K + k) / 2));
        word[i] = __ldg(sf + b * slab_words + mx_word_index(r, k / 128, words));
      }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int64_t k = k0 + i * 256 + lane * 8;
      if (k >= K) break;
      const float s = mx_scale_value((word[i] >> (8 * ((lane >> 2) & 3))) & 255u);
      uint32_t h[4];
      mx_decode8(code[i], h);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
        v[2 * j] = f.x * s;
        v[2 * j + 1] = f.y * s;
      }
      store8<T>(y + row * ld_y + k, v);
    }
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A grid of warps over `items`, at most eight resident blocks per SM.
unsigned warp_grid(int64_t items, int num_sms) {
  const int64_t want = (items + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t most = static_cast<int64_t>(num_sms) * 8;
  return static_cast<unsigned>(want < most ? want : most);
}

template <typename... P, typename... A>
int launch(void (*kern)(P...), dim3 grid, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

int check_device() {
  const DeviceInfo *d = device_info();
  if (!d) return DG_ERR_CUDA;
  return d->ok ? DG_OK : DG_ERR_UNSUPPORTED_ARCH;
}

// Sizes past which an index in elements would leave 62 bits.
bool too_large(int64_t batch, int64_t rows, int64_t cols) {
  constexpr int64_t kMost = int64_t(1) << 31;
  return batch > kMost || rows > kMost || cols > kMost ||
         (rows > 0 && cols > 0 && batch > (int64_t(1) << 62) / rows / cols);
}

}  // namespace

}  // namespace dg

extern "C" int dg_quantize_mxfp4(const void *x, int x_dtype, int64_t batch, int64_t M, int64_t K,
                                 int64_t ld_x, int transpose, uint8_t *q, int32_t *sf,
                                 dg_stream_t stream) {
  using namespace dg;
  if (x_dtype != DG_DTYPE_F32 && x_dtype != DG_DTYPE_BF16) return DG_ERR_INVALID_ARG;
  if (transpose != 0 && transpose != 1) return DG_ERR_INVALID_ARG;
  if (batch < 1 || M < 0 || K <= 0 || K % kMxGroup != 0) return DG_ERR_INVALID_ARG;
  if (too_large(batch, M, K) || ld_x > (int64_t(1) << 31)) return DG_ERR_INVALID_ARG;
  if (ld_x < (transpose ? M : K)) return DG_ERR_INVALID_ARG;
  if (transpose && batch != 1) return DG_ERR_INVALID_ARG;
  if (M == 0) return DG_OK;
  if (!x || !q || !sf) return DG_ERR_INVALID_ARG;
  const int esz = x_dtype == DG_DTYPE_F32 ? 4 : 2;
  if (!aligned16(q) || !aligned16(sf)) return DG_ERR_ALIGNMENT;
  if (transpose ? reinterpret_cast<uintptr_t>(x) % esz != 0
                : (!aligned16(x) || (ld_x * esz) % 16 != 0))
    return DG_ERR_ALIGNMENT;
  const int rc = check_device();
  if (rc) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint32_t *w = reinterpret_cast<uint32_t *>(sf);
  if (transpose) {
    const int vec = ld_x % 2 == 0 && reinterpret_cast<uintptr_t>(x) % (2 * esz) == 0;
    // whole 128-row blocks of scales are written
    const int64_t kt = (K + kTK - 1) / kTK;
    const dim3 grid(static_cast<unsigned>(mx_row_blocks(M) * (128 / kTCols)),
                    static_cast<unsigned>(kt < 65535 ? kt : 65535));
    if (x_dtype == DG_DTYPE_F32)
      return launch(quantize_mxfp4_cols_kernel<float>, grid, s, static_cast<const float *>(x), M,
                    K, ld_x, q, w, vec);
    return launch(quantize_mxfp4_cols_kernel<__nv_bfloat16>, grid, s,
                  static_cast<const __nv_bfloat16 *>(x), M, K, ld_x, q, w, vec);
  }
  const int64_t items =
      batch * mx_row_blocks(M) * 128 * ((K + 256 * kPasses - 1) / (256 * kPasses));
  const dim3 grid(warp_grid(items, effective_num_sms()));
  if (x_dtype == DG_DTYPE_F32)
    return launch(quantize_mxfp4_rows_kernel<float>, grid, s, static_cast<const float *>(x),
                  batch, M, K, ld_x, q, w);
  return launch(quantize_mxfp4_rows_kernel<__nv_bfloat16>, grid, s,
                static_cast<const __nv_bfloat16 *>(x), batch, M, K, ld_x, q, w);
}

extern "C" int dg_dequantize_mxfp4(const uint8_t *q, const int32_t *sf, int64_t batch, int64_t M,
                                   int64_t K, void *y, int y_dtype, int64_t ld_y,
                                   dg_stream_t stream) {
  using namespace dg;
  if (y_dtype != DG_DTYPE_F32 && y_dtype != DG_DTYPE_BF16) return DG_ERR_INVALID_ARG;
  if (batch < 1 || M < 0 || K <= 0 || K % kMxGroup != 0 || ld_y < K) return DG_ERR_INVALID_ARG;
  if (too_large(batch, M, ld_y)) return DG_ERR_INVALID_ARG;
  if (M == 0) return DG_OK;
  if (!q || !sf || !y) return DG_ERR_INVALID_ARG;
  const int esz = y_dtype == DG_DTYPE_F32 ? 4 : 2;
  if (!aligned16(q) || !aligned16(sf) || !aligned16(y) || (ld_y * esz) % 16 != 0)
    return DG_ERR_ALIGNMENT;
  const int rc = check_device();
  if (rc) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const uint32_t *w = reinterpret_cast<const uint32_t *>(sf);
  const dim3 grid(
      warp_grid(batch * M * ((K + 256 * kPasses - 1) / (256 * kPasses)), effective_num_sms()));
  if (y_dtype == DG_DTYPE_F32)
    return launch(dequantize_mxfp4_kernel<float>, grid, s, q, w, batch, M, K,
                  static_cast<float *>(y), ld_y);
  return launch(dequantize_mxfp4_kernel<__nv_bfloat16>, grid, s, q, w, batch, M, K,
                static_cast<__nv_bfloat16 *>(y), ld_y);
}
