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
#include "host.h"
#include "internal.h"
#include "mxfp4.cuh"
#include "ptx.cuh"

namespace dg {

namespace {

constexpr int kThreads = 256;

// A lane's consecutive elements of a row, as loaded, with what the row kernel asks
// of them: the FP32 bits of the largest magnitude (a NaN counts as the
// largest), and the codes of the elements times `inv`.  Compares, selects and
// byte moves (the ALU pipe) bound the kernel before HBM does, so they are what
// is kept few.
template <typename T>
struct Piece;

template <>
struct Piece<float> {
  static constexpr int kElems = 8;
  float v[8];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  }
  __device__ __forceinline__ void load(const float *p) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  static __device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
  }
  __device__ __forceinline__ uint32_t amax_bits() const {
    const float m = max3(max3(v[0], v[1], v[2]), max3(v[3], v[4], v[5]), max3(v[6], v[7], v[7]));
    return __float_as_uint(m);
  }
  __device__ __forceinline__ void encode(float inv, uint32_t *codes) const {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[i] * inv;
    codes[0] = mx_encode8(w);
  }
};

template <>
struct Piece<__nv_bfloat16> {
  static constexpr int kElems = 16;
  uint32_t v[8];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0;
  }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p));
    const uint4 b = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  // the larger magnitudes of two pairs (their signs end up mixed)
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ __forceinline__ uint32_t amax_bits() const {
    const uint32_t m = max2(max2(max2(v[0], v[1]), max2(v[2], v[3])),
                            max2(max2(v[4], v[5]), max2(v[6], v[7]))) & 0x7FFF7FFFu;
    return max(m << 16, m & 0xFFFF0000u);
  }
  __device__ __forceinline__ void encode(float inv, uint32_t *codes) const {
    float w[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[2 * i] = __uint_as_float(v[i] << 16) * inv;
      w[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u) * inv;
    }
    codes[0] = mx_encode8(w);
    codes[1] = mx_encode8(w + 8);
  }
};

// Rows.  A warp takes a chunk of a row: kPasses passes of 32 lanes' pieces, all
// loaded before the first is used.  grid: (chunks, row groups of 8 warps,
// batch), the last two strided.  Rows past M up to the end of the last 128-row
// block only get zero scales.
constexpr int kPasses = 2;

template <typename T>
__global__ void __launch_bounds__(kThreads)
quantize_mxfp4_rows_kernel(const T *__restrict__ x, int batch, int M, int K, int64_t ld_x,
                           uint8_t *__restrict__ q, uint32_t *__restrict__ sf) {
  using P = Piece<T>;
  constexpr int kLanes = kMxGroup / P::kElems;   // lanes per group
  constexpr int kPass = 32 * P::kElems;          // elements per pass
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int words = (K + 127) / 128, rows = (M + 127) / 128 * 128;
  const int k0 = blockIdx.x * (kPass * kPasses) + lane * P::kElems;
  for (int b = blockIdx.z; b < batch; b += gridDim.z) {
    for (int r = blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5); r < rows;
         r += gridDim.y * (kThreads / 32)) {
      const int64_t row = static_cast<int64_t>(b) * M + r;
      const bool live = r < M;
      P piece[kPasses];
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        if (live && k0 + i * kPass < K)
          piece[i].load(x + row * ld_x + k0 + i * kPass);
        else
          piece[i].clear();
      }
      uint8_t *qrow = q + row * (K / 2) + k0 / 2;
      uint32_t *srow = sf + (static_cast<int64_t>(b) * (rows / 128) + (r >> 7)) * words *
                                kMxBlockWords + (r & 31) * 4 + ((r & 127) >> 5);
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        uint32_t a = piece[i].amax_bits();
#pragma unroll
        for (int o = 1; o < kLanes; o *= 2) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
        const uint32_t e = mx_scale_byte(a);
        uint32_t codes[P::kElems / 8];
        piece[i].encode(mx_inv_scale(e), codes);
        if (e == 255u) {  // (the codes of a NaN group are zero)
#pragma unroll
          for (int j = 0; j < P::kElems / 8; ++j) codes[j] = 0;
        }
        if (live && k0 + i * kPass < K) {
          if constexpr (P::kElems == 16)
            *reinterpret_cast<uint2 *>(qrow + i * (kPass / 2)) = make_uint2(codes[0], codes[1]);
          else
            *reinterpret_cast<uint32_t *>(qrow + i * (kPass / 2)) = codes[0];
        }
        // the four groups of a scale word sit in 4 kLanes lanes; groups past K
        // and rows past M are zero (their amax is)
        uint32_t w = e << (8 * ((lane / kLanes) & 3));
        w |= __shfl_xor_sync(0xffffffffu, w, kLanes);
        w |= __shfl_xor_sync(0xffffffffu, w, 2 * kLanes);
        const int p = (k0 + i * kPass) / 128;
        if (lane % (4 * kLanes) == 0 && p < words)
          srow[static_cast<int64_t>(p) * kMxBlockWords] = w;
      }
    }
  }
}

// Columns: x [K][M] (row stride ld_x), the operand's row m is column m of x.
// A block takes 64 columns x 256 K elements: each warp one group of 32 K
// rows, each thread two adjacent columns of it (a warp reads 64 consecutive
// columns of a row).  The codes are turned in shared memory, so that every
// operand row leaves as 128 contiguous bytes, and so are the scale bytes.
constexpr int kTCols = 64, kTK = 256;

// One group of two adjacent columns, as loaded.  `two`: both columns exist and
// their pairs are aligned, so a row is one load.
template <typename T>
struct Columns;

template <>
struct Columns<float> {
  float v[2][kMxGroup];
  __device__ __forceinline__ void load(const float *p, int64_t ld, bool two, bool c0, bool c1) {
    if (two) {
#pragma unroll
      for (int i = 0; i < kMxGroup; ++i) {
        const float2 t = __ldcs(reinterpret_cast<const float2 *>(p + i * ld));
        v[0][i] = t.x;
        v[1][i] = t.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kMxGroup; ++i) {
        v[0][i] = c0 ? __ldcs(p + i * ld) : 0.0f;
        v[1][i] = c1 ? __ldcs(p + i * ld + 1) : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void amax_bits(uint32_t a[2]) const {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float m = v[c][0];
#pragma unroll
      for (int i = 1; i < kMxGroup; i += 2)
        m = Piece<float>::max3(m, v[c][i], v[c][i + 1 < kMxGroup ? i + 1 : i]);
      a[c] = __float_as_uint(m);
    }
  }
  template <int C>
  __device__ __forceinline__ float get(int i) const { return v[C][i]; }
};

template <>
struct Columns<__nv_bfloat16> {
  uint32_t v[kMxGroup];  // column 0 in the low half
  __device__ __forceinline__ void load(const __nv_bfloat16 *p, int64_t ld, bool two, bool c0,
                                       bool c1) {
    if (two) {
#pragma unroll
      for (int i = 0; i < kMxGroup; ++i)
        v[i] = __ldcs(reinterpret_cast<const uint32_t *>(p + i * ld));
    } else {
      const unsigned short *s = reinterpret_cast<const unsigned short *>(p);
#pragma unroll
      for (int i = 0; i < kMxGroup; ++i)
        v[i] = (c0 ? __ldcs(s + i * ld) : 0u) |
               (c1 ? static_cast<uint32_t>(__ldcs(s + i * ld + 1)) << 16 : 0u);
    }
  }
  __device__ __forceinline__ void amax_bits(uint32_t a[2]) const {
    uint32_t m = Piece<__nv_bfloat16>::max2(v[0], v[1]);
#pragma unroll
    for (int i = 2; i < kMxGroup; ++i) m = Piece<__nv_bfloat16>::max2(m, v[i]);
    m &= 0x7FFF7FFFu;
    a[0] = m << 16;
    a[1] = m & 0xFFFF0000u;
  }
  template <int C>
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(C == 0 ? v[i] << 16 : v[i] & 0xFFFF0000u);
  }
};

// The codes and the scale byte of column C of a group, to shared memory.
template <int C, typename T>
__device__ __forceinline__ void encode_column(const Columns<T> &cols, uint32_t amax,
                                              uint8_t *codes, uint8_t *scale) {
  const uint32_t e = mx_scale_byte(amax);
  const float inv = mx_inv_scale(e);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = cols.template get<C>(8 * j + i) * inv;
    w[j] = e == 255u ? 0u : mx_encode8(f);  // (the codes of a NaN group are zero)
  }
  *reinterpret_cast<uint4 *>(codes) = make_uint4(w[0], w[1], w[2], w[3]);
  *scale = static_cast<uint8_t>(e);
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
    const bool live = k0 < K;  // K % 32 == 0: a whole group or none
    Columns<T> cols;
    cols.load(x + k0 * ld_x + m, ld_x, vec != 0 && live && c1, live && c0, live && c1);
    uint32_t a[2];
    cols.amax_bits(a);
    encode_column<0>(cols, a[0], &s_codes[2 * lane][warp * 16], &s_scale[2 * lane][warp]);
    encode_column<1>(cols, a[1], &s_codes[2 * lane + 1][warp * 16], &s_scale[2 * lane + 1][warp]);
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

// Read-back: sixteen codes (half a group) per lane, grid as for the rows.
// In BF16 the products with the scale are exact and two at a time: a code's FP16
// bits moved down three places are a BF16 number 2^-112 times its value, so two
// products by powers of two that are BF16 numbers give the result.
template <typename T>
__device__ __forceinline__ void decode_store(T *p, const uint32_t codes[2], uint32_t e);
template <>
__device__ __forceinline__ void decode_store<float>(float *p, const uint32_t codes[2],
                                                    uint32_t e) {
  const float s = mx_scale_value(e);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t h[4];
    mx_decode8(codes[c], h);
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
      const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&h[j + 1]));
      __stcs(reinterpret_cast<float4 *>(p + 8 * c + 2 * j),
             make_float4(f.x * s, f.y * s, g.x * s, g.y * s));
    }
  }
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <>
__device__ __forceinline__ void decode_store<__nv_bfloat16>(__nv_bfloat16 *p,
                                                            const uint32_t codes[2], uint32_t e) {
  constexpr uint32_t k2p112 = ((112u + 127u) << 7) * 0x10001u;
  // 2^(e - 127) as BF16: its bits are FP32's upper half
  const uint32_t s = (__float_as_uint(mx_scale_value(e)) >> 16) * 0x10001u;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t h[4];
    mx_decode8(codes[c], h);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      h[j] = mul_bf16x2(mul_bf16x2(((h[j] >> 3) & 0x0FFF0FFFu) | (h[j] & 0x80008000u), k2p112),
                        s);
    __stcs(reinterpret_cast<uint4 *>(p) + c, make_uint4(h[0], h[1], h[2], h[3]));
  }
}

constexpr int kReadPass = 32 * 16;  // elements a warp reads back

template <typename T>
__global__ void __launch_bounds__(kThreads)
dequantize_mxfp4_kernel(const uint8_t *__restrict__ q, const uint32_t *__restrict__ sf, int batch,
                        int M, int K, T *__restrict__ y, int64_t ld_y) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int words = (K + 127) / 128, blocks = (M + 127) / 128;
  const int k = blockIdx.x * kReadPass + lane * 16;
  for (int b = blockIdx.z; b < batch; b += gridDim.z) {
    for (int r = blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5); r < M;
         r += gridDim.y * (kThreads / 32)) {
      const int64_t row = static_cast<int64_t>(b) * M + r;
      const uint32_t *srow = sf + (static_cast<int64_t>(b) * blocks + (r >> 7)) * words *
                                      kMxBlockWords + (r & 31) * 4 + ((r & 127) >> 5);
      if (k < K) {
        const uint2 code = __ldcs(reinterpret_cast<const uint2 *>(q + row * (K / 2) + k / 2));
        const uint32_t word = __ldcg(srow + static_cast<int64_t>(k / 128) * kMxBlockWords);
        const uint32_t c[2] = {code.x, code.y};
        decode_store<T>(y + row * ld_y + k, c, (word >> (8 * ((lane >> 1) & 3))) & 255u);
      }
    }
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// (chunks of a row, groups of 8 rows, batch); the kernels stride over what a
// grid's second and third dimensions cannot hold.
dim3 row_grid(int64_t K, int64_t chunk, int64_t rows, int64_t batch) {
  const int64_t y = (rows + kThreads / 32 - 1) / (kThreads / 32);
  return dim3(static_cast<unsigned>((K + chunk - 1) / chunk),
              static_cast<unsigned>(y < 65535 ? y : 65535),
              static_cast<unsigned>(batch < 65535 ? batch : 65535));
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
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, args...));
}

int check_device() {
  const DeviceInfo *d = device_info();
  if (!d) return DG_ERR_CUDA;
  return d->ok ? DG_OK : DG_ERR_UNSUPPORTED_ARCH;
}

// Sizes past which a coordinate (and a grid's stride past it) would leave 31 bits,
// or an index in elements 62.
bool too_large(int64_t batch, int64_t rows, int64_t cols) {
  constexpr int64_t kMost = 0x7FF00000;
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
  const int64_t rows = mx_row_blocks(M) * 128;
  const int b = static_cast<int>(batch), m = static_cast<int>(M), k = static_cast<int>(K);
  if (x_dtype == DG_DTYPE_F32)
    return launch(quantize_mxfp4_rows_kernel<float>,
                  row_grid(K, 32 * Piece<float>::kElems * kPasses, rows, batch), s,
                  static_cast<const float *>(x), b, m, k, ld_x, q, w);
  return launch(quantize_mxfp4_rows_kernel<__nv_bfloat16>,
                row_grid(K, 32 * Piece<__nv_bfloat16>::kElems * kPasses, rows, batch), s,
                static_cast<const __nv_bfloat16 *>(x), b, m, k, ld_x, q, w);
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
  const dim3 grid = row_grid(K, kReadPass, M, batch);
  const int b = static_cast<int>(batch), m = static_cast<int>(M), k = static_cast<int>(K);
  if (y_dtype == DG_DTYPE_F32)
    return launch(dequantize_mxfp4_kernel<float>, grid, s, q, w, b, m, k,
                  static_cast<float *>(y), ld_y);
  return launch(dequantize_mxfp4_kernel<__nv_bfloat16>, grid, s, q, w, b, m, k,
                static_cast<__nv_bfloat16 *>(y), ld_y);
}
