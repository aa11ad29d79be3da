// mxfp4.cuh -- what the MXFP4 kernels share: the layout of the scale words, the
// arithmetic of a 32-element group, and the PTX wrappers of the 4-bit
// block-scaled MMA.
//
// MXFP4 (OCP Microscaling Formats specification 1.0): E2M1 elements (0, 0.5,
// 1, 1.5, 2, 3, 4, 6 and their negatives; two per byte, the element of the
// lower K index in the low nibble) with one UE8M0 scale 2^(e - 127) per 32
// consecutive K elements; scale byte 255 is NaN.
//
// These kernels start before the ones ahead of them on the stream have finished
// (programmatic dependent launch), so they read global memory with coherent
// loads (__ldcg, __ldcs) only: __ldg may use lines that were cached before the
// data was written.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "dg.h"

namespace dg {

constexpr int kMxGroup = 32;  // K elements per scale

// Scale words: int32 [ceil(R/128)][ceil(K/128)][32][4]; word (b, p, r, c)
// holds K groups 4p .. 4p+3 of row 128 b + 32 c + r, group 4p + t in bits
// 8t .. 8t+7.  The 512 bytes of a (b, p) block are tcgen05.cp's 32-row x
// 16-byte source as it stands: one bulk copy brings a block to shared
// memory, one tcgen05.cp to TMEM.
constexpr int kMxBlockWords = 128;
constexpr int kMxBlockBytes = 512;

__host__ __device__ constexpr int64_t mx_row_blocks(int64_t rows) { return (rows + 127) / 128; }
__host__ __device__ constexpr int64_t mx_k_words(int64_t k) { return (k + 127) / 128; }

// Index of the scale word of (row, K word p) in a slab of `words` K words.
__device__ __forceinline__ int64_t mx_word_index(int64_t row, int64_t p, int64_t words) {
  const int64_t b = row >> 7;
  const int i = static_cast<int>(row & 127);
  return (b * words + p) * kMxBlockWords + (i & 31) * 4 + (i >> 5);
}

// Scale byte of a group from the FP32 bits of its amax (sign cleared): the
// smallest e >= 0 with 6 * 2^(e - 127) >= amax, so no code saturates.  6 is
// 1.5 * 4: e is amax's exponent field less 2, plus one where its mantissa
// exceeds 1.5.  255 (NaN) for a group that holds an infinity or a NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255u;
  const int e = static_cast<int>(amax_bits >> 23) - 2 + ((amax_bits & 0x7FFFFFu) > 0x400000u);
  return static_cast<uint32_t>(max(e, 0));
}

// 2^(127 - e) as FP32 (e <= 253: always a normal number, the product with
// an element of the group is exact unless it underflows, far below the
// smallest code); 0 for a NaN group, whose codes are then all zero.
__device__ __forceinline__ float mx_inv_scale(uint32_t e) {
  return e == 255u ? 0.0f : __uint_as_float((254u - e) << 23);
}

// 2^(e - 127) as FP32 (e = 0 is the subnormal 2^-127), NaN for 255.
__device__ __forceinline__ float mx_scale_value(uint32_t e) {
  return e == 255u ? __uint_as_float(0x7FFFFFFFu)
                   : __uint_as_float(e == 0u ? 1u << 22 : e << 23);
}

// Eight E2M1 codes (round to nearest, ties to even) of v[0..7], v[0] in the
// lowest nibble.
__device__ __forceinline__ uint32_t mx_encode8(const float v[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The values of eight codes, as four half2 words (exact), lowest nibble first.
__device__ __forceinline__ void mx_decode8(uint32_t codes, uint32_t h[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

// ------------------------------------------------------------------ tcgen05
// True in one lane of a converged warp.  The tcgen05 and TMA instructions of
// an elected lane are issued back to back; behind `lane == 0` the compiler does
// not know that a single thread is active, and each one cost about a hundred
// cycles (4096 x 7168 x 16384: 297 us behind `lane == 0`, 218 us elected).
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// Instruction descriptor of the block-scaled kind::mxf4: A and B E2M1 (format
// 1), both K-major, UE8M0 scales (bit 23), shape M x N x 64; the FP32
// accumulator is implied.
__host__ __device__ constexpr uint32_t idesc_mxf4(int m, int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// D[tmem] (+)= (A 2^sfa)(B 2^sfb)^T over 64 K elements, two scales per row of
// A and of B (one per 32), read from TMEM at sfa / sfb: bytes `half`,
// `half` + 1 (half 0 or 2) of each 32-bit cell, given in the top two address
// bits and in the instruction descriptor (bits 29-30 and 4-5).  One thread.
__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                          uint32_t half, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], "
      "[%6], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc | (half << 29) | (half << 4)), "r"(accumulate),
      "r"(sfa | (half << 30)), "r"(sfb | (half << 30))
      : "memory");
}

// TMEM -> registers, 16 lanes x 16 columns of 32 bits: thread t gets, of column
// block b (8 columns), r[4b], r[4b+1] = lane t/4, columns 2 (t%4), +1, and
// r[4b+2], r[4b+3] the same of lane t/4 + 8 -- the fragments of 8 x 8 matrices
// that stmatrix takes.
__device__ __forceinline__ void tmem_ld_16x256_x2(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

// Four 8 x 8 matrices of 16-bit elements, transposed, to shared memory: thread
// 8m + i gives the address of the 16 bytes that hold column i of matrix m.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b,
                                                  uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                   addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// The CTA-pair form: M = 256, rows 0-127 of A, of D and A's scales in rank 0,
// rows 128-255 in rank 1; B split along N between the two CTAs' shared memory,
// its scales whole in both CTAs' TMEM.  Issued by one thread of rank 0.
__device__ __forceinline__ void umma_mxf4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                               uint32_t half, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], "
      "[%6], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc | (half << 29) | (half << 4)), "r"(accumulate),
      "r"(sfa | (half << 30)), "r"(sfb | (half << 30))
      : "memory");
}

// tmem_cp_32x128b_x4 in both CTAs of the pair, each from its own shared memory
// (the same offset) to its own TMEM.  Issued by rank 0.
__device__ __forceinline__ void tmem_cp_32x128b_x4_pair(uint32_t taddr, uint64_t src_desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(src_desc)
               : "memory");
}

}  // namespace dg
