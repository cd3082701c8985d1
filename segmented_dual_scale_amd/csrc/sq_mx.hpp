// sq_mx.hpp -- the microscaled 4-bit format (MXFP4): blocks of 32 neighbours
// along K share a power of two, each element is a 4-bit float (sign, 2 bits of
// exponent, 1 of mantissa: 0, 0.5, 1, 1.5, 2, 3, 4, 6) times it.  The format is
// the public one of the OCP Microscaling Formats specification, version 1.0.
// Here: the launch interface of mx_kernels.hip and gemm_mx.hip, and the device
// helpers of every kernel that writes the format.
//
// A matrix of R rows (tokens of an activation, output columns of a weight) and
// K columns is kept in the operand order of the 16x16x128 matrix-core
// instruction, rows and columns padded to whole tiles:
//   codes   tiles of 16 rows x 128 k, 1 KiB, row tiles outermost.  Lane 16 g + j
//           of a wave owns bytes 16 (16 g + j) .. + 15: block g of row j, two
//           codes a byte, the first in the low half.
//   scales  tiles of 16 rows x 512 k, 256 bytes, row tiles outermost.  Lane
//           16 g + j owns 4 bytes, byte s the power of two (biased by 127) of
//           block g of row j in the s-th 128 of the 512: one load feeds four
//           instructions, which pick their byte.
// Both operands then arrive as one contiguous load per instruction, from
// memory or from LDS, and every lane has its own block's scale.
#pragma once

#include "sq_rows.hpp"

namespace sq {

constexpr int kMxTileRows = 16, kMxTileK = 128, kMxScaleK = 512;

__host__ __device__ inline int64_t mx_tiles_k(int64_t K) { return (K + kMxTileK - 1) / kMxTileK; }
__host__ __device__ inline int64_t mx_scale_tiles_k(int64_t K) {
  return (K + kMxScaleK - 1) / kMxScaleK;
}
inline int64_t mx_row_tiles(int64_t R) { return (R + kMxTileRows - 1) / kMxTileRows; }
inline int64_t mx_code_bytes(int64_t R, int64_t K) {
  return mx_row_tiles(R) * mx_tiles_k(K) * 1024;
}
inline int64_t mx_scale_bytes(int64_t R, int64_t K) {
  return mx_row_tiles(R) * mx_scale_tiles_k(K) * 256;
}

// act: 0 none, 1 SiLU, 2 GELU
hipError_t launch_quantize_mx(const uint16_t *x, int64_t M, int64_t K, int64_t ld_x, int32_t act,
                              uint8_t *codes, uint8_t *scales, hipStream_t s);
hipError_t launch_quantize_weight_mx(const float *w, int64_t K, int64_t N, int64_t ld_w,
                                     uint8_t *codes, uint8_t *scales, hipStream_t s);
hipError_t launch_unpack_mx(const uint8_t *codes, const uint8_t *scales, int64_t R, int64_t K,
                            float *x, int64_t ld_x, hipStream_t s);

struct MxGemmProblem {
  int64_t M, N, K;
  const uint8_t *x, *x_scale;  // MXFP4 [M][K]
  const uint8_t *w, *w_scale;  // MXFP4 [N][K]
  uint16_t *y;
  int64_t ld_y;
};

hipError_t launch_gemm_mx(const MxGemmProblem &p, hipStream_t s);
// Its form for more than 16 rows: the tile shape in its table that costs least, or -1
// for the kernel that splits K over its waves.
int mx_choice(int64_t M, int64_t N, int64_t K);
// Whether the product of bf16 input of this size quantises it itself: with any
// activation; with none.  And that product (x and x_scale of the problem unused).
bool mx_quantises_inside(int64_t M, int64_t K);
bool mx_rows_inside(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm_mx_bf16(const MxGemmProblem &p, const uint16_t *z, int64_t ld_z, int32_t act,
                               hipStream_t s);

// ------------------------------------------------------- device helpers --
// The biased power of two of a block whose largest magnitude has these bf16 or
// fp32 exponent bits (0..255): floor(log2 amax) - 2, so that the largest
// element lies in [4, 8) of the scale and saturates at 6 from 7 on.  A block
// with an infinity or a NaN (255) gets 255, which is NaN: so is every product
// with it.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t exp_bits) {
  return exp_bits == 255u ? 255u : exp_bits < 2u ? 0u : exp_bits - 2u;
}

// 1 / scale, exact for every byte but 255, whose codes do not matter.
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// Eight scaled values -> eight codes, the first in the lowest four bits; round
// to nearest, ties to the even code, magnitudes above 6 become 6.
__device__ __forceinline__ uint32_t mx_codes8(const float f[8]) {
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[0], f[1], 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[2], f[3], 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[4], f[5], 1.0f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[6], f[7], 1.0f, 3);
  return c;
}

// Largest value over the four lanes of a quad, in each of them.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
#define SQ_DPP(ctrl) (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xf, 0xf, false)
  v = max(v, SQ_DPP(0xB1));  // quad_perm [1,0,3,2]
  v = max(v, SQ_DPP(0x4E));  // quad_perm [2,3,0,1]
#undef SQ_DPP
  return v;
}

// Byte offsets of block `kb` (32 k) of a row.
__device__ __forceinline__ int64_t mx_code_at(const MxOut &o, int64_t row, int kb) {
  return (((row >> 4) * o.kt + (kb >> 2)) << 10) + (((kb & 3) << 4 | (int)(row & 15)) << 4);
}

__device__ __forceinline__ int64_t mx_scale_at(const MxOut &o, int64_t row, int kb) {
  return (((row >> 4) * o.ks + (kb >> 4)) << 8) + (((kb & 3) << 4 | (int)(row & 15)) << 2) +
         (kb >> 2 & 3);
}

// Bf16 piece v (8 elements at column k, a multiple of 8) of a row: the lanes of
// a quad hold one block and all call this.
__device__ __forceinline__ uint32_t mx_piece(v4u v, uint32_t &byte) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) top = max(top, max(v[j] & 0x7fffu, v[j] >> 16 & 0x7fffu));
  byte = mx_scale_byte(quad_max(top) >> 7);
  // the conversion divides by the power of two in its scale's exponent bits (2^-127
  // for 0), exactly, and rounds as mx_codes8
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const float scale = __uint_as_float(byte << 23);
  const uint32_t x0 = v[0], x1 = v[1], x2 = v[2], x3 = v[3];
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(v2bf, x0), scale, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(v2bf, x1), scale, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(v2bf, x2), scale, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(v2bf, x3), scale, 3);
  return c;
}

__device__ __forceinline__ void mx_emit8(const MxOut &o, int64_t row, int k, v4u v) {
  uint32_t byte;
  const uint32_t c = mx_piece(v, byte);
  const int kb = k >> 5, q = k >> 3 & 3;
  *reinterpret_cast<uint32_t *>(o.codes + mx_code_at(o, row, kb) + 4 * q) = c;
  if (q == 0) o.scales[mx_scale_at(o, row, kb)] = (uint8_t)byte;
}

}  // namespace sq
