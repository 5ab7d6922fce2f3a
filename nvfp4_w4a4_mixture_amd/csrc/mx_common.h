// Device helpers of the MXFP4 kernels (OCP Microscaling: blocks of 32 E2M1
// elements with one E8M0 scale).
//
// E8M0 byte b stands for 2^(b - 127), b = 255 for NaN.  A block's byte is
// floor(log2(amax)) - 2 + 127 (2 = the exponent of the largest E2M1 value, 6),
// so amax / scale lies in [4, 8) and what exceeds 6 saturates.
//
// Operand fragments.  The scaled FP4 MFMA of 32 x 32 x 64 takes, per lane l,
// 32 elements (16 bytes) of row l % 32: one MX block, with that block's scale
// byte in one of the four bytes of a scale register.  The order of the blocks
// along K is free as long as both operands agree; here the 256 columns of one
// column group (8 blocks) are four MFMA steps, and lane half f = l / 32 takes
// block 4 f + s at step s.  A lane's four blocks of a column group are then 64
// consecutive bytes of codes, and their scale bytes one dword.
//
// Result rows.  Lane l holds column l % 32 of the result and, in register
// 4 q + j, row 8 q + 4 (l / 32) + j.  Weights are the row operand, and packed
// so that MFMA row 8 q + 4 h + j is weight row 16 h + 4 q + j of its group of
// 32: a lane then holds 16 consecutive output features of one token.
#pragma once

#include "device_common.h"

namespace moe {

constexpr int kMxBlock = 32;    // elements per scale
constexpr int kMxGroupCols = 256;  // columns of one column group
constexpr int kMxGroupRows = 32;   // rows of one packed row group
// bytes of one packed (row group, column group): codes and scales
constexpr int kMxFragCodes = 4096;
constexpr int kMxFragScales = 256;

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

// Scale byte of a block from the largest |x| of it, given as float bits with
// the sign cleared (as integers these order like the values, infinities above
// every number and NaN above infinity).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// 2^(127 - byte), the exact factor that takes x to its element; 0 for a NaN block.
__device__ __forceinline__ float mx_inverse_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0u : (254u - byte) << 23);
}

// 2^(byte - 127), NaN for byte 255
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
  const uint32_t bits = byte == 0u ? 0x00400000u : (byte == 255u ? 0x7FC00000u : byte << 23);
  return __uint_as_float(bits);
}

// Eight codes (one dword) of x[0..7] under a block's scale byte.  A NaN block has zero codes.
__device__ __forceinline__ uint32_t mx_encode8(const float* x, uint32_t byte) {
  const float inv = mx_inverse_scale(byte);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = x[i] * inv;
  const uint32_t d = e2m1_encode8(v);
  return byte == 255u ? 0u : d;
}

// The elements of eight codes, unscaled
__device__ __forceinline__ void mx_decode8(uint32_t d, float* f) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 3)};
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = p[k >> 1][k & 1];
}

// Two values rounded to nearest even in BF16, the first in the low half; NaN stays NaN
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}

// The value of the lane that DPP control CTRL names: an ALU operand, where a
// shuffle goes through LDS.  kLaneXor1, kLaneXor2: exchange inside quads;
// kLaneHalfMirror, kLaneMirror: lane 7 - i of 8, 15 - i of 16.
enum { kLaneXor1 = 0xB1, kLaneXor2 = 0x4E, kLaneHalfMirror = 0x141, kLaneMirror = 0x140 };
template <int CTRL>
__device__ __forceinline__ uint32_t lane_dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

// Largest of v over aligned groups of four lanes, in every one of them
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, lane_dpp<kLaneXor1>(v));
  return max(v, lane_dpp<kLaneXor2>(v));
}

// A 16-byte store that does not stay in L2: for results larger than it, whose
// lines would push out what is still read.
__device__ __forceinline__ void store16_streaming(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const u32x4_t v = {a, b, c, d};
  __builtin_nontemporal_store(v, static_cast<u32x4_t*>(p));
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// One scaled FP4 MFMA step: c += A . B over 64 columns; S = step = scale byte.
template <int S>
__device__ __forceinline__ float16_t mx_mfma(i32x4_t a, i32x4_t b, float16_t c, int sa, int sb) {
  const i32x8_t a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
  const i32x8_t b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, S, sa, S, sb);
}

// Lane (of 64) and byte of the packed layout for weight row `row` and block `blk` (of 32 columns):
// codes  ((g * KK + c) * 4 + s) * 1024 + lane * 16, scales (g * KK + c) * 256 + lane * 4 + s.
__host__ __device__ __forceinline__ int mx_packed_lane(int64_t row, int64_t blk) {
  const int r = (int)(row & 31), f = (int)((blk >> 2) & 1);
  const int h = r >> 4, q = (r >> 2) & 3, j = r & 3;
  return 32 * f + 8 * q + 4 * h + j;
}

}  // namespace moe
