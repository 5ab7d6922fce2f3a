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
// MXFP8 activations (E4M3 elements under the same kind of scale; the byte is
// floor(log2(amax)) - 8 + 127, 8 = the exponent of 448) multiply the same packed
// weights.  Of an 8-bit operand lane l takes two runs of 16 bytes a step:
// elements 16 f .. 16 f + 15 of the step's first block (s) and of its second
// (4 + s), where a 4-bit operand takes one whole block; scales go by lane as
// above (layout checked on the device).
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

// Scale byte of an MXFP8 block; as mx_scale_byte, with E4M3's exponent
__device__ __forceinline__ uint32_t mx8_scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255u ? 255u : (e > 8u ? e - 8u : 0u);
}

// Four E4M3 elements (one dword) of x[0..3] under a block's scale byte: round to
// nearest even, saturating (the convert alone gives NaN past 448; checked on the
// device against the definition for every BF16 value).  A NaN block is zero.
__device__ __forceinline__ uint32_t mx8_encode4(const float* x, uint32_t byte) {
  const float inv = mx_inverse_scale(byte);
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_fmed3f(x[i] * inv, -kE4M3Max, kE4M3Max);
  int d = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  d = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], d, true);
  return byte == 255u ? 0u : (uint32_t)d;
}

// The elements of four bytes, unscaled
__device__ __forceinline__ void mx8_decode4(uint32_t d, float* f) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)d, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)d, true);
  f[0] = lo[0];
  f[1] = lo[1];
  f[2] = hi[0];
  f[3] = hi[1];
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

// Orders this wave's LDS accesses before its later ones (lanes read what other lanes of the same wave wrote)
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// One scaled FP4 MFMA step: c += A . B over 64 columns; S = step = scale byte.
template <int S>
__device__ __forceinline__ float16_t mx_mfma(i32x4_t a, i32x4_t b, float16_t c, int sa, int sb) {
  const i32x8_t a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
  const i32x8_t b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, S, sa, S, sb);
}

// The same step with 8-bit activations.  The instruction aligns the products of
// a block to the largest of them and drops what lies some 17 binades below, where
// E4M3's elements alone span 18: normal data's products of 6144 columns would be
// off by 4e-6 in the 2-norm, with outliers of 300 times the rest by 7e-5, and
// elements of h then round to another code.  So x is multiplied as two operands
// whose elements each span half of that (the exponent's upper bit tells which),
// and all that is left is the rounding of the FP32 accumulator (3e-8 and 1e-7), for
// twice the matrix instructions.
// Selector of a byte permutation between d and zeros: byte 4 + i where byte i of d is large, i where not.
__device__ __forceinline__ uint32_t mx8_select(uint32_t d) {
  uint32_t r;  // one instruction after the shift; the compiler takes two
  asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(d >> 4), "s"(0x04040404u), "v"(0x03020100u));
  return r;
}
__device__ __forceinline__ uint32_t mx8_large(uint32_t d) { return __builtin_amdgcn_perm(d, 0u, mx8_select(d)); }
__device__ __forceinline__ uint32_t mx8_rest(uint32_t d) { return __builtin_amdgcn_perm(0u, d, mx8_select(d)); }
// Either, by lane
__device__ __forceinline__ i32x8_t mx8_part(i32x8_t b, bool rest) {
  const uint32_t flip = rest ? 0x04040404u : 0u;
  i32x8_t r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (int)__builtin_amdgcn_perm((uint32_t)b[i], 0u, mx8_select((uint32_t)b[i]) ^ flip);
  return r;
}
template <int S>
__device__ __forceinline__ float16_t mx8_part_mfma(i32x4_t a, i32x8_t b, float16_t c, int sa, int sb) {
  const i32x8_t a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b, c, 4, 0, S, sa, S, sb);
}
// HALF: the columns of b hold the large elements and the rest (16 of each); else b is parted here.
template <int S, bool HALF>
__device__ __forceinline__ float16_t mx8_mfma(i32x4_t a, i32x8_t b, float16_t c, int sa, int sb) {
  if constexpr (HALF) return mx8_part_mfma<S>(a, b, c, sa, sb);
  i32x8_t large, rest;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    large[i] = (int)mx8_large((uint32_t)b[i]);
    rest[i] = (int)mx8_rest((uint32_t)b[i]);
  }
  return mx8_part_mfma<S>(a, rest, mx8_part_mfma<S>(a, large, c, sa, sb), sa, sb);
}

// Lane (of 64) and byte of the packed layout for weight row `row` and block `blk` (of 32 columns):
// codes  ((g * KK + c) * 4 + s) * 1024 + lane * 16, scales (g * KK + c) * 256 + lane * 4 + s.
__host__ __device__ __forceinline__ int mx_packed_lane(int64_t row, int64_t blk) {
  const int r = (int)(row & 31), f = (int)((blk >> 2) & 1);
  const int h = r >> 4, q = (r >> 2) & 3, j = r & 3;
  return 32 * f + 8 * q + 4 * h + j;
}

}  // namespace moe
