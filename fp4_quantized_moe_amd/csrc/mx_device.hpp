// Device-side MXFP4 and MXFP8 codecs for the gfx950 kernels.
//
// MXFP4 (OCP Microscaling): blocks of 32 elements along the last axis share
// one E8M0 scale, a power of two 2^E stored as the byte E + 127; the elements
// are E2M1.  For a block with largest magnitude a:
//   E    = floor(log2 a) - 2, clamped to [-127, 125]   (2 = E2M1's largest exponent)
//   code = E2M1 nearest to x * 2^-E, ties to even, saturating at 6
// so magnitudes in (6, 8) * 2^E saturate.  The "even" rule rounds a to E2M1's
// two significant bits before taking its exponent: a >= 1.75 * 2^floor(log2 a)
// takes the next E, and the block's largest value is then off by at most 1/7
// instead of 1/4.  A block of zeros or of values below 2^-125 gets byte 0; a
// block with a NaN or an infinity gets byte 255 (E8M0's NaN) and codes 0, so
// every value it stands for is NaN.  Multiplying by 2^-E is exact except
// where the product is far below the first rounding threshold (0.25).
//
// MXFP8 has the same blocks with E4M3 elements (largest exponent 8, largest
// value 448 = 1.75 * 2^8):
//   E    = floor(log2 a) - 8, at least -127
//   code = E4M3 nearest to x * 2^-E, ties to even, saturating at 448
// so magnitudes in (448, 512) * 2^E saturate (off by at most 1/8).  Zero,
// subnormal and non-finite blocks as above.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace quads {

constexpr uint32_t kMxNan = 255;            // E8M0 NaN
constexpr uint32_t kMxMaxByte = 252;        // 6 * 2^125 is the largest finite fp32/bf16 value of a block
constexpr uint32_t kMxEvenAdd = 0x200000u;  // carries into the exponent from a mantissa of 1.75 on

// E8M0 byte of a block from the bits of its largest magnitude (as an
// unsigned maximum of |x| bit patterns, so a NaN wins); `add` is 0 or kMxEvenAdd.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t abs_bits, uint32_t add) {
  const uint32_t e = (abs_bits + add) >> 23;
  const uint32_t b = min(e < 2u ? 0u : e - 2u, kMxMaxByte);
  return abs_bits >= 0x7F800000u ? kMxNan : b;
}

// 2^-E for a scale byte (byte 255: zero, which makes every code of the block 0).
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) {
  return byte == kMxNan ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// 2^E for a scale byte (2^-127 is a subnormal).
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return byte == 0u ? __uint_as_float(0x00400000u) : byte == kMxNan ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23);
}

// v[0..7] (already multiplied by 2^-E) -> 8 E2M1 codes, element i in nibble i.
// v_cvt_scalef32_pk_fp4_f32 rounds to nearest even and saturates; its own
// scale operand stays 1 (the exact multiplication was done in fp32).
__device__ __forceinline__ uint32_t mx_pack8(const float (&v)[8]) {
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], 1.0f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], 1.0f, 3);
  return c;
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

// 8 codes -> 8 levels (exact).
__device__ __forceinline__ void mx_unpack8(uint32_t c, float (&v)[8]) {
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
  const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
  v[0] = a[0];
  v[1] = a[1];
  v[2] = b[0];
  v[3] = b[1];
  v[4] = d[0];
  v[5] = d[1];
  v[6] = e[0];
  v[7] = e[1];
}

// Maximum over the aligned quad of lanes (quad_perm [1,0,3,2] and [2,3,0,1]).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, true)));
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xF, 0xF, true)));
}

// E8M0 byte of an MXFP8 block from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t mx8_scale_byte(uint32_t abs_bits) {
  const uint32_t e = abs_bits >> 23;
  return abs_bits >= 0x7F800000u ? kMxNan : e < 8u ? 0u : e - 8u;
}

// v[0..7] (already multiplied by 2^-E) -> 8 E4M3 codes, element i in byte i.
// The conversion rounds to nearest even; what it makes of larger magnitudes
// does not matter behind the clamp.
__device__ __forceinline__ uint2 mx8_pack8(const float (&v)[8]) {
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __builtin_amdgcn_fmed3f(v[i], -448.0f, 448.0f);
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], hi, true);
  return make_uint2(static_cast<uint32_t>(lo), static_cast<uint32_t>(hi));
}

// 8 codes -> 8 values (exact; a NaN code stays NaN).
__device__ __forceinline__ void mx8_unpack8(uint2 c, float (&v)[8]) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c.x), false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c.x), true);
  const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c.y), false);
  const f32x2 e = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c.y), true);
  v[0] = a[0];
  v[1] = a[1];
  v[2] = b[0];
  v[3] = b[1];
  v[4] = d[0];
  v[5] = d[1];
  v[6] = e[0];
  v[7] = e[1];
}

// Two floats -> packed bf16, nearest-even (v_cvt_pk_bf16_f32; NaN stays NaN).
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 p = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, p);
}

}  // namespace quads
