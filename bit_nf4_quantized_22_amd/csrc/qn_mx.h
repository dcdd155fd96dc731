// Device helpers of the microscaled kernels: groups of 32 values of a row that
// share one power of two, 2^(byte - 127) (byte 255: NaN), with E2M1 codes (1
// sign, 2 exponent bits of bias 1, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6)
// or E4M3 codes; two E2M1 codes per byte, the even column in the low half.
//
// Scales lie as the matrix instruction takes them: a lane of a 16x16x128 MFMA
// scales its own row's (lane % 16) group lane / 16 of the four, with one of the
// four bytes of a register.  A tile of scales is 64 registers, 256 bytes, of
//   E2M1: 32 rows x 256 columns, byte 2 h + j = row 16 h + lane % 16, group
//         4 j + lane / 16 (tiles [ceil(K / 256)][ceil(R / 32)]);
//   8-bit: 64 rows x 128 columns, byte h = row 16 h + lane % 16, group lane / 16
//         (tiles [ceil(K / 128)][ceil(R / 64)]).
// Bytes of groups past a row's end are 0, for both operands of a product: what
// the codes there hold is then multiplied by 2^-254.
#pragma once

#include "qn_fp8.h"

namespace qn {

// Scale byte of a group whose largest magnitude has the fp32 bits amax: the
// least power of two for which that magnitude rounds to a code, 6 at most (a
// mantissa from 1.75 on would round to 8).  Below 2^-125 the least power, 255
// for a group with an infinity or NaN.
__device__ __forceinline__ uint32_t mx4_scale(uint32_t amax) {
  const int e = static_cast<int>((amax + 0x200000u) >> 23) - 2;
  return amax < 0x7F800000u ? static_cast<uint32_t>(e > 0 ? e : 0) : 255u;
}

// The same for E4M3 codes, 448 at most (past 1.8125 = 464 / 256 the next number
// of 3 mantissa bits would be the code of NaN).
__device__ __forceinline__ uint32_t mx8_scale(uint32_t amax) {
  const int e = static_cast<int>((amax + 0x17FFFFu) >> 23) - 8;
  return amax < 0x7F800000u ? static_cast<uint32_t>(e > 0 ? e : 0) : 255u;
}

// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float mx_power(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}

// E2M1 codes of 8 values over the power s, nearest even; values past 6 s give
// 6.  The conversion divides without rounding, subnormal numbers too.
typedef __bf16 bf16x2_mx_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t mx4_codes8(const uint4& v, float s) {
  uint32_t c = 0;
  auto bf = [](uint32_t w) { return __builtin_bit_cast(bf16x2_mx_t, w); };
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf(v.x), s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf(v.y), s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf(v.z), s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf(v.w), s, 3);
}

__device__ __forceinline__ uint32_t mx4_codes8(const float (&v)[8], float s) {
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
}

// E4M3 codes of 8 values over the power of scale byte b.  The quotient is exact
// (subnormal ones lie far below the least code).
__device__ __forceinline__ uint2 mx8_codes8(const float (&v)[8], uint32_t b) {
  const int e = 127 - static_cast<int>(b);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    q[i] = __builtin_amdgcn_fmed3f(__builtin_amdgcn_ldexpf(v[i], e), -448.0f, 448.0f);
  return make_uint2(fp8_pack4(q[0], q[1], q[2], q[3]), fp8_pack4(q[4], q[5], q[6], q[7]));
}

// Formats of the matrix instruction's operands.
enum MxFormat { kE4M3 = 0, kE5M2 = 1, kE2M1 = 4 };

// c + (a sa) (b sb)^T over 128 values; sa, sb hold the scale bytes at place
// oa, ob, which have to be constants once the loops around are unrolled.
template <int kA, int kB>
__device__ __forceinline__ f32x4_t mfma_mx(const i32x8_t& a, const i32x8_t& b, f32x4_t c, int oa,
                                           int sa, int ob, int sb) {
#define QN_MX_CASE(i, j)                                                                     \
  case 4 * i + j:                                                                            \
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, kA, kB, i, sa, j, sb);
#define QN_MX_ROW(i) QN_MX_CASE(i, 0) QN_MX_CASE(i, 1) QN_MX_CASE(i, 2) QN_MX_CASE(i, 3)
  switch (4 * oa + ob) { QN_MX_ROW(0) QN_MX_ROW(1) QN_MX_ROW(2) QN_MX_ROW(3) }
#undef QN_MX_ROW
#undef QN_MX_CASE
  __builtin_unreachable();
}

// An operand of 16 bytes, 32 E2M1 codes.
__device__ __forceinline__ i32x8_t frag4(const uint4& v) {
  return frag8(v, make_uint4(0, 0, 0, 0));
}

}  // namespace qn
