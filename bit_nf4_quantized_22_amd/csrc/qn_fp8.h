// Device helpers of the block-scaled FP8 kernels: E4M3 codes (1-4-3, bias 7,
// no infinities; largest value 448) with one fp32 scale per 128 columns of a
// row (activations, gradients) or per 128 x 128 block (weights).
#pragma once

#include "qn_device.h"

namespace qn {

// Scale of a group whose largest magnitude has the fp32 bits amax: fl32(amax /
// 448), at least 2^-100, so that no group divides by zero and 1 / s is a normal
// number; NaN for a group with an infinity or NaN, so that every product with
// the group is NaN.
__device__ __forceinline__ float fp8_scale(uint32_t amax) {
  const float s = fmaxf(__fdiv_rn(__uint_as_float(amax), 448.0f), 0x1p-100f);
  return amax < 0x7F800000u ? s : __builtin_nanf("");
}

// fl32(x / s) in the codes' range, inv = fl32(1 / s): one Newton step on
// x inv (x - q s is exact in the fused multiply-add; at the lowest borders of
// a group with the least scale it is a subnormal number, which is kept).  bf16
// values often lie on the border between two codes, where the product x inv
// alone is an ulp to one side.
__device__ __forceinline__ float fp8_ratio(float x, float s, float inv) {
  const float q = x * inv;
  return __builtin_amdgcn_fmed3f(fmaf(fmaf(-q, s, x), inv, q), -448.0f, 448.0f);
}

// E4M3 codes of four values in [-448, 448], round to nearest even.
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}

// Codes of 8 values of one group.
__device__ __forceinline__ uint2 fp8_codes8(const float (&v)[8], float s, float inv) {
  return make_uint2(fp8_pack4(fp8_ratio(v[0], s, inv), fp8_ratio(v[1], s, inv),
                              fp8_ratio(v[2], s, inv), fp8_ratio(v[3], s, inv)),
                    fp8_pack4(fp8_ratio(v[4], s, inv), fp8_ratio(v[5], s, inv),
                              fp8_ratio(v[6], s, inv), fp8_ratio(v[7], s, inv)));
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4& w, float (&v)[8]) {
  v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
  v[4] = bf16_lo(w.z), v[5] = bf16_hi(w.z), v[6] = bf16_lo(w.w), v[7] = bf16_hi(w.w);
}

// Magnitudes are compared as integers: the bits of |x| are ordered as |x| is,
// with infinities and NaN on top, where a maximum of floats drops a NaN.
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));

// Two running maxima of bf16 magnitudes, of the even and the odd values.
__device__ __forceinline__ u16x2_t absmax_pair(u16x2_t m, uint32_t pair) {
  return __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, pair & 0x7FFF7FFFu));
}

__device__ __forceinline__ u16x2_t absmax_pair(u16x2_t m, const uint4& w) {
  return absmax_pair(absmax_pair(absmax_pair(absmax_pair(m, w.x), w.y), w.z), w.w);
}

// The larger of the two, as fp32 bits.
__device__ __forceinline__ uint32_t absmax_bits(u16x2_t m) {
  return static_cast<uint32_t>(m[0] > m[1] ? m[0] : m[1]) << 16;
}

// Max over the lanes that differ in the bits from .. to of their number
// (every lane gets it).
template <int kFrom, int kTo>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
#pragma unroll
  for (int off = kFrom; off <= kTo; off <<= 1) {
    const uint32_t y = static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), off, 64));
    x = x > y ? x : y;
  }
  return x;
}

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// c + a b^T of 16 x 128 E4M3 fragments: lane l gives row l % 16 of a and of
// b, the same 32 of the 128 contraction values each; the result's lane l
// holds column l % 16, rows 4 (l / 16) .. + 3.  No scale in the instruction.
__device__ __forceinline__ f32x4_t mfma_fp8(i32x8_t a, i32x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ i32x8_t frag8(const uint4& lo, const uint4& hi) {
  return i32x8_t{static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(lo.z),
                 static_cast<int>(lo.w), static_cast<int>(hi.x), static_cast<int>(hi.y),
                 static_cast<int>(hi.z), static_cast<int>(hi.w)};
}

// 8 bf16 values p[0 .. 7] of a row with `left` values left, zeros behind the
// row's end; vec: p is 16-byte aligned and left a multiple of 8.
__device__ __forceinline__ uint4 load_bf16x8(const uint16_t* p, int left, bool vec) {
  if (left <= 0) return make_uint4(0, 0, 0, 0);
  if (vec) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = 2 * j < left ? p[2 * j] : 0u;
    const uint32_t hi = 2 * j + 1 < left ? p[2 * j + 1] : 0u;
    w[j] = lo | hi << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two values as sums hi + lo of bf16 numbers (pairs of each): 16 significant
// bits.  What bf16 holds as an infinity or NaN has lo = 0.
struct Bf16Split {
  uint32_t hi, lo;
};

__device__ __forceinline__ Bf16Split split_bf16x2(float a, float b) {
  const uint32_t hi = pack_bf16x2(a, b);
  const float ha = bf16_lo(hi), hb = bf16_hi(hi);
  return {hi, pack_bf16x2(fabsf(ha) < __builtin_inff() ? a - ha : 0.0f,
                          fabsf(hb) < __builtin_inff() ? b - hb : 0.0f)};
}

__device__ __forceinline__ f32x4_t mfma_bf16_32(const uint4& a, const uint4& b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                  __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

}  // namespace qn
