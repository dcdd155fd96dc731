// Device helpers of the products for few tokens on 8- and 4-bit weights: the
// LoRA-up term of the 16 columns that a wave finishes, and its operands.
#pragma once

#include "qn_fp8.h"

namespace qn {

constexpr int kDecodeMaxRank = 128;

// LoRA-up term of 16 tokens: acc += B[n rows] us^T, us rows of `pitch` bf16
// (the two parts of 32 ranks at a time, zero past r) at sus, B's fragments
// already in registers.
template <int kFrags>
__device__ __forceinline__ f32x4_t lora_up(f32x4_t acc, const uint4 (&bf)[kFrags],
                                           const uint16_t* sus, int pitch, int r, int li, int lg) {
#pragma unroll
  for (int q = 0; q < kFrags; ++q)
    if (32 * q < r) {
      const uint16_t* p = sus + li * pitch + 64 * q + 8 * lg;
      acc = mfma_bf16_32(bf[q], *reinterpret_cast<const uint4*>(p), acc);
      acc = mfma_bf16_32(bf[q], *reinterpret_cast<const uint4*>(p + 32), acc);
    }
  return acc;
}

// Rank j of a row of us = the two parts of v.
__device__ __forceinline__ void store_us(uint16_t* row, int j, float v) {
  const Bf16Split p = split_bf16x2(v, 0.0f);
  uint16_t* at = row + (j & ~31) * 2 + (j & 31);
  at[0] = static_cast<uint16_t>(p.hi & 0xFFFF);
  at[32] = static_cast<uint16_t>(p.lo & 0xFFFF);
}

__device__ __forceinline__ void store_columns(uint16_t* y, f32x4_t acc) {
  *reinterpret_cast<uint2*>(y) =
      make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
}

// Where one token's u comes from: no adapter, x A^T computed here (r <= 16),
// or `slices` partial sums of it.
enum TokenU { kNoAdapter, kOwnU, kGivenU };

// B's fragments of rows n0 .. n0 + 15, zeros behind r.
template <int kFrags>
__device__ __forceinline__ void load_up(uint4 (&bf)[kFrags], const uint16_t* B, int64_t n0, int r,
                                        int li, int lg, bool vec_b) {
#pragma unroll
  for (int q = 0; q < kFrags; ++q) {
    bf[q] = make_uint4(0, 0, 0, 0);
    if (32 * q < r)
      bf[q] = load_bf16x8(B + (n0 + li) * r + 32 * q + 8 * lg, r - 32 * q - 8 * lg, vec_b);
  }
}

// One token's u: thread (q0, j) of kThreads adds the slices q0, q0 + par, ... of
// rank j.
template <int kThreads>
__device__ __forceinline__ float add_slices(const float* part, int slices, int r, int t) {
  const int par = kThreads / r, j = t % r, q0 = t / r;
  float s = 0.0f;
  if (q0 < par) {
#pragma unroll 4
    for (int q = q0; q < slices; q += par) s += part[static_cast<int64_t>(q) * r + j];
  }
  return s;
}

// One wave adds the `sums` sums of each rank in s_u, rows of `pitch`, to u, gives
// its bf16 to u_out if not null, and adds (lora_scale u) B^T.
template <int kFrags>
__device__ __forceinline__ f32x4_t token_up(f32x4_t acc, const uint4 (&bf)[kFrags],
                                            const float* s_u, int pitch, int sums, uint16_t* s_us,
                                            int r, float lora_scale, uint16_t* u_out, int lane) {
  for (int j = lane; j < 32 * kFrags && j < ((r + 31) & ~31); j += 64) {
    float s = 0.0f;
    if (j < r) {
#pragma unroll 8
      for (int q = 0; q < sums; ++q) s += s_u[q * pitch + j];
    }
    if (u_out && j < r) u_out[j] = static_cast<uint16_t>(pack_bf16x2(s, 0.f) & 0xFFFF);
    store_us(s_us, j, s * lora_scale);
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  return lora_up(acc, bf, s_us, 0, r, lane & 15, lane >> 4);
}

// The workgroup's rows of us from the par sums of each of the M r values in s_u.
template <int kThreads>
__device__ __forceinline__ void spread_u(const float* s_u, int par, int slices, int mr, int M, int r,
                                         float lora_scale, uint16_t* s_us, uint16_t* u_out, int t) {
  const int rp = (r + 31) & ~31;
  for (int i = t; i < 16 * rp; i += kThreads) {
    const int row = i / rp, j = i % rp;
    float s = 0.0f;
    if (row < M && j < r) {
      for (int q = 0; q < par && q < slices; ++q) s += s_u[q * mr + row * r + j];
      if (u_out) u_out[row * r + j] = static_cast<uint16_t>(pack_bf16x2(s, 0.f) & 0xFFFF);
    }
    store_us(s_us + row * 2 * rp, j, s * lora_scale);
  }
}

}  // namespace qn
