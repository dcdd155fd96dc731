// Block-scaled FP8 quantisation (gfx950): a weight in 128 x 128 blocks, an
// activation or gradient in runs of 128 columns of a row, and the weight's
// values back.
//
// Per block: s = max(fl32(max |x| / 448), 2^-100), code = the E4M3 number
// nearest to fl32(x / s), ties to even.  All three are one pass over the
// data: a block's values stay in registers between its maximum and its codes.

#include "qn_fp8.h"
#include "qn_launch.h"

namespace qn {

namespace {

constexpr int kT = 256;

__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  bf16x8_to_f32(*reinterpret_cast<const uint4*>(p), v);
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// One workgroup per 128 x 128 block: 16 lanes span a row's 128 columns, the
// workgroup 16 rows at a time, 8 passes held in registers.
template <typename T>
__global__ __launch_bounds__(kT) void quantize_blocks_kernel(const T* __restrict__ w, int64_t N,
                                                             int64_t K, uint8_t* __restrict__ codes,
                                                             float* __restrict__ scale) {
  __shared__ float s_max[kT / 64];
  const int64_t kb = (K + 127) / 128;
  const int64_t bn = blockIdx.x / kb, bk = blockIdx.x % kb;
  const int t = threadIdx.x;
  const int64_t k = bk * 128 + (t & 15) * 8;
  const int64_t n0 = bn * 128 + (t >> 4);
  const bool kin = k < K;  // K is a multiple of 16: a run of 8 is in or out
  float v[8][8];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = n0 + 16 * i;
    if (kin && n < N) {
      load8(w + n * K + k, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, absmax8(v[i]));
  m = wave_max(m);
  if ((t & 63) == 0) s_max[t >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  const float s = fp8_scale(m), inv = __fdiv_rn(1.0f, s);
  if (t == 0) scale[blockIdx.x] = s;
  if (!kin) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = n0 + 16 * i;
    if (n < N) *reinterpret_cast<uint2*>(codes + n * K + k) = fp8_codes8(v[i], s, inv);
  }
}

// 16 lanes per run of 128 columns of one row; run q of the launch is row
// q / kb, columns 128 (q % kb) ...
__global__ __launch_bounds__(kT) void quantize_rows_kernel(const uint16_t* __restrict__ x,
                                                           int64_t M, int64_t K,
                                                           uint8_t* __restrict__ codes,
                                                           float* __restrict__ scale) {
  const int64_t kb = (K + 127) / 128;
  const int64_t q = static_cast<int64_t>(blockIdx.x) * (kT / 16) + (threadIdx.x >> 4);
  const int64_t m = q / kb, b = q % kb;
  const int64_t k = b * 128 + (threadIdx.x & 15) * 8;
  const bool in = m < M && k < K;
  float v[8];
  if (in) {
    load8(x + m * K + k, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  }
  const float s = fp8_scale(max16(absmax8(v))), inv = __fdiv_rn(1.0f, s);
  if (m < M && (threadIdx.x & 15) == 0) scale[b * M + m] = s;
  if (in) *reinterpret_cast<uint2*>(codes + m * K + k) = fp8_codes8(v, s, inv);
}

// Quantisation of x [M, L] and its LoRA projection x P^T in one pass over x:
// a wave takes 16 tokens and the blocks of 128 columns of one slice.  Lane
// (li, lg) holds columns 32 c + 8 lg .. + 7 (c = 0..3) of token li, which is
// the bf16 MFMA's operand layout, so the values that are quantised are the
// ones that are multiplied.  P is A [r, L] (forward) or, with kRowsL, B
// [L, r] read in place (backward).  part[slice][M][r] gets the slice's sums.
template <bool kRowsL, int kRT>
__global__ __launch_bounds__(kT) void quantize_project_kernel(
    const uint16_t* __restrict__ x, int64_t M, int64_t L, const uint16_t* __restrict__ P, int r,
    bool vec_p, int per_slice, uint8_t* __restrict__ codes, float* __restrict__ scale,
    float* __restrict__ part) {
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 6) + (threadIdx.x >> 6)) * 16 + li;
  const int64_t m = row < M ? row : M - 1;
  const int64_t blocks = (L + 127) / 128;
  const int64_t b0 = static_cast<int64_t>(blockIdx.y) * per_slice;
  const int64_t b1 = b0 + per_slice < blocks ? b0 + per_slice : blocks;
  f32x4_t acc[kRT];
#pragma unroll
  for (int i = 0; i < kRT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int64_t b = b0; b < b1; ++b) {
    uint4 w[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t k = b * 128 + 32 * c + 8 * lg;
      w[c] = k < L ? *reinterpret_cast<const uint4*>(x + m * L + k) : make_uint4(0, 0, 0, 0);
    }
    float v[4][8], am = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      bf16x8_to_f32(w[c], v[c]);
      am = fmaxf(am, absmax8(v[c]));
    }
    am = fmaxf(am, __shfl_xor(am, 16, 64));
    am = fmaxf(am, __shfl_xor(am, 32, 64));
    const float s = fp8_scale(am), inv = __fdiv_rn(1.0f, s);
    if (row < M) {
      if (lg == 0) scale[b * M + row] = s;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int64_t k = b * 128 + 32 * c + 8 * lg;
        if (k < L) *reinterpret_cast<uint2*>(codes + row * L + k) = fp8_codes8(v[c], s, inv);
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t k = b * 128 + 32 * c + 8 * lg;
#pragma unroll
      for (int i = 0; i < kRT; ++i) {
        const int j = 16 * i + li;
        uint4 pf = make_uint4(0, 0, 0, 0);
        if (j < r && k < L)
          pf = kRowsL ? load_bf16x8_strided(P + k * r + j, r, 8) : load_bf16x8(P + j * L + k, 8, vec_p);
        acc[i] = mfma_bf16_32(pf, w[c], acc[i]);
      }
    }
  }
  if (row >= M) return;
  // lane (li, lg): ranks 16 i + 4 lg .. + 3 of token li
  float* out = part + (static_cast<int64_t>(blockIdx.y) * M + row) * r;
#pragma unroll
  for (int i = 0; i < kRT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = 16 * i + 4 * lg + e;
      if (j < r) out[j] = acc[i][e];
    }
}

// Sum of the slices, in slice order: bf16(scale sum) for the LoRA-up term
// and bf16(sum) for the caller.
__global__ __launch_bounds__(kT) void project_sum_kernel(const float* __restrict__ part, int slices,
                                                         int64_t n, float scale,
                                                         uint16_t* __restrict__ scaled,
                                                         uint16_t* __restrict__ plain) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kT + threadIdx.x;
  if (i >= n) return;
  float s = 0.0f;
  for (int q = 0; q < slices; ++q) s += part[q * n + i];
  scaled[i] = static_cast<uint16_t>(pack_bf16x2(s * scale, 0.f) & 0xFFFF);
  if (plain) plain[i] = static_cast<uint16_t>(pack_bf16x2(s, 0.f) & 0xFFFF);
}

// 16 codes per thread.
template <typename T>
__global__ __launch_bounds__(kT) void dequant_kernel(const uint8_t* __restrict__ codes,
                                                     const float* __restrict__ scale, int64_t N,
                                                     int64_t K, T* __restrict__ out) {
  const int64_t e = (static_cast<int64_t>(blockIdx.x) * kT + threadIdx.x) * 16;
  if (e >= N * K) return;
  const int64_t n = e / K, k = e % K;
  const float s = scale[(n / 128) * ((K + 127) / 128) + k / 128];
  const uint4 c = *reinterpret_cast<const uint4*>(codes + e);
  const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
  float v[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(cw[i]), false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(cw[i]), true);
    v[4 * i] = __fmul_rn(a[0], s), v[4 * i + 1] = __fmul_rn(a[1], s);
    v[4 * i + 2] = __fmul_rn(b[0], s), v[4 * i + 3] = __fmul_rn(b[1], s);
  }
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(out + e + 4 * i) =
          make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint4*>(out + e + 8 * i) =
          make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                     pack_bf16x2(v[8 * i + 4], v[8 * i + 5]),
                     pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
  }
}

}  // namespace

hipError_t launch_fp8_quantize_blocks(const void* w, bool bf16, int64_t N, int64_t K,
                                      uint8_t* codes, float* scale, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>(((N + 127) / 128) * ((K + 127) / 128)));
  if (grid.x == 0) return hipSuccess;
  if (bf16)
    hipLaunchKernelGGL(quantize_blocks_kernel<uint16_t>, grid, dim3(kT), 0, st,
                       static_cast<const uint16_t*>(w), N, K, codes, scale);
  else
    hipLaunchKernelGGL(quantize_blocks_kernel<float>, grid, dim3(kT), 0, st,
                       static_cast<const float*>(w), N, K, codes, scale);
  return hipGetLastError();
}

hipError_t launch_fp8_quantize_rows(const uint16_t* x, int64_t M, int64_t K, uint8_t* codes,
                                    float* scale, hipStream_t st) {
  const int64_t runs = M * ((K + 127) / 128);
  if (runs == 0) return hipSuccess;
  hipLaunchKernelGGL(quantize_rows_kernel,
                     dim3(static_cast<uint32_t>((runs + kT / 16 - 1) / (kT / 16))), dim3(kT), 0, st,
                     x, M, K, codes, scale);
  return hipGetLastError();
}

// Slices of the contraction: enough workgroups to fill the chip for small
// batches, one pass of a few blocks each for large ones.
static int blocks_per_slice(int64_t M, int64_t L) {
  const int64_t blocks = (L + 127) / 128, groups = (M + 63) / 64;
  int64_t slices = (512 + groups - 1) / groups;
  slices = slices < blocks ? slices : blocks;
  return static_cast<int>((blocks + slices - 1) / slices);
}

int fp8_project_slices(int64_t M, int64_t L) {
  const int64_t blocks = (L + 127) / 128;
  const int per = blocks_per_slice(M, L);
  return static_cast<int>((blocks + per - 1) / per);
}

hipError_t launch_fp8_quantize_project(const uint16_t* x, int64_t M, int64_t L, const uint16_t* P,
                                       int r, bool rows_l, uint8_t* codes, float* scale,
                                       float* part, hipStream_t st) {
  if (M == 0) return hipSuccess;
  const int waves = M > 48 ? 4 : static_cast<int>((M + 15) / 16);
  const dim3 grid(static_cast<uint32_t>((M + 16 * waves - 1) / (16 * waves)),
                  static_cast<uint32_t>(fp8_project_slices(M, L)));
  const bool vec_p = (reinterpret_cast<uintptr_t>(P) & 15) == 0;
  const int per = blocks_per_slice(M, L);
  auto go = [&](auto k) {
    hipLaunchKernelGGL(k, grid, dim3(64 * waves), 0, st, x, M, L, P, r, vec_p, per, codes, scale,
                       part);
    return hipGetLastError();
  };
  if (rows_l)
    return r <= 16   ? go(quantize_project_kernel<true, 1>)
           : r <= 32 ? go(quantize_project_kernel<true, 2>)
           : r <= 64 ? go(quantize_project_kernel<true, 4>)
                     : go(quantize_project_kernel<true, 8>);
  return r <= 16   ? go(quantize_project_kernel<false, 1>)
         : r <= 32 ? go(quantize_project_kernel<false, 2>)
         : r <= 64 ? go(quantize_project_kernel<false, 4>)
                   : go(quantize_project_kernel<false, 8>);
}

hipError_t launch_fp8_project_sum(const float* part, int slices, int64_t n, float scale,
                                  uint16_t* scaled, uint16_t* plain, hipStream_t st) {
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(project_sum_kernel, dim3(static_cast<uint32_t>((n + kT - 1) / kT)), dim3(kT),
                     0, st, part, slices, n, scale, scaled, plain);
  return hipGetLastError();
}

hipError_t launch_fp8_dequant(const Fp8View& w, bool out_bf16, void* out, hipStream_t st) {
  const int64_t threads = w.N * w.K / 16;
  if (threads == 0) return hipSuccess;
  const dim3 grid(static_cast<uint32_t>((threads + kT - 1) / kT));
  if (out_bf16)
    hipLaunchKernelGGL(dequant_kernel<uint16_t>, grid, dim3(kT), 0, st, w.codes, w.scale, w.N, w.K,
                       static_cast<uint16_t*>(out));
  else
    hipLaunchKernelGGL(dequant_kernel<float>, grid, dim3(kT), 0, st, w.codes, w.scale, w.N, w.K,
                       static_cast<float*>(out));
  return hipGetLastError();
}

}  // namespace qn
