// Block-scaled FP8 quantisation (gfx950): a weight in 128 x 128 blocks, an
// activation or gradient in runs of 128 columns of a row, and the weight's
// values back.
//
// Per block: s = max(fl32(max |x| / 448), 2^-100), code = the E4M3 number
// nearest to fl32(x / s), ties to even; s = NaN for a block that is not all
// finite.  All three are one pass over the data: a block's values stay in
// registers between its maximum and its codes.

#include "qn_fp8.h"
#include "qn_launch.h"
#include "qn_project.h"

namespace qn {

namespace {

constexpr int kT = 256;

// One workgroup per 128 x 128 block: 16 lanes span a row's 128 columns, the
// workgroup 16 rows at a time, 8 passes held in registers as loaded, so that
// all loads are on their way before the first is used.  Bound by HBM: 11008 x
// 4096 bf16, 135 MB, in 28 us (4.8 TB/s; a large copy reaches 4.7).
template <typename T>
__global__ __launch_bounds__(kT) void quantize_blocks_kernel(const T* __restrict__ w, int64_t N,
                                                             int64_t K, uint8_t* __restrict__ codes,
                                                             float* __restrict__ scale) {
  __shared__ uint32_t s_max[kT / 64];
  const int64_t kb = (K + 127) / 128;
  const int64_t bn = blockIdx.x / kb, bk = blockIdx.x % kb;
  const int t = threadIdx.x;
  const int64_t k = bk * 128 + (t & 15) * 8;
  const int64_t n0 = bn * 128 + (t >> 4);
  const bool kin = k < K;  // K is a multiple of 16: a run of 8 is in or out
  Raw8<T> x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (kin && n0 + 16 * i < N) load8(w + (n0 + 16 * i) * K + k, x[i]);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t mi = absmax8(x[i]);
    m = m > mi ? m : mi;
  }
  m = lanes_max<1, 32>(m);
  if ((t & 63) == 0) s_max[t >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kT / 64; ++i) m = m > s_max[i] ? m : s_max[i];
  const float s = fp8_scale(m), inv = __fdiv_rn(1.0f, s);
  if (t == 0) scale[blockIdx.x] = s;
  if (!kin) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = n0 + 16 * i;
    float v[8];
    values8(x[i], v);
    if (n < N) *reinterpret_cast<uint2*>(codes + n * K + k) = fp8_codes8(v, s, inv);
  }
}

// 16 lanes per run of 128 columns of one row; a workgroup takes 16 rows of one
// block of columns, so that its scales lie together.  Bound by HBM: 2048 x
// 11008, 68 MB, in 16.2 us (4.2 TB/s; runs in the order of the rows 17.3, several
// runs per lane no faster).
__global__ __launch_bounds__(kT) void quantize_rows_kernel(const uint16_t* __restrict__ x,
                                                           int64_t M, int64_t K,
                                                           uint8_t* __restrict__ codes,
                                                           float* __restrict__ scale) {
  const int64_t kb = (K + 127) / 128;
  const int64_t m = blockIdx.x / kb * (kT / 16) + (threadIdx.x >> 4), b = blockIdx.x % kb;
  const int64_t k = b * 128 + (threadIdx.x & 15) * 8;
  const bool in = m < M && k < K;
  Raw8<uint16_t> raw;
  float v[8];
  if (in) load8(x + m * K + k, raw);
  values8(raw, v);
  const float s = fp8_scale(lanes_max<1, 8>(absmax8(raw))), inv = __fdiv_rn(1.0f, s);
  if (m < M && (threadIdx.x & 15) == 0) scale[b * M + m] = s;
  if (in) *reinterpret_cast<uint2*>(codes + m * K + k) = fp8_codes8(v, s, inv);
}

// Of the projection kernels: one scale for the whole block.
struct Fp8Rows {
  typedef uint2 Codes;
  static constexpr int kBytes = 128;
  static constexpr bool kForward = true, kBackward = true;
  uint8_t* codes;
  int64_t pitch;  // bytes of a token
  float* scale;
  int64_t M;

  struct Block {
    Codes c[4];
    float s;
  };
  __device__ __forceinline__ static Block quantize(const uint4 (&x)[4]) {
    Block q;
    float v[4][8];
    u16x2_t am{0, 0};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      bf16x8_to_f32(x[c], v[c]);
      am = absmax_pair(am, x[c]);
    }
    q.s = fp8_scale(lanes_max<16, 32>(absmax_bits(am)));
    const float inv = __fdiv_rn(1.0f, q.s);
#pragma unroll
    for (int c = 0; c < 4; ++c) q.c[c] = fp8_codes8(v[c], q.s, inv);
    return q;
  }
  __device__ __forceinline__ void store_scale(const Block& q, int64_t b, int64_t row, int lg) const {
    if (lg == 0) scale[b * M + row] = q.s;
  }
};

// The LoRA term's token side for the tile kernel: scale u, u the slices' sum in
// slice order, as two bf16 parts in rows of act zero-padded to `ranks`, a
// multiple of 32, so that the parts of 32 ranks are one 128-byte run, like the
// codes of a block; bf16(u) also to `plain` [M, r] for the caller.  Four values
// per thread; kSlices loads go out before the first is added.
__global__ __launch_bounds__(kT) void project_sum_kernel(const float* __restrict__ part, int slices,
                                                         int64_t M, int r, int ranks, float scale,
                                                         uint16_t* __restrict__ act,
                                                         uint16_t* __restrict__ plain) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * kT + threadIdx.x) * 4;
  const int64_t m = i / ranks;
  const int j = static_cast<int>(i % ranks);
  if (m >= M) return;
  f32x4_t s = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int64_t step = M * r;
  const float* p = part + m * r + j;
  if (j < r && (r & 3) == 0) {
    constexpr int kSlices = 16;
    for (int k0 = 0; k0 < slices; k0 += kSlices) {
      f32x4_t v[kSlices];
#pragma unroll
      for (int k = 0; k < kSlices; ++k)  // past the end: the last one again, not added
        v[k] = *reinterpret_cast<const f32x4_t*>(p + (k0 + k < slices ? k0 + k : slices - 1) * step);
#pragma unroll
      for (int k = 0; k < kSlices; ++k)
        if (k0 + k < slices) s += v[k];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e < r)
        for (int k = 0; k < slices; ++k) s[e] += p[k * step + e];
  }
  const Bf16Split a = split_bf16x2(s[0] * scale, s[1] * scale);
  const Bf16Split b = split_bf16x2(s[2] * scale, s[3] * scale);
  uint16_t* at = act + 2 * (i - (j & 31)) + (j & 31);
  *reinterpret_cast<uint2*>(at) = make_uint2(a.hi, b.hi);
  *reinterpret_cast<uint2*>(at + 32) = make_uint2(a.lo, b.lo);
  if (plain) {
    const uint32_t u[2] = {pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e < r) plain[m * r + j + e] = static_cast<uint16_t>(u[e >> 1] >> (16 * (e & 1)));
  }
}

// out = bf16 of the sum of `splits` fp32 parts [splits][n], in their order; 8
// values per thread (n is a multiple of 16).
__global__ __launch_bounds__(kT) void split_sum_kernel(const float* __restrict__ part, int splits,
                                                       int64_t n, uint16_t* __restrict__ out) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * kT + threadIdx.x) * 8;
  if (i >= n) return;
  f32x4_t a = f32x4_t{0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll 4
  for (int q = 0; q < splits; ++q) {
    a += *reinterpret_cast<const f32x4_t*>(part + q * n + i);
    b += *reinterpret_cast<const f32x4_t*>(part + q * n + i + 4);
  }
  *reinterpret_cast<uint4*>(out + i) = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                                  pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]));
}

// 16 codes per thread.  Bound by HBM: 11008 x 4096 to bf16, 135 MB, in 29 us
// (4.6 TB/s).
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
  const int64_t groups = (M + kT / 16 - 1) / (kT / 16) * ((K + 127) / 128);
  if (groups == 0) return hipSuccess;
  hipLaunchKernelGGL(quantize_rows_kernel, dim3(static_cast<uint32_t>(groups)), dim3(kT), 0, st, x,
                     M, K, codes, scale);
  return hipGetLastError();
}

int fp8_project_slices(int64_t M, int64_t L) {
  const int64_t blocks = (L + 127) / 128;
  const int per = project_blocks_per_slice(M, L);
  return static_cast<int>((blocks + per - 1) / per);
}

hipError_t launch_fp8_quantize_project(const uint16_t* x, int64_t M, int64_t L, const uint16_t* P,
                                       int r, bool rows_l, uint8_t* codes, float* scale,
                                       float* part, hipStream_t st) {
  return go_quantize_project(x, M, L, P, r, rows_l, Fp8Rows{codes, L, scale, M},
                             fp8_project_slices(M, L), part, st);
}

int fp8_decode_slices(int64_t L) { return static_cast<int>(((L + 127) / 128 + 3) / 4); }

hipError_t launch_fp8_decode_project(const uint16_t* x, int M, int64_t L, const uint16_t* A, int r,
                                     uint8_t* codes, float* scale, float* part, hipStream_t st) {
  return go_decode_project(x, M, L, A, r, Fp8Rows{codes, L, scale, M}, fp8_decode_slices(L), part,
                           st);
}

hipError_t launch_fp8_project_sum(const float* part, int slices, int64_t M, int r, float scale,
                                  uint16_t* act, uint16_t* plain, hipStream_t st) {
  if (M == 0 || r == 0) return hipSuccess;
  const int ranks = fp8_lora_ranks(r);
  const int64_t threads = M * ranks / 4;
  hipLaunchKernelGGL(project_sum_kernel, dim3(static_cast<uint32_t>((threads + kT - 1) / kT)),
                     dim3(kT), 0, st, part, slices, M, r, ranks, scale, act, plain);
  return hipGetLastError();
}

hipError_t launch_fp8_split_sum(const float* part, int splits, int64_t n, uint16_t* out,
                                hipStream_t st) {
  const int64_t threads = n / 8;
  hipLaunchKernelGGL(split_sum_kernel, dim3(static_cast<uint32_t>((threads + kT - 1) / kT)),
                     dim3(kT), 0, st, part, splits, n, out);
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
