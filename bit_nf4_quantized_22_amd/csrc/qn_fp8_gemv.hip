// Block-scaled FP8 product for up to 16 tokens (gfx950).
//
//   y[m, n] = sum_b xs[b, m] ws[n / 128, b] (xq_b[m] . wq_b[n]) + (s u) B^T
//
// Bound by reading the weight once (N K bytes).  A workgroup owns 16 output
// columns and the whole contraction: its waves take the blocks of 128 in
// turn, each block one 16x16x128 FP8 MFMA with the weight's rows as the first
// operand and the tokens (padded to 16 by re-reading the last) as the second.
// Every lane loads 32 consecutive bytes of its row straight into its
// fragment, kDepth blocks ahead of their products, so the weight needs
// neither LDS nor a second pass.  The waves' fp32 sums meet in LDS and are
// added in wave order, so results are bit-reproducible.

#include "qn_fp8.h"
#include "qn_launch.h"

namespace qn {

namespace {

constexpr int kDepth = 4;  // blocks in flight per wave
constexpr int kMaxRank = 128;

struct Block {
  uint4 w0, w1, x0, x1;
  float s;
};

template <int kWaves>
__global__ __launch_bounds__(64 * kWaves) void fp8_decode_kernel(
    const uint8_t* __restrict__ w, const float* __restrict__ ws, int64_t N, int64_t K,
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int M,
    const float* __restrict__ part, int slices, const uint16_t* __restrict__ B, int r, bool vec_b,
    float lora_scale, uint16_t* __restrict__ y, uint16_t* __restrict__ u_out) {
  constexpr int kThreads = 64 * kWaves;
  __shared__ f32x4_t s_acc[kWaves][64];
  __shared__ float s_u[kFp8DecodeM * kMaxRank];                     // slices of u, then u
  __shared__ __attribute__((aligned(16))) uint16_t s_us[16 * kMaxRank];  // bf16(s u), [16][rp]
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int li = lane & 15, lg = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;  // N is a multiple of 16
  const int64_t kb = (K + 127) / 128;
  const int m = li < M ? li : M - 1;
  const uint8_t* wr = w + (n0 + li) * K;
  const uint8_t* xr = x + static_cast<int64_t>(m) * K;
  const float* wsr = ws + (n0 / 128) * kb;

  auto load = [&](int64_t b, Block& d) {
    const int64_t k = b * 128 + 32 * lg;
    const uint4 z = make_uint4(0, 0, 0, 0);
    d.w0 = d.w1 = d.x0 = d.x1 = z;
    d.s = 0.0f;
    if (b >= kb) return;
    if (k < K) {
      d.w0 = *reinterpret_cast<const uint4*>(wr + k);
      d.x0 = *reinterpret_cast<const uint4*>(xr + k);
    }
    if (k + 16 < K) {
      d.w1 = *reinterpret_cast<const uint4*>(wr + k + 16);
      d.x1 = *reinterpret_cast<const uint4*>(xr + k + 16);
    }
    d.s = xs[b * M + m] * wsr[b];
  };
  Block blk[kDepth];
#pragma unroll
  for (int d = 0; d < kDepth; ++d) load(wave + d * kWaves, blk[d]);

  // u = sum of its slices: as many slices at a time as there are threads,
  // then the partial sums, in a fixed order
  const int mr = M * r;
  if (r > 0) {
    const int par = mr <= kThreads ? kThreads / mr : 1;
    for (int i = t; i < (par > 1 ? par * mr : mr); i += kThreads) {
      const int e = i % mr, q0 = i / mr;
      float s = 0.0f;
#pragma unroll 8
      for (int q = q0; q < slices; q += par) s += part[static_cast<int64_t>(q) * mr + e];
      s_u[i] = s;
    }
    __syncthreads();
    const int rp = (r + 31) & ~31;
    for (int i = t; i < 16 * rp; i += kThreads) {
      const int row = i / rp, j = i % rp;
      float s = 0.0f;
      if (row < M && j < r) {
        for (int q = 0; q < par; ++q) s += s_u[q * mr + row * r + j];
        if (u_out && blockIdx.x == 0)
          u_out[row * r + j] = static_cast<uint16_t>(pack_bf16x2(s, 0.f) & 0xFFFF);
      }
      s_us[i] = static_cast<uint16_t>(pack_bf16x2(s * lora_scale, 0.f) & 0xFFFF);
    }
  }

  f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int64_t b = wave; b < kb; b += kDepth * kWaves) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const f32x4_t c = mfma_fp8(frag8(blk[d].w0, blk[d].w1), frag8(blk[d].x0, blk[d].x1),
                                 f32x4_t{0.f, 0.f, 0.f, 0.f});
      const float s = blk[d].s;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = fmaf(c[e], s, acc[e]);
      load(b + (d + kDepth) * kWaves, blk[d]);
    }
  }
  s_acc[wave][lane] = acc;
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int q = 1; q < kWaves; ++q) acc += s_acc[q][lane];
  if (r > 0) {
    const int rp = (r + 31) & ~31;
    for (int j0 = 0; j0 < r; j0 += 32) {
      const int j = j0 + 8 * lg;
      const uint4 bf = load_bf16x8(B + (n0 + li) * r + j, r - j, vec_b);
      const uint4 uf = *reinterpret_cast<const uint4*>(s_us + li * rp + j);
      acc = mfma_bf16_32(bf, uf, acc);
    }
  }
  // lane (li, lg): columns n0 + 4 lg .. + 3 of token li
  if (li < M)
    *reinterpret_cast<uint2*>(y + static_cast<int64_t>(li) * N + n0 + 4 * lg) =
        make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
}

}  // namespace

hipError_t launch_fp8_decode(const Fp8View& w, const uint8_t* x, const float* xs, int M,
                             const float* part, int slices, const uint16_t* B, int r,
                             float lora_scale, uint16_t* y, uint16_t* u_out, hipStream_t st) {
  if (M == 0) return hipSuccess;
  const dim3 grid(static_cast<uint32_t>(w.N / 16));
  const bool vec_b = (r & 7) == 0 && (reinterpret_cast<uintptr_t>(B) & 15) == 0;
  const int64_t kb = (w.K + 127) / 128;
  auto go = [&](auto k, int waves) {
    hipLaunchKernelGGL(k, grid, dim3(64 * waves), 0, st, w.codes, w.scale, w.N, w.K, x, xs, M, part,
                       slices, B, r, vec_b, lora_scale, y, u_out);
    return hipGetLastError();
  };
  return kb <= 8 ? go(fp8_decode_kernel<4>, 4) : go(fp8_decode_kernel<16>, 16);
}

}  // namespace qn
