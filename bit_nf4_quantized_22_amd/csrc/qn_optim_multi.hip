// AdamW over many LoRA matrices in one launch, states in 32 or in 8 bits, and
// the global gradient norm that clips them (gfx950).
//
// [rkmt "QLORA技术解析" §3.5], [czcl "QLoRA技術解析" §3.2]: the adapter is
// trained with AdamW, its states in 32 or 8 bits.  A 7B model has 448 LoRA
// matrices of 64 K - 176 K elements, so one call per matrix is launch-bound;
// here a workgroup takes one chunk of 2048 elements of one matrix, whose
// addresses it finds in one 64-byte entry of a table that the caller keeps on
// the device.
//
// Per element, fp32, each operation rounded on its own (no fused
// multiply-add, so that the 8-bit codes are a pure function of the inputs):
//   g <- c g                       (c: the clip coefficient, when given)
//   m <- b1 m + (1 - b1) g;   v <- b2 v + (1 - b2) g^2
//   p <- p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// 8-bit states: blocks of 256 elements, one fp32 scale each; m is E4M3
// (scale = max |m| / 448), v is E5M2 (scale = max v / 57344), both at least
// 2^-100.  The update uses the unrounded m and v; only what is kept for the
// next step is rounded, by dithering: element i of a block at step t adds
// frac(i (sqrt 2 - 1) + t (sqrt 5 - 1) / 2), a Weyl sequence over the steps,
// below the last kept mantissa bit and cuts.  Rounding to nearest would
// leave v where it is for good, since one step moves it by 0.1% and the
// codes are 12-25% apart; over the steps the dithered codes move by the
// right amount on average.  A positive v never becomes code 0, so no
// element's denominator drops to eps.  What is not finite takes no part in its
// block's scale and keeps its place: an m as the NaN code, a v as the code of
// infinity or NaN, like 32-bit states.

#include <cmath>

#include "qn_device.h"
#include "qn_launch.h"

namespace qn {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;  // elements per thread
static_assert(kThreads * kPer == kAdamChunk, "chunk split");
static_assert(kAdamChunk % kAdamStateBlock == 0 && kAdamStateBlock == 32 * kPer,
              "a state block is 32 lanes");

typedef float f4_t __attribute__((ext_vector_type(4)));
typedef float f2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

constexpr uint32_t kInfBits = 0x7F800000u;  // of fp32; NaN lies above

struct MultiArgs {
  float beta1, beta2, one_minus_beta1, one_minus_beta2, eps;
  float decay;         // 1 - lr wd
  float step_size;     // lr / (1 - beta1^t)
  float inv_bc2_sqrt;  // 1 / sqrt(1 - beta2^t)
  uint32_t dither;     // t 2^32 (sqrt 5 - 1) / 2 mod 2^32
};

__device__ __forceinline__ void adam_update(float& p, float g, float& m, float& v,
                                            const MultiArgs& a) {
#pragma clang fp contract(off)
  m = a.beta1 * m + a.one_minus_beta1 * g;
  v = a.beta2 * v + a.one_minus_beta2 * (g * g);
  const float den = __fsqrt_rn(v) * a.inv_bc2_sqrt + a.eps;
  p = p * a.decay - a.step_size * __fdiv_rn(m, den);
}

// Max over the 32 lanes of a half wave (every lane gets it).
__device__ __forceinline__ uint32_t half_wave_max(uint32_t x) {
#pragma unroll
  for (int off = 1; off <= 16; off <<= 1) {
    const uint32_t y = static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), off, 64));
    x = x > y ? x : y;
  }
  return x;
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Code of n >= 0 in a format of kMant mantissa bits: fp32 bits plus the
// dither, cut; below the least normal number 2^kMinExp the same on the fixed
// grid of the subnormals.
template <int kMant, int kMinExp, uint32_t kMost>
__device__ __forceinline__ uint32_t dithered_code(float n, uint32_t d) {
  constexpr int kShift = 23 - kMant;
  constexpr uint32_t kOffset = static_cast<uint32_t>(127 + kMinExp - 1) << kMant;
  const uint32_t normal = ((__float_as_uint(n) + d) >> kShift) - kOffset;
  // n 2^(kMant - kMinExp) counts subnormal steps; 2^kShift keeps the fraction
  const float sub = __uint_as_float(static_cast<uint32_t>(127 + kMant - kMinExp + kShift) << 23);
  const uint32_t small = (static_cast<uint32_t>(n * sub) + d) >> kShift;
  const float least = __uint_as_float(static_cast<uint32_t>(127 + kMinExp) << 23);
  const uint32_t c = n >= least ? normal : small;
  return c < kMost ? c : kMost;
}

__device__ __forceinline__ float state_scale(uint32_t most, float top) {
  return fmaxf(__fdiv_rn(__uint_as_float(most), top), 0x1p-100f);
}

// Bound by HBM: 160 M elements, 32-bit states, 30 bytes each, in 892 us (5.4
// TB/s); 40 M, 8-bit states, 18 bytes each, in 113-139 us (5.2-6.4 TB/s, part
// of it from the cache); one 7B layer's 1.25 M with 32-bit states in 9.0 us.
// Chunks of 1024 or 4096 elements and nontemporal accesses were slower.
template <bool kState8, bool kBf16Grad>
__global__ __launch_bounds__(kThreads) void adamw_multi_kernel(
    const AdamChunk* __restrict__ tab, const float* __restrict__ grad_scale, MultiArgs a) {
#pragma clang fp contract(off)
  const AdamChunk d = tab[blockIdx.x];
  float c = 1.0f;
  if (grad_scale) {
    c = *grad_scale;
    if (!(fabsf(c) < __builtin_inff())) return;  // norm not finite: no step
  }
  const int e0 = threadIdx.x * kPer, n = static_cast<int>(d.n);
  const int left = n - e0 >= kPer ? kPer : n > e0 ? n - e0 : 0;
  float p[kPer], g[kPer], m[kPer], v[kPer];
  uint32_t m8[2] = {0, 0}, v8[2] = {0, 0};
  const int blk = e0 / kAdamStateBlock;
  float ms = 0.0f, vs = 0.0f;
  if (left == kPer) {
    const f4_t p0 = *reinterpret_cast<const f4_t*>(d.p + e0);
    const f4_t p1 = *reinterpret_cast<const f4_t*>(d.p + e0 + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = p0[j], p[4 + j] = p1[j];
    if constexpr (kBf16Grad) {
      const u4_t w = *reinterpret_cast<const u4_t*>(static_cast<const uint16_t*>(d.g) + e0);
#pragma unroll
      for (int j = 0; j < 4; ++j) g[2 * j] = bf16_lo(w[j]), g[2 * j + 1] = bf16_hi(w[j]);
    } else {
      const f4_t g0 = *reinterpret_cast<const f4_t*>(static_cast<const float*>(d.g) + e0);
      const f4_t g1 = *reinterpret_cast<const f4_t*>(static_cast<const float*>(d.g) + e0 + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] = g0[j], g[4 + j] = g1[j];
    }
    if constexpr (kState8) {
      const uint2 mw = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(d.m) + e0);
      const uint2 vw = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(d.v) + e0);
      m8[0] = mw.x, m8[1] = mw.y, v8[0] = vw.x, v8[1] = vw.y;
      ms = d.m_scale[blk];
      vs = d.v_scale[blk];
    } else {
      const f4_t m0 = *reinterpret_cast<const f4_t*>(static_cast<const float*>(d.m) + e0);
      const f4_t m1 = *reinterpret_cast<const f4_t*>(static_cast<const float*>(d.m) + e0 + 4);
      const f4_t v0 = *reinterpret_cast<const f4_t*>(static_cast<const float*>(d.v) + e0);
      const f4_t v1 = *reinterpret_cast<const f4_t*>(static_cast<const float*>(d.v) + e0 + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        m[j] = m0[j], m[4 + j] = m1[j], v[j] = v0[j], v[4 + j] = v1[j];
    }
  } else {  // the last 0..7 elements of the matrix, or none
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool in = j < left;
      p[j] = in ? d.p[e0 + j] : 0.0f;
      if constexpr (kBf16Grad)
        g[j] = in ? bf16_to_f32(static_cast<const uint16_t*>(d.g)[e0 + j]) : 0.0f;
      else
        g[j] = in ? static_cast<const float*>(d.g)[e0 + j] : 0.0f;
      if constexpr (kState8) {
        if (in) {
          m8[j >> 2] |= static_cast<uint32_t>(static_cast<const uint8_t*>(d.m)[e0 + j]) << (8 * (j & 3));
          v8[j >> 2] |= static_cast<uint32_t>(static_cast<const uint8_t*>(d.v)[e0 + j]) << (8 * (j & 3));
        }
      } else {
        m[j] = in ? static_cast<const float*>(d.m)[e0 + j] : 0.0f;
        v[j] = in ? static_cast<const float*>(d.v)[e0 + j] : 0.0f;
      }
    }
    if (kState8 && left > 0) {
      ms = d.m_scale[blk];
      vs = d.v_scale[blk];
    }
  }
  if constexpr (kState8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f2_t ma = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(m8[h]), false);
      const f2_t mb = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(m8[h]), true);
      const f2_t va = __builtin_amdgcn_cvt_pk_f32_bf8(static_cast<int>(v8[h]), false);
      const f2_t vb = __builtin_amdgcn_cvt_pk_f32_bf8(static_cast<int>(v8[h]), true);
      m[4 * h] = ma[0] * ms, m[4 * h + 1] = ma[1] * ms;
      m[4 * h + 2] = mb[0] * ms, m[4 * h + 3] = mb[1] * ms;
      v[4 * h] = va[0] * vs, v[4 * h + 1] = va[1] * vs;
      v[4 * h + 2] = vb[0] * vs, v[4 * h + 3] = vb[1] * vs;
    }
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) adam_update(p[j], g[j] * c, m[j], v[j], a);

  uint32_t mc[2] = {0, 0}, vc[2] = {0, 0};
  float ns = 0.0f, nvs = 0.0f;
  if constexpr (kState8) {
    // magnitudes are compared as integers, which keep infinities and NaN on top
    uint32_t mm = 0, vm = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      mm = mm > magnitude(m[j]) ? mm : magnitude(m[j]);
      vm = vm > magnitude(v[j]) ? vm : magnitude(v[j]);
    }
    mm = half_wave_max(mm);
    vm = half_wave_max(vm);
    // the same for all lanes of a block, and rare: with the two tests in every
    // element's way 3 M elements took 14.5 us instead of 13.5
    const bool lost = (mm > vm ? mm : vm) >= kInfBits;
    if (lost) {
      mm = vm = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint32_t am = magnitude(m[j]), av = magnitude(v[j]);
        mm = am < kInfBits && am > mm ? am : mm;
        vm = av < kInfBits && av > vm ? av : vm;
      }
      mm = half_wave_max(mm);
      vm = half_wave_max(vm);
    }
    ns = state_scale(mm, 448.0f);
    nvs = state_scale(vm, 57344.0f);
    const float im = __fdiv_rn(1.0f, ns), iv = __fdiv_rn(1.0f, nvs);
    // dither of this thread's first element, then one step of i at a time
    uint32_t w = (threadIdx.x % 32) * kPer * 0x6A09E667u + a.dither;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float nm = fminf(fabsf(m[j]) * im, 448.0f), nv = fminf(v[j] * iv, 57344.0f);
      uint32_t cm = dithered_code<3, -6, 0x7Eu>(nm, w >> 12);
      cm |= m[j] < 0.0f ? 0x80u : 0u;
      uint32_t cv = dithered_code<2, -14, 0x7Bu>(nv, ~w >> 11);
      cv = v[j] > 0.0f ? (cv > 1u ? cv : 1u) : 0u;
      mc[j >> 2] |= cm << (8 * (j & 3));
      vc[j >> 2] |= cv << (8 * (j & 3));
      w += 0x6A09E667u;
    }
    if (lost) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int at = 8 * (j & 3);
        if (magnitude(m[j]) >= kInfBits) mc[j >> 2] |= 0x7Fu << at;
        if (magnitude(v[j]) >= kInfBits)
          vc[j >> 2] = (vc[j >> 2] & ~(0xFFu << at)) |
                       (magnitude(v[j]) == kInfBits ? 0x7Cu : 0x7Fu) << at;
      }
    }
  }
  if (left == kPer) {
    *reinterpret_cast<f4_t*>(d.p + e0) = f4_t{p[0], p[1], p[2], p[3]};
    *reinterpret_cast<f4_t*>(d.p + e0 + 4) = f4_t{p[4], p[5], p[6], p[7]};
    if (d.p_bf16)
      *reinterpret_cast<u4_t*>(d.p_bf16 + e0) =
          u4_t{pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]), pack_bf16x2(p[4], p[5]),
               pack_bf16x2(p[6], p[7])};
    if constexpr (kState8) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(d.m) + e0) = make_uint2(mc[0], mc[1]);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(d.v) + e0) = make_uint2(vc[0], vc[1]);
    } else {
      *reinterpret_cast<f4_t*>(static_cast<float*>(d.m) + e0) = f4_t{m[0], m[1], m[2], m[3]};
      *reinterpret_cast<f4_t*>(static_cast<float*>(d.m) + e0 + 4) = f4_t{m[4], m[5], m[6], m[7]};
      *reinterpret_cast<f4_t*>(static_cast<float*>(d.v) + e0) = f4_t{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f4_t*>(static_cast<float*>(d.v) + e0 + 4) = f4_t{v[4], v[5], v[6], v[7]};
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (j >= left) break;
      d.p[e0 + j] = p[j];
      if (d.p_bf16)
        d.p_bf16[e0 + j] = static_cast<uint16_t>(pack_bf16x2(p[j], 0.f) & 0xFFFF);
      if constexpr (kState8) {
        static_cast<uint8_t*>(d.m)[e0 + j] = static_cast<uint8_t>(mc[j >> 2] >> (8 * (j & 3)));
        static_cast<uint8_t*>(d.v)[e0 + j] = static_cast<uint8_t>(vc[j >> 2] >> (8 * (j & 3)));
      } else {
        static_cast<float*>(d.m)[e0 + j] = m[j];
        static_cast<float*>(d.v)[e0 + j] = v[j];
      }
    }
  }
  if constexpr (kState8) {
    if (threadIdx.x % 32 == 0 && left > 0) {
      d.m_scale[blk] = ns;
      d.v_scale[blk] = nvs;
    }
  }
}

__device__ __forceinline__ double wave_sum64(double x) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
  return x;
}

// Sum over the workgroup's waves, in wave order (valid in thread 0).
template <int kWaves>
__device__ __forceinline__ double block_sum64(double x) {
  __shared__ double s[kWaves];
  x = wave_sum64(x);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
  __syncthreads();
  double t = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kWaves; ++w) t += s[w];
  return t;
}

// Squares summed in fp64 (the vector unit's fp64 rate is far above what the
// reads of g need, and no gradient's square overflows): workgroup b takes
// chunks b, b + gridDim.x, ..., a fixed order.  1024 workgroups, four chunks in
// flight each: 160 M gradients in 115 us (5.6 TB/s), 40 M in 31.
template <bool kBf16Grad>
__global__ __launch_bounds__(kThreads) void grad_sq_kernel(const AdamChunk* __restrict__ tab,
                                                           int64_t chunks,
                                                           double* __restrict__ part) {
  constexpr int kAhead = 4;  // chunks in flight
  const int e0 = threadIdx.x * kPer;
  double s = 0.0;
  for (int64_t q = blockIdx.x; q < chunks; q += kAhead * static_cast<int64_t>(gridDim.x)) {
    float g[kAhead][kPer];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t c = q + k * static_cast<int64_t>(gridDim.x);
      const void* gp = tab[c < chunks ? c : q].g;
      const int n = c < chunks ? static_cast<int>(tab[c].n) : 0;
      if (e0 + kPer <= n) {
        if constexpr (kBf16Grad) {
          const u4_t w = *reinterpret_cast<const u4_t*>(static_cast<const uint16_t*>(gp) + e0);
#pragma unroll
          for (int j = 0; j < 4; ++j) g[k][2 * j] = bf16_lo(w[j]), g[k][2 * j + 1] = bf16_hi(w[j]);
        } else {
          const f4_t g0 = *reinterpret_cast<const f4_t*>(static_cast<const float*>(gp) + e0);
          const f4_t g1 = *reinterpret_cast<const f4_t*>(static_cast<const float*>(gp) + e0 + 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) g[k][j] = g0[j], g[k][4 + j] = g1[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          if constexpr (kBf16Grad)
            g[k][j] = e0 + j < n ? bf16_to_f32(static_cast<const uint16_t*>(gp)[e0 + j]) : 0.0f;
          else
            g[k][j] = e0 + j < n ? static_cast<const float*>(gp)[e0 + j] : 0.0f;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const double v = static_cast<double>(g[k][j]);
        s = fma(v, v, s);
      }
  }
  const double t = block_sum64<kThreads / 64>(s);
  if (threadIdx.x == 0) part[blockIdx.x] = t;
}

// out[0] = norm, out[1] = min(1, max_norm / (norm + 1e-6)), NaN when the
// norm is not finite.
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const double* __restrict__ part,
                                                             int n, float max_norm,
                                                             float* __restrict__ out) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += part[i];
  const double t = block_sum64<kThreads / 64>(s);
  if (threadIdx.x == 0) {
    const double norm = sqrt(t);
    double c = static_cast<double>(max_norm) / (norm + 1e-6);
    c = c < 1.0 ? c : 1.0;
    out[0] = static_cast<float>(norm);
    out[1] = norm < __builtin_inf() ? static_cast<float>(c) : __builtin_nanf("");
  }
}

}  // namespace

int grad_norm_blocks(int64_t chunks) {
  return static_cast<int>(chunks < kGradNormBlocks ? chunks : kGradNormBlocks);
}

hipError_t launch_adamw_multi(const AdamChunk* tab, int64_t chunks, bool state8, bool bf16_grad,
                              const float* grad_scale, float lr, float beta1, float beta2,
                              float eps, float weight_decay, int step, hipStream_t st) {
  if (chunks == 0) return hipSuccess;
  MultiArgs a;
  a.beta1 = beta1;
  a.beta2 = beta2;
  a.one_minus_beta1 = 1.0f - beta1;
  a.one_minus_beta2 = 1.0f - beta2;
  a.eps = eps;
  a.decay = static_cast<float>(1.0 - static_cast<double>(lr) * static_cast<double>(weight_decay));
  const double bc1 = 1.0 - std::pow(static_cast<double>(beta1), step);
  const double bc2 = 1.0 - std::pow(static_cast<double>(beta2), step);
  a.step_size = static_cast<float>(static_cast<double>(lr) / bc1);
  a.inv_bc2_sqrt = static_cast<float>(1.0 / std::sqrt(bc2));
  a.dither = static_cast<uint32_t>(step) * 0x9E3779B9u;
  const dim3 grid(static_cast<uint32_t>(chunks));
  auto k = state8 ? (bf16_grad ? adamw_multi_kernel<true, true> : adamw_multi_kernel<true, false>)
                  : (bf16_grad ? adamw_multi_kernel<false, true> : adamw_multi_kernel<false, false>);
  hipLaunchKernelGGL(k, grid, dim3(kThreads), 0, st, tab, grad_scale, a);
  return hipGetLastError();
}

hipError_t launch_grad_norm(const AdamChunk* tab, int64_t chunks, bool bf16_grad, float max_norm,
                            double* part, float* out, hipStream_t st) {
  const int blocks = grad_norm_blocks(chunks);
  if (blocks > 0) {
    auto k = bf16_grad ? grad_sq_kernel<true> : grad_sq_kernel<false>;
    hipLaunchKernelGGL(k, dim3(static_cast<uint32_t>(blocks)), dim3(kThreads), 0, st, tab,
                       chunks, part);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kThreads), 0, st, part, blocks, max_norm, out);
  return hipGetLastError();
}

}  // namespace qn
