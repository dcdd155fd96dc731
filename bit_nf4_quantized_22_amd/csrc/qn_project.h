// Quantisation of a batch of rows together with its LoRA projection, for the
// 8-bit and the microscaled layers.  Q says what a block of 128 columns of 16
// tokens becomes: kBytes of codes per token, and what quantize() and
// store_scale() make of the values that lane (li, lg) holds, columns 32 c + 8 lg
// .. + 7 (c = 0 .. 3) of token li.
#pragma once

#include "qn_fp8.h"

namespace qn {

// 8 values as they lie in memory; the bits of their largest magnitude; the
// values as fp32.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2] = {};
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, Raw8<T>& x) {
#pragma unroll
  for (int h = 0; h < static_cast<int>(sizeof(T) / 2); ++h)
    x.w[h] = reinterpret_cast<const uint4*>(p)[h];
}

__device__ __forceinline__ uint32_t absmax8(const Raw8<uint16_t>& x) {
  return absmax_bits(absmax_pair(u16x2_t{0, 0}, x.w[0]));
}

__device__ __forceinline__ uint32_t absmax8(const Raw8<float>& x) {
  uint32_t m = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    for (const uint32_t w : {x.w[h].x, x.w[h].y, x.w[h].z, x.w[h].w}) {
      const uint32_t u = w & 0x7FFFFFFFu;
      m = m > u ? m : u;
    }
  return m;
}

__device__ __forceinline__ void values8(const Raw8<uint16_t>& x, float (&v)[8]) {
  bf16x8_to_f32(x.w[0], v);
}

__device__ __forceinline__ void values8(const Raw8<float>& x, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    v[4 * h] = __uint_as_float(x.w[h].x), v[4 * h + 1] = __uint_as_float(x.w[h].y);
    v[4 * h + 2] = __uint_as_float(x.w[h].z), v[4 * h + 3] = __uint_as_float(x.w[h].w);
  }
}

// Quantisation of x [M, L] and its LoRA projection x P^T in one pass over x:
// a wave takes 16 tokens, its workgroup the blocks of 128 columns of one
// slice.  Lane (li, lg) holds columns 32 c + 8 lg .. + 7 (c = 0..3) of token
// li, which is the bf16 MFMA's operand layout, so the values that are
// quantised are the ones that are multiplied.  P is A [r, L] (forward) or,
// with kRowsL, B [L, r] read in place (backward); its 128 columns (rows) of a
// block are staged in LDS for the workgroup's waves, in the other of two
// buffers, and x and P of the next block are in flight meanwhile.  B's tile
// lies [column][rank] and is read through the transposing LDS loads (4 rows x
// 16 ranks per 16 lanes).  part[slice][M][r] gets the slice's sums.
// Bound by HBM and the turn between two blocks: forward 2048 x 4096, r = 16,
// 25 MB in 8.4 us; 4096 x 8192, r = 64, 101 MB in 29 us (3.5 TB/s); backward
// 2048 x 11008, r = 64, 69 MB in 22 us.
typedef __attribute__((address_space(3))) uint16_t lds_u16_t;

// Places of P's 16-byte (32-byte with kRowsL) chunks in LDS: XOR-swizzled by
// the row so that a wave's reads spread over all banks.
template <bool kRowsL, int kRT>
__device__ __forceinline__ int p_place(int row, int chunk) {
  if constexpr (!kRowsL) return row * 128 + (chunk ^ (row & 15)) * 8;
  const int sw = kRT == 8   ? (row & 3) | ((row >> 3) & 1) << 2
                 : kRT == 4 ? ((row >> 1) & 1) | ((row >> 3) & 1) << 1
                 : kRT == 2 ? (row >> 3) & 1
                            : 0;
  return row * (16 * kRT) + (((chunk >> 1) ^ sw) << 4) + (chunk & 1) * 8;
}

// LDS of a workgroup: two tiles of P, and each wave's codes of a block.
template <typename Q, int kRT, int kWaves>
struct ProjectLds {
  __attribute__((aligned(16))) uint16_t p[2][kRT * 16 * 128];
  __attribute__((aligned(16))) uint8_t q[kWaves][16 * (Q::kBytes + 16)];
};

template <typename Q, bool kRowsL, int kRT, int kWaves>
__device__ __forceinline__ void quantize_project(const uint16_t* __restrict__ x, int64_t M,
                                                 int64_t L, const uint16_t* __restrict__ P, int r,
                                                 bool vec_p, int per_slice, const Q& out_q,
                                                 float* __restrict__ part, int group, int slice,
                                                 ProjectLds<Q, kRT, kWaves>& lds) {
  constexpr int kThreads = 64 * kWaves;
  constexpr int kLoads = kRT * 256 / kThreads;  // 16-byte chunks of P per thread and block
  static_assert(kLoads * kThreads == kRT * 256, "P tile split");
  constexpr int kQPitch = Q::kBytes + 16, kQChunks = Q::kBytes / 16;
  const int t = threadIdx.x, lane = t & 63, li = lane & 15, lg = lane >> 4;
  const int64_t row = (static_cast<int64_t>(group) * kWaves + (t >> 6)) * 16 + li;
  const int64_t m = row < M ? row : M - 1;
  const int64_t blocks = (L + 127) / 128;
  const int64_t b0 = static_cast<int64_t>(slice) * per_slice;
  const int64_t b1 = b0 + per_slice < blocks ? b0 + per_slice : blocks;
  uint4 w[4], p[kLoads];
  auto load_x = [&](int64_t b) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t k = b * 128 + 32 * c + 8 * lg;
      w[c] = k < L ? *reinterpret_cast<const uint4*>(x + m * L + k) : make_uint4(0, 0, 0, 0);
    }
  };
  auto load_p = [&](int64_t b) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int q = i * kThreads + t;
      if constexpr (kRowsL) {
        const int64_t l = b * 128 + q / (2 * kRT);
        const int j = q % (2 * kRT) * 8;
        p[i] = load_bf16x8(P + l * r + j, l < L ? r - j : 0, vec_p);
      } else {
        const int64_t k = b * 128 + q % 16 * 8;
        const int j = q / 16;
        p[i] = load_bf16x8(P + j * L + k, j < r && k < L ? 8 : 0, vec_p);
      }
    }
  };
  f32x4_t acc[kRT];
#pragma unroll
  for (int i = 0; i < kRT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  load_x(b0);
  load_p(b0);
  for (int64_t b = b0; b < b1; ++b) {
    uint16_t* sp = lds.p[(b - b0) & 1];
    uint4 cur[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) cur[c] = w[c];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int q = i * kThreads + t;
      const int at = kRowsL ? p_place<kRowsL, kRT>(q / (2 * kRT), q % (2 * kRT))
                            : p_place<kRowsL, kRT>(q / 16, q % 16);
      *reinterpret_cast<uint4*>(sp + at) = p[i];
    }
    __syncthreads();
    if (b + 1 < b1) {
      load_x(b + 1);
      load_p(b + 1);
    }
    const typename Q::Block q = Q::quantize(cur);
    if (row < M) out_q.store_scale(q, b, row, lg);
    // the codes leave as whole rows of the block, 8 or 16 of them per store (8
    // bytes of 16 rows per store took 40% longer for the whole kernel); sq is
    // the wave's own, so the order of its LDS accesses keeps the turns apart
    uint8_t* sq = lds.q[t >> 6];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<typename Q::Codes*>(sq + li * kQPitch + (4 * c + lg) * sizeof(q.c[0])) =
          q.c[c];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int h = 0; h < kQChunks / 4; ++h) {
      const int rr = (64 / kQChunks) * h + lane / kQChunks, ch = lane % kQChunks * 16;
      const int64_t to = row - li + rr, at = b * Q::kBytes + ch;
      const uint4 w16 = *reinterpret_cast<const uint4*>(sq + rr * kQPitch + ch);
      if (to < M && at < out_q.pitch)
        *reinterpret_cast<uint4*>(out_q.codes + to * out_q.pitch + at) = w16;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < kRT; ++i) {
        uint4 pf;
        if constexpr (kRowsL) {
          uint2 h[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            // lane 4 a + e of a group points at row a, ranks 4 e .. + 3
            const int l = 32 * c + 8 * lg + 4 * q + (li >> 2);
            const i16x4_t d = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_i16x4_t*)(lds_u16_t*)(sp + p_place<kRowsL, kRT>(l, 2 * i + ((li >> 1) & 1)) +
                                           (li & 1) * 4));
            h[q] = __builtin_bit_cast(uint2, d);
          }
          pf = make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
        } else {
          pf = *reinterpret_cast<const uint4*>(sp + p_place<kRowsL, kRT>(16 * i + li, 4 * c + lg));
        }
        acc[i] = mfma_bf16_32(pf, cur[c], acc[i]);
      }
  }
  if (row >= M) return;
  // lane (li, lg): ranks 16 i + 4 lg .. + 3 of token li
  float* out = part + (static_cast<int64_t>(slice) * M + row) * r;
#pragma unroll
  for (int i = 0; i < kRT; ++i) {
    const int j = 16 * i + 4 * lg;
    if ((r & 3) == 0) {
      if (j < r) *reinterpret_cast<f32x4_t*>(out + j) = acc[i];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e < r) out[j + e] = acc[i][e];
    }
  }
}

template <typename Q, bool kRowsL, int kRT, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void quantize_project_kernel(
    const uint16_t* __restrict__ x, int64_t M, int64_t L, const uint16_t* __restrict__ P, int r,
    bool vec_p, int per_slice, Q out_q, float* __restrict__ part) {
  __shared__ ProjectLds<Q, kRT, kWaves> lds;
  quantize_project<Q, kRowsL, kRT, kWaves>(x, M, L, P, r, vec_p, per_slice, out_q, part, blockIdx.x,
                                           blockIdx.y, lds);
}

// The same for the decode path (up to 16 tokens, P = A): a wave takes one
// block, with A's fragments straight in registers, everything asked for at
// once; the four waves' sums are added in LDS, so that the product's
// workgroups, which all add up the slices, find a quarter as many.  16 tokens
// of 11008 values, r = 16: 4 us, one round trip to memory.
template <typename Q, int kRT>
__global__ __launch_bounds__(256) void decode_project_kernel(
    const uint16_t* __restrict__ x, int M, int64_t L, const uint16_t* __restrict__ A, int r,
    bool vec_a, Q out_q, float* __restrict__ part) {
  __shared__ f32x4_t s_part[4][kRT][64];
  const int t = threadIdx.x, lane = t & 63, li = lane & 15, lg = lane >> 4, wave = t >> 6;
  const int64_t b = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  const int m = li < M ? li : M - 1;
  uint4 w[4], a[kRT][4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int64_t k = b * 128 + 32 * c + 8 * lg;
    w[c] = k < L ? *reinterpret_cast<const uint4*>(x + m * L + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kRT; ++i) {
      const int j = 16 * i + li;
      a[i][c] = load_bf16x8(A + j * L + k, j < r && k < L ? 8 : 0, vec_a);
    }
  }
  const typename Q::Block q = Q::quantize(w);
  if (out_q.codes && li < M && b * 128 < L) {
    out_q.store_scale(q, b, li, lg);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t at = b * Q::kBytes + (4 * c + lg) * static_cast<int>(sizeof(q.c[0]));
      if (at < out_q.pitch)
        *reinterpret_cast<typename Q::Codes*>(out_q.codes + li * out_q.pitch + at) = q.c[c];
    }
  }
#pragma unroll
  for (int i = 0; i < kRT; ++i) {
    f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c) acc = mfma_bf16_32(a[i][c], w[c], acc);
    s_part[wave][i][lane] = acc;
  }
  __syncthreads();
  // lane (li, lg): ranks 16 i + 4 lg .. + 3 of token li; wave i's tiles
  for (int i = wave; i < kRT; i += 4) {
    const f32x4_t u = s_part[0][i][lane] + s_part[1][i][lane] + s_part[2][i][lane] +
                      s_part[3][i][lane];
    float* out = part + (static_cast<int64_t>(blockIdx.x) * M + li) * r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = 16 * i + 4 * lg + e;
      if (li < M && j < r) out[j] = u[e];
    }
  }
}

// Slices of the contraction: enough workgroups to fill the chip for small
// batches, one pass of a few blocks each for large ones.
inline int project_blocks_per_slice(int64_t M, int64_t L) {
  const int64_t blocks = (L + 127) / 128, groups = (M + 63) / 64;
  int64_t slices = (512 + groups - 1) / groups;
  slices = slices < blocks ? slices : blocks;
  return static_cast<int>((blocks + slices - 1) / slices);
}

template <typename Q>
hipError_t go_quantize_project(const uint16_t* x, int64_t M, int64_t L, const uint16_t* P, int r,
                               bool rows_l, const Q& q, int slices, float* part, hipStream_t st) {
  if (M == 0) return hipSuccess;
  const int waves = rows_l && M <= 16 ? 1 : 4;
  const dim3 grid(static_cast<uint32_t>((M + 16 * waves - 1) / (16 * waves)),
                  static_cast<uint32_t>(slices));
  // rows of P can be read 16 bytes at a time (a row of A has L values, a
  // multiple of 16; a row of B has r)
  const bool vec_p = (reinterpret_cast<uintptr_t>(P) & 15) == 0 && (!rows_l || (r & 7) == 0);
  const int per = project_blocks_per_slice(M, L);
  auto go = [&](auto k) {
    hipLaunchKernelGGL(k, grid, dim3(64 * waves), 0, st, x, M, L, P, r, vec_p, per, q, part);
    return hipGetLastError();
  };
  if constexpr (Q::kForward) {
    if (!rows_l)
      return r <= 16   ? go(quantize_project_kernel<Q, false, 1, 4>)
             : r <= 32 ? go(quantize_project_kernel<Q, false, 2, 4>)
             : r <= 64 ? go(quantize_project_kernel<Q, false, 4, 4>)
                       : go(quantize_project_kernel<Q, false, 8, 4>);
  }
  if constexpr (Q::kBackward) {
    if (waves == 1)
      return r <= 16   ? go(quantize_project_kernel<Q, true, 1, 1>)
             : r <= 32 ? go(quantize_project_kernel<Q, true, 2, 1>)
             : r <= 64 ? go(quantize_project_kernel<Q, true, 4, 1>)
                       : go(quantize_project_kernel<Q, true, 8, 1>);
    return r <= 16   ? go(quantize_project_kernel<Q, true, 1, 4>)
           : r <= 32 ? go(quantize_project_kernel<Q, true, 2, 4>)
           : r <= 64 ? go(quantize_project_kernel<Q, true, 4, 4>)
                     : go(quantize_project_kernel<Q, true, 8, 4>);
  }
  return hipErrorInvalidValue;
}

template <typename Q>
hipError_t go_decode_project(const uint16_t* x, int M, int64_t L, const uint16_t* A, int r,
                             const Q& q, int slices, float* part, hipStream_t st) {
  const bool vec_a = (reinterpret_cast<uintptr_t>(A) & 15) == 0;
  auto go = [&](auto k) {
    hipLaunchKernelGGL(k, dim3(static_cast<uint32_t>(slices)), dim3(256), 0, st, x, M, L, A, r,
                       vec_a, q, part);
    return hipGetLastError();
  };
  return r <= 16   ? go(decode_project_kernel<Q, 1>)
         : r <= 32 ? go(decode_project_kernel<Q, 2>)
         : r <= 64 ? go(decode_project_kernel<Q, 4>)
                   : go(decode_project_kernel<Q, 8>);
}

}  // namespace qn
