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

namespace qn {

namespace {

constexpr int kT = 256;

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
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;
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

template <bool kRowsL, int kRT, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void quantize_project_kernel(
    const uint16_t* __restrict__ x, int64_t M, int64_t L, const uint16_t* __restrict__ P, int r,
    bool vec_p, int per_slice, uint8_t* __restrict__ codes, float* __restrict__ scale,
    float* __restrict__ part) {
  constexpr int kThreads = 64 * kWaves;
  constexpr int kLoads = kRT * 256 / kThreads;  // 16-byte chunks of P per thread and block
  static_assert(kLoads * kThreads == kRT * 256, "P tile split");
  constexpr int kQPitch = 128 + 16;
  __shared__ __attribute__((aligned(16))) uint16_t sP[2][kRT * 16 * 128];
  __shared__ __attribute__((aligned(16))) uint8_t sQ[kWaves][16 * kQPitch];
  const int t = threadIdx.x, lane = t & 63, li = lane & 15, lg = lane >> 4;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * kWaves + (t >> 6)) * 16 + li;
  const int64_t m = row < M ? row : M - 1;
  const int64_t blocks = (L + 127) / 128;
  const int64_t b0 = static_cast<int64_t>(blockIdx.y) * per_slice;
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
    uint16_t* sp = sP[(b - b0) & 1];
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
    float v[4][8];
    u16x2_t am{0, 0};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      bf16x8_to_f32(cur[c], v[c]);
      am = absmax_pair(am, cur[c]);
    }
    const float s = fp8_scale(lanes_max<16, 32>(absmax_bits(am))), inv = __fdiv_rn(1.0f, s);
    if (row < M && lg == 0) scale[b * M + row] = s;
    // the codes leave as whole 128-byte rows, 8 of them per store (8 bytes of
    // 16 rows per store took 40% longer for the whole kernel); sQ is the
    // wave's own, so the order of its LDS accesses keeps the turns apart
    uint8_t* sq = sQ[t >> 6];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint2*>(sq + li * kQPitch + 32 * c + 8 * lg) = fp8_codes8(v[c], s, inv);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int rr = 8 * h + (lane >> 3);
      const int64_t to = row - li + rr, k = b * 128 + (lane & 7) * 16;
      const uint4 q = *reinterpret_cast<const uint4*>(sq + rr * kQPitch + (lane & 7) * 16);
      if (to < M && k < L) *reinterpret_cast<uint4*>(codes + to * L + k) = q;
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
  float* out = part + (static_cast<int64_t>(blockIdx.y) * M + row) * r;
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

// The same for the decode path (up to 16 tokens, P = A): a wave takes one
// block, with A's fragments straight in registers, everything asked for at
// once; the four waves' sums are added in LDS, so that the product's
// workgroups, which all add up the slices, find a quarter as many.  16 tokens
// of 11008 values, r = 16: 4 us, one round trip to memory.
template <int kRT>
__global__ __launch_bounds__(kT) void decode_project_kernel(
    const uint16_t* __restrict__ x, int M, int64_t L, const uint16_t* __restrict__ A, int r,
    bool vec_a, uint8_t* __restrict__ codes, float* __restrict__ scale, float* __restrict__ part) {
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
  float v[4][8];
  u16x2_t am{0, 0};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    bf16x8_to_f32(w[c], v[c]);
    am = absmax_pair(am, w[c]);
  }
  const float s = fp8_scale(lanes_max<16, 32>(absmax_bits(am))), inv = __fdiv_rn(1.0f, s);
  if (codes && li < M && b * 128 < L) {
    if (lg == 0) scale[b * M + li] = s;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t k = b * 128 + 32 * c + 8 * lg;
      if (k < L) *reinterpret_cast<uint2*>(codes + li * L + k) = fp8_codes8(v[c], s, inv);
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
  const int waves = rows_l && M <= 16 ? 1 : 4;
  const dim3 grid(static_cast<uint32_t>((M + 16 * waves - 1) / (16 * waves)),
                  static_cast<uint32_t>(fp8_project_slices(M, L)));
  // rows of P can be read 16 bytes at a time (a row of A has L values, a
  // multiple of 16; a row of B has r)
  const bool vec_p = (reinterpret_cast<uintptr_t>(P) & 15) == 0 && (!rows_l || (r & 7) == 0);
  const int per = blocks_per_slice(M, L);
  auto go = [&](auto k) {
    hipLaunchKernelGGL(k, grid, dim3(64 * waves), 0, st, x, M, L, P, r, vec_p, per, codes, scale,
                       part);
    return hipGetLastError();
  };
  if (!rows_l)
    return r <= 16   ? go(quantize_project_kernel<false, 1, 4>)
           : r <= 32 ? go(quantize_project_kernel<false, 2, 4>)
           : r <= 64 ? go(quantize_project_kernel<false, 4, 4>)
                     : go(quantize_project_kernel<false, 8, 4>);
  if (waves == 1)
    return r <= 16   ? go(quantize_project_kernel<true, 1, 1>)
           : r <= 32 ? go(quantize_project_kernel<true, 2, 1>)
           : r <= 64 ? go(quantize_project_kernel<true, 4, 1>)
                     : go(quantize_project_kernel<true, 8, 1>);
  return r <= 16   ? go(quantize_project_kernel<true, 1, 4>)
         : r <= 32 ? go(quantize_project_kernel<true, 2, 4>)
         : r <= 64 ? go(quantize_project_kernel<true, 4, 4>)
                   : go(quantize_project_kernel<true, 8, 4>);
}

int fp8_decode_slices(int64_t L) { return static_cast<int>(((L + 127) / 128 + 3) / 4); }

hipError_t launch_fp8_decode_project(const uint16_t* x, int M, int64_t L, const uint16_t* A, int r,
                                     uint8_t* codes, float* scale, float* part, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>(fp8_decode_slices(L)));
  const bool vec_a = (reinterpret_cast<uintptr_t>(A) & 15) == 0;
  auto go = [&](auto k) {
    hipLaunchKernelGGL(k, grid, dim3(kT), 0, st, x, M, L, A, r, vec_a, codes, scale, part);
    return hipGetLastError();
  };
  return r <= 16   ? go(decode_project_kernel<1>)
         : r <= 32 ? go(decode_project_kernel<2>)
         : r <= 64 ? go(decode_project_kernel<4>)
                   : go(decode_project_kernel<8>);
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
