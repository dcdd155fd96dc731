// Microscaled 4-bit quantisation (gfx950): a matrix to E2M1 codes with one
// power of two per 32 values of a row, its values back, scales between rows
// and tiles, the batches of the linear layer together with their LoRA
// projection, and the weight turned for the backward's product.

#include "qn_launch.h"
#include "qn_mx.h"
#include "qn_project.h"

namespace qn {

namespace {

constexpr int kT = 256;

// One workgroup per tile of scales, 32 rows x 256 columns: 32 lanes span a
// row's 256 columns, 4 of them a group, the workgroup 8 rows at a time, and all
// four passes are loaded before the first is used.  The tile's scale bytes
// meet in LDS and leave as 256 consecutive bytes.
//
// Bound by HBM.  Workgroups follow the rows, not the order of the tiles in memory,
// which goes down the columns: 11008 x 4096 bf16 32.6 -> 26.1 us (4.4 TB/s), 22016
// x 8192 106 -> 84 (5.5), fp32 11008 x 4096 52 -> 45 (4.5).
template <typename T>
__global__ __launch_bounds__(kT) void mx_quantize_kernel(const T* __restrict__ x, int64_t R,
                                                         int64_t K, uint8_t* __restrict__ codes,
                                                         uint32_t* __restrict__ scale) {
  __shared__ __attribute__((aligned(4))) uint8_t s_byte[256];
  const int64_t kt = (K + 255) / 256, br = blockIdx.x / kt, bk = blockIdx.x % kt;
  const int64_t tile_at = bk * ((R + 31) / 32) + br;
  const int t = threadIdx.x, sub = t >> 5;
  const int64_t k = bk * 256 + (t & 31) * 8, r0 = br * 32 + sub;
  Raw8<T> v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (k < K && r0 + 8 * i < R) load8(x + (r0 + 8 * i) * K + k, v[i]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = mx4_scale(lanes_max<1, 2>(absmax8(v[i])));
    const float s = mx_power(b);
    uint32_t c;
    if constexpr (sizeof(T) == 2) {
      c = mx4_codes8(v[i].w[0], s);
    } else {
      float f[8];
      values8(v[i], f);
      c = mx4_codes8(f, s);
    }
    const int row = sub + 8 * i, g = (t & 31) >> 2;  // row and group in the tile
    if ((t & 3) == 0)
      s_byte[((g & 3) * 16 + (row & 15)) * 4 + (row >> 4) * 2 + (g >> 2)] = static_cast<uint8_t>(b);
    if (k < K && r0 + 8 * i < R)
      *reinterpret_cast<uint32_t*>(codes + ((r0 + 8 * i) * K + k) / 2) = c;
  }
  __syncthreads();
  if (t < 64)
    scale[tile_at * 64 + t] = reinterpret_cast<const uint32_t*>(s_byte)[t];
}

// The values back, in the same split of the work: 8 codes per lane and pass;
// 11008 x 4096 to bf16 21.5 us (5.3 TB/s).
template <typename T>
__global__ __launch_bounds__(kT) void mx_dequant_kernel(const uint8_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scale,
                                                        int64_t R, int64_t K, T* __restrict__ out) {
  const int64_t kt = (K + 255) / 256, br = blockIdx.x / kt, bk = blockIdx.x % kt;
  const int64_t tile_at = bk * ((R + 31) / 32) + br;
  const int t = threadIdx.x, sub = t >> 5, g = (t & 31) >> 2;
  const int64_t k = bk * 256 + (t & 31) * 8, r0 = br * 32 + sub;
  if (k >= K) return;
  const uint8_t* tile = scale + tile_at * 256;
  uint32_t c[4], b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = sub + 8 * i;
    c[i] = 0, b[i] = 0;
    if (r0 + 8 * i < R) {
      c[i] = *reinterpret_cast<const uint32_t*>(codes + ((r0 + 8 * i) * K + k) / 2);
      b[i] = tile[((g & 3) * 16 + (row & 15)) * 4 + (row >> 4) * 2 + (g >> 2)];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (r0 + 8 * i >= R) return;
    // a NaN scale is put in by hand: the conversion takes the power's exponent
    const float s = mx_power(b[i]), nan = b[i] == 255 ? s : 0.0f;
    const auto f0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], s, 0);
    const auto f1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], s, 1);
    const auto f2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], s, 2);
    const auto f3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], s, 3);
    float v[8] = {f0[0], f0[1], f1[0], f1[1], f2[0], f2[1], f3[0], f3[1]};
    if (b[i] == 255)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = nan;
    T* o = out + (r0 + 8 * i) * K + k;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
  }
}

// Scales between rows [R, K / 32] and tiles, a tile byte per thread.
template <bool kPack>
__global__ __launch_bounds__(kT) void mx_scales_kernel(const uint8_t* __restrict__ in, int64_t R,
                                                       int64_t groups, uint8_t* __restrict__ out) {
  const int64_t rt = (R + 31) / 32;
  const int64_t bk = blockIdx.x / rt, br = blockIdx.x % rt;
  const int t = threadIdx.x, lane = t >> 2, h = (t >> 1) & 1, j = t & 1;
  const int64_t row = br * 32 + 16 * h + (lane & 15), g = bk * 8 + 4 * j + (lane >> 4);
  const bool in_rows = row < R && g < groups;
  const int64_t tile = static_cast<int64_t>(blockIdx.x) * 256 + t;
  if constexpr (kPack)
    out[tile] = in_rows ? in[row * groups + g] : uint8_t{0};
  else if (in_rows)
    out[row * groups + g] = in[tile];
}

// Of the projection kernels, forward: E2M1 codes, a scale per 32 columns.
struct Mx4Rows {
  typedef uint32_t Codes;
  static constexpr int kBytes = 64;
  static constexpr bool kForward = true, kBackward = false;
  uint8_t* codes;
  int64_t pitch;  // bytes of a token
  uint8_t* scale;
  int64_t tiles;  // of 32 tokens
  int64_t blocks;

  struct Block {
    Codes c[4];
    uint32_t b[4];
  };
  __device__ __forceinline__ static Block quantize(const uint4 (&x)[4]) {
    Block q;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      q.b[c] = mx4_scale(lanes_max<16, 32>(absmax_bits(absmax_pair(u16x2_t{0, 0}, x[c]))));
      q.c[c] = mx4_codes8(x[c], mx_power(q.b[c]));
    }
    return q;
  }
  __device__ __forceinline__ void store_scale(const Block& q, int64_t b, int64_t row, int lg) const {
    const uint32_t v = lg == 0 ? q.b[0] : lg == 1 ? q.b[1] : lg == 2 ? q.b[2] : q.b[3];
    uint8_t* at = scale + (((b >> 1) * tiles + (row >> 5)) * 64 + lg * 16 + (row & 15)) * 4 +
                  ((row >> 4) & 1) * 2;
    at[b & 1] = static_cast<uint8_t>(v);
    // the half of the last tile that no block fills
    if (b + 1 == blocks && (b & 1) == 0) at[1] = 0;
  }
};

// Backward: E4M3 codes, rows padded with zeros to whole blocks.
struct Mx8Rows {
  typedef uint2 Codes;
  static constexpr int kBytes = 128;
  static constexpr bool kForward = false, kBackward = false;  // mx_backward_kernel
  uint8_t* codes;
  int64_t pitch;
  uint8_t* scale;
  int64_t tiles;  // of 64 tokens

  struct Block {
    Codes c[4];
    uint32_t b[4];
  };
  __device__ __forceinline__ static Block quantize(const uint4 (&x)[4]) {
    Block q;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float v[8];
      bf16x8_to_f32(x[c], v);
      q.b[c] = mx8_scale(lanes_max<16, 32>(absmax_bits(absmax_pair(u16x2_t{0, 0}, x[c]))));
      q.c[c] = mx8_codes8(v, q.b[c]);
    }
    return q;
  }
  __device__ __forceinline__ void store_scale(const Block& q, int64_t b, int64_t row, int lg) const {
    const uint32_t v = lg == 0 ? q.b[0] : lg == 1 ? q.b[1] : lg == 2 ? q.b[2] : q.b[3];
    scale[((b * tiles + (row >> 6)) * 64 + lg * 16 + (row & 15)) * 4 + ((row >> 4) & 3)] =
        static_cast<uint8_t>(v);
  }
};

// The same without a projection: 16 lanes per block of 128 columns of a row, 8
// values each, a workgroup 16 rows of one block.
template <typename Q>
__global__ __launch_bounds__(kT) void mx_rows_kernel(const uint16_t* __restrict__ x, int64_t M,
                                                     int64_t L, int64_t blocks, Q out) {
  const int64_t b = blockIdx.x % blocks, m = blockIdx.x / blocks * 16 + (threadIdx.x >> 4);
  const int g8 = threadIdx.x & 15;  // 8 columns of the block; 4 lanes a group
  const int64_t k = b * 128 + g8 * 8;
  Raw8<uint16_t> raw;
  if (m < M && k < L) load8(x + m * L + k, raw);
  const uint32_t amax = lanes_max<1, 2>(absmax8(raw));
  typename Q::Block q;
  uint32_t byte;
  if constexpr (Q::kForward) {
    byte = mx4_scale(amax);
    q.c[0] = mx4_codes8(raw.w[0], mx_power(byte));
  } else {
    float v[8];
    values8(raw, v);
    byte = mx8_scale(amax);
    q.c[0] = mx8_codes8(v, byte);
  }
  if (m >= M) return;
  const int64_t at = b * Q::kBytes + g8 * static_cast<int>(sizeof(q.c[0]));
  if (at < out.pitch) *reinterpret_cast<typename Q::Codes*>(out.codes + m * out.pitch + at) = q.c[0];
  if ((g8 & 3) == 0) {
#pragma unroll
    for (int c = 0; c < 4; ++c) q.b[c] = byte;
    out.store_scale(q, b, m, g8 >> 2);
  }
}

// The weight for the backward's product, whose contraction runs over the rows:
// W^T as E5M2 codes [K, Np] (rows of zeros behind N, Np the next multiple of
// 128) with one power of two per 32 rows n of a column k.  All 32 x 32 values
// of a block take the largest scale of its rows, 13 powers down, so that the
// largest code, 6, becomes 6 2^13 of at most 57344: an E2M1 number over a row's
// own scale is an E5M2 number over the block's for scales up to 2^26 apart, and
// what lies further below is read as 0.  A workgroup turns 128 x 128 values:
// a row's group of 32 codes is decoded through a table of its 8 magnitudes (8
// bytes in two registers, looked up by byte permutes), lies [n][k] in LDS, and
// is read by the transposing LDS loads, 8 n of a k at a time.
typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2_t lds_i32x2_t;
typedef __attribute__((address_space(3))) uint8_t lds_u8_t;

__device__ __forceinline__ void turn_tile(const uint8_t* __restrict__ codes,
                                          const uint8_t* __restrict__ scale, int64_t N, int64_t K,
                                          int64_t Np, uint8_t* __restrict__ wt,
                                          uint8_t* __restrict__ ts, int64_t tile, uint8_t* s_w) {
  const int64_t nbn = Np / 128;
  const int64_t n0 = tile % nbn * 128, k0 = tile / nbn * 128;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t rt = (N + 31) / 32, kt = (K + 63) / 64;
  // row n0 + 32 wave + lane % 32, groups lane / 32 and 2 + lane / 32 of the
  // block's four; the 32 lanes of a half wave hold the 32 rows of a block
  const int64_t n = n0 + 32 * wave + (lane & 31);
  uint4 c[2];
  uint32_t b[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t g = k0 / 32 + 2 * i + (lane >> 5);
    c[i] = make_uint4(0, 0, 0, 0);
    b[i] = 0;
    if (n < N && g * 32 < K) {
      c[i] = *reinterpret_cast<const uint4*>(codes + n * (K / 2) + g * 16);
      b[i] = scale[(((g >> 3) * rt + (n >> 5)) * 64 + (g & 3) * 16 + (n & 15)) * 4 +
                   ((n >> 4) & 1) * 2 + ((g >> 2) & 1)];
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int gl = 2 * i + (lane >> 5);
    const uint32_t most = lanes_max<1, 16>(b[i]);
    const int base = most == 255 ? 255 : most > 13 ? static_cast<int>(most) - 13 : 0;
    const int d = static_cast<int>(b[i]) - base;  // at most 13
    uint32_t lo = 0, hi = 0;  // E5M2 of 0, 0.5, 1, 1.5 and 2, 3, 4, 6 times 2^d
    if (d >= -13) {
      const uint32_t up = static_cast<uint32_t>(d + 13) * 4;
      lo = 0x3E3C3800u - 0x34343400u + 0x01010100u * up;
      hi = 0x46444240u - 0x34343434u + 0x01010101u * up;
    }
    const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
    uint32_t o[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // the even columns' magnitudes and signs, the odd ones', then in order
      const uint32_t e = __builtin_amdgcn_perm(hi, lo, w[q] & 0x07070707u) |
                         ((w[q] << 4) & 0x80808080u);
      const uint32_t f = __builtin_amdgcn_perm(hi, lo, (w[q] >> 4) & 0x07070707u) |
                         (w[q] & 0x80808080u);
      o[2 * q] = __builtin_amdgcn_perm(f, e, 0x05010400u);
      o[2 * q + 1] = __builtin_amdgcn_perm(f, e, 0x07030602u);
    }
    // 16-byte chunk ch of row r in place ch ^ (r & 7)
    const int r = 32 * wave + (lane & 31);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<uint4*>(s_w + r * 128 + (((2 * gl + h) ^ (r & 7)) << 4)) =
          make_uint4(o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]);
    // tile [Np / 128][K / 64]: byte k % 64 / 16 of register (n % 128 / 32, k % 16)
    const int64_t k = k0 + 32 * gl + (lane & 31);
    if (k < K)
      ts[((n0 / 128 * kt + (k >> 6)) * 64 + wave * 16 + (k & 15)) * 4 + ((k >> 4) & 3)] =
          static_cast<uint8_t>(base);
  }
  __syncthreads();
  // A transposing read gives lane c of 16 column c of 8 rows, lanes 2 r, 2 r + 1
  // pointing at row r.  Wave w takes columns 32 w .. + 31, a group of 16 lanes
  // the rows 32 g .. + 31 of 16 columns at a time: 32 bytes of a row of W^T each.
  const int li = lane & 15, lg = lane >> 4;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int ch = 2 * wave + h;
    uint32_t o[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = 32 * lg + 8 * q + (li >> 1);
      const i32x2_t v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (lds_i32x2_t*)(lds_u8_t*)(s_w + r * 128 + ((ch ^ (r & 7)) << 4) + (li & 1) * 8));
      o[2 * q] = static_cast<uint32_t>(v[0]);
      o[2 * q + 1] = static_cast<uint32_t>(v[1]);
    }
    const int64_t k = k0 + 16 * ch + li;
    if (k < K) {
      uint8_t* to = wt + k * Np + n0 + 32 * lg;
      *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(to + 16) = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

__global__ __launch_bounds__(kT) void mx_turn_kernel(const uint8_t* __restrict__ codes,
                                                     const uint8_t* __restrict__ scale, int64_t N,
                                                     int64_t K, int64_t Np,
                                                     uint8_t* __restrict__ wt,
                                                     uint8_t* __restrict__ ts) {
  __shared__ __attribute__((aligned(16))) uint8_t s_w[128 * 128];
  turn_tile(codes, scale, N, K, Np, wt, ts, blockIdx.x, s_w);
}

// Both in one launch: the first workgroups quantise and project the batch, which
// waits on memory more than it reads, the others turn the weight meanwhile.  2048
// tokens, 11008 x 4096, r = 64, 137 MB: 35.7 us (3.8 TB/s); as two launches 23 and
// 12.2, and the call 124 -> 118 us; 333 tokens, 1088 x 2112 20 -> 17.
template <int kRT>
__global__ __launch_bounds__(kT) void mx_backward_kernel(
    const uint16_t* __restrict__ x, int64_t M, int64_t L, const uint16_t* __restrict__ P, int r,
    bool vec_p, int per_slice, Mx8Rows out_q, float* __restrict__ part, int slices, int projecting,
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scale, int64_t K,
    uint8_t* __restrict__ wt, uint8_t* __restrict__ ts) {
  typedef ProjectLds<Mx8Rows, kRT, 4> Lds;
  constexpr int kBytes = sizeof(Lds) > 128 * 128 ? sizeof(Lds) : 128 * 128;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kBytes];
  const int bid = blockIdx.x;
  if (bid < projecting)
    quantize_project<Mx8Rows, true, kRT, 4>(x, M, L, P, r, vec_p, per_slice, out_q, part,
                                            bid / slices, bid % slices,
                                            *reinterpret_cast<Lds*>(lds));
  else
    turn_tile(codes, scale, L, K, out_q.pitch, wt, ts, bid - projecting, lds);
}

}  // namespace

hipError_t launch_mx_quantize(const void* x, bool bf16, int64_t R, int64_t K, uint8_t* codes,
                              uint8_t* scale, hipStream_t st) {
  const int64_t tiles = mx_tiles(R, 32) * mx_tiles(K, 256);
  if (tiles == 0) return hipSuccess;
  const dim3 grid(static_cast<uint32_t>(tiles));
  uint32_t* s = reinterpret_cast<uint32_t*>(scale);
  if (bf16)
    hipLaunchKernelGGL(mx_quantize_kernel<uint16_t>, grid, dim3(kT), 0, st,
                       static_cast<const uint16_t*>(x), R, K, codes, s);
  else
    hipLaunchKernelGGL(mx_quantize_kernel<float>, grid, dim3(kT), 0, st,
                       static_cast<const float*>(x), R, K, codes, s);
  return hipGetLastError();
}

hipError_t launch_mx_dequant(const MxView& w, bool out_bf16, void* out, hipStream_t st) {
  const int64_t tiles = mx_tiles(w.N, 32) * mx_tiles(w.K, 256);
  if (tiles == 0) return hipSuccess;
  const dim3 grid(static_cast<uint32_t>(tiles));
  if (out_bf16)
    hipLaunchKernelGGL(mx_dequant_kernel<uint16_t>, grid, dim3(kT), 0, st, w.codes, w.scale, w.N,
                       w.K, static_cast<uint16_t*>(out));
  else
    hipLaunchKernelGGL(mx_dequant_kernel<float>, grid, dim3(kT), 0, st, w.codes, w.scale, w.N, w.K,
                       static_cast<float*>(out));
  return hipGetLastError();
}

hipError_t launch_mx_scales(bool pack, const uint8_t* in, int64_t R, int64_t K, uint8_t* out,
                            hipStream_t st) {
  const int64_t tiles = mx_tiles(R, 32) * mx_tiles(K, 256);
  if (tiles == 0) return hipSuccess;
  const dim3 grid(static_cast<uint32_t>(tiles));
  if (pack)
    hipLaunchKernelGGL(mx_scales_kernel<true>, grid, dim3(kT), 0, st, in, R, K / 32, out);
  else
    hipLaunchKernelGGL(mx_scales_kernel<false>, grid, dim3(kT), 0, st, in, R, K / 32, out);
  return hipGetLastError();
}

static Mx4Rows rows4(uint8_t* codes, uint8_t* scale, int64_t M, int64_t K) {
  return Mx4Rows{codes, K / 2, scale, mx_tiles(M, 32), mx_tiles(K, 128)};
}

hipError_t launch_mx_rows(const uint16_t* x, int64_t M, int64_t L, bool bwd, uint8_t* codes,
                          uint8_t* scale, hipStream_t st) {
  const int64_t blocks = mx_tiles(L, 128), groups = mx_tiles(M, 16) * blocks;
  if (groups == 0) return hipSuccess;
  const dim3 grid(static_cast<uint32_t>(groups));
  if (bwd)
    hipLaunchKernelGGL(mx_rows_kernel<Mx8Rows>, grid, dim3(kT), 0, st, x, M, L, blocks,
                       Mx8Rows{codes, blocks * 128, scale, mx_tiles(M, 64)});
  else
    hipLaunchKernelGGL(mx_rows_kernel<Mx4Rows>, grid, dim3(kT), 0, st, x, M, L, blocks,
                       rows4(codes, scale, M, L));
  return hipGetLastError();
}

hipError_t launch_mx_rows_project(const uint16_t* x, int64_t M, int64_t L, const uint16_t* A, int r,
                                  uint8_t* codes, uint8_t* scale, float* part, hipStream_t st) {
  return go_quantize_project(x, M, L, A, r, false, rows4(codes, scale, M, L),
                             fp8_project_slices(M, L), part, st);
}

hipError_t launch_mx_backward(const MxView& w, const uint16_t* dy, int64_t M, const uint16_t* B,
                              int r, uint8_t* codes, uint8_t* scale, float* part, uint8_t* wt,
                              uint8_t* ts, hipStream_t st) {
  if (M == 0) return hipSuccess;
  const int slices = fp8_project_slices(M, w.N), per = project_blocks_per_slice(M, w.N);
  const int64_t projecting = mx_tiles(M, 64) * slices;
  const int64_t turning = mx_tiles(w.N, 128) * mx_tiles(w.K, 128);
  const bool vec = (reinterpret_cast<uintptr_t>(B) & 15) == 0 && (r & 7) == 0;
  auto go = [&](auto k) {
    hipLaunchKernelGGL(k, dim3(static_cast<uint32_t>(projecting + turning)), dim3(kT), 0, st, dy, M,
                       w.N, B, r, vec, per,
                       Mx8Rows{codes, mx_tiles(w.N, 128) * 128, scale, mx_tiles(M, 64)}, part,
                       slices, static_cast<int>(projecting), w.codes, w.scale, w.K, wt, ts);
    return hipGetLastError();
  };
  return r <= 16   ? go(mx_backward_kernel<1>)
         : r <= 32 ? go(mx_backward_kernel<2>)
         : r <= 64 ? go(mx_backward_kernel<4>)
                   : go(mx_backward_kernel<8>);
}

hipError_t launch_mx_decode_project(const uint16_t* x, int M, int64_t L, const uint16_t* A, int r,
                                    uint8_t* codes, uint8_t* scale, float* part, hipStream_t st) {
  return go_decode_project(x, M, L, A, r, rows4(codes, scale, M, L), fp8_decode_slices(L), part,
                           st);
}

hipError_t launch_mx_turn(const MxView& w, uint8_t* wt, uint8_t* ts, hipStream_t st) {
  const int64_t nbn = mx_tiles(w.N, 128);
  const dim3 grid(static_cast<uint32_t>(nbn * mx_tiles(w.K, 128)));
  hipLaunchKernelGGL(mx_turn_kernel, grid, dim3(kT), 0, st, w.codes, w.scale, w.N, w.K, nbn * 128,
                     wt, ts);
  return hipGetLastError();
}

}  // namespace qn
