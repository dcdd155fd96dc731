// Microscaled products for few tokens, up to 64 (gfx950).
//
//   y[m, n] = xq[m] . wq[n] + (s u) B^T
//
// Bound by reading the weight once (17 N K / 32 bytes).  A workgroup owns 16
// output columns (or 32, see the launch) and the whole contraction: its waves
// take the runs of 256 in turn, each run two 16x16x128 MFMAs with the weight's
// rows as the first operand and 16 tokens (the last one again past the end) as
// the second, the powers of two multiplied in by the instruction.  Every lane
// loads two 16-byte chunks of its row straight into its fragments, and the run's
// scales as one register, some runs ahead of their products.  The waves' fp32
// sums meet in LDS and are added in wave order, so results are
// bit-reproducible.
//
// One token: the same launch quantises x, each wave for its own runs, and,
// where the adapter is small, computes u = x A^T.  More tokens: x's codes and
// u's partial sums come from a launch before.
//
// Times of calls in a graph, the weight not in the caches, r = 16: one token on
// 4096 x 4096 8.3 us (without an adapter 4.6, the bytes at a large copy's rate
// 1.8), on 22016 x 8192 25.6 (22.1, 18.9); 16 tokens on 4096 x 4096 10.6, on 4096 x
// 11008 15.3 (4.9), on 22016 x 8192 31.1.  Small calls are a chain of latencies:
// launch, load, sum over the waves, LoRA term; with many tokens it is x's codes,
// which every workgroup reads from the L2 caches.  16 waves a workgroup: one token
// the same within 10%, 16 tokens 10.8 -> 13.6 us and 15.4 -> 18.2.

#include "qn_decode.h"
#include "qn_launch.h"
#include "qn_mx.h"

namespace qn {

namespace {

// Chunks lg and 4 + lg of run b of a row of K / 2 bytes, zeros behind its end.
struct Run {
  uint4 lo, hi;
};

__device__ __forceinline__ Run row_run(const uint8_t* row, int64_t b, int64_t groups, int lg) {
  const int64_t g = b * 8 + lg;
  Run v{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (g < groups) v.lo = *reinterpret_cast<const uint4*>(row + g * 16);
  if (g + 4 < groups) v.hi = *reinterpret_cast<const uint4*>(row + (g + 4) * 16);
  return v;
}

// acc += W x^T over a run; ws and xs hold the two chunks' scale bytes at places
// 0 and 1.
__device__ __forceinline__ f32x4_t run_product(const Run& w, const Run& x, f32x4_t acc, int ws,
                                               int xs) {
  acc = mfma_mx<kE2M1, kE2M1>(frag4(w.lo), frag4(x.lo), acc, 0, ws, 0, xs);
  return mfma_mx<kE2M1, kE2M1>(frag4(w.hi), frag4(x.hi), acc, 1, ws, 1, xs);
}

template <int kU, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void mx_token_kernel(
    const uint8_t* __restrict__ w, const uint32_t* __restrict__ ws, int64_t N, int64_t K,
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ A, bool vec_a,
    const float* __restrict__ part, int slices, const uint16_t* __restrict__ B, int r, bool vec_b,
    float lora_scale, uint16_t* __restrict__ y, uint16_t* __restrict__ u_out) {
  constexpr int kThreads = 64 * kWaves, kAhead = 2;
  constexpr int kFrags = kU == kGivenU ? kDecodeMaxRank / 32 : 1;
  __shared__ f32x4_t s_acc[kWaves][4];
  __shared__ float s_u[kU == kNoAdapter ? 1 : kThreads];  // kOwnU: [wave][16 ranks]
  __shared__ __attribute__((aligned(16))) uint16_t s_us[64 * kFrags];
  __shared__ __attribute__((aligned(16))) uint2 s_x[kU == kOwnU ? kWaves : 1][kAhead][64];
  __shared__ __attribute__((aligned(16))) uint16_t s_q[kWaves][kAhead][64];  // 4 codes a lane
  const int t = threadIdx.x, lane = t & 63;
  // the wave's part is turned by the workgroup, so that the CUs of an XCD do not
  // ask its L2 for the same lines of A at the same time (4096 x 4096, r = 8 7.3 -> 7.0
  // us)
  const int wave = __builtin_amdgcn_readfirstlane(((t >> 6) + (blockIdx.x >> 3)) & (kWaves - 1));
  static_assert((kWaves & (kWaves - 1)) == 0, "the turn is a bijection");
  const int li = lane & 15, lg = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;  // N is a multiple of 16
  const int64_t groups = K / 32, runs = (K + 255) / 256, rt = (N + 31) / 32;
  const uint8_t* wr = w + (n0 + li) * (K / 2);
  const uint32_t* wsr = ws + (n0 / 32) * 64 + lane;
  const int sh = static_cast<int>(n0 & 16);  // rows 16 .. 31 of a tile: bytes 2 and 3

  uint4 bf[kFrags];
  if (kU != kNoAdapter && wave == 0) load_up<kFrags>(bf, B, n0, r, li, lg, vec_b);
  if constexpr (kU == kGivenU) s_u[t] = add_slices<kThreads>(part, slices, r, t);
  f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f}, ua = acc;
  for (int64_t bw = wave; bw < runs; bw += kAhead * kWaves) {
    // everything that these runs need is asked for first
    Run wv[kAhead];
    uint2 xp[kAhead];  // 4 values of the run
    uint32_t sw[kAhead];
    uint4 av[kAhead][8];
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      const int64_t b = bw + d * kWaves;
      const bool in = b < runs;
      const int64_t k = b * 256 + 4 * lane;
      xp[d] = in && k < K ? *reinterpret_cast<const uint2*>(x + k) : make_uint2(0, 0);
      wv[d] = row_run(wr, in ? b : runs, groups, lg);
      sw[d] = in ? wsr[b * rt * 64] : 0u;
      if constexpr (kU == kOwnU) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int64_t ka = b * 256 + 32 * c + 8 * lg;
          av[d][c] = load_bf16x8(A + li * K + ka, li < r && in && ka < K ? 8 : 0, vec_a);
        }
      }
    }
    int sx[kAhead];
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      u16x2_t am = absmax_pair(absmax_pair(u16x2_t{0, 0}, xp[d].x), xp[d].y);
      const uint32_t byte = mx4_scale(lanes_max<1, 4>(absmax_bits(am)));  // 8 lanes a group
      const float s = mx_power(byte);
      uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(
          0u, __builtin_bit_cast(bf16x2_mx_t, xp[d].x), s, 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_mx_t, xp[d].y), s,
                                                    1);
      s_q[wave][d][lane] = static_cast<uint16_t>(c);
      if constexpr (kU == kOwnU) s_x[wave][d][lane] = xp[d];
      // of groups lg and 4 + lg
      sx[d] = __shfl(static_cast<int>(byte), 8 * lg, 64) |
              __shfl(static_cast<int>(byte), 32 + 8 * lg, 64) << 8;
    }
    // written and read by the same wave: its own LDS order suffices
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      const uint4* q = reinterpret_cast<const uint4*>(&s_q[wave][d][0]);
      acc = run_product(wv[d], Run{q[lg], q[4 + lg]}, acc, static_cast<int>(sw[d] >> sh), sx[d]);
      if constexpr (kU == kOwnU) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          ua = mfma_bf16_32(av[d][k],
                            *reinterpret_cast<const uint4*>(&s_x[wave][d][8 * k + 2 * lg]), ua);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next runs' values
  }
  // all 16 result columns are the same token: keep column 0
  if (li == 0) {
    s_acc[wave][lg] = acc;
    if constexpr (kU == kOwnU) *reinterpret_cast<f32x4_t*>(&s_u[16 * wave + 4 * lg]) = ua;
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int q = 0; q < kWaves; ++q) acc = q == 0 ? s_acc[0][lg] : acc + s_acc[q][lg];
  if constexpr (kU != kNoAdapter) {
    const int pitch = kU == kOwnU ? 16 : r;
    const int sums = kU == kOwnU              ? kWaves
                     : kThreads / r < slices ? kThreads / r
                                             : slices;
    acc = token_up<kFrags>(acc, bf, s_u, pitch, sums, s_us, r, lora_scale,
                           blockIdx.x == 0 ? u_out : nullptr, lane);
  }
  if (li == 0) store_columns(y + n0 + 4 * lg, acc);
}

// Up to 16 kMT tokens, codes and scales of x given; u as `slices` partial
// sums (kMT == 1), or act = s u in two parts in rows of `pitch` values.
template <int kWaves, int kMT, int kRows>
__global__ __launch_bounds__(64 * kWaves) void mx_decode_kernel(
    const uint8_t* __restrict__ w, const uint32_t* __restrict__ ws, int64_t N, int64_t K,
    const uint8_t* __restrict__ x, const uint32_t* __restrict__ xs, int M,
    const float* __restrict__ part, int slices, const uint16_t* __restrict__ act, int pitch,
    const uint16_t* __restrict__ B, int r, bool vec_b, float lora_scale, uint16_t* __restrict__ y,
    uint16_t* __restrict__ u_out) {
  constexpr int kThreads = 64 * kWaves;
  // runs in flight besides the one multiplied; with two more registers hold a
  // workgroup less (2 tokens on 22016 x 8192 27.8 -> 31.6 us, 16 on 11008 x 4096 14.7 ->
  // 15.7)
  constexpr int kAhead = 1;
  constexpr int kTiles = kMT * kRows, kXS = (kMT + 1) / 2;
  static_assert(kTiles <= kWaves, "a wave finishes 16 columns of 16 tokens");
  __shared__ f32x4_t s_acc[kWaves][kTiles][64];
  __shared__ float s_u[kMT == 1 ? kFp8DecodeM * kDecodeMaxRank : 1];
  __shared__ __attribute__((aligned(16))) uint16_t s_us[kMT == 1 ? 32 * kDecodeMaxRank : 8];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int li = lane & 15, lg = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * kRows);
  const int64_t groups = K / 32, runs = (K + 255) / 256, rt = (N + 31) / 32;
  const int64_t xt = (M + 31) / 32;
  // N is a multiple of 16: the last workgroup may have fewer rows of 16, and
  // reads its last ones again
  const uint8_t* wr[kRows];
#pragma unroll
  for (int q = 0; q < kRows; ++q)
    wr[q] = w + ((n0 + 16 * q < N ? n0 + 16 * q : N - 16) + li) * (K / 2);
  const uint32_t* wsr = ws + (n0 / 32) * 64 + lane;
  const int sh = kRows == 1 ? static_cast<int>(n0 & 16) : 0;
  int m[kMT];
#pragma unroll
  for (int i = 0; i < kMT; ++i) m[i] = 16 * i + li < M ? 16 * i + li : M - 1;
  static_assert(kRows <= 2, "the rows are one tile of scales");

  struct Step {
    Run w[kRows], x[kMT];
    uint32_t sw, sx[kXS];
  };
  auto load = [&](int64_t b, Step& d) {
    const bool in = b < runs;
#pragma unroll
    for (int q = 0; q < kRows; ++q) d.w[q] = row_run(wr[q], in ? b : runs, groups, lg);
    d.sw = in ? wsr[b * rt * 64] : 0u;
#pragma unroll
    for (int i = 0; i < kMT; ++i) d.x[i] = row_run(x + m[i] * (K / 2), in ? b : runs, groups, lg);
#pragma unroll
    for (int i = 0; i < kXS; ++i)
      d.sx[i] = in ? xs[(b * xt + (i < xt ? i : xt - 1)) * 64 + lane] : 0u;
  };
  // u = sum of its slices: `par` threads per value, as of 16 tokens for any M, so
  // that a token's result does not depend on its batch; the first kEarly slices
  // of each are asked for before anything else
  constexpr int kEarly = 8;
  const int mr = M * r, most = kFp8DecodeM * r;
  const int par = kMT == 1 && r > 0 && most <= kThreads ? kThreads / most : 1;
  float early[kEarly];
  if (kMT == 1 && r > 0) {
    const int e = t % mr, q0 = t / mr;
#pragma unroll
    for (int k = 0; k < kEarly; ++k) {
      const int q = q0 + k * par;
      early[k] = part[static_cast<int64_t>(q < slices ? q : slices - 1) * mr + e];
    }
  }
  Step blk[kAhead + 1];
#pragma unroll
  for (int d = 0; d <= kAhead; ++d) load(wave + d * kWaves, blk[d]);
  // wave 0 .. kTiles - 1 finishes token tile wave % kMT, row tile wave / kMT
  const int64_t nw = n0 + 16 * (wave / kMT);
  const bool finish = wave < kTiles && nw < N;
  uint4 bf[kDecodeMaxRank / 32];
  if (finish) load_up<kDecodeMaxRank / 32>(bf, B, nw, r, li, lg, vec_b);
  if (kMT == 1 && r > 0) {
    const int q0 = t / mr;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kEarly; ++k)
      if (q0 + k * par < slices) s += early[k];
    if (t < par * mr) s_u[t] = s;
  }

  f32x4_t acc[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int64_t b = wave; b < runs; b += (kAhead + 1) * kWaves) {
#pragma unroll
    for (int d = 0; d <= kAhead; ++d) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const int q = i / kMT, c = i % kMT;
        acc[i] = run_product(blk[d].w[q], blk[d].x[c], acc[i],
                             static_cast<int>(blk[d].sw >> (sh + 16 * q)),
                             static_cast<int>(blk[d].sx[c / 2] >> (16 * (c & 1))));
      }
      load(b + (d + kAhead + 1) * kWaves, blk[d]);
    }
  }
#pragma unroll
  for (int i = 0; i < kTiles; ++i) s_acc[wave][i][lane] = acc[i];
  if constexpr (kMT == 1) {
    if (r > 0) {
      // the slices past the early ones, and the values past the first kThreads
      for (int i = t; i < (par > 1 ? par * mr : mr); i += kThreads) {
        const int e = i % mr, q0 = i / mr;
        float s = i == t ? s_u[i] : 0.0f;
#pragma unroll 8
        for (int q = q0 + (i == t ? kEarly * par : 0); q < slices; q += par)
          s += part[static_cast<int64_t>(q) * mr + e];
        s_u[i] = s;
      }
      __syncthreads();
      spread_u<kThreads>(s_u, par, slices, mr, M, r, lora_scale, s_us,
                         blockIdx.x == 0 ? u_out : nullptr, t);
    }
  }
  __syncthreads();
  if (!finish) return;
  f32x4_t sum = s_acc[0][wave][lane];
#pragma unroll
  for (int q = 1; q < kWaves; ++q) sum += s_acc[q][wave][lane];
  const int row = 16 * (wave % kMT) + li;
  if (r > 0) {
    if constexpr (kMT == 1)
      sum = lora_up(sum, bf, s_us, 2 * ((r + 31) & ~31), r, li, lg);
    else
      sum = lora_up(sum, bf, act + static_cast<int64_t>(row < M ? row - li : M - 1 - li) * pitch,
                    pitch, r, li, lg);
  }
  // lane (li, lg): columns nw + 4 lg .. + 3 of its token
  if (row < M) store_columns(y + row * N + nw + 4 * lg, sum);
}

}  // namespace

// Past 16 tokens x's codes, which every workgroup reads, are what counts; past 64
// MiB of them in all the tiles of the large batches cost less, and from 33 tokens,
// with 16 rows of columns a workgroup, past two rounds of the CUs.  This kernel and
// the tiles, us: 17 to 32 tokens 4096 x 4096 12.5-13.2 and 17-18, 4096 x 11008 21-23 and
// 23-25, 8192 x 8192 21-22 and 24, 16384 x 4096 18-19 and 22, but 22016 x 8192 37-40 and
// 36; 33 to 64 tokens 4096 x 4096 14-16 and 19-20, 4096 x 8192 20-23 and 22-26, 8192 x
// 4096 19-23 and 20-23, but 4096 x 11008 25-29 and 25-27, 8192 x 8192 30-36 and 25-27,
// 11008 x 1024 18-19 and 14-15, 28672 x 1024 33-35 and 15-16.
bool mx_few(int64_t M, int64_t N, int64_t K) {
  const int64_t cols = N > 4096 ? N : 4096;
  return M <= kFp8DecodeM || (M <= kFp8FewM && (M <= 32 || N <= 8192) &&
                              (M + 15) / 16 * cols * K / 2 <= (int64_t{64} << 20));
}

// Every workgroup reads A, from the caches: past 32 MiB in all, or 128 KB each, a
// projection launch of its own costs less.  In this launch and in two: r = 8 on 1024
// x 4096 6.4 and 7.0 us, on 4096 x 4096 7.0 and 8.1; r = 16 on 1088 x 2112 5.2 and 6.5,
// on 4096 x 4096 8.3 and 8.1 (the host has one launch less); but r = 8 on 11008 x 4096
// 17 and 10.8, on 4096 x 11008 13 and 11.8.
bool mx_token_self_u(const MxView& w, int r) {
  const int64_t a = int64_t{2} * r * w.K;
  return r <= 16 && a <= (int64_t{128} << 10) && w.N / 16 * a <= (int64_t{32} << 20);
}

hipError_t launch_mx_token(const MxView& w, const uint16_t* x, const uint16_t* A, const float* part,
                           int slices, const uint16_t* B, int r, float lora_scale, uint16_t* y,
                           uint16_t* u_out, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>(w.N / 16));
  const bool vec_a = (reinterpret_cast<uintptr_t>(A) & 15) == 0;
  const bool vec_b = (r & 7) == 0 && (reinterpret_cast<uintptr_t>(B) & 15) == 0;
  auto go = [&](auto k, int waves) {
    hipLaunchKernelGGL(k, grid, dim3(64 * waves), 0, st, w.codes,
                       reinterpret_cast<const uint32_t*>(w.scale), w.N, w.K, x, A, vec_a, part,
                       slices, B, r, vec_b, lora_scale, y, u_out);
    return hipGetLastError();
  };
  return r == 0 ? go(mx_token_kernel<kNoAdapter, 8>, 8)
         : !part ? go(mx_token_kernel<kOwnU, 8>, 8)
                 : go(mx_token_kernel<kGivenU, 8>, 8);
}

hipError_t launch_mx_decode(const MxView& w, const uint8_t* x, const uint8_t* xs, int M,
                            const float* part, int slices, const uint16_t* act, const uint16_t* B,
                            int r, float lora_scale, uint16_t* y, uint16_t* u_out, hipStream_t st) {
  if (M == 0) return hipSuccess;
  const bool vec_b = (r & 7) == 0 && (reinterpret_cast<uintptr_t>(B) & 15) == 0;
  auto go = [&](auto k, int waves, int rows) {
    const dim3 grid(static_cast<uint32_t>((w.N + 16 * rows - 1) / (16 * rows)));
    hipLaunchKernelGGL(k, grid, dim3(64 * waves), 0, st, w.codes,
                       reinterpret_cast<const uint32_t*>(w.scale), w.N, w.K, x,
                       reinterpret_cast<const uint32_t*>(xs), M, part, slices, act,
                       fp8_lora_pitch(r), B, r, vec_b, lora_scale, y, u_out);
    return hipGetLastError();
  };
  // Two rows of columns a workgroup halve the reads of x, where half the workgroups
  // still keep the chip busy; 16 tokens, one row and two, 8 waves: 4096 x 4096 10.5 and
  // 11.2 us, 6144 x 4096 12.7 and 11.5, 8192 x 8192 17.6 and 16.1, 32 tokens 26.6 and 22.1.
  // Where these are more than the CUs, 4 waves each let more of them reside than 8:
  // 8 waves and 4, 11008 x 4096 16.8 and 14.7 us, 22016 x 8192 34.7 and 30.8, 28672 x 1024
  // 18.5 and 13.9, 32 tokens on 11008 x 4096 19.8 and 18.9; but 8192 x 8192 16.1 and 18.2.
  const int64_t pairs = (w.N + 31) / 32;
  if (M <= 16)
    return pairs > 256   ? go(mx_decode_kernel<4, 1, 2>, 4, 2)
           : pairs > 128 ? go(mx_decode_kernel<8, 1, 2>, 8, 2)
                         : go(mx_decode_kernel<8, 1, 1>, 8, 1);
  if (M <= 32)
    return pairs > 256   ? go(mx_decode_kernel<4, 2, 2>, 4, 2)
           : pairs > 128 ? go(mx_decode_kernel<8, 2, 2>, 8, 2)
                         : go(mx_decode_kernel<8, 2, 1>, 8, 1);
  return go(mx_decode_kernel<8, 4, 1>, 8, 1);
}

}  // namespace qn
