// Block-scaled FP8 products for few tokens, up to 64 (gfx950).
//
//   y[m, n] = sum_b xs[b, m] ws[n / 128, b] (xq_b[m] . wq_b[n]) + (s u) B^T
//
// Bound by reading the weight once (N K bytes), and past one token by x's
// codes, which every workgroup reads from the L2s (16 tokens' are as many bytes
// as the workgroup's weight).  A workgroup owns 16 output columns (or 32, see
// the launch) and the whole contraction: its waves take the blocks of 128 in
// turn, each block one 16x16x128 FP8 MFMA with the weight's rows as the first
// operand and 16 tokens (the last one again past the end) as the second.
// Every lane loads 32 consecutive bytes of its row straight into its
// fragment, some blocks ahead of their products, so the weight needs neither
// LDS nor a second pass.  The waves' fp32 sums meet in LDS and are added in
// wave order, so results are bit-reproducible.  One token: 4096 x 4096 in 5.8
// us (r = 16: 9.4 back to back in a graph, 9.8-10.3 traced alone), 8192 x 8192
// in 14.5 (4.6 TB/s), 22016 x 8192 with r = 16, two launches, in 38 (4.7 TB/s, a
// large copy's rate); 16 tokens of 4096 x 11008: 15 us.
//
// One token: the same launch quantises x, each wave for its own blocks, and,
// where the adapter is small, computes u = x A^T: at 4096 x 4096 the whole
// call is one launch.  More tokens: x's codes and u's partial sums come from
// a launch before.

#include "qn_decode.h"
#include "qn_fp8.h"
#include "qn_launch.h"

namespace qn {

namespace {

// This lane's 32 bytes of block b of a row, zeros behind the row's end.
struct Bytes32 {
  uint4 lo, hi;
};

__device__ __forceinline__ Bytes32 row_bytes(const uint8_t* row, int64_t b, int64_t K, int lg) {
  const int64_t k = b * 128 + 32 * lg;
  Bytes32 v{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (k < K) v.lo = *reinterpret_cast<const uint4*>(row + k);
  if (k + 16 < K) v.hi = *reinterpret_cast<const uint4*>(row + k + 16);
  return v;
}

template <int kU, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void fp8_token_kernel(
    const uint8_t* __restrict__ w, const float* __restrict__ ws, int64_t N, int64_t K,
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ A, bool vec_a,
    const float* __restrict__ part, int slices, const uint16_t* __restrict__ B, int r, bool vec_b,
    float lora_scale, uint16_t* __restrict__ y, uint16_t* __restrict__ u_out) {
  constexpr int kThreads = 64 * kWaves, kAhead = 2;
  constexpr int kFrags = kU == kGivenU ? kDecodeMaxRank / 32 : 1;
  __shared__ f32x4_t s_acc[kWaves][4];
  __shared__ float s_u[kU == kNoAdapter ? 1 : kThreads];  // kOwnU: [wave][16 ranks]
  __shared__ __attribute__((aligned(16))) uint16_t s_us[64 * kFrags];
  __shared__ __attribute__((aligned(16))) uint32_t s_x[kWaves][kAhead][64];   // bf16 pairs
  __shared__ __attribute__((aligned(16))) uint16_t s_q[kWaves][kAhead][64];   // code pairs
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int li = lane & 15, lg = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;  // N is a multiple of 16
  const int64_t kb = (K + 127) / 128;
  const uint8_t* wr = w + (n0 + li) * K;
  const float* wsr = ws + (n0 / 128) * kb;

  uint4 bf[kFrags];
  if (kU != kNoAdapter && wave == 0) load_up<kFrags>(bf, B, n0, r, li, lg, vec_b);
  if constexpr (kU == kGivenU) s_u[t] = add_slices<kThreads>(part, slices, r, t);
  f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f}, ua = acc;
  for (int64_t bw = wave; bw < kb; bw += kAhead * kWaves) {
    // everything that these blocks need is asked for first
    Bytes32 wv[kAhead];
    uint32_t xp[kAhead];
    float sw[kAhead];
    uint4 av[kAhead][4];
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      const int64_t b = bw + d * kWaves;
      const bool in = b < kb;
      const int64_t k = b * 128 + 2 * lane;
      xp[d] = in && k < K ? *reinterpret_cast<const uint32_t*>(x + k) : 0u;
      wv[d] = row_bytes(wr, in ? b : kb, K, lg);
      sw[d] = in ? wsr[b] : 0.0f;
      if constexpr (kU == kOwnU) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int64_t ka = b * 128 + 32 * c + 8 * lg;
          av[d][c] = load_bf16x8(A + li * K + ka, li < r && in && ka < K ? 8 : 0, vec_a);
        }
      }
    }
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      const float x0 = bf16_lo(xp[d]), x1 = bf16_hi(xp[d]);
      const float s =
          fp8_scale(lanes_max<1, 32>(absmax_bits(absmax_pair(u16x2_t{0, 0}, xp[d]))));
      const float inv = __fdiv_rn(1.0f, s);
      if constexpr (kU == kOwnU) s_x[wave][d][lane] = xp[d];
      s_q[wave][d][lane] = static_cast<uint16_t>(__builtin_amdgcn_cvt_pk_fp8_f32(
          fp8_ratio(x0, s, inv), fp8_ratio(x1, s, inv), 0, false));
      sw[d] *= s;
    }
    // written and read by the same wave: its own LDS order suffices
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      const uint4* q = reinterpret_cast<const uint4*>(&s_q[wave][d][16 * lg]);
      const f32x4_t c =
          mfma_fp8(frag8(wv[d].lo, wv[d].hi), frag8(q[0], q[1]), f32x4_t{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = fmaf(c[e], sw[d], acc[e]);
      if constexpr (kU == kOwnU) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          ua = mfma_bf16_32(
              av[d][k], *reinterpret_cast<const uint4*>(&s_x[wave][d][16 * k + 4 * lg]), ua);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next blocks' values
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
    const int sums = kU == kOwnU          ? kWaves
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
__global__ __launch_bounds__(64 * kWaves) void fp8_decode_kernel(
    const uint8_t* __restrict__ w, const float* __restrict__ ws, int64_t N, int64_t K,
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int M,
    const float* __restrict__ part, int slices, const uint16_t* __restrict__ act, int pitch,
    const uint16_t* __restrict__ B, int r, bool vec_b, float lora_scale, uint16_t* __restrict__ y,
    uint16_t* __restrict__ u_out) {
  constexpr int kThreads = 64 * kWaves;
  constexpr int kAhead = kMT <= 2 ? 2 : 1;  // blocks in flight besides the one multiplied
  constexpr int kTiles = kMT * kRows;
  static_assert(kTiles <= kWaves, "a wave finishes 16 columns of 16 tokens");
  __shared__ f32x4_t s_acc[kWaves][kTiles][64];
  __shared__ float s_u[kMT == 1 ? kFp8DecodeM * kDecodeMaxRank : 1];
  __shared__ __attribute__((aligned(16))) uint16_t s_us[kMT == 1 ? 32 * kDecodeMaxRank : 8];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int li = lane & 15, lg = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * kRows);
  const int64_t kb = (K + 127) / 128;
  // N is a multiple of 16: the last workgroup may have fewer rows of 16, and
  // reads its last ones again
  const uint8_t* wr[kRows];
#pragma unroll
  for (int q = 0; q < kRows; ++q)
    wr[q] = w + ((n0 + 16 * q < N ? n0 + 16 * q : N - 16) + li) * K;
  const float* wsr = ws + (n0 / 128) * kb;
  int m[kMT];
#pragma unroll
  for (int i = 0; i < kMT; ++i) m[i] = 16 * i + li < M ? 16 * i + li : M - 1;

  struct Block {
    Bytes32 w[kRows], x[kMT];
    float sw, sx[kMT];
  };
  auto load = [&](int64_t b, Block& d) {
    const bool in = b < kb;
#pragma unroll
    for (int q = 0; q < kRows; ++q) d.w[q] = row_bytes(wr[q], in ? b : kb, K, lg);
    d.sw = in ? wsr[b] : 0.0f;
#pragma unroll
    for (int i = 0; i < kMT; ++i) {
      d.x[i] = row_bytes(x + m[i] * K, in ? b : kb, K, lg);
      d.sx[i] = in ? xs[b * M + m[i]] : 0.0f;
    }
  };
  // u = sum of its slices: `par` threads per value, thread (q0, e) takes the
  // slices q0, q0 + par, ...; the first kEarly of them are asked for before
  // anything else and added while the weight is on its way, the sums over q0
  // (in order) follow behind the product.  par is that of 16 tokens for any M:
  // it decides the order of the sum, and so a token's result does not depend on
  // its batch (as many threads as M r leaves are no faster: r = 16, 2 x 4096 x
  // 11008 17.2 us either way, 5 x 4096 x 4096 10.8 against 10.2).
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
  Block blk[kAhead + 1];
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
  for (int64_t b = wave; b < kb; b += (kAhead + 1) * kWaves) {
#pragma unroll
    for (int d = 0; d <= kAhead; ++d) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const Bytes32 &wv = blk[d].w[i / kMT], &xv = blk[d].x[i % kMT];
        const f32x4_t c =
            mfma_fp8(frag8(wv.lo, wv.hi), frag8(xv.lo, xv.hi), f32x4_t{0.f, 0.f, 0.f, 0.f});
        const float s = blk[d].sx[i % kMT] * blk[d].sw;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(c[e], s, acc[i][e]);
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

bool fp8_few(int64_t M, int64_t N, int64_t K) {
  // x's codes go to every workgroup: 16 tokens' as many bytes from the L2s as
  // the weight has.  From 64 MiB of them over a full round of CUs (4096
  // columns) on, the tiles, which share x among 128 columns, cost less (r =
  // 16: 32 x 4096 x 4096, 32 MiB, 16.2 us against 18.3; 64 x 4096 x 4096, 64
  // MiB, 20.1 and 20.2; 64 x 1008 x 8192, 31 against 21; 64 x 4096 x 11008, 42
  // against 31; 64 x 22016 x 8192, 127 against 53).  Up to 16 tokens this kernel
  // always, which is the faster one for short contractions and about even for
  // long ones, but for few columns (products of given rows, here and as tiles,
  // in us: 16 x 272 x 1040 3.6 and 7.4; 16 x 4096 x 4096 7.5 and 10.0; 16 x 1008
  // x 8192 10.5 and 10.9; 16 x 4096 x 11008 14.0 and 14.2; 16 x 11008 x 4096 15.8
  // and 14.5; 16 x 22016 x 8192 52.9 and 50.8; 16 x 144 x 22016, 9 workgroups
  // here and 2 tiles in parts there, 21.7 and 14.6).
  const int64_t cols = N > 4096 ? N : 4096;
  return M <= kFp8DecodeM ||
         (M <= kFp8FewM && (M + 15) / 16 * cols * K < (int64_t{64} << 20));
}

bool fp8_token_self_u(const Fp8View& w, int r) {
  // A is read by every workgroup, from the caches: past 32 MiB in all, or 128
  // KB each, a projection launch of its own costs less (one token on the
  // device, own and given u: 4096 x 4096, r = 16, 32 MiB, 9.4 us against 9.0 and
  // a launch more for the host; 8192 x 1024, r = 16, 6.4 and 7.7; 8192 x 2048,
  // r = 16, 32 MiB, 9.0 and 8.7; past it 4112 x 4096, which is a second round
  // of the CUs too, 13.9 and 10.2; 11008 x 2048, r = 8, 10.6 and 9.6; 1008 x
  // 8192, r = 16, 256 KB each, 13.8 and 9.7)
  const int64_t a = int64_t{2} * r * w.K;
  return r <= 16 && a <= (int64_t{128} << 10) && w.N / 16 * a <= (int64_t{32} << 20);
}

hipError_t launch_fp8_token(const Fp8View& w, const uint16_t* x, const uint16_t* A,
                            const float* part, int slices, const uint16_t* B, int r,
                            float lora_scale, uint16_t* y, uint16_t* u_out, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>(w.N / 16));
  const bool vec_a = (reinterpret_cast<uintptr_t>(A) & 15) == 0;
  const bool vec_b = (r & 7) == 0 && (reinterpret_cast<uintptr_t>(B) & 15) == 0;
  auto go = [&](auto k, int waves) {
    hipLaunchKernelGGL(k, grid, dim3(64 * waves), 0, st, w.codes, w.scale, w.N, w.K, x, A, vec_a, part,
                       slices, B, r, vec_b, lora_scale, y, u_out);
    return hipGetLastError();
  };
  // Without an adapter, which takes the fewest registers, 16 waves; u given: 16
  // where one workgroup per CU has the whole weight, else 8, of which more fit on
  // a CU at once; u of its own: 8, up to one workgroup per CU as fast as 16 and
  // beyond faster (one token, 8 and 16 waves: r = 0 4096 x 4096 6.6 and 5.8 us;
  // given, r = 64, 4096 x 4096 11.0 and 10.4; own, r = 16, 4096 x 4096 9.4 and
  // 9.4, 2048 x 2048 5.5 and 5.8, 5008 x 2000 7.4 and 9.5)
  return r == 0 ? go(fp8_token_kernel<kNoAdapter, 16>, 16)
         : !part        ? go(fp8_token_kernel<kOwnU, 8>, 8)
         : grid.x > 256 ? go(fp8_token_kernel<kGivenU, 8>, 8)
                        : go(fp8_token_kernel<kGivenU, 16>, 16);
}

hipError_t launch_fp8_decode(const Fp8View& w, const uint8_t* x, const float* xs, int M,
                             const float* part, int slices, const uint16_t* act,
                             const uint16_t* B, int r, float lora_scale, uint16_t* y,
                             uint16_t* u_out, hipStream_t st) {
  if (M == 0) return hipSuccess;
  const bool vec_b = (r & 7) == 0 && (reinterpret_cast<uintptr_t>(B) & 15) == 0;
  const int64_t kb = (w.K + 127) / 128;
  auto go = [&](auto k, int waves, int rows) {
    const dim3 grid(static_cast<uint32_t>((w.N + 16 * rows - 1) / (16 * rows)));
    hipLaunchKernelGGL(k, grid, dim3(64 * waves), 0, st, w.codes, w.scale, w.N, w.K, x, xs, M, part,
                       slices, act, fp8_lora_pitch(r), B, r, vec_b, lora_scale, y, u_out);
    return hipGetLastError();
  };
  // 8 waves: 16 leave room for one workgroup per CU only (5 tokens, 5008 x
  // 2000: 9.9 us against 13.8; 16 tokens, 4096 x 11008: the same)
  // Two row tiles share x's codes, but only one such workgroup fits on a CU:
  // where they are one round of the CUs and more than half of one (r = 16:
  // 16 x 8192 x 8192 27.1 -> 23.9 us, 20 x 5008 x 2000 14.5 -> 12.0; outside,
  // 16 x 4096 x 11008 19.7 -> 24.4, 16 x 11008 x 4096 21.3 -> 22.7).
  const int64_t pairs = (w.N + 31) / 32;
  const bool two = pairs > 128 && pairs <= 256 && kb > 8;
  if (M <= 16)
    return two       ? go(fp8_decode_kernel<8, 1, 2>, 8, 2)
           : kb <= 8 ? go(fp8_decode_kernel<4, 1, 1>, 4, 1)
                     : go(fp8_decode_kernel<8, 1, 1>, 8, 1);
  if (M <= 32)
    return two       ? go(fp8_decode_kernel<8, 2, 2>, 8, 2)
           : kb <= 8 ? go(fp8_decode_kernel<4, 2, 1>, 4, 1)
                     : go(fp8_decode_kernel<8, 2, 1>, 8, 1);
  return kb <= 8 ? go(fp8_decode_kernel<4, 4, 1>, 4, 1) : go(fp8_decode_kernel<8, 4, 1>, 8, 1);
}

}  // namespace qn
