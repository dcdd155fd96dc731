// Microscaled products for token batches (gfx950).
//
// Forward  y[M, N]  = xq wq^T + (s u) B^T     E2M1 codes, contraction K
// Backward dx[M, K] = tq wt^T + (s t) A       tq E4M3, wt E5M2 codes of the
//                                             turned weight, contraction N
//
// Each 32 values of a row of either operand share a power of two, which the
// matrix instruction multiplies in: the accumulators are the sums themselves,
// and a step is LDS reads and MFMAs alone.  The LoRA term comes first on the
// same accumulators.
//
// Tiles.  A wave holds kWTM x 64 outputs; the MFMAs take the weight as first
// operand, so a lane's four results are four columns of one token.  A step
// takes 128 bytes of a row of both operands, 256 E2M1 or 128 8-bit values, and
// the scales of these, brought in by direct-to-LDS DMA one or two steps ahead in
// two or three buffers; a lane's fragments are the 16-byte chunks lane / 16 and 4
// + lane / 16 of its row, the two MFMAs of a 4-bit step or the two halves of an
// 8-bit one.  The chunks of a row are XOR-swizzled by the choice of each lane's
// source address.  A last step that the rows fill only in part reads its last
// chunk again: the scales there are 2^-127 on both sides.
//
// Launches: forward 2048 x 11008 x 4096 59-64 us (2.9-3.1 PFLOP/s), 4096 x 22016 x
// 8192 372-400 us (3.7-4.0; the vendor's 4-bit product of 8192^3 3.1), 2048 x 4096 x
// 11008 56 us (3.3); backward 2048 x 11008 x 4096 83-89 us (2.0-2.2; the vendor's
// 8-bit product of 8192^3 2.7), 4096 x 22016 x 8192 577 us (2.56); the matrix unit's
// own rates are 10 and 5 PFLOP/s at 2.4 GHz, 16 clocks a 4-bit instruction, 32 an
// 8-bit one, and it is busy for a third to half of the time.  A large tile's step is
// 1540 clocks of LDS reads (192 KB a CU at 128 bytes a clock), the DMA of 64 KB and 2050
// clocks of MFMAs on either path, one after the other in large part: its LDS holds
// one workgroup of two waves a SIMD.  A half tile reads LDS a third more often per
// product.  The first MXFP4 step read the chunks of a row behind a uniform branch: it
// spilled, 1513 us.
//
// Sums.  Forward, a group's 32 products are summed exactly, and outputs are those of
// fp32 sums.  Backward, the 8-bit instruction aligns the products of 8 consecutive
// values to the largest of them and cuts what lies below 2^-13 of it: nothing where
// dy's codes have one exponent and the weight's scales spread up to 2^6; on weights
// and gradients as in use the outputs differ from those of fp32 sums by 2.3e-4 to
// 3.3e-4, where rounding to bf16 alone costs 1.7e-3, and the distance to 64 bits is
// 1.6623e-3 instead of 1.6621e-3, without a bias.  bf16 products, which cut nothing,
// run at half the 8-bit rate on twice the bytes.

#include "qn_launch.h"
#include "qn_mx.h"
#include "qn_tile.h"

namespace qn {

namespace {

struct MxArgs {
  const uint8_t* w;     // codes, rows of `bytes` bytes: N of them forward, K backward
  const uint8_t* ws;    // their tiles of scales
  const uint8_t* x;     // codes of the M tokens, rows of `bytes` bytes
  const uint8_t* xs;
  int64_t M, N, K, bytes;
  const uint16_t* act;  // s u or s t in two parts, [M] rows of `pitch` values
  const uint16_t* lw;   // B [N, r] or A [r, K]
  int r, pitch;
  bool vec_w;           // lw can be read 16 bytes at a time
  uint16_t* out;
  float* part;          // [splits][M][ncols] fp32 instead of out, or nullptr
};

template <bool kBwd, int kWTM_, int kGM_, int kGN_, int kBuf_>
struct Tile {
  static constexpr int kWTM = kWTM_, kGM = kGM_, kGN = kGN_;
  static constexpr int kBuf = kBuf_;                      // steps held in LDS
  static constexpr int kBM = kWTM * kGM, kBN = 64 * kGN;
  static constexpr int kWaves = kGM * kGN, kThreads = 64 * kWaves;
  static constexpr int kA = kBM * 128, kB = kBN * 128;    // bytes of an operand tile
  static constexpr int kRows = kBwd ? 64 : 32;            // rows of a tile of scales
  static constexpr int kSA = kBM / kRows, kSB = kBN / kRows;  // tiles of scales
  static constexpr int kScales = kA + kB;                 // offset of the tokens' scales
  static constexpr int kWScales = kScales + kSA * 256;    // and of the weight's
  static constexpr int kStage = kWScales + kSB * 256;
  static constexpr int kDmaA = kA / 1024 / kWaves, kDmaB = kB / 1024 / kWaves;
  static constexpr int kDmaS = (kSA + kSB + kWaves - 1) / kWaves;
  static constexpr int kDma = kDmaA + kDmaB + kDmaS;      // of a wave and step
  static constexpr int kTI = kWTM / 16, kTJ = 4;          // MFMA tiles of a wave
  static constexpr int kXS = kWTM > kRows ? kWTM / kRows : 1, kWS = 64 / kRows;
  static constexpr int kShare = 5;                        // DMAs issued at a time
  static_assert(kDmaA * 1024 * kWaves == kA && kDmaB * 1024 * kWaves == kB, "tile split");
};

// A lane reads chunk lane / 16 of 16 rows: half of the rows that are served at
// once at chunk c, half at c ^ 1, and this swizzle gives them 16 different
// groups of 4 banks.
__device__ __forceinline__ int mx_swz(int row) { return (row >> 1) & 7; }

// 32 bytes of a lane: chunks lg and 4 + lg of its row.
struct Chunks {
  uint4 lo, hi;
};

__device__ __forceinline__ Chunks read_chunks(const uint8_t* rows, int li, int lg) {
  const int slot = lg ^ mx_swz(li);
  const uint8_t* p = rows + li * 128;
  return {*reinterpret_cast<const uint4*>(p + slot * 16),
          *reinterpret_cast<const uint4*>(p + (slot ^ 4) * 16)};
}

// acc += W rows 16 j .. + 15 times tokens 16 i .. + 15 of the wave's tile, one
// step of the contraction.
template <bool kBwd>
__device__ __forceinline__ f32x4_t step_product(const Chunks& b, const Chunks& a, f32x4_t acc,
                                                int j, int ws, int i, int xs) {
  if constexpr (kBwd) {
    return mfma_mx<kE5M2, kE4M3>(frag8(b.lo, b.hi), frag8(a.lo, a.hi), acc, j & 3, ws, i & 3, xs);
  } else {
    acc = mfma_mx<kE2M1, kE2M1>(frag4(b.lo), frag4(a.lo), acc, 2 * (j & 1), ws, 2 * (i & 1), xs);
    return mfma_mx<kE2M1, kE2M1>(frag4(b.hi), frag4(a.hi), acc, 2 * (j & 1) + 1, ws,
                                 2 * (i & 1) + 1, xs);
  }
}

// Fragments of a step that are read ahead of it: the weight's, the first
// tokens' and all scales.
template <typename T>
struct Ahead {
  Chunks a[2], b[T::kTJ];
  int xs[T::kXS], ws[T::kWS];
};

template <typename T>
__device__ __forceinline__ void read_scales(const uint8_t* st, int wm, int wn, Ahead<T>& f) {
  const int lane = threadIdx.x & 63;
  const int* sx = reinterpret_cast<const int*>(st + T::kScales) + lane;
  const int* sw = reinterpret_cast<const int*>(st + T::kWScales) + lane;
  if constexpr (T::kWTM >= T::kRows) {
#pragma unroll
    for (int q = 0; q < T::kXS; ++q) f.xs[q] = sx[(wm * T::kXS + q) * 64];
  } else {
    // the wave's 32 tokens are half of a tile of 64
    f.xs[0] = sx[(wm >> 1) * 64] >> (16 * (wm & 1));
  }
#pragma unroll
  for (int q = 0; q < T::kWS; ++q) f.ws[q] = sw[(wn * T::kWS + q) * 64];
}

// One output tile: rows from m0, columns from c0, nb steps of the contraction
// from step b0 of `steps`; the LoRA term is added where first is set.
template <typename T, bool kBwd>
__device__ __forceinline__ void mx_tile(const MxArgs& g, uint8_t* smem, int64_t m0, int64_t c0,
                                        int b0, int nb, bool first, int split) {
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / T::kGN, wn = wave % T::kGN;
  const int li = lane & 15, lg = lane >> 4;
  const int64_t ncols = kBwd ? g.K : g.N;
  const int chunks = static_cast<int>(g.bytes / 16);  // of a row
  // byte offsets of this lane's DMA sources; rows past the edge re-read the last
  // valid ones (they only feed outputs that are not stored)
  uint32_t offA[T::kDmaA], offB[T::kDmaB];
#pragma unroll
  for (int j = 0; j < T::kDmaA; ++j) {
    const int row = 8 * (wave * T::kDmaA + j) + (lane >> 3);
    const int64_t m = m0 + row < g.M ? row : g.M - 1 - m0;
    offA[j] = static_cast<uint32_t>(m * g.bytes + ((lane & 7) ^ mx_swz(row)) * 16);
  }
#pragma unroll
  for (int j = 0; j < T::kDmaB; ++j) {
    const int row = 8 * (wave * T::kDmaB + j) + (lane >> 3);
    const int64_t n = c0 + row < ncols ? row : ncols - 1 - c0;
    offB[j] = static_cast<uint32_t>(n * g.bytes + ((lane & 7) ^ mx_swz(row)) * 16);
  }
  // the chunks that this lane fetches, of DMAs with an even and an odd number
  static_assert(T::kDmaA % 2 == 0 && T::kDmaB % 2 == 0, "DMA numbers keep their parity");
  const int chunk[2] = {(lane & 7) ^ mx_swz(lane >> 3), (lane & 7) ^ mx_swz(8 + (lane >> 3))};
  const int64_t xt = mx_tiles(g.M, T::kRows), wt = mx_tiles(ncols, T::kRows);
  const uint8_t* baseA = g.x + m0 * g.bytes;
  const uint8_t* baseB = g.w + c0 * g.bytes;
  const uint32_t lds0 = lds_addr(smem);
  // DMAs q kShare .. of step b (of all), into buffer buf
  auto issue = [&](int b, int buf, int q) {
    const uint32_t st = lds0 + buf * T::kStage;
    const uint8_t* pa = baseA + static_cast<int64_t>(b) * 128;
    const uint8_t* pb = baseB + static_cast<int64_t>(b) * 128;
    // forward, a lane whose chunk lies behind the last one of its row reads that
    // (backward, rows are padded to whole steps); without a branch, which would
    // cut the step into pieces
    const int left = chunks - 8 * b < 8 ? chunks - 8 * b : 8;
    uint32_t back[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      back[h] = kBwd || chunk[h] < left ? 0u : static_cast<uint32_t>(chunk[h] - left + 1) * 16;
#pragma unroll
    for (int d = q * T::kShare; d < (q + 1) * T::kShare && d < T::kDma; ++d) {
      if (d < T::kDmaA + T::kDmaB) {
        const bool tok = d < T::kDmaA;
        const int e = tok ? d : d - T::kDmaA;
        dma16((tok ? offA[e] : offB[e]) - back[e & 1], tok ? pa : pb,
              st + (tok ? 0 : T::kA) + (wave * (tok ? T::kDmaA : T::kDmaB) + e) * 1024);
      } else {
        // a tile of scales; waves without one of their own fetch one again
        int s = wave + T::kWaves * (d - T::kDmaA - T::kDmaB);
        s = s < T::kSA + T::kSB ? s : s - (T::kSA + T::kSB);
        const bool tok = s < T::kSA;
        const int64_t at = tok ? m0 / T::kRows + s : c0 / T::kRows + s - T::kSA;
        const int64_t n = tok ? xt : wt;
        const uint8_t* p = (tok ? g.xs : g.ws) + (b * n + (at < n ? at : n - 1)) * 256;
        dma4(static_cast<uint32_t>(lane * 4), p, st + T::kScales + s * 256);
      }
    }
  };

  f32x4_t acc[T::kTI][T::kTJ];
#pragma unroll
  for (int i = 0; i < T::kTI; ++i)
#pragma unroll
    for (int j = 0; j < T::kTJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  constexpr int kShares = (T::kDma + T::kShare - 1) / T::kShare;
  const int last = b0 + nb - 1;
  auto upto = [&](int b) { return b < last ? b : last; };
  auto issue_all = [&](int b, int buf) {
#pragma unroll
    for (int q = 0; q < kShares; ++q) issue(upto(b), buf, q);
  };
  // the LoRA term with the first step's DMAs in flight, in the last buffer
  issue_all(b0, 0);
  const int rank = first ? g.r : 0;
  if (rank > 0) {
    uint8_t* stL = smem + (T::kBuf - 1) * T::kStage;
    LoraRows<T> lw;
    for (int lb = 0; lb * 32 < rank; ++lb) {
      if (lb > 0) __syncthreads();
      lora_tokens<T>(g, lb, m0, stL);
      if ((lb & 1) == 0) {
        lora_load<T, kBwd>(g, lb >> 1, c0, lw);
        lora_store<T, kBwd>(stL, lw);
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      lora_add<T, kBwd>(lb, stL, acc);
    }
    __syncthreads();
  }

  // Step b multiplies what lies in buffer b % kBuf.  Its MFMAs of tokens 16 i run
  // while the fragment of tokens 16 (i + 1) is read.  Before the last i comes
  // the turn: this wave's reads of the buffer have returned and the next step
  // has landed, for all waves after the barrier; from there on its first
  // fragments are read under the last MFMAs, and the DMAs of step b + kBuf go
  // out, a share per i.  Steps past the end are the last one again.
  constexpr int kEnd = T::kTI - 1;
  static_assert(kShares <= T::kTI, "the DMAs of a step go out before the next turn");
#pragma unroll
  for (int b = 1; b < T::kBuf - 1; ++b) issue_all(b0 + b, b);
  // all DMAs but those of the kBuf - 2 youngest steps have landed
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((T::kBuf - 2) * T::kDma) : "memory");
  issue(upto(b0 + T::kBuf - 1), T::kBuf - 1, 0);
  Ahead<T> f;
  f.a[0] = read_chunks(smem + wm * T::kWTM * 128, li, lg);
#pragma unroll
  for (int j = 0; j < T::kTJ; ++j)
    f.b[j] = read_chunks(smem + T::kA + (wn * 64 + j * 16) * 128, li, lg);
  read_scales<T>(smem, wm, wn, f);
  int buf = 0;
  for (int b = b0; b <= last; ++b) {
    const int bnext = buf + 1 == T::kBuf ? 0 : buf + 1;
    const int bprev = buf == 0 ? T::kBuf - 1 : buf - 1;
    const uint8_t* cur = smem + buf * T::kStage;
    const uint8_t* nxt = smem + bnext * T::kStage;
#pragma unroll
    for (int i = 0; i < T::kTI; ++i) {
      if (i < kEnd) {
        f.a[(i + 1) & 1] = read_chunks(cur + (wm * T::kWTM + (i + 1) * 16) * 128, li, lg);
      } else {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((T::kBuf - 2) * T::kDma)
                     : "memory");
        f.a[(i + 1) & 1] = read_chunks(nxt + wm * T::kWTM * 128, li, lg);
      }
      const int xs = f.xs[T::kWTM > T::kRows ? i * 16 / T::kRows : 0];
#pragma unroll
      for (int j = 0; j < T::kTJ; ++j) {
        acc[i][j] = step_product<kBwd>(f.b[j], f.a[i & 1], acc[i][j], j,
                                       f.ws[j * 16 / T::kRows], i, xs);
        if (i == kEnd) f.b[j] = read_chunks(nxt + T::kA + (wn * 64 + j * 16) * 128, li, lg);
      }
      if (i == kEnd) {
        read_scales<T>(nxt, wm, wn, f);
        issue(upto(b + T::kBuf), buf, 0);
      } else if (i + 1 < kShares) {
        issue(upto(b + T::kBuf - 1), bprev, i + 1);
      }
      if (i & 1) __builtin_amdgcn_sched_barrier(0);
    }
    static_assert(T::kTI % 2 == 0, "the first fragment of a step is a[0]");
    buf = bnext;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  if (g.part)
    store_part<T>(g.part + static_cast<int64_t>(split) * g.M * ncols, g.M, ncols, m0, c0, acc);
  else
    store_tile<T>(g.out, g.M, ncols, m0, c0, smem, acc);
}

template <bool kBwd>
using Big = Tile<kBwd, 128, 2, 4, 2>;   // 256 x 256, 8 waves
template <bool kBwd>
using Half = Tile<kBwd, 64, 2, 4, 3>;   // 128 x 256, 8 waves
template <bool kBwd>
using Small = Tile<kBwd, 32, 4, 2, 3>;  // 128 x 128, 8 waves

constexpr int kBig = 256, kHalf = 128, kSmall = 128;

// Workgroups below nbig take one 256 x 256 tile each, the others half of one
// of the remaining tiles.
template <bool kBwd>
__global__ __launch_bounds__(512, 2) void mx_gemm_kernel(MxArgs g, int nbig) {
  typedef Big<kBwd> B;
  typedef Half<kBwd> H;
  static_assert(B::kThreads == 512 && H::kThreads == 512 && B::kBN == H::kBN &&
                    B::kBM == kBig && H::kBM == kHalf,
                "a half tile has the same workgroup");
  constexpr int kLds = B::kBuf * B::kStage > H::kBuf * H::kStage ? B::kBuf * B::kStage
                                                                  : H::kBuf * H::kStage;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kLds];
  const int nc = static_cast<int>(((kBwd ? g.K : g.N) + B::kBN - 1) / B::kBN);
  const int nr = static_cast<int>((g.M + B::kBM - 1) / B::kBM);
  const int bid = blockIdx.x;
  const int steps = static_cast<int>((g.bytes + 127) / 128);
  int row, col;
  if (bid < nbig) {
    tile_of(xcd_run(bid, nbig), nc, nr, row, col);
    mx_tile<B, kBwd>(g, smem, static_cast<int64_t>(row) * B::kBM,
                     static_cast<int64_t>(col) * B::kBN, 0, steps, true, 0);
  } else {
    const int two = g.M > H::kBM ? 1 : 0;  // log2 of the halves of a tile
    const int q = xcd_run(bid - nbig, (nc * nr - nbig) << two);
    tile_of(nbig + (q >> two), nc, nr, row, col);
    const int64_t m0 = static_cast<int64_t>(row) * B::kBM + (q & two) * H::kBM;
    if (m0 < g.M)
      mx_tile<H, kBwd>(g, smem, m0, static_cast<int64_t>(col) * H::kBN, 0, steps, true, 0);
  }
}

// Workgroup row z takes the steps z per .. of the contraction.
template <bool kBwd>
__global__ __launch_bounds__(512) void mx_gemm_small_kernel(MxArgs g, int per) {
  typedef Small<kBwd> S;
  static_assert(S::kThreads == 512 && S::kBM == kSmall && S::kBN == kSmall, "tile");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kBuf * S::kStage];
  const int nc = static_cast<int>(((kBwd ? g.K : g.N) + S::kBN - 1) / S::kBN);
  const int nr = static_cast<int>((g.M + S::kBM - 1) / S::kBM);
  const int steps = static_cast<int>((g.bytes + 127) / 128);
  const int b0 = static_cast<int>(blockIdx.y) * per;
  int row, col;
  tile_of(xcd_run(blockIdx.x, nc * nr), nc, nr, row, col);
  mx_tile<S, kBwd>(g, smem, static_cast<int64_t>(row) * S::kBM,
                   static_cast<int64_t>(col) * S::kBN, b0,
                   steps - b0 < per ? steps - b0 : per, blockIdx.y == 0,
                   static_cast<int>(blockIdx.y));
}

int64_t small_tiles(int64_t M, int64_t ncols) {
  return mx_tiles(ncols, kSmall) * mx_tiles(M, kSmall);
}

// Large tiles where the small ones would take more than one round of the CUs.
// Small and large, calls on 4096 x 4096: 1024 tokens (256 small tiles) 26.6 and 32.4
// us, backward 40 and 45; 1152 tokens 37.5 and 32.4; 2048 38.5 and 35.8, backward 55
// and 49; 11008 x 4096, 256 tokens 24 and 32, 512 39 and 33.
bool large(int64_t M, int64_t ncols) { return small_tiles(M, ncols) > 256; }

}  // namespace

int mx_gemm_splits(int64_t M, int64_t ncols, int64_t bytes, bool bwd) {
  if (M <= 0 || large(M, ncols)) return 1;
  // Up to one workgroup per CU.  A step costs 0.45 us forward and 0.55 us backward,
  // the launch that adds the parts 3.5, a part 4 bytes an output at 5.5 TB/s out and
  // back, half of it hidden: fitted to calls such as 4096 x 11008, 128 tokens in 1, 2, 4
  // and 8 parts (44.5, 36, 30, 29 us), 4096 x 4096, 256 tokens in 1, 2, 4 (21.9, 25.6,
  // 28.9) and backward (38, 34, 29).
  const int64_t steps = mx_tiles(bytes, 128), most = 256 / small_tiles(M, ncols);
  const double out = static_cast<double>(M) * static_cast<double>(ncols) * 4 / 5.5e6;
  const double step = bwd ? 0.55 : 0.45;
  double best = step * static_cast<double>(steps);
  int splits = 1;
  for (int64_t s = 2; s <= most && s <= steps; ++s) {
    const int64_t per = (steps + s - 1) / s, n = (steps + per - 1) / per;
    const double t = step * static_cast<double>(per) + 3.5 + (out + 0.1) * static_cast<double>(n);
    if (t < best) best = t, splits = static_cast<int>(n);
  }
  return splits;
}

hipError_t launch_mx_gemm(const uint8_t* w, const uint8_t* ws, int64_t N, int64_t K, int64_t bytes,
                          const uint8_t* x, const uint8_t* xs, int64_t M, const uint16_t* act,
                          const uint16_t* lw, int r, bool bwd, uint16_t* out, float* part,
                          hipStream_t st) {
  if (M == 0) return hipSuccess;
  // rows of B have r values, those of A K, a multiple of 32
  const bool vec_w = (reinterpret_cast<uintptr_t>(lw) & 15) == 0 && (bwd || (r & 7) == 0);
  const int64_t ncols = bwd ? K : N;
  MxArgs g{w, ws, x, xs, M, N, K, bytes, act, lw, r, fp8_lora_pitch(r), vec_w, out, nullptr};
  if (large(M, ncols)) {
    // whole rounds of the 256 CUs in large tiles, a remainder of up to half
    // a round in halves
    const int64_t tiles = mx_tiles(ncols, kBig) * mx_tiles(M, kBig);
    const int64_t rest = tiles % 256, halves = M > kHalf ? 2 : 1;
    const int64_t nbig = halves == 1 ? 0 : rest <= 128 ? tiles - rest : tiles;
    const dim3 grid(static_cast<uint32_t>(nbig + halves * (tiles - nbig)));
    if (bwd)
      hipLaunchKernelGGL(mx_gemm_kernel<true>, grid, dim3(512), 0, st, g, static_cast<int>(nbig));
    else
      hipLaunchKernelGGL(mx_gemm_kernel<false>, grid, dim3(512), 0, st, g, static_cast<int>(nbig));
    return hipGetLastError();
  }
  const int splits = part ? mx_gemm_splits(M, ncols, bytes, bwd) : 1;
  const int per = static_cast<int>((mx_tiles(bytes, 128) + splits - 1) / splits);
  if (splits > 1) g.part = part;
  const dim3 grid(static_cast<uint32_t>(small_tiles(M, ncols)), static_cast<uint32_t>(splits));
  if (bwd)
    hipLaunchKernelGGL(mx_gemm_small_kernel<true>, grid, dim3(512), 0, st, g, per);
  else
    hipLaunchKernelGGL(mx_gemm_small_kernel<false>, grid, dim3(512), 0, st, g, per);
  const hipError_t e = hipGetLastError();
  return splits > 1 && e == hipSuccess ? launch_fp8_split_sum(part, splits, M * ncols, out, st) : e;
}

}  // namespace qn
