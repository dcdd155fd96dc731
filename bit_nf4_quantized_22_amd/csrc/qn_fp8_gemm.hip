// Block-scaled FP8 products for token batches (gfx950).
//
// Forward  y[M, N]  = sum_b xs[m, b] ws[n / 128, b] (xq_b wq_b^T) + (s u) B^T
// Backward dx[M, K] = sum_b ts[m, b] ws[b, k / 128] (tq_b wq_b)   + (s t) A
//
// b runs over the blocks of 128 of the contraction (K forward, N backward);
// xq, tq and wq are E4M3 codes.  Within a block the product is one
// 16x16x128 FP8 MFMA per 16 x 16 outputs; its fp32 result is multiplied by
// the block's two scales and added to the fp32 accumulator with one fused
// multiply-add per output, so no scale is ever rounded to fewer bits.  The
// LoRA term follows on the same accumulators as bf16 MFMAs.
//
// Tiles.  A wave holds kWTM x 64 outputs, which lie in one 128-block of the
// weight, so the weight's scale is wave-uniform; the MFMAs take the weight as
// first operand, so a lane's four results are four columns of one token and
// the token's scale is one register.  Both operand tiles (128 bytes of the
// contraction per step) are brought in by direct-to-LDS DMA, one step ahead
// in the other of two buffers; 16-byte chunks of a row are XOR-swizzled by
// the choice of each lane's source address, so that the fragment reads hit
// all banks.  The backward's weight tile lies [n][k] in memory while a lane
// needs 32 n of one k: it is read through the transposing LDS loads (8 rows
// x 16 columns of bytes per 16 lanes).

#include "qn_fp8.h"
#include "qn_launch.h"

namespace qn {

namespace {

typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2_t lds_i32x2_t;
typedef __attribute__((address_space(3))) uint8_t lds_u8_t;

struct Fp8Args {
  const uint8_t* w;    // codes [N, K]
  const float* ws;     // scales [ceil(N / 128), ceil(K / 128)]
  const uint8_t* x;    // codes [M, L], L the contraction length
  const float* xs;     // scales [ceil(L / 128), M]
  int64_t M, N, K;
  const uint16_t* lact;  // bf16(s u) or bf16(s t), [M, r]
  const uint16_t* lw;    // B [N, r] or A [r, K]
  int r;
  bool vec_w;            // rows of lw can be read 16 bytes at a time (forward)
  uint16_t* out;
};

template <int kWTM_, int kGM_, int kGN_>
struct Tile {
  static constexpr int kWTM = kWTM_, kGM = kGM_, kGN = kGN_;
  static constexpr int kBM = kWTM * kGM, kBN = 64 * kGN;
  static constexpr int kWaves = kGM * kGN, kThreads = 64 * kWaves;
  static constexpr int kA = kBM * 128, kB = kBN * 128;    // bytes of an operand tile
  static constexpr int kStage = kA + kB + kBM * 4;        // + the tokens' scales
  static constexpr int kDmaA = kA / 1024 / kWaves, kDmaB = kB / 1024 / kWaves;
  static constexpr int kDmaS = kBM / 64;                  // waves that fetch 64 scales each
  static constexpr int kTI = kWTM / 16, kTJ = 4;          // MFMA tiles of a wave
  static_assert(kDmaA * 1024 * kWaves == kA && kDmaB * 1024 * kWaves == kB && kDmaS <= kWaves,
                "tile split");
};

// Slot of 16-byte chunk c in a 128-byte row: 16 consecutive rows' reads of
// one chunk fall into 16 different groups of 4 banks.
__device__ __forceinline__ int row_swz(int row) { return (row >> 1) & 7; }

// The same for the backward's weight tile of kBN bytes a row, whose reads
// take rows 8 q + 32 g .. + 7 of two g at a time.
template <int kBN>
__device__ __forceinline__ int col_swz(int row) {
  if constexpr (kBN == 256) return (row & 7) | ((row >> 5) & 1) << 3;
  return ((row >> 1) & 3) | ((row >> 5) & 1) << 2;
}

// LDS DMAs as inline assembly: the compiler waits for every DMA it knows of
// at each LDS read.  Nothing is returned to registers; the waits below cover
// them.  Lane l writes 16 (or 4) bytes at lds + 16 l (4 l).
__device__ __forceinline__ void dma16(uint32_t off, const void* base, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
}

__device__ __forceinline__ void dma4(uint32_t off, const void* base, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const uint8_t*)p));
}

// Output tile of workgroup bid: the workgroups of one XCD (bid % 8) take a
// contiguous run of the tile order, bands of kBandRows row tiles, column by
// column within a band, so that the tiles an XCD works on at a time share
// their rows of x and columns of W in its L2.
constexpr int kBandRows = 4;

__device__ __forceinline__ void fp8_tile_of(int bid, int nc, int nr, int& row, int& col) {
  const int total = nc * nr, x = bid & 7;
  const int base = total >> 3, rem = total & 7;
  const int q = x * base + (x < rem ? x : rem) + (bid >> 3);
  const int band = q / (kBandRows * nc);
  const int local = q - band * kBandRows * nc;
  const int rows = nr - band * kBandRows < kBandRows ? nr - band * kBandRows : kBandRows;
  col = local / rows;
  row = band * kBandRows + local % rows;
}

template <typename T, bool kBwd>
__device__ __forceinline__ void mma_step(const uint8_t* st, float sw, int wm, int wn, int li, int g,
                                         f32x4_t (&acc)[T::kTI][T::kTJ]) {
  const uint8_t* sA = st;
  const uint8_t* sB = st + T::kA;
  const float* sS = reinterpret_cast<const float*>(st + T::kA + T::kB);
  const int slot = (2 * g) ^ row_swz(li);
  i32x8_t b[T::kTJ];
#pragma unroll
  for (int j = 0; j < T::kTJ; ++j) {
    if constexpr (kBwd) {
      // lanes 2 r, 2 r + 1 of a group point at row 8 q + 32 g + r, columns
      // 0-7 and 8-15; lane c receives column c of the 8 rows
      const int f = col_swz<T::kBN>((li >> 1) + 32 * g);
      const uint8_t* p =
          sB + (32 * g + (li >> 1)) * T::kBN + (((wn * 4 + j) ^ f) << 4) + (li & 1) * 8;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const i32x2_t v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (lds_i32x2_t*)(lds_u8_t*)(p + q * 8 * T::kBN));
        b[j][2 * q] = v[0];
        b[j][2 * q + 1] = v[1];
      }
    } else {
      const uint8_t* p = sB + (wn * 64 + j * 16 + li) * 128;
      b[j] = frag8(*reinterpret_cast<const uint4*>(p + slot * 16),
                   *reinterpret_cast<const uint4*>(p + (slot ^ 1) * 16));
    }
  }
#pragma unroll
  for (int i = 0; i < T::kTI; ++i) {
    const uint8_t* p = sA + (wm * T::kWTM + i * 16 + li) * 128;
    const i32x8_t a = frag8(*reinterpret_cast<const uint4*>(p + slot * 16),
                            *reinterpret_cast<const uint4*>(p + (slot ^ 1) * 16));
    const float s = sS[wm * T::kWTM + i * 16 + li] * sw;
#pragma unroll
    for (int j = 0; j < T::kTJ; ++j) {
      const f32x4_t c = mfma_fp8(b[j], a, f32x4_t{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(c[e], s, acc[i][j][e]);
    }
  }
}

template <typename T, bool kBwd>
__global__ __launch_bounds__(T::kThreads) void fp8_gemm_kernel(Fp8Args g) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * T::kStage];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / T::kGN, wn = wave % T::kGN;
  const int li = lane & 15, lg = lane >> 4;
  const int64_t ncols = kBwd ? g.K : g.N, L = kBwd ? g.N : g.K;
  int trow, tcol;
  fp8_tile_of(blockIdx.x, static_cast<int>((ncols + T::kBN - 1) / T::kBN),
              static_cast<int>((g.M + T::kBM - 1) / T::kBM), trow, tcol);
  const int64_t m0 = static_cast<int64_t>(trow) * T::kBM;
  const int64_t c0 = static_cast<int64_t>(tcol) * T::kBN;
  const int nfull = static_cast<int>(L / 128), tail = static_cast<int>(L % 128);
  const int64_t kb = (g.K + 127) / 128;
  // the weight's scale of contraction block b, the same for the whole wave;
  // a wave past the last column re-reads the last block's
  int64_t cblk = (c0 + wn * 64) / 128;
  const int64_t cmax = (ncols - 1) / 128;
  cblk = cblk < cmax ? cblk : cmax;
  const float* wsp = kBwd ? g.ws + cblk : g.ws + cblk * kb;
  const int64_t ws_step = kBwd ? kb : 1;

  // byte offsets of this lane's DMA sources; rows and columns past the edge
  // re-read the last valid ones (they only feed outputs that are not stored)
  uint32_t offA[T::kDmaA], offB[T::kDmaB];
#pragma unroll
  for (int j = 0; j < T::kDmaA; ++j) {
    const int row = 8 * (wave * T::kDmaA + j) + (lane >> 3);
    const int64_t m = m0 + row < g.M ? row : g.M - 1 - m0;
    offA[j] = static_cast<uint32_t>(m * L + ((lane & 7) ^ row_swz(row)) * 16);
  }
#pragma unroll
  for (int j = 0; j < T::kDmaB; ++j) {
    if constexpr (kBwd) {
      constexpr int kSlots = T::kBN / 16;
      const int row = (64 / kSlots) * (wave * T::kDmaB + j) + lane / kSlots;
      const int64_t c = ((lane % kSlots) ^ col_swz<T::kBN>(row)) * 16;
      offB[j] = static_cast<uint32_t>(row * g.K + (c0 + c < g.K ? c : g.K - 16 - c0));
    } else {
      const int row = 8 * (wave * T::kDmaB + j) + (lane >> 3);
      const int64_t n = c0 + row < g.N ? row : g.N - 1 - c0;
      offB[j] = static_cast<uint32_t>(n * L + ((lane & 7) ^ row_swz(row)) * 16);
    }
  }
  const int64_t srow = m0 + wave * 64 + lane;
  const uint32_t offS = static_cast<uint32_t>((srow < g.M ? wave * 64 + lane : g.M - 1 - m0) * 4);
  const uint8_t* baseA = g.x + m0 * L;
  const uint8_t* baseB = kBwd ? g.w + c0 : g.w + c0 * L;
  const float* baseS = g.xs + m0;
  const uint32_t lds0 = lds_addr(smem);
  auto issue = [&](int b) {
    const uint32_t st = lds0 + (b & 1) * T::kStage;
    const uint8_t* pa = baseA + static_cast<int64_t>(b) * 128;
    const uint8_t* pb = kBwd ? baseB + static_cast<int64_t>(b) * 128 * g.K
                             : baseB + static_cast<int64_t>(b) * 128;
#pragma unroll
    for (int j = 0; j < T::kDmaA; ++j) dma16(offA[j], pa, st + (wave * T::kDmaA + j) * 1024);
#pragma unroll
    for (int j = 0; j < T::kDmaB; ++j)
      dma16(offB[j], pb, st + T::kA + (wave * T::kDmaB + j) * 1024);
    if (wave < T::kDmaS)
      dma4(offS, baseS + static_cast<int64_t>(b) * g.M, st + T::kA + T::kB + wave * 256);
  };

  f32x4_t acc[T::kTI][T::kTJ];
#pragma unroll
  for (int i = 0; i < T::kTI; ++i)
#pragma unroll
    for (int j = 0; j < T::kTJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  if (nfull > 0) issue(0);
  for (int b = 0; b < nfull; ++b) {
    const float sw = wsp[b * ws_step];
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // block b landed (this wave's part)
    __syncthreads();  // everyone's part, and everyone is done with block b - 1
    if (b + 1 < nfull) issue(b + 1);
    mma_step<T, kBwd>(smem + (b & 1) * T::kStage, sw, wm, wn, li, lg, acc);
  }
  if (tail) {
    // the last, partial block: through registers, zeros behind its end
    uint8_t* st = smem + (nfull & 1) * T::kStage;
    const int64_t l0 = static_cast<int64_t>(nfull) * 128;
    auto row_tile = [&](uint8_t* dst, const uint8_t* src, int64_t row0, int64_t rows, int count) {
      for (int q = t; q < count * 8; q += T::kThreads) {
        const int row = q >> 3, c = q & 7;
        const int64_t at = row0 + row < rows ? row0 + row : rows - 1;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (c * 16 < tail) v = *reinterpret_cast<const uint4*>(src + at * L + l0 + c * 16);
        *reinterpret_cast<uint4*>(dst + row * 128 + (c ^ row_swz(row)) * 16) = v;
      }
    };
    row_tile(st, g.x, m0, g.M, T::kBM);
    if constexpr (kBwd) {
      constexpr int kSlots = T::kBN / 16;
      for (int q = t; q < 128 * kSlots; q += T::kThreads) {
        const int row = q / kSlots, c = q % kSlots;
        const int64_t col = c0 + c * 16 < g.K ? c0 + c * 16 : g.K - 16;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < tail) v = *reinterpret_cast<const uint4*>(g.w + (l0 + row) * g.K + col);
        *reinterpret_cast<uint4*>(st + T::kA + row * T::kBN +
                                  (c ^ col_swz<T::kBN>(row)) * 16) = v;
      }
    } else {
      row_tile(st + T::kA, g.w, c0, g.N, T::kBN);
    }
    float* sS = reinterpret_cast<float*>(st + T::kA + T::kB);
    for (int q = t; q < T::kBM; q += T::kThreads)
      sS[q] = g.xs[nfull * g.M + (m0 + q < g.M ? m0 + q : g.M - 1)];
    __syncthreads();
    mma_step<T, kBwd>(st, wsp[nfull * ws_step], wm, wn, li, lg, acc);
  }

  // LoRA term, 32 ranks at a time, operands from the caches: they are a few
  // KB per tile against the main loop's hundreds.
  for (int j0 = 0; j0 < g.r; j0 += 32) {
    const int rj = j0 + 8 * lg, left = g.r - rj;
    uint4 wf[T::kTJ];
#pragma unroll
    for (int j = 0; j < T::kTJ; ++j) {
      int64_t n = c0 + wn * 64 + j * 16 + li;
      n = n < ncols ? n : ncols - 1;
      wf[j] = kBwd ? load_bf16x8_strided(g.lw + rj * g.K + n, g.K, left)
                   : load_bf16x8(g.lw + n * g.r + rj, left, g.vec_w);
    }
#pragma unroll
    for (int i = 0; i < T::kTI; ++i) {
      int64_t m = m0 + wm * T::kWTM + i * 16 + li;
      m = m < g.M ? m : g.M - 1;
      const uint4 af = load_bf16x8(g.lact + m * g.r + rj, left, (g.r & 7) == 0);
#pragma unroll
      for (int j = 0; j < T::kTJ; ++j) acc[i][j] = mfma_bf16_32(wf[j], af, acc[i][j]);
    }
  }

  // Epilogue: lane (li, lg) holds columns 16 j + 4 lg .. + 3 of token 16 i +
  // li.  Each wave turns its tile to bf16 through LDS, 64 tokens at a time,
  // and stores whole 128-byte row segments.
  __syncthreads();
  constexpr int kPitch = 64 + 8;
  uint16_t* stg = reinterpret_cast<uint16_t*>(smem) + wave * 64 * kPitch;
  static_assert(T::kWaves * 64 * kPitch * 2 <= 2 * T::kStage, "staging fits");
#pragma unroll
  for (int h = 0; h < T::kWTM / 64; ++h) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < T::kTJ; ++j) {
        const f32x4_t& c = acc[4 * h + i][j];
        *reinterpret_cast<uint2*>(stg + (i * 16 + li) * kPitch + j * 16 + 4 * lg) =
            make_uint2(pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3]));
      }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int row = s * 8 + (lane >> 3), ch = lane & 7;
      const uint4 v = *reinterpret_cast<const uint4*>(stg + row * kPitch + ch * 8);
      const int64_t m = m0 + wm * T::kWTM + h * 64 + row;
      const int64_t n = c0 + wn * 64 + ch * 8;
      if (m < g.M && n < ncols) *reinterpret_cast<uint4*>(g.out + m * ncols + n) = v;
    }
    __syncthreads();
  }
}

template <typename T>
hipError_t run(const Fp8Args& g, bool bwd, hipStream_t st) {
  const int64_t ncols = bwd ? g.K : g.N;
  const dim3 grid(static_cast<uint32_t>(((ncols + T::kBN - 1) / T::kBN) *
                                        ((g.M + T::kBM - 1) / T::kBM)));
  if (bwd)
    hipLaunchKernelGGL((fp8_gemm_kernel<T, true>), grid, dim3(T::kThreads), 0, st, g);
  else
    hipLaunchKernelGGL((fp8_gemm_kernel<T, false>), grid, dim3(T::kThreads), 0, st, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8View& w, const uint8_t* x, const float* xs, int64_t M,
                           const uint16_t* lact, const uint16_t* lw, int r, bool bwd, uint16_t* out,
                           hipStream_t st) {
  if (M == 0) return hipSuccess;
  const bool vec_w = (r & 7) == 0 && (reinterpret_cast<uintptr_t>(lw) & 15) == 0;
  Fp8Args g{w.codes, w.scale, x, xs, M, w.N, w.K, lact, lw, r, vec_w, out};
  const int64_t ncols = bwd ? w.K : w.N;
  const int64_t big = ((ncols + 255) / 256) * ((M + 255) / 256);
  if (big >= 256) return run<Tile<128, 2, 4>>(g, bwd, st);
  return run<Tile<64, 2, 2>>(g, bwd, st);
}

}  // namespace qn
