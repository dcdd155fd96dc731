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
// LoRA term comes first on the same accumulators, multiplied by bf16 MFMAs: s u
// (s t) is there as two bf16 parts, whose 32 ranks are a block of 128 bytes
// too, and 64 ranks of the adapter are another, both laid out like codes.
//
// Tiles.  A wave holds kWTM x 64 outputs, which lie in one 128-block of the
// weight, so the weight's scale is wave-uniform; the MFMAs take the weight as
// first operand, so a lane's four results are four columns of one token and
// the token's scale is one register.  Both operand tiles (128 bytes of the
// contraction per step) and their scales are brought in by direct-to-LDS DMA,
// one or two steps ahead in two or three buffers; 16-byte chunks of a row are
// XOR-swizzled by the choice of each lane's source address, so that the
// fragment reads hit all banks.  The loop holds no other vector-memory
// instruction: one scale loaded to a register made the compiler wait for all
// outstanding DMAs in every step (4096 x 22016 x 8192: 720 -> 656 us).  The
// backward's weight tile lies [n][k] in memory while a lane needs 32 n of one
// k: it is read through the transposing LDS loads (8 rows x 16 columns of
// bytes per 16 lanes).

#include "qn_fp8.h"
#include "qn_launch.h"

namespace qn {

namespace {

typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2_t lds_i32x2_t;
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;
typedef __attribute__((address_space(3))) uint8_t lds_u8_t;

struct Fp8Args {
  const uint8_t* w;    // codes [N, K]
  const float* ws;     // scales [ceil(N / 128), ceil(K / 128)]
  const uint8_t* x;    // codes [M, L], L the contraction length
  const float* xs;     // scales [ceil(L / 128), M]
  int64_t M, N, K;
  const uint16_t* act;  // s u or s t in two parts, [M] rows of `pitch` values
  const uint16_t* lw;   // B [N, r] or A [r, K]
  int r, pitch;
  bool vec_w;           // lw can be read 16 bytes at a time
  uint16_t* out;
  float* part;          // [splits][M][ncols] fp32 instead of out, or nullptr
};

template <int kWTM_, int kGM_, int kGN_, int kBuf_>
struct Tile {
  static constexpr int kWTM = kWTM_, kGM = kGM_, kGN = kGN_;
  static constexpr int kBuf = kBuf_;                      // blocks held in LDS
  static constexpr int kBM = kWTM * kGM, kBN = 64 * kGN;
  static constexpr int kWaves = kGM * kGN, kThreads = 64 * kWaves;
  static constexpr int kA = kBM * 128, kB = kBN * 128;    // bytes of an operand tile
  static constexpr int kScales = kA + kB;                 // offset of the tokens' scales
  static constexpr int kWScales = kScales + kBM * 4;      // and of the weight's, 64 floats
  static constexpr int kStage = kWScales + 256;
  static constexpr int kDmaA = kA / 1024 / kWaves, kDmaB = kB / 1024 / kWaves;
  static constexpr int kDmaS = kBM / 64;                  // waves that fetch 64 scales each
  static constexpr int kTI = kWTM / 16, kTJ = 4;          // MFMA tiles of a wave
  static constexpr int kShare = 4;                             // DMAs issued at a time
  static_assert(kDmaA * 1024 * kWaves == kA && kDmaB * 1024 * kWaves == kB && kDmaS <= kWaves,
                "tile split");
  static_assert(kDmaS < kWaves, "a wave is left for the weight's scales");
};

// Slot of 16-byte chunk c in a 128-byte row is c ^ row_swz(row).  A 16-byte
// LDS read serves lanes 0-3, 12-15, 20-27 at once (then 4-11, 16-19, 28-31,
// and the same of the upper half): with lane = 16 g + row and chunk 2 g, half
// of the 16 rows are read at chunk c and half at c ^ 2, and this swizzle
// gives them 16 different groups of 4 banks.  ((row >> 1) & 7, right for 16
// consecutive lanes, cost 4 extra cycles a read.)
__device__ __forceinline__ int row_swz(int row) { return (row >> 1) & 5; }

// The same for the backward's weight tile of kBN bytes a row, whose reads
// take rows 8 q + 32 g .. + 7 of two g at a time.
template <int kBN>
__device__ __forceinline__ int col_swz(int row) {
  if constexpr (kBN == 256) return (row & 7) | ((row >> 5) & 1) << 3;
  return ((row >> 1) & 3) | ((row >> 5) & 1) << 2;
}

// And of A's 32-byte chunks of 16 columns in the LoRA term's rank rows, whose
// reads take rows 8 g + 0 .. 3 of all four g at a time.
__device__ __forceinline__ int lora_swz(int row) { return (row & 3) | ((row >> 3) & 1) << 2; }

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

// Place in the tile order of workgroup bid of total: the workgroups of one
// XCD (bid % 8) take a contiguous run of it.
__device__ __forceinline__ int xcd_run(int bid, int total) {
  const int x = bid & 7, base = total >> 3, rem = total & 7;
  return x * base + (x < rem ? x : rem) + (bid >> 3);
}

// Tile q of nr x nc in the tile order: bands of kBandRows row tiles, column
// by column within a band, so that the tiles an XCD works on at a time share
// their rows of x and columns of W in its L2 (2 and 16 rows: 4-10% slower at
// 2048 x 11008 x 4096 and 4096 x 22016 x 8192; 8 the same).
constexpr int kBandRows = 4;

__device__ __forceinline__ void fp8_tile_of(int q, int nc, int nr, int& row, int& col) {
  const int band = q / (kBandRows * nc);
  const int local = q - band * kBandRows * nc;
  const int rows = nr - band * kBandRows < kBandRows ? nr - band * kBandRows : kBandRows;
  col = local / rows;
  row = band * kBandRows + local % rows;
}

// Fragments of a step: weight columns 16 j .. + 15 of the wave's tile, and
// the tokens 16 i .. + 15.
template <typename T, bool kBwd>
__device__ __forceinline__ i32x8_t weight_frag(const uint8_t* sB, int wn, int j, int li, int g) {
  if constexpr (kBwd) {
    // lanes 2 r, 2 r + 1 of a group point at row 32 g + 8 q + r, columns 0-7
    // and 8-15; lane c receives column c of the 8 rows
    const int f = col_swz<T::kBN>((li >> 1) + 32 * g);
    const uint8_t* p =
        sB + (32 * g + (li >> 1)) * T::kBN + (((wn * 4 + j) ^ f) << 4) + (li & 1) * 8;
    i32x8_t b;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const i32x2_t v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (lds_i32x2_t*)(lds_u8_t*)(p + q * 8 * T::kBN));
      b[2 * q] = v[0];
      b[2 * q + 1] = v[1];
    }
    return b;
  }
  const int slot = (2 * g) ^ row_swz(li);
  const uint8_t* p = sB + (wn * 64 + j * 16 + li) * 128;
  return frag8(*reinterpret_cast<const uint4*>(p + slot * 16),
               *reinterpret_cast<const uint4*>(p + (slot ^ 1) * 16));
}

template <typename T>
__device__ __forceinline__ i32x8_t token_frag(const uint8_t* sA, int wm, int i, int li, int g) {
  const int slot = (2 * g) ^ row_swz(li);
  const uint8_t* p = sA + (wm * T::kWTM + i * 16 + li) * 128;
  return frag8(*reinterpret_cast<const uint4*>(p + slot * 16),
               *reinterpret_cast<const uint4*>(p + (slot ^ 1) * 16));
}

// Fragments of a block that are read ahead of it: the weight's, the first
// tokens' and all tokens' scales.
template <typename T>
struct Ahead {
  i32x8_t a[2], b[T::kTJ];
  float s[T::kTI], sw;
};

template <typename T>
__device__ __forceinline__ void read_scales(const uint8_t* st, int wm, int wn, int li,
                                            Ahead<T>& f) {
  const float* sS = reinterpret_cast<const float*>(st + T::kScales) + wm * T::kWTM + li;
#pragma unroll
  for (int i = 0; i < T::kTI; ++i) f.s[i] = sS[16 * i];
  f.sw = reinterpret_cast<const float*>(st + T::kWScales)[wn / 2];
}

template <typename T, bool kBwd>
__device__ __forceinline__ void read_ahead(const uint8_t* st, int wm, int wn, int li, int g,
                                           Ahead<T>& f) {
  f.a[0] = token_frag<T>(st, wm, 0, li, g);
#pragma unroll
  for (int j = 0; j < T::kTJ; ++j) f.b[j] = weight_frag<T, kBwd>(st + T::kA, wn, j, li, g);
  read_scales<T>(st, wm, wn, li, f);
}

// Results of the MFMAs that are still to be scaled and added.
template <typename T>
struct Pending {
  f32x4_t c[T::kTJ];
  float f;
};

template <typename T>
__device__ __forceinline__ void add_pending(const Pending<T>& p, int j, f32x4_t& acc) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = fmaf(p.c[j][e], p.f, acc[e]);
}

// LoRA term: the tokens' side 32 ranks at a time (128 bytes a row, both parts)
// by DMA, the adapter's 64 at a time from where it lies, through registers:
// rows of B as the codes' rows, or A's 64 rows of kBN columns, which the
// transposing LDS loads read.
template <typename T>
struct LoraRows {
  uint4 v[T::kBN * 8 / T::kThreads];
};

template <typename T>
__device__ __forceinline__ void lora_tokens(const Fp8Args& g, int lb, int64_t m0, uint8_t* st) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint16_t* pa = g.act + m0 * g.pitch + lb * 64;
#pragma unroll
  for (int d = 0; d < T::kDmaA; ++d) {
    const int row = 8 * (wave * T::kDmaA + d) + (lane >> 3);
    const int64_t at = m0 + row < g.M ? row : g.M - 1 - m0;
    dma16(static_cast<uint32_t>(at * g.pitch * 2 + ((lane & 7) ^ row_swz(row)) * 16), pa,
          lds_addr(st) + (wave * T::kDmaA + d) * 1024);
  }
}

template <typename T, bool kBwd>
__device__ __forceinline__ void lora_load(const Fp8Args& g, int lb, int64_t c0, LoraRows<T>& w) {
  const int t = threadIdx.x;
#pragma unroll
  for (int q = 0; q < static_cast<int>(sizeof(w.v) / 16); ++q) {
    const int e = q * T::kThreads + t;
    const uint16_t* src;
    bool in;
    int left;
    if constexpr (kBwd) {
      const int64_t c = c0 + e % (T::kBN / 8) * 8;
      const int j = lb * 64 + e / (T::kBN / 8);
      in = j < g.r;
      left = 8;
      src = g.lw + (in ? j : 0) * g.K + (c < g.K ? c : g.K - 8);
    } else {
      const int64_t n = c0 + (e >> 3);
      const int j = lb * 64 + (e & 7) * 8;
      in = j < g.r;
      left = in ? g.r - j : 8;
      src = g.lw + (n < g.N ? n : g.N - 1) * g.r + (in ? j : 0);
    }
    if (g.vec_w) {
      w.v[q] = *reinterpret_cast<const uint4*>(src);
      if (!in) w.v[q] = make_uint4(0, 0, 0, 0);
    } else {
      w.v[q] = load_bf16x8(src, in ? left : 0, false);
    }
  }
}

template <typename T, bool kBwd>
__device__ __forceinline__ void lora_store(uint8_t* st, const LoraRows<T>& w) {
#pragma unroll
  for (int q = 0; q < static_cast<int>(sizeof(w.v) / 16); ++q) {
    const int e = q * T::kThreads + static_cast<int>(threadIdx.x);
    uint8_t* dst = st + T::kA;
    if constexpr (kBwd) {
      const int j = e / (T::kBN / 8), c = e % (T::kBN / 8);
      dst += j * (T::kBN * 2) + (((c >> 1) ^ lora_swz(j)) << 5) + (c & 1) * 16;
    } else {
      dst += (e >> 3) * 128 + ((e & 7) ^ row_swz(e >> 3)) * 16;
    }
    *reinterpret_cast<uint4*>(dst) = w.v[q];
  }
}

// Adds the ranks 32 lb .. + 31, which are the half lb & 1 of the adapter's.
template <typename T, bool kBwd>
__device__ __forceinline__ void lora_add(int lb, const uint8_t* st,
                                         f32x4_t (&acc)[T::kTI][T::kTJ]) {
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / T::kGN, wn = wave % T::kGN;
  const int half = lb & 1;
  uint4 b[T::kTJ];
#pragma unroll
  for (int j = 0; j < T::kTJ; ++j) {
    if constexpr (kBwd) {
      // lane 4 a + e of a group points at rank row a, columns 4 e .. + 3
      uint2 h[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int row = 32 * half + 8 * lg + 4 * q + (li >> 2);
        const i16x4_t d = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_i16x4_t*)(lds_u8_t*)(st + T::kA + row * (T::kBN * 2) +
                                      (((wn * 4 + j) ^ lora_swz(row)) << 5) + (li & 3) * 8));
        h[q] = __builtin_bit_cast(uint2, d);
      }
      b[j] = make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
    } else {
      const int at = ((4 * half + lg) ^ row_swz(li)) * 16;
      b[j] = *reinterpret_cast<const uint4*>(st + T::kA + (wn * 64 + j * 16 + li) * 128 + at);
    }
  }
#pragma unroll 1
  for (int p = 0; p < 2; ++p) {
    const int at = ((4 * p + lg) ^ row_swz(li)) * 16;
#pragma unroll
    for (int i = 0; i < T::kTI; ++i) {
      const uint4 a = *reinterpret_cast<const uint4*>(st + (wm * T::kWTM + i * 16 + li) * 128 + at);
#pragma unroll
      for (int j = 0; j < T::kTJ; ++j) acc[i][j] = mfma_bf16_32(b[j], a, acc[i][j]);
    }
  }
}

// The contraction's last, partial block: through registers, zeros behind its
// end.
template <typename T>
struct TailRows {
  uint4 a[T::kBM * 8 / T::kThreads], b[T::kBN * 8 / T::kThreads];
  float s, ws;
};

template <typename T, bool kBwd>
__device__ __forceinline__ void tail_load(const Fp8Args& g, int tail, int64_t m0, int64_t c0,
                                          int64_t bt, TailRows<T>& w) {
  const int t = threadIdx.x;
  const int64_t ncols = kBwd ? g.K : g.N, L = kBwd ? g.N : g.K;
  const int64_t kb = (g.K + 127) / 128, cmax = (ncols - 1) / 128, l0 = bt * 128;
  auto row_chunk = [&](const uint8_t* src, int64_t row0, int64_t rows, int q) {
    const int c = q & 7;
    const int64_t row = row0 + (q >> 3);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (c * 16 < tail)
      v = *reinterpret_cast<const uint4*>(src + (row < rows ? row : rows - 1) * L + l0 + c * 16);
    return v;
  };
#pragma unroll
  for (int q = 0; q < static_cast<int>(sizeof(w.a) / 16); ++q)
    w.a[q] = row_chunk(g.x, m0, g.M, q * T::kThreads + t);
#pragma unroll
  for (int q = 0; q < static_cast<int>(sizeof(w.b) / 16); ++q) {
    const int e = q * T::kThreads + t;
    if constexpr (kBwd) {
      constexpr int kSlots = T::kBN / 16;
      const int row = e / kSlots;
      const int64_t col = c0 + e % kSlots * 16;
      w.b[q] = make_uint4(0, 0, 0, 0);
      if (row < tail)
        w.b[q] = *reinterpret_cast<const uint4*>(g.w + (l0 + row) * g.K +
                                                 (col < g.K ? col : g.K - 16));
    } else {
      w.b[q] = row_chunk(g.w, c0, g.N, e);
    }
  }
  static_assert(T::kThreads >= T::kBM, "a thread per token's scale");
  const int64_t m = m0 + t < g.M ? m0 + t : g.M - 1;
  const int64_t cb = c0 / 128 + (t & 3), c = cb < cmax ? cb : cmax;
  w.s = g.xs[bt * g.M + m];
  w.ws = g.ws[kBwd ? bt * kb + c : c * kb + bt];
}

template <typename T, bool kBwd>
__device__ __forceinline__ void tail_store(uint8_t* st, const TailRows<T>& w) {
  const int t = threadIdx.x;
#pragma unroll
  for (int q = 0; q < static_cast<int>(sizeof(w.a) / 16); ++q) {
    const int e = q * T::kThreads + t, row = e >> 3;
    *reinterpret_cast<uint4*>(st + row * 128 + ((e & 7) ^ row_swz(row)) * 16) = w.a[q];
  }
#pragma unroll
  for (int q = 0; q < static_cast<int>(sizeof(w.b) / 16); ++q) {
    const int e = q * T::kThreads + t;
    if constexpr (kBwd) {
      constexpr int kSlots = T::kBN / 16;
      const int row = e / kSlots, c = e % kSlots;
      *reinterpret_cast<uint4*>(st + T::kA + row * T::kBN + (c ^ col_swz<T::kBN>(row)) * 16) =
          w.b[q];
    } else {
      const int row = e >> 3;
      *reinterpret_cast<uint4*>(st + T::kA + row * 128 + ((e & 7) ^ row_swz(row)) * 16) = w.b[q];
    }
  }
  if (t < T::kBM) reinterpret_cast<float*>(st + T::kScales)[t] = w.s;
  if (t < 4) reinterpret_cast<float*>(st + T::kWScales)[t] = w.ws;
}

template <typename T, bool kBwd>
__device__ __forceinline__ void tail_add(const uint8_t* st, f32x4_t (&acc)[T::kTI][T::kTJ]) {
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / T::kGN, wn = wave % T::kGN;
  Ahead<T> f;
  read_ahead<T, kBwd>(st, wm, wn, li, lg, f);
#pragma unroll
  for (int i = 0; i < T::kTI; ++i) {
    if (i > 0) f.a[0] = token_frag<T>(st, wm, i, li, lg);
#pragma unroll
    for (int j = 0; j < T::kTJ; ++j) {
      const f32x4_t c = mfma_fp8(f.b[j], f.a[0], f32x4_t{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(c[e], f.s[i] * f.sw, acc[i][j][e]);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// One output tile: rows from m0, columns from c0, the contraction's blocks
// from b0, nfull whole ones and a tail of `tail` values behind them; the LoRA
// term is added where first is set.
template <typename T, bool kBwd>
__device__ __forceinline__ void fp8_tile(const Fp8Args& g, uint8_t* smem, int64_t m0, int64_t c0,
                                         int b0, int nfull, int tail, bool first, int split) {
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / T::kGN, wn = wave % T::kGN;
  const int li = lane & 15, lg = lane >> 4;
  const int64_t ncols = kBwd ? g.K : g.N, L = kBwd ? g.N : g.K;
  const int64_t kb = (g.K + 127) / 128;
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
  // Scales of a block: the first kDmaS waves fetch 64 tokens' each, the
  // others the weight's (lane l that of column block l % 4 of the tile).
  const bool tok = wave < T::kDmaS;
  const int64_t cmax = (ncols - 1) / 128;
  const int srow = wave * 64 + lane;
  int64_t cblk = c0 / 128 + (lane & 3);
  cblk = cblk < cmax ? cblk : cmax;
  const uint32_t offS = static_cast<uint32_t>(
      tok ? (m0 + srow < g.M ? srow : g.M - 1 - m0) * 4 : (cblk - c0 / 128) * (kBwd ? 1 : kb) * 4);
  const float* baseS = tok ? g.xs + m0 : kBwd ? g.ws + c0 / 128 : g.ws + c0 / 128 * kb;
  const int64_t stepS = tok ? g.M : kBwd ? kb : 1;
  baseS += b0 * stepS;
  const uint32_t dstS = tok ? T::kScales + wave * 256 : T::kWScales;
  const uint8_t* baseA = g.x + m0 * L + static_cast<int64_t>(b0) * 128;
  const uint8_t* baseB = kBwd ? g.w + c0 + static_cast<int64_t>(b0) * 128 * g.K
                              : g.w + c0 * L + static_cast<int64_t>(b0) * 128;
  const uint32_t lds0 = lds_addr(smem);
  // share q of the DMAs of block b, into buffer buf
  constexpr int kDma = T::kDmaA + T::kDmaB;
  auto issue = [&](int b, int buf, int q) {
    const uint32_t st = lds0 + buf * T::kStage;
    const uint8_t* pa = baseA + static_cast<int64_t>(b) * 128;
    const uint8_t* pb = kBwd ? baseB + static_cast<int64_t>(b) * 128 * g.K
                             : baseB + static_cast<int64_t>(b) * 128;
#pragma unroll
    for (int d = q * T::kShare; d < (q + 1) * T::kShare && d < kDma; ++d) {
      if (d < T::kDmaA)
        dma16(offA[d], pa, st + (wave * T::kDmaA + d) * 1024);
      else
        dma16(offB[d - T::kDmaA], pb, st + T::kA + (wave * T::kDmaB + d - T::kDmaA) * 1024);
    }
    if (q == 0) dma4(offS, baseS + b * stepS, st + dstS);
  };

  f32x4_t acc[T::kTI][T::kTJ];
#pragma unroll
  for (int i = 0; i < T::kTI; ++i)
#pragma unroll
    for (int j = 0; j < T::kTJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // Before the blocks, with the first block's DMAs in flight: the LoRA term
  // and the tail, whose own memory latency passes meanwhile (behind the last
  // block it was exposed: 3000 x 5008 x 2000 with r = 16 53 -> 51 us).
  constexpr int kShares = (kDma + T::kShare - 1) / T::kShare;
  const int last = nfull - 1;
  auto upto = [&](int b) { return b < last ? b : last; };
  auto issue_all = [&](int b) {
#pragma unroll
    for (int q = 0; q < kShares; ++q) issue(upto(b), b, q);
  };
  if (nfull > 0) issue_all(0);
  const int rank = first ? g.r : 0;
  if (rank > 0 || tail) {
    uint8_t* stL = smem + (T::kBuf - 1) * T::kStage;
    uint8_t* stT = smem + (T::kBuf > 2 ? T::kBuf - 2 : 1) * T::kStage;
    LoraRows<T> lw;
    TailRows<T> tr;
    if (rank > 0) {
      lora_tokens<T>(g, 0, m0, stL);
      lora_load<T, kBwd>(g, 0, c0, lw);
    }
    if (tail) tail_load<T, kBwd>(g, tail, m0, c0, b0 + nfull, tr);
    for (int lb = 0; lb * 32 < rank; ++lb) {
      if (lb > 0) {
        __syncthreads();
        lora_tokens<T>(g, lb, m0, stL);
        if ((lb & 1) == 0) lora_load<T, kBwd>(g, lb >> 1, c0, lw);
      }
      if ((lb & 1) == 0) lora_store<T, kBwd>(stL, lw);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      lora_add<T, kBwd>(lb, stL, acc);
    }
    if (tail) {
      if (T::kBuf == 2) __syncthreads();
      tail_store<T, kBwd>(stT, tr);
      __syncthreads();
      tail_add<T, kBwd>(stT, acc);
    }
    __syncthreads();
  }

  // Step b multiplies block b (buffer b % kBuf).  Its MFMAs of tokens 16 i run
  // while the fragment of tokens 16 (i + 1) is read and the results of tokens
  // 16 (i - 1) are scaled and added.  Before the last i comes the turn: this
  // wave's reads of the buffer have returned and block b + 1 has landed, for
  // all waves after the barrier; from there on block b + 1's first fragments
  // are read under the last MFMAs, and the DMAs of block b + kBuf go out, a
  // share per i (a DMA takes the address unit 16 cycles, so all at once would
  // hold the reads up; too late and the next turn waits for them).  Blocks
  // past the end are the last one again: a branch would cut the
  // step into pieces, and the last steps compiled apart without those DMAs
  // spilled registers (656 -> 745 us at 4096 x 22016 x 8192).
  if (nfull > 0) {
    constexpr int kEnd = T::kTI - 1;
    static_assert(kShares < T::kTI, "the DMAs of a block go out before the next turn");
#pragma unroll
    for (int b = 1; b < T::kBuf - 1; ++b) issue_all(b);
    // all DMAs but those of the kBuf - 2 youngest blocks have landed
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((T::kBuf - 2) * (kDma + 1)) : "memory");
    issue(upto(T::kBuf - 1), T::kBuf - 1, 0);
    Ahead<T> f;
    Pending<T> p;
#pragma unroll
    for (int j = 0; j < T::kTJ; ++j) p.c[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    p.f = 0.0f;
    read_ahead<T, kBwd>(smem, wm, wn, li, lg, f);
    int buf = 0;
    for (int b = 0; b <= last; ++b) {
      const int bnext = buf + 1 == T::kBuf ? 0 : buf + 1;
      const int bprev = buf == 0 ? T::kBuf - 1 : buf - 1;
      const uint8_t* cur = smem + buf * T::kStage;
      const uint8_t* nxt = smem + bnext * T::kStage;
#pragma unroll
      for (int i = 0; i < T::kTI; ++i) {
        if (i < kEnd) {
          f.a[(i + 1) & 1] = token_frag<T>(cur, wm, i + 1, li, lg);
        } else {
          asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((T::kBuf - 2) *
                                                                          (kDma + 1))
                       : "memory");
          f.a[0] = token_frag<T>(nxt, wm, 0, li, lg);
        }
#pragma unroll
        for (int j = 0; j < T::kTJ; ++j) {
          add_pending<T>(p, j, acc[i > 0 ? i - 1 : kEnd][j]);
          p.c[j] = mfma_fp8(f.b[j], f.a[i & 1], f32x4_t{0.f, 0.f, 0.f, 0.f});
          if (i == kEnd) f.b[j] = weight_frag<T, kBwd>(nxt + T::kA, wn, j, li, lg);
        }
        p.f = f.s[i] * f.sw;
        if (i == kEnd) {
          read_scales<T>(nxt, wm, wn, li, f);
          issue(upto(b + T::kBuf), buf, 0);
        } else if (i + 1 < kShares) {
          issue(upto(b + T::kBuf - 1), bprev, i + 1);
        }
        // every second i: within two of them the compiler interleaves better
        // than as written, over the whole step worse (88 us against 92 with a
        // fence at each i and without any, 2048 x 4096 x 11008)
        if (i & 1) __builtin_amdgcn_sched_barrier(0);
      }
      buf = bnext;
    }
#pragma unroll
    for (int j = 0; j < T::kTJ; ++j) add_pending<T>(p, j, acc[kEnd][j]);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }

  if (g.part) {
    float* part = g.part + static_cast<int64_t>(split) * g.M * ncols;
#pragma unroll
    for (int i = 0; i < T::kTI; ++i)
#pragma unroll
      for (int j = 0; j < T::kTJ; ++j) {
        const int64_t m = m0 + wm * T::kWTM + i * 16 + li, n = c0 + wn * 64 + j * 16 + 4 * lg;
        if (m < g.M && n < ncols) *reinterpret_cast<f32x4_t*>(part + m * ncols + n) = acc[i][j];
      }
    return;
  }
  // Epilogue: lane (li, lg) holds columns 16 j + 4 lg .. + 3 of token 16 i +
  // li.  Each wave turns its tile to bf16 through LDS, 64 tokens at a time,
  // and stores whole 128-byte row segments.
  __syncthreads();
  constexpr int kPitch = 64 + 8;
  constexpr int kTurn = T::kWTM < 64 ? T::kWTM : 64;  // tokens of a turn
  uint16_t* stg = reinterpret_cast<uint16_t*>(smem) + wave * kTurn * kPitch;
  static_assert(T::kWaves * kTurn * kPitch * 2 <= 2 * T::kStage, "staging fits");
#pragma unroll
  for (int h = 0; h < T::kWTM / kTurn; ++h) {
#pragma unroll
    for (int i = 0; i < kTurn / 16; ++i)
#pragma unroll
      for (int j = 0; j < T::kTJ; ++j) {
        const f32x4_t& c = acc[kTurn / 16 * h + i][j];
        *reinterpret_cast<uint2*>(stg + (i * 16 + li) * kPitch + j * 16 + 4 * lg) =
            make_uint2(pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3]));
      }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kTurn / 8; ++s) {
      const int row = s * 8 + (lane >> 3), ch = lane & 7;
      const uint4 v = *reinterpret_cast<const uint4*>(stg + row * kPitch + ch * 8);
      const int64_t m = m0 + wm * T::kWTM + h * kTurn + row;
      const int64_t n = c0 + wn * 64 + ch * 8;
      if (m < g.M && n < ncols) *reinterpret_cast<uint4*>(g.out + m * ncols + n) = v;
    }
    __syncthreads();
  }
}

using Big = Tile<128, 2, 4, 2>;    // 256 x 256, 8 waves
using Half = Tile<64, 2, 4, 3>;    // 128 x 256, 8 waves
// 128 x 128, 8 waves: grids of at most one workgroup per CU are bound by the
// latency of a step, which a second wave per SIMD and a third buffer hide
// (333 x 1088 x 2112: 13.7 us; with 4 waves 16.8, with two buffers 15.4, with
// four 14.2; a 32 x 64 wave tile reads LDS 1.5 times as often as 64 x 64).
using Small = Tile<32, 4, 2, 3>;
constexpr int kMixedLds = Big::kBuf * Big::kStage > Half::kBuf * Half::kStage
                              ? Big::kBuf * Big::kStage
                              : Half::kBuf * Half::kStage;

// Measured, median launches of several runs: 4096 x 22016 x 8192 forward 638-645
// us (2.3 PF; least 614), 2048 x 11008 x 4096 forward 94-105, backward 90-105.
// The vendor's FP8 product with one scale per tensor: 616-622 and, forward, 91.
// Without the DMAs the first takes about 80% of its time, without the LDS reads
// 85%, without the MFMAs 85%: none of them alone bounds it.
//
// Workgroups below nbig take one 256 x 256 tile each, the others half of one
// of the remaining tiles: 256-row tiles halve the LDS reads per product, but
// a last round that fills less than half of the 256 CUs with them costs as
// much as a full one, and as halves it takes about 0.6 of that.  A batch of up
// to 128 tokens is one row of upper halves (32 x 65536 x 4096 71 us, in whole
// tiles 82; 100 x 33024 x 4096 37 and 53; 128 x 128256 x 4096 140 and 154).
template <bool kBwd>
__global__ __launch_bounds__(Big::kThreads, 2) void fp8_gemm_kernel(Fp8Args g, int nbig) {
  static_assert(Big::kThreads == Half::kThreads && Big::kBN == Half::kBN &&
                    Big::kBM == 2 * Half::kBM,
                "a half tile has the same workgroup");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kMixedLds];
  const int nc = static_cast<int>(((kBwd ? g.K : g.N) + Big::kBN - 1) / Big::kBN);
  const int nr = static_cast<int>((g.M + Big::kBM - 1) / Big::kBM);
  const int bid = blockIdx.x;
  const int64_t L = kBwd ? g.N : g.K;
  const int nfull = static_cast<int>(L / 128), tail = static_cast<int>(L % 128);
  int row, col;
  if (bid < nbig) {
    fp8_tile_of(xcd_run(bid, nbig), nc, nr, row, col);
    fp8_tile<Big, kBwd>(g, smem, static_cast<int64_t>(row) * Big::kBM,
                        static_cast<int64_t>(col) * Big::kBN, 0, nfull, tail, true, 0);
  } else {
    const int two = g.M > Half::kBM ? 1 : 0;  // log2 of the halves of a tile
    const int q = xcd_run(bid - nbig, (nc * nr - nbig) << two);
    fp8_tile_of(nbig + (q >> two), nc, nr, row, col);
    const int64_t m0 = static_cast<int64_t>(row) * Big::kBM + (q & two) * Half::kBM;
    if (m0 < g.M)
      fp8_tile<Half, kBwd>(g, smem, m0, static_cast<int64_t>(col) * Half::kBN, 0, nfull, tail,
                           true, 0);
  }
}

// Workgroup row z takes the blocks z per .. of the contraction; the last one
// has the tail too.
template <bool kBwd>
__global__ __launch_bounds__(Small::kThreads) void fp8_gemm_small_kernel(Fp8Args g, int per) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[Small::kBuf * Small::kStage];
  const int nc = static_cast<int>(((kBwd ? g.K : g.N) + Small::kBN - 1) / Small::kBN);
  const int nr = static_cast<int>((g.M + Small::kBM - 1) / Small::kBM);
  const int64_t L = kBwd ? g.N : g.K;
  const int whole = static_cast<int>(L / 128), b0 = static_cast<int>(blockIdx.y) * per;
  const bool last = blockIdx.y + 1 == gridDim.y;
  int row, col;
  fp8_tile_of(xcd_run(blockIdx.x, nc * nr), nc, nr, row, col);
  fp8_tile<Small, kBwd>(g, smem, static_cast<int64_t>(row) * Small::kBM,
                        static_cast<int64_t>(col) * Small::kBN, b0, last ? whole - b0 : per,
                        last ? static_cast<int>(L % 128) : 0, blockIdx.y == 0,
                        static_cast<int>(blockIdx.y));
}

int64_t small_tiles(int64_t M, int64_t ncols) {
  return ((ncols + Small::kBN - 1) / Small::kBN) * ((M + Small::kBM - 1) / Small::kBM);
}

// Large tiles where the small ones would take more than one round of the CUs
// (256 small tiles, 1000 x 4096 x 4096 with r = 16: small 33 us, large 40).
bool large(int64_t M, int64_t ncols) { return small_tiles(M, ncols) > 256; }

}  // namespace

int fp8_gemm_splits(int64_t M, int64_t ncols, int64_t L) {
  if (M <= 0 || large(M, ncols)) return 1;
  // Up to one workgroup per CU.  A block takes 0.42 us of a workgroup.  The
  // parts cost a launch, the turn to another workgroup and its latency, 2.4 us
  // in all, 0.1 us each in the sum, and their way out and back, 8 bytes an
  // output at 5.5 TB/s (mostly in the caches): as many as make the total least.
  // Whole and as chosen here, products of given rows, in us: 128 x 4096 x 11008
  // 41.0, in 6 20.1; 1000 x 1024 x 8192 32.2, in 4 20.4; 65 x 4096 x 4096 18.2,
  // in 4 12.6; 512 x 2048 x 4096 18.5, in 3 17.5; 128 x 11008 x 4096 19.8, in 2
  // 19.1; 100 x 1088 x 2112 11.8, in 4 10.2; 333 x 1088 x 2112 13.6, in 4 13.6.
  // Kept whole: 200 x 1040 x 1552 10.3, in 2 to 4 11.3 to 10.6; 333 x 2112 x
  // 1088 8.9, in 2 13.5; 1000 x 1024 x 2048 11.9, in 2 15.3.  More parts than
  // CUs gain nothing (412 x 4416 x 8672, 140 tiles, 45.9 us, in three 44.9).
  const int64_t blocks = L / 128, most = 256 / small_tiles(M, ncols);
  const double out = static_cast<double>(M) * static_cast<double>(ncols) * 8 / 5.5e6;
  double best = 0.42 * static_cast<double>(blocks);
  int splits = 1;
  for (int64_t s = 2; s <= most && s <= blocks; ++s) {
    const int64_t per = (blocks + s - 1) / s, n = (blocks + per - 1) / per;
    const double t = 0.42 * static_cast<double>(per) + 2.4 + (out + 0.1) * static_cast<double>(n);
    if (t < best) best = t, splits = static_cast<int>(n);
  }
  return splits;
}

hipError_t launch_fp8_gemm(const Fp8View& w, const uint8_t* x, const float* xs, int64_t M,
                           const uint16_t* act, const uint16_t* lw, int r, bool bwd, uint16_t* out,
                           float* part, hipStream_t st) {
  if (M == 0) return hipSuccess;
  // rows of B have r values, those of A K, a multiple of 16
  const bool vec_w = (reinterpret_cast<uintptr_t>(lw) & 15) == 0 && (bwd || (r & 7) == 0);
  const int64_t ncols = bwd ? w.K : w.N, L = bwd ? w.N : w.K;
  Fp8Args g{w.codes, w.scale, x, xs, M, w.N, w.K, act, lw, r, fp8_lora_pitch(r), vec_w, out,
            nullptr};
  if (large(M, ncols)) {
    // whole rounds of the 256 CUs in large tiles, a remainder of up to half
    // a round in halves
    const int64_t tiles = ((ncols + Big::kBN - 1) / Big::kBN) * ((M + Big::kBM - 1) / Big::kBM);
    const int64_t rest = tiles % 256, halves = M > Half::kBM ? 2 : 1;
    const int64_t nbig = halves == 1 ? 0 : rest <= 128 ? tiles - rest : tiles;
    const dim3 grid(static_cast<uint32_t>(nbig + halves * (tiles - nbig)));
    if (bwd)
      hipLaunchKernelGGL(fp8_gemm_kernel<true>, grid, dim3(Big::kThreads), 0, st, g,
                         static_cast<int>(nbig));
    else
      hipLaunchKernelGGL(fp8_gemm_kernel<false>, grid, dim3(Big::kThreads), 0, st, g,
                         static_cast<int>(nbig));
    return hipGetLastError();
  }
  const int splits = part ? fp8_gemm_splits(M, ncols, L) : 1;
  const int per = static_cast<int>((L / 128 + splits - 1) / splits);
  if (splits > 1) g.part = part;
  const dim3 grid(static_cast<uint32_t>(small_tiles(M, ncols)), static_cast<uint32_t>(splits));
  if (bwd)
    hipLaunchKernelGGL(fp8_gemm_small_kernel<true>, grid, dim3(Small::kThreads), 0, st, g, per);
  else
    hipLaunchKernelGGL(fp8_gemm_small_kernel<false>, grid, dim3(Small::kThreads), 0, st, g, per);
  const hipError_t e = hipGetLastError();
  return splits > 1 && e == hipSuccess ? launch_fp8_split_sum(part, splits, M * ncols, out, st) : e;
}

}  // namespace qn
