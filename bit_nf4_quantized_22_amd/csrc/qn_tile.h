// Device helpers of the tiled 8- and 4-bit products: DMAs into LDS, the order of
// the output tiles, the LoRA term and the way out.  A tile type T gives the
// tile's rows (tokens) kBM and columns kBN, the wave's kWTM tokens and 64
// columns in a kGM x kGN grid of waves, and the size of an operand's stage,
// whose rows have 128 bytes.
#pragma once

#include "qn_fp8.h"

namespace qn {

typedef __attribute__((address_space(3))) uint8_t lds_u8_t;

// Slot of 16-byte chunk c in a 128-byte row is c ^ row_swz(row).  A 16-byte
// LDS read serves lanes 0-3, 12-15, 20-27 at once (then 4-11, 16-19, 28-31,
// and the same of the upper half): with lane = 16 g + row and chunk 2 g, half
// of the 16 rows are read at chunk c and half at c ^ 2, and this swizzle
// gives them 16 different groups of 4 banks.  ((row >> 1) & 7, right for 16
// consecutive lanes, cost 4 extra cycles a read.)
__device__ __forceinline__ int row_swz(int row) { return (row >> 1) & 5; }

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

__device__ __forceinline__ void tile_of(int q, int nc, int nr, int& row, int& col) {
  const int band = q / (kBandRows * nc);
  const int local = q - band * kBandRows * nc;
  const int rows = nr - band * kBandRows < kBandRows ? nr - band * kBandRows : kBandRows;
  col = local / rows;
  row = band * kBandRows + local % rows;
}

// LoRA term: the tokens' side 32 ranks at a time (128 bytes a row, both parts)
// by DMA, the adapter's 64 at a time from where it lies, through registers:
// rows of B as the codes' rows, or A's 64 rows of kBN columns, which the
// transposing LDS loads read.
template <typename T>
struct LoraRows {
  uint4 v[T::kBN * 8 / T::kThreads];
};

template <typename T, typename G>
__device__ __forceinline__ void lora_tokens(const G& g, int lb, int64_t m0, uint8_t* st) {
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

template <typename T, bool kBwd, typename G>
__device__ __forceinline__ void lora_load(const G& g, int lb, int64_t c0, LoraRows<T>& w) {
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

// fp32 sums of the wave's outputs (columns are a multiple of 16) to part[M][ncols].
template <typename T>
__device__ __forceinline__ void store_part(float* part, int64_t M, int64_t ncols, int64_t m0,
                                           int64_t c0, const f32x4_t (&acc)[T::kTI][T::kTJ]) {
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / T::kGN, wn = wave % T::kGN;
#pragma unroll
  for (int i = 0; i < T::kTI; ++i)
#pragma unroll
    for (int j = 0; j < T::kTJ; ++j) {
      const int64_t m = m0 + wm * T::kWTM + i * 16 + li, n = c0 + wn * 64 + j * 16 + 4 * lg;
      if (m < M && n < ncols) *reinterpret_cast<f32x4_t*>(part + m * ncols + n) = acc[i][j];
    }
}

// The way out: lane (li, lg) holds columns 16 j + 4 lg .. + 3 of token 16 i +
// li.  Each wave turns its tile to bf16 through LDS, 64 tokens at a time, and
// stores whole 128-byte row segments.
template <typename T>
__device__ __forceinline__ void store_tile(uint16_t* out, int64_t M, int64_t ncols, int64_t m0,
                                           int64_t c0, uint8_t* smem,
                                           const f32x4_t (&acc)[T::kTI][T::kTJ]) {
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / T::kGN, wn = wave % T::kGN;
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
      if (m < M && n < ncols) *reinterpret_cast<uint4*>(out + m * ncols + n) = v;
    }
    __syncthreads();
  }
}

}  // namespace qn
