// Momentum and orthogonalised update (Muon) of many LoRA matrices (gfx950).
//
//   m <- mu m + (1 - mu) g;  u = (1 - mu) g + mu m (Nesterov) or m
//   X = u / (|u| + eps), as [r, L] with r <= L;  per step, S = X X^T:
//   X <- a X + (b S + c S^2) X;  p <- p (1 - lr wd) - lr f X
//
// Every iterate is a polynomial of S0 = X0 X0^T times X0, so the long side is
// passed over twice, not twice per step: one pass sums u u^T, the steps run on
// r x r matrices (S and T with X = T X0: Q = a I + b S + c S^2, T <- T Q, S <- S
// Q^2; all of them symmetric, and they commute), one pass multiplies u by T.
// S0 squares the singular values, and the steps raise the least of them by up to
// a factor of a^2 each, so u u^T, the steps and the last product are in 64
// bits, on the 64-bit matrix instruction: in 32 bits the least directions would
// be noise.  For the same reason the host refuses counts of steps that would raise
// 64 bits' own noise to the size of X (kMuonMaxGrowth).
//
// Rows of r are padded to kT tiles of 16 (1, 2, 4 or 8); a symmetric matrix is
// its tiles on and above the diagonal.  A wave's 16 x 16 result holds rows 4 v +
// lane / 16 (register v) of column lane % 16, and an operand's lane element lane
// % 16 of step lane / 16, so that a tile's registers are what it needs as either
// operand of its transpose.
//
// Bound by HBM: 8 bytes an element in the first pass, 22 in the last.  448
// matrices of 16 x 4096 (29 M elements): 58 us (4.0 TB/s) and 116-122 us (5.3-5.6
// TB/s, part of it from the last-level cache), the steps among them; of 64 x 4096 (117
// M): 297 us (3.2 TB/s), the steps 86 us, 540 us (4.8 TB/s), of 4096 x 64 643 us.  All
// adapters of a 7B model: r = 16 256 us, r = 64 1.30 ms, 0.95 at a large copy's rate.  Up
// to r = 64 the matrix instructions would take a third of these times; at r = 128 (100
// matrices of 128 x 4096, 52 M) they are half of them: 300, 234 and 442 us.  The steps
// of a matrix are one CU's work, and above 32 rows its 64-bit rate bounds them (15
// matrices: 64 rows 36 us, 74 rows 63, 100 rows 190, 128 rows 209, for 17 products each).
// Few matrices are a chain of latencies: one layer's 14 of r = 16 19 us.

#include <cmath>

#include "qn_device.h"
#include "qn_launch.h"

namespace qn {

namespace {

typedef double f64x4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = 4;

__device__ __forceinline__ f64x4_t mfma64(double a, double b, f64x4_t c) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

constexpr int upper_tiles(int t) { return t * (t + 1) / 2; }

// Number of tile (a, b), a <= b: column by column, so that the tiles of a smaller
// matrix are the first ones of a larger.
__host__ __device__ constexpr int upper_index(int a, int b) { return b * (b + 1) / 2 + a; }

__device__ __forceinline__ void upper_tile(int q, int& a, int& b) {
  b = 0;
  while (q > b) q -= ++b;
  a = q;
}

struct MuonArgs {
  float mu, one_minus_mu, decay, lr, eps;
  bool nesterov, rms;
  double ca, cb, cc;  // of a step
  int steps;
};

// The table's pointers as what they are: from a pointer that it finds in memory
// the compiler would make flat accesses, which count as LDS accesses too.
template <typename T>
using Global = __attribute__((address_space(1))) T*;

template <typename T>
__device__ __forceinline__ Global<T> global(T* p) {
  return (Global<T>)p;
}

// Element `lane` behind a wave's address: a scalar and 32 bits, which takes one
// register for all vectors of a lane (byte offsets below 2^32).
template <typename T>
__device__ __forceinline__ Global<T> lane_ptr(Global<T> p, uint32_t lane) {
  return (Global<T>)((Global<const char>)p + lane * static_cast<uint32_t>(sizeof(T)));
}

__device__ __forceinline__ float element(float x) { return x; }
__device__ __forceinline__ float element(uint16_t x) { return bf16_to_f32(x); }

// kN consecutive elements in memory, of which n exist; with kVec all or none of
// them do, and they are read and written as one vector.
template <bool kVec, int kN, typename T>
__device__ __forceinline__ void load_some(Global<const T> p, int n, float (&v)[kN]) {
  if constexpr (kVec && kN > 1) {
    typedef T vec_t __attribute__((ext_vector_type(kN)));
    vec_t w = vec_t(0);
    if (n > 0) w = *(Global<const vec_t>)p;
#pragma unroll
    for (int e = 0; e < kN; ++e) v[e] = element(w[e]);
  } else {
#pragma unroll
    for (int e = 0; e < kN; ++e) v[e] = e < n ? element(p[e]) : 0.0f;
  }
}

template <bool kVec, int kN>
__device__ __forceinline__ void store_some(Global<float> p, int n, const float (&v)[kN]) {
  if constexpr (kVec) {
    typedef float vec_t __attribute__((ext_vector_type(kN)));
    vec_t w;
#pragma unroll
    for (int e = 0; e < kN; ++e) w[e] = v[e];
    if (n > 0) *(Global<vec_t>)p = w;
  } else {
#pragma unroll
    for (int e = 0; e < kN; ++e)
      if (e < n) p[e] = v[e];
  }
}

template <bool kVec, int kN>
__device__ __forceinline__ void store_some(Global<uint16_t> p, int n, const float (&v)[kN]) {
  typedef uint32_t vec_t __attribute__((ext_vector_type(kN / 2)));
  vec_t w;
#pragma unroll
  for (int e = 0; e < kN / 2; ++e) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
  if constexpr (kVec) {
    if (n > 0) *(Global<vec_t>)p = w;
  } else {
#pragma unroll
    for (int e = 0; e < kN; ++e)
      if (e < n) p[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
  }
}

// The momentum and the update of n elements.
template <int n>
__device__ __forceinline__ void momentum(const MuonArgs& a, const float (&g)[n], float (&m)[n],
                                         float (&u)[n]) {
#pragma unroll
  for (int e = 0; e < n; ++e) {
    const float gs = g[e] * a.one_minus_mu;
    m[e] = fmaf(m[e], a.mu, gs);
    u[e] = a.nesterov ? fmaf(m[e], a.mu, gs) : m[e];
  }
}

// u u^T of a chunk of the long side, its batches dealt to the waves in turn (so
// that they read the same lines at about the same time: 430 -> 300 us for 448
// matrices of 64 x 4096).  The products' operands are loaded as they are needed,
// without LDS, a batch ahead: lane (li, lg) holds row 16 t + li of the short side;
// a wide matrix gives it 4 consecutive elements of the long side (4 steps, group
// lg's elements at 4 lg: any order that both operands share will do), a tall one a
// single one.
template <int kT, bool kTall, bool kVec, typename G>
__device__ __forceinline__ void gram_blocks(const MuonMatrix& mat, const MuonArgs& a, int start,
                                            int end, int wave, f64x4_t (&acc)[upper_tiles(kT)]) {
  constexpr int kN = kTall ? 1 : kT == 8 ? 2 : 4;  // elements of a load
  constexpr int kH = kT < 4 ? (kTall ? 16 : 4) / kT : kTall ? 2 : 1;  // loads of a row and batch
  constexpr int kBatch = 4 * kN * kH;              // of the long side
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int r = mat.r, len = static_cast<int>(mat.len);
  const Global<const G> g = global(static_cast<const G*>(mat.g));
  const Global<const float> m = global(static_cast<const float*>(mat.m));
  const uint32_t place = kTall ? static_cast<uint32_t>(lg * r + li)
                               : static_cast<uint32_t>(li) * static_cast<uint32_t>(len) + kN * lg;
  float gv[2][kT][kH][kN], mv[2][kT][kH][kN];
  auto load = [&](int n, int buf) {
    const int k0 = start + (wave + n * kWaves) * kBatch;
    // hidden from the compiler, which would keep and step a pointer for each load
    int64_t block = kTall ? static_cast<int64_t>(k0) * r : k0;
    asm volatile("" : "+s"(block));
#pragma unroll
    for (int h = 0; h < kH; ++h)
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        const int k = k0 + 4 * kN * h;
        const int64_t at = block + (kTall ? 4 * kN * h * r + 16 * t
                                          : static_cast<int64_t>(16 * t) * len + 4 * kN * h);
        const int n_in = 16 * t + li < r ? end - k - kN * lg : 0;
        load_some<kVec, kN, G>(lane_ptr(g + at, place), n_in, gv[buf][t][h]);
        load_some<kVec, kN, float>(lane_ptr(m + at, place), n_in, mv[buf][t][h]);
      }
  };
  auto multiply = [&](int buf) {
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      float u[kT][kN];
#pragma unroll
      for (int t = 0; t < kT; ++t) momentum(a, gv[buf][t][h], mv[buf][t][h], u[t]);
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        double f[kT];
#pragma unroll
        for (int t = 0; t < kT; ++t) f[t] = static_cast<double>(u[t][e]);
#pragma unroll
        for (int y = 0; y < kT; ++y)
          if (kT < 4 || 16 * y < r)
#pragma unroll
            for (int x = 0; x <= y; ++x)
              acc[upper_index(x, y)] = mfma64(f[x], f[y], acc[upper_index(x, y)]);
      }
    }
  };
  const int all = (end - start + kBatch - 1) / kBatch;
  const int batches = all > wave ? (all - wave + kWaves - 1) / kWaves : 0;
  if (batches > 0) load(0, 0);
  for (int n = 0; n < batches; n += 2) {
    if (n + 1 < batches) load(n + 1, 1);
    multiply(0);
    if (n + 2 < batches) load(n + 2, 0);
    if (n + 1 < batches) multiply(1);
  }
}

template <int kT, typename G>
__global__ __launch_bounds__(kThreads) void muon_gram_kernel(const MuonMatrix* __restrict__ mats,
                                                             const MuonChunk* __restrict__ chunks,
                                                             MuonArgs a, double* __restrict__ ws) {
  constexpr int kTiles = upper_tiles(kT);
  __shared__ f64x4_t s_acc[kWaves * kWaves * 64];  // [tile of the round][wave][lane]
  const MuonChunk c = chunks[blockIdx.x];
  const MuonMatrix mat = mats[c.matrix];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int start = static_cast<int>(c.index * mat.chunk);
  const int end = static_cast<int>(start + mat.chunk < mat.len ? start + mat.chunk : mat.len);
  f64x4_t acc[kTiles];
#pragma unroll
  for (int q = 0; q < kTiles; ++q) acc[q] = f64x4_t{0.0, 0.0, 0.0, 0.0};
  if (mat.tall)  // of single elements
    gram_blocks<kT, true, false, G>(mat, a, start, end, wave, acc);
  else if ((mat.len & 3) == 0)
    gram_blocks<kT, false, true, G>(mat, a, start, end, wave, acc);
  else
    gram_blocks<kT, false, false, G>(mat, a, start, end, wave, acc);
  // the waves' sums, 4 tiles at a time, one per wave; those that r reaches
  const int rows = (mat.r + 15) / 16, tiles = rows * (rows + 1) / 2;
  f64x4_t* part = reinterpret_cast<f64x4_t*>(ws + mat.part + c.index * (kTiles * 256));
#pragma unroll
  for (int q0 = 0; q0 < kTiles; q0 += kWaves) {
    if (kT >= 4 && q0 >= tiles) break;
    if (q0 > 0) __syncthreads();
#pragma unroll
    for (int q = q0; q < q0 + kWaves && q < kTiles; ++q)
      s_acc[((q - q0) * kWaves + wave) * 64 + lane] = acc[q];
    __syncthreads();
    if (q0 + wave < kTiles) {
      const f64x4_t* s = s_acc + wave * kWaves * 64 + lane;
      part[(q0 + wave) * 64 + lane] = ((s[0] + s[64]) + s[128]) + s[192];
    }
  }
}

// The steps on one matrix's S, a workgroup each: wave w holds the tiles w, w + W,
// ... of S, Q and T in registers (of the kN x kN that r reaches: 5 x 5 for r =
// 74), and products read their operands, two at a time, from LDS.  The diagonal
// tiles of S and Q go there by their upper halves, as the whole matrix does by its
// upper tiles: with the products' own lower halves, which rounding makes others, T
// mixed directions that u has with those that it has not (r = 64, u of rank one, 12
// steps: X off by 1.2 instead of 6e-6, 8 steps 2e-6 instead of 3e-11; T's and S Q's
// lower halves may stay).
constexpr int kStepPitch = 17, kStepTile = 16 * kStepPitch;  // doubles

template <int kN>
__device__ __forceinline__ f64x4_t tile_product(const double* x, const double* y, int a, int b,
                                                int li, int lg) {
  f64x4_t acc = f64x4_t{0.0, 0.0, 0.0, 0.0};
#pragma unroll(kN > 5 ? 2 : kN)
  for (int c = 0; c < kN; ++c) {
    // X(a, c)[li][4 s + lg] and Y(c, b)[4 s + lg][li], or the other half's
    const bool xu = a <= c, yu = c <= b;
    const double* px = x + upper_index(xu ? a : c, xu ? c : a) * kStepTile +
                       (xu ? li * kStepPitch + lg : lg * kStepPitch + li);
    const double* py = y + upper_index(yu ? c : b, yu ? b : c) * kStepTile +
                       (yu ? lg * kStepPitch + li : li * kStepPitch + lg);
    const int dx = xu ? 4 : 4 * kStepPitch, dy = yu ? 4 * kStepPitch : 4;
#pragma unroll
    for (int s = 0; s < 4; ++s) acc = mfma64(px[s * dx], py[s * dy], acc);
  }
  return acc;
}

// Place of T's element (i, j) among the operands of the last pass: step (j / 16,
// q) of row tile i / 16, 64 lanes each.  Lane (li, lg) multiplies its row with the
// element of u that it holds there, 4 q + lg of a wide matrix or 4 lg + q of a
// tall one, and a tall one's rows are turned likewise: result register v of lanes
// lg is row 4 lg + v.
template <int kT>
__device__ __forceinline__ int factor_place(bool tall, int i, int j) {
  const int a = i & 15, b = j & 15;
  const int li = tall ? 4 * (a & 3) + (a >> 2) : a;
  const int lg = tall ? b >> 2 : b & 3, q = tall ? b & 3 : b >> 2;
  return (((i >> 4) * kT + (j >> 4)) * 4 + q) * 64 + lg * 16 + li;
}

template <int kT, int kN, int kWavesOf>
__device__ __forceinline__ void tile_steps(const MuonMatrix& mat, const MuonArgs& a, double* ws,
                                           double* s_x, double* s_y, double* s_diag) {
  constexpr int kTiles = upper_tiles(kN), kOwn = (kTiles + kWavesOf - 1) / kWavesOf;
  const int t = threadIdx.x, lane = t & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  int ta[kOwn], tb[kOwn];
  bool have[kOwn];
  f64x4_t s[kOwn], q[kOwn], x[kOwn];
  // the chunks' sums, in their order
#pragma unroll
  for (int d = 0; d < kOwn; ++d) {
    const int n = wave + kWavesOf * d;
    have[d] = n < kTiles;
    upper_tile(have[d] ? n : 0, ta[d], tb[d]);
    const f64x4_t* part = reinterpret_cast<const f64x4_t*>(ws + mat.part) +
                          upper_index(ta[d], tb[d]) * 64 + lane;
    constexpr int kStride = upper_tiles(kT) * 64;
    f64x4_t sum = f64x4_t{0.0, 0.0, 0.0, 0.0};
    int i = 0;
    for (; i + 8 <= mat.chunks; i += 8) {
      f64x4_t v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = part[static_cast<int64_t>(i + e) * kStride];
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += v[e];
    }
    for (; i < mat.chunks; ++i) sum += part[static_cast<int64_t>(i) * kStride];
    s[d] = sum;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (have[d] && ta[d] == tb[d] && 4 * v + lg == li) s_diag[16 * ta[d] + li] = sum[v];
  }
  __syncthreads();
  double norm2 = 0.0;
#pragma unroll 8
  for (int i = 0; i < 16 * kN; ++i) norm2 += s_diag[i];
  const double inv = 1.0 / (sqrt(norm2) + static_cast<double>(a.eps));

  // (by_upper: of a diagonal tile the upper half, to both places)
  auto store = [&](double* to, const f64x4_t (&m)[kOwn], bool by_upper) {
#pragma unroll
    for (int d = 0; d < kOwn; ++d) {
      if (!have[d]) continue;
      double* tile = to + (wave + kWavesOf * d) * kStepTile;
      const bool diagonal = by_upper && ta[d] == tb[d];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int i = 4 * v + lg;
        if (!diagonal || i <= li) tile[i * kStepPitch + li] = m[d][v];
        if (diagonal && i < li) tile[li * kStepPitch + i] = m[d][v];
      }
    }
  };
  auto product = [&](f64x4_t (&to)[kOwn]) {
#pragma unroll
    for (int d = 0; d < kOwn; ++d)
      if (have[d]) to[d] = tile_product<kN>(s_x, s_y, ta[d], tb[d], li, lg);
  };
#pragma unroll
  for (int d = 0; d < kOwn; ++d) {
    s[d] *= inv * inv;
    x[d] = q[d] = s[d];
  }
  for (int n = 0; n < a.steps; ++n) {
    // Q = a I + b S + c S^2
    store(s_x, s, true);
    __syncthreads();
#pragma unroll
    for (int d = 0; d < kOwn; ++d) {
      if (!have[d]) continue;
      const f64x4_t s2 = tile_product<kN>(s_x, s_x, ta[d], tb[d], li, lg);
#pragma unroll
      for (int v = 0; v < 4; ++v)
        q[d][v] = a.cc * s2[v] + a.cb * s[d][v] +
                  (ta[d] == tb[d] && 4 * v + lg == li ? a.ca : 0.0);
    }
    store(s_y, q, true);
    __syncthreads();
    // T Q, and S Q Q unless this was the last step
    f64x4_t r[kOwn];
    if (n + 1 < a.steps) product(r);
    if (n == 0) {
#pragma unroll
      for (int d = 0; d < kOwn; ++d) x[d] = q[d];
    } else {
      __syncthreads();
      store(s_x, x, false);
      __syncthreads();
      product(x);
    }
    if (n + 1 < a.steps) {
      __syncthreads();
      store(s_x, r, false);
      __syncthreads();
      product(s);
      __syncthreads();
    }
  }
  // T / (|u| + eps) in the order of the last pass's operands
  double* out = ws + mat.factor;
#pragma unroll
  for (int d = 0; d < kOwn; ++d)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int i = 16 * ta[d] + 4 * v + lg, j = 16 * tb[d] + li;
      const double w = x[d][v] * inv;
      if (have[d] && i <= j) {
        out[factor_place<kT>(mat.tall, i, j)] = w;
        out[factor_place<kT>(mat.tall, j, i)] = w;
      }
    }
}

// Waves of a workgroup: one a tile, or of 8 x 8 a third as many.
template <int kT>
constexpr int kStepWaves = kT == 8 ? 12 : upper_tiles(kT);

template <int kT>
__global__ __launch_bounds__(64 * kStepWaves<kT>) void muon_steps_kernel(
    const MuonMatrix* __restrict__ mats, MuonArgs a, double* __restrict__ ws) {
  __shared__ __attribute__((aligned(16))) double s_x[upper_tiles(kT) * kStepTile];
  __shared__ __attribute__((aligned(16))) double s_y[upper_tiles(kT) * kStepTile];
  __shared__ double s_diag[16 * kT];
  const MuonMatrix mat = mats[blockIdx.x];
  constexpr int kW = kStepWaves<kT>;
  const int tiles = (mat.r + 15) / 16;  // more than kT / 2
  if constexpr (kT == 8) {
    if (tiles == 5) return tile_steps<kT, 5, kW>(mat, a, ws, s_x, s_y, s_diag);
    if (tiles == 6) return tile_steps<kT, 6, kW>(mat, a, ws, s_x, s_y, s_diag);
    if (tiles == 7) return tile_steps<kT, 7, kW>(mat, a, ws, s_x, s_y, s_diag);
  }
  if constexpr (kT == 4)
    if (tiles == 3) return tile_steps<kT, 3, kW>(mat, a, ws, s_x, s_y, s_diag);
  tile_steps<kT, kT, kW>(mat, a, ws, s_x, s_y, s_diag);
}

// The update of blocks of 16 kC of the long side, a wave each: u once more, times
// T, and into p.  A lane holds 4 kC elements of 16 rows, of a wide matrix as 4
// vectors along the long side (vector q: row 4 q + lg, columns kC li ..), of a tall
// one as kC vectors along the short one (vector c: columns 4 lg .. + 3 of row 16 c
// + li).  Step q and column tile c of the product take element c of vector q, or
// element q of vector c; rows of T are put in the order in which the results then
// lie in the same places, so that nothing moves between lanes.
// (Loads of the next block, and of p before the products, cost the registers of a
// resident wave: 100 -> 145 us for 448 matrices of 16 x 4096.)
template <int kT, int kC, int kWavesOf, bool kTall, bool kVec, typename G>
__device__ __forceinline__ void apply_blocks(const MuonMatrix& mat, const MuonArgs& a, float step,
                                             int start, int end, int wave, const double* s_w) {
  constexpr int kN = kTall ? 4 : kC, kX = kTall ? kC : 4;  // elements of a vector, vectors
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int r = mat.r, len = static_cast<int>(mat.len);
  const Global<const G> g = global(static_cast<const G*>(mat.g));
  const Global<float> m = global(mat.m), p = global(mat.p);
  const Global<uint16_t> p_bf16 = global(mat.p_bf16);
  uint32_t place[kX];  // of the lane's vectors behind a tile's first element
#pragma unroll
  for (int x = 0; x < kX; ++x)
    place[x] = kTall ? static_cast<uint32_t>((16 * x + li) * r + 4 * lg)
                     : static_cast<uint32_t>(4 * x + lg) * static_cast<uint32_t>(len) + kC * li;
  // a block's first element in tile t, and how many elements of vector x there are;
  // the block's place is hidden from the compiler, which would keep a pointer for
  // each vector and step all of them (128 registers)
  auto tile_at = [&](int64_t block, int t) {
    return block + (kTall ? 16 * t : static_cast<int64_t>(16 * t) * len);
  };
  auto count = [&](int k0, int t, int x) {
    if constexpr (kTall) return k0 + 16 * x + li < end ? r - 16 * t - 4 * lg : 0;
    return 16 * t + 4 * x + lg < r ? end - k0 - kC * li : 0;
  };
  float gv[2][kX][kN], mv[2][kX][kN];
  auto load = [&](int k0, int64_t block, int t) {
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      const int n = count(k0, t, x);
      load_some<kVec, kN, G>(lane_ptr(g + tile_at(block, t), place[x]), n, gv[t & 1][x]);
      load_some<kVec, kN, float>(lane_ptr((Global<const float>)m + tile_at(block, t), place[x]), n,
                                 mv[t & 1][x]);
    }
  };
  for (int k0 = start + wave * 16 * kC; k0 < end; k0 += kWavesOf * 16 * kC) {
    int64_t block = kTall ? static_cast<int64_t>(k0) * r : k0;
    asm volatile("" : "+s"(block));
    f64x4_t acc[kT][kC];
#pragma unroll
    for (int h = 0; h < kT; ++h)
#pragma unroll
      for (int c = 0; c < kC; ++c) acc[h][c] = f64x4_t{0.0, 0.0, 0.0, 0.0};
    // T's operands are read in every block anew: held over the loop, as they would
    // be if the compiler knew where they lie, they take 32 kT^2 registers
    int from = lane;
    asm volatile("" : "+v"(from));
    load(k0, block, 0);
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      if (kT >= 4 && 16 * t >= r) continue;
      if (t + 1 < kT) load(k0, block, t + 1);
      float u[kX][kN];
#pragma unroll
      for (int x = 0; x < kX; ++x) {
        momentum(a, gv[t & 1][x], mv[t & 1][x], u[x]);
        store_some<kVec>(lane_ptr(m + tile_at(block, t), place[x]), count(k0, t, x), mv[t & 1][x]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        double b[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) b[c] = static_cast<double>(kTall ? u[c][q] : u[q][c]);
#pragma unroll
        for (int h = 0; h < kT; ++h) {
          if (kT >= 4 && 16 * h >= r) continue;
          const double w = s_w[((h * kT + t) * 4 + q) * 64 + from];
#pragma unroll
          for (int c = 0; c < kC; ++c) acc[h][c] = mfma64(w, b[c], acc[h][c]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int h = 0; h < kT; ++h) {
      if (kT >= 4 && 16 * h >= r) continue;
      float pv[kX][kN];
#pragma unroll
      for (int x = 0; x < kX; ++x)
        load_some<kVec, kN, float>(lane_ptr((Global<const float>)p + tile_at(block, h), place[x]),
                                   count(k0, h, x), pv[x]);
#pragma unroll
      for (int x = 0; x < kX; ++x) {
        float (&v)[kN] = pv[x];
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const double o = kTall ? acc[h][x][e] : acc[h][e][x];
          v[e] = fmaf(-step, static_cast<float>(o), v[e] * a.decay);
        }
        const int n = count(k0, h, x);
        store_some<kVec>(lane_ptr(p + tile_at(block, h), place[x]), n, v);
        if (p_bf16) store_some<kVec>(lane_ptr(p_bf16 + tile_at(block, h), place[x]), n, v);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// Product of two symmetric 16 x 16 matrices that commute, in the order of the
// results: a register is what the instruction takes of either operand.
__device__ __forceinline__ f64x4_t tile_product(f64x4_t x, f64x4_t y) {
  f64x4_t acc = f64x4_t{0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int s = 0; s < 4; ++s) acc = mfma64(x[s], y[s], acc);
  return acc;
}

// The steps on one tile, in every workgroup that needs the result and in each of
// its waves alike, in registers: 17 products of 4 instructions, which costs less
// than a launch between the passes.  The chunks' sums are added a quarter per
// wave first.  T is multiplied from the left: what rounding mixes of u's directions
// into one that u has not grows like T there, ns[0]^n.  From the right, step n adds
// Q's rounding, grown by as much, times T's factor there (u of rank one, 12 steps: X
// off by 3e-4 instead of 1e-9).
__device__ __forceinline__ void one_tile_steps(const MuonMatrix& mat, const MuonArgs& a,
                                               const double* ws, int wave, double* s_w) {
  __shared__ f64x4_t s_sum[kWaves][64];
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const f64x4_t* part = reinterpret_cast<const f64x4_t*>(ws + mat.part) + lane;
  f64x4_t s = f64x4_t{0.0, 0.0, 0.0, 0.0};
#pragma unroll 8
  for (int i = wave; i < mat.chunks; i += kWaves) s += part[static_cast<int64_t>(i) * 64];
  s_sum[wave][lane] = s;
  __syncthreads();
  s = s_sum[0][lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) s += s_sum[w][lane];
  // lane (li, lg) holds the diagonal's li where lg = li % 4
  double norm2 = 0.0;
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (4 * v + lg == li) norm2 = s[v];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) norm2 += __shfl_xor(norm2, off, 64);
  const double inv = 1.0 / (sqrt(norm2) + static_cast<double>(a.eps));
  s *= inv * inv;
  f64x4_t x = s;
  for (int n = 0; n < a.steps; ++n) {
    f64x4_t q = a.cc * tile_product(s, s) + a.cb * s;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (4 * v + lg == li) q[v] += a.ca;
    x = n == 0 ? q : tile_product(q, x);
    s = tile_product(tile_product(s, q), q);
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) s_w[factor_place<1>(mat.tall, 4 * v + lg, li)] = x[v] * inv;
}

// 8 waves where T takes all of a CU's LDS but for one workgroup.
template <int kT>
constexpr int kApplyWaves = kT == 8 ? 8 : kWaves;

template <int kT, typename G>
__global__ __launch_bounds__(64 * kApplyWaves<kT>, kT <= 2 ? 4 : kT == 4 ? 3 : 2) void
muon_apply_kernel(const MuonMatrix* __restrict__ mats, const MuonChunk* __restrict__ chunks,
                  MuonArgs a, const double* __restrict__ ws) {
  __shared__ __attribute__((aligned(16))) double s_w[256 * kT * kT];
  const MuonChunk c = chunks[blockIdx.x];
  const MuonMatrix mat = mats[c.matrix];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int start = static_cast<int>(c.index * mat.span);
  const int end = static_cast<int>(start + mat.span < mat.len ? start + mat.span : mat.len);
  const double rows = static_cast<double>(mat.tall ? mat.len : mat.r);
  const double cols = static_cast<double>(mat.tall ? mat.r : mat.len);
  const double most = rows > cols ? rows : cols;
  const double f = a.rms ? 0.2 * sqrt(most) : rows > cols ? sqrt(rows / cols) : 1.0;
  const float step = static_cast<float>(static_cast<double>(a.lr) * f);
  if constexpr (kT == 1) {
    one_tile_steps(mat, a, ws, wave, s_w);
  } else {
    for (int i = threadIdx.x * 2; i < 256 * kT * kT; i += 128 * kApplyWaves<kT>)
      *reinterpret_cast<double2*>(s_w + i) =
          *reinterpret_cast<const double2*>(ws + mat.factor + i);
  }
  __syncthreads();
  constexpr int kC = kT == 1 ? 4 : 2, kW = kApplyWaves<kT>;
  if (mat.tall && (mat.r & 3) == 0)
    apply_blocks<kT, kC, kW, true, true, G>(mat, a, step, start, end, wave, s_w);
  else if (mat.tall)
    apply_blocks<kT, kC, kW, true, false, G>(mat, a, step, start, end, wave, s_w);
  else if ((mat.len & 3) == 0)
    apply_blocks<kT, kC, kW, false, true, G>(mat, a, step, start, end, wave, s_w);
  else
    apply_blocks<kT, kC, kW, false, false, G>(mat, a, step, start, end, wave, s_w);
}

template <int kT>
hipError_t launch_class(const MuonMatrix* mats, const MuonMatrix* of, int64_t matrices,
                        const MuonChunk* chunks, int64_t nchunks, int64_t nspans, bool bf16_grad,
                        const MuonArgs& a, double* ws, hipStream_t st) {
  if (matrices == 0) return hipSuccess;
  const dim3 grid(static_cast<uint32_t>(nchunks)), grid2(static_cast<uint32_t>(nspans));
  const MuonChunk* spans = chunks + nchunks;
  if (bf16_grad)
    hipLaunchKernelGGL((muon_gram_kernel<kT, uint16_t>), grid, dim3(kThreads), 0, st, mats, chunks,
                       a, ws);
  else
    hipLaunchKernelGGL((muon_gram_kernel<kT, float>), grid, dim3(kThreads), 0, st, mats, chunks, a,
                       ws);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if constexpr (kT > 1) {
    hipLaunchKernelGGL(muon_steps_kernel<kT>, dim3(static_cast<uint32_t>(matrices)),
                       dim3(64 * kStepWaves<kT>), 0, st, of, a, ws);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (bf16_grad)
    hipLaunchKernelGGL((muon_apply_kernel<kT, uint16_t>), grid2, dim3(64 * kApplyWaves<kT>), 0, st,
                       mats, spans, a, ws);
  else
    hipLaunchKernelGGL((muon_apply_kernel<kT, float>), grid2, dim3(64 * kApplyWaves<kT>), 0, st,
                       mats, spans, a, ws);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_muon(const MuonMatrix* mats, const MuonChunk* chunks, const MuonCounts& n,
                       bool bf16_grad, const MuonStep& h, void* ws, hipStream_t st) {
  MuonArgs a;
  a.mu = h.momentum;
  a.one_minus_mu = static_cast<float>(1.0 - static_cast<double>(h.momentum));
  a.decay = static_cast<float>(1.0 - static_cast<double>(h.lr) * static_cast<double>(h.weight_decay));
  a.lr = h.lr;
  a.eps = h.eps;
  a.ca = h.a, a.cb = h.b, a.cc = h.c;
  a.steps = h.steps;
  a.nesterov = h.nesterov;
  a.rms = h.rms;
  double* w = static_cast<double*>(ws);
  const MuonMatrix* of = mats;  // a chunk names its matrix from the table's start
  hipError_t e = hipSuccess;
  for (int k = 0; k < kMuonClasses && e == hipSuccess; ++k) {
    const int64_t m = n.matrices[k], c = n.chunks[k], s = n.spans[k];
    e = k == 0   ? launch_class<1>(mats, of, m, chunks, c, s, bf16_grad, a, w, st)
        : k == 1 ? launch_class<2>(mats, of, m, chunks, c, s, bf16_grad, a, w, st)
        : k == 2 ? launch_class<4>(mats, of, m, chunks, c, s, bf16_grad, a, w, st)
                 : launch_class<8>(mats, of, m, chunks, c, s, bf16_grad, a, w, st);
    of += m;
    chunks += c + s;
  }
  return e;
}

}  // namespace qn
