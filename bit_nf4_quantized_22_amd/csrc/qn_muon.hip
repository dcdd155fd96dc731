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
// be noise.
//
// Rows of r are padded to kT tiles of 16 (1, 2, 4 or 8); a symmetric matrix is
// its tiles on and above the diagonal.  A wave's 16 x 16 result holds rows 4 v +
// lane / 16 (register v) of column lane % 16, and an operand's lane element lane
// % 16 of step lane / 16, so that a tile's registers are what it needs as either
// operand of its transpose.

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

// Tile (row, column) number q of those on and above the diagonal.
template <int kT>
__device__ __forceinline__ void upper_tile(int q, int& a, int& b) {
  a = 0;
  while (q >= kT - a) q -= kT - a++;
  b = a + q;
}

struct MuonArgs {
  float mu, one_minus_mu, decay, lr;
  bool nesterov, rms;
};

// 4 consecutive elements in memory, of which n (at most 4) exist.
template <typename T>
__device__ __forceinline__ void load4(const T* p, int64_t n, bool vec, float (&v)[4]) {
  if (vec && n >= 4) {
    if constexpr (sizeof(T) == 4) {
      const float4 w = *reinterpret_cast<const float4*>(p);
      v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = 0.0f;
    if (e < n) {
      if constexpr (sizeof(T) == 4)
        v[e] = p[e];
      else
        v[e] = bf16_to_f32(p[e]);
    }
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, int64_t n, bool vec, const float (&v)[4]) {
  if (vec && n >= 4) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) {
      if constexpr (sizeof(T) == 4)
        p[e] = v[e];
      else
        p[e] = static_cast<uint16_t>(pack_bf16x2(v[e], 0.0f) & 0xFFFF);
    }
}

// How a workgroup's threads take a run of kLen elements of the long side, 4096
// in all: group j of a thread is 4 elements that lie together in memory, along
// the long side of a wide matrix and the short one of a tall one.
template <int kT, int kPitch>
struct Runs {
  static constexpr int kLen = 256 / kT, kGroups = 4;
  static_assert(kT * 16 * kLen == kThreads * kGroups * 4, "16 elements a thread");
  int64_t first[kGroups];   // the group's first element, of the run at 0
  int64_t behind[kGroups];  // elements of the run before it in its direction
  int place[kGroups][4];    // [short][long] in LDS, -1: no element of the matrix
  int64_t stride;           // of one element of the long side
  bool vec;                 // all groups can be read as vectors

  __device__ __forceinline__ explicit Runs(const MuonMatrix& mat) {
    const bool tall = mat.tall != 0;
    const int r = mat.r;
    vec = tall || (mat.len & 3) == 0;
    stride = tall ? r : 1;
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      const int q = j * kThreads + static_cast<int>(threadIdx.x);
      int i, k;
      if (tall) {
        k = q * 4 / r;
        i = q * 4 - k * r;
        first[j] = q * 4;
        behind[j] = q * 4;
      } else {
        i = q / (kLen / 4);
        k = q % (kLen / 4) * 4;
        first[j] = i * mat.len + k;
        behind[j] = k;
      }
      if (k >= kLen || i >= r) behind[j] = int64_t{1} << 60;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        place[j][e] = k < kLen && i < r ? i * kPitch + k : -1;
        i += tall ? 1 : 0;
        k += tall ? 0 : 1;
        if (tall && i == r) i = 0, ++k;
      }
    }
  }
  __device__ __forceinline__ int64_t at(int j, int64_t k0) const { return first[j] + k0 * stride; }
  // How many elements from group j's first on lie before `end` of the long side
  // (0 or less: none; more than 4 for whole groups).
  __device__ __forceinline__ int64_t left(int j, int64_t k0, int64_t end) const {
    return (end - k0) * stride - behind[j];
  }
};

// The momentum and the update of 4 elements.
__device__ __forceinline__ void momentum4(const MuonArgs& a, const float (&g)[4], float (&m)[4],
                                          float (&u)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float gs = g[e] * a.one_minus_mu;
    m[e] = fmaf(m[e], a.mu, gs);
    u[e] = a.nesterov ? fmaf(m[e], a.mu, gs) : m[e];
  }
}

// u u^T of one chunk of the long side.  Runs of it are staged in LDS [short]
// [long] as fp32, the next one on its way meanwhile; each wave multiplies a
// quarter of a run into all tiles, and the waves' sums are added in order.
template <int kT, typename G>
__global__ __launch_bounds__(kThreads) void muon_gram_kernel(const MuonMatrix* __restrict__ mats,
                                                             const MuonChunk* __restrict__ chunks,
                                                             MuonArgs a, double* __restrict__ ws) {
  constexpr int kLen = 256 / kT, kPitch = kLen + 4, kTiles = upper_tiles(kT);
  typedef Runs<kT, kPitch> R;
  constexpr int kFloats = kT * 16 * kPitch;
  __shared__ __attribute__((aligned(16))) float s_u[2 * kFloats];
  const MuonChunk c = chunks[blockIdx.x];
  const MuonMatrix mat = mats[c.matrix];
  const int t = threadIdx.x, lane = t & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t start = c.index * mat.chunk;
  const int64_t end = start + mat.chunk < mat.len ? start + mat.chunk : mat.len;
  const R runs(mat);
  const G* g = static_cast<const G*>(mat.g);
  for (int i = t; i < 2 * kFloats; i += kThreads) s_u[i] = 0.0f;
  float gv[R::kGroups][4], mv[R::kGroups][4];
  auto load = [&](int64_t k0) {
#pragma unroll
    for (int j = 0; j < R::kGroups; ++j) {
      const int64_t at = runs.at(j, k0), left = runs.left(j, k0, end);
      load4(g + at, left, runs.vec, gv[j]);
      load4(mat.m + at, left, runs.vec, mv[j]);
    }
  };
  f64x4_t acc[kTiles];
#pragma unroll
  for (int q = 0; q < kTiles; ++q) acc[q] = f64x4_t{0.0, 0.0, 0.0, 0.0};
  load(start);
  __syncthreads();
  int buf = 0;
  for (int64_t k0 = start; k0 < end; k0 += kLen, buf ^= 1) {
    float* su = s_u + buf * kFloats;
#pragma unroll
    for (int j = 0; j < R::kGroups; ++j) {
      float u[4];
      momentum4(a, gv[j], mv[j], u);
      const int64_t left = runs.left(j, k0, end);
#pragma unroll
      for (int e = 0; e < 4; ++e)  // past the chunk's end zeros, over what the buffer held
        if (runs.place[j][e] >= 0) su[runs.place[j][e]] = e < left ? u[e] : 0.0f;
    }
    __syncthreads();
    if (k0 + kLen < end) load(k0 + kLen);
    constexpr int kSteps = kLen / 4 / kWaves;
#pragma unroll 2
    for (int s = 0; s < kSteps; ++s) {
      double f[kT];
#pragma unroll
      for (int q = 0; q < kT; ++q)
        f[q] = static_cast<double>(su[(16 * q + li) * kPitch + 4 * (wave * kSteps + s) + lg]);
      int q = 0;
#pragma unroll
      for (int x = 0; x < kT; ++x)
#pragma unroll
        for (int y = x; y < kT; ++y, ++q) acc[q] = mfma64(f[x], f[y], acc[q]);
    }
  }
  // 4 tiles at a time, one per wave
  __syncthreads();
  f64x4_t* s_acc = reinterpret_cast<f64x4_t*>(s_u);  // [tile][wave][lane]
  static_assert(2 * kFloats * 4 >= kWaves * kWaves * 64 * 32, "the sums fit");
  f64x4_t* part = reinterpret_cast<f64x4_t*>(ws + mat.part + c.index * (kTiles * 256));
#pragma unroll
  for (int q0 = 0; q0 < kTiles; q0 += kWaves) {
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
// ... of S, Q and T in registers, and products read their operands, two at a
// time, from LDS.
template <int kT>
struct Steps {
  static constexpr int kTiles = upper_tiles(kT);
  static constexpr int kOwn = kT == 8 ? 3 : 1, kWavesOf = kTiles / kOwn;
  static constexpr int kPitch = 17, kTile = 16 * kPitch;  // doubles
  static_assert(kOwn * kWavesOf == kTiles, "tiles of a wave");
};

__device__ __forceinline__ int upper_index(int t, int a, int b) {
  return a * t - a * (a - 1) / 2 + (b - a);
}

template <int kT>
__device__ __forceinline__ f64x4_t tile_product(const double* x, const double* y, int a, int b,
                                                int li, int lg) {
  typedef Steps<kT> P;
  f64x4_t acc = f64x4_t{0.0, 0.0, 0.0, 0.0};
#pragma unroll(kT == 8 ? 2 : kT)
  for (int c = 0; c < kT; ++c) {
    // X(a, c)[li][4 s + lg] and Y(c, b)[4 s + lg][li], or the other half's
    const bool xu = a <= c, yu = c <= b;
    const double* px = x + upper_index(kT, xu ? a : c, xu ? c : a) * P::kTile +
                       (xu ? li * P::kPitch + lg : lg * P::kPitch + li);
    const double* py = y + upper_index(kT, yu ? c : b, yu ? b : c) * P::kTile +
                       (yu ? lg * P::kPitch + li : li * P::kPitch + lg);
    const int dx = xu ? 4 : 4 * P::kPitch, dy = yu ? 4 * P::kPitch : 4;
#pragma unroll
    for (int s = 0; s < 4; ++s) acc = mfma64(px[s * dx], py[s * dy], acc);
  }
  return acc;
}

template <int kT>
__global__ __launch_bounds__(64 * Steps<kT>::kWavesOf) void muon_steps_kernel(
    const MuonMatrix* __restrict__ mats, double ca, double cb, double cc, int steps, float eps,
    double* __restrict__ ws) {
  typedef Steps<kT> P;
  __shared__ __attribute__((aligned(16))) double s_x[P::kTiles * P::kTile];
  __shared__ __attribute__((aligned(16))) double s_y[P::kTiles * P::kTile];
  __shared__ double s_diag[16 * kT];
  const MuonMatrix mat = mats[blockIdx.x];
  const int t = threadIdx.x, lane = t & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  int ta[P::kOwn], tb[P::kOwn];
  f64x4_t s[P::kOwn], q[P::kOwn], x[P::kOwn];
  // the chunks' sums, in their order
#pragma unroll
  for (int d = 0; d < P::kOwn; ++d) {
    const int n = wave + P::kWavesOf * d;
    upper_tile<kT>(n, ta[d], tb[d]);
    const f64x4_t* part = reinterpret_cast<const f64x4_t*>(ws + mat.part) + n * 64 + lane;
    f64x4_t sum = f64x4_t{0.0, 0.0, 0.0, 0.0};
    int i = 0;
    for (; i + 8 <= mat.chunks; i += 8) {
      f64x4_t v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = part[static_cast<int64_t>(i + e) * (P::kTiles * 64)];
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += v[e];
    }
    for (; i < mat.chunks; ++i) sum += part[static_cast<int64_t>(i) * (P::kTiles * 64)];
    s[d] = sum;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (ta[d] == tb[d] && 4 * v + lg == li) s_diag[16 * ta[d] + li] = sum[v];
  }
  __syncthreads();
  double norm2 = 0.0;
#pragma unroll 8
  for (int i = 0; i < 16 * kT; ++i) norm2 += s_diag[i];
  const double inv = 1.0 / (sqrt(norm2) + static_cast<double>(eps));

  auto store = [&](double* to, const f64x4_t (&m)[P::kOwn]) {
#pragma unroll
    for (int d = 0; d < P::kOwn; ++d)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        to[(wave + P::kWavesOf * d) * P::kTile + (4 * v + lg) * P::kPitch + li] = m[d][v];
  };
  auto product = [&](f64x4_t (&to)[P::kOwn]) {
#pragma unroll
    for (int d = 0; d < P::kOwn; ++d) to[d] = tile_product<kT>(s_x, s_y, ta[d], tb[d], li, lg);
  };
#pragma unroll
  for (int d = 0; d < P::kOwn; ++d) s[d] *= inv * inv;
  for (int n = 0; n < steps; ++n) {
    // Q = a I + b S + c S^2
    store(s_x, s);
    __syncthreads();
#pragma unroll
    for (int d = 0; d < P::kOwn; ++d) {
      const f64x4_t s2 = tile_product<kT>(s_x, s_x, ta[d], tb[d], li, lg);
#pragma unroll
      for (int v = 0; v < 4; ++v)
        q[d][v] = cc * s2[v] + cb * s[d][v] +
                  (ta[d] == tb[d] && 4 * v + lg == li ? ca : 0.0);
    }
    store(s_y, q);
    __syncthreads();
    // T Q, and S Q Q unless this was the last step
    f64x4_t r[P::kOwn];
    if (n + 1 < steps) product(r);
    if (n == 0) {
#pragma unroll
      for (int d = 0; d < P::kOwn; ++d) x[d] = q[d];
    } else {
      __syncthreads();
      store(s_x, x);
      __syncthreads();
      product(x);
    }
    if (n + 1 < steps) {
      __syncthreads();
      store(s_x, r);
      __syncthreads();
      product(s);
      __syncthreads();
    }
  }
  // T / (|u| + eps) in the order of the last pass's operands: [16 rows][4 columns]
  // a lane each
  double* out = ws + mat.factor;
#pragma unroll
  for (int d = 0; d < P::kOwn; ++d)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int i = 16 * ta[d] + 4 * v + lg, j = 16 * tb[d] + li;
      const double w = x[d][v] * inv;
      out[((i >> 4) * (4 * kT) + (j >> 2)) * 64 + (j & 3) * 16 + (i & 15)] = w;
      out[((j >> 4) * (4 * kT) + (i >> 2)) * 64 + (i & 3) * 16 + (j & 15)] = w;
    }
}

// The update of one chunk: u once more, times T, and into p.
template <int kT, typename G>
__global__ __launch_bounds__(kThreads) void muon_apply_kernel(const MuonMatrix* __restrict__ mats,
                                                              const MuonChunk* __restrict__ chunks,
                                                              MuonArgs a,
                                                              const double* __restrict__ ws) {
  constexpr int kLen = 256 / kT, kPitch = kLen + 16;  // a step's 4 rows in different banks
  typedef Runs<kT, kPitch> R;
  // a wave's row tiles and column tiles of a run, 4 tiles in all
  constexpr int kRT = kT == 8 ? 2 : 1, kCT = 4 / kRT;
  constexpr int kRowGroups = kT / kRT, kSteps = 4 * kT;
  __shared__ __attribute__((aligned(16))) float s_u[kT * 16 * kPitch], s_o[kT * 16 * kPitch];
  const MuonChunk c = chunks[blockIdx.x];
  const MuonMatrix mat = mats[c.matrix];
  const int t = threadIdx.x, lane = t & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int row_tile = wave % kRowGroups, col_tile = wave / kRowGroups * kCT;
  const int64_t start = c.index * mat.chunk;
  const int64_t end = start + mat.chunk < mat.len ? start + mat.chunk : mat.len;
  const R runs(mat);
  const G* g = static_cast<const G*>(mat.g);
  for (int i = t; i < kT * 16 * kPitch; i += kThreads) s_u[i] = 0.0f;
  const double rows = static_cast<double>(mat.tall ? mat.len : mat.r);
  const double cols = static_cast<double>(mat.tall ? mat.r : mat.len);
  const double most = rows > cols ? rows : cols;
  const double f = a.rms ? 0.2 * sqrt(most) : rows > cols ? sqrt(rows / cols) : 1.0;
  const float step = static_cast<float>(static_cast<double>(a.lr) * f);
  double w[kRT][kSteps];
#pragma unroll
  for (int h = 0; h < kRT; ++h)
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      w[h][s] = ws[mat.factor + ((row_tile + h * kRowGroups) * kSteps + s) * 64 + lane];
  float gv[R::kGroups][4], mv[R::kGroups][4], pv[R::kGroups][4];
  auto load = [&](int64_t k0) {
#pragma unroll
    for (int j = 0; j < R::kGroups; ++j) {
      const int64_t at = runs.at(j, k0), left = runs.left(j, k0, end);
      load4(g + at, left, runs.vec, gv[j]);
      load4(mat.m + at, left, runs.vec, mv[j]);
    }
  };
  load(start);
  __syncthreads();
  for (int64_t k0 = start; k0 < end; k0 += kLen) {
#pragma unroll
    for (int j = 0; j < R::kGroups; ++j) {
      const int64_t at = runs.at(j, k0), left = runs.left(j, k0, end);
      float u[4];
      momentum4(a, gv[j], mv[j], u);
      store4(mat.m + at, left, runs.vec, mv[j]);
      load4(mat.p + at, left, runs.vec, pv[j]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (runs.place[j][e] >= 0) s_u[runs.place[j][e]] = e < left ? u[e] : 0.0f;
    }
    __syncthreads();
    if (k0 + kLen < end) load(k0 + kLen);
    f64x4_t acc[kRT][kCT];
#pragma unroll
    for (int h = 0; h < kRT; ++h)
#pragma unroll
      for (int q = 0; q < kCT; ++q) acc[h][q] = f64x4_t{0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      double b[kCT];
#pragma unroll
      for (int q = 0; q < kCT; ++q)
        b[q] = static_cast<double>(s_u[(4 * s + lg) * kPitch + 16 * (col_tile + q) + li]);
#pragma unroll
      for (int h = 0; h < kRT; ++h)
#pragma unroll
        for (int q = 0; q < kCT; ++q) acc[h][q] = mfma64(w[h][s], b[q], acc[h][q]);
    }
#pragma unroll
    for (int h = 0; h < kRT; ++h)
#pragma unroll
      for (int q = 0; q < kCT; ++q)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          s_o[(16 * (row_tile + h * kRowGroups) + 4 * v + lg) * kPitch + 16 * (col_tile + q) + li] =
              static_cast<float>(acc[h][q][v]);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < R::kGroups; ++j) {
      const int64_t at = runs.at(j, k0), left = runs.left(j, k0, end);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (runs.place[j][e] >= 0)
          pv[j][e] = fmaf(-step, s_o[runs.place[j][e]], pv[j][e] * a.decay);
      store4(mat.p + at, left, runs.vec, pv[j]);
      if (mat.p_bf16) store4(mat.p_bf16 + at, left, runs.vec, pv[j]);
    }
  }
}

template <int kT>
hipError_t launch_class(const MuonMatrix* mats, const MuonMatrix* of, int64_t matrices,
                        const MuonChunk* chunks, int64_t n, bool bf16_grad, const MuonStep& h, const MuonArgs& a, double* ws,
                        hipStream_t st) {
  if (n == 0) return hipSuccess;
  const dim3 grid(static_cast<uint32_t>(n));
  if (bf16_grad)
    hipLaunchKernelGGL((muon_gram_kernel<kT, uint16_t>), grid, dim3(kThreads), 0, st, mats, chunks,
                       a, ws);
  else
    hipLaunchKernelGGL((muon_gram_kernel<kT, float>), grid, dim3(kThreads), 0, st, mats, chunks, a,
                       ws);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  hipLaunchKernelGGL(muon_steps_kernel<kT>, dim3(static_cast<uint32_t>(matrices)),
                     dim3(64 * Steps<kT>::kWavesOf), 0, st, of, h.a, h.b, h.c, h.steps, h.eps, ws);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (bf16_grad)
    hipLaunchKernelGGL((muon_apply_kernel<kT, uint16_t>), grid, dim3(kThreads), 0, st, mats,
                       chunks, a, ws);
  else
    hipLaunchKernelGGL((muon_apply_kernel<kT, float>), grid, dim3(kThreads), 0, st, mats, chunks, a,
                       ws);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_muon(const MuonMatrix* mats, const MuonChunk* chunks,
                       const int64_t (&matrices)[kMuonClasses], const int64_t (&nchunks)[kMuonClasses],
                       bool bf16_grad, const MuonStep& h, void* ws, hipStream_t st) {
  MuonArgs a;
  a.mu = h.momentum;
  a.one_minus_mu = static_cast<float>(1.0 - static_cast<double>(h.momentum));
  a.decay = static_cast<float>(1.0 - static_cast<double>(h.lr) * static_cast<double>(h.weight_decay));
  a.lr = h.lr;
  a.nesterov = h.nesterov;
  a.rms = h.rms;
  double* w = static_cast<double*>(ws);
  int64_t m = 0, c = 0;
  hipError_t e = hipSuccess;
  for (int k = 0; k < kMuonClasses && e == hipSuccess; ++k) {
    // a chunk names its matrix from the table's start, the steps from the class's
    const MuonMatrix* of = mats + m;
    const int64_t n = matrices[k], nc = nchunks[k];
    e = k == 0   ? launch_class<1>(mats, of, n, chunks + c, nc, bf16_grad, h, a, w, st)
        : k == 1 ? launch_class<2>(mats, of, n, chunks + c, nc, bf16_grad, h, a, w, st)
        : k == 2 ? launch_class<4>(mats, of, n, chunks + c, nc, bf16_grad, h, a, w, st)
                 : launch_class<8>(mats, of, n, chunks + c, nc, bf16_grad, h, a, w, st);
    m += n, c += nc;
  }
  return e;
}

}  // namespace qn
