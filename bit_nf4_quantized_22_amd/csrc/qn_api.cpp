// C ABI of the QLoRA NF4 library: argument validation on the host, then the
// launches on the caller's stream.  See include/qlora_nf4.h for the contract
// of every entry point.

#include "qlora_nf4.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <vector>

#include "qn_launch.h"
#include "qn_tables.h"

namespace {

constexpr int kBlock = 64;
constexpr int kGroup = 256;
constexpr int kMaxRank = 128;
constexpr int64_t kGemvMaxM = 16;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

int hip_status(hipError_t e) { return e == hipSuccess ? QN_OK : QN_ERR_HIP; }

// The adapter of a call: r == 0, or A and B both NULL, is the frozen layer
// (rank 0); exactly one of A, B NULL with r > 0 is an error.
int adapter_rank(int32_t r, const void* A, const void* B, int32_t& r_eff) {
  r_eff = r;
  if (r > 0 && !A && !B) r_eff = 0;
  else if (r > 0 && (!A || !B)) return QN_ERR_NULL;
  return QN_OK;
}

// Validates a quantised weight for the linear ops and fills a view.
int check_weight(const qn_weight* w, qn::WeightView& v, bool linear) {
  if (!w || !w->packed) return QN_ERR_NULL;
  if (w->blocksize != kBlock || w->group != kGroup) return QN_ERR_UNSUPPORTED;
  if (w->quant_type != QN_NF4 && w->quant_type != QN_FP4) return QN_ERR_UNSUPPORTED;
  if (w->scale_type != QN_SCALE_U8 && w->scale_type != QN_SCALE_FP8 &&
      w->scale_type != QN_SCALE_CENTRED)
    return QN_ERR_UNSUPPORTED;
  if (!qn::tables(w->quant_type)) return QN_ERR_UNSUPPORTED;
  if (w->N < 0 || w->K < 0) return QN_ERR_SHAPE;
  if (linear && (w->N <= 0 || w->K <= 0 || w->N % 64 != 0 || w->K % 64 != 0)) return QN_ERR_SHAPE;
  const bool centred = w->qscale && w->scale_type == QN_SCALE_CENTRED;
  if (w->qscale) {
    if (!w->gscale || (centred && !w->offset)) return QN_ERR_NULL;
  } else if (!w->absmax) {
    return QN_ERR_NULL;
  }
  if (!aligned(w->packed, 16)) return QN_ERR_ALIGN;
  if ((w->gscale && !aligned(w->gscale, 4)) || (w->absmax && !aligned(w->absmax, 4)) ||
      (centred && !aligned(w->offset, 4)))
    return QN_ERR_ALIGN;
  v.packed = w->packed;
  v.qscale = w->qscale;
  v.gscale = w->gscale;
  v.absmax = w->qscale ? nullptr : w->absmax;
  v.N = w->N;
  v.K = w->K;
  v.quant_type = w->quant_type == QN_FP4 ? qn::kQuantFP4 : qn::kQuantNF4;
  v.l2 = !w->qscale ? qn::kL2Grid8
        : w->scale_type == QN_SCALE_FP8 ? qn::kL2E4M3
        : w->scale_type == QN_SCALE_CENTRED ? qn::kL2Centred
                                            : qn::kL2Grid8;
  v.mu = centred ? w->offset : nullptr;
  return QN_OK;
}

// fp32 partial sums of u (or t) over L-slices: up to kDecodeMaxSlices of
// them on the decode path, kWideMaxSlices for token batches.
size_t lora_part_bytes(int64_t M, int32_t r) {
  const size_t mr = static_cast<size_t>(M) * static_cast<size_t>(r);
  const size_t slices = M <= kGemvMaxM ? qn::kDecodeMaxSlices : qn::kWideMaxSlices;
  return round_up(mr * 4 * slices, 256);
}

// bf16(s u) or bf16(s t), the LoRA operand of the fused GEMM.
size_t lora_bf16_bytes(int64_t M, int32_t r) {
  return round_up(static_cast<size_t>(M) * static_cast<size_t>(r) * 2, 256);
}

// Forward workspace: the partial sums of u, then bf16(s u).
size_t fwd_ws(int64_t M, int32_t r) {
  if (r == 0 || M == 0) return 0;
  return lora_part_bytes(M, r) + lora_bf16_bytes(M, r);
}

// Backward workspace: the partial sums of t, then bf16(s t).
size_t bwd_ws(int64_t M, int64_t N, int32_t r) {
  (void)N;
  if (r == 0 || M == 0) return 0;
  return lora_part_bytes(M > kGemvMaxM ? M : kGemvMaxM + 1, r) + lora_bf16_bytes(M, r);
}

// Backward with dropout: the backward's workspace, then the fp32 product
// dy W [M, K] that the masked LoRA pass adds to before rounding once.
size_t bwd_drop_ws(int64_t M, int64_t N, int64_t K, int32_t r) {
  if (r == 0 || M == 0) return 0;
  return bwd_ws(M, N, r) + round_up(static_cast<size_t>(M) * static_cast<size_t>(K) * 4, 256);
}

// Gradient workspace: bf16 u and t (recomputed when not given), the
// partial sums of those projections, then the split-M partial sums.
size_t grads_ws(int64_t M, int64_t N, int64_t K, int32_t r) {
  if (r == 0) return 0;
  return 2 * lora_bf16_bytes(M, r) + lora_part_bytes(M > kGemvMaxM ? M : kGemvMaxM + 1, r) +
         round_up(qn::grads_workspace_bytes(M, N, K, r), 256);
}

int codebook(int qt, float out[16]) {
  if (!out) return QN_ERR_NULL;
  const qn::Tables* t = qn::tables(qt);
  if (!t) return QN_ERR_UNSUPPORTED;
  std::memcpy(out, t->q32, sizeof(t->q32));
  return QN_OK;
}

int quantize(int qt, const void* w, int32_t dtype, int64_t numel, int32_t blocksize,
             uint8_t* packed, float* absmax, void* stream) {
  if (blocksize != kBlock) return QN_ERR_UNSUPPORTED;
  if (dtype != QN_F32 && dtype != QN_BF16) return QN_ERR_UNSUPPORTED;
  if (numel < 0 || (numel & 1)) return QN_ERR_SHAPE;
  if (numel == 0) return QN_OK;
  if (!w || !packed || !absmax) return QN_ERR_NULL;
  if (!aligned(w, 16) || !aligned(packed, 16) || !aligned(absmax, 4)) return QN_ERR_ALIGN;
  if (!qn::tables(qt)) return QN_ERR_UNSUPPORTED;
  (void)hipGetLastError();
  return hip_status(
      qn::launch_quantize(w, dtype == QN_BF16, numel, qt, packed, absmax, as_stream(stream)));
}

int dq(bool fp8, const float* absmax, int64_t nblocks, int32_t group, uint8_t* qscale,
       float* gscale, void* stream) {
  if (group != kGroup) return QN_ERR_UNSUPPORTED;
  if (nblocks < 0) return QN_ERR_SHAPE;
  if (nblocks == 0) return QN_OK;
  if (!absmax || !qscale || !gscale) return QN_ERR_NULL;
  if (!aligned(absmax, 4) || !aligned(gscale, 4)) return QN_ERR_ALIGN;
  (void)hipGetLastError();
  return hip_status(qn::launch_dq(absmax, nblocks, fp8, qscale, gscale, as_stream(stream)));
}

// Forward with the LoRA-down input xa (x itself, or the dropped x).
int fwd_impl(const qn_weight* w, const qn_bf16* x, const qn_bf16* xa, int64_t M, const qn_bf16* A,
             const qn_bf16* B, int32_t r, float alpha, qn_bf16* y, qn_bf16* u_out, void* ws,
             size_t ws_bytes, void* stream, bool own_scratch = false) {
  qn::WeightView v;
  int st = check_weight(w, v, true);
  if (st != QN_OK) return st;
  if (M < 0 || r < 0) return QN_ERR_SHAPE;
  if (r > kMaxRank) return QN_ERR_UNSUPPORTED;
  if (M == 0 || w->N == 0) return QN_OK;
  if ((st = adapter_rank(r, A, B, r)) != QN_OK) return st;
  if (!x || !xa || !y) return QN_ERR_NULL;
  if (!aligned(x, 16) || !aligned(xa, 16) || !aligned(y, 2) || (r > 0 && (!aligned(A, 16) || !aligned(B, 2))) ||
      (u_out && !aligned(u_out, 2)))
    return QN_ERR_ALIGN;
  const size_t need = fwd_ws(M, r);
  if (own_scratch) {
    // the library's per-device array stands in for the caller's workspace
    if (need > qn::kScratchBytes) return QN_ERR_WORKSPACE;
    ws = nullptr;
    ws_bytes = 0;
    if (need > 0) {
      if (qn::scratch_address(as_stream(stream), &ws) != hipSuccess) return QN_ERR_HIP;
      ws_bytes = qn::kScratchBytes;
    }
  }
  if (need > 0 && (!ws || ws_bytes < need)) return QN_ERR_WORKSPACE;
  if (need > 0 && !aligned(ws, 16)) return QN_ERR_ALIGN;
  if (!qn::tables()) return QN_ERR_UNSUPPORTED;
  hipStream_t s = as_stream(stream);
  (void)hipGetLastError();
  const float scale = r > 0 ? alpha / static_cast<float>(r) : 0.0f;
  // u = x A^T as fp32 partial sums over L-slices, added up (in slice order)
  // by the GEMV or GEMM that applies the LoRA-up term
  float* u32 = static_cast<float*>(ws);
  const bool decode = M <= kGemvMaxM;
  const int ks = decode ? qn::skinny_splits(M, w->K, r, qn::gemv_threads(w->N, w->K))
                        : qn::skinny_wide_splits(M, w->K);
  // one token on a one-pass GEMV (and no dropout): the GEMV launch computes
  // u from the x it stages, and no LoRA-down launch runs
  const bool self_u = decode && r > 0 && xa == x && qn::gemv_self_u(v, static_cast<int>(M), r);
  if (r > 0 && !self_u) {
    if (qn::launch_skinny(xa, M, w->K, A, r, scale, u32, nullptr, nullptr, ks, s) != hipSuccess)
      return QN_ERR_HIP;
  }
  if (decode)
    return hip_status(qn::launch_gemv(v, x, static_cast<int>(M), u32, ks, B, r, scale, y,
                                      r > 0 ? u_out : nullptr, s, self_u ? A : nullptr));
  uint16_t* us = nullptr;
  if (r > 0) {
    us = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + lora_part_bytes(M, r));
    if (qn::launch_lora_reduce(u32, ks, M * r, scale, us, u_out, s) != hipSuccess) return QN_ERR_HIP;
  }
  return hip_status(qn::launch_gemm_fwd(v, x, M, us, B, r, y, s));
}

// Backward to the input; with drop, the LoRA term is masked by the dropout
// of the adapter's input (base GEMM alone, then dx += D * (s t A)).
int bwd_impl(const qn_weight* w, const qn_bf16* dy, int64_t M, const qn_bf16* A, const qn_bf16* B,
             int32_t r, float alpha, const float* drop_p, uint64_t seed, qn_bf16* dx,
             qn_bf16* t_out, void* ws, size_t ws_bytes, void* stream) {
  qn::WeightView v;
  int st = check_weight(w, v, true);
  if (st != QN_OK) return st;
  if (M < 0 || r < 0) return QN_ERR_SHAPE;
  if (r > kMaxRank) return QN_ERR_UNSUPPORTED;
  if (M == 0 || w->K == 0) return QN_OK;
  if ((st = adapter_rank(r, A, B, r)) != QN_OK) return st;
  if (!dy || !dx) return QN_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(dx, 2) || (r > 0 && (!aligned(A, 2) || !aligned(B, 2))) ||
      (t_out && !aligned(t_out, 2)))
    return QN_ERR_ALIGN;
  const size_t need = drop_p ? bwd_drop_ws(M, w->N, w->K, r) : bwd_ws(M, w->N, r);
  if (need > 0 && (!ws || ws_bytes < need)) return QN_ERR_WORKSPACE;
  if (need > 0 && !aligned(ws, 16)) return QN_ERR_ALIGN;
  if (!qn::tables()) return QN_ERR_UNSUPPORTED;
  hipStream_t s = as_stream(stream);
  (void)hipGetLastError();
  const float scale = r > 0 ? alpha / static_cast<float>(r) : 0.0f;
  // t = dy B as fp32 partial sums over N-slices (B read where it lies,
  // [N, r]), added up in slice order into bf16(s t), the GEMM's operand
  uint16_t* ts = nullptr;
  const int64_t mp = M > kGemvMaxM ? M : kGemvMaxM + 1;
  const int ks = qn::skinny_wide_splits(mp, w->N);
  if (r > 0) {
    char* base = static_cast<char*>(ws);
    float* t32 = reinterpret_cast<float*>(base);
    ts = reinterpret_cast<uint16_t*>(base + lora_part_bytes(mp, r));
    if (qn::launch_skinny(dy, M, w->N, B, r, scale, t32, nullptr, nullptr, ks, s, true) !=
        hipSuccess)
      return QN_ERR_HIP;
    if (qn::launch_lora_reduce(t32, ks, M * r, scale, ts, t_out, s) != hipSuccess) return QN_ERR_HIP;
  }
  if (!drop_p || r == 0) return hip_status(qn::launch_gemm_bwd(v, dy, M, ts, A, r, dx, s));
  float* base32 = reinterpret_cast<float*>(static_cast<char*>(ws) + bwd_ws(M, w->N, r));
  if (qn::launch_gemm_bwd(v, dy, M, nullptr, nullptr, 0, dx, s, base32) != hipSuccess)
    return QN_ERR_HIP;
  return hip_status(qn::launch_dx_lora_dropout(base32, dx, ts, A, M, w->K, r, *drop_p, seed, s));
}

// --- block-scaled FP8 ---------------------------------------------------

constexpr int64_t kFp8MaxDim = int64_t{1} << 23;  // 32-bit offsets within a tile

int64_t blocks128(int64_t n) { return (n + 127) / 128; }

int check_fp8_weight(const qn_fp8_weight* w, qn::Fp8View& v) {
  if (!w || !w->codes || !w->scale) return QN_ERR_NULL;
  if (w->N <= 0 || w->K <= 0 || w->N % 16 != 0 || w->K % 16 != 0 || w->N > kFp8MaxDim ||
      w->K > kFp8MaxDim)
    return QN_ERR_SHAPE;
  if (!aligned(w->codes, 16) || !aligned(w->scale, 4)) return QN_ERR_ALIGN;
  v = qn::Fp8View{w->codes, w->scale, w->N, w->K};
  return QN_OK;
}

// Rows of a batch: every launch over M rows of n columns has less than 2^32
// threads (at most 16 per run of 128 columns, 32 per row).
bool fp8_rows_ok(int64_t M, int64_t n) {
  return M >= 0 && M <= (int64_t{1} << 26) && M * blocks128(n) <= (int64_t{1} << 27);
}

// Workspace of a quantised batch [M, L] with `cols` output columns: codes, row
// scales, partial sums of the LoRA projection and its scaled bf16 sum in
// padded rows, partial sums of a split contraction.
struct Fp8Ws {
  size_t scale, part, act, split, total;
};

Fp8Ws fp8_ws(bool bwd, int64_t M, int64_t N, int64_t K, int32_t r) {
  Fp8Ws f{};
  if (M <= 0 || N <= 0 || K <= 0) return f;
  const int64_t L = bwd ? N : K, cols = bwd ? K : N;
  const size_t m = static_cast<size_t>(M);
  f.scale = round_up(m * static_cast<size_t>(L), 256);
  f.part = f.scale + round_up(m * static_cast<size_t>(blocks128(L)) * 4, 256);
  f.act = f.part;
  const int slices = !bwd && M <= qn::kFp8DecodeM ? qn::fp8_decode_slices(L)
                                                  : qn::fp8_project_slices(M, L);
  if (r > 0)
    f.act += round_up(m * static_cast<size_t>(r) * 4 * static_cast<size_t>(slices), 256);
  f.split = f.act;
  if (r > 0 && (bwd || M > qn::kFp8DecodeM))
    f.split += round_up(m * static_cast<size_t>(qn::fp8_lora_pitch(r)) * 2, 256);
  f.total = f.split;
  const int splits = bwd || !qn::fp8_few(M, N, K) ? qn::fp8_gemm_splits(M, cols, L) : 1;
  if (splits > 1)
    f.total += m * static_cast<size_t>(cols) * 4 * static_cast<size_t>(splits);
  return f;
}

// Forward (bwd false: in = x [M, K], down = A, up = B) or backward to the
// input (in = dy [M, N], down = B read in place, up = A).
int fp8_linear(bool bwd, const qn_fp8_weight* w, const qn_bf16* in, int64_t M, const qn_bf16* A,
               const qn_bf16* B, int32_t r, float alpha, qn_bf16* out, qn_bf16* low_out, void* ws,
               size_t ws_bytes, void* stream) {
  qn::Fp8View v;
  int st = check_fp8_weight(w, v);
  if (st != QN_OK) return st;
  const int64_t L = bwd ? v.N : v.K;
  if (r < 0 || !fp8_rows_ok(M, v.N) || !fp8_rows_ok(M, v.K)) return QN_ERR_SHAPE;
  if (r > kMaxRank) return QN_ERR_UNSUPPORTED;
  if (M == 0) return QN_OK;
  if ((st = adapter_rank(r, A, B, r)) != QN_OK) return st;
  if (!in || !out) return QN_ERR_NULL;
  if (!aligned(in, 16) || !aligned(out, 16) || (r > 0 && (!aligned(A, 2) || !aligned(B, 2))) ||
      !aligned(low_out, 2))
    return QN_ERR_ALIGN;
  const Fp8Ws f = fp8_ws(bwd, M, v.N, v.K, r);
  if (!ws || ws_bytes < f.total) return QN_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return QN_ERR_ALIGN;
  hipStream_t s = as_stream(stream);
  (void)hipGetLastError();
  const float ls = r > 0 ? alpha / static_cast<float>(r) : 0.0f;
  qn_bf16* low = r > 0 ? low_out : nullptr;
  uint8_t* codes = static_cast<uint8_t*>(ws);
  float* scale = reinterpret_cast<float*>(codes + f.scale);
  float* part = reinterpret_cast<float*>(codes + f.part);
  uint16_t* act = reinterpret_cast<uint16_t*>(codes + f.act);
  float* split = f.total > f.split ? reinterpret_cast<float*>(codes + f.split) : nullptr;
  if (!bwd && M == 1) {
    const bool own_u = qn::fp8_token_self_u(v, r);
    if (!own_u && qn::launch_fp8_decode_project(in, 1, L, A, r, nullptr, nullptr, part, s) !=
                      hipSuccess)
      return QN_ERR_HIP;
    return hip_status(qn::launch_fp8_token(v, in, A, own_u ? nullptr : part,
                                           qn::fp8_decode_slices(L), B, r, ls, out, low, s));
  }
  const bool decode = !bwd && M <= qn::kFp8DecodeM, few = !bwd && qn::fp8_few(M, v.N, v.K);
  const int m32 = static_cast<int>(few ? M : 0);
  hipError_t e = r == 0   ? qn::launch_fp8_quantize_rows(in, M, L, codes, scale, s)
                 : decode ? qn::launch_fp8_decode_project(in, m32, L, A, r, codes, scale, part, s)
                          : qn::launch_fp8_quantize_project(in, M, L, bwd ? B : A, r, bwd, codes,
                                                            scale, part, s);
  if (e != hipSuccess) return QN_ERR_HIP;
  if (r > 0 && !decode &&
      qn::launch_fp8_project_sum(part, qn::fp8_project_slices(M, L), M, r, ls, act, low, s) !=
          hipSuccess)
    return QN_ERR_HIP;
  if (few)
    return hip_status(qn::launch_fp8_decode(v, codes, scale, m32, part, qn::fp8_decode_slices(L),
                                            act, B, r, ls, out, low, s));
  return hip_status(qn::launch_fp8_gemm(v, codes, scale, M, act, bwd ? A : B, r, bwd, out, split, s));
}

// --- microscaled 4-bit ---------------------------------------------------

// 32-bit offsets within a tile; tiles of scales and blocks below 2^31.
constexpr int64_t kMxMaxDim = int64_t{1} << 23;

bool mx_size_ok(int64_t R, int64_t K) {
  return R >= 0 && K >= 0 && K % 32 == 0 && K <= kMxMaxDim && R <= (int64_t{1} << 26) &&
         qn::mx_tiles(R, 32) * qn::mx_tiles(K, 256) < (int64_t{1} << 24);
}

int check_mx_weight(const qn_mxfp4_weight* w, qn::MxView& v) {
  if (!w || !w->codes || !w->scale) return QN_ERR_NULL;
  if (w->N <= 0 || w->K <= 0 || w->N % 16 != 0 || w->N > kMxMaxDim || !mx_size_ok(w->N, w->K))
    return QN_ERR_SHAPE;
  if (!aligned(w->codes, 16) || !aligned(w->scale, 4)) return QN_ERR_ALIGN;
  v = qn::MxView{w->codes, w->scale, w->N, w->K};
  return QN_OK;
}

// Workspace of a batch [M, L]: codes and their scales, backward the turned
// weight and its scales, partial sums of the LoRA projection and its scaled
// sum in padded rows, partial sums of a split contraction.
struct MxWs {
  size_t scale, turned, tscale, part, act, split, total;
  int64_t bytes;  // of a row of codes
};

MxWs mx_ws(bool bwd, int64_t M, int64_t N, int64_t K, int32_t r) {
  MxWs f{};
  if (M <= 0 || N <= 0 || K <= 0) return f;
  const int64_t L = bwd ? N : K, cols = bwd ? K : N;
  const size_t m = static_cast<size_t>(M);
  f.bytes = bwd ? qn::mx_tiles(L, 128) * 128 : L / 2;
  auto tiles = [&](int64_t rows) {
    const int64_t n = bwd ? qn::mx_tiles(rows, 64) * qn::mx_tiles(L, 128)
                          : qn::mx_tiles(rows, 32) * qn::mx_tiles(L, 256);
    return static_cast<size_t>(n) * 256;
  };
  f.scale = round_up(m * static_cast<size_t>(f.bytes), 256);
  f.turned = f.scale + tiles(M);
  f.tscale = f.turned + (bwd ? static_cast<size_t>(K * f.bytes) : 0);
  f.tscale = round_up(f.tscale, 256);
  f.part = f.tscale + (bwd ? tiles(K) : 0);
  f.act = f.part;
  const int slices = !bwd && M <= qn::kFp8DecodeM ? qn::fp8_decode_slices(L)
                                                  : qn::fp8_project_slices(M, L);
  if (r > 0)
    f.act += round_up(m * static_cast<size_t>(r) * 4 * static_cast<size_t>(slices), 256);
  f.split = f.act;
  if (r > 0 && (bwd || M > qn::kFp8DecodeM))
    f.split += round_up(m * static_cast<size_t>(qn::fp8_lora_pitch(r)) * 2, 256);
  f.total = f.split;
  const int splits = bwd || !qn::mx_few(M, N, K) ? qn::mx_gemm_splits(M, cols, f.bytes, bwd) : 1;
  if (splits > 1)
    f.total += m * static_cast<size_t>(cols) * 4 * static_cast<size_t>(splits);
  return f;
}

// Batches of the products: the launches over M rows have less than 2^32
// threads, and the tiles of scales are counted in 32 bits.
bool mx_rows_ok(int64_t M, int64_t N, int64_t K) {
  return fp8_rows_ok(M, N) && fp8_rows_ok(M, K);
}

// Forward (bwd false: in = x [M, K], down = A, up = B) or backward to the
// input (in = dy [M, N], down = B read in place, up = A).
int mx_linear(bool bwd, const qn_mxfp4_weight* w, const qn_bf16* in, int64_t M, const qn_bf16* A,
              const qn_bf16* B, int32_t r, float alpha, qn_bf16* out, qn_bf16* low_out, void* ws,
              size_t ws_bytes, void* stream) {
  qn::MxView v;
  int st = check_mx_weight(w, v);
  if (st != QN_OK) return st;
  const int64_t L = bwd ? v.N : v.K;
  if (r < 0 || !mx_rows_ok(M, v.N, v.K)) return QN_ERR_SHAPE;
  if (r > kMaxRank) return QN_ERR_UNSUPPORTED;
  if (M == 0) return QN_OK;
  if ((st = adapter_rank(r, A, B, r)) != QN_OK) return st;
  if (!in || !out) return QN_ERR_NULL;
  if (!aligned(in, 16) || !aligned(out, 16) || (r > 0 && (!aligned(A, 2) || !aligned(B, 2))) ||
      !aligned(low_out, 2))
    return QN_ERR_ALIGN;
  const MxWs f = mx_ws(bwd, M, v.N, v.K, r);
  if (!ws || ws_bytes < f.total) return QN_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return QN_ERR_ALIGN;
  hipStream_t s = as_stream(stream);
  (void)hipGetLastError();
  const float ls = r > 0 ? alpha / static_cast<float>(r) : 0.0f;
  qn_bf16* low = r > 0 ? low_out : nullptr;
  uint8_t* codes = static_cast<uint8_t*>(ws);
  uint8_t* scale = codes + f.scale;
  float* part = reinterpret_cast<float*>(codes + f.part);
  uint16_t* act = reinterpret_cast<uint16_t*>(codes + f.act);
  float* split = f.total > f.split ? reinterpret_cast<float*>(codes + f.split) : nullptr;
  if (!bwd && M == 1) {
    const bool own_u = qn::mx_token_self_u(v, r);
    if (!own_u && qn::launch_mx_decode_project(in, 1, L, A, r, nullptr, nullptr, part, s) !=
                      hipSuccess)
      return QN_ERR_HIP;
    return hip_status(qn::launch_mx_token(v, in, A, own_u ? nullptr : part,
                                          qn::fp8_decode_slices(L), B, r, ls, out, low, s));
  }
  const bool decode = !bwd && M <= qn::kFp8DecodeM, few = !bwd && qn::mx_few(M, v.N, v.K);
  const int m32 = static_cast<int>(few ? M : 0);
  uint8_t* turned = codes + f.turned;
  uint8_t* tscale = codes + f.tscale;
  hipError_t e = r == 0   ? qn::launch_mx_rows(in, M, L, bwd, codes, scale, s)
                 : decode ? qn::launch_mx_decode_project(in, m32, L, A, r, codes, scale, part, s)
                 : bwd    ? qn::launch_mx_backward(v, in, M, B, r, codes, scale, part, turned,
                                                   tscale, s)
                          : qn::launch_mx_rows_project(in, M, L, A, r, codes, scale, part, s);
  if (e != hipSuccess) return QN_ERR_HIP;
  if (bwd && r == 0 && qn::launch_mx_turn(v, turned, tscale, s) != hipSuccess) return QN_ERR_HIP;
  if (r > 0 && !decode &&
      qn::launch_fp8_project_sum(part, qn::fp8_project_slices(M, L), M, r, ls, act, low, s) !=
          hipSuccess)
    return QN_ERR_HIP;
  if (few)
    return hip_status(qn::launch_mx_decode(v, codes, scale, m32, part, qn::fp8_decode_slices(L),
                                           act, B, r, ls, out, low, s));
  return hip_status(qn::launch_mx_gemm(bwd ? turned : v.codes, bwd ? tscale : v.scale, v.N, v.K,
                                       f.bytes, codes, scale, M, act, bwd ? A : B, r, bwd, out,
                                       split, s));
}

bool adamw_hyper_ok(float lr, float beta1, float beta2, float eps, float weight_decay) {
  return lr >= 0.0f && beta1 >= 0.0f && beta1 < 1.0f && beta2 >= 0.0f && beta2 < 1.0f &&
         eps > 0.0f && weight_decay >= 0.0f;
}

constexpr int64_t kAdamMaxChunks = int64_t{1} << 24;  // 256 threads each, under 2^32

// Chunks of the matrices of an AdamW table, -1 for sizes out of range.
int64_t adamw_chunks(const qn_adamw_tensor* t, int32_t count) {
  int64_t chunks = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].n < 0) return -1;
    if (t[i].n == 0) continue;
    chunks += (t[i].n - 1) / qn::kAdamChunk + 1;
    if (chunks >= kAdamMaxChunks) return -1;
  }
  return chunks;
}

size_t adamw_table_size(int64_t chunks) {
  return static_cast<size_t>(chunks) * sizeof(qn::AdamChunk);
}

// Memory that a step reads or writes.
struct Range {
  uintptr_t lo, hi;
  bool written;
};

// Whether one that is written overlaps any other.
bool ranges_overlap(std::vector<Range>& all) {
  std::sort(all.begin(), all.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t any = 0, written = 0;  // furthest end so far, of all and of the written
  for (const Range& r : all) {
    if (r.lo < (r.written ? any : written)) return true;
    any = std::max(any, r.hi);
    if (r.written) written = std::max(written, r.hi);
  }
  return false;
}

// Whether memory that a step writes overlaps anything else of the table.
bool adamw_overlaps(const qn_adamw_tensor* t, int32_t count, size_t grad_size, bool state8) {
  std::vector<Range> all;
  all.reserve(static_cast<size_t>(count) * 7);
  for (int32_t i = 0; i < count; ++i) {
    const size_t n = static_cast<size_t>(t[i].n);
    if (n == 0) continue;
    auto add = [&](const void* p, size_t bytes, bool written) {
      const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
      if (p) all.push_back({lo, lo + bytes, written});
    };
    const size_t state = n * (state8 ? 1 : 4);
    const size_t blocks = (n - 1) / qn::kAdamStateBlock + 1;
    add(t[i].p, n * 4, true);
    add(t[i].g, n * grad_size, false);
    add(t[i].m, state, true);
    add(t[i].v, state, true);
    add(t[i].p_bf16, n * 2, true);
    if (state8) {
      add(t[i].m_scale, blocks * 4, true);
      add(t[i].v_scale, blocks * 4, true);
    }
  }
  return ranges_overlap(all);
}

int check_adamw_plan(const qn_adamw_plan* plan, const void* table) {
  if (!plan) return QN_ERR_NULL;
  if ((plan->grad_dtype != QN_F32 && plan->grad_dtype != QN_BF16) ||
      (plan->state != QN_STATE_F32 && plan->state != QN_STATE_8BIT))
    return QN_ERR_UNSUPPORTED;
  if (plan->chunks < 0 || plan->chunks >= kAdamMaxChunks ||
      plan->bytes != static_cast<int64_t>(adamw_table_size(plan->chunks)))
    return QN_ERR_SHAPE;
  if (plan->chunks > 0 && !table) return QN_ERR_NULL;
  if (!aligned(table, 16)) return QN_ERR_ALIGN;
  return QN_OK;
}

const qn::AdamChunk* adamw_table(const void* table) {
  return static_cast<const qn::AdamChunk*>(table);
}

// --- Muon over many matrices ----------------------------------------------

// Chunks and spans of a table, at least one of each for a matrix: the first pass
// has 256 threads a chunk, the last up to 512 a span, the steps up to 768 a matrix,
// each launch less than 2^32.
constexpr int64_t kMuonMaxChunks = int64_t{1} << 23;
constexpr int64_t kMuonMaxLong = (int64_t{1} << 24) - 1;
// Bits by which the steps may raise what rounding leaves of S0's null directions,
// eigenvalues of 2^-53 or a little more of either sign: ns[0]^2 a step.  A negative
// one near 1 runs away (12 steps of 3.4445, 42.8 bits: X off by 1e-4 on singular
// values over 10 decades; 14 steps 2e-2, 16 steps 1e1, 20 steps NaN).
constexpr double kMuonMaxGrowth = 43.0;

// How a matrix is split; -1 for one that is not offered.
struct MuonShape {
  int64_t r, len;
  int cls, tiles;  // class, tiles of 16 of the short side
  int64_t run;     // kMuonRun of the class
  int64_t runs;    // of the long side
};

int muon_shape(const qn_muon_tensor& t, MuonShape& s) {
  if (t.rows < 0 || t.cols < 0) return QN_ERR_SHAPE;
  s.r = std::min(t.rows, t.cols);
  s.len = std::max(t.rows, t.cols);
  if (s.r == 0) {
    s.len = 0;
    return QN_OK;
  }
  if (s.r > kMaxRank) return QN_ERR_UNSUPPORTED;
  if (s.len > kMuonMaxLong) return QN_ERR_SHAPE;
  s.cls = 0;
  while (16 * qn::kMuonTiles[s.cls] < s.r) ++s.cls;
  s.tiles = qn::kMuonTiles[s.cls];
  s.run = qn::kMuonRun[s.cls];
  s.runs = qn::mx_tiles(s.len, s.run);
  return QN_OK;
}

// Runs of each chunk or span of a matrix, for about `target` workgroups of a pass
// in all, at most 256 chunks of a matrix, whose sums one workgroup adds; nearly
// equal ones.
int64_t muon_runs_of(const MuonShape& s, int64_t total_runs, int64_t target, bool capped) {
  const int64_t per = std::max({int64_t{1}, (total_runs + target - 1) / target,
                                capped ? (s.runs + 255) / 256 : int64_t{1}});
  const int64_t n = (s.runs + per - 1) / per;
  return (s.runs + n - 1) / n;
}

// The first pass leaves tiles (tiles + 1) KB of sums per chunk, which are few
// for up to 32 rows.  Targets, the chunks that they give, and times: a step on all
// adapters of a 7B model, r = 32, 2048 (2272) 596-601 us, 4096 (4192) 585-589, 8192
// (6656) 587-588, r = 16 the same within 1%; 448 matrices of 64 x 4096, 2048 (2240)
// first pass 287-297 us and steps 80-86, 8192 (7168) 296-301 and 104.
int64_t muon_chunk_runs(const MuonShape& s, int64_t total_runs) {
  return muon_runs_of(s, total_runs, s.tiles <= 2 ? 4096 : 2048, true);
}

// The last pass takes the steps' result once per workgroup, which for up to 16
// rows means to compute it.  Targets, the spans that they give, and times: a step on
// all adapters of a 7B model, r = 4, 3200 (2464) 114-118 us, 4096 (3552) 128, 8192
// (4928) 139, r = 16 261, 260 and 257; the pass on 448 matrices of 64 x 4096, 8192
// (7168) 541-643 us, 4096 (3584) 567-671, 2048 (2240) 616-714.
int64_t muon_span_runs(const MuonShape& s, int64_t total_runs) {
  return muon_runs_of(s, total_runs, s.tiles == 1 ? 3200 : 8192, false);
}

// Doubles of a chunk's sums and of a matrix's left factor, of `tiles` tiles of rows.
int64_t muon_sums(int64_t tiles) { return tiles * (tiles + 1) / 2 * 256; }
int64_t muon_factor(int64_t tiles) { return tiles * tiles * 256; }

// Matrices and chunks by class, table and workspace of `count` matrices.
int muon_sizes(const qn_muon_tensor* t, int32_t count, qn_muon_plan& plan, int64_t& total_runs) {
  plan = qn_muon_plan{};
  total_runs = 0;
  MuonShape s;
  for (int32_t i = 0; i < count; ++i) {
    if (int st = muon_shape(t[i], s); st != QN_OK) return st;
    if (s.len > 0) total_runs += s.runs;
  }
  int64_t matrices = 0, chunks = 0, doubles = 0;
  for (int32_t i = 0; i < count; ++i) {
    muon_shape(t[i], s);
    if (s.len == 0) continue;
    const int64_t n = qn::mx_tiles(s.runs, muon_chunk_runs(s, total_runs));
    const int64_t spans = qn::mx_tiles(s.runs, muon_span_runs(s, total_runs));
    ++plan.matrices[s.cls];
    plan.chunks[s.cls] += n;
    plan.spans[s.cls] += spans;
    ++matrices;
    chunks += n + spans;
    doubles += n * muon_sums(s.tiles) + muon_factor(s.tiles);
    if (chunks >= kMuonMaxChunks) return QN_ERR_SHAPE;
  }
  plan.bytes = matrices * static_cast<int64_t>(sizeof(qn::MuonMatrix)) +
               chunks * static_cast<int64_t>(sizeof(qn::MuonChunk));
  plan.ws_bytes = doubles * 8;
  return QN_OK;
}

int check_muon_plan(const qn_muon_plan* plan, const void* table) {
  if (!plan) return QN_ERR_NULL;
  if (plan->grad_dtype != QN_F32 && plan->grad_dtype != QN_BF16) return QN_ERR_UNSUPPORTED;
  int64_t matrices = 0, chunks = 0, doubles = 0;
  for (int k = 0; k < qn::kMuonClasses; ++k) {
    const int64_t m = plan->matrices[k], c = plan->chunks[k], s = plan->spans[k];
    if (m < 0 || c < m || c >= kMuonMaxChunks || s < m || s >= kMuonMaxChunks ||
        (m == 0 && (c > 0 || s > 0)))
      return QN_ERR_SHAPE;
    matrices += m;
    chunks += c + s;
    doubles += c * muon_sums(qn::kMuonTiles[k]) + m * muon_factor(qn::kMuonTiles[k]);
  }
  if (chunks >= kMuonMaxChunks || plan->ws_bytes != doubles * 8 ||
      plan->bytes != matrices * static_cast<int64_t>(sizeof(qn::MuonMatrix)) +
                         chunks * static_cast<int64_t>(sizeof(qn::MuonChunk)))
    return QN_ERR_SHAPE;
  if (chunks > 0 && !table) return QN_ERR_NULL;
  if (!aligned(table, 16)) return QN_ERR_ALIGN;
  return QN_OK;
}

}  // namespace

extern "C" {

const char* qn_status_string(int status) {
  switch (status) {
    case QN_OK: return "ok";
    case QN_ERR_NULL: return "a required pointer is NULL";
    case QN_ERR_SHAPE: return "invalid or inconsistent sizes";
    case QN_ERR_ALIGN: return "pointer not 16-byte aligned";
    case QN_ERR_UNSUPPORTED: return "unsupported parameter (blocksize 64, group 256, fp32/bf16 only)";
    case QN_ERR_WORKSPACE: return "workspace missing or too small";
    case QN_ERR_HIP: return "HIP launch failed";
    default: return "unknown status";
  }
}

int nf4_codebook(float out[16]) { return codebook(qn::kQuantNF4, out); }

int fp4_codebook(float out[16]) { return codebook(qn::kQuantFP4, out); }

int nf4_quantize(const void* w, int32_t dtype, int64_t numel, int32_t blocksize,
                 uint8_t* packed, float* absmax, void* stream) {
  return quantize(qn::kQuantNF4, w, dtype, numel, blocksize, packed, absmax, stream);
}

int fp4_quantize(const void* w, int32_t dtype, int64_t numel, int32_t blocksize,
                 uint8_t* packed, float* absmax, void* stream) {
  return quantize(qn::kQuantFP4, w, dtype, numel, blocksize, packed, absmax, stream);
}

int dq_quantize_scales(const float* absmax, int64_t nblocks, int32_t group, uint8_t* qscale,
                       float* gscale, void* stream) {
  return dq(false, absmax, nblocks, group, qscale, gscale, stream);
}

int dq_quantize_scales_fp8(const float* absmax, int64_t nblocks, int32_t group,
                           uint8_t* qscale, float* gscale, void* stream) {
  return dq(true, absmax, nblocks, group, qscale, gscale, stream);
}

int nf4_quantize_dq(const void* w, int32_t dtype, int64_t numel, int32_t blocksize, int32_t group,
                    int32_t quant_type, int32_t scale_type, uint8_t* packed, float* absmax,
                    uint8_t* qscale, float* gscale, void* stream) {
  if (blocksize != kBlock || group != kGroup) return QN_ERR_UNSUPPORTED;
  if (dtype != QN_F32 && dtype != QN_BF16) return QN_ERR_UNSUPPORTED;
  if (quant_type != QN_NF4 && quant_type != QN_FP4) return QN_ERR_UNSUPPORTED;
  if (scale_type != QN_SCALE_U8 && scale_type != QN_SCALE_FP8) return QN_ERR_UNSUPPORTED;
  if (numel < 0 || (numel & 1)) return QN_ERR_SHAPE;
  if (numel == 0) return QN_OK;
  if (!w || !packed || !qscale || !gscale) return QN_ERR_NULL;
  if (!aligned(w, 16) || !aligned(packed, 16) || !aligned(gscale, 4) ||
      (absmax && !aligned(absmax, 4)))
    return QN_ERR_ALIGN;
  const int qt = quant_type == QN_FP4 ? qn::kQuantFP4 : qn::kQuantNF4;
  if (!qn::tables(qt)) return QN_ERR_UNSUPPORTED;
  (void)hipGetLastError();
  return hip_status(qn::launch_quantize_dq(w, dtype == QN_BF16, numel, qt,
                                           scale_type == QN_SCALE_FP8, packed, absmax, qscale,
                                           gscale, as_stream(stream)));
}

int nf4_quantize_dq_batch(int32_t n, const void* const* w, const int64_t* numel, int32_t dtype,
                          int32_t blocksize, int32_t group, int32_t quant_type,
                          int32_t scale_type, uint8_t* const* packed, float* const* absmax,
                          uint8_t* const* qscale, float* const* gscale, void* stream) {
  if (blocksize != kBlock || group != kGroup) return QN_ERR_UNSUPPORTED;
  if (dtype != QN_F32 && dtype != QN_BF16) return QN_ERR_UNSUPPORTED;
  if (quant_type != QN_NF4 && quant_type != QN_FP4) return QN_ERR_UNSUPPORTED;
  if (scale_type != QN_SCALE_U8 && scale_type != QN_SCALE_FP8) return QN_ERR_UNSUPPORTED;
  if (n < 0 || n > qn::kQdqMaxBatch) return QN_ERR_SHAPE;
  if (n == 0) return QN_OK;
  if (!w || !numel || !packed || !qscale || !gscale) return QN_ERR_NULL;
  qn::QdqBatch b{};
  const int64_t per = static_cast<int64_t>(kBlock) * kGroup;  // weights per group
  int64_t groups = 0;
  for (int i = 0; i < n; ++i) {
    const int64_t m = numel[i];
    if (m < 0 || (m & 1)) return QN_ERR_SHAPE;
    if (m > 0) {
      float* am = absmax ? absmax[i] : nullptr;
      if (!w[i] || !packed[i] || !qscale[i] || !gscale[i]) return QN_ERR_NULL;
      if (!aligned(w[i], 16) || !aligned(packed[i], 16) || !aligned(gscale[i], 4) ||
          (am && !aligned(am, 4)))
        return QN_ERR_ALIGN;
      b.w[b.n] = w[i];
      b.numel[b.n] = m;
      b.packed[b.n] = packed[i];
      b.absmax[b.n] = am;
      b.qscale[b.n] = qscale[i];
      b.gscale[b.n] = gscale[i];
      groups += (m + per - 1) / per;
      if (groups > INT32_MAX) return QN_ERR_SHAPE;
      b.gend[b.n] = static_cast<uint32_t>(groups);
      ++b.n;
    }
  }
  if (b.n == 0) return QN_OK;
  const int qt = quant_type == QN_FP4 ? qn::kQuantFP4 : qn::kQuantNF4;
  if (!qn::tables(qt)) return QN_ERR_UNSUPPORTED;
  (void)hipGetLastError();
  return hip_status(qn::launch_quantize_dq_batch(b, dtype == QN_BF16, qt,
                                                 scale_type == QN_SCALE_FP8, as_stream(stream)));
}

int dq_quantize_scales_centred(const float* absmax, int64_t nblocks, int32_t group,
                               uint8_t* qscale, float* gscale, float* offset, void* stream) {
  if (group != kGroup) return QN_ERR_UNSUPPORTED;
  if (nblocks < 0) return QN_ERR_SHAPE;
  if (nblocks == 0) return QN_OK;
  if (!absmax || !qscale || !gscale || !offset) return QN_ERR_NULL;
  if (!aligned(absmax, 4) || !aligned(gscale, 4) || !aligned(offset, 4)) return QN_ERR_ALIGN;
  (void)hipGetLastError();
  return hip_status(
      qn::launch_dq_centred(absmax, nblocks, qscale, gscale, offset, as_stream(stream)));
}

int nf4_dequant(const qn_weight* w, int32_t out_dtype, void* out, void* stream) {
  qn::WeightView v;
  int st = check_weight(w, v, false);
  if (st != QN_OK) return st;
  if (out_dtype != QN_F32 && out_dtype != QN_BF16) return QN_ERR_UNSUPPORTED;
  if ((w->N * w->K) % 32 != 0) return QN_ERR_SHAPE;
  if (w->N * w->K == 0) return QN_OK;
  if (!out) return QN_ERR_NULL;
  if (!aligned(out, 16)) return QN_ERR_ALIGN;
  if (!qn::tables()) return QN_ERR_UNSUPPORTED;
  (void)hipGetLastError();
  return hip_status(qn::launch_dequant(v, out_dtype == QN_BF16, out, as_stream(stream)));
}

size_t qn_workspace_bytes(int32_t op, int64_t M, int64_t N, int64_t K, int32_t r) {
  if (M < 0 || N < 0 || K < 0 || r < 0 || r > kMaxRank) return 0;
  switch (op) {
    case QN_OP_FWD: return fwd_ws(M, r);
    case QN_OP_BWD_DX: return bwd_ws(M, N, r);
    case QN_OP_LORA_GRADS: return grads_ws(M, N, K, r);
    case QN_OP_BWD_DX_DROPOUT: return bwd_drop_ws(M, N, K, r);
    case QN_OP_FP8_FWD: return fp8_ws(false, M, N, K, r).total;
    case QN_OP_FP8_BWD_DX: return fp8_ws(true, M, N, K, r).total;
    case QN_OP_MXFP4_FWD: return mx_ws(false, M, N, K, r).total;
    case QN_OP_MXFP4_BWD_DX: return mx_ws(true, M, N, K, r).total;
    default: return 0;
  }
}

int qlora_linear_fwd(const qn_weight* w, const qn_bf16* x, int64_t M, const qn_bf16* A,
                     const qn_bf16* B, int32_t r, float alpha, qn_bf16* y, qn_bf16* u_out,
                     void* ws, size_t ws_bytes, void* stream) {
  return fwd_impl(w, x, x, M, A, B, r, alpha, y, u_out, ws, ws_bytes, stream);
}

int qn_hbm_read_probe(const void* buf, int64_t bytes, uint32_t* sink, void* stream) {
  if (bytes < 0 || bytes % 16 != 0) return QN_ERR_SHAPE;
  if (bytes == 0) return QN_OK;
  if (!buf || !sink) return QN_ERR_NULL;
  if (!aligned(buf, 16) || !aligned(sink, 4)) return QN_ERR_ALIGN;
  (void)hipGetLastError();
  return hip_status(qn::launch_read_probe(buf, bytes, sink, as_stream(stream)));
}

int qlora_linear_fwd_noalloc(const qn_weight* w, const qn_bf16* x, int64_t M, const qn_bf16* A,
                             const qn_bf16* B, int32_t r, float alpha, qn_bf16* y,
                             qn_bf16* u_out, void* stream) {
  return fwd_impl(w, x, x, M, A, B, r, alpha, y, u_out, nullptr, 0, stream, true);
}

int qlora_linear_fwd_dropout(const qn_weight* w, const qn_bf16* x, const qn_bf16* x_drop,
                             int64_t M, const qn_bf16* A, const qn_bf16* B, int32_t r,
                             float alpha, qn_bf16* y, qn_bf16* u_out, void* ws, size_t ws_bytes,
                             void* stream) {
  return fwd_impl(w, x, x_drop, M, A, B, r, alpha, y, u_out, ws, ws_bytes, stream);
}

int qlora_linear_bwd_dx(const qn_weight* w, const qn_bf16* dy, int64_t M, const qn_bf16* A,
                        const qn_bf16* B, int32_t r, float alpha, qn_bf16* dx, qn_bf16* t_out,
                        void* ws, size_t ws_bytes, void* stream) {
  return bwd_impl(w, dy, M, A, B, r, alpha, nullptr, 0, dx, t_out, ws, ws_bytes, stream);
}

int qlora_linear_bwd_dx_dropout(const qn_weight* w, const qn_bf16* dy, int64_t M,
                                const qn_bf16* A, const qn_bf16* B, int32_t r, float alpha,
                                float p, uint64_t seed, qn_bf16* dx, qn_bf16* t_out, void* ws,
                                size_t ws_bytes, void* stream) {
  if (!(p >= 0.0f && p < 1.0f)) return QN_ERR_SHAPE;
  return bwd_impl(w, dy, M, A, B, r, alpha, &p, seed, dx, t_out, ws, ws_bytes, stream);
}

int lora_dropout(const qn_bf16* x, int64_t M, int64_t K, float p, uint64_t seed, qn_bf16* x_drop,
                 void* stream) {
  if (M < 0 || K < 0 || K % 8 != 0 || !(p >= 0.0f && p < 1.0f)) return QN_ERR_SHAPE;
  if (M == 0 || K == 0) return QN_OK;
  if (!x || !x_drop) return QN_ERR_NULL;
  if (!aligned(x, 16) || !aligned(x_drop, 16)) return QN_ERR_ALIGN;
  (void)hipGetLastError();
  return hip_status(qn::launch_dropout(x, M, K, p, seed, x_drop, as_stream(stream)));
}

int qlora_merge(const qn_weight* w, const qn_bf16* A, const qn_bf16* B, int32_t r, float alpha,
                qn_bf16* out, void* stream) {
  qn::WeightView v;
  int st = check_weight(w, v, true);
  if (st != QN_OK) return st;
  if (r < 0) return QN_ERR_SHAPE;
  if (r > kMaxRank) return QN_ERR_UNSUPPORTED;
  if ((st = adapter_rank(r, A, B, r)) != QN_OK) return st;
  if (!out) return QN_ERR_NULL;
  if (!aligned(out, 16) || (r > 0 && (!aligned(A, 2) || !aligned(B, 2)))) return QN_ERR_ALIGN;
  if (!qn::tables()) return QN_ERR_UNSUPPORTED;
  (void)hipGetLastError();
  const float scale = r > 0 ? alpha / static_cast<float>(r) : 0.0f;
  return hip_status(qn::launch_merge(v, A, B, r, scale, out, as_stream(stream)));
}

int lora_adamw_step(float* p, const float* g, float* m, float* v, qn_bf16* p_bf16, int64_t n,
                    float lr, float beta1, float beta2, float eps, float weight_decay, int32_t step,
                    void* stream) {
  if (n < 0 || step < 1) return QN_ERR_SHAPE;
  if (n == 0) return QN_OK;
  if (!p || !g || !m || !v) return QN_ERR_NULL;
  if (!aligned(p, 16) || !aligned(g, 16) || !aligned(m, 16) || !aligned(v, 16) ||
      (p_bf16 && !aligned(p_bf16, 8)))
    return QN_ERR_ALIGN;
  if (!adamw_hyper_ok(lr, beta1, beta2, eps, weight_decay)) return QN_ERR_SHAPE;
  (void)hipGetLastError();
  return hip_status(qn::launch_adamw(p, g, m, v, p_bf16, n, lr, beta1, beta2, eps, weight_decay,
                                     step, as_stream(stream)));
}

int fp8_quantize_blocks(const void* w, int32_t dtype, int64_t N, int64_t K, uint8_t* codes,
                        float* scale, void* stream) {
  if (dtype != QN_F32 && dtype != QN_BF16) return QN_ERR_UNSUPPORTED;
  if (N < 0 || K < 0 || N % 16 != 0 || K % 16 != 0 || N > kFp8MaxDim || K > kFp8MaxDim ||
      blocks128(N) * blocks128(K) >= (int64_t{1} << 24))
    return QN_ERR_SHAPE;
  if (N == 0 || K == 0) return QN_OK;
  if (!w || !codes || !scale) return QN_ERR_NULL;
  if (!aligned(w, 16) || !aligned(codes, 16) || !aligned(scale, 4)) return QN_ERR_ALIGN;
  (void)hipGetLastError();
  return hip_status(qn::launch_fp8_quantize_blocks(w, dtype == QN_BF16, N, K, codes, scale,
                                                   as_stream(stream)));
}

int fp8_quantize_rows(const qn_bf16* x, int64_t M, int64_t K, uint8_t* codes, float* scale,
                      void* stream) {
  if (K < 0 || K % 16 != 0 || K > kFp8MaxDim || !fp8_rows_ok(M, K)) return QN_ERR_SHAPE;
  if (M == 0 || K == 0) return QN_OK;
  if (!x || !codes || !scale) return QN_ERR_NULL;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scale, 4)) return QN_ERR_ALIGN;
  (void)hipGetLastError();
  return hip_status(qn::launch_fp8_quantize_rows(x, M, K, codes, scale, as_stream(stream)));
}

int fp8_dequant(const qn_fp8_weight* w, int32_t out_dtype, void* out, void* stream) {
  qn::Fp8View v;
  if (int st = check_fp8_weight(w, v); st != QN_OK) return st;
  if (out_dtype != QN_F32 && out_dtype != QN_BF16) return QN_ERR_UNSUPPORTED;
  if (v.N * v.K / 16 > (int64_t{1} << 31)) return QN_ERR_SHAPE;
  if (!out) return QN_ERR_NULL;
  if (!aligned(out, 16)) return QN_ERR_ALIGN;
  (void)hipGetLastError();
  return hip_status(qn::launch_fp8_dequant(v, out_dtype == QN_BF16, out, as_stream(stream)));
}

int fp8_matmul(const qn_fp8_weight* w, const uint8_t* x, const float* xscale, int64_t M,
               int32_t transposed, qn_bf16* out, void* ws, size_t ws_bytes, void* stream) {
  qn::Fp8View v;
  if (int st = check_fp8_weight(w, v); st != QN_OK) return st;
  if (transposed != 0 && transposed != 1) return QN_ERR_UNSUPPORTED;
  if (!fp8_rows_ok(M, v.N) || !fp8_rows_ok(M, v.K)) return QN_ERR_SHAPE;
  if (M == 0) return QN_OK;
  if (!x || !xscale || !out) return QN_ERR_NULL;
  if (!aligned(x, 16) || !aligned(xscale, 4) || !aligned(out, 16)) return QN_ERR_ALIGN;
  const Fp8Ws f = fp8_ws(transposed == 1, M, v.N, v.K, 0);
  if (!ws || ws_bytes < f.total) return QN_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return QN_ERR_ALIGN;
  float* split =
      f.total > f.split ? reinterpret_cast<float*>(static_cast<char*>(ws) + f.split) : nullptr;
  (void)hipGetLastError();
  hipStream_t s = as_stream(stream);
  if (!transposed && qn::fp8_few(M, v.N, v.K))
    return hip_status(qn::launch_fp8_decode(v, x, xscale, static_cast<int>(M), nullptr, 0, nullptr,
                                            nullptr, 0, 0.0f, out, nullptr, s));
  return hip_status(
      qn::launch_fp8_gemm(v, x, xscale, M, nullptr, nullptr, 0, transposed == 1, out, split, s));
}

int fp8_linear_fwd(const qn_fp8_weight* w, const qn_bf16* x, int64_t M, const qn_bf16* A,
                   const qn_bf16* B, int32_t r, float alpha, qn_bf16* y, qn_bf16* u_out, void* ws,
                   size_t ws_bytes, void* stream) {
  return fp8_linear(false, w, x, M, A, B, r, alpha, y, u_out, ws, ws_bytes, stream);
}

int fp8_linear_bwd_dx(const qn_fp8_weight* w, const qn_bf16* dy, int64_t M, const qn_bf16* A,
                      const qn_bf16* B, int32_t r, float alpha, qn_bf16* dx, qn_bf16* t_out,
                      void* ws, size_t ws_bytes, void* stream) {
  return fp8_linear(true, w, dy, M, A, B, r, alpha, dx, t_out, ws, ws_bytes, stream);
}

size_t mxfp4_scale_bytes(int64_t R, int64_t K) {
  if (!mx_size_ok(R, K)) return 0;
  return static_cast<size_t>(qn::mx_tiles(R, 32) * qn::mx_tiles(K, 256)) * 256;
}

int mxfp4_quantize(const void* x, int32_t dtype, int64_t R, int64_t K, uint8_t* codes,
                   uint8_t* scale, void* stream) {
  if (dtype != QN_F32 && dtype != QN_BF16) return QN_ERR_UNSUPPORTED;
  if (!mx_size_ok(R, K)) return QN_ERR_SHAPE;
  if (R == 0 || K == 0) return QN_OK;
  if (!x || !codes || !scale) return QN_ERR_NULL;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scale, 4)) return QN_ERR_ALIGN;
  (void)hipGetLastError();
  return hip_status(
      qn::launch_mx_quantize(x, dtype == QN_BF16, R, K, codes, scale, as_stream(stream)));
}

int mxfp4_dequant(const uint8_t* codes, const uint8_t* scale, int64_t R, int64_t K,
                  int32_t out_dtype, void* out, void* stream) {
  if (out_dtype != QN_F32 && out_dtype != QN_BF16) return QN_ERR_UNSUPPORTED;
  if (!mx_size_ok(R, K)) return QN_ERR_SHAPE;
  if (R == 0 || K == 0) return QN_OK;
  if (!codes || !scale || !out) return QN_ERR_NULL;
  if (!aligned(codes, 16) || !aligned(scale, 4) || !aligned(out, 16)) return QN_ERR_ALIGN;
  (void)hipGetLastError();
  return hip_status(qn::launch_mx_dequant(qn::MxView{codes, scale, R, K}, out_dtype == QN_BF16, out,
                                          as_stream(stream)));
}

static int mx_scales(bool pack, const uint8_t* in, int64_t R, int64_t K, uint8_t* out,
                     void* stream) {
  if (!mx_size_ok(R, K)) return QN_ERR_SHAPE;
  if (R == 0 || K == 0) return QN_OK;
  if (!in || !out) return QN_ERR_NULL;
  if (!aligned(pack ? out : in, 4)) return QN_ERR_ALIGN;
  (void)hipGetLastError();
  return hip_status(qn::launch_mx_scales(pack, in, R, K, out, as_stream(stream)));
}

int mxfp4_pack_scales(const uint8_t* rows, int64_t R, int64_t K, uint8_t* scale, void* stream) {
  return mx_scales(true, rows, R, K, scale, stream);
}

int mxfp4_unpack_scales(const uint8_t* scale, int64_t R, int64_t K, uint8_t* rows, void* stream) {
  return mx_scales(false, scale, R, K, rows, stream);
}

int mxfp4_matmul(const qn_mxfp4_weight* w, const uint8_t* x, const uint8_t* xscale, int64_t M,
                 qn_bf16* out, void* ws, size_t ws_bytes, void* stream) {
  qn::MxView v;
  if (int st = check_mx_weight(w, v); st != QN_OK) return st;
  if (!mx_rows_ok(M, v.N, v.K)) return QN_ERR_SHAPE;
  if (M == 0) return QN_OK;
  if (!x || !xscale || !out) return QN_ERR_NULL;
  if (!aligned(x, 16) || !aligned(xscale, 4) || !aligned(out, 16)) return QN_ERR_ALIGN;
  const MxWs f = mx_ws(false, M, v.N, v.K, 0);
  if (!ws || ws_bytes < f.total) return QN_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return QN_ERR_ALIGN;
  float* split =
      f.total > f.split ? reinterpret_cast<float*>(static_cast<char*>(ws) + f.split) : nullptr;
  (void)hipGetLastError();
  hipStream_t s = as_stream(stream);
  if (qn::mx_few(M, v.N, v.K))
    return hip_status(qn::launch_mx_decode(v, x, xscale, static_cast<int>(M), nullptr, 0, nullptr,
                                           nullptr, 0, 0.0f, out, nullptr, s));
  return hip_status(qn::launch_mx_gemm(v.codes, v.scale, v.N, v.K, f.bytes, x, xscale, M, nullptr,
                                       nullptr, 0, false, out, split, s));
}

int mxfp4_linear_fwd(const qn_mxfp4_weight* w, const qn_bf16* x, int64_t M, const qn_bf16* A,
                     const qn_bf16* B, int32_t r, float alpha, qn_bf16* y, qn_bf16* u_out, void* ws,
                     size_t ws_bytes, void* stream) {
  return mx_linear(false, w, x, M, A, B, r, alpha, y, u_out, ws, ws_bytes, stream);
}

int mxfp4_linear_bwd_dx(const qn_mxfp4_weight* w, const qn_bf16* dy, int64_t M, const qn_bf16* A,
                        const qn_bf16* B, int32_t r, float alpha, qn_bf16* dx, qn_bf16* t_out,
                        void* ws, size_t ws_bytes, void* stream) {
  return mx_linear(true, w, dy, M, A, B, r, alpha, dx, t_out, ws, ws_bytes, stream);
}

size_t lora_adamw_table_bytes(const qn_adamw_tensor* t, int32_t count) {
  if (!t || count < 0) return 0;
  const int64_t chunks = adamw_chunks(t, count);
  return chunks < 0 ? 0 : adamw_table_size(chunks);
}

int lora_adamw_table(const qn_adamw_tensor* t, int32_t count, int32_t grad_dtype, int32_t state,
                     void* table, size_t bytes, qn_adamw_plan* plan) {
  if (!plan || (count > 0 && !t)) return QN_ERR_NULL;
  if ((grad_dtype != QN_F32 && grad_dtype != QN_BF16) ||
      (state != QN_STATE_F32 && state != QN_STATE_8BIT))
    return QN_ERR_UNSUPPORTED;
  if (count < 0) return QN_ERR_SHAPE;
  const int64_t chunks = adamw_chunks(t, count);
  if (chunks < 0) return QN_ERR_SHAPE;
  const bool state8 = state == QN_STATE_8BIT;
  for (int32_t i = 0; i < count; ++i) {
    const qn_adamw_tensor& a = t[i];
    if (a.n == 0) continue;
    if (!a.p || !a.g || !a.m || !a.v || (state8 && (!a.m_scale || !a.v_scale)))
      return QN_ERR_NULL;
    if (!aligned(a.p, 16) || !aligned(a.g, 16) || !aligned(a.m, 16) || !aligned(a.v, 16) ||
        !aligned(a.p_bf16, 16) ||
        (state8 && (!aligned(a.m_scale, 4) || !aligned(a.v_scale, 4))))
      return QN_ERR_ALIGN;
  }
  const size_t need = adamw_table_size(chunks);
  if (need > 0 && (!table || bytes < need)) return QN_ERR_WORKSPACE;
  if (!aligned(table, 8)) return QN_ERR_ALIGN;
  try {
    if (adamw_overlaps(t, count, grad_dtype == QN_BF16 ? 2 : 4, state8)) return QN_ERR_SHAPE;
  } catch (...) {  // no host memory for the ranges
    return QN_ERR_WORKSPACE;
  }
  *plan = qn_adamw_plan{chunks, static_cast<int64_t>(need), grad_dtype, state};
  qn::AdamChunk* d = static_cast<qn::AdamChunk*>(table);
  for (int32_t i = 0; i < count; ++i) {
    const qn_adamw_tensor& a = t[i];
    for (int64_t e = 0; e < a.n; e += qn::kAdamChunk) {
      const int64_t blk = e / qn::kAdamStateBlock, state = state8 ? e : e * 4;
      *d++ = qn::AdamChunk{a.p + e,
                           static_cast<const char*>(a.g) + e * (grad_dtype == QN_BF16 ? 2 : 4),
                           static_cast<char*>(a.m) + state,
                           static_cast<char*>(a.v) + state,
                           state8 ? a.m_scale + blk : nullptr,
                           state8 ? a.v_scale + blk : nullptr,
                           a.p_bf16 ? a.p_bf16 + e : nullptr,
                           std::min<int64_t>(a.n - e, qn::kAdamChunk)};
    }
  }
  return QN_OK;
}

size_t lora_grad_norm_workspace_bytes(const qn_adamw_plan* plan) {
  if (!plan || plan->chunks <= 0) return 0;
  return static_cast<size_t>(qn::grad_norm_blocks(plan->chunks)) * sizeof(double);
}

int lora_grad_norm(const qn_adamw_plan* plan, const void* table, float max_norm, float* out,
                   void* ws, size_t ws_bytes, void* stream) {
  if (int st = check_adamw_plan(plan, table); st != QN_OK) return st;
  if (!out) return QN_ERR_NULL;
  if (!(max_norm > 0.0f)) return QN_ERR_SHAPE;
  if (!aligned(out, 4)) return QN_ERR_ALIGN;
  const size_t need = lora_grad_norm_workspace_bytes(plan);
  if (need > 0 && (!ws || ws_bytes < need)) return QN_ERR_WORKSPACE;
  if (!aligned(ws, 8)) return QN_ERR_ALIGN;
  (void)hipGetLastError();
  return hip_status(qn::launch_grad_norm(adamw_table(table), plan->chunks,
                                         plan->grad_dtype == QN_BF16, max_norm,
                                         static_cast<double*>(ws), out, as_stream(stream)));
}

int lora_adamw_multi_step(const qn_adamw_plan* plan, const void* table, const float* grad_scale,
                          float lr, float beta1, float beta2, float eps, float weight_decay,
                          int32_t step, void* stream) {
  if (int st = check_adamw_plan(plan, table); st != QN_OK) return st;
  if (!aligned(grad_scale, 4)) return QN_ERR_ALIGN;
  if (step < 1 || !adamw_hyper_ok(lr, beta1, beta2, eps, weight_decay)) return QN_ERR_SHAPE;
  (void)hipGetLastError();
  return hip_status(qn::launch_adamw_multi(
      adamw_table(table), plan->chunks, plan->state == QN_STATE_8BIT,
      plan->grad_dtype == QN_BF16, grad_scale, lr, beta1, beta2, eps, weight_decay, step,
      as_stream(stream)));
}

size_t lora_muon_table_bytes(const qn_muon_tensor* t, int32_t count) {
  qn_muon_plan plan;
  int64_t runs;
  if (!t || count < 0 || muon_sizes(t, count, plan, runs) != QN_OK) return 0;
  return static_cast<size_t>(plan.bytes);
}

int lora_muon_table(const qn_muon_tensor* t, int32_t count, int32_t grad_dtype, void* table,
                    size_t bytes, qn_muon_plan* plan) {
  if (!plan || (count > 0 && !t)) return QN_ERR_NULL;
  if (grad_dtype != QN_F32 && grad_dtype != QN_BF16) return QN_ERR_UNSUPPORTED;
  if (count < 0) return QN_ERR_SHAPE;
  qn_muon_plan made;
  int64_t total_runs;
  if (int st = muon_sizes(t, count, made, total_runs); st != QN_OK) return st;
  made.grad_dtype = grad_dtype;
  const int64_t grad_size = grad_dtype == QN_BF16 ? 2 : 4;
  for (int32_t i = 0; i < count; ++i) {
    const qn_muon_tensor& a = t[i];
    if (a.rows == 0 || a.cols == 0) continue;
    if (!a.p || !a.g || !a.m) return QN_ERR_NULL;
    if (!aligned(a.p, 16) || !aligned(a.g, 16) || !aligned(a.m, 16) || !aligned(a.p_bf16, 16))
      return QN_ERR_ALIGN;
  }
  if (made.bytes > 0 && (!table || bytes < static_cast<size_t>(made.bytes)))
    return QN_ERR_WORKSPACE;
  if (!aligned(table, 8)) return QN_ERR_ALIGN;
  try {
    std::vector<Range> all;
    all.reserve(static_cast<size_t>(count) * 4);
    for (int32_t i = 0; i < count; ++i) {
      const int64_t n = t[i].rows * t[i].cols;
      auto add = [&](const void* p, int64_t size, bool written) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        if (p && n > 0) all.push_back({lo, lo + static_cast<uintptr_t>(size), written});
      };
      add(t[i].p, n * 4, true);
      add(t[i].g, n * grad_size, false);
      add(t[i].m, n * 4, true);
      add(t[i].p_bf16, n * 2, true);
    }
    if (ranges_overlap(all)) return QN_ERR_SHAPE;
  } catch (...) {  // no host memory for the ranges
    return QN_ERR_WORKSPACE;
  }
  *plan = made;
  int64_t matrices = 0;
  for (int64_t m : made.matrices) matrices += m;
  qn::MuonMatrix* mats = static_cast<qn::MuonMatrix*>(table);
  qn::MuonChunk* chunk = reinterpret_cast<qn::MuonChunk*>(mats + matrices);
  int64_t at = 0;  // in the workspace
  int32_t index = 0;
  MuonShape s;
  for (int cls = 0; cls < qn::kMuonClasses; ++cls) {
    qn::MuonChunk* span = chunk + made.chunks[cls];
    for (int32_t i = 0; i < count; ++i) {
      muon_shape(t[i], s);
      if (s.len == 0 || s.cls != cls) continue;
      const int64_t per = muon_chunk_runs(s, total_runs), per2 = muon_span_runs(s, total_runs);
      const int32_t n = static_cast<int32_t>(qn::mx_tiles(s.runs, per));
      const int32_t n2 = static_cast<int32_t>(qn::mx_tiles(s.runs, per2));
      const int64_t factor = at + n * muon_sums(s.tiles);
      *mats++ = qn::MuonMatrix{t[i].p, t[i].g, t[i].m, t[i].p_bf16, s.len, per * s.run,
                               per2 * s.run, at, factor, static_cast<int32_t>(s.r),
                               t[i].rows > t[i].cols ? 1 : 0, n, n2};
      for (int32_t c = 0; c < n; ++c) *chunk++ = qn::MuonChunk{index, c};
      for (int32_t c = 0; c < n2; ++c) *span++ = qn::MuonChunk{index, c};
      at = factor + muon_factor(s.tiles);
      ++index;
    }
    chunk = span;
  }
  return QN_OK;
}

size_t lora_muon_workspace_bytes(const qn_muon_plan* plan) {
  return plan && plan->ws_bytes > 0 ? static_cast<size_t>(plan->ws_bytes) : 0;
}

int lora_muon_multi_step(const qn_muon_plan* plan, const void* table, const qn_muon_step* step,
                         void* ws, size_t ws_bytes, void* stream) {
  if (int st = check_muon_plan(plan, table); st != QN_OK) return st;
  if (!step) return QN_ERR_NULL;
  if (step->adjust != QN_MUON_ORIGINAL && step->adjust != QN_MUON_MATCH_RMS)
    return QN_ERR_UNSUPPORTED;
  if (!(step->lr >= 0.0f) || !(step->momentum >= 0.0f && step->momentum < 1.0f) ||
      !(step->weight_decay >= 0.0f) || !(step->eps > 0.0f) || step->ns_steps < 1 ||
      step->ns_steps > 32 || !std::isfinite(step->ns[0]) || !std::isfinite(step->ns[1]) ||
      !std::isfinite(step->ns[2]) || (step->nesterov != 0 && step->nesterov != 1))
    return QN_ERR_SHAPE;
  if (2.0 * step->ns_steps * std::log2(std::fabs(step->ns[0])) > kMuonMaxGrowth)
    return QN_ERR_UNSUPPORTED;
  if (plan->ws_bytes > 0 && (!ws || ws_bytes < static_cast<size_t>(plan->ws_bytes)))
    return QN_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return QN_ERR_ALIGN;
  (void)hipGetLastError();
  qn::MuonCounts n;
  int64_t matrices = 0;
  for (int k = 0; k < qn::kMuonClasses; ++k) {
    n.matrices[k] = plan->matrices[k], n.chunks[k] = plan->chunks[k], n.spans[k] = plan->spans[k];
    matrices += plan->matrices[k];
  }
  const qn::MuonMatrix* mats = static_cast<const qn::MuonMatrix*>(table);
  const qn::MuonStep h{step->lr,     step->momentum, step->weight_decay, step->eps,
                       step->ns[0],  step->ns[1],    step->ns[2],        step->ns_steps,
                       step->nesterov == 1, step->adjust == QN_MUON_MATCH_RMS};
  return hip_status(qn::launch_muon(mats, reinterpret_cast<const qn::MuonChunk*>(mats + matrices),
                                    n, plan->grad_dtype == QN_BF16, h, ws, as_stream(stream)));
}

int lora_grads(const qn_bf16* x, const qn_bf16* dy, const qn_bf16* u, const qn_bf16* t,
               const qn_bf16* A, const qn_bf16* B, int64_t M, int64_t N, int64_t K, int32_t r,
               float alpha, float* dA, float* dB, void* ws, size_t ws_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0 || r < 0) return QN_ERR_SHAPE;
  if (r == 0) return QN_ERR_SHAPE;
  if (r > kMaxRank) return QN_ERR_UNSUPPORTED;
  if (N == 0 || K == 0 || N % 64 != 0 || K % 64 != 0) return QN_ERR_SHAPE;
  if (!dA || !dB) return QN_ERR_NULL;
  if (M > 0 && (!x || !dy || (!u && !A) || (!t && !B))) return QN_ERR_NULL;
  if ((x && !aligned(x, 16)) || (dy && !aligned(dy, 16)) || (A && !aligned(A, 16)) ||
      (B && !aligned(B, 2)) || (u && !aligned(u, 2)) || (t && !aligned(t, 2)) ||
      !aligned(dA, 4) || !aligned(dB, 4))
    return QN_ERR_ALIGN;
  const size_t need = grads_ws(M, N, K, r);
  if (!ws || ws_bytes < need) return QN_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return QN_ERR_ALIGN;
  if (!qn::tables()) return QN_ERR_UNSUPPORTED;
  hipStream_t s = as_stream(stream);
  (void)hipGetLastError();
  const float scale = alpha / static_cast<float>(r);
  // u and t, when not given, are recomputed as bf16 by the launches the
  // forward and the backward use for u_out and t_out (same splits, same
  // fixed-order sums), so they equal the saved ones bit for bit for M > 16
  // (t at every M)
  char* base = static_cast<char*>(ws);
  const int64_t mp = M > kGemvMaxM ? M : kGemvMaxM + 1;
  uint16_t* u16 = reinterpret_cast<uint16_t*>(base);
  uint16_t* t16 = reinterpret_cast<uint16_t*>(base + lora_bf16_bytes(M, r));
  float* lpart = reinterpret_cast<float*>(base + 2 * lora_bf16_bytes(M, r));
  void* part = base + 2 * lora_bf16_bytes(M, r) + lora_part_bytes(mp, r);
  if (M > 0 && !u) {
    const int ks = qn::skinny_wide_splits(mp, K);
    if (qn::launch_skinny(x, M, K, A, r, 1.0f, lpart, nullptr, nullptr, ks, s) != hipSuccess ||
        qn::launch_lora_reduce(lpart, ks, M * r, 1.0f, u16, nullptr, s) != hipSuccess)
      return QN_ERR_HIP;
  }
  if (M > 0 && !t) {
    const int ks = qn::skinny_wide_splits(mp, N);
    if (qn::launch_skinny(dy, M, N, B, r, 1.0f, lpart, nullptr, nullptr, ks, s, true) != hipSuccess ||
        qn::launch_lora_reduce(lpart, ks, M * r, 1.0f, t16, nullptr, s) != hipSuccess)
      return QN_ERR_HIP;
  }
  return hip_status(qn::launch_grads_impl(x, dy, u ? u : u16, t ? t : t16, M, N, K, r, scale, dA,
                                          dB, part, s));
}

}  // extern "C"
