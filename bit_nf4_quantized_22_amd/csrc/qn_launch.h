// Host-side launch functions, one per kernel family.  The C ABI in
// qn_api.cpp validates arguments and then calls these; each returns the
// hipError_t of its launch(es).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qn {

struct CodeParams;  // qn_device.h

// Kinds of level-2 code of the block constants.
constexpr int kL2Grid8 = 0;    // uint8 grid fl32(q / 255) of c / c2
constexpr int kL2E4M3 = 1;     // E4M3 number of c / c2
constexpr int kL2Centred = 2;  // signed grid fl32(k / 127) of (c - mu) / c2

struct WeightView {
  const uint8_t* packed;
  const uint8_t* qscale;  // nullptr: not double-quantised
  const float* gscale;
  const float* absmax;
  int64_t N, K;
  int quant_type;  // kQuantNF4 or kQuantFP4 (the code table)
  int l2;          // level-2 code: 0 uint8 grid, 1 E4M3, 2 mean-centred signed grid
  const float* mu; // the centred code's offset (device, one fp32), else nullptr
};

// Code values and level-2 kind of a weight, for the kernels.
CodeParams code_params(const WeightView& w);

hipError_t launch_quantize(const void* w, bool bf16, int64_t numel, int quant_type,
                           uint8_t* packed, float* absmax, hipStream_t s);
hipError_t launch_dq(const float* absmax, int64_t nblocks, bool fp8, uint8_t* qscale,
                     float* gscale, hipStream_t s);
// Both in one launch (one workgroup per 256-block group); absmax may be
// nullptr.
hipError_t launch_quantize_dq(const void* w, bool bf16, int64_t numel, int quant_type, bool fp8,
                              uint8_t* packed, float* absmax, uint8_t* qscale, float* gscale,
                              hipStream_t s);
// Several weights of one dtype and code type in one launch: entry i is
// weight w[i] of numel[i] elements and its outputs; gend[i] is one past the
// last group (workgroup) of entries 0..i.  The struct travels by value as
// a kernel argument.
constexpr int kQdqMaxBatch = 8;
struct QdqBatch {
  const void* w[kQdqMaxBatch];
  int64_t numel[kQdqMaxBatch];
  uint8_t* packed[kQdqMaxBatch];
  float* absmax[kQdqMaxBatch];
  uint8_t* qscale[kQdqMaxBatch];
  float* gscale[kQdqMaxBatch];
  uint32_t gend[kQdqMaxBatch];
  int n;
};
hipError_t launch_quantize_dq_batch(const QdqBatch& batch, bool bf16, int quant_type, bool fp8,
                                    hipStream_t s);
// Mean-centred level-2 code: mu (pairwise fp64 sum of the constants / n,
// written to *mu), then per 256-group c2 = max |c - mu| and signed codes.
// gscale doubles as scratch for the partial sums before its final values.
hipError_t launch_dq_centred(const float* absmax, int64_t nblocks, uint8_t* qscale, float* gscale,
                             float* mu, hipStream_t s);
hipError_t launch_dequant(const WeightView& w, bool out_bf16, void* out, hipStream_t s);

// out[M, r] = in[M, L] * P^T, P row-major [r, L] (in and P 16-byte
// aligned, L % 32 == 0).  ksplit == 1 writes any of: fp32 result,
// bf16(scale * result), bf16(result); ksplit > 1 splits L over ksplit
// workgroups and writes fp32 partial sums out_f32[ksplit][M][r].
// With p_rows_l, P is stored [L, r] instead (B for t = dy B, read in place).
hipError_t launch_skinny(const uint16_t* in, int64_t M, int64_t L, const uint16_t* P, int r,
                         float scale, float* out_f32, uint16_t* out_scaled_bf16,
                         uint16_t* out_bf16, int ksplit, hipStream_t s, bool p_rows_l = false);
// Largest number of L-slices of the decode LoRA-down (the forward
// workspace holds that many fp32 partial sums of u).
constexpr int kDecodeMaxSlices = 512;
// Largest number of L-slices of the token-batch LoRA projections u = x A^T
// and t = dy B, whose fp32 partial sums the fused GEMM adds up.
constexpr int kWideMaxSlices = 16;
// Number of L-slices launch_skinny uses for M > 16 tokens.
int skinny_wide_splits(int64_t M, int64_t L);

// Streaming read of `bytes` (a multiple of 16) with 16-byte loads (a
// measurement aid).
hipError_t launch_read_probe(const void* buf, int64_t bytes, uint32_t* sink, hipStream_t st);

// Size of the library's own per-device scratch array (qn_scratch.hip), the
// workspace of the allocation-free forward.
constexpr size_t kScratchBytes = static_cast<size_t>(64) << 20;
// Device address of the scratch array of the device that `stream` belongs
// to (the current device for the null stream), resolved once per device
// with that device current, then cached.
hipError_t scratch_address(hipStream_t stream, void** out);

// Threads per workgroup of the decode GEMV for an N x K weight.
int gemv_threads(int64_t N, int64_t K);
// Number of L-slices launch_skinny uses for the decode path (M <= 16),
// given the GEMV's threads per workgroup (which bounds the partial sums it
// can take).
int skinny_splits(int64_t M, int64_t L, int r, int gemv_thr);

// Decode path (M <= 16): y = x W^T + s u B^T with u given as usplit fp32
// partial sums [usplit][M][r]; optionally writes bf16(u) to u_out.
// With A_self (A [r, K]; only where gemv_self_u holds) the GEMV launch
// computes u itself from x, and u / usplit are not read.
hipError_t launch_gemv(const WeightView& w, const uint16_t* x, int M, const float* u, int usplit,
                       const uint16_t* B, int r, float s, uint16_t* y, uint16_t* u_out,
                       hipStream_t st, const uint16_t* A_self = nullptr);
// Whether the GEMV for this weight, M and r computes the LoRA-down in the
// same launch (one token, r <= 16, one pass of the 16-wave kernel, and A
// re-read by all bands in at most about 40 MB).
bool gemv_self_u(const WeightView& w, int M, int r);

// Fused dequant GEMM, forward: y[M,N] = x W^T + us B^T (us = bf16(s*u), [M, r]).
hipError_t launch_gemm_fwd(const WeightView& w, const uint16_t* x, int64_t M,
                           const uint16_t* us, const uint16_t* B, int r, uint16_t* y,
                           hipStream_t st);

// Fused dequant GEMM, backward to the input: dx[M,K] = dy W + ts A; with
// dx32 the fp32 result goes to dx32 [M, K] instead (dx untouched).
hipError_t launch_gemm_bwd(const WeightView& w, const uint16_t* dy, int64_t M,
                           const uint16_t* ts, const uint16_t* A, int r, uint16_t* dx,
                           hipStream_t st, float* dx32 = nullptr);

// Sum of nslice (<= kWideMaxSlices) fp32 partial sums part[nslice][n] in
// slice order: writes bf16(scale * sum) to out_scaled (and bf16(sum) to out
// if non-null).
hipError_t launch_lora_reduce(const float* part, int nslice, int64_t n, float scale,
                              uint16_t* out_scaled, uint16_t* out, hipStream_t st);

// A weight in E4M3 codes with one scale per 128 x 128 block.
struct Fp8View {
  const uint8_t* codes;  // [N, K]
  const float* scale;    // [ceil(N / 128), ceil(K / 128)]
  int64_t N, K;          // multiples of 16
};

// Block-scaled FP8 (see the fp8_* entries of the C ABI).  Row scales are
// [ceil(K / 128), M].
hipError_t launch_fp8_quantize_blocks(const void* w, bool bf16, int64_t N, int64_t K,
                                      uint8_t* codes, float* scale, hipStream_t st);
hipError_t launch_fp8_quantize_rows(const uint16_t* x, int64_t M, int64_t K, uint8_t* codes,
                                    float* scale, hipStream_t st);
// launch_fp8_quantize_rows of x [M, L], and partial sums part[slices][M][r]
// of its LoRA projection x P^T (P [r, L], or [L, r] with rows_l; r >= 1).
int fp8_project_slices(int64_t M, int64_t L);
hipError_t launch_fp8_quantize_project(const uint16_t* x, int64_t M, int64_t L, const uint16_t* P,
                                       int r, bool rows_l, uint8_t* codes, float* scale,
                                       float* part, hipStream_t st);
// y [M, N] = x W^T + (lora_scale u) B^T for fp8_few(..) tokens, u given as
// slices partial sums [slices][M][r] (M <= kFp8DecodeM; bf16(u) to u_out if
// not null) or as act (see launch_fp8_project_sum).
constexpr int kFp8DecodeM = 16, kFp8FewM = 64;
bool fp8_few(int64_t M, int64_t N, int64_t K);
hipError_t launch_fp8_decode(const Fp8View& w, const uint8_t* x, const float* xs, int M,
                             const float* part, int slices, const uint16_t* act,
                             const uint16_t* B, int r, float lora_scale, uint16_t* y,
                             uint16_t* u_out, hipStream_t st);
// launch_fp8_quantize_project of M <= kFp8DecodeM tokens with P = A, into
// fp8_decode_slices(L) slices; codes == nullptr: the projection alone.
int fp8_decode_slices(int64_t L);
hipError_t launch_fp8_decode_project(const uint16_t* x, int M, int64_t L, const uint16_t* A, int r,
                                     uint8_t* codes, float* scale, float* part, hipStream_t st);
// One token, x quantised by the product's workgroups; u = x A^T given as
// slices partial sums, or (part == nullptr, where fp8_token_self_u holds)
// computed by them too.
bool fp8_token_self_u(const Fp8View& w, int r);
hipError_t launch_fp8_token(const Fp8View& w, const uint16_t* x, const uint16_t* A,
                            const float* part, int slices, const uint16_t* B, int r,
                            float lora_scale, uint16_t* y, uint16_t* u_out, hipStream_t st);
// out = bf16(sum of `splits` fp32 parts of n values).
hipError_t launch_fp8_split_sum(const float* part, int splits, int64_t n, uint16_t* out,
                                hipStream_t st);
hipError_t launch_fp8_dequant(const Fp8View& w, bool out_bf16, void* out, hipStream_t st);
// The LoRA term's token side for launch_fp8_gemm: act[M], scale * the sum of
// the slices of part, each value as a sum hi + lo of two bf16 numbers: one
// bf16 alone would cost 2^-8 of the term before the result is rounded.  Rows of
// fp8_lora_pitch(r) values: for each 32 ranks their 32 hi, then their 32 lo,
// zeros behind r.  The sum's bf16 without the scale goes to plain [M, r] if
// not null.
inline int fp8_lora_ranks(int r) { return (r + 31) / 32 * 32; }
inline int fp8_lora_pitch(int r) { return 2 * fp8_lora_ranks(r); }
hipError_t launch_fp8_project_sum(const float* part, int slices, int64_t M, int r, float scale,
                                  uint16_t* act, uint16_t* plain, hipStream_t st);
// out = x W^T + act lw^T (x [M, K], lw = B [N, r]), or with bwd
// out = x W + act lw (x [M, N], lw = A [r, K]); x in codes with row scales
// (r == 0: no LoRA term).  The contraction (L) is split over
// fp8_gemm_splits(M, ncols, L) workgroups where the tiles are few and part,
// fp32 [splits][M][ncols], is given.
int fp8_gemm_splits(int64_t M, int64_t ncols, int64_t L);
hipError_t launch_fp8_gemm(const Fp8View& w, const uint8_t* x, const float* xs, int64_t M,
                           const uint16_t* act, const uint16_t* lw, int r, bool bwd, uint16_t* out,
                           float* part, hipStream_t st);

// A weight in microscaled E2M1 codes.
struct MxView {
  const uint8_t* codes;  // [N, K / 2]
  const uint8_t* scale;  // tiles of 32 rows x 256 columns, [ceil(K / 256)][ceil(N / 32)][256]
  int64_t N, K;          // multiples of 16 and 32
};

// Tiles of t that cover n.
constexpr int64_t mx_tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }

// Microscaled 4-bit (see the mxfp4_* entries of the C ABI).  x [R, K].
hipError_t launch_mx_quantize(const void* x, bool bf16, int64_t R, int64_t K, uint8_t* codes,
                              uint8_t* scale, hipStream_t st);
hipError_t launch_mx_dequant(const MxView& w, bool out_bf16, void* out, hipStream_t st);
// Scales from rows [R, K / 32] to tiles (pack) or back.
hipError_t launch_mx_scales(bool pack, const uint8_t* in, int64_t R, int64_t K, uint8_t* out,
                            hipStream_t st);
// A batch x [M, L] in codes: forward E2M1 [M, L / 2] with tiles as a weight's,
// backward E4M3 [M, mx_tiles(L, 128) * 128] with tiles of 64 rows x 128 columns.
// The second form, forward, also gives fp8_project_slices(M, L) partial sums
// part[slices][M][r] of the LoRA projection x A^T (A [r, L], r >= 1).
hipError_t launch_mx_rows(const uint16_t* x, int64_t M, int64_t L, bool bwd, uint8_t* codes,
                          uint8_t* scale, hipStream_t st);
hipError_t launch_mx_rows_project(const uint16_t* x, int64_t M, int64_t L, const uint16_t* A, int r,
                                  uint8_t* codes, uint8_t* scale, float* part, hipStream_t st);
// The same of M <= kFp8DecodeM tokens, forward, in fp8_decode_slices(L) slices.
hipError_t launch_mx_decode_project(const uint16_t* x, int M, int64_t L, const uint16_t* A, int r,
                                    uint8_t* codes, uint8_t* scale, float* part, hipStream_t st);
// W^T in E5M2 codes wt [K, mx_tiles(N, 128) * 128] with tiles ts of 64 rows x
// 128 columns, for the backward's product.
hipError_t launch_mx_turn(const MxView& w, uint8_t* wt, uint8_t* ts, hipStream_t st);
// launch_mx_rows of dy [M, N] with fp8_project_slices(M, N) partial sums of dy B (B
// [N, r], r >= 1), and launch_mx_turn, in one launch.
hipError_t launch_mx_backward(const MxView& w, const uint16_t* dy, int64_t M, const uint16_t* B,
                              int r, uint8_t* codes, uint8_t* scale, float* part, uint8_t* wt,
                              uint8_t* ts, hipStream_t st);
// y [M, N] = x W^T + (lora_scale u) B^T for mx_few(..) tokens in codes, u given as
// to launch_fp8_decode.
bool mx_few(int64_t M, int64_t N, int64_t K);
hipError_t launch_mx_decode(const MxView& w, const uint8_t* x, const uint8_t* xs, int M,
                            const float* part, int slices, const uint16_t* act, const uint16_t* B,
                            int r, float lora_scale, uint16_t* y, uint16_t* u_out, hipStream_t st);
// One token, quantised by the product's workgroups; u = x A^T given as slices
// partial sums, or (part == nullptr, where mx_token_self_u holds) computed by
// them too.
bool mx_token_self_u(const MxView& w, int r);
hipError_t launch_mx_token(const MxView& w, const uint16_t* x, const uint16_t* A, const float* part,
                           int slices, const uint16_t* B, int r, float lora_scale, uint16_t* y,
                           uint16_t* u_out, hipStream_t st);
// out [M, N] = x w^T + act B^T (w, x E2M1 codes, bytes = K / 2), or with bwd
// out [M, K] = x w^T + act A (w the turned weight, x E4M3 codes, bytes a multiple
// of 128); act as launch_fp8_project_sum gives it (r == 0: no LoRA term).  The
// contraction is split over mx_gemm_splits(M, ncols, bytes, bwd) workgroups where the
// tiles are few and part, fp32 [splits][M][ncols], is given.
int mx_gemm_splits(int64_t M, int64_t ncols, int64_t bytes, bool bwd);
hipError_t launch_mx_gemm(const uint8_t* w, const uint8_t* ws, int64_t N, int64_t K, int64_t bytes,
                          const uint8_t* x, const uint8_t* xs, int64_t M, const uint16_t* act,
                          const uint16_t* lw, int r, bool bwd, uint16_t* out, float* part,
                          hipStream_t st);

// LoRA merge: out[N, K] = bf16(dequant(W) + s B A) (A [r, K], B [N, r]).
hipError_t launch_merge(const WeightView& w, const uint16_t* A, const uint16_t* B, int r, float s,
                        uint16_t* out, hipStream_t st);

// AdamW step (see lora_adamw_step in the C ABI).
hipError_t launch_adamw(float* p, const float* g, float* m, float* v, uint16_t* p_bf16, int64_t n,
                        float lr, float beta1, float beta2, float eps, float weight_decay, int step,
                        hipStream_t st);

// AdamW over many matrices (see lora_adamw_multi_step in the C ABI): the
// device table holds one entry per workgroup, a chunk of up to kAdamChunk
// elements of one matrix with the addresses of its first element.
struct AdamChunk {
  float* p;
  const void* g;  // fp32 or bf16
  void* m;        // fp32, or E4M3 codes
  void* v;        // fp32, or E5M2 codes
  float* m_scale;
  float* v_scale;
  uint16_t* p_bf16;
  int64_t n;
};
constexpr int kAdamChunk = 2048;
constexpr int kAdamStateBlock = 256;  // elements per scale of the 8-bit states
constexpr int kGradNormBlocks = 1024;  // most partial sums of the gradient norm
int grad_norm_blocks(int64_t chunks);
hipError_t launch_adamw_multi(const AdamChunk* tab, int64_t chunks, bool state8, bool bf16_grad,
                              const float* grad_scale, float lr, float beta1, float beta2,
                              float eps, float weight_decay, int step, hipStream_t st);
// part: grad_norm_blocks(chunks) doubles; out[0] = norm, out[1] = clip
// coefficient.
hipError_t launch_grad_norm(const AdamChunk* tab, int64_t chunks, bool bf16_grad, float max_norm,
                            double* part, float* out, hipStream_t st);

// Muon over many matrices (see lora_muon_multi_step in the C ABI).  The device
// table holds the matrices, in the order of their classes (short sides up to 16,
// 32, 64 and 128), then for each class one entry per workgroup of the first pass,
// a chunk of a matrix's long side, and one per workgroup of the last, a span.
struct MuonMatrix {
  float* p;
  const void* g;  // fp32 or bf16
  float* m;
  uint16_t* p_bf16;
  int64_t len;      // the long side; row-major [r, len], or with tall [len, r]
  int64_t chunk;    // elements of the long side in a chunk
  int64_t span;     // and in a span
  int64_t part;     // in the workspace, in doubles: the chunks' sums
  int64_t factor;   // and the product's left factor
  int32_t r, tall, chunks;
  int32_t spans;    // for readers of the table on the host: a span names itself
};
struct MuonChunk {
  int32_t matrix;  // in the table
  int32_t index;   // among the matrix's chunks or spans
};
constexpr int kMuonClasses = 4;
constexpr int kMuonTiles[kMuonClasses] = {1, 2, 4, 8};  // of 16 rows
// What a workgroup of the passes takes at a time of the long side: 64 (or 32) for
// each of its waves.
constexpr int kMuonRun[kMuonClasses] = {256, 128, 128, 256};
struct MuonStep {
  float lr, momentum, weight_decay, eps;
  double a, b, c;
  int steps;
  bool nesterov, rms;
};
struct MuonCounts {
  int64_t matrices[kMuonClasses], chunks[kMuonClasses], spans[kMuonClasses];
};
hipError_t launch_muon(const MuonMatrix* mats, const MuonChunk* chunks, const MuonCounts& n,
                       bool bf16_grad, const MuonStep& h, void* ws, hipStream_t st);

// LoRA dropout on the adapter branch (see lora_dropout in the C ABI):
// threshold = floor(p 2^32) on the 32-bit Philox halves, inv_keep =
// fl32(1 / (1 - p)), both from fp64 on the host.
struct DropoutParams {
  uint32_t threshold;
  float inv_keep;
};
DropoutParams dropout_params(float p);
// out[M, K] = x * keep / (1 - p) in bf16 (dropped elements +0); K % 8 == 0.
hipError_t launch_dropout(const uint16_t* x, int64_t M, int64_t K, float p, uint64_t seed,
                          uint16_t* out, hipStream_t st);
// dx[M, K] = bf16(base[M, K] + keep * (ts A) / (1 - p)), base the fp32
// product dy W, ts = bf16(s t) [M, r], A [r, K]: one rounding.
hipError_t launch_dx_lora_dropout(const float* base, uint16_t* dx, const uint16_t* ts,
                                  const uint16_t* A, int64_t M, int64_t K, int r, float p,
                                  uint64_t seed, hipStream_t st);

// LoRA gradients (see lora_grads in the C ABI).  u and t are bf16 [M, r];
// ws holds grads_workspace_bytes() of split-M partials.
size_t grads_workspace_bytes(int64_t M, int64_t N, int64_t K, int r);
hipError_t launch_grads_impl(const uint16_t* x, const uint16_t* dy, const uint16_t* u,
                             const uint16_t* t, int64_t M, int64_t N, int64_t K, int r, float s,
                             float* dA, float* dB, void* ws, hipStream_t st);

}  // namespace qn
