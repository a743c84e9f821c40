// internal.hpp -- launchers shared between the C ABI layer and the kernel sources.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

// Number of compute units of the current device (cached per device).
int device_cu_count();

// Rowwise quantize: line l = row l of src, K = cols.  flat: the whole problem is one
// dense run of blocks (ld_src == K == Kp, ld_codes == Kp, ld_scales == nb).
// vec: every 8-element chunk of src can be read with 16-byte loads.  rule: the scale
// rule, kRuleCeil (0, the pages') or kRuleOcp (1, the OCP MX specification's).
hipError_t launch_quant_rows(const void* src, int src_bf16, int64_t rows, int64_t K, int64_t ld_src,
                             int fmt, int rule, uint8_t* codes, int64_t ld_codes, uint8_t* scales,
                             int64_t ld_scales, bool flat, bool vec, hipStream_t stream);

// Columnwise quantize: line l = column l of src [rows][ld_src], K = rows, codes and
// scales stored [cols][ld].
hipError_t launch_quant_cols(const void* src, int src_bf16, int64_t rows, int64_t cols, int64_t ld_src,
                             int fmt, int rule, uint8_t* codes, int64_t ld_codes, uint8_t* scales,
                             int64_t ld_scales, hipStream_t stream);

// Both orientations in one pass: rowwise codes [rows][ld_rc] (K = cols) and columnwise
// codes [cols][ld_cc] (K = rows), with their scales.
hipError_t launch_quant_dual(const void* src, int src_bf16, int64_t rows, int64_t cols, int64_t ld_src, int fmt,
                             uint8_t* rcodes, int64_t ld_rc, uint8_t* rscales, int64_t ld_rs, uint8_t* ccodes,
                             int64_t ld_cc, uint8_t* cscales, int64_t ld_cs, bool vec, hipStream_t stream);

// Quantize with stochastically rounded codes (rowwise, or colwise with transposed output);
// seed keys the Philox4x32-10 stream, element n of the padded code array draws word n % 4
// of counter n / 4.
hipError_t launch_quant_sr(const void* src, int src_bf16, int64_t rows, int64_t cols, int64_t ld_src, bool colwise,
                           int fmt, uint8_t* codes, int64_t ld_codes, uint8_t* scales, int64_t ld_scales, bool vec,
                           uint64_t seed, hipStream_t stream);

// Quantize with caller-owned scale bytes given [L][ld_given] (RNE-satfinite codes) and
// optional per-block diagnostics: amax (fp32), clipped and flushed counts (null = skip).
hipError_t launch_quant_scaled(const void* src, int src_bf16, int64_t rows, int64_t cols, int64_t ld_src, bool colwise,
                               int fmt, const uint8_t* given, int64_t ld_given, uint8_t* codes, int64_t ld_codes,
                               float* amax, int64_t ld_amax, uint8_t* clipped, uint8_t* flushed, int64_t ld_diag,
                               bool vec, hipStream_t stream);

hipError_t launch_dequant(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales,
                          int fmt, int64_t L, int64_t K, void* dst, int dst_bf16, int64_t ld_dst,
                          bool vec, hipStream_t stream);

// What a GEMM launch writes: v = act(alpha * acc + bias[col]) (act 0: identity, 1: SiLU);
// y (may be null) receives v rounded to its type; qc/qs (qc may be null) receive the MX
// codes (format q_fmt) and E8M0 scales of bf16(v) in 32-column blocks along N, i.e. the
// bytes the rowwise quantize gives for a bf16 Y.  y_vec16: y and its rows are 16-byte
// aligned.
struct GemmEpilogue {
  float alpha;
  const float* bias;
  int act;
  void* y;
  int y_bf16;
  int64_t ld_y;
  int y_vec16;
  uint8_t* qc;
  int64_t ld_qc;
  uint8_t* qs;
  int64_t ld_qs;
  int q_fmt;
};

// The GEMM kernels (gemm_exact.hip, gemm_fp8.hip, gemm_fallback.hip); launch_gemm picks one.
// Exact-product GEMM.  workspace: device memory for the K split of the last round's tiles
// (gemm_exact_workspace_bytes(M, N, K) bytes; with less, or none, the tiles run whole).
int64_t gemm_exact_workspace_bytes(int64_t M, int64_t N, int64_t K);
// The exact GEMM's plan for `cus` CUs (host logic only): tile width, K ranges per split
// tile, split tiles, whole tiles and workspace bytes.
void gemm_exact_plan(int64_t M, int64_t N, int64_t K, int cus, int* tile_n, int* ranges, int* split_tiles,
                     int* whole_tiles, int64_t* workspace_bytes);
hipError_t launch_gemm_exact(int64_t M, int64_t N, int64_t K, const uint8_t* xc, int64_t ld_x, const uint8_t* xs,
                             int64_t ld_xs, int x_fmt, const uint8_t* wc, int64_t ld_w, const uint8_t* ws,
                             int64_t ld_ws, int w_fmt, const GemmEpilogue& ep, void* workspace,
                             int64_t workspace_bytes, hipStream_t stream);
hipError_t launch_gemm_fp8(int64_t M, int64_t N, int64_t K, const uint8_t* xc, int64_t ld_x, const uint8_t* xs,
                           int64_t ld_xs, int x_fmt, const uint8_t* wc, int64_t ld_w, const uint8_t* ws, int64_t ld_ws,
                           int w_fmt, const GemmEpilogue& ep, hipStream_t stream);
hipError_t launch_gemm_fallback(int64_t M, int64_t N, int64_t K, const uint8_t* xc, int64_t ld_x, const uint8_t* xs,
                                int64_t ld_xs, int x_fmt, const uint8_t* wc, int64_t ld_w, const uint8_t* ws,
                                int64_t ld_ws, int w_fmt, const GemmEpilogue& ep, int exact, hipStream_t stream);

// workspace / workspace_bytes: device memory the exact kernel may use for its K split;
// may_alloc: when it is too small, take one from the stream-ordered pool for the call.
hipError_t launch_gemm(int64_t M, int64_t N, int64_t K,
                       const uint8_t* x_codes, int64_t ld_x, const uint8_t* x_scales, int64_t ld_xs, int x_fmt,
                       const uint8_t* w_codes, int64_t ld_w, const uint8_t* w_scales, int64_t ld_ws, int w_fmt,
                       const GemmEpilogue& ep, int exact, void* workspace, int64_t workspace_bytes, bool may_alloc,
                       hipStream_t stream);

// ---- MXFP4 (quantize_fp4.hip, gemm_fp4.hip, moe_fp4.hip).  Code rows hold 16 bytes per block;
// ld_codes is in bytes.

// One orientation: RNE codes under `rule`, or stochastically rounded ones (sr; ceil rule).
hipError_t launch_quant4(const void* src, int src_bf16, int64_t rows, int64_t cols, int64_t ld_src, bool colwise,
                         int rule, bool sr, uint64_t seed, uint8_t* codes, int64_t ld_codes, uint8_t* scales,
                         int64_t ld_scales, hipStream_t stream);
hipError_t launch_quant4_dual(const void* src, int src_bf16, int64_t rows, int64_t cols, int64_t ld_src, uint8_t* rcodes,
                              int64_t ld_rc, uint8_t* rscales, int64_t ld_rs, uint8_t* ccodes, int64_t ld_cc,
                              uint8_t* cscales, int64_t ld_cs, hipStream_t stream);
hipError_t launch_dequant4(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales, int64_t L,
                           int64_t K, void* dst, int dst_bf16, int64_t ld_dst, hipStream_t stream);

// How the MXFP4 product runs M x N x K on `cus` CUs (host logic only): its tile and the waves that share
// one, 0 where a thread takes a row of a tile of 1 x 4.  aligned: the scale rows are 16-byte aligned.
struct GemmFp4Plan {
  int tile_m, tile_n, waves;
};
GemmFp4Plan gemm_fp4_plan(int64_t M, int64_t N, int64_t K, bool x_fp4, bool aligned, int cus);

// X in bf16 (ld_x in elements, xs null) or MXFP4 (ld_x in bytes), W in MXFP4.
hipError_t launch_gemm_fp4(int64_t M, int64_t N, int64_t K, const void* x, bool x_fp4, int64_t ld_x, const uint8_t* xs,
                           int64_t ld_xs, const uint8_t* wc, int64_t ld_w, const uint8_t* ws, int64_t ld_ws,
                           const GemmEpilogue& ep, hipStream_t stream);

// The 256 x 256 tile kernel behind it: X and W in MXFP4, scale rows 16-byte aligned, ld_x < 2^24.
hipError_t launch_gemm_fp4_tile(int64_t M, int64_t N, int64_t K, const uint8_t* xc, int64_t ld_x, const uint8_t* xs,
                                int64_t ld_xs, const uint8_t* wc, int64_t ld_w, const uint8_t* ws, int64_t ld_ws,
                                const GemmEpilogue& ep, hipStream_t stream);

// A mixture-of-experts layer; ld_ are row pitches and st_ expert pitches, in bytes for codes
// and scales, in elements for x, logits and y.
struct MoeFp4 {
  int64_t T, H, I, E, k;
  bool renorm;
  const void* x;
  int64_t ld_x;
  const float* logits;
  int64_t ld_logits;
  const uint8_t* w13;
  int64_t ld_w13, st_w13;
  const uint8_t* s13;
  int64_t ld_s13, st_s13;
  const uint8_t* w2;
  int64_t ld_w2, st_w2;
  const uint8_t* s2;
  int64_t ld_s2, st_s2;
  void* y;
  int64_t ld_y;
  bool y_bf16;
  void* workspace;
};
// How the expert layer runs on `cus` CUs (host logic only): its launches, 2 or 4; of 4, the columns of I and of
// H that a workgroup takes (128 and 256: the persistent kernels) and the ranges of I of the down product.
// aligned: rows of x and scale rows are 16-byte aligned.
struct MoeFp4Plan {
  int launches, up_columns, down_columns, down_parts;
};
MoeFp4Plan moe_fp4_plan(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, bool y_bf16, bool aligned, int cus);
int64_t moe_fp4_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, bool y_bf16);
hipError_t launch_moe_fp4(const MoeFp4& p, hipStream_t stream);

// ---- FP8 in blocks of 128 with FP32 scales (quantize_b128.hip, gemm_b128*.hip).  Code lines hold 128 bytes
// per block; scales are [block][line], or [tile][block] of tiles.

// rc / rs: along rows; cc / cs: along columns (either pair may be null).  tile: one scale for each 128 x 128, in
// rs; rc as it is, cc transposed.  offsets (device, experts + 1): columns' blocks begin anew with each expert's rows.
hipError_t launch_quant_b128(const void* src, int src_bf16, int64_t rows, int64_t cols, int64_t ld_src, int fmt, int rule,
                             bool tile, uint8_t* rc, int64_t ld_rc, float* rs, int64_t ld_rs, uint8_t* cc, int64_t ld_cc,
                             float* cs, int64_t ld_cs, const int* offsets, int experts, hipStream_t stream);

// Y = act(alpha X W + bias).  mode: one matrix; the rows of each expert with its W; each expert's blocks of K.
enum : int { kB128Plain = 0, kB128Rows = 1, kB128Blocks = 2 };
struct GemmB128 {
  int mode, M, N, nb;          // nb: blocks of K; kB128Blocks: those that a line has room for
  int x_fmt, w_fmt, exact, w_line;
  const uint8_t* x;
  int64_t ld_x;
  const float* xs;             // line m, block b: xs[b ld_xs + m]
  int64_t ld_xs;
  const uint8_t* w;
  int64_t ld_w, st_w;          // st_: from one expert to the next
  const float* ws;             // line (w_line) or tile n, block b: ws[n ws_n + b ws_k]
  int64_t ws_n, ws_k, st_ws;
  const int* offsets;
  int experts, rows;           // rows: sorted lines (kB128Blocks; M where they are X's own)
  float alpha;
  const float* bias;
  int act;
  void* y;
  int y_bf16;
  int64_t ld_y, st_y;
  int past_caches;             // y is written past the caches
};
// The most tiles of tm x tn outputs that the problem may have.
int64_t gemm_b128_tiles(const GemmB128& a, int tm, int tn);
// How it runs on `cus` CUs (host logic only): its tile, and the waves that share one along K (0: a workgroup's
// waves share its tile's rows and columns, step by step).
struct GemmB128Plan {
  int tile_m, tile_n, waves;
};
GemmB128Plan gemm_b128_plan(const GemmB128& a, int cus);
hipError_t launch_gemm_b128(const GemmB128& a, hipStream_t stream);
hipError_t launch_gemm_b128_tile(const GemmB128& a, hipStream_t stream);
hipError_t launch_gemm_b128_mid(const GemmB128& a, const GemmB128Plan& p, hipStream_t stream);
hipError_t launch_gemm_b128_rows(const GemmB128& a, const GemmB128Plan& p, hipStream_t stream);

// ---- routing (moe_route.hip): experts and shares [T][k], counts [E], offsets [E + 1], order [T k], loss [1], slope [E]
struct MoeRoute {
  int64_t T, E, k;
  int renorm, bf16;
  const void* logits;
  int64_t ld_logits;
  const uint8_t* mask;
  int* experts;
  float* shares;
  int* counts;
  int* offsets;
  int* order;
  float* loss;
  float* slope;
  void* workspace;
};
int64_t moe_route_workspace_bytes(int64_t T, int64_t E, int64_t k);
hipError_t launch_moe_route(const MoeRoute& p, hipStream_t stream);
// Uses logits, mask, experts, shares and slope.
hipError_t launch_moe_route_grad(const MoeRoute& p, const float* d_shares, int64_t ld_ds, const float* d_loss, void* d,
                                 int64_t ld_d, hipStream_t stream);

}  // namespace mxq
