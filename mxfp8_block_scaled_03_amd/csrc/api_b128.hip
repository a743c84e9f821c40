// api_b128.hip -- the entry points for blocks of 128 and for routing (include/mxq.h): host-side argument
// validation and dispatch, on the terms of api.hip (validation before anything is enqueued, no
// synchronization, no allocation).
#include "mxq.h"

#include <math.h>

#include "b128.hpp"
#include "codec.hpp"
#include "internal.hpp"

namespace {

constexpr int64_t kMaxLines = (int64_t)1 << 30;
constexpr int64_t kMaxK = (int64_t)1 << 24;          // also the most bytes from one line of codes to the next
constexpr int64_t kMaxTiles = 0x7FFFFFFF - ((int64_t)1 << 22);
constexpr int64_t kMaxScales = (int64_t)1 << 29;     // scales of one matrix, in elements from first to last
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxChoices = 64;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
bool is_wide(int t) { return t == MXQ_F32 || t == MXQ_BF16; }
bool is_fp8(int t) { return t == MXQ_E4M3 || t == MXQ_E5M2; }
bool mul_ok(int64_t a, int64_t b) { return a == 0 || b <= INT64_MAX / a; }
int64_t blocks_of(int64_t k) { return (k + mxq::kB - 1) / mxq::kB; }
int64_t blocks_of16(int64_t n) { return (n + 15) / 16; }
int hip_status(hipError_t e) { return e == hipSuccess ? MXQ_OK : MXQ_ERR_HIP; }
int fmt_of(int elem) { return elem == MXQ_E4M3 ? mxq::kE4M3 : mxq::kE5M2; }

// Code lines of nb blocks.
int check_codes(const void* p, int64_t lines, int64_t ld, int64_t nb) {
  if (ld < mxq::kB * nb) return MXQ_ERR_LD;
  if (!mul_ok(lines, ld)) return MXQ_ERR_SHAPE;
  if (!aligned(p, 16) || ld % 16 != 0) return MXQ_ERR_ALIGN;
  return MXQ_OK;
}

// Scales of lines: [nb][ld].
int check_scales(const void* p, int64_t lines, int64_t ld, int64_t nb) {
  if (ld < lines) return MXQ_ERR_LD;
  if (!mul_ok(nb, ld)) return MXQ_ERR_SHAPE;
  if (!aligned(p, 4)) return MXQ_ERR_ALIGN;
  return MXQ_OK;
}

// What both sides of a product share: limits, formats, epilogue, pointers.
int check_product(const mxq::GemmB128& a, int64_t M, int64_t N, int64_t K, int64_t nb, int x_elem, int w_elem, int w_block,
                  int accum, int act, int y_type, int64_t scale_lines_x) {
  if (!is_fp8(x_elem) || !is_fp8(w_elem) || !is_wide(y_type)) return MXQ_ERR_DTYPE;
  if (accum != MXQ_ACC_FP8_MFMA && accum != MXQ_ACC_FP32) return MXQ_ERR_ARG;
  if (act != MXQ_ACT_NONE && act != MXQ_ACT_SILU) return MXQ_ERR_ARG;
  if (w_block != 1 && w_block != mxq::kB) return MXQ_ERR_ARG;
  if (!isfinite(a.alpha)) return MXQ_ERR_ARG;
  if (M < 0 || N < 0 || K < 0 || M >= kMaxLines || N >= kMaxLines || K >= kMaxK || nb * mxq::kB > kMaxK) return MXQ_ERR_SHAPE;
  if (M == 0 || N == 0) return MXQ_OK;
  if (!a.y || (nb > 0 && (!a.x || !a.xs || !a.w || !a.ws))) return MXQ_ERR_NULL;
  if (nb > 0) {
    if (a.ld_x >= kMaxK || a.ld_w >= kMaxK) return MXQ_ERR_LD;
    int st = check_codes(a.x, M, a.ld_x, nb);
    if (st == MXQ_OK) st = check_codes(a.w, N, a.ld_w, nb);
    if (st == MXQ_OK) st = check_scales(a.xs, scale_lines_x, a.ld_xs, nb);
    if (st != MXQ_OK) return st;
    if (a.ws_n < 0 || a.ws_k < 0) return MXQ_ERR_LD;
    if (w_block == 1 && ((N > 1 && a.ws_n != 1) || (nb > 1 && a.ws_k < N))) return MXQ_ERR_LD;
    if (!aligned(a.ws, 4)) return MXQ_ERR_ALIGN;
    const int64_t lines_w = w_block == 1 ? N : blocks_of(N);
    if (!mul_ok(nb, a.ld_xs) || nb * a.ld_xs > kMaxScales || !mul_ok(nb, a.ws_k) || !mul_ok(lines_w, a.ws_n) ||
        nb * a.ws_k > kMaxScales || lines_w * a.ws_n > kMaxScales)
      return MXQ_ERR_SHAPE;
  }
  const int64_t ey = y_type == MXQ_BF16 ? 2 : 4;
  if (a.ld_y < N) return MXQ_ERR_LD;
  if (!mul_ok(a.ld_y, ey) || !mul_ok(M, a.ld_y * ey)) return MXQ_ERR_SHAPE;
  if (!aligned(a.y, (uintptr_t)ey) || (a.bias && !aligned(a.bias, 4))) return MXQ_ERR_ALIGN;
  // the smallest tile is 16 x 16: numbers of tiles are 32-bit
  const int64_t tm = blocks_of16(M) + (a.mode == mxq::kB128Rows ? a.experts : 0);
  const int64_t times = a.mode == mxq::kB128Blocks ? a.experts : 1;
  if (tm * blocks_of16(N) > kMaxTiles / times) return MXQ_ERR_SHAPE;
  return MXQ_OK;
}

int check_experts(const int* offsets, int64_t E) {
  if (E < 1 || E > kMaxExperts) return MXQ_ERR_SHAPE;
  if (!offsets) return MXQ_ERR_NULL;
  if (!aligned(offsets, 4)) return MXQ_ERR_ALIGN;
  return MXQ_OK;
}

void fill(mxq::GemmB128& a, int64_t M, int64_t N, int64_t nb, int x_elem, int w_elem, int w_block, int accum, int act,
          int y_type) {
  a.M = (int)M;
  a.N = (int)N;
  a.nb = (int)nb;
  a.x_fmt = fmt_of(x_elem);
  a.w_fmt = fmt_of(w_elem);
  a.exact = accum == MXQ_ACC_FP32;
  a.w_line = w_block == 1;
  a.act = act == MXQ_ACT_SILU ? 1 : 0;
  a.y_bf16 = y_type == MXQ_BF16;
}

}  // namespace

extern "C" {

int mxq_quantize_b128(const void* src, int src_type, int64_t rows, int64_t cols, int64_t ld_src, int elem, int rule,
                      int tile, uint8_t* row_codes, int64_t ld_row_codes, float* row_scales, int64_t ld_row_scales,
                      uint8_t* col_codes, int64_t ld_col_codes, float* col_scales, int64_t ld_col_scales,
                      const int32_t* offsets, int64_t experts, void* stream) {
  if (!is_wide(src_type) || !is_fp8(elem)) return MXQ_ERR_DTYPE;
  if ((rule != MXQ_SCALE_AMAX && rule != MXQ_SCALE_CEIL) || (tile != 0 && tile != 1)) return MXQ_ERR_ARG;
  if (rows < 0 || cols < 0 || rows >= kMaxLines || cols >= kMaxLines) return MXQ_ERR_SHAPE;
  if (offsets) {
    if (tile) return MXQ_ERR_ARG;
    const int st = check_experts(offsets, experts);
    if (st != MXQ_OK) return st;
  }
  const bool row = row_codes != nullptr, col = col_codes != nullptr;
  if (!row && !col) return MXQ_ERR_NULL;
  if (offsets && !col) return MXQ_ERR_ARG;
  if (rows == 0 || cols == 0) return MXQ_OK;
  if (!src || (tile && !row) || (row && !row_scales) || (col && !tile && !col_scales)) return MXQ_ERR_NULL;
  const int64_t es = src_type == MXQ_BF16 ? 2 : 4;
  if (ld_src < cols) return MXQ_ERR_LD;
  if (!mul_ok(ld_src, es) || !mul_ok(rows, ld_src * es)) return MXQ_ERR_SHAPE;
  const int64_t nbc = blocks_of(cols), nbr = mxq::grouped_tiles(rows, offsets ? experts : 1, mxq::kB);
  int st = MXQ_OK;
  if (row) {
    st = check_codes(row_codes, rows, ld_row_codes, nbc);
    if (st == MXQ_OK) st = tile ? check_scales(row_scales, nbc, ld_row_scales, nbr) : check_scales(row_scales, rows, ld_row_scales, nbc);
  }
  if (col && st == MXQ_OK) st = check_codes(col_codes, cols, ld_col_codes, nbr);
  if (col && !tile && st == MXQ_OK) st = check_scales(col_scales, cols, ld_col_scales, nbr);
  if (st != MXQ_OK) return st;
  if (!aligned(src, (uintptr_t)es)) return MXQ_ERR_ALIGN;
  if (nbr * nbc > 0x7FFFFF) return MXQ_ERR_SHAPE;
  return hip_status(mxq::launch_quant_b128(src, src_type == MXQ_BF16, rows, cols, ld_src, fmt_of(elem),
                                           rule == MXQ_SCALE_CEIL ? 1 : 0, tile != 0, row_codes, ld_row_codes, row_scales,
                                           ld_row_scales, col_codes, ld_col_codes, col_scales, ld_col_scales, offsets,
                                           offsets ? (int)experts : 1, (hipStream_t)stream));
}

int mxq_gemm_b128(int64_t M, int64_t N, int64_t K, const uint8_t* x_codes, int64_t ld_x, const float* x_scales,
                  int64_t ld_xs, int x_elem, const uint8_t* w_codes, int64_t ld_w, const float* w_scales, int64_t ws_line,
                  int64_t ws_block, int w_block, int w_elem, float alpha, const float* bias, int act, int accum, void* y,
                  int y_type, int64_t ld_y, void* stream) {
  mxq::GemmB128 a{};
  a.mode = mxq::kB128Plain;
  a.x = x_codes;
  a.ld_x = ld_x;
  a.xs = x_scales;
  a.ld_xs = ld_xs;
  a.w = w_codes;
  a.ld_w = ld_w;
  a.ws = w_scales;
  a.ws_n = ws_line;
  a.ws_k = ws_block;
  a.experts = 1;
  a.alpha = alpha;
  a.bias = bias;
  a.y = y;
  a.ld_y = ld_y;
  const int st = check_product(a, M, N, K, K < 0 ? 0 : blocks_of(K), x_elem, w_elem, w_block, accum, act, y_type, M);
  if (st != MXQ_OK || M == 0 || N == 0) return st;
  fill(a, M, N, blocks_of(K), x_elem, w_elem, w_block, accum, act, y_type);
  return hip_status(mxq::launch_gemm_b128(a, (hipStream_t)stream));
}

int mxq_moe_gemm_b128(int64_t rows, int64_t N, int64_t K, int64_t E, const int32_t* offsets, const uint8_t* x_codes,
                      int64_t ld_x, const float* x_scales, int64_t ld_xs, int x_elem, const uint8_t* w_codes, int64_t ld_w,
                      int64_t expert_w, const float* w_scales, int64_t ws_line, int64_t ws_block, int64_t expert_ws,
                      int w_block, int w_elem, int accum, void* y, int y_type, int64_t ld_y, void* stream) {
  int st = check_experts(offsets, E);
  if (st != MXQ_OK) return st;
  mxq::GemmB128 a{};
  a.mode = mxq::kB128Rows;
  a.x = x_codes;
  a.ld_x = ld_x;
  a.xs = x_scales;
  a.ld_xs = ld_xs;
  a.w = w_codes;
  a.ld_w = ld_w;
  a.st_w = expert_w;
  a.ws = w_scales;
  a.ws_n = ws_line;
  a.ws_k = ws_block;
  a.st_ws = expert_ws;
  a.offsets = offsets;
  a.experts = (int)E;
  a.rows = (int)rows;
  a.alpha = 1.0f;
  a.y = y;
  a.ld_y = ld_y;
  const int64_t nb = K < 0 ? 0 : blocks_of(K);
  st = check_product(a, rows, N, K, nb, x_elem, w_elem, w_block, accum, MXQ_ACT_NONE, y_type, rows);
  if (st != MXQ_OK || rows == 0 || N == 0) return st;
  if (E > 1 && nb > 0) {
    if (expert_w < 0 || expert_ws < 0) return MXQ_ERR_LD;
    if (expert_w % 16 != 0) return MXQ_ERR_ALIGN;
    if (!mul_ok(E, expert_w) || !mul_ok(4 * E, expert_ws)) return MXQ_ERR_SHAPE;
  }
  fill(a, rows, N, nb, x_elem, w_elem, w_block, accum, MXQ_ACT_NONE, y_type);
  return hip_status(mxq::launch_gemm_b128(a, (hipStream_t)stream));
}

int mxq_moe_wgrad_b128(int64_t M, int64_t N, int64_t rows, int64_t E, const int32_t* offsets, const uint8_t* x_codes,
                       int64_t ld_x, const float* x_scales, int64_t ld_xs, int x_elem, const uint8_t* w_codes, int64_t ld_w,
                       const float* w_scales, int64_t ld_ws, int w_elem, int accum, void* y, int y_type, int64_t ld_y,
                       int64_t expert_y, void* stream) {
  int st = check_experts(offsets, E);
  if (st != MXQ_OK) return st;
  if (rows < 0 || rows >= kMaxK) return MXQ_ERR_SHAPE;
  mxq::GemmB128 a{};
  a.mode = mxq::kB128Blocks;
  a.x = x_codes;
  a.ld_x = ld_x;
  a.xs = x_scales;
  a.ld_xs = ld_xs;
  a.w = w_codes;
  a.ld_w = ld_w;
  a.ws = w_scales;
  a.ws_n = 1;
  a.ws_k = ld_ws;
  a.offsets = offsets;
  a.experts = (int)E;
  a.rows = (int)rows;
  a.alpha = 1.0f;
  a.y = y;
  a.ld_y = ld_y;
  a.st_y = expert_y;
  const int64_t nb = mxq::grouped_tiles(rows, E, mxq::kB);
  st = check_product(a, M, N, rows, nb, x_elem, w_elem, 1, accum, MXQ_ACT_NONE, y_type, M);
  if (st != MXQ_OK || M == 0 || N == 0) return st;
  if (nb > 0 && ld_ws < N) return MXQ_ERR_LD;
  if (E > 1) {
    if (expert_y < 0 || expert_y < (M - 1) * ld_y + N) return MXQ_ERR_LD;
    if (!mul_ok(4 * E, expert_y)) return MXQ_ERR_SHAPE;
  }
  fill(a, M, N, nb, x_elem, w_elem, 1, accum, MXQ_ACT_NONE, y_type);
  return hip_status(mxq::launch_gemm_b128(a, (hipStream_t)stream));
}

int mxq_gemm_b128_plan(int mode, int64_t M, int64_t N, int64_t K, int64_t E, int w_block, int accum, int cus, int* tile_m,
                       int* tile_n, int* waves) {
  if (!tile_m || !tile_n || !waves) return MXQ_ERR_NULL;
  if (mode < mxq::kB128Plain || mode > mxq::kB128Blocks || cus < 1 || (w_block != 1 && w_block != mxq::kB) ||
      (accum != MXQ_ACC_FP8_MFMA && accum != MXQ_ACC_FP32))
    return MXQ_ERR_ARG;
  if (mode == mxq::kB128Plain) E = 1;
  if (M < 1 || N < 1 || K < 0 || M >= kMaxLines || N >= kMaxLines || K >= kMaxK || E < 1 || E > kMaxExperts)
    return MXQ_ERR_SHAPE;
  mxq::GemmB128 a{};
  a.mode = mode;
  a.experts = (int)E;
  a.rows = (int)(mode == mxq::kB128Blocks ? K : M);
  a.M = (int)M;
  a.N = (int)N;
  a.nb = (int)(mode == mxq::kB128Blocks ? mxq::grouped_tiles(K, E, mxq::kB) : blocks_of(K));
  a.exact = accum == MXQ_ACC_FP32;
  a.w_line = w_block == 1;
  const mxq::GemmB128Plan p = mxq::gemm_b128_plan(a, cus);
  *tile_m = p.tile_m;
  *tile_n = p.tile_n;
  *waves = p.waves;
  return MXQ_OK;
}

static int check_route(int64_t T, int64_t E, int64_t k) {
  if (T < 0 || T >= kMaxLines || E < 1 || E > kMaxExperts) return MXQ_ERR_SHAPE;
  if (k < 1 || k > E || k > kMaxChoices) return MXQ_ERR_ARG;
  if (T * k >= kMaxLines) return MXQ_ERR_SHAPE;
  return MXQ_OK;
}

int mxq_moe_route_workspace(int64_t T, int64_t E, int64_t k, int64_t* bytes) {
  if (!bytes) return MXQ_ERR_NULL;
  const int st = check_route(T, E, k);
  if (st != MXQ_OK) return st;
  *bytes = mxq::moe_route_workspace_bytes(T, E, k);
  return MXQ_OK;
}

int mxq_moe_route(int64_t T, int64_t E, int64_t k, int renormalize, const void* logits, int logits_type, int64_t ld_logits,
                  const uint8_t* mask, int32_t* experts, float* shares, int32_t* counts, int32_t* offsets, int32_t* order,
                  float* loss, float* slope, void* workspace, int64_t workspace_bytes, void* stream) {
  const int st = check_route(T, E, k);
  if (st != MXQ_OK) return st;
  if (!is_wide(logits_type)) return MXQ_ERR_DTYPE;
  if (renormalize != 0 && renormalize != 1) return MXQ_ERR_ARG;
  const int64_t need = mxq::moe_route_workspace_bytes(T, E, k);
  if (!counts || !offsets || !loss || !slope || (T > 0 && (!logits || !experts || !shares || !order)) ||
      (need > 0 && !workspace))
    return MXQ_ERR_NULL;
  const int64_t es = logits_type == MXQ_BF16 ? 2 : 4;
  if (ld_logits < E) return MXQ_ERR_LD;
  if (!mul_ok(ld_logits, es) || !mul_ok(T, ld_logits * es)) return MXQ_ERR_SHAPE;
  if (!aligned(logits, (uintptr_t)es) || !aligned(experts, 4) || !aligned(shares, 4) || !aligned(counts, 4) ||
      !aligned(offsets, 4) || !aligned(order, 4) || !aligned(loss, 4) || !aligned(slope, 4) ||
      (need > 0 && !aligned(workspace, 256)))
    return MXQ_ERR_ALIGN;
  if (workspace_bytes < need) return MXQ_ERR_SCRATCH;
  mxq::MoeRoute p{};
  p.T = T;
  p.E = E;
  p.k = k;
  p.renorm = renormalize;
  p.bf16 = logits_type == MXQ_BF16;
  p.logits = logits;
  p.ld_logits = ld_logits;
  p.mask = mask;
  p.experts = experts;
  p.shares = shares;
  p.counts = counts;
  p.offsets = offsets;
  p.order = order;
  p.loss = loss;
  p.slope = slope;
  p.workspace = workspace;
  return hip_status(mxq::launch_moe_route(p, (hipStream_t)stream));
}

int mxq_moe_route_grad(int64_t T, int64_t E, int64_t k, int renormalize, const void* logits, int logits_type,
                       int64_t ld_logits, const uint8_t* mask, const int32_t* experts, const float* shares,
                       const float* slope, const float* d_shares, int64_t ld_d_shares, const float* d_loss, void* d_logits,
                       int64_t ld_d_logits, void* stream) {
  const int st = check_route(T, E, k);
  if (st != MXQ_OK) return st;
  if (!is_wide(logits_type)) return MXQ_ERR_DTYPE;
  if (renormalize != 0 && renormalize != 1) return MXQ_ERR_ARG;
  if (T == 0) return MXQ_OK;
  if (!logits || !d_logits || (d_shares && (!experts || !shares)) || (d_loss && !slope)) return MXQ_ERR_NULL;
  const int64_t es = logits_type == MXQ_BF16 ? 2 : 4;
  if (ld_logits < E || ld_d_logits < E || (d_shares && ld_d_shares < k)) return MXQ_ERR_LD;
  if (!mul_ok(ld_logits, es) || !mul_ok(T, ld_logits * es) || !mul_ok(ld_d_logits, es) || !mul_ok(T, ld_d_logits * es) ||
      (d_shares && (!mul_ok(ld_d_shares, 4) || !mul_ok(T, ld_d_shares * 4))))
    return MXQ_ERR_SHAPE;
  if (!aligned(logits, (uintptr_t)es) || !aligned(d_logits, (uintptr_t)es) || !aligned(experts, 4) || !aligned(shares, 4) ||
      !aligned(slope, 4) || !aligned(d_shares, 4) || !aligned(d_loss, 4))
    return MXQ_ERR_ALIGN;
  mxq::MoeRoute p{};
  p.T = T;
  p.E = E;
  p.k = k;
  p.renorm = renormalize;
  p.bf16 = logits_type == MXQ_BF16;
  p.logits = logits;
  p.ld_logits = ld_logits;
  p.mask = mask;
  p.experts = const_cast<int32_t*>(experts);
  p.shares = const_cast<float*>(shares);
  p.slope = const_cast<float*>(slope);
  return hip_status(mxq::launch_moe_route_grad(p, d_shares, ld_d_shares, d_loss, d_logits, ld_d_logits, (hipStream_t)stream));
}

}  // extern "C"
