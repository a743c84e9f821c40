// api_fp4.hip -- the MXFP4 entry points of include/mxq.h: host-side argument validation and
// dispatch, on the terms of api.hip (validation before anything is enqueued, no
// synchronization, no allocation).
#include "mxq.h"

#include <math.h>

#include "codec.hpp"
#include "internal.hpp"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxK = (int64_t)1 << 24;
constexpr int64_t kMaxMoeTokens = 1024;
constexpr int64_t kMaxExperts = 1024;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
bool is_wide(int t) { return t == MXQ_F32 || t == MXQ_BF16; }
bool mul_ok(int64_t a, int64_t b) { return a == 0 || b <= INT64_MAX / a; }
int64_t blocks_of(int64_t k) { return (k + 31) / 32; }
int hip_status(hipError_t e) { return e == hipSuccess ? MXQ_OK : MXQ_ERR_HIP; }

// A code array of L lines: 16 bytes per block, 16-byte aligned.
int check_codes(const void* p, int64_t L, int64_t ld, int64_t ld_scales, int64_t nb) {
  if (ld < 16 * nb || ld_scales < nb) return MXQ_ERR_LD;
  if (!mul_ok(L, ld) || !mul_ok(L, ld_scales)) return MXQ_ERR_SHAPE;
  if (!aligned(p, 16) || ld % 16 != 0) return MXQ_ERR_ALIGN;
  return MXQ_OK;
}

int quantize(const void* src, int src_type, int64_t rows, int64_t cols, int64_t ld_src, int axis, int rule, bool sr,
             uint64_t seed, uint8_t* codes, int64_t ld_codes, uint8_t* scales, int64_t ld_scales, void* stream) {
  if (!is_wide(src_type)) return MXQ_ERR_DTYPE;
  if (axis != MXQ_ROWWISE && axis != MXQ_COLWISE) return MXQ_ERR_ARG;
  if (rule != MXQ_SCALE_CEIL && rule != MXQ_SCALE_OCP) return MXQ_ERR_ARG;
  if (rows < 0 || cols < 0 || rows >= kMaxDim || cols >= kMaxDim) return MXQ_ERR_SHAPE;
  const int64_t L = axis == MXQ_ROWWISE ? rows : cols, K = axis == MXQ_ROWWISE ? cols : rows;
  if (L == 0 || K == 0) return MXQ_OK;
  if (!src || !codes || !scales) return MXQ_ERR_NULL;
  const int64_t es = src_type == MXQ_BF16 ? 2 : 4;
  if (ld_src < cols) return MXQ_ERR_LD;
  if (!mul_ok(ld_src, es) || !mul_ok(rows, ld_src * es)) return MXQ_ERR_SHAPE;
  const int st = check_codes(codes, L, ld_codes, ld_scales, blocks_of(K));
  if (st != MXQ_OK) return st;
  if (!aligned(src, (uintptr_t)es)) return MXQ_ERR_ALIGN;
  return hip_status(mxq::launch_quant4(src, src_type == MXQ_BF16, rows, cols, ld_src, axis == MXQ_COLWISE,
                                       rule == MXQ_SCALE_OCP ? mxq::kRuleOcp : mxq::kRuleCeil, sr, seed, codes,
                                       ld_codes, scales, ld_scales, (hipStream_t)stream));
}

}  // namespace

extern "C" {

int mxq_quantize_fp4(const void* src, int src_type, int64_t rows, int64_t cols, int64_t ld_src, int axis, int rule,
                     uint8_t* codes, int64_t ld_codes, uint8_t* scales, int64_t ld_scales, void* stream) {
  return quantize(src, src_type, rows, cols, ld_src, axis, rule, false, 0, codes, ld_codes, scales, ld_scales, stream);
}

int mxq_quantize_fp4_sr(const void* src, int src_type, int64_t rows, int64_t cols, int64_t ld_src, int axis,
                        uint64_t seed, uint8_t* codes, int64_t ld_codes, uint8_t* scales, int64_t ld_scales,
                        void* stream) {
  return quantize(src, src_type, rows, cols, ld_src, axis, MXQ_SCALE_CEIL, true, seed, codes, ld_codes, scales,
                  ld_scales, stream);
}

int mxq_quantize_fp4_dual(const void* src, int src_type, int64_t rows, int64_t cols, int64_t ld_src,
                          uint8_t* row_codes, int64_t ld_row_codes, uint8_t* row_scales, int64_t ld_row_scales,
                          uint8_t* col_codes, int64_t ld_col_codes, uint8_t* col_scales, int64_t ld_col_scales,
                          void* stream) {
  if (!is_wide(src_type)) return MXQ_ERR_DTYPE;
  if (rows < 0 || cols < 0 || rows >= kMaxDim || cols >= kMaxDim) return MXQ_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MXQ_OK;
  if (!src || !row_codes || !row_scales || !col_codes || !col_scales) return MXQ_ERR_NULL;
  const int64_t es = src_type == MXQ_BF16 ? 2 : 4;
  if (ld_src < cols) return MXQ_ERR_LD;
  if (!mul_ok(ld_src, es) || !mul_ok(rows, ld_src * es)) return MXQ_ERR_SHAPE;
  int st = check_codes(row_codes, rows, ld_row_codes, ld_row_scales, blocks_of(cols));
  if (st == MXQ_OK) st = check_codes(col_codes, cols, ld_col_codes, ld_col_scales, blocks_of(rows));
  if (st != MXQ_OK) return st;
  if (!aligned(src, (uintptr_t)es)) return MXQ_ERR_ALIGN;
  return hip_status(mxq::launch_quant4_dual(src, src_type == MXQ_BF16, rows, cols, ld_src, row_codes, ld_row_codes,
                                            row_scales, ld_row_scales, col_codes, ld_col_codes, col_scales,
                                            ld_col_scales, (hipStream_t)stream));
}

int mxq_dequantize_fp4(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales, int64_t L,
                       int64_t K, void* dst, int dst_type, int64_t ld_dst, void* stream) {
  if (!is_wide(dst_type)) return MXQ_ERR_DTYPE;
  if (L < 0 || K < 0 || L >= kMaxDim || K >= kMaxDim) return MXQ_ERR_SHAPE;
  if (L == 0 || K == 0) return MXQ_OK;
  if (!codes || !scales || !dst) return MXQ_ERR_NULL;
  const int64_t es = dst_type == MXQ_BF16 ? 2 : 4;
  if (ld_dst < K) return MXQ_ERR_LD;
  if (!mul_ok(ld_dst, es) || !mul_ok(L, ld_dst * es)) return MXQ_ERR_SHAPE;
  const int st = check_codes(codes, L, ld_codes, ld_scales, blocks_of(K));
  if (st != MXQ_OK) return st;
  if (!aligned(dst, (uintptr_t)es)) return MXQ_ERR_ALIGN;
  return hip_status(mxq::launch_dequant4(codes, ld_codes, scales, ld_scales, L, K, dst, dst_type == MXQ_BF16, ld_dst,
                                         (hipStream_t)stream));
}

int mxq_gemm_fp4(int64_t M, int64_t N, int64_t K, const void* x, int x_type, int64_t ld_x, const uint8_t* x_scales,
                 int64_t ld_xs, const uint8_t* w_codes, int64_t ld_w, const uint8_t* w_scales, int64_t ld_ws,
                 float alpha, const float* bias, int act, void* y, int y_type, int64_t ld_y, void* stream) {
  if ((x_type != MXQ_BF16 && x_type != MXQ_E2M1) || !is_wide(y_type)) return MXQ_ERR_DTYPE;
  if (act != MXQ_ACT_NONE && act != MXQ_ACT_SILU) return MXQ_ERR_ARG;
  if (M < 0 || N < 0 || K < 0 || M >= kMaxDim || N >= kMaxDim || K >= kMaxK) return MXQ_ERR_SHAPE;
  if (!isfinite(alpha)) return MXQ_ERR_ARG;
  if (M == 0 || N == 0) return MXQ_OK;
  const bool x_fp4 = x_type == MXQ_E2M1;
  const int64_t nb = blocks_of(K);
  if (!y || (K > 0 && (!x || !w_codes || !w_scales || (x_fp4 && !x_scales)))) return MXQ_ERR_NULL;
  if (K > 0) {
    if (ld_w >= kMaxK || ld_ws >= kMaxK || ld_x >= (x_fp4 ? kMaxK : kMaxDim) || ld_xs >= (x_fp4 ? kMaxK : INT64_MAX))
      return MXQ_ERR_LD;
    int st = check_codes(w_codes, N, ld_w, ld_ws, nb);
    if (st == MXQ_OK && x_fp4) st = check_codes(x, M, ld_x, ld_xs, nb);
    if (st != MXQ_OK) return st;
    if (!x_fp4) {
      if (ld_x < K) return MXQ_ERR_LD;
      if (!aligned(x, 2)) return MXQ_ERR_ALIGN;
      if (!mul_ok(M, 2 * ld_x)) return MXQ_ERR_SHAPE;
    }
  }
  const int64_t ey = y_type == MXQ_BF16 ? 2 : 4;
  if (ld_y < N) return MXQ_ERR_LD;
  if (!mul_ok(ld_y, ey) || !mul_ok(M, ld_y * ey)) return MXQ_ERR_SHAPE;
  if (!aligned(y, (uintptr_t)ey) || (bias && !aligned(bias, 4))) return MXQ_ERR_ALIGN;
  mxq::GemmEpilogue ep{};
  ep.alpha = alpha;
  ep.bias = bias;
  ep.act = act == MXQ_ACT_SILU ? 1 : 0;
  ep.y = y;
  ep.y_bf16 = y_type == MXQ_BF16;
  ep.ld_y = ld_y;
  ep.y_vec16 = aligned(y, 16) && (ld_y * ey) % 16 == 0;
  return hip_status(mxq::launch_gemm_fp4(M, N, K, x, x_fp4, ld_x, x_scales, ld_xs, w_codes, ld_w, w_scales, ld_ws, ep,
                                         (hipStream_t)stream));
}

int mxq_gemm_fp4_plan(int64_t M, int64_t N, int64_t K, int x_type, int aligned, int cus, int* tile_m, int* tile_n,
                      int* waves) {
  if (!tile_m || !tile_n || !waves) return MXQ_ERR_NULL;
  if (x_type != MXQ_BF16 && x_type != MXQ_E2M1) return MXQ_ERR_DTYPE;
  if (M < 1 || N < 1 || K < 0 || M >= kMaxDim || N >= kMaxDim || K >= kMaxK) return MXQ_ERR_SHAPE;
  if (cus < 1 || (aligned != 0 && aligned != 1)) return MXQ_ERR_ARG;
  const mxq::GemmFp4Plan p = mxq::gemm_fp4_plan(M, N, K, x_type == MXQ_E2M1, aligned != 0, cus);
  *tile_m = p.tile_m;
  *tile_n = p.tile_n;
  *waves = p.waves;
  return MXQ_OK;
}

int mxq_moe_fp4_plan(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int y_type, int aligned, int cus,
                     int* launches, int* up_columns, int* down_columns, int* down_parts) {
  if (!launches || !up_columns || !down_columns || !down_parts) return MXQ_ERR_NULL;
  if (!is_wide(y_type)) return MXQ_ERR_DTYPE;
  if (T < 1 || T > kMaxMoeTokens || H < 1 || H >= kMaxK || I < 1 || I >= kMaxK || E < 1 || E > kMaxExperts)
    return MXQ_ERR_SHAPE;
  if (k < 1 || k > E || cus < 1 || (aligned != 0 && aligned != 1)) return MXQ_ERR_ARG;
  const mxq::MoeFp4Plan p = mxq::moe_fp4_plan(T, H, I, E, k, y_type == MXQ_BF16, aligned != 0, cus);
  *launches = p.launches;
  *up_columns = p.up_columns;
  *down_columns = p.down_columns;
  *down_parts = p.down_parts;
  return MXQ_OK;
}

int mxq_moe_fp4_workspace(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int y_type, int64_t* bytes) {
  if (!bytes) return MXQ_ERR_NULL;
  if (!is_wide(y_type)) return MXQ_ERR_DTYPE;
  if (T < 0 || T > kMaxMoeTokens || H < 0 || H >= kMaxK || I < 0 || I >= kMaxK || E < 1 || E > kMaxExperts)
    return MXQ_ERR_SHAPE;
  if (k < 1 || k > E) return MXQ_ERR_ARG;
  *bytes = T == 0 || H == 0 ? 0 : mxq::moe_fp4_workspace_bytes(T, H, I, E, k, y_type == MXQ_BF16);
  return MXQ_OK;
}

int mxq_moe_fp4(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int renormalize, const void* x, int64_t ld_x,
                const float* logits, int64_t ld_logits, const uint8_t* w13_codes, int64_t ld_w13,
                int64_t expert_w13, const uint8_t* w13_scales, int64_t ld_s13, int64_t expert_s13,
                const uint8_t* w2_codes, int64_t ld_w2, int64_t expert_w2, const uint8_t* w2_scales, int64_t ld_s2,
                int64_t expert_s2, void* y, int y_type, int64_t ld_y, void* workspace, int64_t workspace_bytes,
                void* stream) {
  int64_t need = 0;
  int st = mxq_moe_fp4_workspace(T, H, I, E, k, y_type, &need);
  if (st != MXQ_OK) return st;
  if (renormalize != 0 && renormalize != 1) return MXQ_ERR_ARG;
  if (T == 0 || H == 0) return MXQ_OK;
  if (I == 0) return MXQ_ERR_SHAPE;
  if (!x || !logits || !w13_codes || !w13_scales || !w2_codes || !w2_scales || !y || !workspace) return MXQ_ERR_NULL;
  const int64_t ey = y_type == MXQ_BF16 ? 2 : 4;
  if (ld_x < H || ld_logits < E || ld_y < H) return MXQ_ERR_LD;
  if (ld_x >= kMaxDim || ld_logits >= kMaxDim || ld_y >= kMaxDim) return MXQ_ERR_LD;
  st = check_codes(w13_codes, 2 * I, ld_w13, ld_s13, blocks_of(H));
  if (st == MXQ_OK) st = check_codes(w2_codes, H, ld_w2, ld_s2, blocks_of(I));
  if (st != MXQ_OK) return st;
  // row tiles are reached with 32-bit offsets; a gate row and its up row, which have 64-bit addresses, are kept
  // within 4 GiB all the same, as the contract says
  if (ld_w13 >= kMaxK || ld_w2 >= kMaxK || ld_s13 >= kMaxK || ld_s2 >= kMaxK) return MXQ_ERR_LD;
  if ((I + 128) * ld_w13 > 0xFFFFFFFFll || (I + 128) * ld_s13 > 0xFFFFFFFFll) return MXQ_ERR_SHAPE;
  if (expert_w13 < (E > 1 ? 2 * I * ld_w13 : 0) || expert_w2 < (E > 1 ? H * ld_w2 : 0)) return MXQ_ERR_LD;
  if (E > 1 && (expert_s13 < (2 * I - 1) * ld_s13 + blocks_of(H) || expert_s2 < (H - 1) * ld_s2 + blocks_of(I)))
    return MXQ_ERR_LD;
  if (!mul_ok(E, expert_w13) || !mul_ok(E, expert_w2) || !mul_ok(E, expert_s13) || !mul_ok(E, expert_s2))
    return MXQ_ERR_SHAPE;
  if (!aligned(x, 2) || !aligned(logits, 4) || !aligned(y, (uintptr_t)ey) || expert_w13 % 16 != 0 ||
      expert_w2 % 16 != 0 || !aligned(workspace, 256))
    return MXQ_ERR_ALIGN;
  if (workspace_bytes < need) return MXQ_ERR_SCRATCH;
  mxq::MoeFp4 p{};
  p.T = T;
  p.H = H;
  p.I = I;
  p.E = E;
  p.k = k;
  p.renorm = renormalize != 0;
  p.x = x;
  p.ld_x = ld_x;
  p.logits = logits;
  p.ld_logits = ld_logits;
  p.w13 = w13_codes;
  p.ld_w13 = ld_w13;
  p.st_w13 = expert_w13;
  p.s13 = w13_scales;
  p.ld_s13 = ld_s13;
  p.st_s13 = expert_s13;
  p.w2 = w2_codes;
  p.ld_w2 = ld_w2;
  p.st_w2 = expert_w2;
  p.s2 = w2_scales;
  p.ld_s2 = ld_s2;
  p.st_s2 = expert_s2;
  p.y = y;
  p.ld_y = ld_y;
  p.y_bf16 = y_type == MXQ_BF16;
  p.workspace = workspace;
  return hip_status(mxq::launch_moe_fp4(p, (hipStream_t)stream));
}

}  // extern "C"
