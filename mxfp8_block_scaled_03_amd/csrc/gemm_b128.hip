// gemm_b128.hip -- the product in blocks of 128: how a problem runs.
#include "b128.hpp"
#include "internal.hpp"

namespace mxq {
namespace {

int64_t cover(int64_t n, int64_t size) { return (n + size - 1) / size; }

}  // namespace

int64_t gemm_b128_tiles(const GemmB128& a, int tm, int tn) {
  const int64_t n = cover(a.N, tn);
  if (a.mode == kB128Rows) return n * grouped_tiles(a.M, a.experts, tm);
  return n * cover(a.M, tm) * (a.mode == kB128Blocks ? a.experts : 1);
}

GemmB128Plan gemm_b128_plan(const GemmB128& a, int cus) {
  const int64_t rows = a.mode == kB128Rows ? cover(a.M, a.experts) : a.M;
  if (a.mode == kB128Rows && rows <= 64) return rows <= 12 ? GemmB128Plan{16, 64, 1} : rows <= 24 ? GemmB128Plan{32, 64, 1} : GemmB128Plan{64, 64, 1};
  if (rows <= 16) return {16, 16, 8};
  if (rows <= 32) return {32, 16, 8};
  const int64_t tiles = gemm_b128_tiles(a, 256, 256);
  if (rows > 64 && 5 * tiles >= 2 * cus) return {256, 256, 0};
  return rows <= 64 ? GemmB128Plan{64, 32, 8} : GemmB128Plan{64, 64, 8};
}

hipError_t launch_gemm_b128(const GemmB128& a, hipStream_t stream) {
  const GemmB128Plan p = gemm_b128_plan(a, device_cu_count());
  return p.waves == 0 ? launch_gemm_b128_tile(a, stream) : launch_gemm_b128_rows(a, p, stream);
}

}  // namespace mxq
