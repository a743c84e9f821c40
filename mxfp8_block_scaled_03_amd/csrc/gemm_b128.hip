// gemm_b128.hip -- the product in blocks of 128: how a problem runs.
#include <math.h>

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

// The plan is the cheapest of the kernels' estimates, in us, from timing all of them on 60 shapes (256 CUs, graphs of 20
// calls, other weights each; the estimates are within some 10 % of what they were fitted to):
//   small tiles  1.8 and, in rounds of a tile for each CU, 1.1 and 33 KB of both sides' lines a us (16 x 4096 x 4096
//                7.0 us by 16 x 16 and 11.0 by 64 x 32; 128 rows 31.9 and 15.3)
//   64 x 64      4 and 0.34 a block (exact 0.4, after a round of two 0.47) for one tile a CU, 0.55 (0.83) for two
//                (512 x 4096 x 4096 22.8 fp8, 128 x 128 25.1; exact 28.7 and 39.5)
//   128 x 128    5 and 0.66 (1.1) for one tile a CU, 1.2 (2.06) for two (1024 rows 27, 256 x 256 55; exact 42 and 109)
//                (experts: 2048 rows of 64 x 4096 x 2048 114, 64 x 64 117, 256 x 256 138)
//   256 x 256    5 and a round of 1.75 (3.2) a block (4096 rows 63, 128 x 128 99; up to half the CUs 1.55)
GemmB128Plan gemm_b128_plan(const GemmB128& a, int cus) {
  // (an expert's last block counts whole)
  const double nb = a.mode == kB128Blocks ? (double)a.rows / (kB * a.experts) + 0.5 : a.nb;
  // Rows of experts: of E experts E (1 - (1 - 1/E)^rows) have some, if rows choose freely; their last tiles are taken
  // to be a quarter full, since some have many more rows than others.  The weights come at 5.5 MB a us (128 rows of
  // 64 x 4096 x 2048, some 50 experts with rows: 5.9 in 72 us, as the layer's one set of weights or six in turn).
  const double E = a.experts, active = E * (1 - pow(1 - 1 / E, (double)a.M)), mean = a.M / active;
  const bool by_rows = a.mode == kB128Rows;
  auto tiles = [&](int tm, int tn) {
    if (!by_rows) return (double)gemm_b128_tiles(a, tm, tn);
    return active * fmax(1.0, mean / tm + 0.75) * (double)cover(a.N, tn);
  };
  const double memory = by_rows ? active * a.N * nb * kB / 5.5e6 : 0;
  GemmB128Plan best{};
  double least = 1e30;
  auto offer = [&](int tm, int tn, int waves, double us) {
    us = fmax(us, memory + 4);
    if (us < least) least = us, best = GemmB128Plan{tm, tn, waves};
  };
  const int small[3][2] = {{16, 16}, {32, 16}, {64, 32}};
  // (up to three rows an expert on average, whoever has them: 128 rows of 64 x 4096 x 2048 67-71 us by 16 x 64, 74 by
  // 64 x 64; 32 of 8 x 8192 x 5120, past it, 58 and 49)
  if (by_rows && a.M <= 3 * E) return {16, 64, 1};
  // the experts' weight gradients: each round's outputs too, which a large tile writes with nothing beside it
  const bool grads = a.mode == kB128Blocks;
  for (const auto& s : small)
    if (!by_rows)
      offer(s[0], s[1], 8, 1.8 + ceil(tiles(s[0], s[1]) / cus) * ((grads ? 2.1 : 1.1) + (s[0] + s[1]) * nb * kB / 33e3));
  const double t64 = tiles(64, 64), t128 = tiles(128, 128), t256 = tiles(256, 256);
  // rounds of two tiles a CU, the last of one where that is enough
  auto pairs = [&](double n, double one, double two) {
    const double whole = floor(n / (2 * cus)), rest = n - whole * 2 * cus;
    return whole * two + (rest > cus ? two : rest > 0 ? one : 0);
  };
  auto out = [&](double n, double us) { return grads ? ceil(n / (2 * cus)) * us : 0; };
  const double one64 = !a.exact ? 0.34 : t64 <= cus ? 0.4 : 0.47;
  offer(64, 64, 0, 4 + nb * pairs(t64, one64, a.exact ? 0.83 : 0.55) + out(t64, a.exact ? 0.9 : 1.2));
  offer(128, 128, 0, 5 + nb * (a.exact ? pairs(t128, 1.1, 2.06) : pairs(t128, 0.66, 1.2)) + out(t128, a.exact ? 4.0 : 4.7));
  // (W's scales by lines: a product more for each sum, 76 us instead of 63 and 131 instead of 113; experts' own blocks
  // differ in number, which a round or two of large tiles show: 16384 rows over 8 experts, exact fp32, 2048 x 1024
  // 161 us, 128 x 128 80; 4096 x 2048 280 and 303)
  const double step = a.exact ? (a.w_line ? 3.8 : 3.2) : a.w_line ? 2.15 : 2 * t256 <= cus ? 1.55 : 1.75;
  const double rounds = ceil(t256 / cus), write = grads ? 10 : 2;
  offer(256, 256, 0, (5 + rounds * (nb * step + write)) * (grads && a.experts > 1 ? 1 + 0.4 / (rounds * rounds) : 1));
  return best;
}

// Every expert's weight gradients are far more than the codes they are made from, and a program's next pass over them
// (an optimizer's) is not the next launch: past 128 MiB, half the last cache, they are written past the caches, which
// then keep the codes (16 of 4096 x 2048 in fp32 from 8192 rows 243 -> 214 us exact, 202 -> 159 fp8, and a pass over
// them right after is no slower; bf16 206 -> 200; 8 of 2048 x 1024 48 and 48, the pass 1 us slower).  A layer's
// outputs are read at once and stay (16384 x 8192 x 2048 in bf16 272 and 276 us, with a quantization of them 383 and 394).
constexpr int64_t kPastCaches = (int64_t)128 << 20;

hipError_t launch_gemm_b128(const GemmB128& given, hipStream_t stream) {
  GemmB128 a = given;
  const GemmB128Plan p = gemm_b128_plan(a, device_cu_count());
  a.past_caches = a.mode == kB128Blocks && (double)a.experts * a.M * a.N * (a.y_bf16 ? 2 : 4) > kPastCaches;
  if (p.waves != 0) return launch_gemm_b128_rows(a, p, stream);
  return p.tile_m == 256 ? launch_gemm_b128_tile(a, stream) : launch_gemm_b128_mid(a, p, stream);
}

}  // namespace mxq
