// moe_fp4.hip -- a mixture-of-experts layer for a few tokens with MXFP4 weights, for gfx950.
//
//   p = softmax(logits);  the k largest p of a token choose its experts (ties to the lower
//   index), their shares optionally renormalized to sum 1;
//   h = share * silu(x W1_e) * (x W3_e)      (gate rows [0, I) and up rows [I, 2I) of w13[e])
//   y = sum over the token's experts, in the order of their rank, of h W2_e
//
// Where hardly an expert has two tokens: two launches (moe_fp4_few.hip).  Otherwise four:
// k_moe_route (ranks and shares, one wave a token), k_moe_up (gate and up products, h),
// k_moe_down (down products, one partial row per token and expert), k_moe_sum (the sum of a
// token's rows).  The weights of every expert that a token chose are read once and bound the
// time (fp4_stream.hpp); everything else is kept out of their way: a workgroup finds the tokens
// of its expert with one ballot, h goes to memory in the fragment order that k_moe_down reads, and
// the workgroups of experts that nobody chose end at once.
//
// An expert with logit -inf is never taken: its share is zero, and a token whose logits are
// all -inf gets y = 0.  NaN logits order above +inf; their shares are NaN, as softmax's.
#include <math.h>

#include "moe_fp4.hpp"

namespace mxq {
namespace {

// ---- routing: a wave a token, which takes its experts one maximum after the other.  share = exp(l - max)
// over the sum of the chosen experts' exponentials (renorm) or of all.
template <int KEYS>
__global__ __launch_bounds__(kThreads) void k_moe_route(const MoeArgs a) {
  const int t = blockIdx.x * kWaves + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= a.T) return;                                  // the whole wave
  Logits<KEYS> lg;
  lg.load(a, t, lane);
  const float top = lg.top();
  int rank[KEYS];
#pragma unroll
  for (int q = 0; q < KEYS; ++q) rank[q] = -1;
  bool left = true;
  for (int r = 0; r < a.k; ++r) {
    const int e = left ? lg.take(lane) : -1;
    left = e >= 0;
    if (lane == 0) a.chosen[t * a.k + r] = e;
#pragma unroll
    for (int q = 0; q < KEYS; ++q)
      if (e == 64 * q + lane) rank[q] = r;
  }
  float p[KEYS], sum = 0.0f;
#pragma unroll
  for (int q = 0; q < KEYS; ++q) {
    p[q] = expf(lg.l[q] - top);
    if (a.renorm ? rank[q] >= 0 : 64 * q + lane < a.E) sum += p[q];
  }
  sum = wave_sum(sum);
#pragma unroll
  for (int q = 0; q < KEYS; ++q) {
    const int j = 64 * q + lane;
    if (j < a.E) a.rank[(int64_t)j * a.T + t] = (int16_t)rank[q];
    if (rank[q] >= 0) a.share[t * a.k + rank[q]] = p[q] / sum;
  }
}

// The work of a workgroup: neighbours on one XCD where every slot has some; dealt round where many
// slots may have none, whose XCDs would be left idle.
__device__ __forceinline__ int work_of(const MoeArgs& a, int wg) {
  return a.by_token ? wg : xcd_order(wg, a.slots * a.tiles);
}

// The expert of a slot, or -1.
__device__ __forceinline__ int slot_expert(const MoeArgs& a, int slot) { return a.by_token ? a.chosen[slot] : slot; }

// The tokens of a slot's expert e, in order: s_row[m] = t * k + rank.  Returns their number, 0
// where there is nothing to do: no token, or (by_token) an earlier token's slot has the expert
// already.  Holds a barrier.
__device__ __forceinline__ int slot_tokens(const MoeArgs& a, int slot, int e, int* s_row, int* s_cnt) {
  const int lane = threadIdx.x & 63;
  if (threadIdx.x < 64) {
    int cnt = 0;
    for (int t0 = 0; t0 < a.T; t0 += 64) {
      const int t = t0 + lane;
      const int r = t < a.T ? a.rank[(int64_t)e * a.T + t] : -1;
      const uint64_t b = __ballot(r >= 0);
      if (r >= 0) s_row[cnt + __popcll(b & ((1ull << lane) - 1))] = t * a.k + r;
      cnt += __popcll(b);
    }
    if (lane == 0) *s_cnt = cnt;
  }
  __syncthreads();
  const int cnt = *s_cnt;
  return cnt > 0 && a.by_token && s_row[0] != slot ? 0 : cnt;
}

// ---- gate and up products.  A workgroup: one slot, 8 * NTW columns of I: row tiles
// 0 .. NTW/2-1 of its 16 * NTW rows of w13 are gate rows, the others the up rows.
template <int NTW, int KIND>
__global__ __launch_bounds__(kThreads, 2) void k_moe_up(const MoeArgs a) {
  constexpr int IC = 8 * NTW, NG = NTW / 2;
  int* s_row = reinterpret_cast<int*>(smem + stream_lds<1, NTW>());
  __shared__ int s_cnt;
  const int wg = workgroup_at(blockIdx.x, blockIdx.y);
  if (blockIdx.y > 0 && wg >= a.slots * a.tiles) return;
  const int work = work_of(a, wg), slot = work / a.tiles, tile = work % a.tiles;
  const int lane = threadIdx.x & 63, i = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = slot_expert(a, slot);
  if (e < 0) return;
  const int i0 = tile * IC, nb = (a.H + 31) / 32;
  const int rows = min(IC, a.I - i0);
  const uint8_t* w = a.w13 + e * a.st_w13 + i0 * a.ld_w13;
  const uint8_t* s = a.s13 + e * a.st_s13 + i0 * a.ld_s13;
  Lines l = lines_of(w, a.ld_w13, s, a.ld_s13, rows, nb, a.s13_words);
  l.first = NG;
  l.far_c = (uint64_t)(a.I * a.ld_w13);
  l.far_s = (uint64_t)(a.I * a.ld_s13);
  const ItemOffsets wo = item_offsets(l.ld_c, l.ld_s, lane);
  const uint32_t ring = (uint32_t)wave * kWaveLds, lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)smem + ring;
  const int chunks = (a.I + kChunk - 1) / kChunk;
  const Run run = run_of<NTW>(a.H, wave);
  auto issue = [&](int t, int c, uint32_t lds) { issue_item(l, wo, t, c, lds); };
  // few tokens come straight into registers, and the first weights are on their way while they
  // are looked up; more pass through the ring a chunk at a time
  const bool through = a.T <= 4 || a.T * a.k <= 2 * a.E || !a.x_pieces;
  if (through) fill_ring<NTW>(run.it0, run.it1, lds0, issue);
  const int cnt = slot_tokens(a, slot, e, s_row, &s_cnt);
  if (cnt == 0) {
    wait_vm<0>();
    return;
  }
  for (int m0 = 0; m0 < cnt; m0 += 16) {
    if (m0 > 0) {
      __syncthreads();
      if (through) fill_ring<NTW>(run.it0, run.it1, lds0, issue);
    }
    v4f acc[1][NTW];
#pragma unroll
    for (int n = 0; n < NTW; ++n) acc[0][n] = {0.0f, 0.0f, 0.0f, 0.0f};
    const uint8_t* row = a.x + (int64_t)(s_row[min(m0 + i, cnt - 1)] / a.k) * a.ld_x;
    stream<XWide<1, 1>, 1, NTW>(
        run, wave, lane, a.s13_words, through, issue,
        [&](XWide<1, 1>& x, int c) {
          const int left = a.H - kChunk * c;
          if (through || left < kChunk) {
            x.load_direct(0, row + 2 * kChunk * (int64_t)c, m0 + i < cnt, left, a.H, lane);
          } else {
            stage_rows((uint64_t)(uintptr_t)row, min(16, cnt - m0), c, lds0, lane);
            wait_vm<0>();
            asm volatile("" ::: "memory");
            x.read_staged(0, ring, lane);
            reads_done();
          }
        },
        [&](int t, int c, uint32_t slot_at) { return item_scales(l, slot_at, t, c, nb, lane); }, acc);
    __syncthreads();
    store_part<1, NTW>(wave, lane, acc);
    __syncthreads();
    for (int q = threadIdx.x; q < 16 * (IC / 8); q += kThreads) {
      const int m = q / (IC / 8), c = 8 * (q % (IC / 8));
      if (m0 + m >= cnt || i0 + c >= a.I) continue;
      const float share = a.share[s_row[m0 + m]];
      const int k = i0 + c;
      uint8_t* dst = a.h + (((int64_t)slot * a.mt_cap + m0 / 16) * chunks) * hidden_chunk(KIND) + h_offset<KIND>(m, k);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const v4f gt = sum_part<1, NTW>(m, c + 4 * hf), u = sum_part<1, NTW>(m, IC + c + 4 * hf);
        float v[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) v[p] = k + 4 * hf + p < a.I ? gated(share, gt[p], u[p]) : 0.0f;   // zeros past I
        store_hidden<KIND>(dst, hf, v);
      }
    }
  }
}

// ---- down products.  A workgroup: one slot, 16 * NTW columns of H; h comes in fragment order.
template <int NTW, int KIND>
__global__ __launch_bounds__(kThreads, 2) void k_moe_down(const MoeArgs a) {
  int* s_row = reinterpret_cast<int*>(smem + stream_lds<1, NTW>());
  __shared__ int s_cnt;
  const int wg = workgroup_at(blockIdx.x, blockIdx.y);
  if (blockIdx.y > 0 && wg >= a.slots * a.tiles) return;
  const int work = work_of(a, wg), slot = work / a.tiles, tile = work % a.tiles;
  const int lane = threadIdx.x & 63, i = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = slot_expert(a, slot);
  if (e < 0) return;
  const int n0 = 16 * NTW * tile, nb = (a.I + 31) / 32;
  const Lines w = lines_of(a.w2 + e * a.st_w2 + n0 * a.ld_w2, a.ld_w2, a.s2 + e * a.st_s2 + n0 * a.ld_s2, a.ld_s2,
                           min(16 * NTW, a.H - n0), nb, a.s2_words);
  const ItemOffsets wo = item_offsets(w.ld_c, w.ld_s, lane);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)smem + (uint32_t)wave * kWaveLds;
  const int chunks = (a.I + kChunk - 1) / kChunk;
  const Run run = run_of<NTW>(a.I, wave);
  auto issue = [&](int t, int c, uint32_t lds) { issue_item(w, wo, t, c, lds); };
  fill_ring<NTW>(run.it0, run.it1, lds0, issue);
  const int cnt = slot_tokens(a, slot, e, s_row, &s_cnt);
  if (cnt == 0) {
    wait_vm<0>();
    return;
  }
  for (int m0 = 0; m0 < cnt; m0 += 16) {
    if (m0 > 0) {
      __syncthreads();
      fill_ring<NTW>(run.it0, run.it1, lds0, issue);
    }
    const uint8_t* h = a.h + ((int64_t)slot * a.mt_cap + m0 / 16) * chunks * hidden_chunk(KIND) + 16 * lane;
    v4f acc[1][NTW];
#pragma unroll
    for (int n = 0; n < NTW; ++n) acc[0][n] = {0.0f, 0.0f, 0.0f, 0.0f};
    stream<XWide<1, KIND>, 1, NTW>(
        run, wave, lane, a.s2_words, true, issue,
        [&](XWide<1, KIND>& x, int c) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int p = 0; p < KIND; ++p)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                // rows past the last token and elements past I have nothing in h
                const int k = kChunk * c + 32 * (4 * (lane >> 4) + u) + 8 * j;
                v4i v = {0, 0, 0, 0};
                if (k < a.I && m0 + i < cnt)
                  v = *reinterpret_cast<const v4i*>(h + (((int64_t)4 * c + u) * KIND + p) * 4096 + 1024 * j);
                x.f[u][j][0][p] = v;
              }
        },
        [&](int t, int c, uint32_t slot_at) { return item_scales(w, slot_at, t, c, nb, lane); }, acc);
    __syncthreads();
    store_part<1, NTW>(wave, lane, acc);
    __syncthreads();
    for (int q = threadIdx.x; q < 16 * 4 * NTW; q += kThreads) {
      const int m = q / (4 * NTW), n = 4 * (q % (4 * NTW));
      if (m0 + m >= cnt || n0 + n >= a.H) continue;
      const v4f v = sum_part<1, NTW>(m, n);
      float* p = a.part + (int64_t)s_row[m0 + m] * a.H + n0 + n;
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (n0 + n + x < a.H) p[x] = v[x];
    }
  }
}

// ---- y[t] = sum of the token's rows, in the order of rank; masked experts, which come last,
// have none.  Four columns a thread, four rows on their way at a time (a column and a row at a time: 6.6
// us against 5.1 for 16 tokens of 5120 columns).
__global__ __launch_bounds__(64) void k_moe_sum(const MoeArgs a) {
  const int t = blockIdx.y, n = 4 * (blockIdx.x * 64 + threadIdx.x);
  int kept = 0;
  for (int r = 0; r < a.k; ++r) kept += a.chosen[t * a.k + r] >= 0 ? 1 : 0;
  if (n >= a.H) return;
  const float* part = a.part + (int64_t)t * a.k * a.parts * a.H + n;
  const int rows = kept * a.parts, cols = min(4, a.H - n);
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int r0 = 0; r0 < rows; r0 += 4) {
    float v[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float* row = part + (int64_t)min(r0 + r, rows - 1) * a.H;
      if (cols == 4) {
        __builtin_memcpy(v[r], row, 16);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[r][e] = row[min(e, cols - 1)];
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (r0 + r < rows) s[e] += v[r][e];
  }
  if (a.y_bf16) {
    uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + t * a.ld_y + n;
    const uint32_t d[2] = {pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3])};
    if (cols == 4) {
      __builtin_memcpy(y, d, 8);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < cols) y[e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
    }
  } else {
    float* y = reinterpret_cast<float*>(a.y) + t * a.ld_y + n;
    if (cols == 4) {
      __builtin_memcpy(y, s, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < cols) y[e] = s[e];
    }
  }
}

template <int NTW, int KIND>
hipError_t launch_up(MoeArgs a, hipStream_t st) {
  static bool set[64] = {false};
  a.tiles = (a.I + 8 * NTW - 1) / (8 * NTW);
  if ((int64_t)a.slots * a.tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  auto kern = k_moe_up<NTW, KIND>;
  const hipError_t e = allow_lds(kern, stream_lds<1, NTW>() + 4 * 1024, set);
  if (e != hipSuccess) return e;
  const Grid grid = grid_of((int64_t)a.slots * a.tiles);
  hipLaunchKernelGGL(kern, dim3(grid.x, grid.y), dim3(kThreads), (stream_lds<1, NTW>() + 4 * a.T), st, a);
  return hipGetLastError();
}

template <int NTW, int KIND>
hipError_t launch_down(MoeArgs a, hipStream_t st) {
  static bool set[64] = {false};
  a.tiles = (a.H + 16 * NTW - 1) / (16 * NTW);
  if ((int64_t)a.slots * a.tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  auto kern = k_moe_down<NTW, KIND>;
  const hipError_t e = allow_lds(kern, stream_lds<1, NTW>() + 4 * 1024, set);
  if (e != hipSuccess) return e;
  const Grid grid = grid_of((int64_t)a.slots * a.tiles);
  hipLaunchKernelGGL(kern, dim3(grid.x, grid.y), dim3(kThreads), (stream_lds<1, NTW>() + 4 * a.T), st, a);
  return hipGetLastError();
}

// Experts that some token chooses, if the choices were independent.
double active_experts(int64_t T, int64_t E, int64_t k) { return E * (1.0 - pow(1.0 - (double)k / E, (double)T)); }

// How a product over `experts` matrices of `rows` x `K` runs: by the workgroups of this file, `tiles`
// row tiles each, or by the persistent ones of moe_fp4_wide.hip with K in `parts` ranges.  The
// estimates, in us, are fits to runs on 256 CUs:
//   this file  rounds of two workgroups a CU, each 6 us and, per row tile and chunk, 0.33 us going up
//              and 0.4 down (0.6 for three terms of h), or the weights at 4.3 TB/s
//   persistent rounds of one work a CU, 3.5 us a chunk and 8 us going up, 4.3 a chunk and 6 us down (5
//              and 12 for three terms), 0.3 us more for every range after the first, or the weights at
//              5.2 TB/s
// Tokens are taken to choose independently, and an expert to have 16 at most: both repeat its weights for every
// 16, which the estimates leave out.
// Measured, this file's against the persistent ones': up 133 and 122 us (64 tokens, 64 experts of
// 4096 x 2048), 80 and 71 (16, 8 of 5120 x 8192); down 74 and 76, 58 and 46; with y in fp32 10.8 and
// 18.4 (30 tokens, 32 experts of 1000 x 500).
struct Way {
  bool wide;
  int tiles, parts;
  double us;
};

Way way_of(double experts, int64_t rows, int64_t K, bool up, bool f32, double cus) {
  const double mb = experts * rows * K * 17 / 32 * 1e-6;
  const int64_t chunks = (K + kChunk - 1) / kChunk;
  Way best{false, 8, 1, 1e30};
  for (int t = f32 && !up ? 2 : 8; t >= 2; t /= 2) {   // three terms of h leave registers for two row tiles
    const double rounds = ceil(experts * ceil((double)rows / (16 * t)) / (2 * cus));
    const double us = fmax(rounds * (6 + (up ? 0.33 : f32 ? 0.6 : 0.4) * t * chunks), mb / 4.3);
    if (us < best.us) best = Way{false, t, 1, us};
  }
  const double works = experts * ceil((double)rows / 256);
  for (int p = 1; p <= (up ? 1 : 8) && p <= chunks; p *= 2) {
    const double chunk = up ? 3.5 : f32 ? 5.0 : 4.3;
    const double us = fmax(ceil(works * p / cus) * ((chunks + p - 1) / p) * chunk, mb / 5.2) + (up ? 8 : f32 ? 12 : 6) + 0.3 * (p - 1);
    if (us < best.us) best = Way{true, 8, p, us};
  }
  return best;
}

// The two launches of moe_fp4_few.hip read an expert's weights once for every token that chose it, the
// four here and in moe_fp4_wide.hip once, but these cost 12 us of routing, adding up and launching, and the
// estimates above are low for few tokens.  Measured, two launches' kernels against four: 23 and 38 us (1
// token, 4 of 64 experts of 4096 x 2048), 83 and 131 (8 tokens), 160 and 212 (16); 47 and 70 (7, 6 of 60,
// 2000 x 1064, y in fp32); 12 and 24 (2, 2 of 32, 1000 x 700).
struct Plan {
  Way up, down;
  bool few;
};

Plan plan_of(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, bool f32, int cus) {
  const double experts = active_experts(T, E, k);
  Plan p{way_of(experts, 2 * I, H, true, f32, cus), way_of(experts, H, I, false, f32, cus), false};
  p.few = moe_few_us(T, H, I, E, k, cus) < 1.2 * (p.up.us + p.down.us) + 12;
  return p;
}

// The persistent kernels need whole 16-byte pieces: of rows of X and of scales going up, of scales down.
bool up_wide(const Plan& p, int64_t H, bool pieces) { return p.up.wide && H % 8 == 0 && pieces; }
bool down_wide(const Plan& p, bool pieces) { return p.down.wide && pieces; }
// Row tiles of a workgroup going down otherwise: three terms of h leave registers for two.
int down_tiles(const Plan& p, bool f32) { return f32 ? 2 : p.down.tiles; }

template <int KIND>
hipError_t launch_all(const MoeArgs& a, const Plan& plan, hipStream_t st) {
  if (plan.few) return launch_moe_few(a, st);
  auto route = a.E <= 64 ? k_moe_route<1> : a.E <= 256 ? k_moe_route<4> : k_moe_route<16>;
  hipLaunchKernelGGL(route, dim3((unsigned)((a.T + kWaves - 1) / kWaves)), dim3(kThreads), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int nu = plan.up.tiles, nd = down_tiles(plan, KIND == kThree);
  if (up_wide(plan, a.H, a.x_pieces && a.s13_pieces))
    e = launch_moe_up_wide<KIND>(a, st);
  else
    e = nu == 8 ? launch_up<8, KIND>(a, st) : nu == 4 ? launch_up<4, KIND>(a, st) : launch_up<2, KIND>(a, st);
  if (e != hipSuccess) return e;
  MoeArgs d = a;
  const bool wide = down_wide(plan, a.s2_pieces);
  d.parts = wide ? plan.down.parts : 1;
  if (wide)
    e = launch_moe_down_wide<KIND>(d, st);
  else
    e = KIND == kTwo && nd == 8 ? launch_down<8, kTwo>(d, st)
        : KIND == kTwo && nd == 4 ? launch_down<4, kTwo>(d, st) : launch_down<2, KIND>(d, st);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_moe_sum, dim3((unsigned)((a.H + 255) / 256), (unsigned)a.T), dim3(64), 0, st, d);
  return hipGetLastError();
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// Slots: one per expert, or, where the tokens can choose fewer, one per token and rank.
void moe_layout(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int kind, int parts, MoeArgs* a, int64_t off[5],
                int64_t* total) {
  a->by_token = T * k < E;
  a->slots = (int)(a->by_token ? T * k : E);
  a->mt_cap = (int)((T + 15) / 16);
  const int64_t chunks = (I + kChunk - 1) / kChunk;
  off[0] = 0;
  off[1] = up256(T * k * 4);
  off[2] = off[1] + up256(T * k * 4);
  off[3] = off[2] + up256(E * T * 2);
  off[4] = off[3] + (int64_t)a->slots * a->mt_cap * chunks * hidden_chunk(kind);
  *total = off[4] + up256(T * k * parts * H * 4);
}

}  // namespace

MoeFp4Plan moe_fp4_plan(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, bool y_bf16, bool aligned, int cus) {
  const Plan p = plan_of(T, H, I, E, k, !y_bf16, cus);
  if (p.few) return MoeFp4Plan{2, 0, 0, 0};
  const bool up = up_wide(p, H, aligned), down = down_wide(p, aligned);
  return MoeFp4Plan{4, up ? 128 : 8 * p.up.tiles, down ? 256 : 16 * down_tiles(p, !y_bf16), down ? p.down.parts : 1};
}

int64_t moe_fp4_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, bool y_bf16) {
  MoeArgs a{};
  int64_t off[5], total;
  const Plan plan = plan_of(T, H, I, E, k, !y_bf16, device_cu_count());
  if (plan.few) return moe_few_bytes(T, I, k);
  moe_layout(T, H, I, E, k, y_bf16 ? kTwo : kThree, plan.down.parts, &a, off, &total);
  return total;
}

hipError_t launch_moe_fp4(const MoeFp4& p, hipStream_t st) {
  MoeArgs a{};
  int64_t off[5], total;
  const Plan plan = plan_of(p.T, p.H, p.I, p.E, p.k, !p.y_bf16, device_cu_count());
  moe_layout(p.T, p.H, p.I, p.E, p.k, p.y_bf16 ? kTwo : kThree, plan.down.parts, &a, off, &total);
  a.T = (int)p.T;
  a.H = (int)p.H;
  a.I = (int)p.I;
  a.E = (int)p.E;
  a.k = (int)p.k;
  a.renorm = p.renorm;
  a.x = (const uint8_t*)p.x;
  a.ld_x = 2 * p.ld_x;
  a.logits = p.logits;
  a.ld_logits = p.ld_logits;
  a.w13 = p.w13;
  a.ld_w13 = p.ld_w13;
  a.st_w13 = p.st_w13;
  a.s13 = p.s13;
  a.ld_s13 = p.ld_s13;
  a.st_s13 = p.st_s13;
  a.w2 = p.w2;
  a.ld_w2 = p.ld_w2;
  a.st_w2 = p.st_w2;
  a.s2 = p.s2;
  a.ld_s2 = p.ld_s2;
  a.st_s2 = p.st_s2;
  uint8_t* ws = (uint8_t*)p.workspace;
  a.chosen = (int*)(ws + off[0]);
  a.share = (float*)(ws + off[1]);
  a.rank = (int16_t*)(ws + off[2]);
  a.h = plan.few ? ws : ws + off[3];
  a.part = (float*)(ws + off[4]);
  a.x_pieces = (uintptr_t)p.x % 16 == 0 && a.ld_x % 16 == 0;
  a.s13_words = (uintptr_t)p.s13 % 4 == 0 && p.ld_s13 % 4 == 0 && p.st_s13 % 4 == 0;
  a.s2_words = (uintptr_t)p.s2 % 4 == 0 && p.ld_s2 % 4 == 0 && p.st_s2 % 4 == 0;
  a.s13_pieces = (uintptr_t)p.s13 % 16 == 0 && p.ld_s13 % 16 == 0 && p.st_s13 % 16 == 0;
  a.s2_pieces = (uintptr_t)p.s2 % 16 == 0 && p.ld_s2 % 16 == 0 && p.st_s2 % 16 == 0;
  a.y = p.y;
  a.ld_y = p.ld_y;
  a.y_bf16 = p.y_bf16;
  return p.y_bf16 ? launch_all<kTwo>(a, plan, st) : launch_all<kThree>(a, plan, st);
}

}  // namespace mxq
