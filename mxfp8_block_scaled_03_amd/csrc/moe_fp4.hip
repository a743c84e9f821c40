// moe_fp4.hip -- a mixture-of-experts layer for a few tokens with MXFP4 weights, for gfx950.
//
//   p = softmax(logits);  the k largest p of a token choose its experts (ties to the lower
//   index), their shares optionally renormalized to sum 1;
//   h = share * silu(x W1_e) * (x W3_e)      (gate rows [0, I) and up rows [I, 2I) of w13[e])
//   y = sum over the token's experts, in the order of their rank, of h W2_e
//
// Three launches: k_moe_up (routing, gate and up products, h), k_moe_down (down products, one
// partial row per token and expert), k_moe_sum (the sum of a token's rows).  The weights of
// every expert that a token chose are read once and bound the time; everything else is kept
// out of their way: each workgroup of k_moe_up works out the tokens of its own expert (one
// ballot per token), h goes to memory in the fragment order that k_moe_down reads, and
// experts that nobody chose end their workgroups at once.
//
// An expert with logit -inf is never taken: its share is zero, and a token whose logits are
// all -inf gets y = 0.  NaN logits order above +inf; their shares are NaN, as softmax's.
#include "fp4_mma.hpp"

namespace mxq {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr uint32_t kMasked = 0x007FFFFFu;   // order key of -inf

struct MoeArgs {
  int T, H, I, E, k, renorm;
  int slots, by_token;                 // by_token: slot = (token, rank), else slot = expert
  int mt_cap;                          // 16-row tiles that a slot's part of h holds
  int tiles;                           // column tiles of a launch
  const uint8_t* x;
  int64_t ld_x;                        // bytes
  const float* logits;
  int64_t ld_logits;
  const uint8_t *w13, *s13, *w2, *s2;
  int64_t ld_w13, st_w13, ld_s13, st_s13, ld_w2, st_w2, ld_s2, st_s2;   // rows and experts, bytes
  int* table;                          // [slots][2 + T]: expert, tokens, rows t * k + rank
  uint8_t* h;                          // [slots][mt_cap][units][terms][4][64][16 bytes]
  float* part;                         // [T * k][H]
  void* y;
  int64_t ld_y;
  int y_bf16;
};

// Order key of a logit: greater for greater values, equal for -0 and +0, NaN above +inf.
__device__ __forceinline__ uint32_t order_key(float l) {
  if (l != l) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(l + 0.0f);
  return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}

// How many logits of the row come before expert e (the whole wave calls).
__device__ __forceinline__ int rank_of(const float* row, int E, int e, uint32_t ke, int lane) {
  int n = 0;
  for (int j0 = 0; j0 < E; j0 += 64) {
    const int j = j0 + lane;
    const uint32_t kj = j < E ? order_key(row[j]) : 0u;
    n += __popcll(__ballot(j < E && (kj > ke || (kj == ke && j < e))));
  }
  return n;
}

// The rank of the lane's own expert j (key kj) in the row.
__device__ __forceinline__ int rank_of_lane(const float* row, int E, int j, uint32_t kj, int lane) {
  int n = 0;
  for (int i0 = 0; i0 < E; i0 += 64) {
    const uint32_t ki = i0 + lane < E ? order_key(row[i0 + lane]) : 0u;
#pragma unroll 16
    for (int i = 0; i < 64; ++i) {
      const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)ki, i);
      n += i0 + i < E && (o > kj || (o == kj && i0 + i < j)) ? 1 : 0;
    }
  }
  return n;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// The share of expert e of a row that chose it: exp(l_e - max) over the sum of the chosen
// experts' exponentials (renorm) or of all.
__device__ __forceinline__ float share_of(const float* row, const MoeArgs& a, int e, int lane) {
  float top = -__builtin_inff(), s = 0.0f;
  bool nan = false;
  for (int j = lane; j < a.E; j += 64) {
    top = fmaxf(top, row[j]);
    nan |= row[j] != row[j];
  }
  top = wave_max(top);
  if (__any(nan)) return __builtin_nanf("");
  for (int j0 = 0; j0 < a.E; j0 += 64) {
    const int j = j0 + lane;
    const float l = j < a.E ? row[j] : -__builtin_inff();
    bool in = j < a.E;
    if (a.renorm) in &= rank_of_lane(row, a.E, j, order_key(l), lane) < a.k;
    s += in ? expf(l - top) : 0.0f;
  }
  return expf(row[e] - top) / wave_sum(s);
}

// Rounds v to `TERMS` bf16 terms whose sum is v to 8 * TERMS bits.
template <int TERMS>
__device__ __forceinline__ void split_bf16(float v, uint32_t out[TERMS]) {
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
    const uint32_t b = f32_to_bf16_rne(v);
    out[t] = b;
    v = (b & 0x7F80u) == 0x7F80u ? 0.0f : v - __uint_as_float(b << 16);
  }
}

// ---- gate and up products.  A workgroup: one slot, 8 * NT columns of I (16 * NT rows of w13).
template <int MT, int NT, int TERMS>
__global__ __launch_bounds__(kThreads) void k_moe_up(const MoeArgs a) {
  constexpr int IC = 8 * NT;
  extern __shared__ __align__(16) float part[];
  __shared__ int s_e, s_cnt;
  __shared__ int16_t s_rank[1024], s_tok[1024];
  __shared__ float s_share[1024];
  const int slot = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // ---- the slot's expert and tokens
  int e = slot, t0 = 0;
  if (a.by_token) {
    t0 = slot / a.k;
    const int r0 = slot % a.k;
    const float* row = a.logits + t0 * a.ld_logits;
    if (threadIdx.x == 0) s_e = -1;
    __syncthreads();
    for (int j0 = 64 * wave; j0 < a.E; j0 += kThreads) {
      const int j = j0 + lane;
      const uint32_t kj = j < a.E ? order_key(row[j]) : 0u;
      const int n = rank_of_lane(row, a.E, j, kj, lane);
      if (j < a.E && n == r0 && kj != kMasked) s_e = j;          // ranks are distinct: one lane
    }
    __syncthreads();
    e = s_e;
  }
  if (e >= 0)
    for (int t = wave; t < a.T; t += kWaves) {
      const float* row = a.logits + t * a.ld_logits;
      const uint32_t ke = order_key(row[e]);
      const int n = rank_of(row, a.E, e, ke, lane);
      const bool in = n < a.k && ke != kMasked;
      const float s = in ? share_of(row, a, e, lane) : 0.0f;
      if (lane == 0) {
        s_rank[t] = (int16_t)(in ? n : -1);
        s_share[t] = s;
      }
    }
  __syncthreads();
  if (wave == 0) {
    int cnt = 0;
    if (e >= 0)
      for (int j0 = 0; j0 < a.T; j0 += 64) {
        const bool in = j0 + lane < a.T && s_rank[j0 + lane] >= 0;
        const uint64_t b = __ballot(in);
        if (in) s_tok[cnt + __popcll(b & ((1ull << lane) - 1))] = (int16_t)(j0 + lane);
        cnt += __popcll(b);
      }
    // by_token: an earlier token's slot has the expert already
    if (a.by_token && cnt > 0 && s_tok[0] != t0) cnt = 0;
    if (lane == 0) s_cnt = cnt;
    if (tile == 0) {
      int* tab = a.table + (int64_t)slot * (2 + a.T);
      if (lane == 0) {
        tab[0] = e;
        tab[1] = cnt;
      }
      for (int m = lane; m < cnt; m += 64) tab[2 + m] = s_tok[m] * a.k + s_rank[s_tok[m]];
    }
  }
  __syncthreads();
  const int cnt = s_cnt;
  if (cnt == 0) return;
  // ---- the product
  const int i0 = tile * IC;
  const int units = (a.I + kUnit - 1) / kUnit;
  Rows<MT, NT> r;
  r.w = a.w13 + e * a.st_w13 + i0 * a.ld_w13;
  r.ws = a.s13 + e * a.st_s13 + i0 * a.ld_s13;
#pragma unroll
  for (int n = 0; n < NT; ++n) {                       // columns past I read the last one again
    const int64_t row = min(16 * (n % (NT / 2)) + i, a.I - 1 - i0) + (n < NT / 2 ? 0 : a.I);
    r.wo[n] = (uint32_t)(row * a.ld_w13) + 16u * g;
    r.so[n] = (uint32_t)(row * a.ld_s13) + (uint32_t)g;
  }
  for (int m0 = 0; m0 < cnt; m0 += 16 * MT) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      r.x[m] = a.x + s_tok[min(m0 + 16 * m + i, cnt - 1)] * a.ld_x;
      r.xs[m] = nullptr;
    }
    v4f acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = {0.0f, 0.0f, 0.0f, 0.0f};
    sum_units<kXBf16, MT, NT, 2>(r, wave, kWaves, g, a.H, acc);
    if (m0 > 0) __syncthreads();
    store_part<MT, NT>(part, wave, lane, acc);
    __syncthreads();
    for (int q = threadIdx.x; q < 16 * MT * (IC / 8); q += kThreads) {
      const int m = q / (IC / 8), c = 8 * (q % (IC / 8));
      if (m0 + m >= cnt || i0 + c >= a.I) continue;
      const float share = s_share[s_tok[m0 + m]];
      uint32_t o[TERMS][4];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const v4f gt = sum_part<MT, NT>(part, kWaves, m, c + 4 * hf);
        const v4f up = sum_part<MT, NT>(part, kWaves, m, IC + c + 4 * hf);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint32_t b0[TERMS], b1[TERMS];
          const int col = i0 + c + 4 * hf + 2 * p;     // zeros past I
          split_bf16<TERMS>(col < a.I ? share * (silu(gt[2 * p]) * up[2 * p]) : 0.0f, b0);
          split_bf16<TERMS>(col + 1 < a.I ? share * (silu(gt[2 * p + 1]) * up[2 * p + 1]) : 0.0f, b1);
#pragma unroll
          for (int t = 0; t < TERMS; ++t) o[t][2 * hf + p] = b0[t] | (b1[t] << 16);
        }
      }
      const int k = i0 + c, mt = (m0 + m) / 16;
      uint8_t* dst = a.h + (((int64_t)slot * a.mt_cap + mt) * units + k / kUnit) * (TERMS * 4096) +
                     ((k % 32) / 8) * 1024 + (16 * ((k % kUnit) / 32) + m % 16) * 16;
#pragma unroll
      for (int t = 0; t < TERMS; ++t)
        *reinterpret_cast<uint4*>(dst + 4096 * t) = make_uint4(o[t][0], o[t][1], o[t][2], o[t][3]);
    }
  }
}

// ---- down products.  A workgroup: one slot, 16 * NT columns of H; h comes in fragment order.
template <int MT, int NT, int TERMS>
struct HUnit {
  v4i w[NT];
  uint32_t ws[NT];
  v4i x[MT][TERMS][4];
};

template <int MT, int NT, int TERMS>
__global__ __launch_bounds__(kThreads) void k_moe_down(const MoeArgs a) {
  extern __shared__ __align__(16) float part[];
  const int slot = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
  const int* tab = a.table + (int64_t)slot * (2 + a.T);
  const int e = tab[0], cnt = tab[1];
  if (cnt == 0) return;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = 16 * NT * tile;
  const int units = (a.I + kUnit - 1) / kUnit;
  const uint8_t* w = a.w2 + e * a.st_w2 + (int64_t)n0 * a.ld_w2;
  const uint8_t* ws = a.s2 + e * a.st_s2 + (int64_t)n0 * a.ld_s2;
  uint32_t wo[NT], so[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int row = min(16 * n + i, a.H - 1 - n0);
    wo[n] = (uint32_t)(row * a.ld_w2) + 16u * g;
    so[n] = (uint32_t)(row * a.ld_s2) + (uint32_t)g;
  }
  const int mtiles = (cnt + 15) / 16;
  for (int mt0 = 0; mt0 < mtiles; mt0 += MT) {
    const uint8_t* hx[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
      hx[m] = a.h + ((int64_t)slot * a.mt_cap + min(mt0 + m, mtiles - 1)) * units * (TERMS * 4096);
    auto load = [&](HUnit<MT, NT, TERMS>& t, int u) {
      // codes past I are zeroed, and so are the blocks past the end, under scale 1
      const int left = a.I - kUnit * u - 32 * g;
      const v4i zero = {0, 0, 0, 0};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        t.w[n] = zero;
        t.ws[n] = 127u;
        if (left > 0) {
          t.w[n] = *reinterpret_cast<const v4i*>(w + (wo[n] + 64u * (uint32_t)u));
          t.ws[n] = ws[so[n] + 4u * (uint32_t)u];
        }
        if (left < 32) t.w[n] = keep_codes(t.w[n], left);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int p = 0; p < TERMS; ++p)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            t.x[m][p][j] = zero;                       // h has nothing at k >= I
            if (8 * j < left)
              t.x[m][p][j] = *reinterpret_cast<const v4i*>(hx[m] + ((int64_t)u * TERMS + p) * 4096 + 1024 * j + 16 * lane);
          }
    };
    v4f acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = {0.0f, 0.0f, 0.0f, 0.0f};
    HUnit<MT, NT, TERMS> t;
    for (int u = wave; u < units; u += kWaves) {
      load(t, u);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float s = e8m0_to_f32(t.ws[n]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t d[4];
          fp4::decode8_bf16((uint32_t)t.w[n][j], s, d);
          const v4i dv = {(int)d[0], (int)d[1], (int)d[2], (int)d[3]};
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int p = TERMS - 1; p >= 0; --p)
              acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(v8bf, dv), __builtin_bit_cast(v8bf, t.x[m][p][j]), acc[m][n], 0, 0, 0);
        }
      }
    }
    if (mt0 > 0) __syncthreads();
    store_part<MT, NT>(part, wave, lane, acc);
    __syncthreads();
    for (int q = threadIdx.x; q < 16 * MT * 4 * NT; q += kThreads) {
      const int m = 16 * mt0 + q / (4 * NT), n = 4 * (q % (4 * NT));
      if (m >= cnt || n0 + n >= a.H) continue;
      const v4f v = sum_part<MT, NT>(part, kWaves, q / (4 * NT), n);
      float* p = a.part + (int64_t)tab[2 + m] * a.H + n0 + n;
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (n0 + n + x < a.H) p[x] = v[x];
    }
  }
}

// ---- y[t] = sum of the token's rows, in the order of rank; masked experts come last and
// have none.
__global__ __launch_bounds__(256) void k_moe_sum(const MoeArgs a) {
  const int t = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;
  const int lane = threadIdx.x & 63;
  int valid = 0;
  for (int j0 = 0; j0 < a.E; j0 += 64)
    valid += __popcll(__ballot(j0 + lane < a.E && order_key(a.logits[t * a.ld_logits + j0 + lane]) != kMasked));
  if (valid > a.k) valid = a.k;
  if (n >= a.H) return;
  float s = 0.0f;
  for (int r = 0; r < valid; ++r) s += a.part[((int64_t)t * a.k + r) * a.H + n];
  if (a.y_bf16)
    reinterpret_cast<uint16_t*>(a.y)[t * a.ld_y + n] = (uint16_t)f32_to_bf16_rne(s);
  else
    reinterpret_cast<float*>(a.y)[t * a.ld_y + n] = s;
}

template <typename K>
hipError_t launch_lds(K kern, bool* set, unsigned grid, int lds, const MoeArgs& a, hipStream_t st) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) dev = 0;
  if (lds > 49152 && !set[dev]) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    set[dev] = true;
  }
  hipLaunchKernelGGL(kern, dim3(grid), dim3(kThreads), lds, st, a);
  return hipGetLastError();
}

template <int MT, int NT, int TERMS>
hipError_t launch_up(MoeArgs a, hipStream_t st) {
  static bool set[64] = {false};
  a.tiles = (a.I + 8 * NT - 1) / (8 * NT);
  if ((int64_t)a.slots * a.tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  return launch_lds(k_moe_up<MT, NT, TERMS>, set, (unsigned)(a.slots * a.tiles), kWaves * part_wave<MT, NT>() * 4, a, st);
}

template <int MT, int NT, int TERMS>
hipError_t launch_down(MoeArgs a, hipStream_t st) {
  static bool set[64] = {false};
  a.tiles = (a.H + 16 * NT - 1) / (16 * NT);
  if ((int64_t)a.slots * a.tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  return launch_lds(k_moe_down<MT, NT, TERMS>, set, (unsigned)(a.slots * a.tiles), kWaves * part_wave<MT, NT>() * 4, a,
                    st);
}

// Column tiles as wide as still give every CU a workgroup (a slot's expert may be unused, so
// the count is an upper bound).
template <int MT, int TERMS>
hipError_t launch_all(const MoeArgs& a, hipStream_t st) {
  const int64_t cus = device_cu_count();
  hipError_t e = (int64_t)a.slots * ((a.I + 31) / 32) >= cus ? launch_up<MT, 4, TERMS>(a, st) : launch_up<MT, 2, TERMS>(a, st);
  if (e != hipSuccess) return e;
  if ((int64_t)a.slots * ((a.H + 63) / 64) >= 2 * cus)
    e = launch_down<MT, 4, TERMS>(a, st);
  else if ((int64_t)a.slots * ((a.H + 31) / 32) >= cus)
    e = launch_down<MT, 2, TERMS>(a, st);
  else
    e = launch_down<MT, 1, TERMS>(a, st);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_moe_sum, dim3((unsigned)((a.H + 255) / 256), (unsigned)a.T), dim3(256), 0, st, a);
  return hipGetLastError();
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// Slots: one per expert, or, where the tokens can choose fewer, one per token and rank.
void moe_layout(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int terms, MoeArgs* a, int64_t off[3],
                int64_t* total) {
  a->by_token = T * k < E;
  a->slots = (int)(a->by_token ? T * k : E);
  a->mt_cap = (int)((T + 15) / 16);
  const int64_t units = (I + kUnit - 1) / kUnit;
  off[0] = 0;
  off[1] = up256((int64_t)a->slots * (2 + T) * 4);
  off[2] = off[1] + (int64_t)a->slots * a->mt_cap * units * terms * 4096;
  *total = off[2] + up256(T * k * H * 4);
}

int terms_of(bool y_bf16) { return y_bf16 ? 2 : 3; }

}  // namespace

int64_t moe_fp4_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, bool y_bf16) {
  MoeArgs a{};
  int64_t off[3], total;
  moe_layout(T, H, I, E, k, terms_of(y_bf16), &a, off, &total);
  return total;
}

hipError_t launch_moe_fp4(const MoeFp4& p, hipStream_t st) {
  MoeArgs a{};
  int64_t off[3], total;
  moe_layout(p.T, p.H, p.I, p.E, p.k, terms_of(p.y_bf16), &a, off, &total);
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
  a.table = (int*)((uint8_t*)p.workspace + off[0]);
  a.h = (uint8_t*)p.workspace + off[1];
  a.part = (float*)((uint8_t*)p.workspace + off[2]);
  a.y = p.y;
  a.ld_y = p.ld_y;
  a.y_bf16 = p.y_bf16;
  // rows that an expert can expect: 32-row tiles once its share of the tokens passes 16
  const bool wide = p.T > 16 && p.T * p.k > 12 * p.E;
  if (p.y_bf16) return wide ? launch_all<2, 2>(a, st) : launch_all<1, 2>(a, st);
  return wide ? launch_all<2, 3>(a, st) : launch_all<1, 3>(a, st);
}

}  // namespace mxq
