// moe_route.hip -- routing tokens to experts, for training and serving: softmax, the k greatest, shares,
// counts, the order of the slots by expert, the balance loss (mxq_moe_route) and the gradient of the logits
// (mxq_moe_route_grad).
//
// Mathematics: p = softmax(l); the k greatest logits choose (ties to the lower index); share = p, or p over the
// sum of the chosen.  With n tokens that count, c_e slots of expert e:  f_e = c_e / (n k),
// P_e = sum p_e / n,  L = E sum_e f_e P_e.  f is a constant of the gradient, so dL / dp_e of a token is
// slope_e = E f_e / n, and with g the gradient of p, d that of the shares:
//   dl = p (g - sum p g)  [+ share (d - sum share d) over the chosen, where the shares sum to 1].
//
// A wave has a token: lane l holds the logits of experts l, 64 + l, ...; the maximum of a wave takes six lane
// steps (DPP), its expert a ballot.  Waves take runs of consecutive tokens, so that one wave's counters (lane l
// those of experts l, 64 + l, ...) number the slots of an expert in order, and sums over the waves' and
// workgroups' counts give every slot its place: no atomics, and nothing depends on how workgroups are scheduled.
// Up to 256 tokens take one workgroup and one launch, more take three (tokens; sums over the groups; places and
// loss): 64 tokens of 64 experts, k 8, 10.5 us by one; 257 of 256 experts 15 by three, but 256 of 256 63 by one.
#include "codec.hpp"
#include "internal.hpp"

namespace mxq {
namespace {

constexpr int kGroups = 512, kWaves = 8;      // workgroups at most, and a workgroup's runs of tokens
constexpr int kSumRun = 256;                  // tokens whose p are added one after the other
constexpr int kSmallTokens = 256, kSmallSlots = 4096, kSmallExperts = 256, kSmallWaves = 16;

struct RouteArgs {
  const void* logits;
  int64_t ld;
  const uint8_t* mask;
  int T, E, k, renorm, bf16, groups;
  int* experts;
  float* shares;
  int* counts;
  int* offsets;
  int* order;
  float* loss;
  float* slope;
  // workspace: per group, E + 1 slot counts (the last: tokens that count) and E sums of p; per wave, E counts of
  // the group's waves before it; each slot's number among its wave's slots of the expert; E sums of p; the
  // number of tokens that count
  int* cnt;
  float* psum;
  int* before;
  int* rank;
  float* total;
  int* live;
};

__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
#define MXQ_STEP(ctrl, rows)                                                                       \
  {                                                                                                \
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xF, false);   \
    v = v > o ? v : o;                                                                             \
  }
  MXQ_STEP(0x111, 0xF) MXQ_STEP(0x112, 0xF) MXQ_STEP(0x114, 0xF) MXQ_STEP(0x118, 0xF)   // row_shr 1 2 4 8
  MXQ_STEP(0x142, 0xA) MXQ_STEP(0x143, 0xC)                                             // row_bcast 15, 31
#undef MXQ_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Sum over the wave, the same in every lane, in a fixed order.
__device__ __forceinline__ float dpp_sum(float v) {
#define MXQ_STEP(ctrl, rows) \
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, rows, 0xF, false));
  MXQ_STEP(0x111, 0xF) MXQ_STEP(0x112, 0xF) MXQ_STEP(0x114, 0xF) MXQ_STEP(0x118, 0xF)
  MXQ_STEP(0x142, 0xA) MXQ_STEP(0x143, 0xC)
#undef MXQ_STEP
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Order of the logits as unsigned numbers: NaN above all, -0 like +0; kMasked is -inf.
constexpr uint32_t kMasked = 0x007FFFFFu;
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float logit(const RouteArgs& a, int64_t t, int e) {
  const int64_t at = t * a.ld + e;
  return a.bf16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.logits)[at] << 16)
                : reinterpret_cast<const float*>(a.logits)[at];
}

// e^x for x <= 0 within a few u: 2^(x log2 e) by v_exp_f32, the rounding of the exponent put back by its first-order term
// (ocml's expf is the same to the last bits at three times the instructions; the kernels are bound by those).
__device__ __forceinline__ float exp_below(float x) {
  x = fmaxf(x, -200.0f);                         // (e^-200 is 0, and -inf has no remainder)
  const float t = x * 0x1.715476p+0f;
  const float r = __builtin_fmaf(x, 0x1.4ae0c0p-26f, __builtin_fmaf(x, 0x1.715476p+0f, -t));   // log2 e = high + low
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, r * 0x1.62e430p-1f, e);
}

template <int V>
__device__ __forceinline__ void load_token(const RouteArgs& a, int64_t t, int lane, float x[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 64 * v + lane;
    x[v] = e < a.E ? logit(a, t, e) : -INFINITY;
  }
}

// The softmax of a token's logits before division by `sum`, all zero where every expert is masked; their keys.
template <int V>
__device__ __forceinline__ void softmax(const RouteArgs& a, int lane, const float x[V], uint32_t key[V], float ex[V],
                                        float& sum) {
  uint32_t top = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    key[v] = key_of(x[v]);
    top = max(top, key[v]);
  }
  top = dpp_max(top);
  if (top == kMasked) {
#pragma unroll
    for (int v = 0; v < V; ++v) ex[v] = 0.0f;
    sum = 1.0f;
    return;
  }
  float s = 0.0f;
  if (top >= 0xFF800000u) {                      // +inf or NaN: NaN all over
#pragma unroll
    for (int v = 0; v < V; ++v) ex[v] = __uint_as_float(0x7FC00000u);
    sum = ex[0];
    return;
  }
  const float m = __uint_as_float(top & 0x80000000u ? top & 0x7FFFFFFFu : ~top);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    ex[v] = exp_below(x[v] - m);                 // (experts past the last one are -inf here: 0)
    s += ex[v];
  }
  sum = dpp_sum(s);
}

// The tokens t0 .. t1 - 1 in turn: experts, shares, and slot by slot the number among the run's slots of the
// expert; `put` takes (slot in the array, expert or -1, number).  In the loop over the k greatest a lane only
// learns which of its experts was taken and when (28 instructions a round with four experts a lane, and those
// bound the kernel); the lanes that own the chosen write what there is to write.
template <int V, typename Put>
__device__ __forceinline__ void route_unit(const RouteArgs& a, int t0, int t1, int lane, int cnt[V], float psum[V], int& live,
                                           Put put) {
  // p is summed in two levels, or terms that hardly differ, rounded the same way each time, would drift as the run grows:
  // 2^27 equal tokens of 5 experts, 32768 a wave, left the loss 2.6e-4 off, 3.2e-6 so (16384 x 256: 29.2 us, 29.6 so)
  float part[V];
#pragma unroll
  for (int v = 0; v < V; ++v) cnt[v] = 0, psum[v] = part[v] = 0.0f;
  live = 0;
  float next[V];
  uint32_t next_on = 0;          // (compared where it is used: a comparison here would wait for the loads)
  if (t0 < t1) {
    load_token<V>(a, t0, lane, next);
    next_on = a.mask == nullptr ? 1 : a.mask[t0];
  }
  for (int t = t0; t < t1; ++t) {
    float x[V];
    const bool on = next_on != 0;
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = next[v];
    if (t + 1 < t1) {            // the next token's logits are on their way while this one is routed
      load_token<V>(a, t + 1, lane, next);
      next_on = a.mask == nullptr ? 1 : a.mask[t + 1];
    }
    int taken = 0;
    const int64_t row = (int64_t)t * a.k;
    if (on) {
      ++live;
      uint32_t key[V];
      float ex[V], sum;
      softmax<V>(a, lane, x, key, ex, sum);
      const float inv = 1.0f / sum;
      int slot[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        part[v] += ex[v] * inv;
        slot[v] = -1;              // (experts past the last one have -inf's key, which nobody takes)
      }
      for (; taken < a.k; ++taken) {
        uint32_t top = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) top = max(top, key[v]);
        top = dpp_max(top);
        if (top <= kMasked) break;
        bool found = false;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const uint64_t who = __ballot(key[v] == top);
          const bool me = __builtin_amdgcn_inverse_ballot_w64(found ? 0 : who & (0 - who));
          found = found || who != 0;
          key[v] = me ? 0u : key[v];
          slot[v] = me ? taken : slot[v];
        }
      }
      float scale = inv;
      if (a.renorm) {
        float chosen = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) chosen += slot[v] >= 0 ? ex[v] : 0.0f;
        scale = 1.0f / dpp_sum(chosen);
      }
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (slot[v] >= 0) {
          a.experts[row + slot[v]] = 64 * v + lane;
          a.shares[row + slot[v]] = ex[v] * scale;
          put(row + slot[v], 64 * v + lane, cnt[v]++);
        }
    }
    if (lane >= taken && lane < a.k) {
      a.experts[row + lane] = -1;
      a.shares[row + lane] = 0.0f;
      put(row + lane, -1, 0);
    }
    if (t + 1 == t1 || (t - t0) % kSumRun == kSumRun - 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) psum[v] += part[v], part[v] = 0.0f;
    }
  }
}

// What follows from the counts, by 256 threads or more: thread e < E has count and sum of p of expert e.
__device__ __forceinline__ float loss_term(const RouteArgs& a, int e, int count, float psum, int live) {
  const float n = (float)max(live, 1);
  const float slope = (float)a.E * ((float)count / (n * (float)a.k)) / n;
  a.slope[e] = slope;
  return slope * psum;
}

// Exclusive sums over s[0 .. n), n <= 1024, by one wave; the total.
__device__ __forceinline__ int scan_wave(int* s, int n, int lane) {
  int before = 0;
  for (int e0 = 0; e0 < n; e0 += 64) {
    const int e = e0 + lane, mine = e < n ? s[e] : 0;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(sum, d, 64);
      sum += lane >= d ? o : 0;
    }
    if (e < n) s[e] = before + sum - mine;
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  return before;
}

// ---- few tokens: everything in one workgroup of 16 waves
template <int V>
__global__ __launch_bounds__(64 * kSmallWaves) void k_route_small(const RouteArgs a) {
  __shared__ int s_cnt[kSmallWaves][kSmallExperts], s_slot[kSmallSlots], s_off[kSmallExperts], s_live[kSmallWaves];
  __shared__ float s_p[kSmallWaves][kSmallExperts], s_loss[kSmallWaves];
  __shared__ int s_total;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int per = (a.T + kSmallWaves - 1) / kSmallWaves;
  int cnt[V], live;
  float psum[V];
  route_unit<V>(a, min(wave * per, a.T), min((wave + 1) * per, a.T), lane, cnt, psum, live,
                [&](int64_t at, int e, int n) { s_slot[at] = e < 0 ? -1 : (n << 8) | e; });
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (64 * v + lane < a.E) s_cnt[wave][64 * v + lane] = cnt[v], s_p[wave][64 * v + lane] = psum[v];
  if (lane == 0) s_live[wave] = live;
  __syncthreads();
  float term = 0.0f;
  if (tid < a.E) {
    int sum = 0, n = 0;
    float p = 0.0f;
    for (int w = 0; w < kSmallWaves; ++w) {
      const int c = s_cnt[w][tid];
      s_cnt[w][tid] = sum;
      sum += c;
      p += s_p[w][tid];
      n += s_live[w];
    }
    s_off[tid] = sum;
    a.counts[tid] = sum;
    term = loss_term(a, tid, sum, p, n);
  }
  term = dpp_sum(term);
  if (lane == 0) s_loss[wave] = term;
  __syncthreads();
  if (wave == 0) {
    const int total = scan_wave(s_off, a.E, lane);
    if (lane == 0) s_total = total;
  }
  if (tid == 0) {
    float l = 0.0f;
    for (int w = 0; w < kSmallWaves; ++w) l += s_loss[w];
    a.loss[0] = l;
  }
  __syncthreads();
  if (tid < a.E) a.offsets[tid] = s_off[tid];
  if (tid == 0) a.offsets[a.E] = s_total;
  const int slots = a.T * a.k;
  for (int at = tid; at < slots; at += 64 * kSmallWaves) {
    const int s = s_slot[at];
    if (s >= 0) a.order[s_off[s & 255] + s_cnt[(at / a.k) / per][s & 255] + (s >> 8)] = at;
    if (at >= s_total) a.order[at] = -1;
  }
}

// Wave w of the `groups` x 8: its run of tokens.
__device__ __forceinline__ int first_token(const RouteArgs& a, int w) { return (int)((int64_t)a.T * w / (a.groups * kWaves)); }

// ---- many tokens, one: a run of tokens a wave, then the counts and sums of the group
template <int V>
__global__ __launch_bounds__(64 * kWaves) void k_route_tokens(const RouteArgs a) {
  __shared__ int s_sum[kWaves][64 * V];
  __shared__ int s_live[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int w = blockIdx.x * kWaves + wave;
  int cnt[V], live;
  float psum[V];
  route_unit<V>(a, first_token(a, w), first_token(a, w + 1), lane, cnt, psum, live,
                [&](int64_t at, int, int n) { a.rank[at] = n; });
#pragma unroll
  for (int v = 0; v < V; ++v) s_sum[wave][64 * v + lane] = cnt[v];
  if (lane == 0) s_live[wave] = live;
  __syncthreads();
  for (int e = tid; e < a.E; e += 64 * kWaves) {
    int sum = 0;
#pragma unroll
    for (int u = 0; u < kWaves; ++u) {
      a.before[(int64_t)(blockIdx.x * kWaves + u) * a.E + e] = sum;
      sum += s_sum[u][e];
    }
    a.cnt[(int64_t)blockIdx.x * (a.E + 1) + e] = sum;
  }
  if (tid == 0) {
    int n = 0;
    for (int u = 0; u < kWaves; ++u) n += s_live[u];
    a.cnt[(int64_t)blockIdx.x * (a.E + 1) + a.E] = n;
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) s_sum[wave][64 * v + lane] = __float_as_int(psum[v]);
  __syncthreads();
  for (int e = tid; e < a.E; e += 64 * kWaves) {
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < kWaves; ++u) sum += __int_as_float(s_sum[u][e]);
    a.psum[(int64_t)blockIdx.x * a.E + e] = sum;
  }
}

// ---- two: sums over the groups, 8 columns (experts, then the tokens that count) a workgroup, 128 runs of at
// most four groups, whose counts stay in registers
__global__ __launch_bounds__(1024) void k_route_scan(const RouteArgs a) {
  constexpr int kRuns = 128, kRun = kGroups / kRuns;
  __shared__ int s_c[kRuns][9];
  __shared__ float s_p[kRuns][9];
  const int c = threadIdx.x & 7, run = threadIdx.x >> 3, e = blockIdx.x * 8 + c;
  int n[kRun];
  int sum = 0;
  float p = 0.0f;
#pragma unroll
  for (int u = 0; u < kRun; ++u) {
    const int g = run * kRun + u;
    n[u] = 0;
    if (g < a.groups && e <= a.E) {
      n[u] = a.cnt[(int64_t)g * (a.E + 1) + e];
      if (e < a.E) p += a.psum[(int64_t)g * a.E + e];
    }
    sum += n[u];
  }
  s_c[run][c] = sum;
  s_p[run][c] = p;
  // sums of the runs up to each, and of all p: log2(128) steps
  for (int d = 1; d < kRuns; d <<= 1) {
    __syncthreads();
    const int oc = run >= d ? s_c[run - d][c] : 0;
    const float op = run >= d ? s_p[run - d][c] : 0.0f;
    __syncthreads();
    s_c[run][c] += oc;
    s_p[run][c] += op;
  }
  if (e > a.E) return;
  int before = s_c[run][c] - sum;
#pragma unroll
  for (int u = 0; u < kRun; ++u) {
    const int g = run * kRun + u;
    if (g < a.groups) a.cnt[(int64_t)g * (a.E + 1) + e] = before;
    before += n[u];
  }
  if (run == kRuns - 1) {
    if (e < a.E) {
      a.counts[e] = before;
      a.total[e] = s_p[run][c];
    } else {
      a.live[0] = before;
    }
  }
}

// ---- three: every slot's place; the first workgroup also offsets, loss and slope
__global__ __launch_bounds__(256) void k_route_order(const RouteArgs a) {
  __shared__ int s_off[1024];
  __shared__ float s_loss[4];
  __shared__ int s_total;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < a.E; e += 256) s_off[e] = a.counts[e];
  __syncthreads();
  if (wave == 0) {
    const int total = scan_wave(s_off, a.E, lane);
    if (lane == 0) s_total = total;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    float term = 0.0f;
    const int live = a.live[0];
    for (int e = tid; e < a.E; e += 256) {
      a.offsets[e] = s_off[e];
      term += loss_term(a, e, a.counts[e], a.total[e], live);
    }
    term = dpp_sum(term);
    if (lane == 0) s_loss[wave] = term;
    __syncthreads();
    if (tid == 0) {
      a.loss[0] = (s_loss[0] + s_loss[1]) + (s_loss[2] + s_loss[3]);
      a.offsets[a.E] = s_total;
    }
  }
  const int64_t slots = (int64_t)a.T * a.k;
  for (int64_t at = (int64_t)blockIdx.x * 256 + tid; at < slots; at += (int64_t)gridDim.x * 256) {
    const int e = a.experts[at];
    if (e >= 0) {
      const int t = (int)(at / a.k), waves = a.groups * kWaves;
      // the wave whose run has the token
      int w = (int)(((int64_t)t * waves) / a.T);
      while (w + 1 < waves && first_token(a, w + 1) <= t) ++w;
      a.order[s_off[e] + a.cnt[(int64_t)(w / kWaves) * (a.E + 1) + e] + a.before[(int64_t)w * a.E + e] + a.rank[at]] = (int)at;
    }
    if (at >= s_total) a.order[at] = -1;
  }
}

// ---- the gradient of the logits: a token a wave
struct GradArgs {
  RouteArgs r;
  const float* d_shares;
  int64_t ld_ds;
  const float* d_loss;
  void* d;
  int64_t ld_d;
};

// Orders the wave's own LDS accesses.
__device__ __forceinline__ void wave_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

template <int V>
__global__ __launch_bounds__(256) void k_route_grad(const GradArgs a) {
  __shared__ float s_row[4][64 * V];
  float* row = s_row[threadIdx.x >> 6];
  const int lane = threadIdx.x & 63;
  const int wave = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = gridDim.x * 4;
  const float up = a.d_loss ? a.d_loss[0] : 0.0f;
  float slope[V];
#pragma unroll
  for (int v = 0; v < V; ++v) slope[v] = a.d_loss && 64 * v + lane < a.r.E ? a.r.slope[64 * v + lane] * up : 0.0f;
  for (int64_t t = wave; t < a.r.T; t += waves) {
    float out[V], x[V];
    const uint32_t on = a.r.mask == nullptr ? 1 : a.r.mask[t];
    load_token<V>(a.r, t, lane, x);
    // lane j: slot j
    int ej = -1;
    float d = 0.0f, share = 0.0f;
    if (a.d_shares && lane < a.r.k) {
      ej = a.r.experts[t * a.r.k + lane];
      d = a.d_shares[t * a.ld_ds + lane];
      share = a.r.renorm ? a.r.shares[t * a.r.k + lane] : 0.0f;
      if ((uint32_t)ej >= (uint32_t)a.r.E) ej = -1, d = share = 0.0f;   // (also what no forward pass writes)
    }
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = 0.0f;
    if (on != 0) {
      uint32_t key[V];
      float p[V], g[V], sum;
      softmax<V>(a.r, lane, x, key, p, sum);
      const float inv = 1.0f / sum;
#pragma unroll
      for (int v = 0; v < V; ++v) p[v] *= inv, g[v] = slope[v];
      if (a.d_shares) {
        const float q = a.r.renorm ? share * (d - dpp_sum(share * d)) : d;
        // slot by slot to expert by expert, through the wave's own LDS
#pragma unroll
        for (int v = 0; v < V; ++v) row[64 * v + lane] = 0.0f;
        wave_lds();
        if (ej >= 0) row[ej] = q;
        wave_lds();
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (a.r.renorm)
            out[v] = row[64 * v + lane];
          else
            g[v] += row[64 * v + lane];
        }
        wave_lds();
      }
      float dot = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) dot += p[v] * g[v];
      dot = dpp_sum(dot);
#pragma unroll
      for (int v = 0; v < V; ++v) out[v] += p[v] * (g[v] - dot);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = 64 * v + lane;
      if (e >= a.r.E) continue;
      if (a.r.bf16)
        reinterpret_cast<uint16_t*>(a.d)[t * a.ld_d + e] = (uint16_t)f32_to_bf16_rne(out[v]);
      else
        reinterpret_cast<float*>(a.d)[t * a.ld_d + e] = out[v];
    }
  }
}

bool small(int64_t T, int64_t E, int64_t k) { return T <= kSmallTokens && T * k <= kSmallSlots && E <= kSmallExperts; }
// At least one: without tokens its waves' runs are empty, and their counts and sums of zero are written.
int64_t groups_of(int64_t T) { return T < 1 ? 1 : T < kGroups * kWaves ? (T + kWaves - 1) / kWaves : kGroups; }
int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

template <int V>
hipError_t launch_v(RouteArgs a, hipStream_t s) {
  if (small(a.T, a.E, a.k)) {
    if constexpr (V <= kSmallExperts / 64) hipLaunchKernelGGL(k_route_small<V>, dim3(1), dim3(64 * kSmallWaves), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_route_tokens<V>, dim3(a.groups), dim3(64 * kWaves), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_route_scan, dim3(a.E / 8 + 1), dim3(1024), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  // (one workgroup at least: offsets, loss and slope are written without tokens too)
  const int64_t n = ((int64_t)a.T * a.k + 255) / 256;
  hipLaunchKernelGGL(k_route_order, dim3((unsigned)(n < 1 ? 1 : n < 1024 ? n : 1024)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int V>
hipError_t launch_grad_v(const GradArgs& a, hipStream_t s) {
  const int64_t groups = ((int64_t)a.r.T + 3) / 4;
  hipLaunchKernelGGL(k_route_grad<V>, dim3((unsigned)(groups < 8192 ? groups : 8192)), dim3(256), 0, s, a);
  return hipGetLastError();
}

RouteArgs args_of(const MoeRoute& p) {
  RouteArgs a{};
  a.logits = p.logits;
  a.ld = p.ld_logits;
  a.mask = p.mask;
  a.T = (int)p.T;
  a.E = (int)p.E;
  a.k = (int)p.k;
  a.renorm = p.renorm;
  a.bf16 = p.bf16;
  a.groups = (int)groups_of(p.T);
  a.experts = p.experts;
  a.shares = p.shares;
  a.counts = p.counts;
  a.offsets = p.offsets;
  a.order = p.order;
  a.loss = p.loss;
  a.slope = p.slope;
  return a;
}

}  // namespace

int64_t moe_route_workspace_bytes(int64_t T, int64_t E, int64_t k) {
  if (small(T, E, k)) return 0;
  const int64_t g = groups_of(T);
  return up256(4 * g * (E + 1)) + up256(4 * g * E) + up256(4 * g * kWaves * E) + up256(4 * T * k) + up256(4 * E) + 256;
}

hipError_t launch_moe_route(const MoeRoute& p, hipStream_t s) {
  RouteArgs a = args_of(p);
  if (!small(p.T, p.E, p.k)) {
    char* w = (char*)p.workspace;
    a.cnt = (int*)w;
    w += up256(4 * (int64_t)a.groups * (a.E + 1));
    a.psum = (float*)w;
    w += up256(4 * (int64_t)a.groups * a.E);
    a.before = (int*)w;
    w += up256(4 * (int64_t)a.groups * kWaves * a.E);
    a.rank = (int*)w;
    w += up256(4 * p.T * p.k);
    a.total = (float*)w;
    w += up256(4 * p.E);
    a.live = (int*)w;
  }
  if (p.E <= 64) return launch_v<1>(a, s);
  if (p.E <= 128) return launch_v<2>(a, s);
  if (p.E <= 256) return launch_v<4>(a, s);
  if (p.E <= 512) return launch_v<8>(a, s);
  return launch_v<16>(a, s);
}

hipError_t launch_moe_route_grad(const MoeRoute& p, const float* d_shares, int64_t ld_ds, const float* d_loss, void* d,
                                 int64_t ld_d, hipStream_t s) {
  GradArgs a{};
  a.r = args_of(p);
  a.d_shares = d_shares;
  a.ld_ds = ld_ds;
  a.d_loss = d_loss;
  a.d = d;
  a.ld_d = ld_d;
  if (p.E <= 64) return launch_grad_v<1>(a, s);
  if (p.E <= 128) return launch_grad_v<2>(a, s);
  if (p.E <= 256) return launch_grad_v<4>(a, s);
  if (p.E <= 512) return launch_grad_v<8>(a, s);
  return launch_grad_v<16>(a, s);
}

}  // namespace mxq
