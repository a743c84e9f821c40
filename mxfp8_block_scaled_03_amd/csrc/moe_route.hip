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
// those of experts l, 64 + l, ...) number the slots of an expert in order, and a scan over the waves' counts
// gives every slot its place: no atomics, and nothing depends on how workgroups are scheduled.  Bound by
// HBM for many tokens (logits once), by launches for few: up to 256 tokens take one workgroup and one launch, more
// take three (tokens; scan over waves; places and loss).
#include "codec.hpp"
#include "internal.hpp"

namespace mxq {
namespace {

constexpr int kUnits = 1024;      // runs of tokens, at most
constexpr int kSmallTokens = 256, kSmallSlots = 4096, kSmallExperts = 256, kSmallWaves = 16;

struct RouteArgs {
  const void* logits;
  int64_t ld;
  const uint8_t* mask;
  int T, E, k, renorm, bf16, units;
  int* experts;
  float* shares;
  int* counts;
  int* offsets;
  int* order;
  float* loss;
  float* slope;
  // workspace: per unit, E + 1 slot counts (the last: tokens that count) and E sums of p; each slot's number
  // among its unit's slots of the expert; E sums of p; the number of tokens that count
  int* cnt;
  float* psum;
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

// A token's logits, their maximum and the softmax; all zero where every expert is masked.
template <int V>
__device__ __forceinline__ void softmax(const RouteArgs& a, int64_t t, int lane, float x[V], float ex[V], float& sum) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 64 * v + lane;
    x[v] = e < a.E ? logit(a, t, e) : -INFINITY;
  }
  uint32_t top = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) top = max(top, key_of(x[v]));
  top = dpp_max(top);
  if (top == kMasked) {
#pragma unroll
    for (int v = 0; v < V; ++v) ex[v] = 0.0f;
    sum = 1.0f;
    return;
  }
  const float m = top == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u)
                                     : __uint_as_float(top & 0x80000000u ? top & 0x7FFFFFFFu : ~top);
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    // (an expert past the last one stays 0 also beside a NaN)
    ex[v] = 64 * v + lane < a.E ? expf(x[v] - m) : 0.0f;
    s += ex[v];
  }
  sum = dpp_sum(s);
}

// The tokens of one unit in turn: experts, shares, and slot by slot the number among the unit's slots of the
// expert; `put` takes (slot in the array, expert or -1, number).
template <int V, typename Put>
__device__ __forceinline__ void route_unit(const RouteArgs& a, int t0, int t1, int lane, int cnt[V], float psum[V], int& live,
                                           Put put) {
#pragma unroll
  for (int v = 0; v < V; ++v) cnt[v] = 0, psum[v] = 0.0f;
  live = 0;
  for (int t = t0; t < t1; ++t) {
    int mine = -1, number = 0;   // lane j: slot j
    float share = 0.0f;
    if (a.mask == nullptr || a.mask[t]) {
      ++live;
      float x[V], ex[V], sum;
      softmax<V>(a, t, lane, x, ex, sum);
      const float inv = 1.0f / sum;
      uint32_t key[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        psum[v] += ex[v] * inv;
        key[v] = 64 * v + lane < a.E ? key_of(x[v]) : 0u;
      }
      float chosen = 0.0f;
      for (int j = 0; j < a.k; ++j) {
        uint32_t top = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) top = max(top, key[v]);
        top = dpp_max(top);
        if (top <= kMasked) break;
        bool found = false;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const uint64_t who = __ballot(key[v] == top);
          if (!found && who) {
            found = true;
            const int l = __builtin_ctzll(who);
            const float e = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ex[v]), l));
            const int n = __builtin_amdgcn_readlane(cnt[v], l);
            if (lane == l) key[v] = 0u, ++cnt[v];
            chosen += e;
            if (lane == j) mine = 64 * v + l, number = n, share = e;
          }
        }
      }
      if (mine >= 0) share *= a.renorm ? 1.0f / chosen : inv;
    }
    if (lane < a.k) {
      const int64_t at = (int64_t)t * a.k + lane;
      a.experts[at] = mine;
      a.shares[at] = share;
      put(at, mine, number);
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

// ---- many tokens, one: a unit a wave
template <int V>
__global__ __launch_bounds__(256) void k_route_tokens(const RouteArgs a) {
  const int lane = threadIdx.x & 63, unit = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= a.units) return;
  const int t0 = (int)((int64_t)a.T * unit / a.units), t1 = (int)((int64_t)a.T * (unit + 1) / a.units);
  int cnt[V], live;
  float psum[V];
  route_unit<V>(a, t0, t1, lane, cnt, psum, live, [&](int64_t at, int, int n) { a.rank[at] = n; });
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 64 * v + lane;
    if (e < a.E) {
      a.cnt[(int64_t)unit * (a.E + 1) + e] = cnt[v];
      a.psum[(int64_t)unit * a.E + e] = psum[v];
    }
  }
  if (lane == 0) a.cnt[(int64_t)unit * (a.E + 1) + a.E] = live;
}

// ---- two: sums over the units, 16 columns (experts, then the tokens that count) a workgroup, 64 runs of units
__global__ __launch_bounds__(1024) void k_route_scan(const RouteArgs a) {
  __shared__ int s_c[64][17];
  __shared__ float s_p[64][17];
  const int c = threadIdx.x & 15, run = threadIdx.x >> 4, e = blockIdx.x * 16 + c;
  const int u0 = a.units * run / 64, u1 = a.units * (run + 1) / 64;
  int sum = 0;
  float p = 0.0f;
  if (e <= a.E)
    for (int u = u0; u < u1; ++u) {
      sum += a.cnt[(int64_t)u * (a.E + 1) + e];
      if (e < a.E) p += a.psum[(int64_t)u * a.E + e];
    }
  s_c[run][c] = sum;
  s_p[run][c] = p;
  __syncthreads();
  if (e > a.E) return;
  int before = 0;
  for (int r = 0; r < run; ++r) before += s_c[r][c];
  if (run == 63) {
    float q = 0.0f;
    for (int r = 0; r < 64; ++r) q += s_p[r][c];
    if (e < a.E) {
      a.counts[e] = before + sum;
      a.total[e] = q;
    } else {
      a.live[0] = before + sum;
    }
  }
  for (int u = u0; u < u1; ++u) {
    int* at = a.cnt + (int64_t)u * (a.E + 1) + e;
    const int n = *at;
    *at = before;
    before += n;
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
      const int t = (int)(at / a.k);
      // the unit whose run [T u / units, T (u + 1) / units) has the token
      int u = (int)(((int64_t)t * a.units) / a.T);
      while (u + 1 < a.units && (int64_t)a.T * (u + 1) / a.units <= t) ++u;
      a.order[s_off[e] + a.cnt[(int64_t)u * (a.E + 1) + e] + a.rank[at]] = (int)at;
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

template <int V>
__global__ __launch_bounds__(256) void k_route_grad(const GradArgs a) {
  const int lane = threadIdx.x & 63;
  const int wave = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = gridDim.x * 4;
  const float up = a.d_loss ? a.d_loss[0] : 0.0f;
  float slope[V];
#pragma unroll
  for (int v = 0; v < V; ++v) slope[v] = a.d_loss && 64 * v + lane < a.r.E ? a.r.slope[64 * v + lane] * up : 0.0f;
  for (int64_t t = wave; t < a.r.T; t += waves) {
    float out[V];
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = 0.0f;
    if (a.r.mask == nullptr || a.r.mask[t]) {
      float x[V], p[V], g[V], sum;
      softmax<V>(a.r, t, lane, x, p, sum);
      const float inv = 1.0f / sum;
#pragma unroll
      for (int v = 0; v < V; ++v) p[v] *= inv, g[v] = slope[v];
      if (a.d_shares) {
        const int e = lane < a.r.k ? a.r.experts[t * a.r.k + lane] : -1;
        const float d = e >= 0 ? a.d_shares[t * a.ld_ds + lane] : 0.0f;
        float q = d;
        if (a.r.renorm) {
          const float s = e >= 0 ? a.r.shares[t * a.r.k + lane] : 0.0f;
          q = s * (d - dpp_sum(e >= 0 ? s * d : 0.0f));
        }
        for (int j = 0; j < a.r.k; ++j) {
          const int ej = __builtin_amdgcn_readlane(e, j);
          const float qj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(q), j));
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (ej == 64 * v + lane) {
              if (a.r.renorm)
                out[v] = qj;
              else
                g[v] += qj;
            }
        }
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
int64_t units_of(int64_t T) { return T < kUnits ? T : kUnits; }
int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

template <int V>
hipError_t launch_v(RouteArgs a, hipStream_t s) {
  if (small(a.T, a.E, a.k)) {
    if constexpr (V <= kSmallExperts / 64) hipLaunchKernelGGL(k_route_small<V>, dim3(1), dim3(64 * kSmallWaves), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_route_tokens<V>, dim3((a.units + 3) / 4), dim3(256), 0, s, a);
  hipLaunchKernelGGL(k_route_scan, dim3((a.E + 16) / 16), dim3(1024), 0, s, a);
  const int64_t groups = ((int64_t)a.T * a.k + 255) / 256;
  hipLaunchKernelGGL(k_route_order, dim3((unsigned)(groups < 1024 ? groups : 1024)), dim3(256), 0, s, a);
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
  a.units = (int)units_of(p.T);
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
  const int64_t u = units_of(T);
  return up256(4 * u * (E + 1)) + up256(4 * u * E) + up256(4 * T * k) + up256(4 * E) + 256;
}

hipError_t launch_moe_route(const MoeRoute& p, hipStream_t s) {
  RouteArgs a = args_of(p);
  if (!small(p.T, p.E, p.k)) {
    char* w = (char*)p.workspace;
    a.cnt = (int*)w;
    w += up256(4 * (int64_t)a.units * (a.E + 1));
    a.psum = (float*)w;
    w += up256(4 * (int64_t)a.units * a.E);
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
