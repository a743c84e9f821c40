// moe_fp4_wide.hip -- the expert layer's gate, up and down products where there are weights for
// every CU to stream for long: one persistent workgroup per CU over an equal run of works.
//
// A work is 16 tokens of one expert x 128 columns of I (up: 16 gate and 16 up rows of w13 for
// each of eight waves) or 256 columns of H (down: 32 rows of w2 a wave), over all of K or one
// range of it.  A wave owns its columns, so nothing is added across waves: its weights move as
// in fp4_stream.hpp (items of 16 rows x 512 elements, LDS DMA into a ring of its own, three
// slots, or two) without a pause from chunk to chunk and from work to work, because the DMA runs a
// ring's items ahead of the products through the whole run.  X is shared: the workgroup stages it
// by DMA, a stage or two ahead, and meets at one barrier per stage.
//
// Scale bytes come for several chunks at a time (GROUP: 4 or 2; 64 or 32 bytes of a row), since 16
// bytes of a row per chunk would fetch each of its memory lines anew every time.  They are read
// into registers when the group begins.
//
// Every stage issues at least the same number of loads (those past the run's end, and rows of X
// that no token has, go through an empty descriptor), so the waits are constants: an item's
// wait counts the loads that are sure to be issued after it.
//
// HBM bounds it: up 4.9-5.2 TB/s (70 us for 16 tokens over 8 experts of 5120 x 8192, 357 MB; 120 us
// for 64 over 64 of 4096 x 2048, 570 MB; a copy reaches 5.0), down 3.8 (46 and 76 us), which reads the
// hidden values from LDS twice as wide and meets twice a chunk.  The finer workgroups of moe_fp4.hip,
// whose fixed costs (looking up tokens, filling the ring, adding the waves' sums) come at the same
// time on every CU, take 80 and 133 us going up.
#include "moe_fp4.hpp"

namespace mxq {
namespace {
namespace wide {

constexpr int kW = 8;                        // waves
constexpr int kT = 64 * kW;
constexpr int kRingW = 3;                    // slots going up, and down with hidden values of two terms
constexpr int kCodes = 4096;                 // bytes of an item's codes
constexpr int kStage = 16384;                // bytes of X per stage going up
constexpr int kDownStages = 3;
// LDS of the two kernels: ring, X stages, scales, works.  A stage going down is half a chunk of h; three
// terms leave room for two slots of the ring.
constexpr int ring_slots(int kind) { return kind == kThree ? 2 : kRingW; }
constexpr int down_stage(int kind) { return hidden_chunk(kind) / 2; }
constexpr int kUpX = kW * kRingW * kCodes, kUpScales = kUpX + 2 * kStage, kUpLds = kUpScales + kW * 2048;
constexpr int down_x(int kind) { return kW * ring_slots(kind) * kCodes; }
constexpr int down_scales(int kind) { return down_x(kind) + kDownStages * down_stage(kind); }
constexpr int down_lds(int kind) { return down_scales(kind) + kW * 1024; }
static_assert(down_lds(kTwo) + 4096 <= 160 * 1024 && down_lds(kThree) + 4096 <= 160 * 1024, "LDS of a CU");

// The run of works of this workgroup, and where a work lies: s_end[s] is the number of works of
// slots 0 .. s.  A slot's works: its 16-token tiles, of each its K ranges, of each its columns.
struct Works {
  const int* s_end;
  int tiles, parts;
};

struct Pos {
  int w, slot, m, part, tile;
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ void seek(Pos& p, const Works& q, int w) {
  p.w = w;
  while (uniform(q.s_end[p.slot]) <= w) ++p.slot;
  const int i = w - (p.slot > 0 ? uniform(q.s_end[p.slot - 1]) : 0);
  const int per = q.tiles * q.parts;
  p.m = i / per;
  p.part = (i % per) / q.tiles;
  p.tile = i % q.tiles;
}

__device__ __forceinline__ int expert_of(const MoeArgs& a, int slot) { return a.by_token ? uniform(a.chosen[slot]) : slot; }

// The wave's lanes 0 .. 15: t * k + rank + 1 of the expert's tokens 16 m .. 16 m + 15, 0 past the
// last; other lanes: anything.
__device__ __forceinline__ int rows_of(const MoeArgs& a, int e, int m, int lane) {
  int got = 0, before = 0;
  for (int t0 = 0; t0 < a.T; t0 += 64) {
    const int t = t0 + lane;
    const int r = t < a.T ? a.rank[(int64_t)e * a.T + t] : -1;
    const uint64_t b = __ballot(r >= 0);
    const int at = before + __popcll(b & ((1ull << lane) - 1)) - 16 * m;
    const bool mine = r >= 0 && at >= 0 && at < 16;
    got |= __builtin_amdgcn_ds_permute(4 * (mine ? at : 63), mine ? t * a.k + r + 1 : 0);
    before += __popcll(b);
  }
  return got;
}

// Counts every slot's works into s_end (all waves; barriers inside) and returns the total.
__device__ __forceinline__ int count_works(const MoeArgs& a, int per, int* s_end, int lane, int wave) {
  for (int s = wave; s < a.slots; s += kW) {
    const int e = expert_of(a, s);
    int cnt = 0, first = -1;
    if (e >= 0)
      for (int t0 = 0; t0 < a.T; t0 += 64) {
        const int r = t0 + lane < a.T ? a.rank[(int64_t)e * a.T + t0 + lane] : -1;
        const uint64_t b = __ballot(r >= 0);
        if (b != 0 && first < 0) {
          const int l = __ffsll((unsigned long long)b) - 1;
          first = (t0 + l) * a.k + __builtin_amdgcn_readlane(r, l);
        }
        cnt += __popcll(b);
      }
    if (a.by_token && first != s) cnt = 0;               // an earlier token's slot has the expert
    if (lane == 0) s_end[s] = (cnt + 15) / 16 * per;
  }
  __syncthreads();
  if (wave == 0) {
    int base = 0;
    for (int s0 = 0; s0 < a.slots; s0 += 64) {
      int v = s0 + lane < a.slots ? s_end[s0 + lane] : 0;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
      }
      if (s0 + lane < a.slots) s_end[s0 + lane] = base + v;
      base += __shfl(v, 63);
    }
  }
  __syncthreads();
  return uniform(s_end[a.slots - 1]);
}

// The next item of a wave: row tile t = 0, 1 of chunk c of work p, into slot n.
struct Feed {
  Pos p;
  int c, c1, t, n;
  bool live;
  uint64_t at[2];                            // the tiles' codes
  uint32_t bytes[2];
};

__device__ __forceinline__ void issue_codes(const Feed& f, const ItemOffsets& o, uint32_t ring) {
  const uint32_t off = 256u * (uint32_t)f.c, bytes = f.t == 0 ? f.bytes[0] : f.bytes[1];
  const v4i r = rsrc_of((f.t == 0 ? f.at[0] : f.at[1]) + off, f.live && off < bytes ? bytes - off : 0u);
#pragma unroll
  for (int d = 0; d < 4; ++d) dma16(ring + f.n * kCodes + 1024 * d, o.c[d], r);
}

// Bytes from a tile's first row to its last block; 0 without rows.
__device__ __forceinline__ uint32_t code_bytes(int rows, int64_t ld, int nb) {
  return rows > 0 ? (uint32_t)((rows - 1) * ld + 16 * nb) : 0u;
}

// Scales of a group of chunks for both tiles of a wave: GROUP 4: two loads of 16 rows x 64 bytes;
// GROUP 2: one of 32 rows x 32 bytes (the second tile `step` bytes behind the first).  Row r of
// tile t lies at (16 t + r) * 16 * GROUP.
template <int GROUP>
__device__ __forceinline__ void issue_scales(const uint8_t* base, int64_t ld, int64_t step, int rows0, int rows1, int nb, int c,
                                             uint32_t lds, int lane) {
  constexpr int PIECES = GROUP;              // 16-byte pieces of a row
  const uint32_t nb4 = (uint32_t)(nb + 3) & ~3u, off = 16u * (uint32_t)c;
#pragma unroll
  for (int t = 0; t < (GROUP == 4 ? 2 : 1); ++t) {
    const int r = lane / PIECES;             // 0 .. 15, or 0 .. 31 over both tiles
    const uint32_t voff = (uint32_t)((r & 15) * ld) + (r >= 16 ? (uint32_t)step : 0u) + 16u * (uint32_t)(lane % PIECES);
    const int rows = GROUP == 4 ? (t == 0 ? rows0 : rows1) : (rows1 > 0 ? rows1 : rows0);
    uint32_t bytes = rows > 0 ? (uint32_t)((rows - 1) * ld) + nb4 + (GROUP == 2 && rows1 > 0 ? (uint32_t)step : 0u) : 0u;
    bytes = off < bytes ? bytes - off : 0u;
    dma16(lds + 1024 * t, voff, rsrc_of((uint64_t)(uintptr_t)base + (uint64_t)(t * step) + off, bytes));
  }
}

// The scale dwords of row i, blocks 4g .. 4g+3 of the group's chunks.
template <int GROUP>
__device__ __forceinline__ void read_scales(uint32_t s[2][GROUP], uint32_t at, int lane) {
  const int i = lane & 15, g = lane >> 4;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int c = 0; c < GROUP; ++c)
      s[t][c] = *reinterpret_cast<const uint32_t*>(smem + at + (16 * t + i) * (16 * GROUP) + 16 * c + 4 * g);
}

// The last loads of the wave that LDS reads of this stage have to see are there, and the wave's
// reads of the stage before are done: then all waves meet.
__device__ __forceinline__ void meet() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  lds_barrier();
}

template <int N>
__device__ __forceinline__ void landed() {
  wait_vm<N>();
  asm volatile("" ::: "memory");
}

// ---- gate and up.
template <int KIND>
__global__ __launch_bounds__(kT, 1) void k_moe_up_wide(const MoeArgs a) {
  constexpr int GROUP = 4;
  int* s_end = reinterpret_cast<int*>(smem + kUpLds);
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
  const int total = count_works(a, a.tiles, s_end, lane, wave);
  const int wg = xcd_order(blockIdx.x, gridDim.x);
  const int w0 = (int)((int64_t)total * wg / gridDim.x), w1 = (int)((int64_t)total * (wg + 1) / gridDim.x);
  if (w0 >= w1) return;
  const Works works{s_end, a.tiles, 1};
  const int nb = (a.H + 31) / 32, chunks = (a.H + kChunk - 1) / kChunk, h_chunks = (a.I + kChunk - 1) / kChunk;
  const uint32_t ring = (uint32_t)wave * (kRingW * kCodes), my_scales = kUpScales + (uint32_t)wave * 2048;
  const uint32_t lds = (uint32_t)(uintptr_t)(lds_ptr_t)smem;
  const ItemOffsets wo = item_offsets((uint32_t)a.ld_w13, (uint32_t)a.ld_s13, lane);

  Feed f;
  auto feed_work = [&](int w) {
    f.live = w < w1;
    f.c = 0;
    f.t = 0;
    if (!f.live) return;
    seek(f.p, works, w);
    const int e = expert_of(a, f.p.slot), i0 = 128 * f.p.tile + 16 * wave;
    f.at[0] = (uint64_t)(uintptr_t)(a.w13 + e * a.st_w13 + (int64_t)i0 * a.ld_w13);
    f.at[1] = f.at[0] + (uint64_t)(a.I * a.ld_w13);
    f.bytes[0] = f.bytes[1] = code_bytes(min(16, a.I - i0), a.ld_w13, nb);
  };
  auto feed = [&]() {
    issue_codes(f, wo, lds + ring);
    f.n = f.n + 1 == kRingW ? 0 : f.n + 1;
    f.t ^= 1;
    if (f.t == 0 && ++f.c == chunks) feed_work(f.p.w + 1);
  };
  // scales of the next group
  Pos sp{0, 0, 0, 0, 0};
  int sc = 0, sw = w0 - 1;
  auto scales = [&]() {
    if (sw < w0 || sc >= chunks) {
      sc = 0;
      if (++sw >= w1) return;
      seek(sp, works, sw);
    }
    const int e = expert_of(a, sp.slot), i0 = 128 * sp.tile + 16 * wave, rows = min(16, a.I - i0);
    issue_scales<GROUP>(a.s13 + e * a.st_s13 + (int64_t)i0 * a.ld_s13, a.ld_s13, a.I * a.ld_s13, rows, rows, nb, sc,
                        lds + my_scales, lane);
    sc += GROUP;
  };
  // X: this wave's two rows of the next stage
  Pos xp{0, 0, 0, 0, 0};
  int xc = -1, xn = 0, xrows = 0;
  bool xlive = true;
  auto stage = [&]() {
    if (xc < 0 || ++xc == chunks) {
      const int w = xc < 0 ? w0 : xp.w + 1, slot = xc < 0 ? -1 : xp.slot, m = xp.m;
      xlive = w < w1;
      xc = 0;
      if (xlive) {
        seek(xp, works, w);
        if (xp.slot != slot || xp.m != m) xrows = rows_of(a, expert_of(a, xp.slot), xp.m, lane);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 2 * wave + r, id = __builtin_amdgcn_readlane(xrows, row);
      const int left = xlive && id > 0 ? min(2 * (a.H - kChunk * xc), 1024) : 0;
      const uint64_t at = (uint64_t)(uintptr_t)a.x + (uint64_t)((id > 0 ? id - 1 : 0) / a.k) * (uint64_t)a.ld_x + 1024u * (uint64_t)xc;
      dma16(lds + kUpX + xn * kStage + 1024 * row, 16u * (uint32_t)(lane ^ row), rsrc_of(at, (uint32_t)left));
    }
    xn ^= 1;
  };

  f.p = Pos{0, 0, 0, 0, 0};
  f.n = 0;
  feed_work(w0);
  scales();
  stage();
  feed();
  feed();
  feed();
  landed<0>();
  meet();
  Pos p{0, 0, 0, 0, 0};
  int xbuf = 0, slot = 0;                                // stage and ring slot of the products
  uint32_t sg[2][GROUP];
  for (int w = w0; w < w1; ++w) {
    seek(p, works, w);
    const int rows = xrows;
    v4f acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
    for (int c = 0; c < chunks; ++c) {
      XWide<1, 1> x;
      x.read_staged(0, kUpX + xbuf * kStage, lane);
      xbuf ^= 1;
      if (c % GROUP == 0) {
        read_scales<GROUP>(sg, my_scales, lane);
        reads_done();
        scales();
      }
      stage();
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        // behind the item: two items and the stages of this chunk and the one before (t = 0), or
        // two items and this chunk's stage
        if (t == 0) landed<12>();
        else landed<10>();
        const uint32_t at = ring + slot * kCodes;
        slot = slot + 1 == kRingW ? 0 : slot + 1;
        v4i wf[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) wf[u] = item_codes(at, lane, u);
        uint32_t ws = sg[t][0];
        sg[t][0] = sg[t][1];
        sg[t][1] = sg[t][2];
        sg[t][2] = sg[t][3];
        if (16 * c + 16 > nb) ws = keep_scales(ws, nb - 16 * c - 4 * g);
        reads_done();
        feed();
        x.mma(wf, ws, &acc[t], 1);
      }
      landed<8>();                                       // this chunk's stage, behind it two items
      meet();
    }
    // lane (i, g): columns 4g .. 4g+3 of the wave's 16, token row i
    const int id = __shfl(rows, i), col = 128 * p.tile + 16 * wave + 4 * g;
    if (id > 0 && (col & ~7) < a.I) {
      const float share = a.share[id - 1];
      float v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = col + q < a.I ? gated(share, acc[0][q], acc[1][q]) : 0.0f;
      store_hidden<KIND>(a.h + ((int64_t)p.slot * a.mt_cap + p.m) * h_chunks * hidden_chunk(KIND) + h_offset<KIND>(i, col & ~7), (col >> 2) & 1, v);
    }
  }
  landed<0>();                                           // no load may land after the workgroup
}

// ---- down.  A stage is half a chunk of h (steps 0, 1 or 2, 3) in the order in which it lies in
// memory.
template <int KIND>
__global__ __launch_bounds__(kT, 1) void k_moe_down_wide(const MoeArgs a) {
  constexpr int GROUP = 2, RING = ring_slots(KIND), STAGE = down_stage(KIND), LOADS = STAGE / (1024 * kW);   // a wave's loads a stage
  int* s_end = reinterpret_cast<int*>(smem + down_lds(KIND));
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
  const int total = count_works(a, a.tiles * a.parts, s_end, lane, wave);
  const int wg = xcd_order(blockIdx.x, gridDim.x);
  const int w0 = (int)((int64_t)total * wg / gridDim.x), w1 = (int)((int64_t)total * (wg + 1) / gridDim.x);
  if (w0 >= w1) return;
  const Works works{s_end, a.tiles, a.parts};
  const int nb = (a.I + 31) / 32, chunks = (a.I + kChunk - 1) / kChunk;
  const uint32_t ring = (uint32_t)wave * (RING * kCodes), my_scales = down_scales(KIND) + (uint32_t)wave * 1024;
  const uint32_t lds = (uint32_t)(uintptr_t)(lds_ptr_t)smem;
  const ItemOffsets wo = item_offsets((uint32_t)a.ld_w2, (uint32_t)a.ld_s2, lane);

  Feed f;
  auto feed_work = [&](int w) {
    f.live = w < w1;
    f.c = f.t = 0;
    f.c1 = 1;
    if (!f.live) return;
    seek(f.p, works, w);
    f.c = chunks * f.p.part / a.parts;
    f.c1 = chunks * (f.p.part + 1) / a.parts;
    const int n0 = 256 * f.p.tile + 32 * wave;
    f.at[0] = (uint64_t)(uintptr_t)(a.w2 + expert_of(a, f.p.slot) * a.st_w2 + (int64_t)n0 * a.ld_w2);
    f.at[1] = f.at[0] + (uint64_t)(16 * a.ld_w2);
    f.bytes[0] = code_bytes(min(16, a.H - n0), a.ld_w2, nb);
    f.bytes[1] = code_bytes(min(16, a.H - n0 - 16), a.ld_w2, nb);
  };
  auto feed = [&]() {
    issue_codes(f, wo, lds + ring);
    f.n = f.n + 1 == RING ? 0 : f.n + 1;
    f.t ^= 1;
    if (f.t == 0 && ++f.c == f.c1) feed_work(f.live ? f.p.w + 1 : w1);
  };
  Pos sp{0, 0, 0, 0, 0};
  int sc = 0, sc1 = 0, sw = w0 - 1;
  auto scales = [&]() {
    if (sc >= sc1) {
      if (++sw >= w1) return;
      seek(sp, works, sw);
      sc = chunks * sp.part / a.parts;
      sc1 = chunks * (sp.part + 1) / a.parts;
    }
    const int n0 = 256 * sp.tile + 32 * wave;
    issue_scales<GROUP>(a.s2 + expert_of(a, sp.slot) * a.st_s2 + (int64_t)n0 * a.ld_s2, a.ld_s2, 16 * a.ld_s2,
                        min(16, a.H - n0), min(16, a.H - n0 - 16), nb, sc, lds + my_scales, lane);
    sc += GROUP;
  };
  Pos xp{0, 0, 0, 0, 0};
  int xs = 0, xs1 = 0, xn = 0, xw = w0 - 1;              // next stage of the work, its end, buffer, work
  uint64_t xat = 0;
  auto stage = [&]() {
    if (xs == xs1 && xw < w1) {
      if (++xw < w1) {
        seek(xp, works, xw);
        xs = 2 * (chunks * xp.part / a.parts);
        xs1 = 2 * (chunks * (xp.part + 1) / a.parts);
        xat = (uint64_t)(uintptr_t)a.h + ((uint64_t)xp.slot * a.mt_cap + xp.m) * (uint64_t)chunks * hidden_chunk(KIND);
      }
    }
    const v4i rs = rsrc_of(xat + (uint64_t)xs * STAGE, xw < w1 ? (uint32_t)STAGE : 0u);
    const uint32_t to = lds + down_x(KIND) + xn * STAGE;
#pragma unroll
    for (int r = 0; r < LOADS; ++r) dma16(to + 1024 * (LOADS * wave + r), (uint32_t)(1024 * (LOADS * wave + r) + 16 * lane), rs);
    if (xw < w1) ++xs;
    xn = xn + 1 == kDownStages ? 0 : xn + 1;
  };

  f.p = Pos{0, 0, 0, 0, 0};
  f.n = 0;
  feed_work(w0);
  scales();
  stage();
  stage();
#pragma unroll
  for (int r = 0; r < RING; ++r) feed();
  landed<0>();
  meet();
  Pos p{0, 0, 0, 0, 0};
  int xbuf = 0, slot = 0, rows = 0, old_slot = -1, old_m = 0;
  uint32_t sg[2][GROUP];
  for (int w = w0; w < w1; ++w) {
    seek(p, works, w);
    if (p.slot != old_slot || p.m != old_m) rows = rows_of(a, expert_of(a, p.slot), p.m, lane);
    old_slot = p.slot;
    old_m = p.m;
    v4f acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
    const int c0 = chunks * p.part / a.parts, c1 = chunks * (p.part + 1) / a.parts;
    for (int c = c0; c < c1; ++c) {
      v4i wf[2][4];
      uint32_t ws[2];
      const bool begins = (c - c0) % GROUP == 0;
#pragma unroll
      for (int hs = 0; hs < 2; ++hs) {
        v4i x[2][4][KIND];
        const uint32_t from = down_x(KIND) + xbuf * STAGE + 16 * lane;
        xbuf = xbuf + 1 == kDownStages ? 0 : xbuf + 1;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int q = 0; q < KIND; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[u][j][q] = lds16(from, ((u * KIND + q) * 4 + j) * 1024);
        if (kChunk * (c + 1) > a.I) {                    // h has nothing at k >= I
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (kChunk * c + 32 * (4 * g + 2 * hs + u) + 8 * j >= a.I) {
#pragma unroll
                for (int q = 0; q < KIND; ++q) x[u][j][q] = v4i{0, 0, 0, 0};
              }
        }
        if (hs == 0 && begins) {
          read_scales<GROUP>(sg, my_scales, lane);
          reads_done();
          scales();
        }
        stage();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (hs == 0) {
            // behind the item, with three slots: two items and four stages (t = 0), or two items and
            // two stages; with two slots: one item and two stages
            if (RING == 2) landed<4 + 2 * LOADS>();
            else if (t == 0) landed<8 + 4 * LOADS>();
            else landed<8 + 2 * LOADS>();
            const uint32_t at = ring + slot * kCodes;
            slot = slot + 1 == RING ? 0 : slot + 1;
#pragma unroll
            for (int u = 0; u < 4; ++u) wf[t][u] = item_codes(at, lane, u);
            ws[t] = sg[t][0];
            sg[t][0] = sg[t][1];
            if (16 * c + 16 > nb) ws[t] = keep_scales(ws[t], nb - 16 * c - 4 * g);
            reads_done();
            feed();
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float s = e8m0_to_f32((ws[t] >> (8 * (2 * hs + u))) & 255u);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t d[4];
              fp4::decode8_bf16((uint32_t)wf[t][2 * hs + u][j], s, d);
              const v4i dv = {(int)d[0], (int)d[1], (int)d[2], (int)d[3]};
#pragma unroll
              for (int q = KIND - 1; q >= 0; --q) acc[t] = mma_bf16(dv, x[u][j][q], acc[t]);
            }
          }
        }
        // the next stage: behind it one stage and two items
        landed<8 + LOADS>();
        meet();
      }
    }
    const int id = __shfl(rows, i);
    if (id > 0) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int n = 256 * p.tile + 32 * wave + 16 * t + 4 * g;
        float* to = a.part + ((int64_t)(id - 1) * a.parts + p.part) * a.H + n;
        if (n + 4 <= a.H) {
          __builtin_memcpy(to, &acc[t], 16);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < a.H) to[e] = acc[t][e];
        }
      }
    }
  }
  landed<0>();
}

}  // namespace wide
}  // namespace

template <int KIND>
hipError_t launch_moe_up_wide(const MoeArgs& args, hipStream_t st) {
  static bool set[64] = {false};
  MoeArgs a = args;
  a.tiles = (a.I + 127) / 128;
  auto kern = wide::k_moe_up_wide<KIND>;
  constexpr int lds = wide::kUpLds;
  const hipError_t e = allow_lds(kern, lds + 4 * 1024, set);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)device_cu_count()), dim3(wide::kT), lds + 4 * a.slots, st, a);
  return hipGetLastError();
}

template hipError_t launch_moe_up_wide<kTwo>(const MoeArgs&, hipStream_t);
template hipError_t launch_moe_up_wide<kThree>(const MoeArgs&, hipStream_t);

template <int KIND>
hipError_t launch_moe_down_wide(const MoeArgs& args, hipStream_t st) {
  static bool set[64] = {false};
  MoeArgs a = args;
  a.tiles = (a.H + 255) / 256;
  auto kern = wide::k_moe_down_wide<KIND>;
  constexpr int lds = wide::down_lds(KIND);
  const hipError_t e = allow_lds(kern, lds + 4 * 1024, set);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)device_cu_count()), dim3(wide::kT), lds + 4 * a.slots, st, a);
  return hipGetLastError();
}

template hipError_t launch_moe_down_wide<kTwo>(const MoeArgs&, hipStream_t);
template hipError_t launch_moe_down_wide<kThree>(const MoeArgs&, hipStream_t);

}  // namespace mxq
