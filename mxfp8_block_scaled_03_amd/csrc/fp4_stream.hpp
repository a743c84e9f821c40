// fp4_stream.hpp -- the product of few rows X with streamed MXFP4 weights on gfx950, as the expert
// layer uses it (moe_fp4.hip, moe_fp4_wide.hip): a workgroup multiplies 16 * NTW rows of W with
// 16 * MT rows of X, its waves splitting the work along K.  The weights are read once and bound the
// time, so everything is arranged to keep their loads in flight.
//
// An item is 16 rows of W x 512 elements of K: 4 KiB of codes and 16 scale bytes a row.  It
// moves to LDS by DMA in whole 256-byte row pieces (4 rows an instruction; fragment-shaped
// register loads, 16 bytes of 16 different rows by neighbouring lanes, cost the address unit
// four times as much), into a ring of four slots that belongs to one wave: no barriers, 16 KiB in
// flight per wave, 128 KiB per CU.  The 16-byte block b of row r lies at position b ^ r, which makes
// the fragment reads conflict free.
//
// A step u (of 4) multiplies blocks u, 4 + u, 8 + u, 12 + u of the item: lane l = 16 g + i
// holds block 4g + u of row i, so its scale bytes for the four steps are one dword.  The block's 32
// codes are decoded with their scale to bf16 (exact) and feed four v_mfma_f32_16x16x32_bf16 (exact
// products, FP32 sums); MFMA j holds elements 8j .. 8j+7.  Both operands share the assignment of k to
// (step, lane group, element), so any is right.  W is the A operand: lane (i, g) ends up with W
// rows 4g .. 4g+3 (output columns) of X row i.
//
// The items of a workgroup, chunk of K by chunk and row tile by row tile inside one, are dealt to
// its waves in equal runs.  A wave keeps the X fragments of its chunk in registers and sums
// for every row tile; the waves' sums meet in LDS at the end and are added in wave order.
#pragma once
#include "codec4.hpp"
#include "fp4_ranges.hpp"
#include "gemm_common.hpp"

namespace mxq {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kChunk = 512;                  // elements of K per item
constexpr int kSlot = 4096 + 256;            // codes and scales of an item
constexpr int kRing = 4;
constexpr int kWaveLds = kRing * kSlot;

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 4 bytes per lane into LDS at lds + 4 * lane.
__device__ __forceinline__ void dma4(uint32_t lds, uint32_t voff, v4i rsrc) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// This wave's LDS reads are complete: its slots may be written again.
__device__ __forceinline__ void reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Keep the first n (any int) of the 32 codes in four dwords.
__device__ __forceinline__ v4i keep_codes(v4i v, int n) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int r = n - 8 * d;
    const uint32_t m = r >= 8 ? 0xFFFFFFFFu : r <= 0 ? 0u : (1u << (4 * r)) - 1u;
    v[d] = (int)((uint32_t)v[d] & m);
  }
  return v;
}

// Scale bytes of four blocks, of which the first n (any int) exist: the others are 127.
__device__ __forceinline__ uint32_t keep_scales(uint32_t s, int n) {
  const uint32_t m = n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
  return (s & m) | (0x7F7F7F7Fu & ~m);
}

// Consecutive rows of codes and scales (uniform).  Row tiles from `first` on lie `far_c` and
// `far_s` bytes further (the up rows behind the gate rows of an expert).
struct Lines {
  uint64_t c, s;
  uint32_t c_bytes, s_bytes;
  uint32_t ld_c, ld_s;
  bool s_words;                              // scale rows are whole 4-byte words
  int first;
  uint64_t far_c, far_s;
};

__device__ __forceinline__ Lines lines_of(const uint8_t* c, int64_t ld_c, const uint8_t* s, int64_t ld_s, int rows,
                                          int nb, bool s_words) {
  Lines l;
  l.c = (uint64_t)(uintptr_t)c;
  l.s = (uint64_t)(uintptr_t)s;
  l.ld_c = (uint32_t)ld_c;
  l.ld_s = (uint32_t)ld_s;
  l.c_bytes = (uint32_t)((int64_t)(rows - 1) * ld_c + 16 * nb);
  l.s_bytes = scale_bytes(rows, ld_s, nb, s_words);
  l.s_words = s_words;
  l.first = 1 << 30;
  l.far_c = l.far_s = 0;
  return l;
}

// The lane's offsets in an item: code instruction d covers rows 4d .. 4d+3.
struct ItemOffsets {
  uint32_t c[4], s;
};

__device__ __forceinline__ ItemOffsets item_offsets(uint32_t ld_c, uint32_t ld_s, int lane) {
  ItemOffsets o;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const uint32_t r = 4u * d + (uint32_t)(lane >> 4);
    o.c[d] = r * ld_c + 16u * ((uint32_t)(lane & 15) ^ r);
  }
  o.s = (uint32_t)(lane >> 2) * ld_s + 4u * (uint32_t)(lane & 3);
  return o;
}

// Rows 16 t .. 16 t + 15, chunk c, into the slot at `lds`: five loads, or four where scales are
// not read by words.  What lies past the last row's end reads as zero.
__device__ __forceinline__ void issue_item(const Lines& l, const ItemOffsets& o, int t, int c, uint32_t lds) {
  const bool far = t >= l.first;
  const uint32_t n = (uint32_t)(far ? t - l.first : t);
  const uint32_t oc = 16u * n * l.ld_c + 256u * c, os = 16u * n * l.ld_s + 16u * c;
  const v4i rc = rsrc_of(l.c + (far ? l.far_c : 0) + oc, oc < l.c_bytes ? l.c_bytes - oc : 0u);
#pragma unroll
  for (int d = 0; d < 4; ++d) dma16(lds + 1024 * d, o.c[d], rc);
  if (l.s_words) dma4(lds + 4096, o.s, rsrc_of(l.s + (far ? l.far_s : 0) + os, os < l.s_bytes ? l.s_bytes - os : 0u));
}

// Step u's fragment of the item in the slot at byte `slot` of LDS.
__device__ __forceinline__ v4i item_codes(uint32_t slot, int lane, int u) {
  const uint32_t i = lane & 15, b = 4u * (lane >> 4) + u;
  return lds16(slot + 256u * i + 16u * (b ^ i), 0);
}

// The scale bytes of blocks 4g .. 4g+3 of row i of rows 16 t .., chunk c; blocks past nb: 127.
__device__ __forceinline__ uint32_t item_scales(const Lines& l, uint32_t slot, int t, int c, int nb, int lane) {
  const int i = lane & 15, g = lane >> 4;
  const int left = nb - 16 * c - 4 * g;
  uint32_t s = 0;
  if (l.s_words) {
    s = *reinterpret_cast<const uint32_t*>(smem + slot + 4096 + 16 * i + 4 * g);
  } else {
    const bool far = t >= l.first;
    const uint64_t at = (uint64_t)(16 * (far ? t - l.first : t) + i) * l.ld_s + 16 * c + 4 * g;
    const uint8_t* p = reinterpret_cast<const uint8_t*>(l.s + (far ? l.far_s : 0));
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (u < left && at + u < l.s_bytes) s |= (uint32_t)p[at + u] << (8 * u);
  }
  return 16 * c + 16 > nb ? keep_scales(s, left) : s;
}

template <int U>
__device__ __forceinline__ v4f mma_fp4(v4i a, uint32_t sa, v4i b, uint32_t sb, v4f acc) {
  const v8i wa = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, wb = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, wb, acc, 4, 4, U, (int)sa, U, (int)sb);
}

__device__ __forceinline__ v4f mma_bf16(v4i w, v4i x, v4f acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, w), __builtin_bit_cast(v8bf, x), acc, 0, 0, 0);
}

// Eight 16-bit elements without the first n (0 .. 7), zeros behind.
__device__ __forceinline__ v4i drop_low(v4i v, int n) {
  uint32_t d[4] = {(uint32_t)v[0], (uint32_t)v[1], (uint32_t)v[2], (uint32_t)v[3]};
  if (n & 4) {
    d[0] = d[2];
    d[1] = d[3];
    d[2] = d[3] = 0;
  }
  if (n & 2) {
    d[0] = d[1];
    d[1] = d[2];
    d[2] = d[3];
    d[3] = 0;
  }
  if (n & 1) {
    d[0] = __builtin_amdgcn_alignbit(d[1], d[0], 16);
    d[1] = __builtin_amdgcn_alignbit(d[2], d[1], 16);
    d[2] = __builtin_amdgcn_alignbit(d[3], d[2], 16);
    d[3] >>= 16;
  }
  return v4i{(int)d[0], (int)d[1], (int)d[2], (int)d[3]};
}

// ---- X fragments of a chunk.

// What the fragments hold of an element: a bf16 (rows of X), or the two or three bf16 that add up to a
// hidden value, 16 or all 24 of its significant bits, a plane of 16 bytes per 8 elements each.
enum : int { kOne = 1, kTwo = 2, kThree = 3 };

template <int MT, int KIND>
struct XWide {
  v4i f[4][4][MT][KIND];                     // step, MFMA, row tile, plane: the smallest term last

  __device__ __forceinline__ void mma(const v4i w[4], uint32_t ws, v4f* acc, int stride) const {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float s = e8m0_to_f32((ws >> (8 * u)) & 255u);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t d[4];
        fp4::decode8_bf16((uint32_t)w[u][j], s, d);
        const v4i dv = {(int)d[0], (int)d[1], (int)d[2], (int)d[3]};
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int p = KIND - 1; p >= 0; --p) acc[m * stride] = mma_bf16(dv, f[u][j][m][p], acc[m * stride]);
      }
    }
  }

  // Straight from memory: the lane's row at the chunk, whether it is one, the elements left in it
  // and the row's length.  A piece that the row's end cuts is read from the last 8 elements.
  __device__ __forceinline__ void load_direct(int m, const uint8_t* row, bool live, int left, int K, int lane) {
    const int g = lane >> 4;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = 32 * (4 * g + u) + 8 * j;
        v4i v = {0, 0, 0, 0};
        if (live && k < left && K >= 8) __builtin_memcpy(&v, row + 2 * min(k, left - 8), 16);
        f[u][j][m][0] = v;
      }
    if (left < kChunk) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = 32 * (4 * g + u) + 8 * j, cut = k < left ? max(k + 8 - left, 0) : 0;
          f[u][j][m][0] = drop_low(f[u][j][m][0], cut);
        }
    }
    if (K < 8 && g == 0 && live) {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < K) f[0][0][m][0][e >> 1] |= (int)((uint32_t)reinterpret_cast<const uint16_t*>(row)[e] << (16 * (e & 1)));
    }
  }

  // From 16 rows of 1 KiB in LDS, 16-byte piece p of row r at p ^ r.
  __device__ __forceinline__ void read_staged(int m, uint32_t lds, int lane) {
    const uint32_t i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) f[u][j][m][0] = lds16(lds + 1024u * i + 16u * ((16u * g + 4u * u + j) ^ i), 0);
  }
};

// Stage 16 rows of X in bf16 (1 KiB of chunk c each) in the wave's ring: row r's pointer comes
// from lane r of `row`, rows past `rows` are left as they are.
__device__ __forceinline__ void stage_rows(uint64_t row, int rows, int c, uint32_t lds, int lane) {
  for (int r = 0; r < rows; ++r) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)row, r);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(row >> 32), r);
    const uint64_t at = (((uint64_t)hi << 32) | lo) + 1024u * (uint64_t)c;
    dma16(lds + 1024 * r, 16u * (uint32_t)(lane ^ r), rsrc_of(at, 1024u));
  }
}

// ---- the stream.  A wave's run of items [it0, it1), item c * NTW + t being row tile t of chunk c.
struct Run {
  int it0, it1;
};

template <int NTW>
__device__ __forceinline__ Run run_of(int K, int wave) {
  const int items = ((K + kChunk - 1) / kChunk) * NTW;
  return Run{items * wave / kWaves, items * (wave + 1) / kWaves};
}

// Starts the DMA of up to a ring's worth of items from `it` on, those before `end`.  A loop: what a
// workgroup runs but once is paid for in instruction fetches.
template <int NTW, typename Issue>
__device__ __forceinline__ void fill_ring(int it, int end, uint32_t lds0, Issue issue) {
#pragma unroll 1
  for (int n = 0; n < min(kRing, end - it); ++n)
    issue((int)((uint32_t)(it + n) % NTW), (int)((uint32_t)(it + n) / NTW), lds0 + n * kSlot);
}

// issue(t, c, lds) starts an item's DMA; load_x(x, c) brings a chunk's X fragments;
// scales_of(t, c, slot) gives an item's scale dword.  acc[m][t] sums row tile m of X, t of W.
// through: load_x leaves the ring alone, so items of the next chunk are in flight already when
// a chunk ends, and the caller has filled the ring for the first one; otherwise X passes
// through the ring and every chunk starts with it empty.
template <typename X, int MT, int NTW, typename Issue, typename Load, typename Scales>
__device__ __forceinline__ void stream(Run run, int wave, int lane, bool s_words, bool through, Issue issue, Load load_x,
                                       Scales scales_of, v4f acc[MT][NTW]) {
  const uint32_t ring = (uint32_t)wave * kWaveLds;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)smem + ring;
  int n = 0;                                             // the slot of the next item
  for (int c = run.it0 / NTW; c * NTW < run.it1; ++c) {
    const int lo = max(run.it0 - c * NTW, 0), hi = min(run.it1 - c * NTW, NTW);
    const int end = through ? run.it1 : c * NTW + hi;    // items that may be in flight
    X x;
    load_x(x, c);
    if (!through) {
      fill_ring<NTW>(c * NTW + lo, end, lds0, issue);
      n = 0;
    }
#pragma unroll
    for (int t = 0; t < NTW; ++t) {
      if (t < lo || t >= hi) continue;
      const int it = c * NTW + t;
      // in flight behind this item: up to three more
      const int after = end - 1 - it;
      if (!s_words || after == 0)
        wait_vm<0>();
      else if (after == 1)
        wait_vm<5>();
      else if (after == 2)
        wait_vm<10>();
      else
        wait_vm<15>();
      asm volatile("" ::: "memory");
      const uint32_t slot = ring + n * kSlot;
      v4i w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) w[u] = item_codes(slot, lane, u);
      const uint32_t ws = scales_of(t, c, slot);
      reads_done();
      if (it + kRing < end) issue((int)((uint32_t)(it + kRing) % NTW), (int)((uint32_t)(it + kRing) / NTW), lds0 + n * kSlot);
      n = (n + 1) % kRing;
      x.mma(w, ws, &acc[0][t], NTW);
    }
  }
}

// The waves' sums side by side in LDS: wave w's value of X row m, W row n is at [w][m][n], rows
// of 16 * NTW + 4 floats.
template <int NTW>
constexpr int part_row() { return 16 * NTW + 4; }
template <int MT, int NTW>
constexpr int part_wave() { return 16 * MT * part_row<NTW>(); }
template <int MT, int NTW>
constexpr int stream_lds() {
  return part_wave<MT, NTW>() * 4 > kWaveLds ? kWaves * part_wave<MT, NTW>() * 4 : kWaves * kWaveLds;
}

template <int MT, int NTW>
__device__ __forceinline__ void store_part(int wave, int lane, const v4f acc[MT][NTW]) {
  float* part = reinterpret_cast<float*>(smem);
  const int i = lane & 15, g = lane >> 4;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NTW; ++n)
      *reinterpret_cast<v4f*>(part + wave * part_wave<MT, NTW>() + (16 * m + i) * part_row<NTW>() + 16 * n + 4 * g) =
          acc[m][n];
}

// Sum over the waves, in wave order, of X row m, W rows n .. n+3.
template <int MT, int NTW>
__device__ __forceinline__ v4f sum_part(int m, int n) {
  const float* part = reinterpret_cast<const float*>(smem);
  v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int w = 0; w < kWaves; ++w)
    s += *reinterpret_cast<const v4f*>(part + w * part_wave<MT, NTW>() + m * part_row<NTW>() + n);
  return s;
}

// Raises a kernel's LDS limit once per device.
template <typename K>
hipError_t allow_lds(K kern, int lds, bool set[64]) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) dev = 0;
  if (set[dev]) return hipSuccess;
  const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e == hipSuccess) set[dev] = true;
  return e;
}

}  // namespace
}  // namespace mxq
