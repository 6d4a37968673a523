// Device code shared by the two attention kernels over the 4-bit cache.
#pragma once

#include "moe_device.h"
#include "moe_kv4.h"

namespace moe {

constexpr float kNegInf = -__builtin_huge_valf();

constexpr float kLog2e = 1.4426950408889634f;

// Scaled log2 units a score may exceed the running reference by before the
// accumulators are rescaled: weights stay below 2^8, far from overflow, and
// the rescale runs once or twice a row instead of at every new maximum. The
// reference is kept unscaled and a weight is exp2((score - reference) * scale):
// the difference to a near reference is exact, so this holds for scores of any
// size, where the difference of two scaled scores would be off by a step of
// theirs (128 from 2^31 on, an overflow).
constexpr float kSlack = 8.0f;

typedef const __attribute__((address_space(4))) int32_t kv_const_i32;

// Pages of a tile's two halves (-1: no place).
struct TilePages {
  int page[2];
};

// The page table's entries (scalar loads), to be looked at a tile later, when
// they have arrived.
__device__ __forceinline__ TilePages tile_entries(const Kv4Dims &dm, const int32_t *table, int tile) {
  TilePages p;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const long long t = (long long)tile * kKvTile + 16 * u;
    p.page[u] = ((kv_const_i32 *)table)[t < kv4_capacity(dm) ? (int)(t >> dm.page_shift) : 0];
  }
  return p;
}

__device__ __forceinline__ TilePages tile_pages(const Kv4Dims &dm, const TilePages &entries, int tile) {
  TilePages p;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const bool in = (long long)tile * kKvTile + 16 * u < kv4_capacity(dm);
    p.page[u] = in && kv4_page_ok(dm, entries.page[u]) ? entries.page[u] : -1;
  }
  return p;
}

// Query rows of a workgroup: row r of a sequence and cache head is new token
// r / G, head (cache head) * G + r % G.
struct RowTile {
  int seq, head, row0, rows;  // rows: rows of this sequence and head (n * G)
  Kv4Span sp;
};

__device__ __forceinline__ RowTile row_tile(const Kv4Dims &dm, const Kv4Batch &bt, int max_new,
                                            int tile, int head, int seq, int rows_tile) {
  RowTile t;
  t.head = head;
  t.seq = seq;
  t.row0 = tile * rows_tile;
  t.sp = kv4_span(bt.cu[seq], bt.cu[seq + 1], bt.len[seq], bt.T);
  t.rows = min(t.sp.n, max_new) * (dm.Hq / dm.Hkv);
  return t;
}

// Partial results of row r of a row tile, split `split` of `splits`: D sums at
// part + index * D; reference and sum of weights, all rows' after all sums.
__device__ __forceinline__ long long part_index(const Kv4Dims &dm, const Kv4Attn &at, const RowTile &t, int r,
                                                int splits, int split) {
  const int G = dm.Hq / dm.Hkv, x = t.row0 + r;
  const long long first = at.room > 0 ? (long long)t.seq * at.room : t.sp.begin;
  return ((first + x / G) * dm.Hq + t.head * G + x % G) * splits + split;
}

__device__ __forceinline__ float *part_stats(const Kv4Dims &dm, const Kv4Batch &bt, const Kv4Attn &at, int splits,
                                             float *part) {
  const long long tokens = at.room > 0 ? (long long)dm.B * at.room : bt.T;
  return part + tokens * dm.Hq * splits * dm.D;
}

// Fewest tiles a split of the prefill kernel's keys has.
constexpr int kPfMinTiles = 32;

}  // namespace moe
