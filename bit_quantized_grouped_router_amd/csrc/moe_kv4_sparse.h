// Attention over the pages that a score selects (see moe_kv4_sparse.hip): the
// selection's shape, its workspace and the launchers.
#pragma once

#include "moe_kv4.h"

namespace moe {

// Pages a token at position pos attends to: 0 .. own, all of them but those
// scored (lo .. hi, empty when hi < lo), of which the best `top`.
struct Kv4Scored {
  int lo, hi, own;
};

MOE_HD Kv4Scored kv4_scored(const Kv4Dims &dm, long long pos, int first, int recent) {
  const long long last = kv4_capacity(dm) - 1;
  Kv4Scored s;
  s.own = pos < 0 ? -1 : (int)((pos < last ? pos : last) >> dm.page_shift);
  s.lo = first;
  s.hi = s.own - recent;
  return s;
}

#ifdef __HIPCC__
struct Kv4Select {
  const uint16_t *bounds;  // [num_pages][Hkv][2][D] bf16
  const uint16_t *q;
  long long q_stride;
  int max_new, top, first, recent;
  int32_t *blocks;  // [T][Hkv][top + first + recent], may be null
};

constexpr int kSelectMostPages = 1 << 20;  // columns of the page table
constexpr int kSelectMostTaken = 4096;     // top + first + recent

size_t kv4_sparse_ws(const Kv4Dims &dm, int T, const Kv4Select &sel);
hipError_t launch_kv4_bounds(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Batch &bt, uint16_t *bounds,
                             hipStream_t s);
hipError_t launch_kv4_sparse(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc, const Kv4Batch &bt,
                             const Kv4Select &sel, uint16_t *out, long long out_stride, float scale, void *ws,
                             hipStream_t s);
#endif

}  // namespace moe
