// Rotary positions: what a call passes, and the launchers (see moe_rope.hip).
#pragma once

#include "moe_device.h"
#include "moe_kv4.h"

namespace moe {

constexpr int kRopeMaxD = 512;

struct Rope {
  const float *freqs;  // radians a position, [rot / 2]
  int rot;             // the first rot channels turn
  bool interleaved;    // pairs (2i, 2i + 1), otherwise (i, i + rot / 2)
  float magnitude;
};

struct HeadNorm {
  const uint16_t *weight;  // null: no norm
  float eps;
  bool plus_one;
};

// dtype: 0 bf16, 1 fp32
hipError_t launch_rope(int T, int H, int D, const void *x, long long x_stride, int x_dtype, const int32_t *positions,
                       const Rope &rope, const HeadNorm &norm, void *out, long long out_stride, int out_dtype,
                       hipStream_t s);

struct RopeAppend {
  const void *q, *k, *v;  // of one type
  long long q_stride, k_stride, v_stride;
  uint16_t *out;  // rotated queries
  long long out_stride;
  HeadNorm q_norm, k_norm;
};

hipError_t launch_kv4_rope_append(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc, const Kv4Batch &bt,
                                  const Rope &rope, const RopeAppend &a, int dtype, hipStream_t s);

}  // namespace moe
