// Launcher of the root-mean-square norm (see moe_norm.hip).
#pragma once

#include "moe_device.h"

namespace moe {

enum { kOutBf16 = 0, kOutF32 = 1, kOutE4m3 = 2, kOutInt8 = 3 };

struct NormArgs {
  int T, d;
  const void *x;
  long long x_stride;
  const void *r;  // null: none
  long long r_stride;
  void *h;  // null: not stored; the type of r
  long long h_stride;
  const uint16_t *weight;
  float eps;
  bool plus_one;
  void *y;
  long long y_stride;
  int out;
  float *scales;  // 8-bit outputs
  int group;      // channels that share one
};

constexpr int kNormMaxD = 32768;

// x_dtype, r_dtype: 0 bf16, 1 fp32
hipError_t launch_rmsnorm(const NormArgs &a, int x_dtype, int r_dtype, hipStream_t s);

}  // namespace moe
