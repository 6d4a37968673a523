// Launcher of the dense int4-g64 projection (see moe_linear.hip).
#pragma once

#include "moe_device.h"

namespace moe {

enum { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };

struct LinearArgs {
  int T, rows, cols;
  const uint16_t *x;
  long long x_stride;
  W4 w;
  const uint16_t *bias;  // null: none
  int act;
  const void *residual;  // null: none; the type of y
  long long r_stride;
  void *y;
  long long y_stride;
};

bool linear_grid_ok(const LinearArgs &a);
// dtype of y and the residual: 0 bf16, 1 fp32
hipError_t launch_linear(const LinearArgs &a, int dtype, hipStream_t s);

}  // namespace moe
