// Dense projection with int4-g64 weights:
//   y[t][n] = act(sum_c x[t][c] W[n][c] + bias[n]) + residual[t][n],
//   W = bf16(fp32(s q + b)), products of bf16 values exact, sums in fp32.
//
// Small batches are bound by the weights' bytes. One workgroup takes 16
// weight rows and 16, 32 or 64 tokens; its 8 wavefronts take the 64-column
// groups in turn, rebuild them in registers as the A operand of 16x16x32
// MFMAs (lane l: row l % 16, columns 16 (l / 16) .. +15 of the group) against
// the tokens' activations read straight from memory, and join their sums
// through LDS, where the epilogue runs.
#include "moe_linear.h"

namespace moe {

constexpr int kLnWaves = 8;
constexpr int kLnRows = 16;

__device__ __forceinline__ float activate(float z, int act) {
  if (act == kActRelu) return z > 0.f ? z : (z == z ? 0.f : z);
  if (act == kActSilu) return z / (1.0f + expf(-z));
  if (act == kActGelu) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
  return z;
}

// Bias, activation and residual of one output, and its store.
template <bool F32>
__device__ __forceinline__ void linear_store(const LinearArgs &a, int t, int n, float z) {
  if (a.bias) z += bf16_to_f32(a.bias[n]);
  z = activate(z, a.act);
  if (F32) {
    if (a.residual) z += ((const float *)a.residual)[t * a.r_stride + n];
    ((float *)a.y)[t * a.y_stride + n] = z;
  } else {
    if (a.residual) z += bf16_to_f32(((const uint16_t *)a.residual)[t * a.r_stride + n]);
    ((uint16_t *)a.y)[t * a.y_stride + n] = to_bf16(z);
  }
}

template <int NT, bool F32>
__global__ __launch_bounds__(kLnWaves *kWave) void linear_kernel(LinearArgs a) {
  __shared__ float part[kLnWaves][16 * NT][kLnRows + 1];
  const int blocks = (a.rows + kLnRows - 1) / kLnRows;
  const int n0 = (blockIdx.x % blocks) * kLnRows, t0 = (blockIdx.x / blocks) * 16 * NT;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c16 = (lane >> 4) * 16;
  const int ng = a.cols / kGroup;
  const long long wrow = min(n0 + (lane & 15), a.rows - 1);
  const uint8_t *codes = a.w.codes + wrow * (a.cols / 2) + c16 / 2;
  const uint16_t *sp = a.w.scales + wrow * ng, *bp = a.w.biases + wrow * ng;
  const uint16_t *xp[NT];
  f32x4_t acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int t = min(t0 + i * 16 + (lane & 15), a.T - 1);
    xp[i] = a.x + t * a.x_stride + c16;
    acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  for (int g = wave; g < ng; g += kLnWaves) {
    const uint2 c = *(const uint2 *)(codes + g * 32);
    const float s = bf16_to_f32(sp[g]), b = bf16_to_f32(bp[g]);
    uint4 x[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      x[i][0] = *(const uint4 *)(xp[i] + g * kGroup);
      x[i][1] = *(const uint4 *)(xp[i] + g * kGroup + 8);
    }
    const bf16x8_t w0 = __builtin_bit_cast(bf16x8_t, dequant8(c.x, s, b));
    const bf16x8_t w1 = __builtin_bit_cast(bf16x8_t, dequant8(c.y, s, b));
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0, __builtin_bit_cast(bf16x8_t, x[i][0]), acc[i], 0, 0, 0);
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w1, __builtin_bit_cast(bf16x8_t, x[i][1]), acc[i], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) part[wave][i * 16 + (lane & 15)][(lane >> 4) * 4 + r] = acc[i][r];
  __syncthreads();
  for (int e = threadIdx.x; e < 16 * NT * kLnRows; e += kLnWaves * kWave) {
    const int t = e / kLnRows, n = e % kLnRows;
    if (t0 + t >= a.T || n0 + n >= a.rows) continue;
    float z = 0.f;
#pragma unroll
    for (int w = 0; w < kLnWaves; ++w) z += part[w][t][n];
    linear_store<F32>(a, t0 + t, n0 + n, z);
  }
}

static long long linear_blocks(int T, int rows) {
  return (long long)((rows + kLnRows - 1) / kLnRows) * ((T + 15) / 16);
}

bool linear_grid_ok(int T, int rows) { return linear_blocks(T, rows) < (1ll << 31); }

template <int NT>
static void launch(const LinearArgs &a, int dtype, hipStream_t s) {
  const int grid = (int)((long long)((a.rows + kLnRows - 1) / kLnRows) * ((a.T + 16 * NT - 1) / (16 * NT)));
  auto *kernel = dtype ? linear_kernel<NT, true> : linear_kernel<NT, false>;
  kernel<<<grid, kLnWaves * kWave, 0, s>>>(a);
}

hipError_t launch_linear(const LinearArgs &a, int dtype, hipStream_t s) {
  if (a.T <= 16)
    launch<1>(a, dtype, s);
  else if (a.T <= 32)
    launch<2>(a, dtype, s);
  else
    launch<4>(a, dtype, s);
  return hipGetLastError();
}

}  // namespace moe
