// Root-mean-square norm of rows, with the residual's addition before it.
//
//   s = x + r,   h = s rounded to r's type,   y = s / sqrt(mean s^2 + eps) * w
// with w the weight or 1 + the weight. To 8 bits: per group of channels a = max
// |y|, scale = a / 448 (e4m3) or a / 127 (int8), q = y / scale rounded to
// nearest, ties to even. Everything up to the last rounding is fp32; the norm
// is that of the unrounded sum.
//
// Bound by memory: one pass, a row stays in registers between the sum of its
// squares and its output. L threads take a row, 8 channels (one 16-byte or two)
// at a time and C times, so that a group of 64 or 128 channels is 8 or 16
// neighbouring lanes and its maximum three or four DPP steps. us: 8192 x 2048 in fp32
// with an fp32 residual 43.0 (235 MB, 5.5 TB/s); 777 x 5120 in bf16 to e4m3 10.1 (28 MB,
// 2.8 TB/s: three or four rows a CU, so that little overlaps); one row 2.3. Where the width
// or a stride is no multiple of 8, all is read and written element by element, and rows
// above 8192 channels spill (124 to 324 bytes a lane): 4096 x 2047 52 (2048 channels: 17),
// 4096 x 12001 641 (12000: 126).
#include "moe_norm.h"

namespace moe {

constexpr int kNormThreads = 256;

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// Channels at .. at + 7 of a row as they lie in memory (F32: 8 words, else 4). Lanes past the
// row's n channels load its first ones, so that all of a thread's loads are under way
// together: under a condition each would be waited for (4096 rows in bf16 with an fp32
// residual, 5120 channels 43 us, so 38; 16384 channels 216 and 151).
template <bool F32>
struct Raw8 {
  u32x4_t v[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ void norm_load8(const void *row, int at, int n, Raw8<F32> &x) {
  const int c = at < n ? at : 0;
  if constexpr (F32) {
    x.v[0] = *(const u32x4_t *)((const float *)row + c);
    x.v[1] = *(const u32x4_t *)((const float *)row + c + 4);
  } else {
    x.v[0] = *(const u32x4_t *)((const uint16_t *)row + c);
  }
}

template <bool F32>
__device__ __forceinline__ void norm_unpack8(const Raw8<F32> &r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (F32)
      x[i] = __uint_as_float(r.v[i / 4][i % 4]);
    else
      x[i] = __uint_as_float((i & 1) ? r.v[0][i / 2] & 0xFFFF0000u : r.v[0][i / 2] << 16);
  }
}

// Channels at .. at + 7 of a row of any alignment, those from n on as 0.
template <bool F32>
__device__ __forceinline__ void norm_gather8(const void *row, int at, int n, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = 0.f;
    if (at + i < n) x[i] = F32 ? ((const float *)row)[at + i] : bf16_to_f32(((const uint16_t *)row)[at + i]);
  }
}

// A thread's C times 8 channels of a row, L * 8 apart. VEC: loaded in whole 16 bytes, all at
// once; otherwise where they are asked for.
template <int L, int C, bool F32, bool VEC>
struct RowPart {
  const void *row;
  int lane, n;
  Raw8<F32> raw[VEC ? C : 1];

  __device__ __forceinline__ RowPart(const void *row, int lane, int n) : row(row), lane(lane), n(n) {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < C; ++j) norm_load8<F32>(row, (lane + j * L) * 8, n, raw[j]);
    }
  }

  __device__ __forceinline__ void get(int j, float (&v)[8]) const {
    if constexpr (VEC)
      norm_unpack8<F32>(raw[j], v);
    else
      norm_gather8<F32>(row, (lane + j * L) * 8, n, v);
  }
};

template <bool VEC>
__device__ __forceinline__ void norm_store8(void *row, bool f32, int at, int n, const float (&x)[8]) {
  if constexpr (VEC) {
    if (f32) {
      *(float4 *)((float *)row + at) = make_float4(x[0], x[1], x[2], x[3]);
      *(float4 *)((float *)row + at + 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      *(uint4 *)((uint16_t *)row + at) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                    pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at + i < n) {
        if (f32)
          ((float *)row)[at + i] = x[i];
        else
          ((uint16_t *)row)[at + i] = to_bf16(x[i]);
      }
  }
}

// Sum of the L threads of a row, the same in each; sm is the row's own.
template <int L>
__device__ __forceinline__ float row_sum(float v, float *sm) {
  v = wave_sum_dpp(v);
  if constexpr (L > kWave) {
    __syncthreads();  // what the row before left has been read
    if ((threadIdx.x & (kWave - 1)) == 0) sm[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < L / kWave; ++i) v += sm[i];
  }
  return v;
}

template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *sm) {
  v = wave_max_u32(v);
  if constexpr (L > kWave) {
    __syncthreads();
    if ((threadIdx.x & (kWave - 1)) == 0) sm[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < L / kWave; ++i) v = max(v, sm[i]);
  }
  return v;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false));
}

// Bit pattern of a group's largest |y| (an infinity's or a NaN's is larger than
// any finite one's) as its scale, NaN where the group is not finite.
__device__ __forceinline__ float group_scale(uint32_t top, float largest) {
  return top >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float(top) / largest;
}

// Eight values over their scale, rounded; zeros where that is 0 or NaN. With the
// rounded reciprocal and one step of the remainder a quotient is the rounded one, in
// three operations instead of a division's ten, while nothing under- or overflows.
__device__ __forceinline__ uint2 to_8bit(const float (&y)[8], float scale, bool e4m3) {
  const float largest = e4m3 ? 448.f : 127.f;
  float t[8];
  if (scale >= 0x1p-60f && scale <= 0x1p60f) {
    const float inv = 1.0f / scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = y[i] * inv;
      t[i] = fmaf(fmaf(-q, scale, y[i]), inv, q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = scale > 0.f ? y[i] / scale : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = __builtin_amdgcn_fmed3f(t[i], -largest, largest);  // no NaN is left
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float *p = t + 4 * i;
    if (e4m3) {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(p[0], p[1], 0, false);
      w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(p[2], p[3], lo, true);
    } else {
      w[i] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[i] |= ((uint32_t)(int)rintf(p[j]) & 0xFFu) << (8 * j);
    }
  }
  return make_uint2(w[0], w[1]);
}

// RK: the residual's type, 0 none, 1 bf16, 2 fp32. A workgroup takes its rows in
// steps of the grid (launch_norm bounds it).
template <int L, int C, bool X32, int RK, bool VEC>
__global__ __launch_bounds__(L > kNormThreads ? L : kNormThreads) void rmsnorm_kernel(NormArgs a) {
  constexpr int kThreads = L > kNormThreads ? L : kNormThreads, kRows = kThreads / L;
  __shared__ uint32_t sm[kThreads / kWave];
  const int lane = threadIdx.x % L;
  const float largest = a.out == kOutE4m3 ? 448.f : 127.f;
  for (long long row = (long long)blockIdx.x * kRows + threadIdx.x / L; row < a.T; row += (long long)gridDim.x * kRows) {
    const char *x = (const char *)a.x + row * a.x_stride * (X32 ? 4 : 2);
    const char *r = (const char *)a.r + row * a.r_stride * (RK == 2 ? 4 : 2);
    const RowPart<L, C, X32, VEC> px(x, lane, a.d);
    const RowPart<L, C, RK == 2, VEC && RK != 0> pr(r, lane, a.d);
    const RowPart<L, C, false, VEC> pw(a.weight, lane, a.d);
    float s[C][8], sum = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      px.get(j, s[j]);
      if constexpr (RK != 0) {
        float v[8];
        pr.get(j, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j][i] += v[i];
      }
      const bool in = (lane + j * L) * 8 < a.d;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[j][i] = in ? s[j][i] : 0.f;
        sum = fmaf(s[j][i], s[j][i], sum);
      }
    }
    sum = row_sum<L>(sum, (float *)sm);
    if (RK != 0 && a.h != nullptr) {
      char *h = (char *)a.h + row * a.h_stride * (RK == 2 ? 4 : 2);
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int at = (lane + j * L) * 8;
        if (at < a.d) norm_store8<VEC>(h, RK == 2, at, a.d, s[j]);
      }
    }
    const float inv = 1.0f / sqrtf(sum / (float)a.d + a.eps), one = a.plus_one ? 1.f : 0.f;
    uint32_t top[C];
#pragma unroll
    for (int j = 0; j < C; ++j) {
      float w[8];
      pw.get(j, w);
      const bool in = (lane + j * L) * 8 < a.d;  // the others' weights are not theirs
      top[j] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[j][i] = s[j][i] * inv * ((in ? w[i] : 0.f) + one);
        top[j] = max(top[j], __float_as_uint(s[j][i]) & 0x7FFFFFFFu);
      }
    }
    if (a.out <= kOutF32) {
      char *y = (char *)a.y + row * a.y_stride * (a.out == kOutF32 ? 4 : 2);
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int at = (lane + j * L) * 8;
        if (at < a.d) norm_store8<VEC>(y, a.out == kOutF32, at, a.d, s[j]);
      }
      continue;
    }
    uint8_t *y = (uint8_t *)a.y + row * a.y_stride;
    const int shift = a.group == a.d ? 30 : a.group == 128 ? 7 : 6, mask = (1 << shift) - 1;  // d < 2^30
    uint32_t all = 0;
    if (a.group == a.d) {
#pragma unroll
      for (int j = 0; j < C; ++j) all = max(all, top[j]);
      all = row_max<L>(all, sm);
    }
    float *scales = a.scales + row * (a.d / a.group);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int at = (lane + j * L) * 8;
      uint32_t m = all;
      if (a.group != a.d) {
        m = dpp_max<0x141>(dpp_max<0x4e>(dpp_max<0xb1>(top[j])));  // 8 lanes
        if (a.group == 128) m = dpp_max<0x140>(m);                 // 16 lanes
      }
      if (at >= a.d) continue;
      const float scale = group_scale(m, largest);
      if ((at & mask) == 0) scales[at >> shift] = scale;
      const uint2 q = to_8bit(s[j], scale, a.out == kOutE4m3);
      if constexpr (VEC) {
        *(uint2 *)(y + at) = q;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (at + i < a.d) y[at + i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
      }
    }
  }
}

template <int L, int C, bool X32, int RK>
static hipError_t launch_norm(const NormArgs &a, hipStream_t s) {
  constexpr int kThreads = L > kNormThreads ? L : kNormThreads, kRows = kThreads / L;
  const long long need = ((long long)a.T + kRows - 1) / kRows;
  const unsigned grid = (unsigned)(need < (1 << 20) ? need : 1 << 20);
  const bool vec = a.d % 8 == 0 && ((a.x_stride | a.r_stride | a.h_stride | a.y_stride) & 7) == 0;
  if (vec)
    rmsnorm_kernel<L, C, X32, RK, true><<<grid, kThreads, 0, s>>>(a);
  else
    rmsnorm_kernel<L, C, X32, RK, false><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <bool X32, int RK>
static hipError_t launch_rows(const NormArgs &a, hipStream_t s) {
  const int chunks = (a.d + 7) / 8;
  // 256 threads a row rather than a wavefront with four times the steps: 8192 x 2048 in
  // fp32 with an fp32 residual, 42 us and 52
  if (chunks <= 64) return launch_norm<64, 1, X32, RK>(a, s);
  if (chunks <= 256) return launch_norm<256, 1, X32, RK>(a, s);
  if (chunks <= 512) return launch_norm<256, 2, X32, RK>(a, s);
  if (chunks <= 768) return launch_norm<256, 3, X32, RK>(a, s);
  if (chunks <= 1024) return launch_norm<256, 4, X32, RK>(a, s);
  return launch_norm<1024, 4, X32, RK>(a, s);
}

hipError_t launch_rmsnorm(const NormArgs &a, int x_dtype, int r_dtype, hipStream_t s) {
  if (a.r == nullptr) return x_dtype ? launch_rows<true, 0>(a, s) : launch_rows<false, 0>(a, s);
  if (r_dtype) return x_dtype ? launch_rows<true, 2>(a, s) : launch_rows<false, 2>(a, s);
  return x_dtype ? launch_rows<true, 1>(a, s) : launch_rows<false, 1>(a, s);
}

}  // namespace moe
