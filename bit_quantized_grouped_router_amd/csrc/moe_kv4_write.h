// Device code shared by the kernels that write the 4-bit cache: where a token
// lies in it, and how 64 channels are quantised (see moe_kv4_cache.hip for the
// formulas).
#pragma once

#include "moe_device.h"
#include "moe_kv4.h"

namespace moe {

// A wavefront's own LDS accesses are done, and none is moved across.
__device__ __forceinline__ void wave_lds_sync() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Minimum and maximum over aligned groups of 8 lanes.
template <int CTRL>
__device__ __forceinline__ float dpp_get(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL,
                                                               0xf, 0xf, false));
}
__device__ __forceinline__ float min8(float v) {
  v = fminf(v, dpp_get<0xb1>(v));      // pairs
  v = fminf(v, dpp_get<0x4e>(v));      // quads
  return fminf(v, dpp_get<0x141>(v));  // half rows
}
__device__ __forceinline__ float max8(float v) {
  v = fmaxf(v, dpp_get<0xb1>(v));
  v = fmaxf(v, dpp_get<0x4e>(v));
  return fmaxf(v, dpp_get<0x141>(v));
}

// The code of t = x - b for scale s > 0 (rs about 1/s): t/s rounded to the
// nearest integer, ties to even, then clamped. f is floor(t/s) or one off when
// t/s is within a few ulp of an integer, where both choices lead to that
// integer; d has the sign of t/s - (f + 1/2) because an FMA rounds once.
__device__ __forceinline__ uint32_t code_of(float t, float s, float rs) {
  float f = floorf(t * rs);
  f = fminf(fmaxf(f, -1.0f), 15.0f);
  const float d = fmaf(-(f + 0.5f), s, t);
  const int q = (int)f;
  const int up = (d > 0.0f) || (d == 0.0f && (q & 1));
  return (uint32_t)min(max(q + up, 0), 15);
}

// The sequence of token row tok, and its position: wave-uniform, every lane
// active. cu is searched 64 entries at a time, so B <= 64 costs one round of
// loads. Returns false for rows past the last sequence.
__device__ __forceinline__ bool find_token(const Kv4Dims &dm, const Kv4Batch &bt, int tok, int *seq,
                                           long long *pos) {
  const int lane = threadIdx.x & (kWave - 1);
  int lo = 0, n = dm.B;
  while (n > kWave) {
    const int step = (n + kWave - 1) / kWave;
    const int last = lo + min((lane + 1) * step, n) - 1;  // last sequence of this lane's share
    const uint64_t m = __builtin_amdgcn_ballot_w64(bt.cu[last + 1] > tok);
    if (m == 0) return false;
    const int skip = __builtin_ctzll(m) * step;
    lo += skip;
    n = min(step, n - skip);
  }
  const int b = lo + min(lane, n - 1);
  const int c0 = bt.cu[b], c1 = bt.cu[b + 1], ln = bt.len[b];
  const uint64_t m = __builtin_amdgcn_ballot_w64(lane < n && c1 > tok);
  if (m == 0) return false;
  const int w = __builtin_ctzll(m);
  const Kv4Span sp = kv4_span(__builtin_amdgcn_readlane(c0, w), __builtin_amdgcn_readlane(c1, w),
                              __builtin_amdgcn_readlane(ln, w), bt.T);
  if (tok < sp.begin || tok >= sp.begin + sp.n) return false;
  *seq = lo + w;
  *pos = sp.first + (tok - sp.begin);
  return true;
}

// Page and slot of a token row. page < 0: it has no place in the cache.
// Returns false for rows past the last sequence.
__device__ __forceinline__ bool find_slot(const Kv4Dims &dm, const Kv4Batch &bt, int tok, int *page,
                                          int *slot) {
  int seq;
  long long pos;
  if (!find_token(dm, bt, tok, &seq, &pos)) return false;
  *page = -1;
  *slot = 0;
  if (pos >= 0 && pos < kv4_capacity(dm)) {
    const int p = bt.table[(long long)seq * dm.max_pages + (int)(pos >> dm.page_shift)];
    if (kv4_page_ok(dm, p)) *page = p;
    *slot = (int)(pos & (dm.page - 1));
  }
  return true;
}

template <bool F32>
__device__ __forceinline__ void load8(const void *p, long long at, float (&x)[8]) {
  if (F32) {
    const float4 a = *(const float4 *)((const float *)p + at);
    const float4 b = *(const float4 *)((const float *)p + at + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 a = *(const uint4 *)((const uint16_t *)p + at);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
}

// What 8 lanes with 8 channels each hold of their group of 64.
struct Quant8 {
  uint32_t word;  // this lane's codes
  uint16_t scale, bias;
};

__device__ __forceinline__ Quant8 quantise8(const float (&x)[8], int lane) {
  float lo = x[0], hi = x[0];
  bool bad = !(fabsf(x[0]) <= 3.402823466e38f);
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    bad |= !(fabsf(x[i]) <= 3.402823466e38f);
  }
  lo = min8(lo) + 0.0f;  // -0 becomes +0: the minimum of zeros of both signs is one value
  hi = max8(hi);
  const uint64_t bads = __builtin_amdgcn_ballot_w64(bad);
  Quant8 r;
  r.bias = to_bf16(lo);
  const float b = bf16_to_f32(r.bias);
  const float span = hi - b;
  r.scale = to_bf16(span * (1.0f / 15.0f));
  const float s = bf16_to_f32(r.scale);
  r.word = 0;
  const bool nan = ((bads >> (lane & 56)) & 0xFF) != 0 || !(fabsf(b) <= 3.402823466e38f) ||
                   !(fabsf(span) <= 3.402823466e38f);
  if (nan) {
    r.scale = r.bias = 0x7FC0;
  } else if (s < 1.17549435e-38f) {
    r.scale = 0;
  } else {
    const float rs = __builtin_amdgcn_rcpf(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) r.word |= code_of(x[i] - b, s, rs) << (4 * i);
  }
  return r;
}

// Channels col .. col + 7 of a cache row.
__device__ __forceinline__ void store8(const Kv4Plane &pl, long long row, int D, int col, const Quant8 &q, int lane) {
  *(uint32_t *)(pl.codes + row * (D / 2) + col / 2) = q.word;
  if ((lane & 7) == 0) {
    const long long g = row * (D / kGroup) + col / kGroup;
    pl.scales[g] = q.scale;
    pl.biases[g] = q.bias;
  }
}

}  // namespace moe
