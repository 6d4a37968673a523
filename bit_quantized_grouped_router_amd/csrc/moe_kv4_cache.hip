// Writing keys and values into the paged int4-g64 cache, and reading them back.
//
//   write   per group of 64 channels x:  b = bf16(min x),
//           s = bf16(fp32((max x - b) * fp32(1/15))), 0 below 2^-126,
//           q = clamp(rne((x - b) / s), 0, 15)
//   read    x' = s * q + b, rounded once to fp32 and, for bf16, once more
//
// x - b is rounded to fp32 (for bf16 inputs it is exact unless the two differ
// by a factor above 2^16); the quotient is rounded exactly, by the sign of
// x - b - (q + 1/2) s taken in one FMA, so a code never depends on how a
// divide or reciprocal rounds. A group that holds a NaN or an infinity, or
// that spans more than fp32 can hold, is written as s = b = NaN: it reads back
// as NaN rather than as a wrong finite value.
//
// Both kernels are bound by memory. One wavefront takes a token: its Hkv key
// rows and Hkv value rows, 512 channels at a time, 8 to a lane, so that a
// wavefront reads 1 KB (bf16) or 2 KB (fp32) and writes 256 bytes of codes
// per step; 8 lanes share a group and reduce its minimum and maximum with
// three DPP steps. Measured: 72,400 tokens of 4 x 128 channels read to bf16 (190
// MB) in 39 us, 4.9 TB/s; 7480 tokens of 8 x 128 channels written from fp32 (70 MB)
// in 19 us and read back in 16; 8 tokens in 4.2 and 3.1, three dependent loads.
#include "moe_device.h"
#include "moe_kv4.h"

namespace moe {

constexpr int kCacheWaves = 4;  // wavefronts (tokens in flight) per workgroup
constexpr int kGridRow = 1 << 20;

// Token row of a wavefront; may be past the last (by kGridRow workgroups at the most,
// so below 2^32).
__device__ __forceinline__ uint32_t token_row(int wave) {
  return (blockIdx.y * kGridRow + blockIdx.x) * kCacheWaves + wave;
}

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

template <bool F32>
__global__ __launch_bounds__(kCacheWaves *kWave) void kv4_append_kernel(
    Kv4Dims dm, Kv4Plane kc, Kv4Plane vc, Kv4Batch bt, const void *__restrict__ k,
    const void *__restrict__ v, long long k_stride, long long v_stride) {
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t t = token_row(wave);
  if (t >= (uint32_t)bt.T) return;
  const int tok = (int)t;
  int page, slot;
  if (!find_slot(dm, bt, tok, &page, &slot) || page < 0) return;
  const int width = dm.Hkv * dm.D, total = 2 * width;
  for (int e = lane * 8; e < total; e += kWave * 8) {
    const bool is_v = e >= width;
    const int c = is_v ? e - width : e;
    float x[8];
    load8<F32>(is_v ? v : k, (long long)tok * (is_v ? v_stride : k_stride) + c, x);
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
    uint16_t bb = to_bf16(lo);
    const float b = bf16_to_f32(bb);
    const float span = hi - b;
    uint16_t sb = to_bf16(span * (1.0f / 15.0f));
    float s = bf16_to_f32(sb);
    uint32_t word = 0;
    const bool nan = ((bads >> (lane & 56)) & 0xFF) != 0 || !(fabsf(b) <= 3.402823466e38f) ||
                     !(fabsf(span) <= 3.402823466e38f);
    if (nan) {
      sb = bb = 0x7FC0;
    } else if (s < 1.17549435e-38f) {
      sb = 0;
    } else {
      const float rs = __builtin_amdgcn_rcpf(s);
#pragma unroll
      for (int i = 0; i < 8; ++i) word |= code_of(x[i] - b, s, rs) << (4 * i);
    }
    const int head = c / dm.D, col = c - head * dm.D;
    const long long row = kv4_row(dm, page, head, slot);
    const Kv4Plane &pl = is_v ? vc : kc;
    *(uint32_t *)(pl.codes + row * (dm.D / 2) + col / 2) = word;
    if ((lane & 7) == 0) {
      const long long g = row * (dm.D / kGroup) + col / kGroup;
      pl.scales[g] = sb;
      pl.biases[g] = bb;
    }
  }
}

// 16 bytes past the caches: a read of whole sequences does not fit them, and
// kept there its lines push out the codes that follow (190 MB with another
// batch's reads between: 59 -> 40 us). Not for fp32, whose stores fill a line
// only in pairs (140 MB: 38 -> 41 us).
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void store16(void *p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  __builtin_nontemporal_store(u32x4_t{a, b, c, d}, (u32x4_t *)p);
}

template <bool F32>
__global__ __launch_bounds__(kCacheWaves *kWave) void kv4_read_kernel(
    Kv4Dims dm, Kv4Plane kc, Kv4Plane vc, Kv4Batch bt, void *__restrict__ k, void *__restrict__ v,
    long long k_stride, long long v_stride) {
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t t = token_row(wave);
  if (t >= (uint32_t)bt.T) return;
  const int tok = (int)t;
  int page, slot;
  if (!find_slot(dm, bt, tok, &page, &slot)) return;
  const int width = dm.Hkv * dm.D, total = 2 * width;
  for (int e = lane * 8; e < total; e += kWave * 8) {
    const bool is_v = e >= width;
    const int c = is_v ? e - width : e;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (page >= 0) {
      const int head = c / dm.D, col = c - head * dm.D;
      const long long row = kv4_row(dm, page, head, slot);
      const Kv4Plane &pl = is_v ? vc : kc;
      const uint32_t word = *(const uint32_t *)(pl.codes + row * (dm.D / 2) + col / 2);
      const long long g = row * (dm.D / kGroup) + col / kGroup;
      const float s = bf16_to_f32(pl.scales[g]), b = bf16_to_f32(pl.biases[g]);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf(s, (float)((word >> (4 * i)) & 15u), b);
    }
    const long long at = (long long)tok * (is_v ? v_stride : k_stride) + c;
    void *out = is_v ? v : k;
    if (F32) {
      *(float4 *)((float *)out + at) = make_float4(x[0], x[1], x[2], x[3]);
      *(float4 *)((float *)out + at + 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      store16((uint16_t *)out + at, pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
              pack_bf16x2(x[6], x[7]));
    }
  }
}

// Workgroups of a call, in rows of kGridRow (a launch dimension holds fewer than
// 2^32 threads, and T may be any int32).
static dim3 token_grid(int T) {
  const long long n = ((long long)T + kCacheWaves - 1) / kCacheWaves;
  return n <= kGridRow ? dim3((unsigned)n) : dim3(kGridRow, (unsigned)((n + kGridRow - 1) / kGridRow));
}

hipError_t launch_kv4_append(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc,
                             const Kv4Batch &bt, const void *k, const void *v, long long k_stride,
                             long long v_stride, int dtype, hipStream_t s) {
  auto *kernel = dtype ? kv4_append_kernel<true> : kv4_append_kernel<false>;
  kernel<<<token_grid(bt.T), kCacheWaves * kWave, 0, s>>>(dm, kc, vc, bt, k, v, k_stride, v_stride);
  return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc,
                           const Kv4Batch &bt, void *k, void *v, long long k_stride,
                           long long v_stride, int dtype, hipStream_t s) {
  auto *kernel = dtype ? kv4_read_kernel<true> : kv4_read_kernel<false>;
  kernel<<<token_grid(bt.T), kCacheWaves * kWave, 0, s>>>(dm, kc, vc, bt, k, v, k_stride, v_stride);
  return hipGetLastError();
}

}  // namespace moe
