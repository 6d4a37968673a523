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
#include "moe_kv4_write.h"

namespace moe {

constexpr int kCacheWaves = 4;  // wavefronts (tokens in flight) per workgroup
constexpr int kGridRow = 1 << 20;

// Token row of a wavefront; may be past the last (by kGridRow workgroups at the most,
// so below 2^32).
__device__ __forceinline__ uint32_t token_row(int wave) {
  return (blockIdx.y * kGridRow + blockIdx.x) * kCacheWaves + wave;
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
    const Quant8 q = quantise8(x, lane);
    const int head = c / dm.D, col = c - head * dm.D;
    const long long row = kv4_row(dm, page, head, slot);
    store8(is_v ? vc : kc, row, dm.D, col, q, lane);
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
