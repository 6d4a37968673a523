// Rotary positions of heads, and the same fused with the write of the 4-bit cache.
//
//   (a', b') = magnitude * (a cos t - b sin t, a sin t + b cos t),  t = position * freq
// for each pair of the first rot channels of a head: (2i, 2i + 1) interleaved,
// (i, i + rot / 2) otherwise; the other channels pass. A norm of the head, x /
// sqrt(mean x^2 + eps) * w, may come before. fp32 throughout, rounded once at
// the end; only angle, sine and cosine are taken in 64 bits (in fp32 the angle of
// position 131,072 would be off by 2^-8 radians), as a number of turns whose
// whole part is dropped, and rounded to fp32. The two products are rounded one by
// one and not fused, so that a and b are treated alike and a key next to a border of
// the quantisation falls on the side that the formula in fp32 says.
//
// Bound by memory for many tokens, by launch and latency for few. P lanes take
// a head, 8 channels each, and a wavefront 64 / P heads at a time. The sines of a token are
// worked out once by its wavefront, one pair a lane, and handed over through
// LDS; each lane keeps those of its 8 channels for all of the token's heads. A
// wavefront has one step's loads in flight and few registers, so that more of them
// share a SIMD: with four steps' at a time 8192 tokens of 16 x 128 in bf16 take 15.6
// us instead of 13.9 (13.8 to 14.2 from run to run, 4.7 TB/s). Prompts of 7480 tokens, 32 + 2 x 8 heads of 128 from
// fp32, rotated and written in 61 us (4.1 TB/s); 8 tokens of 16 + 2 x 2 heads of 256 in
// 5.1. Heads between the powers of two leave lanes idle: 8192 x 16 heads of 72, 80 or 96
// channels take 12.6 us, those of 64 9.5; of 136 or 192 19.2 and 20.6, those of 128 13.8.
#include "moe_rope.h"

#include "moe_kv4_write.h"

namespace moe {

constexpr int kRopeWaves = 4;

// LDS of a wavefront: (cos, sin) of the token's pairs, and the 8 channels of
// each lane while partners are fetched.
struct RopeLds {
  float2 turn[kRopeMaxD / 2];
  float stage[kWave * 8];
};

// Sum over the P lanes of a head.
template <int P>
__device__ __forceinline__ float head_sum(float v) {
  if constexpr (P <= 16) return group_sum_dpp<P>(v);
  v = group_sum_dpp<16>(v);
#pragma unroll
  for (int off = 16; off < P; off *= 2) v += __shfl_xor(v, off, kWave);
  return v;
}

// Sine and cosine of p f: the nearest quarter turn is taken off and the rest, at most pi /
// 4, goes into the Taylor series, whose next terms are below 2^-45. The product of a 32-bit
// position and fp32's 24 bits can have 55, so what fp64 rounds off it (2^-23 at position
// 2^31) goes along. Turns are it times 1 / (2 pi) in two parts, so that no more is lost
// for large angles than for small ones.
__device__ __forceinline__ void sincos64(double p, double f, double &sn, double &cs) {
  constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnRest = -0x1.6b01ec5417056p-57;
  const double a = p * f, off = fma(p, f, -a);
  const double t = a * kTurn, rest = fma(off, kTurn, fma(a, kTurnRest, fma(a, kTurn, -t)));
  const double quarter = rint(4.0 * t);
  const double x = (fma(-0.25, quarter, t) + rest) * 6.28318530717958647693, y = x * x;
  double s = 1.0 / 6227020800.0, c = -1.0 / 87178291200.0;
  s = fma(s, y, -1.0 / 39916800.0), c = fma(c, y, 1.0 / 479001600.0);
  s = fma(s, y, 1.0 / 362880.0), c = fma(c, y, -1.0 / 3628800.0);
  s = fma(s, y, -1.0 / 5040.0), c = fma(c, y, 1.0 / 40320.0);
  s = fma(s, y, 1.0 / 120.0), c = fma(c, y, -1.0 / 720.0);
  s = fma(s, y, -1.0 / 6.0), c = fma(c, y, 1.0 / 24.0);
  c = fma(c, y, -0.5);
  s = fma(s * y, x, x), c = fma(c, y, 1.0);
  const int q = (int)(quarter - 4.0 * floor(0.25 * quarter));  // the quarters left after whole turns
  sn = q & 1 ? c : s;
  cs = q & 1 ? s : c;
  sn = q & 2 ? -sn : sn;
  cs = (q + 1) & 2 ? -cs : cs;
}

// What a lane's 8 channels are turned by. c, s: cosine and signed sine.
struct LaneTurn {
  float c[8], s[8];
};

__device__ __forceinline__ void lane_turn(const Rope &rope, int position, int at, RopeLds &lds, LaneTurn &t) {
  const int lane = threadIdx.x & (kWave - 1), half = rope.rot / 2;
  for (int i = lane; i < half; i += kWave) {
    double sn, cs;
    sincos64(position, rope.freqs[i], sn, cs);
    lds.turn[i] = make_float2((float)(cs * rope.magnitude), (float)(sn * rope.magnitude));
  }
  wave_lds_sync();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ch = at + i;
    const bool second = rope.interleaved ? (ch & 1) : ch >= half;
    const int pair = rope.interleaved ? ch / 2 : second ? ch - half : ch;
    const float2 u = lds.turn[ch < rope.rot ? pair : 0];
    t.c[i] = u.x;
    t.s[i] = second ? u.y : -u.y;
  }
}

// a c + b s, the products rounded (hipcc fuses them, __fmul_rn's too, unless told not to).
__device__ __forceinline__ float products_sum(float a, float c, float b, float s) {
#pragma clang fp contract(off)
  const float p = a * c, q = b * s;
  return p + q;
}

// Turns 8 channels of a head whose channel 0 is lane `first`'s.
__device__ __forceinline__ void rotate8(const Rope &rope, const LaneTurn &t, int at, int first, float *stage,
                                        float (&x)[8]) {
  float y[8];
  if (rope.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
  } else {
    const int lane = threadIdx.x & (kWave - 1), half = rope.rot / 2;
    *(float4 *)(stage + lane * 8) = make_float4(x[0], x[1], x[2], x[3]);
    *(float4 *)(stage + lane * 8 + 4) = make_float4(x[4], x[5], x[6], x[7]);
    wave_lds_sync();
    const float *head = stage + first * 8;
    if (half % 4 == 0) {  // four channels have their partners side by side
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const int ch = at + i, to = ch < half ? ch + half : ch < rope.rot ? ch - half : ch;
        const float4 v = *(const float4 *)(head + to);
        y[i] = v.x, y[i + 1] = v.y, y[i + 2] = v.z, y[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int ch = at + i;
        y[i] = head[ch < half ? ch + half : ch < rope.rot ? ch - half : ch];
      }
    }
    wave_lds_sync();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = products_sum(x[i], t.c[i], y[i], t.s[i]);
    x[i] = at + i < rope.rot ? v : x[i];
  }
}

struct LaneNorm {
  uint4 w;  // this lane's weights, as they are in memory
};

__device__ __forceinline__ void lane_norm(const HeadNorm &n, int at, int D, LaneNorm &l) {
  if (n.weight == nullptr) return;
  l.w = *(const uint4 *)(n.weight + (at < D ? at : 0));
}

// Norm and rotation of a head's 8 channels (lanes without a head or channels hold zeros).
template <int P>
__device__ __forceinline__ void turn_head(const Rope &rope, const HeadNorm &norm, const LaneTurn &t, const LaneNorm &l,
                                          int at, int D, float *stage, float (&x)[8]) {
  if (norm.weight != nullptr) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
    const float inv = 1.0f / sqrtf(head_sum<P>(sum) / (float)D + norm.eps);
    const uint32_t u[4] = {l.w.x, l.w.y, l.w.z, l.w.w};
    const float one = norm.plus_one ? 1.f : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = x[i] * inv * (((i & 1) ? __uint_as_float(u[i / 2] & 0xFFFF0000u) : __uint_as_float(u[i / 2] << 16)) + one);
  }
  const int lane = threadIdx.x & (kWave - 1);
  rotate8(rope, t, at, lane - lane % P, stage, x);
}

template <bool F32>
__device__ __forceinline__ void put8(void *p, long long at, const float (&x)[8]) {
  if (F32) {
    *(float4 *)((float *)p + at) = make_float4(x[0], x[1], x[2], x[3]);
    *(float4 *)((float *)p + at + 4) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *(uint4 *)((uint16_t *)p + at) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
}

// A token's heads are shared by `parts` wavefronts, each taking every parts-th
// step of 64 / P heads.
template <int P, bool X32, bool O32>
__global__ __launch_bounds__(kRopeWaves *kWave) void rope_kernel(int T, int H, int D, const void *x, long long x_stride,
                                                                 const int32_t *positions, Rope rope, HeadNorm norm,
                                                                 void *out, long long out_stride, int parts) {
  __shared__ __attribute__((aligned(16))) RopeLds lds[kRopeWaves];
  constexpr int kHeads = kWave / P;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int at = (lane % P) * 8, steps = (H + kHeads - 1) / kHeads;
  const long long all = (long long)T * parts, stride = (long long)gridDim.x * kRopeWaves;
  for (long long unit = (long long)blockIdx.x * kRopeWaves + wave; unit < all; unit += stride) {
    const long long tok = unit / parts;
    const int part = (int)(unit - tok * parts);
    float v[8];
    const auto load = [&](int st) {
      const int head = st * kHeads + lane / P;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
      if (head < H && at < D) load8<X32>(x, tok * x_stride + (long long)head * D + at, v);
    };
    load(part);
    LaneTurn turn;
    LaneNorm ln;
    lane_turn(rope, positions[tok], at, lds[wave], turn);
    lane_norm(norm, at, D, ln);
    for (int st = part; st < steps; st += parts) {
      if (st != part) load(st);
      turn_head<P>(rope, norm, turn, ln, at, D, lds[wave].stage, v);
      const int head = st * kHeads + lane / P;
      if (head < H && at < D) put8<O32>(out, tok * out_stride + (long long)head * D + at, v);
    }
    wave_lds_sync();
  }
}

// The same for a token's queries, and its keys and values into the cache: steps
// are those of the query heads, then of the key heads, then of the value heads.
template <int P, bool X32>
__global__ __launch_bounds__(kRopeWaves *kWave) void kv4_rope_append_kernel(Kv4Dims dm, Kv4Plane kc, Kv4Plane vc,
                                                                            Kv4Batch bt, Rope rope, RopeAppend a,
                                                                            int parts) {
  __shared__ __attribute__((aligned(16))) RopeLds lds[kRopeWaves];
  constexpr int kHeads = kWave / P, D = P * 8;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int at = (lane % P) * 8;
  const int nq = (dm.Hq + kHeads - 1) / kHeads, nk = (dm.Hkv + kHeads - 1) / kHeads, steps = nq + 2 * nk;
  const long long all = (long long)bt.T * parts, stride = (long long)gridDim.x * kRopeWaves;
  for (long long unit = (long long)blockIdx.x * kRopeWaves + wave; unit < all; unit += stride) {
    const int tok = (int)(unit / parts);
    const int part = (int)(unit - (long long)tok * parts);
    float v[8];
    const auto load = [&](int st) {
      const int kind = st < nq ? 0 : st < nq + nk ? 1 : 2;
      const int head = (st - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * kHeads + lane / P;
      const void *src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
      const long long row = tok * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
      if (head < (kind == 0 ? dm.Hq : dm.Hkv)) load8<X32>(src, row + (long long)head * D + at, v);
    };
    int seq, page = -1, slot = 0;
    long long pos;
    LaneTurn turn;
    LaneNorm qn, kn;
    for (int st = part; st < steps; st += parts) {
      load(st);
      if (st == part) {  // behind the first loads
        if (!find_token(dm, bt, tok, &seq, &pos)) break;
        if (pos >= 0 && pos < kv4_capacity(dm)) {
          const int p = bt.table[(long long)seq * dm.max_pages + (int)(pos >> dm.page_shift)];
          if (kv4_page_ok(dm, p)) page = p;
          slot = (int)(pos & (dm.page - 1));
        }
        lane_turn(rope, (int)pos, at, lds[wave], turn);
        lane_norm(a.q_norm, at, D, qn);
        lane_norm(a.k_norm, at, D, kn);
      }
      if (st < nq) {
        const int head = st * kHeads + lane / P;
        turn_head<P>(rope, a.q_norm, turn, qn, at, D, lds[wave].stage, v);
        if (head < dm.Hq) put8<false>(a.out, tok * a.out_stride + (long long)head * D + at, v);
      } else {
        const bool is_k = st < nq + nk;
        const int head = (st - (is_k ? nq : nq + nk)) * kHeads + lane / P;
        if (is_k) turn_head<P>(rope, a.k_norm, turn, kn, at, D, lds[wave].stage, v);
        const Quant8 q = quantise8(v, lane);
        if (page >= 0 && head < dm.Hkv) store8(is_k ? kc : vc, kv4_row(dm, page, head, slot), D, at, q, lane);
      }
    }
    wave_lds_sync();
  }
}

// Wavefronts a token's steps are shared by: with few tokens as many as there are
// steps, since one after the other is latency; with many one, which works the
// sines out once.
static int rope_parts(long long T, int steps) {
  const long long want = 4096 / (T > 0 ? T : 1);
  const int most = steps < 65536 ? steps : 65536;
  return want < 1 ? 1 : want < most ? (int)want : most;
}

static unsigned rope_grid(long long waves) {
  const long long n = (waves + kRopeWaves - 1) / kRopeWaves;
  return (unsigned)(n < (1 << 20) ? n : 1 << 20);
}

template <int P>
static hipError_t launch_p(int T, int H, int D, const void *x, long long x_stride, int x_dtype,
                           const int32_t *positions, const Rope &rope, const HeadNorm &norm, void *out,
                           long long out_stride, int out_dtype, hipStream_t s) {
  const int parts = rope_parts(T, (H + kWave / P - 1) / (kWave / P));
  auto *kernel = x_dtype ? (out_dtype ? rope_kernel<P, true, true> : rope_kernel<P, true, false>)
                         : (out_dtype ? rope_kernel<P, false, true> : rope_kernel<P, false, false>);
  kernel<<<rope_grid((long long)T * parts), kRopeWaves * kWave, 0, s>>>(T, H, D, x, x_stride, positions, rope, norm,
                                                                        out, out_stride, parts);
  return hipGetLastError();
}

hipError_t launch_rope(int T, int H, int D, const void *x, long long x_stride, int x_dtype, const int32_t *positions,
                       const Rope &rope, const HeadNorm &norm, void *out, long long out_stride, int out_dtype,
                       hipStream_t s) {
  auto *launch = D <= 64 ? launch_p<8> : D <= 128 ? launch_p<16> : D <= 256 ? launch_p<32> : launch_p<64>;
  return launch(T, H, D, x, x_stride, x_dtype, positions, rope, norm, out, out_stride, out_dtype, s);
}

template <int P>
static hipError_t launch_append(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc, const Kv4Batch &bt,
                                const Rope &rope, const RopeAppend &a, int dtype, hipStream_t s) {
  constexpr int kHeads = kWave / P;
  const int parts = rope_parts(bt.T, (dm.Hq + kHeads - 1) / kHeads + 2 * ((dm.Hkv + kHeads - 1) / kHeads));
  auto *kernel = dtype ? kv4_rope_append_kernel<P, true> : kv4_rope_append_kernel<P, false>;
  kernel<<<rope_grid((long long)bt.T * parts), kRopeWaves * kWave, 0, s>>>(dm, kc, vc, bt, rope, a, parts);
  return hipGetLastError();
}

hipError_t launch_kv4_rope_append(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc, const Kv4Batch &bt,
                                  const Rope &rope, const RopeAppend &a, int dtype, hipStream_t s) {
  if (dm.D == 64) return launch_append<8>(dm, kc, vc, bt, rope, a, dtype, s);
  if (dm.D == 128) return launch_append<16>(dm, kc, vc, bt, rope, a, dtype, s);
  return launch_append<32>(dm, kc, vc, bt, rope, a, dtype, s);
}

}  // namespace moe
