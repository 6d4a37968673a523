// Dense projection with int4-g64 weights:
//   y[t][n] = act(sum_c x[t][c] W[n][c] + bias[n]) + residual[t][n],
//   W = bf16(fp32(s q + b)), products of bf16 values exact, sums in fp32.
//
// Small batches are bound by the latency of one or two rounds of loads, and from 17
// tokens on by activations too, which every 16 weight rows read again (37 by 2048 x
// 4096: 64 MB from the L2 for 5 MB of operands; 52% of the time is waiting). One
// workgroup takes 16 weight rows and 16 NT tokens; its 8 wavefronts take four
// 64-column groups at a time, rebuild the rows' weights in registers as the A operand of 16x16x32 MFMAs
// (lane l: row l % 16, columns 16 (l / 16) .. +15 of the group) against the
// tokens' activations read straight from memory, and join their sums through
// LDS, where the epilogue runs. Measured, rows x columns: 1 token by 5120 x 2048
// 6.0 us in a graph, 37 by 2048 x 4096 12.1 us. (Activations brought in whole
// lines and turned in LDS took 13 and 27 us.) The tile kernels below: 777
// by 1001 x 2048 14 us, 8192 by 5120 x 2048 173 to 180 us (a library product of
// bf16 weights of that size 175 to 178).
#include <type_traits>

#include "moe_lds.h"
#include "moe_linear.h"

namespace moe {

constexpr int kLnWaves = 8;

// GELU by erfc: 1 + erf cancels below zero and leaves nothing from z = -5.6 on
// (8192 x 5120 x 2048 with GELU 209 -> 223 us, small and middle batches the same).
template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == kActRelu) return z > 0.f ? z : (z == z ? 0.f : z);
  if constexpr (ACT == kActSilu) return z / (1.0f + expf(-z));
  if constexpr (ACT == kActGelu) return 0.5f * z * erfcf(z * -0.70710678118654752f);
  return z;
}

// Calls f with the activation as a compile-time constant.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    default: f(std::integral_constant<int, kActNone>{}); break;
  }
}

template <bool F32>
__device__ __forceinline__ float load_residual(const LinearArgs &a, int t, int n) {
  if (!a.residual) return 0.f;
  if (F32) return ((const float *)a.residual)[t * a.r_stride + n];
  return bf16_to_f32(((const uint16_t *)a.residual)[t * a.r_stride + n]);
}

// y = act(z + bias) + residual, rounded once.
template <int ACT, bool F32>
__device__ __forceinline__ void store_output(const LinearArgs &a, int t, int n, float z, float bias,
                                             float residual) {
  z = activate<ACT>(z + bias) + residual;
  if (F32)
    ((float *)a.y)[t * a.y_stride + n] = z;
  else
    ((uint16_t *)a.y)[t * a.y_stride + n] = to_bf16(z);
}

// The same for outputs n .. n + 7, with wide accesses. STREAM: past the caches,
// which the outputs of a large batch do not fit (8192 x 5120 x 2048, other
// batches between: 188 -> 181 us); smaller ones are left for whoever reads them.
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
template <int ACT, bool F32, bool STREAM>
__device__ __forceinline__ void store_outputs8(const LinearArgs &a, int t, int n, const float (&z)[8],
                                               const float (&bias)[8]) {
  float r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, y[8];
  if (a.residual) {
    if (F32) {
      const float4 *p = (const float4 *)((const float *)a.residual + t * a.r_stride + n);
      const float4 u = p[0], v = p[1];
      r[0] = u.x, r[1] = u.y, r[2] = u.z, r[3] = u.w, r[4] = v.x, r[5] = v.y, r[6] = v.z, r[7] = v.w;
    } else {
      const uint4 u = *(const uint4 *)((const uint16_t *)a.residual + t * a.r_stride + n);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
        r[2 * i + 1] = bf16_to_f32(w[i] >> 16);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = activate<ACT>(z[i] + bias[i]) + r[i];
  if (F32) {
    float4 *p = (float4 *)((float *)a.y + t * a.y_stride + n);
    p[0] = make_float4(y[0], y[1], y[2], y[3]);
    p[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    const u32x4_t v = {pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7])};
    u32x4_t *p = (u32x4_t *)((uint16_t *)a.y + t * a.y_stride + n);
    if (STREAM)
      __builtin_nontemporal_store(v, p);
    else
      *p = v;
  }
}

template <int NT, bool F32>
__global__ __launch_bounds__(kLnWaves *kWave, 2) void linear_kernel(LinearArgs a) {
  constexpr int kTokens = 16 * NT;
  constexpr int kBatch = 4;  // groups whose loads are in flight together
  __shared__ float part[kLnWaves][kTokens][16 + 1];
  const int blocks = (a.rows + 15) / 16;
  const int n0 = (blockIdx.x % blocks) * 16, t0 = (blockIdx.x / blocks) * kTokens;
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
    xp[i] = a.x + min(t0 + i * 16 + (lane & 15), a.T - 1) * a.x_stride + c16;
    acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  // the epilogue's operands: of one output a thread, on their way meanwhile
  static_assert(kTokens * 16 <= kLnWaves * kWave, "one output a thread");
  const int te = t0 + threadIdx.x / 16, ne = n0 + threadIdx.x % 16;
  const bool mine = threadIdx.x < kTokens * 16 && te < a.T && ne < a.rows;
  const float bias = mine && a.bias ? bf16_to_f32(a.bias[ne]) : 0.f;
  const float res = mine ? load_residual<F32>(a, te, ne) : 0.f;
  // a wavefront takes kBatch groups in a row: whole lines of codes, and where rows
  // of scales are 8-byte aligned one load for the four of them (eight 16-bit
  // loads instead cost 1 x 5120 x 2048 3 us of 8.7)
  const bool wide = ng % kBatch == 0;
  for (int g0 = wave * kBatch; g0 < ng; g0 += kLnWaves * kBatch) {
    uint2 c[kBatch];
    uint32_t s[kBatch], b[kBatch];
    uint4 x[kBatch][NT][2];
    if (wide) {
      const uint2 s4 = *(const uint2 *)(sp + g0), b4 = *(const uint2 *)(bp + g0);
      s[0] = s4.x & 0xFFFFu, s[1] = s4.x >> 16, s[2] = s4.y & 0xFFFFu, s[3] = s4.y >> 16;
      b[0] = b4.x & 0xFFFFu, b[1] = b4.x >> 16, b[2] = b4.y & 0xFFFFu, b[3] = b4.y >> 16;
    } else {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int g = min(g0 + j, ng - 1);
        s[j] = sp[g];
        b[j] = bp[g];
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int g = min(g0 + j, ng - 1);
      c[j] = *(const uint2 *)(codes + g * 32);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        x[j][i][0] = *(const uint4 *)(xp[i] + g * kGroup);
        x[j][i][1] = *(const uint4 *)(xp[i] + g * kGroup + 8);
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // all loads first
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (g0 + j >= ng) break;
      const float sc = bf16_to_f32(s[j]), bi = bf16_to_f32(b[j]);
      const bf16x8_t w0 = __builtin_bit_cast(bf16x8_t, dequant8(c[j].x, sc, bi));
      const bf16x8_t w1 = __builtin_bit_cast(bf16x8_t, dequant8(c[j].y, sc, bi));
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0, __builtin_bit_cast(bf16x8_t, x[j][i][0]), acc[i], 0, 0, 0);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w1, __builtin_bit_cast(bf16x8_t, x[j][i][1]), acc[i], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) part[wave][i * 16 + (lane & 15)][(lane >> 4) * 4 + r] = acc[i][r];
  __syncthreads();
  if (!mine) return;
  float z = 0.f;
#pragma unroll
  for (int w = 0; w < kLnWaves; ++w) z += part[w][threadIdx.x / 16][threadIdx.x % 16];
  with_act(a.act, [&](auto act) { store_output<act.value, F32>(a, te, ne, z, bias, res); });
}

// ------------------------------------------------------------------ large batches
//
// WT wavefronts take a tile of 32 MB tokens x 32 NB WT weight rows, each all the
// tokens and its own 32 NB rows, so every weight is rebuilt once per tile, in
// registers, as the B operand of 32x32x16 MFMAs (C: lane = weight row,
// registers = tokens). Per K step of 64 (one group):
//   - activations (4 MB KB) come by LDS DMA into a ring of three stages shared by
//     the team, 16-byte chunks XOR-swizzled by row so that fragment reads of 8
//     or 16 rows hit distinct banks;
//   - codes come by LDS DMA too, into the wavefront's own ring, where each lane
//     reads back the 16 bytes it fetched (32 columns of one row);
//   - scales and biases sit in an LDS table of 8 groups of the wavefront's rows,
//     refilled every 8 steps.
// All loads of the loop are DMA, two steps ahead, and the loop waits for them
// by count: a load into registers there would make the compiler wait for every
// DMA behind it.
//   large batches   MB = 4, NB = 2: two workgroups share a CU (80 KB of LDS, 256
//                   registers), so one rebuilds weights while the other multiplies;
//   middle ones     MB = 2, NB = 1 and KS = 2 teams of four wavefronts that split
//                   the K steps and add up in LDS: there are few tiles then, and
//                   a step takes its latency, not its work;
//   narrow ones     the same with KS = 4 teams of WT = 2, half as many rows a tile:
//                   twice the workgroups where middle tiles leave CUs empty.
constexpr int kBgStages = 3, kBgChunk = 8;

template <int MB, int NB, int KS, int WT>
struct Bg {
  static constexpr int kTokens = 32 * MB, kWaveRows = 32 * NB, kRows = WT * kWaveRows;
  static constexpr int kThreads = KS * WT * kWave;
  static constexpr int kX = kTokens * kGroup * 2;      // bytes of activations a stage
  static constexpr int kCodes = kRows * kGroup / 2;    // bytes of codes a stage
  static constexpr int kTable = kBgChunk * kRows * 4;  // (scale | bias << 16) words
  static constexpr int kTeam = kBgStages * (kX + kCodes) + kTable;
  static constexpr int kLds = KS * kTeam;
  static constexpr int kXLoads = 4 * MB / WT, kLoads = kXLoads + NB;  // DMA instructions a wavefront and stage
  static constexpr int kPasses = MB == 4 ? 2 : 1;      // of the epilogue
  static constexpr int kPassTokens = kTokens / kPasses;
  static_assert((KS == 4 ? 1 : 2) * kLds <= 160 * 1024, "two workgroups a CU, one of four teams");
  static_assert(KS * WT * kPassTokens * kWaveRows * 4 <= kLds, "the epilogue fits");
};

#define MOE_LN_WAIT_VMCNT(n) \
  __builtin_amdgcn_s_waitcnt(((n) & 0xF) | (0x7 << 4) | (0xF << 8) | (((n) >> 4) << 14))

typedef __attribute__((address_space(3))) void ln_lds_void;
typedef uint32_t ln_u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t ln_lds_address(const void *p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(ln_lds_void *)p);
}

__device__ __forceinline__ ln_u32x4 ln_rsrc(const void *base, uint32_t bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  ln_u32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane((uint32_t)b);
  r[1] = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32) & 0xFFFFu);
  r[2] = __builtin_amdgcn_readfirstlane(bytes);
  r[3] = 0x00020000;
  return r;
}

// 16 bytes a lane from buffer r at off (per lane) + step (scalar) to LDS dst +
// 16 * lane. No register is written; the no-ops cover m0 (one wait state) and
// scalar operands fresh from the VALU (five).
__device__ __forceinline__ void ln_dma(const ln_u32x4 &r, uint32_t off, uint32_t step, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               ::"s"(dst), "v"(off), "s"(r), "s"(step) : "memory");
}

// Token tile and weight block of workgroup bid: XCD bid % 8 takes a contiguous
// run of the list in which 8 token tiles go through all weight blocks together,
// so that what an XCD works on at a time (about 8 x 8 tiles) shares its L2.
__device__ __forceinline__ bool bg_tile(int bid, int tt, int nn, int &t, int &n) {
  const int total = tt * nn, per = (total + 7) / 8;
  const int i = (bid % 8) * per + bid / 8;
  if (bid / 8 >= per || i >= total) return false;
  const int band = i / (8 * nn), in = i - band * 8 * nn;
  const int height = min(8, tt - 8 * band);
  n = in / height;
  t = 8 * band + in - n * height;
  return true;
}

template <int MB, int NB, int KS, int WT, bool F32>
__global__ __launch_bounds__(KS * WT * kWave, KS == 1 ? 2 : 4) void linear_tiles_kernel(LinearArgs a) {
  using B = Bg<MB, NB, KS, WT>;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  int ti, ni;
  if (!bg_tile(blockIdx.x, (a.T + B::kTokens - 1) / B::kTokens, (a.rows + B::kRows - 1) / B::kRows, ti, ni)) return;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave8 = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wave = wave8 & (WT - 1), team = wave8 / WT;
  const int t0 = ti * B::kTokens, n0 = ni * B::kRows + wave * B::kWaveRows;
  const int ng = a.cols / kGroup;
  const int tokens = min(B::kTokens, a.T - t0);
  // the team's groups: common steps for all teams, and what is left for the first
  const int common = ng / KS, left = ng - common * KS;
  const int first = team == 0 ? 0 : team * common + left;
  const int steps = common + (team == 0 ? left : 0);
  uint8_t *const lds = smem + team * B::kTeam;

  // activations: DMA instruction i of wavefront w fills rows 8 (WT i + w) .. +7,
  // lane l row l / 8 of those, LDS chunk l % 8, which holds the row's chunk
  // (l % 8) ^ (row % 8) ^ (row / 8 % 2). Rows past the last re-read it.
  const ln_u32x4 xr = ln_rsrc(a.x + t0 * a.x_stride, (uint32_t)(((tokens - 1) * a.x_stride + a.cols) * 2));
  uint32_t x_off[B::kXLoads];
#pragma unroll
  for (int i = 0; i < B::kXLoads; ++i) {
    const int r = min(8 * (WT * i + wave) + (lane >> 3), tokens - 1);
    x_off[i] = (uint32_t)(r * (int)a.x_stride + first * kGroup + (((lane & 7) ^ (lane >> 3) ^ (wave & 1)) * 8)) * 2u;
  }
  // codes: instruction b fetches row 32 b + l % 32, columns 32 (l / 32) .. +31
  const int wrow0 = min(n0, a.rows - 1), wrows = max(min(B::kWaveRows, a.rows - n0), 1);
  const ln_u32x4 cr = ln_rsrc(a.w.codes + (long long)wrow0 * (a.cols / 2), (uint32_t)(wrows * (a.cols / 2)));
  uint32_t c_off[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
    c_off[b] = (uint32_t)(min(32 * b + (lane & 31), wrows - 1) * (a.cols / 2) + first * (kGroup / 2) + (lane >> 5) * 16);
  const uint32_t x_lds = ln_lds_address(lds) + wave * 1024;
  uint8_t *cring = lds + kBgStages * B::kX + wave * (NB * 1024);  // this wavefront's part of a stage
  const uint32_t c_lds = ln_lds_address(cring);
  uint32_t *table = (uint32_t *)(lds + kBgStages * (B::kX + B::kCodes)) + wave * B::kWaveRows;
  // third i of a stage's DMA instructions: activations first, then codes
  auto dma_part = [&](int step, int slot, int i) {
#pragma unroll
    for (int j = i * B::kLoads / 3; j < (i + 1) * B::kLoads / 3; ++j) {
      constexpr int X = B::kXLoads;
      if (j < X)
        ln_dma(xr, x_off[j < X ? j : 0], step * (kGroup * 2), x_lds + slot * B::kX + j * (WT * 1024));
      else
        ln_dma(cr, c_off[j < X ? 0 : j - X], step * (kGroup / 2), c_lds + slot * B::kCodes + (j - X) * 1024);
    }
  };
  auto dma = [&](int step, int slot) {
#pragma unroll
    for (int i = 0; i < 3; ++i) dma_part(step, slot, i);
  };

  // scales and biases of 8 groups of row `lane` of the wavefront
  const int trow = min(lane & (B::kWaveRows - 1), wrows - 1);
  const long long srow = (long long)(wrow0 + trow) * ng + first;
  const uint16_t *sp = a.w.scales + srow, *bp = a.w.biases + srow;
  const bool vec = ng % 8 == 0 && first % 8 == 0 && steps % 8 == 0;  // 16-byte loads stay aligned and inside
  uint4 sv, bv;
  auto fetch = [&](int g0) {
    if (vec) {
      sv = *(const uint4 *)(sp + g0);
      bv = *(const uint4 *)(bp + g0);
    } else {
      uint32_t s[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int g = min(g0 + 2 * i, steps - 1), h = min(g0 + 2 * i + 1, steps - 1);
        s[i] = sp[g] | (uint32_t)sp[h] << 16;
        b[i] = bp[g] | (uint32_t)bp[h] << 16;
      }
      sv = make_uint4(s[0], s[1], s[2], s[3]);
      bv = make_uint4(b[0], b[1], b[2], b[3]);
    }
  };
  auto fill = [&]() {
    const uint32_t s[4] = {sv.x, sv.y, sv.z, sv.w}, b[4] = {bv.x, bv.y, bv.z, bv.w};
    uint32_t *t = table + (lane & (B::kWaveRows - 1));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t[(2 * i) * B::kRows] = (s[i] & 0xFFFFu) | (b[i] << 16);
      t[(2 * i + 1) * B::kRows] = (s[i] >> 16) | (b[i] & 0xFFFF0000u);
    }
  };
  bool ok = true;  // every group of the wavefront's rows takes the fast dequantisation
  if (steps > 0) {
    dma(0, 0);
    if (steps > 1) dma(1, 1);
#pragma unroll 4
    for (int g0 = (steps - 1) / kBgChunk * kBgChunk; g0 >= 0; g0 -= kBgChunk) {  // the first chunk's stay
      fetch(g0);
      const uint32_t s[4] = {sv.x, sv.y, sv.z, sv.w}, b[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        ok &= (int)dq_fast_ok((s[i] & 0xFFFFu) | (b[i] << 16)) & (int)dq_fast_ok((s[i] >> 16) | (b[i] & 0xFFFF0000u));
    }
    fill();
  }
  const bool fast = __builtin_amdgcn_ballot_w64(!ok) == 0;

  f32x16_t acc[MB][NB];
#pragma unroll
  for (int rb = 0; rb < MB; ++rb)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[rb][b] = f32x16_t{0};
  const DqRegs dk = dq_regs();
  const int lrow = (lane & 31) * 128, lx = (lane & 7) ^ ((lane >> 3) & 1), lh = 4 * (lane >> 5);

  // Wait for stage kt (only the DMA of stage kt + 1 may still be in flight) and
  // for every wavefront to be done with stage kt - 1.
  auto enter = [&](int kt) {
    if (kt + 1 < steps)
      MOE_LN_WAIT_VMCNT(B::kLoads);
    else
      MOE_LN_WAIT_VMCNT(0);
    lds_barrier();
    asm volatile("" ::: "memory");
  };
  // one K step; the weights of a slice of 16 columns are rebuilt, and its
  // activation fragments read, while the slice before it is multiplied
  int slot = 0;
  auto step = [&](auto fast_tag, int kt) {
    constexpr bool FAST = decltype(fast_tag)::value;
    if (kt % kBgChunk == kBgChunk - 1 && kt + 1 < steps) fetch(kt + 1);
    const uint8_t *xs = lds + slot * B::kX + lrow;
    uint32_t word[NB][4];
    DqGroup q[NB];
    float sc[NB], bi[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint4 c = *(const uint4 *)(cring + slot * B::kCodes + b * 1024 + lane * 16);
      word[b][0] = c.x, word[b][1] = c.y, word[b][2] = c.z, word[b][3] = c.w;
      const uint32_t sb = table[(kt % kBgChunk) * B::kRows + b * 32 + (lane & 31)];
      if (FAST) {
        q[b] = dq_consts(sb);
      } else {
        sc[b] = bf16_to_f32(sb & 0xFFFFu);
        bi[b] = bf16_to_f32(sb >> 16);
      }
    }
    auto weights = [&](int ks, bf16x8_t (&w)[NB]) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint4 v = FAST ? dequant8_fast(word[b][ks], q[b], dk) : dequant8(word[b][ks], sc[b], bi[b]);
        w[b] = __builtin_bit_cast(bf16x8_t, v);
      }
    };
    auto fragments = [&](int ks, bf16x8_t (&x)[MB]) {
      const uint8_t *p = xs + (((lh + ks) ^ lx) << 4);
#pragma unroll
      for (int rb = 0; rb < MB; ++rb) x[rb] = __builtin_bit_cast(bf16x8_t, *(const uint4 *)(p + rb * 4096));
    };
    bf16x8_t w[2][NB], x[2][MB];
    fragments(0, x[0]);
    weights(0, w[0]);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks < 3) {
        fragments(ks + 1, x[(ks + 1) & 1]);
        weights(ks + 1, w[(ks + 1) & 1]);
      }
#pragma unroll
      for (int rb = 0; rb < MB; ++rb)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          acc[rb][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[ks & 1][rb], w[ks & 1][b], acc[rb][b], 0, 0, 0);
      if (FAST && ks < 3) {
        __builtin_amdgcn_sched_group_barrier(0x100, MB, 0);  // the next fragments' reads
#pragma unroll
        for (int i = 0; i < MB * NB; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);             // one MFMA (32 cycles)
          __builtin_amdgcn_sched_group_barrier(0x002, NB == 2 ? 5 : 9, 0);  // VALU operations of 4
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      // a third of the DMA of stage kt + 2 behind each slice's MFMAs, whose time
      // covers its issue
      if (ks < 3 && kt + 2 < steps) dma_part(kt + 2, slot == 0 ? 2 : slot - 1, ks);
    }
    slot = slot == kBgStages - 1 ? 0 : slot + 1;
  };
  // two whole loops, so that the accumulators meet no branch inside
  auto run = [&](auto fast_tag) {
    for (int k0 = 0; k0 < common; k0 += kBgChunk) {
      if (k0 > 0) {
        MOE_LN_WAIT_VMCNT(0);
        fill();
      }
      const int k1 = min(k0 + kBgChunk, common);
      for (int kt = k0; kt < k1; ++kt) {
        enter(kt);
        step(fast_tag, kt);
      }
    }
    // the first team's steps over: every wavefront keeps the barriers
    for (int kt = common; kt < common + left; ++kt) {
      if (team == 0 && kt % kBgChunk == 0 && kt > 0) {
        MOE_LN_WAIT_VMCNT(0);
        fill();
      }
      enter(kt);
      if (team == 0) step(fast_tag, kt);
    }
  };
  if (fast)
    run(std::true_type{});
  else
    run(std::false_type{});

  // Epilogue. The sums go through LDS ([team][wavefront][token][32 NB rows]), in
  // one or two passes; the teams share the tokens and add up their parts. C
  // layout: lane l holds weight row l % 32 of its block, register r token
  // 8 (r / 4) + 4 (l / 32) + r % 4.
  constexpr int kCols = B::kWaveRows, kLanesTok = kCols / 8, kPart = B::kPassTokens * kCols;
  float *const ep = (float *)smem + wave * kPart;
  // lane l: outputs 8 (l % kLanesTok) .. +7 of a token
  const int c8 = (lane % kLanesTok) * 8, n = n0 + c8;
  // 16-byte (bf16) and 32-byte (fp32) accesses where rows keep their alignment
  const bool wide = n + 8 <= a.rows && a.y_stride % 8 == 0 && (!a.residual || a.r_stride % 8 == 0);
  float bias[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) bias[i] = a.bias && n + i < a.rows ? bf16_to_f32(a.bias[n + i]) : 0.f;
#pragma unroll
  for (int pass = 0; pass < B::kPasses; ++pass) {
    if (pass == 0) lds_barrier();  // the rings are done with
#pragma unroll
    for (int rb = 0; rb < MB / B::kPasses; ++rb)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          ep[team * WT * kPart + (rb * 32 + (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3)) * kCols + b * 32 + (lane & 31)] =
              acc[pass * (MB / B::kPasses) + rb][b][r];
    if (KS > 1) lds_barrier();
    with_act(a.act, [&](auto act) {
      constexpr int kTurn = kWave / kLanesTok, kMine = B::kPassTokens / KS;  // tokens a turn, tokens a team
#pragma unroll 2
      for (int i = 0; i < kMine / kTurn; ++i) {
        const int tl = team * kMine + i * kTurn + lane / kLanesTok, t = t0 + pass * B::kPassTokens + tl;
        if (t >= a.T) continue;
        float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const float4 z0 = *(const float4 *)(ep + k * WT * kPart + tl * kCols + c8);
          const float4 z1 = *(const float4 *)(ep + k * WT * kPart + tl * kCols + c8 + 4);
          z[0] += z0.x, z[1] += z0.y, z[2] += z0.z, z[3] += z0.w;
          z[4] += z1.x, z[5] += z1.y, z[6] += z1.z, z[7] += z1.w;
        }
        if (wide) {
          store_outputs8<act.value, F32, KS == 1>(a, t, n, z, bias);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (n + j < a.rows) store_output<act.value, F32>(a, t, n + j, z[j], bias[j], load_residual<F32>(a, t, n + j));
        }
      }
    });
  }
}

// Where the kernels change over (5120 x 2048 weights unless said otherwise).
// Large tiles from 220 of them: 1500 tokens (240 tiles) 49 us against 55 on
// middle tiles, 1024 tokens (160) 49 against 44.
constexpr int kBgMinTiles = 220;
// The small kernel up to 16 tokens, and where its workgroups of 32 tokens do not
// outnumber the CUs: 64 tokens by 2048 rows (256 of them) 7 us against 10 on
// narrow tiles, 37 by 2048 x 4096 (256) 12 against 16, 32 tokens (320) 12
// against 10, 64 tokens (640) 16 against 10.
constexpr int kSmallMaxBlocks = 256;
// Narrow tiles while each has a CU to itself: 777 tokens by 1001 rows (208) 13 us
// against 19 on middle tiles, 512 by 2048 (256) 11 against 16, 300 tokens (400) 21
// against 17, 1000 by 2048 (512) 23 against 20.
constexpr int kNarrowMaxTiles = 256;

template <int MB, int NB, int KS, int WT>
static long long bg_tiles(int T, int rows) {
  using B = Bg<MB, NB, KS, WT>;
  return (long long)((T + B::kTokens - 1) / B::kTokens) * ((rows + B::kRows - 1) / B::kRows);
}

template <int NT>
static long long ln_blocks(int T, int rows) {
  return (long long)((rows + 15) / 16) * ((T + 16 * NT - 1) / (16 * NT));
}

template <int NT>
static hipError_t launch(const LinearArgs &a, int dtype, hipStream_t s) {
  auto *kernel = dtype ? linear_kernel<NT, true> : linear_kernel<NT, false>;
  kernel<<<(int)ln_blocks<NT>(a.T, a.rows), kLnWaves * kWave, 0, s>>>(a);
  return hipGetLastError();
}

template <int MB, int NB, int KS, int WT>
static hipError_t launch_tiles(const LinearArgs &a, int dtype, hipStream_t s) {
  using B = Bg<MB, NB, KS, WT>;
  auto *kernel = dtype ? linear_tiles_kernel<MB, NB, KS, WT, true> : linear_tiles_kernel<MB, NB, KS, WT, false>;
  static std::atomic<uint64_t> asked[2];
  const hipError_t st = allow_lds((const void *)kernel, B::kLds, asked[dtype ? 1 : 0]);
  if (st != hipSuccess) return st;
  kernel<<<(int)((bg_tiles<MB, NB, KS, WT>(a.T, a.rows) + 7) / 8 * 8), B::kThreads, B::kLds, s>>>(a);
  return hipGetLastError();
}

enum class LinearKind { kLargeTiles, kMiddleTiles, kNarrowTiles, kSmall16, kSmall32 };  // 16 and 32 tokens a workgroup

static LinearKind linear_kind(const LinearArgs &a) {
  if (a.T <= 16) return LinearKind::kSmall16;
  // the tile kernels keep 32-bit byte offsets within a tile
  const bool tiles = a.x_stride < (1 << 23) && a.cols < (1 << 23);
  if (tiles && bg_tiles<4, 2, 1, 4>(a.T, a.rows) >= kBgMinTiles) return LinearKind::kLargeTiles;
  if (!tiles || ln_blocks<2>(a.T, a.rows) <= kSmallMaxBlocks) return LinearKind::kSmall32;
  return bg_tiles<2, 1, 4, 2>(a.T, a.rows) <= kNarrowMaxTiles ? LinearKind::kNarrowTiles : LinearKind::kMiddleTiles;
}

bool linear_grid_ok(const LinearArgs &a) {
  long long threads = 0;
  switch (linear_kind(a)) {
    case LinearKind::kLargeTiles: threads = bg_tiles<4, 2, 1, 4>(a.T, a.rows) * 256; break;
    case LinearKind::kMiddleTiles: threads = bg_tiles<2, 1, 2, 4>(a.T, a.rows) * 512; break;
    case LinearKind::kNarrowTiles: threads = bg_tiles<2, 1, 4, 2>(a.T, a.rows) * 512; break;
    case LinearKind::kSmall16: threads = ln_blocks<1>(a.T, a.rows) * 512; break;
    case LinearKind::kSmall32: threads = ln_blocks<2>(a.T, a.rows) * 512; break;
  }
  return threads < (1ll << 32) - 8 * 512;  // of one launch dimension
}

hipError_t launch_linear(const LinearArgs &a, int dtype, hipStream_t s) {
  switch (linear_kind(a)) {
    case LinearKind::kLargeTiles: return launch_tiles<4, 2, 1, 4>(a, dtype, s);
    case LinearKind::kMiddleTiles: return launch_tiles<2, 1, 2, 4>(a, dtype, s);
    case LinearKind::kNarrowTiles: return launch_tiles<2, 1, 4, 2>(a, dtype, s);
    case LinearKind::kSmall16: return launch<1>(a, dtype, s);
    case LinearKind::kSmall32: break;
  }
  return launch<2>(a, dtype, s);
}

}  // namespace moe
