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
#include <type_traits>

#include "moe_linear.h"

namespace moe {

constexpr int kLnWaves = 8;
constexpr int kLnRows = 16;

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == kActRelu) return z > 0.f ? z : (z == z ? 0.f : z);
  if constexpr (ACT == kActSilu) return z / (1.0f + expf(-z));
  if constexpr (ACT == kActGelu) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
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

template <int NT, bool F32>
__global__ __launch_bounds__(kLnWaves *kWave, 2) void linear_kernel(LinearArgs a) {
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
  // four groups at a time: their loads are in flight together
  constexpr int kBatch = 4;
  for (int g0 = wave; g0 < ng; g0 += kLnWaves * kBatch) {
    uint2 c[kBatch];
    uint32_t s[kBatch], b[kBatch];
    uint4 x[kBatch][NT][2];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int g = min(g0 + j * kLnWaves, ng - 1);
      c[j] = *(const uint2 *)(codes + g * 32);
      s[j] = sp[g];
      b[j] = bp[g];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        x[j][i][0] = *(const uint4 *)(xp[i] + g * kGroup);
        x[j][i][1] = *(const uint4 *)(xp[i] + g * kGroup + 8);
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // all loads first
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (g0 + j * kLnWaves >= ng) break;
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
  with_act(a.act, [&](auto act) {
    for (int e = threadIdx.x; e < 16 * NT * kLnRows; e += kLnWaves * kWave) {
      const int t = e / kLnRows, n = e % kLnRows;
      if (t0 + t >= a.T || n0 + n >= a.rows) continue;
      float z = 0.f;
#pragma unroll
      for (int w = 0; w < kLnWaves; ++w) z += part[w][t][n];
      store_output<act.value, F32>(a, t0 + t, n0 + n, z, a.bias ? bf16_to_f32(a.bias[n0 + n]) : 0.f,
                                   load_residual<F32>(a, t0 + t, n0 + n));
    }
  });
}

// ------------------------------------------------------------------ large batches
//
// One workgroup = 4 wavefronts = 128 tokens x 256 weight rows; a wavefront
// takes all 128 tokens and its own 64 rows, so every weight is rebuilt once per
// 128 tokens, in registers, as the B operand of 32x32x16 MFMAs (C: lane =
// weight row, registers = tokens). Per K step of 64 (one group):
//   - activations (16 KB) come by LDS DMA into a ring of three stages shared by
//     the workgroup, 16-byte chunks XOR-swizzled by row so that fragment reads
//     of 8 or 16 rows hit distinct banks;
//   - codes come by LDS DMA too, into the wavefront's own ring, where each lane
//     reads back the 16 bytes it fetched (32 columns of one row);
//   - scales and biases sit in an LDS table of 8 groups of the wavefront's rows,
//     refilled every 8 steps.
// All loads of the loop are DMA, two steps ahead, and the loop waits for them
// by count: a load into registers there would make the compiler wait for every
// DMA behind it. Two workgroups share a CU (80 KB of LDS, 256 registers), so
// one rebuilds weights while the other multiplies.
constexpr int kBgTokens = 128, kBgRows = 256, kBgWaves = 4, kBgThreads = kBgWaves * kWave;
constexpr int kBgK = kGroup, kBgStages = 3, kBgChunk = 8;
constexpr int kBgX = kBgTokens * kBgK * 2;                   // bytes of activations a stage
constexpr int kBgCodes = kBgRows * kBgK / 2;                 // bytes of codes a stage
constexpr int kBgTable = kBgChunk * kBgRows * 4;             // (scale | bias << 16) words
constexpr int kBgLds = kBgStages * (kBgX + kBgCodes) + kBgTable;
constexpr int kBgLoads = kBgX / 4096 + kBgCodes / 4096;      // DMA instructions a wavefront and stage
static_assert(2 * kBgLds <= 160 * 1024, "two workgroups a CU");
static_assert(kBgWaves * 64 * 64 * 4 <= kBgLds, "the epilogue fits");

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

template <bool F32>
__global__ __launch_bounds__(kBgThreads, 2) void linear_tiles_kernel(LinearArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  int ti, ni;
  if (!bg_tile(blockIdx.x, (a.T + kBgTokens - 1) / kBgTokens, (a.rows + kBgRows - 1) / kBgRows, ti, ni)) return;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int t0 = ti * kBgTokens, n0 = ni * kBgRows + wave * 64;
  const int ng = a.cols / kGroup;
  const int tokens = min(kBgTokens, a.T - t0);

  // activations: DMA instruction i of wavefront w fills rows 32 i + 8 w .. +7,
  // lane l row l / 8 of those, LDS chunk l % 8, which holds the row's chunk
  // (l % 8) ^ (row % 8) ^ (row / 8 % 2). Rows past the last re-read it.
  const ln_u32x4 xr = ln_rsrc(a.x + t0 * a.x_stride, (uint32_t)(((tokens - 1) * a.x_stride + a.cols) * 2));
  uint32_t x_off[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = min(32 * i + 8 * wave + (lane >> 3), tokens - 1);
    x_off[i] = (uint32_t)(r * (int)a.x_stride + (((lane & 7) ^ (lane >> 3) ^ (wave & 1)) * 8)) * 2u;
  }
  // codes: instruction b fetches row 32 b + l % 32, columns 32 (l / 32) .. +31
  const uint8_t *codes = a.w.codes + (long long)min(n0, a.rows - 1) * (a.cols / 2);
  const int wrows = max(min(64, a.rows - n0), 1);
  const ln_u32x4 cr = ln_rsrc(codes, (uint32_t)(wrows * (a.cols / 2)));
  uint32_t c_off[2];
#pragma unroll
  for (int b = 0; b < 2; ++b)
    c_off[b] = (uint32_t)(min(32 * b + (lane & 31), wrows - 1) * (a.cols / 2) + (lane >> 5) * 16);
  const uint32_t x_lds = ln_lds_address(smem) + wave * 1024;
  uint8_t *cring = smem + kBgStages * kBgX + wave * 2048;  // this wavefront's part of a stage
  const uint32_t c_lds = ln_lds_address(cring);
  uint32_t *table = (uint32_t *)(smem + kBgStages * (kBgX + kBgCodes)) + wave * 64;
  auto dma = [&](int step, int slot) {
#pragma unroll
    for (int i = 0; i < 4; ++i) ln_dma(xr, x_off[i], step * (kBgK * 2), x_lds + slot * kBgX + i * 4096);
#pragma unroll
    for (int b = 0; b < 2; ++b) ln_dma(cr, c_off[b], step * (kBgK / 2), c_lds + slot * kBgCodes + b * 1024);
  };

  // scales and biases of 8 groups of row `lane` of the wavefront
  const long long srow = (long long)(min(n0, a.rows - 1) + min(lane, wrows - 1)) * ng;
  const uint16_t *sp = a.w.scales + srow, *bp = a.w.biases + srow;
  const bool vec = ng % 8 == 0;  // 16-byte loads stay aligned
  uint4 sv, bv;
  auto fetch = [&](int g0) {
    if (vec) {
      sv = *(const uint4 *)(sp + g0);
      bv = *(const uint4 *)(bp + g0);
    } else {
      uint32_t s[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int g = min(g0 + 2 * i, ng - 1), h = min(g0 + 2 * i + 1, ng - 1);
        s[i] = sp[g] | (uint32_t)sp[h] << 16;
        b[i] = bp[g] | (uint32_t)bp[h] << 16;
      }
      sv = make_uint4(s[0], s[1], s[2], s[3]);
      bv = make_uint4(b[0], b[1], b[2], b[3]);
    }
  };
  auto fill = [&]() {
    const uint32_t s[4] = {sv.x, sv.y, sv.z, sv.w}, b[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      table[(2 * i) * kBgRows + lane] = (s[i] & 0xFFFFu) | (b[i] << 16);
      table[(2 * i + 1) * kBgRows + lane] = (s[i] >> 16) | (b[i] & 0xFFFF0000u);
    }
  };
  // does every group of the wavefront's rows take the fast dequantisation?
  bool ok = true;
#pragma unroll 4
  for (int g0 = 0; g0 < ng; g0 += kBgChunk) {
    fetch(g0);
    const uint32_t s[4] = {sv.x, sv.y, sv.z, sv.w}, b[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ok &= (int)dq_fast_ok((s[i] & 0xFFFFu) | (b[i] << 16)) & (int)dq_fast_ok((s[i] >> 16) | (b[i] & 0xFFFF0000u));
  }
  const bool fast = __builtin_amdgcn_ballot_w64(!ok) == 0;

  fetch(0);
  fill();
  dma(0, 0);
  if (ng > 1) dma(1, 1);

  f32x16_t acc[4][2];
#pragma unroll
  for (int rb = 0; rb < 4; ++rb) acc[rb][0] = acc[rb][1] = f32x16_t{0};
  const DqRegs dk = dq_regs();
  const int lrow = (lane & 31) * 128, lx = (lane & 7) ^ ((lane >> 3) & 1), lh = 4 * (lane >> 5);

  // one K step; the weights of a slice of 16 columns are rebuilt, and its
  // activation fragments read, while the slice before it is multiplied
  int slot = 0;
  auto step = [&](auto fast_tag, int kt) {
    constexpr bool FAST = decltype(fast_tag)::value;
    // stage kt has landed (only the DMA of stage kt + 1 may still be in flight);
    // the barrier also tells that every wavefront is done with stage kt - 1
    if (kt + 1 < ng)
      MOE_LN_WAIT_VMCNT(kBgLoads);
    else
      MOE_LN_WAIT_VMCNT(0);
    lds_barrier();
    asm volatile("" ::: "memory");
    if (kt % kBgChunk == kBgChunk - 1 && kt + 1 < ng) fetch(kt + 1);
    if (kt + 2 < ng) dma(kt + 2, slot == 0 ? 2 : slot - 1);
    const uint8_t *xs = smem + slot * kBgX + lrow;
    uint32_t word[2][4];
    DqGroup q[2];
    float sc[2], bi[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint4 c = *(const uint4 *)(cring + slot * kBgCodes + b * 1024 + lane * 16);
      word[b][0] = c.x, word[b][1] = c.y, word[b][2] = c.z, word[b][3] = c.w;
      const uint32_t sb = table[(kt % kBgChunk) * kBgRows + b * 32 + (lane & 31)];
      if (FAST) {
        q[b] = dq_consts(sb);
      } else {
        sc[b] = bf16_to_f32(sb & 0xFFFFu);
        bi[b] = bf16_to_f32(sb >> 16);
      }
    }
    auto weights = [&](int ks, bf16x8_t (&w)[2]) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint4 v = FAST ? dequant8_fast(word[b][ks], q[b], dk) : dequant8(word[b][ks], sc[b], bi[b]);
        w[b] = __builtin_bit_cast(bf16x8_t, v);
      }
    };
    auto fragments = [&](int ks, bf16x8_t (&x)[4]) {
      const uint8_t *p = xs + (((lh + ks) ^ lx) << 4);
#pragma unroll
      for (int rb = 0; rb < 4; ++rb) x[rb] = __builtin_bit_cast(bf16x8_t, *(const uint4 *)(p + rb * 4096));
    };
    bf16x8_t w[2][2], x[2][4];
    fragments(0, x[0]);
    weights(0, w[0]);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks < 3) {
        fragments(ks + 1, x[(ks + 1) & 1]);
        weights(ks + 1, w[(ks + 1) & 1]);
      }
#pragma unroll
      for (int rb = 0; rb < 4; ++rb)
#pragma unroll
        for (int b = 0; b < 2; ++b)
          acc[rb][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[ks & 1][rb], w[ks & 1][b], acc[rb][b], 0, 0, 0);
      if (FAST && ks < 3) {
        __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);  // the next fragments' reads
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one MFMA (32 cycles)
          __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);  // five VALU operations (20)
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    slot = slot == kBgStages - 1 ? 0 : slot + 1;
  };
  // two whole loops, so that the accumulators meet no branch inside
  auto run = [&](auto fast_tag) {
    for (int k0 = 0; k0 < ng; k0 += kBgChunk) {
      if (k0 > 0) {
        MOE_LN_WAIT_VMCNT(0);
        fill();
      }
      const int k1 = min(k0 + kBgChunk, ng);
      for (int kt = k0; kt < k1; ++kt) step(fast_tag, kt);
    }
  };
  if (fast)
    run(std::true_type{});
  else
    run(std::false_type{});

  // Epilogue. The sums go through the wavefront's quarter of the LDS, 64 tokens
  // by 64 rows at a time, and leave a token's 64 outputs to a wavefront store.
  // C layout: lane l holds weight row l % 32 of its block, register r token
  // 8 (r / 4) + 4 (l / 32) + r % 4.
  lds_barrier();
  float *ep = (float *)(smem + wave * (64 * 64 * 4));
  const int n = n0 + lane;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          ep[(rb * 32 + (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3)) * 64 + b * 32 + (lane & 31)] =
              acc[half * 2 + rb][b][r];
    const int tb = t0 + half * 64, te = min(64, a.T - tb);
    if (n < a.rows) {
      const float bias = a.bias ? bf16_to_f32(a.bias[n]) : 0.f;
      with_act(a.act, [&](auto act) {
#pragma unroll 4
        for (int t = 0; t < te; ++t)
          store_output<act.value, F32>(a, tb + t, n, ep[t * 64 + lane], bias, load_residual<F32>(a, tb + t, n));
      });
    }
  }
}

static long long linear_blocks(int T, int rows) {
  return (long long)((rows + kLnRows - 1) / kLnRows) * ((T + 15) / 16);
}

// Below this many tokens the 16-row kernel is faster.
constexpr int kBgMinT = 128;

static bool tiles_fit(const LinearArgs &a) {
  // 32-bit byte offsets within a tile
  return a.T >= kBgMinT && a.x_stride < (1 << 23) && a.cols < (1 << 23);
}

bool linear_grid_ok(int T, int rows) { return linear_blocks(T, rows) < (1ll << 23); }

template <int NT>
static void launch(const LinearArgs &a, int dtype, hipStream_t s) {
  const int grid = (int)((long long)((a.rows + kLnRows - 1) / kLnRows) * ((a.T + 16 * NT - 1) / (16 * NT)));
  auto *kernel = dtype ? linear_kernel<NT, true> : linear_kernel<NT, false>;
  kernel<<<grid, kLnWaves * kWave, 0, s>>>(a);
}

static hipError_t launch_tiles(const LinearArgs &a, int dtype, hipStream_t s) {
  auto *kernel = dtype ? linear_tiles_kernel<true> : linear_tiles_kernel<false>;
  static const hipError_t st = [] {  // more than 64 KB of LDS needs an opt-in, once per process
    const hipError_t e = hipFuncSetAttribute((const void *)linear_tiles_kernel<true>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kBgLds);
    return e != hipSuccess ? e
                           : hipFuncSetAttribute((const void *)linear_tiles_kernel<false>,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, kBgLds);
  }();
  if (st != hipSuccess) return st;
  const int tiles = ((a.T + kBgTokens - 1) / kBgTokens) * ((a.rows + kBgRows - 1) / kBgRows);
  kernel<<<(tiles + 7) / 8 * 8, kBgThreads, kBgLds, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_linear(const LinearArgs &a, int dtype, hipStream_t s) {
  if (tiles_fit(a)) return launch_tiles(a, dtype, s);
  if (a.T <= 16)
    launch<1>(a, dtype, s);
  else if (a.T <= 32)
    launch<2>(a, dtype, s);
  else
    launch<4>(a, dtype, s);
  return hipGetLastError();
}

}  // namespace moe
