// Attention over the paged int4-g64 key/value cache.
//
//   o[r] = sum_t softmax_t(scale * q_r . k_t) v_t,   k_t, v_t = s * code + b
// over the keys t that query row r (a new token of a sequence and a head)
// sees; a row that sees no key gives zeros. The G = Hq / Hkv heads of one
// cache head are rows of the same tile, so its keys are read once for all.
//
// The scales and biases never touch the 4-bit codes. With c = 16 + code as an
// exact bf16 integer (0x4180 | code << 3):
//   q.k_t   = sum_g [ s_tg (q_g . c_tg) + (b_tg - 16 s_tg) sum(q_g) ]
//   o       = sum_t (p_t s_tg) c_t - 24 sum_t (p_t s_tg) + sum_t p_t (b_tg + 8 s_tg)
// per group g of 64 channels, so the matrix cores multiply codes, at one VALU
// operation per code for the conversion, and the affine part costs a few
// fp32 operations per key and group. p_t s_tg is rounded to bf16 for the
// matrix cores (each term off by at most 2^-9 of itself, like any bf16 softmax
// weight); the same rounded weights are summed for the second term, so the
// centred code (code - 8) is what carries the rounding. Scores, softmax
// statistics, the affine sums and all accumulators are fp32.
//
// Everything is transposed so that no operand changes lanes between the two
// products (16x16x32 MFMA, lane l: column l % 16, lane group l / 16):
//   S^T = K Q^T   rows are keys, columns query rows: a lane ends up with keys
//                 4 (l/16) .. +3 of each 16-key half for its own query row;
//   O^T = V^T P^T contracts over those keys, 8 to a lane; the lane's V operand
//                 are the 8 keys' codes of channel 16 j + l % 16, which one
//                 transposing LDS read (16 keys by 16 channels of 4 bits a
//                 lane group) delivers for two j at once.
// The order inside a contraction is free, so the nibbles of a word are taken
// in the order 0 4 1 5 2 6 3 7 (one shift and one and-or give two of them),
// and the query and the weights are laid out to match.
//
// Bound by memory for many or long sequences, by its chain of dependent loads
// (offsets, pages, codes) for few short ones. us, one new token a sequence, 16
// heads on 2: 64 sequences of up to 8101, D = 256 (113 MB) 33.2 and 5.4 for the
// join, 3.4 TB/s; one of 131,150, D = 128 (38 MB) 16.9 and 6.8; one of 500, D =
// 256 11.7. 3000 lists of 1024 keys of their own, 8 heads, D = 128: 74.3 (90.1 with
// half the columns empty), 90% of it vector instructions: the codes' conversion is 128
// of 214 a tile, and a workgroup's start and end cost as much as three tiles.
#include "moe_kv4_device.h"
#include "moe_lds.h"

namespace moe {

constexpr int kAtRows = 16;  // query rows (token, head of the group) per workgroup; its wavefronts split the keys

// Constants of the conversion, kept in registers and opaque to the compiler so
// that it is one shift and one v_and_or_b32 (which takes no literals).
struct CodeRegs {
  uint32_t mask, magic;  // 0x00780078 (scalar), 0x41804180 (vector)
};

__device__ __forceinline__ CodeRegs code_regs() {
  CodeRegs k;
  asm("s_mov_b32 %0, 0x00780078" : "=s"(k.mask));
  asm("v_mov_b32 %0, 0x41804180" : "=v"(k.magic));
  return k;
}

// Nibble i of both halves of x as two bf16 16 + code.
__device__ __forceinline__ uint32_t codes2(uint32_t x, int i, const CodeRegs &k) {
  return and_or(i == 0 ? x << 3 : x >> (4 * i - 3), k.mask, k.magic);
}

__device__ __forceinline__ bf16x8_t codes8(uint32_t c, const CodeRegs &k) {
  const uint4 r = make_uint4(codes2(c, 0, k), codes2(c, 1, k), codes2(c, 2, k), codes2(c, 3, k));
  return __builtin_bit_cast(bf16x8_t, r);
}

// a plus the two bf16 values of w (products with 1 are exact).
__device__ __forceinline__ float sum_bf16x2(uint32_t w, float a) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w),
                                         __builtin_bit_cast(bf16x2_t, 0x3F803F80u), a, false);
}

// The affine part of the scores, sum_g (b_tg - 16 s_tg) qsum_g, as one more
// MFMA of a 16-key half: the operand of the keys is their biases and scales as
// they lie in the cache, the other one qsum cut into three bf16 (hi, lo, lo2:
// 24 bits, so nothing is lost) and -16 times that. Contraction slots, by lane
// group (8 each): b x hi, b x lo | b x lo2, s x hi | s x lo, s x lo2 | none for
// NG = 4; b x hi, lo, lo2, s x hi | s x lo, lo2 | none for NG = 2; all six in
// the first group for NG = 1.
template <int NG>
__device__ __forceinline__ bf16x8_t affine_query(const float (&qsum)[NG], int group) {
  float v[6 * NG];  // [slot][g]
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    float rest = qsum[g];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const float part = bf16_to_f32(to_bf16(rest));
      v[i * NG + g] = part;
      v[(3 + i) * NG + g] = -16.0f * part;
      rest -= part;
    }
  }
  uint32_t e[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e[i] = 0;
#pragma unroll
    for (int lg = 0; lg < 4; ++lg) {
      const int at = lg * 8 + i * 2;
      if (at < 6 * NG) e[i] = group == lg ? pack_bf16x2(v[at], v[at + 1]) : e[i];
    }
  }
  return __builtin_bit_cast(bf16x8_t, make_uint4(e[0], e[1], e[2], e[3]));
}

// Sum and maximum over the four lane groups (lanes l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float groups_sum(float v) {
  v += __shfl_xor(v, 16, kWave);
  return v + __shfl_xor(v, 32, kWave);
}
__device__ __forceinline__ float groups_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
}

// bf16 number i of packed words w.
template <int N>
__device__ __forceinline__ float bf16_at(const uint32_t (&w)[N], int i) {
  return (i & 1) ? __uint_as_float(w[i / 2] & 0xFFFF0000u) : __uint_as_float(w[i / 2] << 16);
}

// ---- a wavefront's ring of key tiles in LDS
//
// Each wavefront fills its own ring with LDS DMA (no registers, no barriers)
// and waits only for its own vector-memory counter. A stage holds a tile of
// 32 keys: codes of the keys, codes of the values, then their scales and
// biases in the cache's own order. A row's 32-byte groups are XOR-swizzled by
// (key / 4), so that the 16 rows of a key operand and the 4 rows of a value
// operand lie in different banks; the DMA's source address carries the
// swizzle, since its LDS side is in lane order.
constexpr int kStages = 2;

template <int D>
struct Ring {
  static constexpr int NG = D / kGroup;
  static constexpr int kRow = D / 2;                      // bytes of codes a key
  static constexpr int kCodes = kKvTile * kRow;           // bytes of a tile's key (or value) codes
  static constexpr int kMeta = kKvTile * NG * 2;          // bytes of a tile's scales (or biases)
  static constexpr int kStage = 2 * kCodes + 4 * kMeta;
  static constexpr int kCodeLoads = kCodes / 1024;        // DMA instructions of 64 x 16 bytes
  static constexpr int kLoads = 2 * kCodeLoads + 1;       // one takes all the scales and biases
};

// s_waitcnt with only the vector-memory counter limited.
#define MOE_KV_WAIT_VMCNT(n) \
  __builtin_amdgcn_s_waitcnt(((n) & 0xF) | (0x7 << 4) | (0xF << 8) | (((n) >> 4) << 14))

typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2_t kv_lds_i32x2;
typedef __attribute__((address_space(3))) void kv_lds_void;
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// LDS DMA, 16 bytes a lane, to LDS address dst + 16 * lane (dst wave-uniform).
// Written as assembly because the compiler, which cannot tell the ring's stages
// apart, would wait for every DMA in flight before each LDS read; here the
// waits are the explicit ones in the loop. No register is written. The no-ops
// cover m0 (one wait state) and scalar operands fresh from the VALU (five).
__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(kv_lds_void *)p);
}

// From base + off, base wave-uniform with `bytes` readable bytes.
__device__ __forceinline__ void load_lds16(const uint8_t *base, uint32_t bytes, uint32_t off, uint32_t dst) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  u32x4_t r;
  r[0] = __builtin_amdgcn_readfirstlane((uint32_t)b);
  r[1] = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32) & 0xFFFFu);
  r[2] = bytes;
  r[3] = 0x00020000;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               ::"s"(dst), "v"(off), "s"(r) : "memory");
}

// From each lane's own address.
__device__ __forceinline__ void load_lds16(const void *p, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, off"
               ::"s"(dst), "v"(p) : "memory");
}

// What a lane's DMA and LDS addresses are made of: few registers, from which
// each tile's addresses follow in an operation or two.
template <int D>
struct LaneParts {
  uint32_t code;             // byte of this lane's chunk in a half's codes, with the swizzle
  const uint16_t *meta;      // this lane's 16 bytes of the first row's scales or biases
  uint32_t key, value, scale;  // LDS bytes of its key codes, value codes, scales in a stage
  uint32_t affine0, affine1;   // and of what affine_keys reads
};

template <int D, bool HALF>
__device__ __forceinline__ LaneParts<D> lane_parts(const Kv4Plane &kc, const Kv4Plane &vc, int lane) {
  using R = Ring<D>;
  constexpr int NG = R::NG, kChunks = R::kRow / 16;
  LaneParts<D> p;
  const int key = lane / kChunks, at = lane % kChunks;
  p.code = (key & 15) * R::kRow + ((((at >> 1) ^ ((key >> 2) & (NG - 1))) << 1) | (at & 1)) * 16;
  const int array = lane / (4 * NG);  // of 2 NG chunks a half; lanes past 16 NG have none
  p.meta = (array & 1 ? (array & 2 ? vc.biases : kc.biases) : (array & 2 ? vc.scales : kc.scales)) +
           (lane % (2 * NG)) * 8;
  p.key = (lane & 15) * R::kRow + (lane >> 4) * 8 + (((lane >> 2) & (NG - 1)) << 5);
  // lane k % 8 of a lane group supplies the row of the group's k-th key (4 of
  // the first half, 4 of the second), lanes 8 .. 15 the next 16 channels; HALF: in
  // the order in which codes8 puts the halves one behind the other
  const int of = HALF ? 2 * (lane & 1) + (lane >> 2 & 1) + 8 * (lane & 2) : (lane & 3) + 4 * (lane & 4);
  p.value = R::kCodes + (4 * (lane >> 4) + of) * R::kRow + (lane & 8) + (((lane >> 4) & (NG - 1)) << 5);
  p.scale = 2 * R::kCodes + (lane >> 4) * 4 * NG * 2 + (HALF ? (lane >> 3 & 1) * 16 * NG * 2 : 0);
  const uint32_t s_at = 2 * R::kCodes + (lane & 15) * NG * 2, b_at = s_at + R::kMeta;
  p.affine0 = lane >> 4 <= (NG == 4 ? 1 : 0) ? b_at : s_at;
  p.affine1 = NG == 4 && lane >> 4 == 0 ? b_at : s_at;
  return p;
}

// Starts the DMA of one tile into a stage. A half without a page reads page 0
// (its keys are masked).
template <int D>
__device__ __forceinline__ void load_tile(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc,
                                          const TilePages &p, int head, int tile, uint32_t dst,
                                          const LaneParts<D> &lp, int lane) {
  using R = Ring<D>;
  constexpr int NG = R::NG;
  long long row[2];
#pragma unroll
  for (int u = 0; u < 2; ++u)
    row[u] = kv4_row(dm, p.page[u] < 0 ? 0 : p.page[u], head, (tile * kKvTile + 16 * u) & (dm.page - 1));
#pragma unroll
  for (int i = 0; i < R::kCodeLoads; ++i) {
    if constexpr (NG >= 2) {
      // an instruction stays in one half: a scalar base and a 32-bit lane
      // offset (D = 256: the half's second 8 keys, whose swizzle differs by 2)
      const uint32_t off = NG == 4 && (i & 1) ? (lp.code ^ 64u) + 8 * R::kRow : lp.code;
      const long long r = row[i / (R::kCodeLoads / 2)] * R::kRow;
      load_lds16(kc.codes + r, 16 * R::kRow, off, dst + i * 1024);
      load_lds16(vc.codes + r, 16 * R::kRow, off, dst + R::kCodes + i * 1024);
    } else {
      const long long r = (lane >= 32 ? row[1] : row[0]) * R::kRow + lp.code;
      load_lds16(kc.codes + r, dst + i * 1024);
      load_lds16(vc.codes + r, dst + R::kCodes + i * 1024);
    }
  }
  if (NG == 4 || lane < 16 * NG)
    load_lds16(lp.meta + (lane & (2 * NG) ? row[1] : row[0]) * NG, dst + 2 * R::kCodes);
}

// This lane's scales or biases of one 16-key half: keys 4 (l / 16) .. +3, NG
// groups each, as packed bf16 pairs.
template <int NG>
__device__ __forceinline__ void read_meta(const uint8_t *p, uint32_t (&w)[2 * NG]) {
  if constexpr (NG == 1) {
    const uint2 x = *(const uint2 *)p;
    w[0] = x.x, w[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < NG / 2; ++i) {
      const uint4 x = *(const uint4 *)(p + 16 * i);
      w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
    }
  }
}

// The operand of affine_query for the keys of half u: key l % 16.
template <int NG>
__device__ __forceinline__ bf16x8_t affine_keys(const uint8_t *stage, const LaneParts<NG * kGroup> &lp, int u) {
  const uint8_t *p0 = stage + lp.affine0 + 16 * u * NG * 2, *p1 = stage + lp.affine1 + 16 * u * NG * 2;
  uint4 r;
  if constexpr (NG == 4) {
    const uint2 x = *(const uint2 *)p0, y = *(const uint2 *)p1;
    r = make_uint4(x.x, x.y, y.x, y.y);
  } else if constexpr (NG == 2) {
    const uint32_t x = *(const uint32_t *)p0, y = *(const uint32_t *)p1;
    r = make_uint4(x, x, x, y);
  } else {
    const uint32_t x = *(const uint16_t *)p0, y = *(const uint16_t *)p1;
    r = make_uint4(x | x << 16, x | y << 16, y | y << 16, 0u);
  }
  return __builtin_bit_cast(bf16x8_t, r);
}

// What one wavefront has summed up for its 16 query rows; a lane holds its row
// (column l % 16) and, for each group, channels 64 g + 16 j + 4 (l / 16) + r.
template <int D>
struct RowSums {
  static constexpr int NG = D / kGroup;
  f32x4_t o[NG][4];  // [g][j]: register r
  float w[NG];       // sum of the rounded weights p s, this lane's keys only
  float c[NG];       // sum of p (b + 8 s), this lane's keys only
  float m, l;        // reference score (unscaled); sum of p, this lane's keys only
};

// One 32-key tile. masked (wave-uniform): some row does not see some key (t0 ..
// t1 - 1 is what this lane's row sees) or a page does not exist.
//
// HALF: there are at most 8 query rows, and each is two columns: column c has its
// weights of the tile's first half of the keys, column c + 8 of the second half, so
// that no lane's work on scores and weights is for nothing. The columns are joined
// at the end like two wavefronts' parts.
template <int D, bool HALF>
__device__ __forceinline__ void attend_tile(const uint8_t *stage, const LaneParts<D> &lp,
                                            const bf16x8_t (&q)[D / kGroup][2],
                                            const bf16x8_t &qaff, float scale2,
                                            bool masked, int lane, int key0, int t0, int t1,
                                            const TilePages &pages, RowSums<D> &a) {
  using R = Ring<D>;
  constexpr int NG = R::NG;
  const uint8_t *meta = stage + lp.scale;
  const CodeRegs kr = code_regs();
  constexpr int H = HALF ? 1 : 2;  // halves whose keys are this lane's
  const bool second = (lane & 8) != 0;
  float s[4 * H];
  if constexpr (HALF) {
    f32x4_t x, acc[NG];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4_t v = {0.f, 0.f, 0.f, 0.f};
      v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(affine_keys<NG>(stage, lp, u), qaff, v, 0, 0, 0);
      x = u == 0 || second ? v : x;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint2 c = *(const uint2 *)(stage + (lp.key ^ (g << 5)) + 16 * u * R::kRow);
        f32x4_t y = {0.f, 0.f, 0.f, 0.f};
        y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes8(c.x, kr), q[g][0], y, 0, 0, 0);
        y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes8(c.y, kr), q[g][1], y, 0, 0, 0);
        acc[g] = u == 0 || second ? y : acc[g];
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    uint32_t ws[2 * NG];
    read_meta<NG>(meta, ws);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      s[r] = x[r];
#pragma unroll
      for (int g = 0; g < NG; ++g) s[r] = fmaf(bf16_at(ws, r * NG + g), acc[g][r], s[r]);
    }
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t ws[2 * NG];
      read_meta<NG>(meta + 16 * u * NG * 2, ws);
      f32x4_t x = {0.f, 0.f, 0.f, 0.f};
      x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(affine_keys<NG>(stage, lp, u), qaff, x, 0, 0, 0);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint2 c = *(const uint2 *)(stage + (lp.key ^ (g << 5)) + 16 * u * R::kRow);
        f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes8(c.x, kr), q[g][0], acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes8(c.y, kr), q[g][1], acc, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = fmaf(bf16_at(ws, r * NG + g), acc[r], x[r]);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) s[4 * u + r] = x[r];
      __builtin_amdgcn_sched_barrier(0);  // one half's operands at a time: registers
    }
  }
  uint32_t ws[H][2 * NG], wb[H][2 * NG];
#pragma unroll
  for (int u = 0; u < H; ++u) {
    read_meta<NG>(meta + 2 * R::kMeta + 16 * u * NG * 2, ws[u]);
    read_meta<NG>(meta + 3 * R::kMeta + 16 * u * NG * 2, wb[u]);
  }
  if (masked) {
    // An unseen slot may hold anything, NaN included: its score becomes -inf
    // and its value's scale and bias 0, by selection and never by a product.
#pragma unroll
    for (int i = 0; i < 4 * H; ++i) {
      const int u = i >> 2, r = i & 3, t = key0 + (HALF ? 2 * (lane & 8) : u * 16) + (lane >> 4) * 4 + r;
      const bool seen = (HALF && second ? pages.page[1] : pages.page[u]) >= 0 && t >= t0 && t < t1;
      s[i] = seen ? s[i] : kNegInf;
      if constexpr (NG == 1) {
        const uint32_t keep = seen ? 0xFFFFFFFFu : (r & 1 ? 0x0000FFFFu : 0xFFFF0000u);
        ws[u][r / 2] &= keep;
        wb[u][r / 2] &= keep;
      } else {
#pragma unroll
        for (int k = 0; k < NG / 2; ++k) {
          ws[u][r * NG / 2 + k] = seen ? ws[u][r * NG / 2 + k] : 0u;
          wb[u][r * NG / 2 + k] = seen ? wb[u][r * NG / 2 + k] : 0u;
        }
      }
    }
  }
  float mx = s[0];
#pragma unroll
  for (int i = 1; i < 4 * H; ++i) mx = fmaxf(mx, s[i]);
  if (__builtin_amdgcn_ballot_w64((mx - a.m) * scale2 > kSlack) != 0) {
    const float m = fmaxf(a.m, groups_max(mx));
    const float alpha = a.m == kNegInf ? 0.f : __builtin_amdgcn_exp2f((a.m - m) * scale2);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) a.o[g][j][r] *= alpha;
      a.w[g] *= alpha;
      a.c[g] *= alpha;
    }
    a.l *= alpha;
    a.m = m;
  }
  const float ref = a.m == kNegInf ? 0.f : a.m;  // nothing seen yet: every weight is exp2(-inf) = 0
  float p[4 * H];
#pragma unroll
  for (int i = 0; i < 4 * H; ++i) {
    p[i] = __builtin_amdgcn_exp2f((s[i] - ref) * scale2);  // see kSlack for this order
    a.l += p[i];
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    i32x2_t vc[2];  // 8 keys' codes of channels 64 g + 16 j + l % 16, j = 0, 1 and 2, 3
#pragma unroll
    for (int i = 0; i < 2; ++i)
      vc[i] = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
          (kv_lds_i32x2 *)(stage + (lp.value ^ (g << 5)) + 16 * i));
    float ps[4 * H];
#pragma unroll
    for (int i = 0; i < 4 * H; ++i) {
      const float sc = bf16_at(ws[i >> 2], (i & 3) * NG + g), bi = bf16_at(wb[i >> 2], (i & 3) * NG + g);
      ps[i] = p[i] * sc;
      a.c[g] = fmaf(p[i], fmaf(8.0f, sc, bi), a.c[g]);
    }
    // the keys in the order codes8 takes nibbles
    uint4 pw;
    if constexpr (HALF) {
      const uint32_t w0 = pack_bf16x2(ps[0], ps[1]), w1 = pack_bf16x2(ps[2], ps[3]);
      a.w[g] = sum_bf16x2(w0, sum_bf16x2(w1, a.w[g]));
      pw = make_uint4(second ? 0u : w0, second ? 0u : w1, second ? w0 : 0u, second ? w1 : 0u);
    } else {
      pw = make_uint4(pack_bf16x2(ps[0], ps[4]), pack_bf16x2(ps[1], ps[5]), pack_bf16x2(ps[2], ps[6]),
                      pack_bf16x2(ps[3], ps[7]));
      a.w[g] = sum_bf16x2(pw.x, sum_bf16x2(pw.y, sum_bf16x2(pw.z, sum_bf16x2(pw.w, a.w[g]))));
    }
    const bf16x8_t pb = __builtin_bit_cast(bf16x8_t, pw);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      a.o[g][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes8((uint32_t)vc[j >> 1][j & 1], kr), pb,
                                                          a.o[g][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Keys the tile's rows can see.
__device__ __forceinline__ Kv4Range tile_range(const Kv4Dims &dm, const RowTile &t, int rows, bool causal,
                                               int window) {
  const int G = dm.Hq / dm.Hkv;
  const int last = min(t.row0 + rows, t.rows) - 1;
  return kv4_range(dm, t.sp.first + t.row0 / G, t.sp.first + last / G, t.sp.len, causal, window);
}

// What a part of a row (reference m_i, sum l_i) counts for at reference m: one
// that saw no key (l_i = 0) nothing; one whose scores were all NaN has no
// reference and passes its NaN on.
__device__ __forceinline__ float part_weight(float m_i, float l_i, float m, float scale2) {
  const float none = l_i == 0.f ? kNegInf : 0.f;
  return __builtin_amdgcn_exp2f(m_i == kNegInf ? none : (m_i - m) * scale2);
}

// Channels c .. c + 3 of a token's head, divided by the row's sum; a row that
// saw no key is zero.
__device__ __forceinline__ void store_row(const Kv4Dims &dm, const Kv4Attn &at, int tok, int head, int c,
                                          float l, const float4 &o) {
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  *(uint2 *)(at.out + tok * at.out_stride + (long long)head * dm.D + c) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

// LDS of a workgroup of W wavefronts: their rings, and over them, at the end,
// their results ([wave][16 rows][D + 4] floats).
template <int D, int W>
constexpr int at_lds_bytes() {
  static_assert(kAtRows * (D + 4) * 4 <= kStages * Ring<D>::kStage, "the results fit over the rings");
  return W * kStages * Ring<D>::kStage;
}

// Splitting a sequence's keys over workgroups of 4 wavefronts: at least
// kMinTiles tiles each (4 a wavefront), and no more workgroups than the card's
// 256 CUs hold at a time. A workgroup too many runs alone after the others: 516
// instead of 512 took a batch of 64 mixed sequences from 33 to 57 us.
constexpr int kMinTiles = 16;
// Of rows that are sequences, which have few keys: two a wavefront (us of this kernel and
// the join for 2048 keys of one token, 16 heads on 2, D = 128: 9.5 + 2.9 with four,
// 7.4 + 3.4 with two, 6.2 + 4.8 with one).
constexpr int kMinTilesRows = 8;
// Workgroups of 4 wavefronts a CU holds: wavefronts a SIMD by their registers
// (214, 130 and 90; a 4-wavefront limit at D = 128 spills a pointer of the loop,
// and its reload waits for the DMA in flight).
template <int D>
constexpr int at_blocks() { return D == 256 ? 2 : D == 128 ? 3 : 5; }
template <int D>
constexpr int at_slots() { return 256 * at_blocks<D>(); }
// Batches up to this size spread their keys evenly over the workgroups (the
// lengths are on the device, so each wavefront adds them up, 64 at a time);
// larger ones have enough sequences to fill the card with.
constexpr int kEvenMaxB = 256;

// Tiles a workgroup takes of a sequence, so that all workgroups of the call
// have about the same and all fit the card: sum ceil(n_b / per) <= total / per +
// tasks. (kv4_share raises it where `splits` are too few.)
template <int D>
__device__ __forceinline__ int tiles_per_split(const Kv4Dims &dm, const Kv4Batch &bt, const Kv4Attn &at) {
  if (dm.B > kEvenMaxB) return kMinTiles;
  const int lane = threadIdx.x & (kWave - 1), G = dm.Hq / dm.Hkv;
  const int cap = (int)kv4_capacity(dm);
  float total = 0.f, tasks = 0.f;  // rough figures will do
  for (int b = lane; b < dm.B; b += kWave) {
    int n = min(min(max(bt.cu[b + 1], 0), bt.T) - min(max(bt.cu[b], 0), bt.T), at.max_new);
    if (n * G > at.most) n = 0;
    float keys = (float)min(max(bt.len[b], 0), cap);
    if (at.window > 0) keys = fminf(keys, (float)at.window + (float)n);
    const float tiles = n > 0 ? ceilf((float)n * G * (1.0f / kAtRows)) : 0.f;
    total += tiles * (keys * (1.0f / kKvTile) + 1.0f);
    tasks += tiles;
  }
  total = wave_sum_dpp(total) * dm.Hkv;
  tasks = wave_sum_dpp(tasks) * dm.Hkv;
  const float room = fmaxf(at_slots<D>() - tasks, at_slots<D>() / 4);
  return max(kMinTiles, (int)fminf(ceilf(total / room), 67108864.0f));
}

// Work item `item` of a call whose sequences have one row tile each: the
// sequences in order, each with its heads and their splits. Returns false past
// the last. Listing only the splits that have keys keeps the workgroups of a
// ragged batch evenly spread: with a grid of all possible splits, most of them
// empty, 128 of 442 waited for a free CU while others idled (49 us, not 33).
struct Item {
  int seq, head, split;
};

__device__ __forceinline__ bool work_item(const Kv4Dims &dm, const Kv4Batch &bt, const Kv4Attn &at, int per,
                                          int splits, int item, Item &it) {
  const int lane = threadIdx.x & (kWave - 1);
  for (int b0 = 0; b0 < dm.B; b0 += kWave) {
    const int b = min(b0 + lane, dm.B - 1);
    const Kv4Span sp = kv4_seq_span(bt, b);
    const int n = min(sp.n, at.max_new);
    const Kv4Range r = kv4_range(dm, sp.first, sp.first + max(n, 1) - 1, sp.len, at.causal, at.window);
    const int used = b0 + lane < dm.B && n > 0 && n * (dm.Hq / dm.Hkv) <= at.most ? kv4_share(r, per, splits, 0).used : 0;
    const int upto = wave_scan(used * dm.Hkv);
    const uint64_t after = __builtin_amdgcn_ballot_w64(upto > item);
    if (after != 0) {
      const int w = __builtin_ctzll(after);
      const int u = __builtin_amdgcn_readlane(used, w);
      const int at_ = item - (__builtin_amdgcn_readlane(upto, w) - u * dm.Hkv);
      it.seq = b0 + w;
      it.head = at_ / u;
      it.split = at_ - it.head * u;
      return true;
    }
    item -= __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  return false;
}

// One row tile of a sequence and head (tile_i of `tiles`), and one split of its keys.
template <int D, int W, bool HALF>
__device__ __forceinline__ void attend_rows(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc,
                                            const Kv4Batch &bt, const Kv4Attn &at, int seq, int head,
                                            int tile_i, int split, int splits, int per,
                                            uint8_t *smem, float (*sm)[kAtRows], float (*sl)[kAtRows],
                                            float *__restrict__ part) {
  constexpr int NG = D / kGroup;
  const RowTile rt = row_tile(dm, bt, at.max_new, tile_i, head, seq, kAtRows);
  if (rt.row0 >= rt.rows || rt.rows > at.most) return;
  const int G = dm.Hq / dm.Hkv;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);

  // the tile's first and last token, and this lane's query row
  const int tok0 = HALF || rt.row0 == 0 ? 0 : rt.row0 / G;
  const int in0 = rt.row0 - tok0 * G;  // head of the first row in its group
  const int col = HALF ? lane & 7 : lane & 15;
  const int row = min(rt.row0 + col, rt.rows - 1) - rt.row0 + in0;
  const bool real = rt.row0 + col < rt.rows;
  const int tok = HALF ? 0 : tok0 + row / G, hd = rt.head * G + (HALF ? row : row % G);
  const int tok1 = HALF ? 0 : __builtin_amdgcn_readlane(tok, 15);
  // its channels, in the order codes8 takes a word's nibbles
  bf16x8_t q[NG][2];
  float qsum[NG];
  const uint16_t *qp = at.q + (rt.sp.begin + tok) * at.q_stride + (long long)hd * D + (lane >> 4) * 16;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 x = *(const uint4 *)(qp + g * kGroup + j * 8);
      sum = sum_bf16x2(x.x, sum_bf16x2(x.y, sum_bf16x2(x.z, sum_bf16x2(x.w, sum))));
      // pairs (0,4) (1,5) (2,6) (3,7)
      const uint4 y = make_uint4((x.x & 0xFFFFu) | (x.z << 16), (x.x >> 16) | (x.z & 0xFFFF0000u),
                                 (x.y & 0xFFFFu) | (x.w << 16), (x.y >> 16) | (x.w & 0xFFFF0000u));
      q[g][j] = __builtin_bit_cast(bf16x8_t, y);
    }
    qsum[g] = sum;
  }
  // keys the first and the last token see: all rows see those from all0 to all1
  // and none sees any outside lo .. hi
  const Kv4Range r0 = kv4_range(dm, rt.sp.first + tok0, rt.sp.first + tok0, rt.sp.len, at.causal, at.window);
  const Kv4Range r1 = kv4_range(dm, rt.sp.first + tok1, rt.sp.first + tok1, rt.sp.len, at.causal, at.window);
  const long long all0 = r1.lo, all1 = r0.hi;
  const Kv4Share share = kv4_share(Kv4Range{r0.lo, r1.hi}, per, splits, split);
  if (split >= share.used) return;

  const int32_t *table =
      bt.table + (bt.rows ? (long long)rt.seq * dm.Hkv + rt.head : (long long)rt.seq) * dm.max_pages;
  uint8_t *ring = smem + wave * kStages * Ring<D>::kStage;
  const uint32_t ring_at = lds_address(ring);
  LaneParts<D> lp = lane_parts<D, HALF>(kc, vc, lane);
  int tile = share.begin + wave;
  const int end = share.end;
  // pages of the tile in use, of the next one and (not loaded yet) of the one after
  TilePages here{}, next{}, after{};
  if (tile < end) {
    const int t1 = min(tile + W, end - 1);
    here = tile_entries(dm, table, tile);
    next = tile_entries(dm, table, t1);
    after = tile_entries(dm, table, min(tile + 2 * W, end - 1));
    here = tile_pages(dm, here, tile);
    next = tile_pages(dm, next, t1);
    load_tile<D>(dm, kc, vc, here, rt.head, tile, ring_at, lp, lane);
    if (tile + W < end) load_tile<D>(dm, kc, vc, next, rt.head, tile + W, ring_at + Ring<D>::kStage, lp, lane);
  }

  // keys this lane's row sees (positions in the table fit 31 bits)
  int t0 = 0, t1 = 0;
  if (real) {
    const Kv4Range mine = kv4_range(dm, rt.sp.first + tok, rt.sp.first + tok, rt.sp.len, at.causal, at.window);
    t0 = (int)(mine.lo < mine.hi ? mine.lo : 0);
    t1 = (int)(mine.lo < mine.hi ? mine.hi : 0);
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) qsum[g] = groups_sum(qsum[g]);
  const bf16x8_t qaff = affine_query<NG>(qsum, lane >> 4);
  const float scale2 = at.scale * kLog2e;  // scores in log2 units
  RowSums<D> a;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
#pragma unroll
    for (int j = 0; j < 4; ++j) a.o[g][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    a.w[g] = a.c[g] = 0.f;
  }
  a.m = kNegInf;
  a.l = 0.f;

  for (int stage = 0; tile < end; tile += W, stage ^= 1) {
    // keeps the compiler from holding every address made of the parts in a register
    asm volatile("" : "+v"(lp.code), "+v"(lp.key), "+v"(lp.value), "+v"(lp.scale));
    // this tile has landed; the next one's loads may still be in flight
    if (tile + W < end)
      MOE_KV_WAIT_VMCNT(Ring<D>::kLoads);
    else
      MOE_KV_WAIT_VMCNT(0);
    asm volatile("" ::: "memory");
    const int key0 = tile * kKvTile;
    const bool masked = key0 < all0 || key0 + (long long)kKvTile > all1 || here.page[0] < 0 || here.page[1] < 0;
    attend_tile<D, HALF>(ring + stage * Ring<D>::kStage, lp, q, qaff, scale2, masked, lane, key0, t0, t1, here, a);
    // every LDS read of this stage is done before the DMA refills it
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    here = next;
    if (tile + 2 * W < end) {
      next = tile_pages(dm, after, tile + 2 * W);
      load_tile<D>(dm, kc, vc, next, rt.head, tile + 2 * W, ring_at + stage * Ring<D>::kStage, lp, lane);
      after = tile_entries(dm, table, min(tile + 3 * W, end - 1));
    }
  }

  // Join the wavefronts: each scales what it has to the workgroup's reference
  // and leaves it in its own ring's place; then the parts are added up, D / 4
  // threads a row.
  a.l = groups_sum(a.l);
  if (lane < kAtRows) {
    sm[wave][lane] = a.m;
    sl[wave][lane] = a.l;
  }
  __syncthreads();
  float m = kNegInf;
#pragma unroll
  for (int w = 0; w < W; ++w)
    m = HALF ? fmaxf(m, fmaxf(sm[w][lane & 7], sm[w][(lane & 7) + 8])) : fmaxf(m, sm[w][lane & 15]);
  const float f = part_weight(a.m, a.l, m, scale2);
  float *so = (float *)ring + (lane & 15) * (D + 4) + 4 * (lane >> 4);
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const float off = groups_sum(fmaf(-24.0f, a.w[g], a.c[g]));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *(float4 *)(so + g * kGroup + 16 * j) =
          make_float4(f * (a.o[g][j][0] + off), f * (a.o[g][j][1] + off), f * (a.o[g][j][2] + off),
                      f * (a.o[g][j][3] + off));
  }
  __syncthreads();
  constexpr int kThreadsRow = D / 4, kParts = HALF ? 2 * W : W;
  for (int r = threadIdx.x / kThreadsRow; r < kAtRows && rt.row0 + r < rt.rows; r += W * kWave / kThreadsRow) {
    const int c = (threadIdx.x % kThreadsRow) * 4;
    float mr = kNegInf, l = 0.f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) mr = fmaxf(mr, sm[i % W][r + i / W * 8]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      const int w = i % W, x_row = r + i / W * 8;
      const float4 x = *(const float4 *)((float *)(smem + w * kStages * Ring<D>::kStage) + x_row * (D + 4) + c);
      o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
      l = fmaf(part_weight(sm[w][x_row], sl[w][x_row], mr, scale2), sl[w][x_row], l);
    }
    if (share.used > 1) {
      const long long pr = part_index(dm, at, rt, r, splits, split);
      *(float4 *)(part + pr * D + c) = o;
      if (c == 0) *(float2 *)(part_stats(dm, bt, at, splits, part) + pr * 2) = make_float2(mr, l);
    } else {
      const int x = r + in0, i = HALF ? 0 : tok0 + x / G, h = rt.head * G + (HALF ? x : x % G);
      store_row(dm, at, rt.sp.begin + i, h, c, l, o);
    }
  }
}

// Grid: x = row tile * splits + split, y = cache head, z = sequence; or, where
// keys are split and a sequence has one row tile (flat), x = work items.
template <int D, int W, bool HALF>
__global__ __launch_bounds__(W *kWave, at_blocks<D>()) void kv4_attention_kernel(Kv4Dims dm, Kv4Plane kc, Kv4Plane vc,
                                                                    Kv4Batch bt, Kv4Attn at, int splits,
                                                                    bool flat, float *__restrict__ part) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ float sm[W][kAtRows], sl[W][kAtRows];
  const int per = splits > 1 && at.per == 0 ? tiles_per_split<D>(dm, bt, at) : at.per;
  int seq = blockIdx.z, head = blockIdx.y, tile_i = blockIdx.x, split = 0;
  if (flat) {
    // there are never more items than workgroups: a task has at most `splits`
    Item it;
    if (!work_item(dm, bt, at, per, splits, blockIdx.x, it)) return;
    seq = it.seq;
    head = it.head;
    split = it.split;
    tile_i = 0;
  } else if (splits > 1) {
    tile_i = blockIdx.x / splits;
    split = blockIdx.x - tile_i * splits;
  }
  attend_rows<D, W, HALF>(dm, kc, vc, bt, at, seq, head, tile_i, split, splits, per, smem, sm, sl, part);
}

// Joins the splits' partial results of a row tile of ROWS. Few splits (C = D): D /
// 4 threads a row, each over all its splits. Many (C = 32): a workgroup for 32
// channels of a row, 32 parts at a time.
template <int D, int C, int ROWS>
__global__ __launch_bounds__(256) void kv4_join_kernel(Kv4Dims dm, Kv4Batch bt, Kv4Attn at, int splits,
                                                       float *__restrict__ part) {
  constexpr int kThreadsRow = C / 4, kGroups = 256 / kThreadsRow;
  constexpr int kParts = C < D ? kGroups : 1, kRows = C < D ? 1 : kGroups, kChunks = D / C;
  static_assert(ROWS % kRows == 0, "a workgroup's rows are of one tile");
  __shared__ float4 so[kParts][kThreadsRow];
  __shared__ float sl[kParts];
  const int tid = threadIdx.x, c = tid % kThreadsRow, group = tid / kThreadsRow;
  const int chunk = blockIdx.x % kChunks, first = blockIdx.x / kChunks * kRows;
  const int tile_i = first / ROWS, r = first - tile_i * ROWS + (C < D ? 0 : group), part_i = C < D ? group : 0;
  const RowTile rt = row_tile(dm, bt, at.max_new, tile_i, blockIdx.y, blockIdx.z, ROWS);
  if (rt.row0 + first - tile_i * ROWS >= rt.rows || rt.rows <= at.above || rt.rows > at.most) return;
  const Kv4Range range = tile_range(dm, rt, ROWS, at.causal, at.window);
  const int per = ROWS != kAtRows ? kPfMinTiles : at.per > 0 ? at.per : tiles_per_split<D>(dm, bt, at);
  const int used = kv4_share(range, per, splits, 0).used;
  if (used <= 1 || rt.row0 + r >= rt.rows) return;
  const float *ml = part_stats(dm, bt, at, splits, part);
  const long long pr0 = part_index(dm, at, rt, r, splits, 0);
  // the row's reference
  float m = kNegInf;
  if constexpr (C < D) {  // every wavefront looks at all the splits'
    for (int s = tid & (kWave - 1); s < used; s += kWave) m = fmaxf(m, ml[(pr0 + s) * 2]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, kWave));
  } else {
    for (int s = 0; s < used; ++s) m = fmaxf(m, ml[(pr0 + s) * 2]);
  }
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = part_i; s < used; s += kParts) {
    const long long pr = pr0 + s;
    const float2 mls = *(const float2 *)(ml + pr * 2);
    const float4 x = *(const float4 *)(part + pr * D + chunk * C + c * 4);
    const float f = part_weight(mls.x, mls.y, m, at.scale * kLog2e);
    l = fmaf(f, mls.y, l);
    o.x = fmaf(f, x.x, o.x), o.y = fmaf(f, x.y, o.y), o.z = fmaf(f, x.z, o.z), o.w = fmaf(f, x.w, o.w);
  }
  if constexpr (kParts > 1) {
    so[part_i][c] = o;
    if (c == 0) sl[part_i] = l;
    __syncthreads();
    if (part_i != 0) return;
#pragma unroll
    for (int i = 1; i < kParts; ++i) {
      const float4 x = so[i][c];
      o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
      l += sl[i];
    }
  }
  const int G = dm.Hq / dm.Hkv, x = rt.row0 + r;
  store_row(dm, at, rt.sp.begin + x / G, rt.head * G + x % G, chunk * C + c * 4, l, o);
}

// Query rows of a sequence and head above which the prefill kernel can take it.
constexpr int kManyRows = 64;

// Row tiles of a sequence and head (an upper bound: it may have fewer new
// tokens), and over all sequences and heads.
static long long kv4_row_tiles(const Kv4Dims &dm, int tokens) {
  const long long rows = (long long)tokens * (dm.Hq / dm.Hkv);
  return (rows + kAtRows - 1) / kAtRows;
}
static long long kv4_tasks(const Kv4Dims &dm, int tokens) {
  return kv4_row_tiles(dm, tokens) * dm.Hkv * dm.B;
}

// Keys a row tile can see (of the table's width: the host does not know the lengths).
static long long kv4_keys(const Kv4Dims &dm, int tokens, int window) {
  const long long keys = kv4_capacity(dm);
  return window > 0 && (long long)window + tokens < keys ? (long long)window + tokens : keys;
}

// The most workgroups a row tile's keys are split over: as many as have
// kMinTiles each, and no more than the card's slots over all tasks, or twice
// that where sequences have one row tile each (work_item() evens those out).
//
// Rows that are sequences each take the same number of workgroups, by the room of their
// tables, and none has to look at the lengths of all (64 tokens of 24 pages of 64 keys,
// 16 heads on 2, D = 256: 19.6 + 4.0 us so, 21.5 + 4.7 by the lengths). That is for tables
// about as wide as the lists: 64 of 2048 keys in tables of 512 pages leave all to one
// workgroup of four (60 us for the whole call, 36 in tables of 32 pages).
static int row_tiles_all(const Kv4Dims &dm) { return (int)((kv4_capacity(dm) + kKvTile - 1) / kKvTile); }
static int few_splits(const Kv4Dims &dm, int tokens, int window, bool rows) {
  const long long tasks = kv4_tasks(dm, tokens);
  const int slots = dm.D == 256 ? at_slots<256>() : dm.D == 128 ? at_slots<128>() : at_slots<64>();
  if (rows) {
    const int all = row_tiles_all(dm);
    const long long n = slots / tasks < all / kMinTilesRows ? slots / tasks : all / kMinTilesRows;
    return n < 1 ? 1 : (int)n;
  }
  const long long most = kv4_keys(dm, tokens, window) / (kKvTile * kMinTiles);
  long long n = (kv4_row_tiles(dm, tokens) == 1 ? 2 : 1) * slots / tasks;
  if (n > most) n = most;
  return n < 1 ? 1 : (int)n;
}

// How a call's sequences are shared between the two kernels.
struct Kv4Plan {
  bool many;       // the prefill kernel takes those with more than kManyRows rows
  int few;         // new tokens a sequence of the row kernel can have; 0: it has none
  int pre_splits, row_splits;
  int room;        // Kv4Attn::room of the row kernel
};

// The prefill kernel reads and rebuilds keys once for 128 rows instead of 16, but
// starts slower and needs rows to fill its tiles. us of the prefill kernel / of
// this one, D = 128, 16 query heads on 2 (and 8 on 8), by new tokens + earlier
// ones: 128 + 0: 14 / 7 (15 / 7), 1024 + 0: 36 / 28 (37 / 19), 2048 + 0: 65 / 70
// (48 / 45), 128 + 8000: 49 / 42 (45 / 28), 512 + 60000: 339 / 778 (215 / 398),
// 1024 + 16000: 244 / 385 (136 / 223); D = 64 and 256 cross over at the same
// products of rows and keys. Below 4096 rows it gains 20% at the most.
static bool kv4_many(const Kv4Dims &dm, int T, long long keys) {
  const long long rows = (long long)T * dm.Hq;
  return rows >= 4096 && rows * keys >= 1ll << 25;
}

static Kv4Plan kv4_plan(const Kv4Dims &dm, int T, int max_new, int window, bool rows) {
  const int G = dm.Hq / dm.Hkv;
  Kv4Plan p{false, max_new, 1, 1, 0};
  const long long keys = kv4_keys(dm, 128 / G, window);
  if ((long long)max_new * G > kManyRows && kv4_many(dm, T, keys)) {
    p.many = true;
    p.few = dm.B == 1 ? 0 : kManyRows / G;
    // enough workgroups for every slot (two a CU, one for D = 256)
    const long long tiles = (long long)T * dm.Hq / 128 + (long long)(dm.B < T ? dm.B : T) * dm.Hkv;
    long long n = ((dm.D == 256 ? 256 : 512) + tiles / 2) / tiles;
    if (n > keys / (kKvTile * kPfMinTiles)) n = keys / (kKvTile * kPfMinTiles);
    p.pre_splits = n < 1 ? 1 : (int)n;
  }
  if (p.few > 0) p.row_splits = few_splits(dm, p.few, window, rows);
  // beside a prompt few of the call's rows are the row kernel's (32768 tokens and one
  // sequence of a single one, 64 heads on 8, D = 128: 12 GB of workspace by row, 6 MB so)
  if ((long long)dm.B * p.few < T) p.room = p.few;
  return p;
}

bool kv4_grid_ok(const Kv4Dims &dm, int max_new) {
  // a launch dimension holds fewer than 2^32 threads: 256 for 16 rows, at the
  // most (splits only multiply small grids)
  return (long long)max_new * (dm.Hq / dm.Hkv) < (1ll << 28) - 128;
}

size_t kv4_attention_ws(const Kv4Dims &dm, int T, int max_new, int window, bool rows) {
  const Kv4Plan p = kv4_plan(dm, T, max_new, window, rows);
  const size_t row = (size_t)dm.Hq * (dm.D + 2) * sizeof(float);  // bytes of a token and split
  const size_t pre = p.pre_splits > 1 ? row * T * p.pre_splits : 0;
  const size_t few = p.row_splits > 1 ? row * p.row_splits * (p.room > 0 ? (size_t)dm.B * p.room : T) : 0;
  return pre > few ? pre : few;
}

template <int D, int W, bool HALF>
static hipError_t launch_rows(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc, const Kv4Batch &bt,
                              const Kv4Attn &at, int tokens, int splits, float *part, hipStream_t s) {
  if constexpr (at_lds_bytes<D, W>() > 64 * 1024) {
    static std::atomic<uint64_t> asked;
    const hipError_t st = allow_lds((const void *)kv4_attention_kernel<D, W, HALF>, at_lds_bytes<D, W>(), asked);
    if (st != hipSuccess) return st;
  }
  const long long tiles = kv4_row_tiles(dm, tokens);
  const bool flat = splits > 1 && tiles == 1 && dm.B <= kEvenMaxB && at.per == 0;
  const dim3 grid = flat ? dim3((unsigned)(kv4_tasks(dm, tokens) * splits))
                         : dim3((unsigned)(tiles * splits), dm.Hkv, dm.B);
  kv4_attention_kernel<D, W, HALF><<<grid, W * kWave, at_lds_bytes<D, W>(), s>>>(dm, kc, vc, bt, at, splits, flat, part);
  return hipGetLastError();
}

template <int D, int ROWS>
static hipError_t launch_join(const Kv4Dims &dm, const Kv4Batch &bt, const Kv4Attn &at, int tokens, int splits,
                              float *part, hipStream_t s) {
  const long long rows = (long long)tokens * (dm.Hq / dm.Hkv);
  const unsigned all = (unsigned)((rows + ROWS - 1) / ROWS * ROWS);
  if (splits > 16)
    kv4_join_kernel<D, 32, ROWS><<<dim3(all * (D / 32), dm.Hkv, dm.B), 256, 0, s>>>(dm, bt, at, splits, part);
  else
    kv4_join_kernel<D, D, ROWS><<<dim3(all / (1024 / D), dm.Hkv, dm.B), 256, 0, s>>>(dm, bt, at, splits, part);
  return hipGetLastError();
}

template <int D>
static hipError_t launch_all(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc, const Kv4Batch &bt,
                             Kv4Attn at, float *part, hipStream_t s) {
  const Kv4Plan p = kv4_plan(dm, bt.T, at.max_new, at.window, bt.rows);
  hipError_t e = hipSuccess;
  if (p.many) {
    at.above = p.few > 0 ? kManyRows : 0;
    at.most = 0x7FFFFFFF;
    at.room = 0;
    e = launch_kv4_prefill(dm, kc, vc, bt, at, p.pre_splits, part, s);
    if (e == hipSuccess && p.pre_splits > 1) e = launch_join<D, 128>(dm, bt, at, at.max_new, p.pre_splits, part, s);
    if (e != hipSuccess || p.few == 0) return e;
  }
  // the partial results of the one above have been read when this one's come
  at.above = 0;
  at.most = p.many ? kManyRows : 0x7FFFFFFF;
  at.room = p.room;
  at.per = bt.rows && p.row_splits > 1 ? (row_tiles_all(dm) + p.row_splits - 1) / p.row_splits : 0;
  // Eight wavefronts where every workgroup has a CU to itself (a short sequence
  // ends sooner), four where there are more of them or keys are split.
  const bool alone = p.row_splits == 1 && kv4_tasks(dm, p.few) <= 256;
  // Rows that are sequences, of 8 heads or fewer: two columns a query row; and from three
  // lists for every wavefront the card holds, a wavefront each, which joins nothing. us of
  // the whole call with four / one, D = 128: 8 heads a list, 32 pages of 32 keys: 112 / 126
  // for 3000 lists, 304 / 286 for 10,000, 543 / 505 for 18,000; 4 heads, 16 pages of 16:
  // 228 / 202 for 12,000; 8 heads, 124 pages of 32: 256 / 337 for 3000, 710 / 701 for 9000.
  const bool half = bt.rows && dm.Hq / dm.Hkv <= kAtRows / 2;
  const bool single = half && p.row_splits == 1 && kv4_tasks(dm, p.few) >= 12ll * at_slots<D>();
  e = single ? launch_rows<D, 1, true>(dm, kc, vc, bt, at, p.few, p.row_splits, part, s)
      : alone ? half ? launch_rows<D, 8, true>(dm, kc, vc, bt, at, p.few, p.row_splits, part, s)
                   : launch_rows<D, 8, false>(dm, kc, vc, bt, at, p.few, p.row_splits, part, s)
      : half ? launch_rows<D, 4, true>(dm, kc, vc, bt, at, p.few, p.row_splits, part, s)
             : launch_rows<D, 4, false>(dm, kc, vc, bt, at, p.few, p.row_splits, part, s);
  if (e == hipSuccess && p.row_splits > 1) e = launch_join<D, kAtRows>(dm, bt, at, p.few, p.row_splits, part, s);
  return e;
}

hipError_t launch_kv4_attention(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc,
                                const Kv4Batch &bt, const Kv4Attn &at, void *ws, hipStream_t s) {
  if (dm.D == 64) return launch_all<64>(dm, kc, vc, bt, at, (float *)ws, s);
  if (dm.D == 128) return launch_all<128>(dm, kc, vc, bt, at, (float *)ws, s);
  return launch_all<256>(dm, kc, vc, bt, at, (float *)ws, s);
}

}  // namespace moe
