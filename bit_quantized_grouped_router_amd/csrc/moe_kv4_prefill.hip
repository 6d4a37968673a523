// Attention over the paged int4-g64 cache for sequences with many query rows
// (prompts): the same sums as moe_kv4_attention.hip, arranged for the matrix
// cores rather than for memory.
//
// One workgroup = 4 wavefronts = 128 query rows of one sequence and cache head,
// 32 to a wavefront; it goes through the keys in tiles of 32. A tile's keys and
// values are rebuilt once for all 128 rows, s * code + b rounded to fp16 in one
// packed FMA, and put into LDS; 32x32x16 MFMAs multiply
//   S^T = K Q^T   (lane: query row l % 32, registers: 16 of the 32 keys)
//   O^T = V^T P^T (lane: query row, registers: channels),
// so that the scores of a row stay in the two lanes (l, l ^ 32) that need them as
// weights, and nothing but the row's maximum and sum ever crosses lanes. The
// value operand is read with the transposing LDS read (4 keys by 16 channels a
// lane group).
//
// A pass of the loop scores tile i + 1 while it turns tile i's scores into
// weights, then multiplies tile i's weights and values while it rebuilds tile i
// + 2, whose codes were loaded a pass before: matrix and vector instructions
// alternate in the order written here (the compiler would put them one after
// the other). One barrier a pass; two buffers of keys, three of values.
//
// fp16 rather than bf16 for the operands: keys, values and weights lose 2^-12 of
// themselves at most instead of 2^-9, so that the result is as exact as its
// own rounding to bf16 (rms error against fp64 1.7e-3 of the result, of which
// the rounding is all; bf16 operands would make it 3.2e-3). Its range is the
// price: where a tile has a value or key of 2^15 or more, or a scale so small
// that codes would fall among fp16's subnormals, or a query is too large or
// too small, or scores pass kMostHalf, the workgroup starts over with bf16
// operands, one tile after the other. That run also takes NaN and infinities: a
// group of values that holds one, or that passes bf16's range at code 0 or 15, is
// replaced by zeros, and the rows that see its key get NaN in the group's
// channels, so that a key no row may look at never reaches one.
//
// Keys are split over workgroups, as in the other kernel, where the row tiles
// do not fill the card (512 tokens behind 60000, 16 heads on 2, D = 128: 1531 us
// unsplit, 308 split eight ways: 821 TFLOP/s).
//
// Measured (us; TFLOP/s of the products that causality leaves), 16 heads on 2:
//   4096 tokens behind 1003   D = 128 147 (696)
//   3000 tokens               D = 64 60 (307)   128 82 (450)
//   4096 tokens               D = 64 79 (435)   128 110 (625)   256 203 (677)
//   8192 tokens               D = 128 329 (836)
//   4096 tokens, values past fp16, D = 128 331
// next to 1224 TFLOP/s of a library product of 8192^3. Bound by the vector
// instructions that a tile needs besides its products (about 150 a wavefront,
// 16 exponentials among them, next to 512 cycles of MFMA; of the SIMDs' time at
// 4096 tokens behind 1003, matrix instructions took 28%, vector ones 42%). Rows of
// 64 to a wavefront halve the rebuilding per row but leave one wavefront a SIMD:
// the same time without a mask (251 us against 254, as first written), longer
// with one (229 against 176).
#include <type_traits>

#include "moe_kv4_device.h"
#include "moe_lds.h"

namespace moe {

constexpr int kPfWaves = 4, kPfRows = 32 * kPfWaves;
// Products whose LDS operands are on their way (D = 64: 103 us, 108 with four of
// them; D = 128: the same).
template <bool HALF, int D>
constexpr int ahead() { return !HALF ? 1 : D == 256 ? 2 : 3; }
// Weights are kept times 2^7: up to 2^15 (the reference lags by kSlack), and off
// by no more than 2^-32 of the largest where fp16 runs out of exponents, so that
// even a million keys in a faint tail lose less than 2^-12 of it together.
constexpr float kShift = 7.0f;
// Scaled scores up to here take one FMA to their distance from the scaled
// reference. That is off by half a step of theirs, 1/2 at most, so weights stay below
// 2^15.5; the same for all of a reference's weights, and taken into account where
// they meet those of another.
constexpr float kMostHalf = 0x1p23f;
constexpr int kSalu = 0x4;  // sched_barrier: scalar instructions may pass

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t kv_lds_s16x4;

template <int D>
struct Pf {
  static constexpr int NG = D / kGroup, NM = D / 32, NK = D / 16;
  static constexpr int kWords = D / 32;        // code words (8 channels) a thread rebuilds
  // A rebuilt row: its 16-byte chunks, those of the four threads that write it
  // next to each other, and one more, so that in all three accesses (sixteen
  // rows' equal chunks, four rows by four threads' chunks, four rows by four
  // chunks of 32 channels) sixteen lanes meet sixteen different chunks of 256 bytes.
  static constexpr int kRow = 2 * D + 16;
  static constexpr __host__ __device__ int place(int chunk) {
    return (chunk / kWords + 4 * (chunk % kWords)) * 16;
  }
  static constexpr int kPlane = kKvTile * kRow;
  // two buffers of keys, three of values: the scores are one tile ahead
  static constexpr int kValues = 2 * kPlane, kLds = 5 * kPlane;
};

// A thread's share of a tile as it lies in the cache: D / 4 channels of one key
// (or value) row.
template <int D>
struct Packed {
  uint32_t c[D / 32];
  uint32_t s, b;  // of this group and the one beside it (16-bit loads take longer)
  bool seen;  // by some row of the workgroup, and of a page that exists
};

// Whether all groups so far can go through fp16: scales stay below 2^10 and
// biases below 2^14, so that values stay below 2^15, and a scale (or, without
// one, a bias) is at least 2^-13: its sixteenth is then exact (8 bits above
// 2^-24) and fp16's smallest step is no more than 2^-11 of it. NaN and infinities
// fail. Bits of the magnitudes are compared; a zero's, less one, are the largest.
struct HalfRange {
  uint32_t hi = 0, lo = ~0u;
  __device__ __forceinline__ void add(uint32_t sb) {
    const uint32_t s = sb & 0x7FFFu, b = (sb >> 16) & 0x7FFFu;
    hi = max(max(hi, s + 0x200u), b);
    lo = min(lo, (s != 0 ? s : b) - 1u);
  }
  __device__ __forceinline__ bool bad() const { return hi >= 0x4680u || lo < 0x38FFu; }
};

// Values of a code word as fp16: those of codes 0 4 1 5, and of 2 6 3 7 from the
// word shifted by 8. Codes become 1024 + q or 1024 + 16 q, exactly, and then one
// packed FMA each.
__device__ __forceinline__ uint2 rebuild_half(uint32_t c, f16x2_t s, f16x2_t s16, f16x2_t b, const DqRegs &k) {
  const f16x2_t off = {(_Float16)1024.0f, (_Float16)1024.0f};
  const f16x2_t h0 = __builtin_bit_cast(f16x2_t, and_or(c, k.m_lo, k.magic)) - off;  // 0, 4
  const f16x2_t h1 = __builtin_bit_cast(f16x2_t, and_or(c, k.m_hi, k.magic)) - off;  // 1, 5 (times 16)
  return make_uint2(__builtin_bit_cast(uint32_t, __builtin_elementwise_fma(h0, s, b)),
                    __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(h1, s16, b)));
}

// The same as bf16.
__device__ __forceinline__ uint4 rebuild_bf16(uint32_t c, float s, float b) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = pack_bf16x2(fmaf(s, (float)((c >> (4 * i)) & 15u), b), fmaf(s, (float)((c >> (4 * i + 16)) & 15u), b));
  return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  f16x2_t v;
  v[0] = (_Float16)a;
  v[1] = (_Float16)b;
  return __builtin_bit_cast(uint32_t, v);
}

template <bool HALF>
__device__ __forceinline__ f32x16_t mfma32(const uint4 &a, const uint4 &b, const f32x16_t &c) {
  if constexpr (HALF)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Whether any thread of the workgroup says so: a barrier, and a scalar branch.
__device__ __forceinline__ bool any_thread(bool x) {
  return __builtin_amdgcn_readfirstlane(__syncthreads_or(x)) != 0;
}

// The tile's rows with fp16 or bf16 operands. False, with nothing written, where
// fp16 will not do; the same for all threads of the workgroup.
template <int D, bool HALF>
__device__ __forceinline__ bool prefill(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc, const Kv4Batch &bt,
                                        const Kv4Attn &at, const RowTile &rt, int split, int splits, float *part,
                                        int thread, uint8_t *smem, uint8_t (*vnan)[4]) {
  using P = Pf<D>;
  constexpr int NG = P::NG, NM = P::NM, NK = P::NK, kAhead = ahead<HALF, D>();
  const int G = dm.Hq / dm.Hkv;
  const int lane = thread & (kWave - 1), half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(thread / kWave);

  // the tile's first and last token, and this lane's query row
  const int tok0 = rt.row0 / G, in0 = rt.row0 - tok0 * G;
  const int last = min(rt.row0 + kPfRows, rt.rows) - 1, tok1 = last / G;
  const int row = rt.row0 + 32 * wave + (lane & 31);
  const bool real = row <= last;
  const int rel = min(row, last) - rt.row0 + in0;
  const int tok = tok0 + rel / G, hd = rt.head * G + rel % G;
  // its channels in the order rebuilt rows have
  const uint16_t *qp = at.q + (rt.sp.begin + tok) * at.q_stride + (long long)hd * D + half * 8;
  uint4 q[NK];
  float most = 0.f;
  bool nan_q = false;
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    const uint4 x = *(const uint4 *)(qp + k * 16);
    uint32_t w[4] = {(x.x & 0xFFFFu) | (x.z << 16), (x.x >> 16) | (x.z & 0xFFFF0000u),
                     (x.y & 0xFFFFu) | (x.w << 16), (x.y >> 16) | (x.w & 0xFFFF0000u)};
    if constexpr (HALF) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xFFFF0000u);
        most = fmaxf(most, fmaxf(fabsf(a), fabsf(b)));
        nan_q |= a != a || b != b;
        w[i] = pack_half(a, b);
      }
    }
    q[k] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if constexpr (HALF) {
    // a row whose largest channel is small would fall among fp16's subnormals
    most = fmaxf(most, __shfl_xor(most, 32, kWave));
    if (any_thread(nan_q || !(most < 32768.0f) || (most < 0x1p-8f && most != 0.f))) return false;
  }

  // keys the first and the last token see, and this lane's row
  const Kv4Range r0 = kv4_range(dm, rt.sp.first + tok0, rt.sp.first + tok0, rt.sp.len, at.causal, at.window);
  const Kv4Range r1 = kv4_range(dm, rt.sp.first + tok1, rt.sp.first + tok1, rt.sp.len, at.causal, at.window);
  const Kv4Range both{r0.lo, r1.hi};
  const Kv4Share share = kv4_share(both, splits > 1 ? kPfMinTiles : 0, splits, split);
  if (split >= share.used) return true;
  const int tiles = share.end - share.begin, first = share.begin;
  const int key_lo = (int)both.lo, key_hi = (int)(tiles > 0 ? both.hi : 0);  // positions fit 31 bits
  int t0 = 0, t1 = 0;
  {
    const Kv4Range mine = kv4_range(dm, rt.sp.first + tok, rt.sp.first + tok, rt.sp.len, at.causal, at.window);
    t0 = (int)(mine.lo < mine.hi ? mine.lo : 0);
    t1 = (int)(mine.lo < mine.hi ? mine.hi : 0);
  }
  const int all0 = (int)r1.lo, all1 = (int)(tiles > 0 && r0.hi > 0 ? r0.hi : 0);  // what every row sees

  // rebuilding: wavefronts 0, 1 take the keys' halves, 2, 3 the values'; four
  // threads a row
  const int32_t *table = bt.table + (long long)rt.seq * dm.max_pages;
  const int hf = wave & 1, plane = wave >> 1, quarter = lane & 3, krow = ((lane >> 4) & 3) | ((lane & 12)), key = 16 * hf + krow;
  const Kv4Plane pl = plane ? vc : kc;
  const DqRegs dk = dq_regs();
  const uint32_t g = (uint32_t)(krow * NG + quarter * NG / 4);  // its group in the half tile
  const bool odd = g & 1;
  auto fetch = [&](int tile, const TilePages &pg, Packed<D> &r) {
    const int t = tile * kKvTile + key, page = hf ? pg.page[1] : pg.page[0];
    const uint64_t row0 = (((uint64_t)(uint32_t)max(page, 0) * (uint32_t)dm.Hkv + rt.head) << dm.page_shift) |
                          (uint32_t)((tile * kKvTile + 16 * hf) & (dm.page - 1));
    const uint8_t *c = pl.codes + row0 * (D / 2) + (uint32_t)(krow * (D / 2) + quarter * (D / 8));
    if constexpr (D == 64) {
      const uint2 x = *(const uint2 *)c;
      r.c[0] = x.x, r.c[1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        const uint4 x = *(const uint4 *)(c + 16 * i);
        r.c[4 * i] = x.x, r.c[4 * i + 1] = x.y, r.c[4 * i + 2] = x.z, r.c[4 * i + 3] = x.w;
      }
    }
    r.s = *(const uint32_t *)(pl.scales + row0 * NG + (g & ~1u));
    r.b = *(const uint32_t *)(pl.biases + row0 * NG + (g & ~1u));
    r.seen = (page | (t - key_lo) | (key_hi - 1 - t)) >= 0;
  };
  // Rebuilding, to buffer kb of the keys, the values' at byte vb: what the groups
  // of a row have in common, and then two steps a code word.
  struct Rebuild {
    uint8_t *row;
    f16x2_t s2, s16, b2;
    float s, b;
    uint2 first;
  };
  auto begin = [&](const Packed<D> &r, int kb, int vb, HalfRange &range) {
    // what no row of the workgroup sees may be anything: it becomes zeros
    const uint32_t pair = odd ? __builtin_amdgcn_perm(r.b, r.s, 0x07060302u) : __builtin_amdgcn_perm(r.b, r.s, 0x05040100u);
    const uint32_t sb = r.seen ? pair : 0u;
    Rebuild c;
    c.row = smem + (plane ? P::kValues + vb : kb * P::kPlane) + key * P::kRow + quarter * 16;
    c.s = bf16_to_f32(sb & 0xFFFFu), c.b = bf16_to_f32(sb >> 16);
    if constexpr (HALF) {
      const _Float16 s = (_Float16)c.s, b = (_Float16)c.b;
      c.s2 = f16x2_t{s, s}, c.b2 = f16x2_t{b, b}, c.s16 = c.s2 * (_Float16)0.0625f;
      range.add(sb);
    } else if (plane == 1) {
      // values run from b to 15 s + b; a scale of 2e37 overflows there though it is finite
      const float end = bf16_to_f32(to_bf16(fmaf(15.0f, c.s, c.b)));
      const bool nan = !(fabsf(c.b) <= 3.402823466e38f) || !(fabsf(end) <= 3.402823466e38f);
      if ((quarter * NG) % 4 == 0) vnan[key][quarter * NG / 4] = nan;
      if (nan) c.s = c.b = 0.f;
    }
    return c;
  };
  auto step = [&](const Packed<D> &r, Rebuild &c, int i) {
    const int w = i / 2;
    if constexpr (HALF) {
      const uint2 y = rebuild_half(i % 2 ? r.c[w] >> 8 : r.c[w], c.s2, c.s16, c.b2, dk);
      if (i % 2)
        *(uint4 *)(c.row + P::place(w)) = make_uint4(c.first.x, c.first.y, y.x, y.y);
      else
        c.first = y;
    } else if (i % 2) {
      *(uint4 *)(c.row + P::place(w)) = rebuild_bf16(r.c[w], c.s, c.b);
    }
  };
  auto convert = [&](const Packed<D> &r, int kb, int vb, HalfRange &range) {
    Rebuild c = begin(r, kb, vb, range);
#pragma unroll
    for (int i = 0; i < 2 * P::kWords; ++i) step(r, c, i);
  };

  const float scale2 = at.scale * kLog2e;  // scores in log2 units
  // Keys: chunk 2 k + half of row l % 32. Values: lane group member j supplies
  // key j / 4 of a step of four, channels 4 (j % 4) .. +3.
  const int vk = 4 * half + ((lane >> 2) & 3);  // + 8 a step
  const uint32_t kbase = (lane & 31) * P::kRow + P::place(half);
  const uint32_t vbase = P::kValues + vk * P::kRow + P::place(2 * ((lane >> 4) & 1) + ((lane >> 1) & 1)) + (lane & 1) * 8;

  // Scores of the tile in key buffer kb; other(k) is what runs beside product k.
  auto scores = [&](int kb, auto other) {
    const uint8_t *st = smem + kb * P::kPlane + kbase;
    f32x16_t s = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    uint4 a[NK];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) a[k] = *(const uint4 *)(st + P::place(2 * k));
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      if (k + kAhead < NK) a[k + kAhead] = *(const uint4 *)(st + P::place(2 * (k + kAhead)));
      s = mfma32<HALF>(a[k], q[k], s);
      other(k);
      __builtin_amdgcn_sched_barrier(kSalu);
    }
    return s;
  };
  // the scores that this lane's row must not see become -infinity
  auto mask = [&](int key0, const TilePages &pg, f32x16_t &s, uint32_t &nan) {
    const bool all = (pg.page[0] | pg.page[1] | (key0 - all0) | (all1 - kKvTile - key0)) >= 0;
    if (__builtin_expect(!all || !HALF, 0)) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {  // register r: key 8 (r / 4) + 4 half + r % 4
        const int k = 8 * (r >> 2) + 4 * half + (r & 3), t = key0 + k;
        const bool seen = pg.page[r >> 3] >= 0 && t >= t0 && t < t1;
        s[r] = seen ? s[r] : kNegInf;
        if (!HALF) nan |= seen ? *(const uint32_t *)vnan[k] : 0u;
      }
    }
  };
  HalfRange range;
  // what a score is scaled and then taken from, as fp16 weights have it
  auto scaled = [&](float m) { return fmaf(m, scale2, -kShift); };
  // moves the reference m where a score exceeds it by too much
  auto rescale = [&](float mx, f32x16_t (&o)[NM], float &m, float &l) {
    if (__builtin_expect(__builtin_amdgcn_ballot_w64((mx - m) * scale2 > kSlack) != 0, 0)) {
      const float mn = fmaxf(m, fmaxf(mx, __shfl_xor(mx, 32, kWave)));
      const float alpha = m == kNegInf ? 0.f : __builtin_amdgcn_exp2f(HALF ? scaled(m) - scaled(mn) : (m - mn) * scale2);
      if (HALF && mn != kNegInf && !(fabsf(mn * scale2) < kMostHalf)) range.hi = ~0u;
#pragma unroll
      for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] *= alpha;
      l *= alpha;
      m = mn;
    }
  };

  // Weights of keys e, e + 1 and their sum. ref: the reference, for fp16 scaled and
  // less kShift.
  auto weigh = [&](const f32x16_t &s, int e, float ref, float &l) {
    const f16x2_t ones = {(_Float16)1.0f, (_Float16)1.0f};
    const float p0 = __builtin_amdgcn_exp2f(HALF ? fmaf(s[e], scale2, -ref) : (s[e] - ref) * scale2);
    const float p1 = __builtin_amdgcn_exp2f(HALF ? fmaf(s[e + 1], scale2, -ref) : (s[e + 1] - ref) * scale2);
    uint32_t w = HALF ? pack_half(p0, p1) : pack_bf16x2(p0, p1);
    if constexpr (HALF) {
      asm volatile("" : "+v"(w));  // in this place, not behind the next branch
      l = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2_t, w), ones, l, false);  // of the rounded weights
    } else {
      l += p0 + p1;
    }
    return w;
  };
  // Value operand of product n: keys 16 (n / NM) + 4 half .. +3 and 8 more, channels 32 (n % NM) + l % 32.
  auto value = [&](int n, int vb) {
    uint2 v[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      v[e] = __builtin_bit_cast(
          uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                     (kv_lds_s16x4 *)(smem + vb + vbase + P::place(4 * (n % NM)) + (16 * (n / NM) + 8 * e) * P::kRow)));
    return make_uint4(v[0].x, v[0].y, v[1].x, v[1].y);
  };
  auto product = [&](int n, const uint4 &v, const uint32_t (&pw)[8], f32x16_t (&o)[NM]) {
    const uint32_t *w = pw + n / NM * 4;
    o[n % NM] = mfma32<HALF>(v, make_uint4(w[0], w[1], w[2], w[3]), o[n % NM]);
  };

  f32x16_t o[NM];
#pragma unroll
  for (int i = 0; i < NM; ++i) o[i] = f32x16_t{0};
  float m = kNegInf, l = 0.f;
  uint32_t nan = 0;  // value groups (a byte each) that are NaN at a key this row sees
  // Page numbers of 32 tiles at a time lie in a register, two lanes a tile:
  // scalar loads would return out of order with LDS reads, so that every tile
  // waited for them. Tile numbers are clamped to the last tile's.
  const int last_page = (key_hi - 1) >> dm.page_shift;
  auto entries = [&](int t) {
    const int p = (first + min(t + (lane >> 1), tiles - 1)) * kKvTile + (lane & 1) * 16;
    return table[min(p >> dm.page_shift, last_page)];
  };
  auto checked = [&](int page) { return kv4_page_ok(dm, page) ? page : -1; };
  auto pages = [&](int now, int t) {
    TilePages pg;
#pragma unroll
    for (int u = 0; u < 2; ++u) pg.page[u] = __builtin_amdgcn_readlane(now, 2 * (t & 31) + u);
    return pg;
  };
  Packed<D> r;
  if (HALF && tiles > 0) {
    // A tile is loaded three tiles ahead of its weights, rebuilt two ahead and
    // scored one ahead; past the last one it is the last that is rebuilt and
    // scored again, rather than branched around.
    auto load = [&](int t, const TilePages &pg) { fetch(first + min(t, tiles - 1), pg, r); };
    int now = checked(entries(0)), later = entries(32);
    TilePages pg1 = pages(now, 0), pg2 = pages(now, 1), pg3 = pages(now, 2);
    load(0, pg1);
    convert(r, 0, 0, range);
    load(1, pg2);
    if (any_thread(range.bad())) return false;  // most caches that need bf16 do so at once
    lds_barrier();
    f32x16_t s0 = scores(0, [](int) {}), s1;
    convert(r, 1, P::kPlane, range);
    load(2, pg3);
    mask(first * kKvTile, pg1, s0, nan);
    float mx = s0[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) mx = fmaxf(mx, s0[e]);
    rescale(mx, o, m, l);
    pg1 = pg2, pg2 = pg3, pg3 = pages(now, 3);
    lds_barrier();
    int vb = 0, wb = 2 * P::kPlane;
    // Tile i, whose scores are s, and the scores sn of tile i + 1.
    auto tile = [&](int i, int kb, const f32x16_t &s, f32x16_t &sn) __attribute__((always_inline)) {
      const float ref = m == kNegInf ? 0.f : scaled(m);
      uint32_t pw[8];
      // the wavefront that scores goes first, its neighbour's rebuilding can wait (4096
      // tokens by 5099 keys without a mask 248 -> 240 us, with one within 2%; D = 64
      // the same, 256 has no neighbour)
      if (D == 128) __builtin_amdgcn_s_setprio(1);
      sn = scores(kb, [&](int k) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e * NK / 8 == k) pw[e] = weigh(s, 2 * e, ref, l);
        asm volatile("" : "+v"(l));
      });
      mask((first + min(i + 1, tiles - 1)) * kKvTile, pg1, sn, nan);
      __builtin_amdgcn_sched_barrier(0);
      if (D == 128) __builtin_amdgcn_s_setprio(0);
      // the products of tile i next to the rebuilding of tile i + 2 and the
      // largest of the new scores
      uint4 v[2 * NM];
#pragma unroll
      for (int n = 0; n < kAhead; ++n) v[n] = value(n, vb);
      Rebuild c = begin(r, kb ^ 1, wb, range);
      mx = kNegInf;
#pragma unroll
      for (int n = 0; n < 2 * NM; ++n) {
        if (n + kAhead < 2 * NM) v[n + kAhead] = value(n + kAhead, vb);
        product(n, v[n], pw, o);
        step(r, c, n);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (e * NM / 8 == n) mx = fmaxf(mx, sn[e]);
        asm volatile("" : "+v"(mx));
        __builtin_amdgcn_sched_barrier(kSalu);
      }
      load(i + 3, pg3);
      if (((i + 4) & 31) == 0) {
        now = checked(later);
        later = entries(i + 36);
      }
      pg1 = pg2, pg2 = pg3, pg3 = pages(now, i + 4);
      rescale(mx, o, m, l);
      vb = vb == 2 * P::kPlane ? 0 : vb + P::kPlane;
      wb = wb == 2 * P::kPlane ? 0 : wb + P::kPlane;
      lds_barrier();
    };
    for (int i = 0;;) {
      tile(i, 1, s0, s1);
      if (++i == tiles) break;
      tile(i, 0, s1, s0);
      if (++i == tiles) break;
    }
  }
  if (!HALF) {  // one tile after the other: with the above twice, registers spill
    int now = 0;
    for (int i = 0; i < tiles; ++i) {
      if ((i & 31) == 0) now = checked(entries(i));
      const TilePages pg = pages(now, i);
      fetch(first + i, pg, r);
      convert(r, 0, 0, range);
      lds_barrier();
      f32x16_t s = scores(0, [](int) {});
      mask((first + i) * kKvTile, pg, s, nan);
      float mx = s[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) mx = fmaxf(mx, s[e]);
      rescale(mx, o, m, l);
      uint32_t pw[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) pw[e] = weigh(s, 2 * e, m == kNegInf ? 0.f : m, l);
#pragma unroll
      for (int n = 0; n < 2 * NM; ++n) {
        product(n, value(n, 0), pw, o);
        __builtin_amdgcn_sched_barrier(0);
      }
      lds_barrier();
    }
  }
  if (HALF && any_thread(range.bad())) return false;
  l += __shfl_xor(l, 32, kWave);
  if (!HALF) nan |= __shfl_xor(nan, 32, kWave);
  // register 4 a + b of tile i: channels 32 i + 8 a + 0 4 1 5 (half 0) or 2 6 3 7
  // (no return from here for rows behind the last: a branch of lanes would have
  // the second attempt's registers beside the first's)
  const bool partial = share.used > 1;
  // parts leave relative to m itself, without kShift and the rounding of scaled(m)
  const float unit = HALF && m != kNegInf ? __builtin_amdgcn_exp2f(-fmaf(m, scale2, -scaled(m))) : 1.0f;
  const float sum_inv = partial ? unit : l == 0.f ? 0.f : 1.0f / l;
  const long long pr = part_index(dm, at, rt, real ? row - rt.row0 : 0, splits, split);
  float *sums = part + pr * D + 2 * half;
  if (partial && real && half == 0) *(float2 *)(part_stats(dm, bt, at, splits, part) + pr * 2) = make_float2(m, l * unit);
  uint16_t *out = at.out + (rt.sp.begin + tok) * at.out_stride + (long long)hd * D + 2 * half;
  if (real) {
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      const float inv = !HALF && ((nan >> (8 * (i / 2))) & 0xFFu) ? __builtin_nanf("") : sum_inv;
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const float c0 = o[i][4 * a] * inv, c1 = o[i][4 * a + 2] * inv;  // channels + 0, 1
        const float c4 = o[i][4 * a + 1] * inv, c5 = o[i][4 * a + 3] * inv;
        if (partial) {
          *(float2 *)(sums + 32 * i + 8 * a) = make_float2(c0, c1);
          *(float2 *)(sums + 32 * i + 8 * a + 4) = make_float2(c4, c5);
        } else {
          *(uint32_t *)(out + 32 * i + 8 * a) = pack_bf16x2(c0, c1);
          *(uint32_t *)(out + 32 * i + 8 * a + 4) = pack_bf16x2(c4, c5);
        }
      }
    }
  }
  return true;
}

// Grid: x = row tile * splits + split, y = cache head, z = sequence. Sequences
// with at most at.above rows are left to the other kernel.
template <int D>
__global__ __launch_bounds__(kPfWaves *kWave, D == 256 ? 1 : 2) void kv4_prefill_kernel(Kv4Dims dm, Kv4Plane kc,
                                                                                      Kv4Plane vc, Kv4Batch bt,
                                                                                      Kv4Attn at, int splits,
                                                                                      float *__restrict__ part) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ __attribute__((aligned(4))) uint8_t vnan[kKvTile][4];  // value groups of a tile that are NaN (bf16)
  // Pairs where two workgroups share a CU and no keys are split (D = 256, one a CU,
  // 4096 tokens: 300 us with pairs, whose second round would come as the shorter
  // tiles of the first end, and 218 without).
  const int x = blockIdx.x / splits, split = blockIdx.x - x * splits;
  const Kv4Place place = kv4_prompt_place(x, blockIdx.y + (long long)gridDim.y * blockIdx.z, gridDim.x / splits,
                                          (long long)gridDim.y * gridDim.z, at.causal, D < 256 && splits == 1);
  const int seq = (int)(place.hs / gridDim.y), head = (int)(place.hs - (long long)seq * gridDim.y);
  const RowTile rt = row_tile(dm, bt, at.max_new, place.tile, head, seq, kPfRows);
  if (rt.row0 >= rt.rows || rt.rows <= at.above) return;
  int thread = threadIdx.x;
  if (prefill<D, true>(dm, kc, vc, bt, at, rt, split, splits, part, thread, smem, vnan)) return;
  asm volatile("" : "+v"(thread));  // nothing of the first attempt is kept in registers for the second
  prefill<D, false>(dm, kc, vc, bt, at, rt, split, splits, part, thread, smem, vnan);
}

template <int D>
static hipError_t launch_prefill(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc, const Kv4Batch &bt,
                                 const Kv4Attn &at, int splits, float *part, hipStream_t s) {
  if constexpr (Pf<D>::kLds >= 64 * 1024) {
    static std::atomic<uint64_t> asked;
    const hipError_t st = allow_lds((const void *)kv4_prefill_kernel<D>, Pf<D>::kLds, asked);
    if (st != hipSuccess) return st;
  }
  const long long rows = (long long)at.max_new * (dm.Hq / dm.Hkv);
  const dim3 grid((unsigned)((rows + kPfRows - 1) / kPfRows * splits), dm.Hkv, dm.B);
  kv4_prefill_kernel<D><<<grid, kPfWaves * kWave, Pf<D>::kLds, s>>>(dm, kc, vc, bt, at, splits, part);
  return hipGetLastError();
}

hipError_t launch_kv4_prefill(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc, const Kv4Batch &bt,
                              const Kv4Attn &at, int splits, float *part, hipStream_t s) {
  if (dm.D == 64) return launch_prefill<64>(dm, kc, vc, bt, at, splits, part, s);
  if (dm.D == 128) return launch_prefill<128>(dm, kc, vc, bt, at, splits, part, s);
  return launch_prefill<256>(dm, kc, vc, bt, at, splits, part, s);
}

}  // namespace moe
