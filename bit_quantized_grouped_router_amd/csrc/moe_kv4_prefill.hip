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
// lane group). Codes come straight from memory into registers one tile ahead;
// the rebuilt tiles are double buffered, one barrier a tile.
//
// fp16 rather than bf16 for the operands: keys, values and weights lose 2^-12 of
// themselves at most instead of 2^-9, so that the result is as exact as its
// own rounding to bf16 (rms error against fp64 1.7e-3 of the result, of which
// the rounding is all; bf16 operands would make it 3.2e-3). Its range is the
// price: where a tile has a value or key of 2^15 or more, or a scale so small
// that codes would fall among fp16's subnormals, or a query is that large, the
// workgroup starts over with bf16 operands. That run also takes NaN and
// infinities: such values are replaced by zeros, and the rows that see their
// key get NaN in the group's channels, so that a key no row may look at never
// reaches one.
//
// Bound by the vector units: a 32-key tile costs a wavefront about 240 VALU
// operations (16 exponentials at a quarter rate among them) next to 512 cycles
// of MFMA; two workgroups share a CU, so one's softmax runs under the other's
// products.
#include <type_traits>

#include "moe_kv4_device.h"

namespace moe {

constexpr int kPfWaves = 4, kPfRows = 32 * kPfWaves;

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
  uint16_t s, b;
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

// Eight values of a code word as fp16, in the order 0 4 1 5 2 6 3 7: codes as
// 1024 + q or 1024 + 16 q, exactly, then one packed FMA each.
__device__ __forceinline__ uint4 rebuild_half(uint32_t c, f16x2_t s, f16x2_t s16, f16x2_t b, const DqRegs &k) {
  const f16x2_t off = {(_Float16)1024.0f, (_Float16)1024.0f};
  const uint32_t y = c >> 8;
  const f16x2_t h0 = __builtin_bit_cast(f16x2_t, and_or(c, k.m_lo, k.magic)) - off;  // 0, 4
  const f16x2_t h1 = __builtin_bit_cast(f16x2_t, and_or(c, k.m_hi, k.magic)) - off;  // 1, 5 (times 16)
  const f16x2_t h2 = __builtin_bit_cast(f16x2_t, and_or(y, k.m_lo, k.magic)) - off;  // 2, 6
  const f16x2_t h3 = __builtin_bit_cast(f16x2_t, and_or(y, k.m_hi, k.magic)) - off;  // 3, 7 (times 16)
  return make_uint4(__builtin_bit_cast(uint32_t, __builtin_elementwise_fma(h0, s, b)),
                    __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(h1, s16, b)),
                    __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(h2, s, b)),
                    __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(h3, s16, b)));
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

__device__ __forceinline__ uint32_t half_to_bf16x2(uint32_t w) {
  const f16x2_t v = __builtin_bit_cast(f16x2_t, w);
  return pack_bf16x2((float)v[0], (float)v[1]);
}

template <bool HALF>
__device__ __forceinline__ f32x16_t mfma32(const uint4 &a, const uint4 &b, const f32x16_t &c) {
  if constexpr (HALF)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// The row tile of workgroup i of n, for causal calls longest first. Where all
// workgroups are on the card at once (two a CU), every second round of 256 runs
// the other way, so that a long tile shares its CU with a short one.
__device__ __forceinline__ int prefill_tile(int i, int n, bool causal) {
  if (!causal) return i;
  const int heads = gridDim.y * gridDim.z;
  if ((long long)n * heads <= 512) {
    const int linear = i + n * (blockIdx.y + gridDim.y * blockIdx.z);
    if (n <= 256) return (linear >> 8) & 1 ? i : n - 1 - i;
    if (i >= 256) return i - 256;
  }
  return n - 1 - i;
}

// Sequences with at most `few` rows are left to the other kernel.
template <int D>
__global__ __launch_bounds__(kPfWaves *kWave, D == 256 ? 1 : 2) void kv4_prefill_kernel(Kv4Dims dm, Kv4Plane kc,
                                                                                     Kv4Plane vc, Kv4Batch bt,
                                                                                     Kv4Attn at, int few) {
  using P = Pf<D>;
  constexpr int NG = P::NG, NM = P::NM, NK = P::NK;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ __attribute__((aligned(4))) uint8_t vnan[2][kKvTile][4];  // its value groups that are NaN (bf16 run)
  const int tile_i = prefill_tile(blockIdx.x, gridDim.x, at.causal);
  const RowTile rt = row_tile(dm, bt, at.max_new, tile_i, blockIdx.y, blockIdx.z, kPfRows);
  if (rt.row0 >= rt.rows || rt.rows <= few) return;
  const int G = dm.Hq / dm.Hkv;
  const int lane = threadIdx.x & (kWave - 1), half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);

  // the tile's first and last token, and this lane's query row
  const int tok0 = rt.row0 / G, in0 = rt.row0 - tok0 * G;
  const int last = min(rt.row0 + kPfRows, rt.rows) - 1, tok1 = last / G;
  const int row = rt.row0 + 32 * wave + (lane & 31);
  const bool real = row <= last;
  const int rel = min(row, last) - rt.row0 + in0;
  const int tok = tok0 + rel / G, hd = rt.head * G + rel % G;
  // its channels in the order rebuilt rows have, as fp16 unless some query of
  // the workgroup is too large (read twice: cheaper than keeping them meanwhile)
  const uint16_t *qp = at.q + (rt.sp.begin + tok) * at.q_stride + (long long)hd * D + half * 8;
  bool large = false;
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    const uint4 x = *(const uint4 *)(qp + k * 16);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)  // exponent of either half at least 2^15's, NaN and infinities among them
      large |= (w[i] & 0x7FFFu) >= 0x4700u || (w[i] & 0x7FFF0000u) >= 0x47000000u;
  }
  const bool any_large = __syncthreads_or(large);
  uint4 q[NK];
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    const uint4 x = *(const uint4 *)(qp + k * 16);
    uint32_t w[4] = {(x.x & 0xFFFFu) | (x.z << 16), (x.x >> 16) | (x.z & 0xFFFF0000u),
                     (x.y & 0xFFFFu) | (x.w << 16), (x.y >> 16) | (x.w & 0xFFFF0000u)};
    if (!any_large) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack_half(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    q[k] = make_uint4(w[0], w[1], w[2], w[3]);
  }

  // keys the first and the last token see, and this lane's row
  const Kv4Range r0 = kv4_range(dm, rt.sp.first + tok0, rt.sp.first + tok0, rt.sp.len, at.causal, at.window);
  const Kv4Range r1 = kv4_range(dm, rt.sp.first + tok1, rt.sp.first + tok1, rt.sp.len, at.causal, at.window);
  const Kv4Range range{r0.lo, r1.hi};
  const int tiles = kv4_tiles(range), first = (int)(range.lo / kKvTile);
  const int key_lo = (int)range.lo, key_hi = (int)(tiles > 0 ? range.hi : 0);  // positions fit 31 bits
  int t0 = 0, t1 = 0;
  {
    const Kv4Range mine = kv4_range(dm, rt.sp.first + tok, rt.sp.first + tok, rt.sp.len, at.causal, at.window);
    t0 = (int)(mine.lo < mine.hi ? mine.lo : 0);
    t1 = (int)(mine.lo < mine.hi ? mine.hi : 0);
  }
  const int all0 = (int)r1.lo, all1 = (int)(tiles > 0 ? r0.hi : 0);  // what every row sees

  // rebuilding: wavefronts 0, 1 take the keys' halves, 2, 3 the values'; four
  // threads a row
  const int32_t *table = bt.table + (long long)rt.seq * dm.max_pages;
  const int hf = wave & 1, plane = wave >> 1, part = lane & 3, krow = ((lane >> 4) & 3) | ((lane & 12)), key = 16 * hf + krow;
  const Kv4Plane pl = plane ? vc : kc;
  const DqRegs dk = dq_regs();
  auto fetch = [&](int tile, const TilePages &pg, Packed<D> &r) {
    const int t = tile * kKvTile + key, page = hf ? pg.page[1] : pg.page[0];
    const long long row0 = kv4_row(dm, page < 0 ? 0 : page, rt.head, (tile * kKvTile + 16 * hf) & (dm.page - 1));
    const uint8_t *c = pl.codes + row0 * (D / 2) + (uint32_t)(krow * (D / 2) + part * (D / 8));
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
    const uint32_t g = (uint32_t)(krow * NG + part * NG / 4);
    r.s = (pl.scales + row0 * NG)[g];
    r.b = (pl.biases + row0 * NG)[g];
    r.seen = page >= 0 && t >= key_lo && t < key_hi;
  };
  // to buffer kb of the keys, the values' at byte vb
  auto convert = [&](auto half_tag, const Packed<D> &r, int kb, int vb, HalfRange &seen) {
    // what no row of the workgroup sees may be anything: it becomes zeros
    const uint32_t sb = r.seen ? r.s | ((uint32_t)r.b << 16) : 0u;
    const int at_row = (plane ? P::kValues + vb : kb * P::kPlane) + key * P::kRow + part * 16;
    auto slot = [&](int w) { return (uint4 *)(smem + at_row + P::place(w)); };
    if constexpr (decltype(half_tag)::value) {
      const _Float16 s = (_Float16)bf16_to_f32(sb & 0xFFFFu), b = (_Float16)bf16_to_f32(sb >> 16);
      const f16x2_t s2 = {s, s}, b2 = {b, b}, s16 = s2 * (_Float16)0.0625f;
#pragma unroll
      for (int w = 0; w < P::kWords; ++w) *slot(w) = rebuild_half(r.c[w], s2, s16, b2, dk);
      seen.add(sb);
    } else {
      float s = bf16_to_f32(sb & 0xFFFFu), b = bf16_to_f32(sb >> 16);
      if (plane == 1) {
        const bool nan = !(fabsf(s) <= 3.402823466e38f) || !(fabsf(b) <= 3.402823466e38f);
        if ((part * NG) % 4 == 0) vnan[kb][key][part * NG / 4] = nan;
        if (nan) s = b = 0.f;
      }
#pragma unroll
      for (int w = 0; w < P::kWords; ++w) *slot(w) = rebuild_bf16(r.c[w], s, b);
    }
  };

  const float scale2 = at.scale * 1.4426950408889634f;  // scores in log2 units
  // Keys: chunk 2 k + half of row l % 32. Values: lane group member j supplies
  // key j / 4 of a step of four, channels 4 (j % 4) .. +3.
  const int vk = 4 * half + ((lane >> 2) & 3);  // + 8 a step
  const uint32_t kbase = (lane & 31) * P::kRow + P::place(half);
  const uint32_t vbase = P::kValues + vk * P::kRow + P::place(2 * ((lane >> 4) & 1) + ((lane >> 1) & 1)) + (lane & 1) * 8;

  // scores of the tile in key buffer kb
  auto scores = [&](auto half_tag, int kb) {
    constexpr bool HALF = decltype(half_tag)::value;
    const uint8_t *st = smem + kb * P::kPlane;
    f32x16_t s = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      const uint4 a = *(const uint4 *)(st + kbase + P::place(2 * k));
      uint4 b = q[k];
      if constexpr (!HALF) {
        asm volatile("" : "+v"(b.x), "+v"(b.y), "+v"(b.z), "+v"(b.w));  // converted here, not kept
        b.x = any_large ? b.x : half_to_bf16x2(b.x);
        b.y = any_large ? b.y : half_to_bf16x2(b.y);
        b.z = any_large ? b.z : half_to_bf16x2(b.z);
        b.w = any_large ? b.w : half_to_bf16x2(b.w);
      }
      s = mfma32<HALF>(a, b, s);
      if (!HALF) __builtin_amdgcn_sched_barrier(0);
    }
    return s;
  };
  // the scores that this lane's row must not see become -infinity
  auto mask = [&](auto half_tag, int kb, int key0, const TilePages &pg, f32x16_t &s, uint32_t &nan) {
    constexpr bool HALF = decltype(half_tag)::value;
    const bool masked = key0 < all0 || key0 > all1 - kKvTile || (pg.page[0] | pg.page[1]) < 0;
    if (masked || !HALF) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {  // register r: key 8 (r / 4) + 4 half + r % 4
        const int k = 8 * (r >> 2) + 4 * half + (r & 3), t = key0 + k;
        const bool seen = pg.page[r >> 3] >= 0 && t >= t0 && t < t1;
        s[r] = seen ? s[r] : kNegInf;
        if (!HALF) nan |= seen ? *(const uint32_t *)vnan[kb][k] : 0u;
      }
    }
  };
  // moves the reference m where the scores exceed it by too much
  auto rescale = [&](const f32x16_t &s, f32x16_t (&o)[NM], float &m, float &l) {
    float mx = s[0];
#pragma unroll
    for (int r = 1; r < 16; ++r) mx = fmaxf(mx, s[r]);
    mx *= scale2;
    if (__builtin_amdgcn_ballot_w64(mx > m + kSlack) != 0) {
      const float mn = fmaxf(m, fmaxf(mx, __shfl_xor(mx, 32, kWave)));
      const float alpha = m == kNegInf ? 0.f : __builtin_amdgcn_exp2f(m - mn);
#pragma unroll
      for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] *= alpha;
      l *= alpha;
      m = mn;
    }
  };

  // All tiles, and the rows' results; false where a tile asks for bf16.
  auto run = [&](auto half_tag) -> bool {
    constexpr bool HALF = decltype(half_tag)::value;
    f32x16_t o[NM];
#pragma unroll
    for (int i = 0; i < NM; ++i) o[i] = f32x16_t{0};
    float m = kNegInf, l = 0.f;
    HalfRange seen;
    uint32_t nan = 0;  // value groups (a byte each) that are NaN at a key this row sees
    if (tiles > 0) {
      // Tile numbers are clamped to the last one, which is rebuilt, and scored,
      // once or twice too often rather than branched around.
      const int last_page = (key_hi - 1) >> dm.page_shift;
      auto entries = [&](int t) {  // of the page table, not looked at until the tile after
        const int p = (first + min(t, tiles - 1)) * kKvTile;
        TilePages pg;
#pragma unroll
        for (int u = 0; u < 2; ++u)
          pg.page[u] = ((kv_const_i32 *)table)[min((p + 16 * u) >> dm.page_shift, last_page)];
        return pg;
      };
      auto pages = [&](TilePages pg) {
#pragma unroll
        for (int u = 0; u < 2; ++u) pg.page[u] = kv4_page_ok(dm, pg.page[u]) ? pg.page[u] : -1;
        return pg;
      };
      auto load = [&](int t, const TilePages &pg, Packed<D> &r) { fetch(first + min(t, tiles - 1), pg, r); };
      Packed<D> r;
      TilePages pg1 = pages(entries(0)), pg2 = pages(entries(1)), pg3 = pages(entries(2)), pg4 = entries(3);
      load(0, pg1, r);
      convert(half_tag, r, 0, 0, seen);
      load(1, pg2, r);
      if (HALF && __syncthreads_or(seen.bad())) return false;  // most caches that need bf16 do so at once
      lds_barrier();
      f32x16_t s = scores(half_tag, 0);
      convert(half_tag, r, 1, P::kPlane, seen);
      load(2, pg3, r);
      mask(half_tag, 0, first * kKvTile, pg1, s, nan);
      rescale(s, o, m, l);
      pg1 = pg2, pg2 = pg3, pg3 = pages(pg4), pg4 = entries(4);
      lds_barrier();
      int vb = 0, wb = 2 * P::kPlane;
      for (int i = 0; i < tiles; ++i) {
        const int kb = (i + 1) & 1;
        // scores of tile i + 1 next to the weights of tile i
        f32x16_t sn = scores(half_tag, kb);
        if (!HALF || D == 256) __builtin_amdgcn_sched_barrier(0);  // registers
        const float ref = m == kNegInf ? 0.f : m;
        uint32_t pw[8];
        const f16x2_t ones = {(_Float16)1.0f, (_Float16)1.0f};
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float p0 = __builtin_amdgcn_exp2f(fmaf(s[e], scale2, -ref));
          const float p1 = __builtin_amdgcn_exp2f(fmaf(s[e + 1], scale2, -ref));
          if constexpr (HALF) {
            pw[e / 2] = pack_half(p0, p1);  // and the sum is that of the rounded weights
            l = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2_t, pw[e / 2]), ones, l, false);
          } else {
            l += p0 + p1;
            pw[e / 2] = pack_bf16x2(p0, p1);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        // the products of tile i next to the rebuilding of tile i + 2
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 p = make_uint4(pw[4 * j], pw[4 * j + 1], pw[4 * j + 2], pw[4 * j + 3]);
#pragma unroll
          for (int c = 0; c < NM; ++c) {
            // keys 16 j + 4 half .. +3 and 8 more, channels 32 c + l % 32
            uint2 v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
              v[e] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                   (kv_lds_s16x4 *)(smem + vb + vbase + P::place(4 * c) +
                                                                    (16 * j + 8 * e) * P::kRow)));
            o[c] = mfma32<HALF>(make_uint4(v[0].x, v[0].y, v[1].x, v[1].y), p, o[c]);
            if (!HALF) __builtin_amdgcn_sched_barrier(0);
          }
        }
        convert(half_tag, r, i & 1, wb, seen);
        __builtin_amdgcn_sched_barrier(0);
        load(i + 3, pg3, r);
        mask(half_tag, kb, (first + min(i + 1, tiles - 1)) * kKvTile, pg1, sn, nan);
        rescale(sn, o, m, l);
        s = sn;
        pg1 = pg2, pg2 = pg3, pg3 = pages(pg4), pg4 = entries(i + 5);
        vb = vb == 2 * P::kPlane ? 0 : vb + P::kPlane;
        wb = wb == 2 * P::kPlane ? 0 : wb + P::kPlane;
        lds_barrier();
      }
    }
    // register 4 a + b of tile i: channels 32 i + 8 a + 0 4 1 5 (half 0) or 2 6 3 7
    if (HALF && __syncthreads_or(seen.bad())) return false;
    l += __shfl_xor(l, 32, kWave);
    if (!HALF) nan |= __shfl_xor(nan, 32, kWave);
    if (!real) return true;
    const float sum_inv = l == 0.f ? 0.f : 1.0f / l;
    uint16_t *out = at.out + (rt.sp.begin + tok) * at.out_stride + (long long)hd * D + 2 * half;
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      const float inv = !HALF && ((nan >> (8 * (i / 2))) & 0xFFu) ? __builtin_nanf("") : sum_inv;
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        *(uint32_t *)(out + 32 * i + 8 * a) = pack_bf16x2(o[i][4 * a] * inv, o[i][4 * a + 2] * inv);
        *(uint32_t *)(out + 32 * i + 8 * a + 4) = pack_bf16x2(o[i][4 * a + 1] * inv, o[i][4 * a + 3] * inv);
      }
    }
    return true;
  };
  if (!any_large && run(std::true_type{})) return;
  __syncthreads();  // every wavefront has read the flags
  run(std::false_type{});
}

template <int D>
static hipError_t launch_prefill(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc, const Kv4Batch &bt,
                                 const Kv4Attn &at, int few, hipStream_t s) {
  if constexpr (Pf<D>::kLds >= 64 * 1024) {  // needs an opt-in, once per process
    static const hipError_t st = hipFuncSetAttribute(
        (const void *)kv4_prefill_kernel<D>, hipFuncAttributeMaxDynamicSharedMemorySize, Pf<D>::kLds);
    if (st != hipSuccess) return st;
  }
  const long long rows = (long long)at.max_new * (dm.Hq / dm.Hkv);
  const dim3 grid((unsigned)((rows + kPfRows - 1) / kPfRows), dm.Hkv, dm.B);
  kv4_prefill_kernel<D><<<grid, kPfWaves * kWave, Pf<D>::kLds, s>>>(dm, kc, vc, bt, at, few);
  return hipGetLastError();
}

hipError_t launch_kv4_prefill(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc, const Kv4Batch &bt,
                              const Kv4Attn &at, int few, hipStream_t s) {
  if (dm.D == 64) return launch_prefill<64>(dm, kc, vc, bt, at, few, s);
  if (dm.D == 128) return launch_prefill<128>(dm, kc, vc, bt, at, few, s);
  return launch_prefill<256>(dm, kc, vc, bt, at, few, s);
}

}  // namespace moe
