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
//   O^T = V^T P^T contracts over those keys, 8 to a lane, in that same order;
//                 the lane's V operand are the 8 keys' codes of channels
//                 64 g + 4 (l % 16) + j, nibble j of one 16-bit load a key.
// The order of the channels inside a contraction is free, so the nibbles of a
// word are taken in the order 0 4 1 5 2 6 3 7 (one shift and one and-or give
// two of them) and the query is laid out once to match.
#include "moe_device.h"
#include "moe_kv4.h"

namespace moe {

constexpr int kAtWaves = 4;  // wavefronts per workgroup: they share 16 query rows and split the keys
constexpr int kAtRows = 16;  // query rows (token, head of the group) per workgroup

constexpr float kNegInf = -__builtin_huge_valf();

// Scaled log2 units a score may exceed the running reference by before the
// accumulators are rescaled: weights stay below 2^8, far from overflow, and
// the rescale runs once or twice a row instead of at every new maximum.
constexpr float kSlack = 8.0f;

// Two codes of a word, at bits 0..3 and 16..19 of x, as bf16 16 + code.
// Shift: where they sit before (bit 4 i goes to bit 3).
__device__ __forceinline__ uint32_t codes2(uint32_t x, int i) {
  const uint32_t y = i == 0 ? x << 3 : x >> (4 * i - 3);
  return (y & 0x00780078u) | 0x41804180u;
}

__device__ __forceinline__ bf16x8_t codes8(uint32_t c) {
  const uint4 r = make_uint4(codes2(c, 0), codes2(c, 1), codes2(c, 2), codes2(c, 3));
  return __builtin_bit_cast(bf16x8_t, r);
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

// This lane's scales and biases of one 16-key half: 4 keys x NG groups.
template <int NG>
struct HalfScales {
  uint32_t s[2 * NG], b[2 * NG];
};

template <int NG>
__device__ __forceinline__ void load_half_scales(const uint16_t *s, const uint16_t *b, long long at,
                                                 HalfScales<NG> &h) {
  if constexpr (NG == 1) {
    const uint2 x = *(const uint2 *)(s + at), y = *(const uint2 *)(b + at);
    h.s[0] = x.x, h.s[1] = x.y, h.b[0] = y.x, h.b[1] = y.y;
  } else {
#pragma unroll
    for (int i = 0; i < NG / 2; ++i) {
      const uint4 x = *(const uint4 *)(s + at + 8 * i), y = *(const uint4 *)(b + at + 8 * i);
      h.s[4 * i] = x.x, h.s[4 * i + 1] = x.y, h.s[4 * i + 2] = x.z, h.s[4 * i + 3] = x.w;
      h.b[4 * i] = y.x, h.b[4 * i + 1] = y.y, h.b[4 * i + 2] = y.z, h.b[4 * i + 3] = y.w;
    }
  }
}

// Where a 32-key tile lies: the cache rows of its two halves' first keys, and
// whether their pages exist (a half without one is masked and reads page 0).
struct TilePlace {
  long long row[2];
  bool ok[2];
};

__device__ __forceinline__ TilePlace tile_place(const Kv4Dims &dm, const int32_t *__restrict__ table,
                                                int head, int tile) {
  TilePlace p;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const long long t = (long long)tile * kKvTile + 16 * u;
    const bool in = t < kv4_capacity(dm);
    const int page = table[in ? (int)(t >> dm.page_shift) : 0];
    p.ok[u] = in && kv4_page_ok(dm, page);
    p.row[u] = kv4_row(dm, p.ok[u] ? page : 0, head, (int)(t & (dm.page - 1)));
  }
  return p;
}

template <int D>
struct KeyTile {
  static constexpr int NG = D / kGroup;
  uint2 c[2][NG];
  HalfScales<NG> h[2];
};

template <int D>
struct ValueTile {
  static constexpr int NG = D / kGroup;
  uint32_t c[NG][4];  // 16 bits of two keys: (0,1) (2,3) of the first half, then of the second
  HalfScales<NG> h[2];
};

template <int D>
__device__ __forceinline__ void load_keys(const Kv4Plane &pl, const TilePlace &p, int lane,
                                          KeyTile<D> &t) {
  constexpr int NG = D / kGroup;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t *c = pl.codes + p.row[u] * (D / 2);
    const uint32_t at = (lane & 15) * (D / 2) + (lane >> 4) * 8;
#pragma unroll
    for (int g = 0; g < NG; ++g) t.c[u][g] = *(const uint2 *)(c + at + g * 32);
    load_half_scales<NG>(pl.scales + p.row[u] * NG, pl.biases + p.row[u] * NG, (lane >> 4) * 4 * NG,
                         t.h[u]);
  }
}

template <int D>
__device__ __forceinline__ void load_values(const Kv4Plane &pl, const TilePlace &p, int lane,
                                            ValueTile<D> &t) {
  constexpr int NG = D / kGroup;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t *c = pl.codes + p.row[u] * (D / 2);
    const uint32_t at = (lane >> 4) * 4 * (D / 2) + (lane & 15) * 2;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t a = *(const uint16_t *)(c + at + (2 * r) * (D / 2) + g * 32);
        const uint32_t b = *(const uint16_t *)(c + at + (2 * r + 1) * (D / 2) + g * 32);
        t.c[g][2 * u + r] = a | (b << 16);
      }
    load_half_scales<NG>(pl.scales + p.row[u] * NG, pl.biases + p.row[u] * NG, (lane >> 4) * 4 * NG,
                         t.h[u]);
  }
}

// What one wavefront has summed up for its 16 query rows; a lane holds its row
// (column l % 16) and, for each group, channels 64 g + 16 (l / 16) + 4 r + j.
template <int D>
struct RowSums {
  static constexpr int NG = D / kGroup;
  f32x4_t o[NG][4];  // [g][j]: register r
  f32x4_t w[NG];     // sum of the rounded weights p s (every register the same)
  float c[NG];       // sum of p (b + 8 s), this lane's keys only
  float m, l;        // reference maximum (scaled log2 units); sum of p, this lane's keys only
};

// One 32-key tile. MASKED: some row does not see some key (t0 .. t1 - 1 is what
// this lane's row sees) or a page does not exist.
template <int D, bool MASKED>
__device__ __forceinline__ void attend_tile(const KeyTile<D> &kt, const ValueTile<D> &vt,
                                            const bf16x8_t (&q)[D / kGroup][2],
                                            const float (&qsum)[D / kGroup], float scale2,
                                            int lane, long long key0, long long t0, long long t1,
                                            const bool (&ok)[2], RowSums<D> &a) {
  constexpr int NG = D / kGroup;
  float s[8];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes8(kt.c[u][g].x), q[g][0], acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes8(kt.c[u][g].y), q[g][1], acc, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float sc = bf16_at(kt.h[u].s, r * NG + g), bi = bf16_at(kt.h[u].b, r * NG + g);
        x[r] = fmaf(sc, acc[r], fmaf(fmaf(-16.0f, sc, bi), qsum[g], x[r]));
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) s[4 * u + r] = x[r];
  }
  bool seen[8];
  if (MASKED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long t = key0 + (i >> 2) * 16 + (lane >> 4) * 4 + (i & 3);
      seen[i] = ok[i >> 2] && t >= t0 && t < t1;
      s[i] = seen[i] ? s[i] : kNegInf;
    }
  }
  float mx = s[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s[i]);
  mx *= scale2;
  if (__builtin_amdgcn_ballot_w64(mx > a.m + kSlack) != 0) {
    const float m = fmaxf(a.m, groups_max(mx));
    const float alpha = a.m == kNegInf ? 0.f : __builtin_amdgcn_exp2f(a.m - m);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) a.o[g][j][r] *= alpha;
#pragma unroll
      for (int r = 0; r < 4; ++r) a.w[g][r] *= alpha;
      a.c[g] *= alpha;
    }
    a.l *= alpha;
    a.m = m;
  }
  const float ref = a.m == kNegInf ? 0.f : a.m;  // nothing seen yet: every weight is exp2(-inf) = 0
  float p[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p[i] = __builtin_amdgcn_exp2f(fmaf(s[i], scale2, -ref));
    a.l += p[i];
  }
  bf16x8_t ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = (__bf16)1.0f;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    float ps[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const HalfScales<NG> &h = vt.h[i >> 2];
      const float sc = bf16_at(h.s, (i & 3) * NG + g), bi = bf16_at(h.b, (i & 3) * NG + g);
      // a masked slot may hold anything, NaN included: select, never multiply by zero
      ps[i] = !MASKED || seen[i] ? p[i] * sc : 0.f;
      const float mid = fmaf(8.0f, sc, bi);
      a.c[g] = !MASKED || seen[i] ? fmaf(p[i], mid, a.c[g]) : a.c[g];
    }
    const uint4 pw = make_uint4(pack_bf16x2(ps[0], ps[1]), pack_bf16x2(ps[2], ps[3]),
                                pack_bf16x2(ps[4], ps[5]), pack_bf16x2(ps[6], ps[7]));
    const bf16x8_t pb = __builtin_bit_cast(bf16x8_t, pw);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 vw = make_uint4(codes2(vt.c[g][0], j), codes2(vt.c[g][1], j),
                                  codes2(vt.c[g][2], j), codes2(vt.c[g][3], j));
      a.o[g][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, vw), pb,
                                                          a.o[g][j], 0, 0, 0);
    }
    a.w[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, pb, a.w[g], 0, 0, 0);
  }
}

// Query rows of a workgroup: row r of a sequence and cache head is new token
// r / G, head (cache head) * G + r % G.
struct RowTile {
  int seq, head, row0, rows;  // rows: rows of this sequence and head (n * G)
  Kv4Span sp;
};

__device__ __forceinline__ RowTile row_tile(const Kv4Dims &dm, const Kv4Batch &bt, int max_new,
                                            int task) {
  const int G = dm.Hq / dm.Hkv;
  const int tiles = (int)(((long long)max_new * G + kAtRows - 1) / kAtRows);
  RowTile t;
  const int tile = task % tiles;
  task /= tiles;
  t.head = task % dm.Hkv;
  t.seq = task / dm.Hkv;
  t.row0 = tile * kAtRows;
  t.sp = kv4_span(bt.cu[t.seq], bt.cu[t.seq + 1], bt.len[t.seq], bt.T);
  t.rows = min(t.sp.n, max_new) * G;
  return t;
}

// Keys the tile's rows can see.
__device__ __forceinline__ Kv4Range tile_range(const Kv4Dims &dm, const RowTile &t, bool causal,
                                               int window) {
  const int G = dm.Hq / dm.Hkv;
  const int last = min(t.row0 + kAtRows, t.rows) - 1;
  return kv4_range(dm, t.sp.first + t.row0 / G, t.sp.first + last / G, t.sp.len, causal, window);
}

// Adds one part (reference m_i, sum l_i, unnormalised outputs x) to a row's
// total at reference m. A part that saw no key (l_i = 0) is left out; one whose
// scores were all NaN has no reference and passes its NaN on.
__device__ __forceinline__ void join_part(float m_i, float l_i, float m, const float4 &x, float &l,
                                          float4 &o) {
  if (m_i == kNegInf && l_i == 0.f) return;
  const float f = m_i == kNegInf ? 1.f : __builtin_amdgcn_exp2f(m_i - m);
  l = fmaf(f, l_i, l);
  o.x = fmaf(f, x.x, o.x), o.y = fmaf(f, x.y, o.y), o.z = fmaf(f, x.z, o.z), o.w = fmaf(f, x.w, o.w);
}

// Channels c .. c + 3 of row r of a tile, divided by the row's sum; a row that
// saw no key is zero.
__device__ __forceinline__ void store_row(const Kv4Dims &dm, const Kv4Attn &at, const RowTile &rt, int r,
                                          int c, float l, const float4 &o) {
  const int G = dm.Hq / dm.Hkv;
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  const int i = (rt.row0 + r) / G, h = rt.head * G + (rt.row0 + r) % G;
  *(uint2 *)(at.out + (rt.sp.begin + i) * at.out_stride + (long long)h * dm.D + c) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

template <int D>
__global__ __launch_bounds__(kAtWaves *kWave, 2) void kv4_attention_kernel(
    Kv4Dims dm, Kv4Plane kc, Kv4Plane vc, Kv4Batch bt, Kv4Attn at, int splits,
    float *__restrict__ part) {
  constexpr int NG = D / kGroup;
  constexpr int kPad = 4;  // floats between rows in LDS
  constexpr int kJoin = D < 128 ? D : 128;  // channels joined at a time
  __shared__ __attribute__((aligned(16))) float so[kAtWaves][kAtRows][kJoin + kPad];
  __shared__ float sm[kAtWaves][kAtRows], sl[kAtWaves][kAtRows];
  const int task = blockIdx.x / splits, split = blockIdx.x % splits;
  const RowTile rt = row_tile(dm, bt, at.max_new, task);
  if (rt.row0 >= rt.rows) return;
  const Kv4Range range = tile_range(dm, rt, at.causal, at.window);
  const Kv4Share share = kv4_share(range, splits, split);
  if (split >= share.used) return;

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int G = dm.Hq / dm.Hkv;
  const float scale2 = at.scale * 1.4426950408889634f;  // scores in log2 units

  // this lane's query row, its channels in the order codes8 takes a word's nibbles
  const int row = rt.row0 + (lane & 15);
  const bool real = row < rt.rows;
  const int tok = (real ? row : rt.row0) / G, hd = rt.head * G + (real ? row : rt.row0) % G;
  bf16x8_t q[NG][2];
  float qsum[NG];
  {
    const uint16_t *qp = at.q + (rt.sp.begin + tok) * at.q_stride + (long long)hd * D;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 x = *(const uint4 *)(qp + g * kGroup + (2 * (lane >> 4) + j) * 8);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += bf16_at(w, i);
        // pairs (0,4) (1,5) (2,6) (3,7)
        const uint4 y = make_uint4((w[0] & 0xFFFFu) | (w[2] << 16), (w[0] >> 16) | (w[2] & 0xFFFF0000u),
                                   (w[1] & 0xFFFFu) | (w[3] << 16), (w[1] >> 16) | (w[3] & 0xFFFF0000u));
        q[g][j] = __builtin_bit_cast(bf16x8_t, y);
      }
      qsum[g] = groups_sum(sum);
    }
  }
  // keys this lane's row sees
  long long t0 = 0, t1 = 0;
  if (real) {
    const Kv4Range mine = kv4_range(dm, rt.sp.first + tok, rt.sp.first + tok, rt.sp.len, at.causal, at.window);
    t0 = mine.lo;
    t1 = mine.hi;
  }
  // keys every real row sees: tiles inside need no mask
  const int last = min(rt.row0 + kAtRows, rt.rows) - 1;
  const long long all1 = kv4_range(dm, rt.sp.first + rt.row0 / G, rt.sp.first + rt.row0 / G, rt.sp.len,
                                   at.causal, at.window).hi;
  const long long all0 = kv4_range(dm, rt.sp.first + last / G, rt.sp.first + last / G, rt.sp.len,
                                   at.causal, at.window).lo;

  RowSums<D> a;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
#pragma unroll
    for (int j = 0; j < 4; ++j) a.o[g][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    a.w[g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    a.c[g] = 0.f;
  }
  a.m = kNegInf;
  a.l = 0.f;

  const int32_t *table = bt.table + (long long)rt.seq * dm.max_pages;
  int tile = share.begin + wave;
  if (tile < share.end) {
    KeyTile<D> kt;
    ValueTile<D> vt;
    TilePlace here = tile_place(dm, table, rt.head, tile);
    load_keys<D>(kc, here, lane, kt);
    load_values<D>(vc, here, lane, vt);
    for (; tile < share.end; tile += kAtWaves) {
      const long long key0 = (long long)tile * kKvTile;
      const bool full = key0 >= all0 && key0 + kKvTile <= all1 && here.ok[0] && here.ok[1];
      if (full)
        attend_tile<D, false>(kt, vt, q, qsum, scale2, lane, key0, t0, t1, here.ok, a);
      else
        attend_tile<D, true>(kt, vt, q, qsum, scale2, lane, key0, t0, t1, here.ok, a);
      if (tile + kAtWaves < share.end) {
        here = tile_place(dm, table, rt.head, tile + kAtWaves);
        load_keys<D>(kc, here, lane, kt);
        load_values<D>(vc, here, lane, vt);
      }
    }
  }

  // join the wavefronts through LDS, kJoin channels at a time: o, reference and
  // sum of each wavefront's rows, then kThreadsRow threads a row, 4 channels each
  a.l = groups_sum(a.l);
  if (lane < kAtRows) {
    sm[wave][lane] = a.m;
    sl[wave][lane] = a.l;
  }
  constexpr int kThreadsRow = kJoin / 4;
#pragma unroll
  for (int c0 = 0; c0 < D; c0 += kJoin) {
    if (c0 > 0) __syncthreads();
#pragma unroll
    for (int g = c0 / kGroup; g < (c0 + kJoin) / kGroup; ++g) {
      const float sum = groups_sum(a.c[g]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float off = fmaf(-24.0f, a.w[g][r], sum);
        *(float4 *)&so[wave][lane & 15][g * kGroup - c0 + (lane >> 4) * 16 + 4 * r] = make_float4(
            a.o[g][0][r] + off, a.o[g][1][r] + off, a.o[g][2][r] + off, a.o[g][3][r] + off);
      }
    }
    __syncthreads();
    for (int r = threadIdx.x / kThreadsRow; r < kAtRows && rt.row0 + r < rt.rows;
         r += kAtWaves * kWave / kThreadsRow) {
      const int c = (threadIdx.x % kThreadsRow) * 4;
      float m = sm[0][r];
#pragma unroll
      for (int w = 1; w < kAtWaves; ++w) m = fmaxf(m, sm[w][r]);
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kAtWaves; ++w) join_part(sm[w][r], sl[w][r], m, *(const float4 *)&so[w][r][c], l, o);
      if (share.used > 1) {
        // partial [task][split][16][D], then reference and sum [task][split][16][2]
        const long long pr = ((long long)task * splits + split) * kAtRows + r;
        float *ml = part + (long long)gridDim.x * kAtRows * D + pr * 2;
        *(float4 *)(part + pr * D + c0 + c) = o;
        if (c0 + c == 0) {
          ml[0] = m;
          ml[1] = l;
        }
      } else {
        store_row(dm, at, rt, r, c0 + c, l, o);
      }
    }
  }
}

// Joins the splits' partial results: one workgroup per row of a task.
template <int D>
__global__ __launch_bounds__(256) void kv4_join_kernel(Kv4Dims dm, Kv4Batch bt, Kv4Attn at, int splits,
                                                       long long tasks,
                                                       const float *__restrict__ part) {
  constexpr int kThreadsRow = D / 4, kParts = 256 / kThreadsRow;
  __shared__ float4 so[kParts][kThreadsRow];
  __shared__ float sl[kParts];
  const int task = blockIdx.x / kAtRows, r = blockIdx.x % kAtRows;
  const RowTile rt = row_tile(dm, bt, at.max_new, task);
  if (rt.row0 + r >= rt.rows) return;
  const Kv4Range range = tile_range(dm, rt, at.causal, at.window);
  const int used = kv4_share(range, splits, 0).used;
  if (used <= 1) return;
  const float *ml = part + tasks * splits * kAtRows * D;
  const long long pr0 = (long long)task * splits * kAtRows + r;
  // the row's reference: every thread looks at all the splits' (few, and cached)
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  float m = kNegInf;
  for (int s = lane; s < used; s += kWave) m = fmaxf(m, ml[(pr0 + (long long)s * kAtRows) * 2]);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, kWave));
  const int c = tid % kThreadsRow, part_i = tid / kThreadsRow;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = part_i; s < used; s += kParts) {
    const long long pr = pr0 + (long long)s * kAtRows;
    join_part(ml[pr * 2], ml[pr * 2 + 1], m, *(const float4 *)(part + pr * D + c * 4), l, o);
  }
  so[part_i][c] = o;
  if (c == 0) sl[part_i] = l;
  __syncthreads();
  if (part_i == 0) {
#pragma unroll
    for (int i = 1; i < kParts; ++i) {
      const float4 x = so[i][c];
      o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
      l += sl[i];
    }
    store_row(dm, at, rt, r, c * 4, l, o);
  }
}

// Row tiles of a call (an upper bound: a sequence may have fewer new tokens
// than max_new) over all sequences and cache heads.
static long long kv4_tasks(const Kv4Dims &dm, int max_new) {
  const long long rows = (long long)max_new * (dm.Hq / dm.Hkv);
  return (rows + kAtRows - 1) / kAtRows * dm.Hkv * dm.B;
}

// Workgroups to aim for: two per CU fit (their LDS and registers), so this is
// one round of the card's 256 CUs.
constexpr int kTargetBlocks = 512;

int kv4_splits(const Kv4Dims &dm, int max_new, int window) {
  const long long tasks = kv4_tasks(dm, max_new);
  long long keys = kv4_capacity(dm);
  if (window > 0 && (long long)window + max_new < keys) keys = (long long)window + max_new;
  const long long most = (keys + kKvTile * kMinSplitTiles - 1) / (kKvTile * kMinSplitTiles);
  long long n = (kTargetBlocks + tasks - 1) / tasks;
  if (n > most) n = most;
  return n < 1 ? 1 : (int)n;
}

bool kv4_grid_ok(const Kv4Dims &dm, int max_new, int window) {
  return kv4_tasks(dm, max_new) * kAtRows * kv4_splits(dm, max_new, window) < (1ll << 31);
}

size_t kv4_attention_ws(const Kv4Dims &dm, int max_new, int window) {
  const int splits = kv4_splits(dm, max_new, window);
  if (splits == 1) return 0;
  return (size_t)kv4_tasks(dm, max_new) * splits * kAtRows * (dm.D + 2) * sizeof(float);
}

template <int D>
static hipError_t launch(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc, const Kv4Batch &bt,
                         const Kv4Attn &at, float *part, hipStream_t s) {
  const long long tasks = kv4_tasks(dm, at.max_new);
  const int splits = kv4_splits(dm, at.max_new, at.window);
  kv4_attention_kernel<D><<<(int)(tasks * splits), kAtWaves * kWave, 0, s>>>(dm, kc, vc, bt, at, splits, part);
  if (const hipError_t e = hipGetLastError()) return e;
  if (splits > 1)
    kv4_join_kernel<D><<<(int)(tasks * kAtRows), 256, 0, s>>>(dm, bt, at, splits, tasks, part);
  return hipGetLastError();
}

hipError_t launch_kv4_attention(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc,
                                const Kv4Batch &bt, const Kv4Attn &at, void *ws, hipStream_t s) {
  if (dm.D == 64) return launch<64>(dm, kc, vc, bt, at, (float *)ws, s);
  if (dm.D == 128) return launch<128>(dm, kc, vc, bt, at, (float *)ws, s);
  return launch<256>(dm, kc, vc, bt, at, (float *)ws, s);
}

}  // namespace moe
