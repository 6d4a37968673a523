// Attention of each new token over the cache pages that a score selects for it.
//
//   bounds   per page, cache head and channel the smallest and largest key lo, hi
//   score    of a page for a token and cache head: sum over the group's query
//            heads and the channels of max(q lo, q hi), the most that any key of
//            the page could score, summed over the heads. With q+ = sum over the
//            heads of max(q, 0) and q- = sum of min(q, 0) it is q- . lo + q+ . hi
//            where all are finite; otherwise it is worked out head by head
//   pages    the first `first`, the last `recent` (the token's own among them)
//            and of the others the `top` with the best scores, ties to the lowest
//   output   softmax attention over the keys of those pages
//
// A page is taken or not by its score in 64 bits, rounded once to fp32, so that the
// choice does not depend on the order of a sum or on what else is in the batch.
// Most pages are far from the border, though: scores are first worked out on the
// matrix cores, q+ and q- cut into three bf16, with a bound of how far off they may
// be, and only the pages within that of the border are scored in 64 bits (on average
// fewer than one a list). All in 64 bits, on the fp64 matrix instruction, took 80 us
// for the scores of 1500 tokens behind 60,000, 16 heads on 2, D = 128, pages of 32.
//
// The selected pages become page tables of their own, one for each token and
// cache head, and the attention kernel for few query rows runs over those.
//
// us of scores + selection + attention (+ join of split keys), 16 heads on 2: one token
// behind 131,149, D = 128, 32 of 2050 pages 5.3 + 8.1 + 7.3 + 3.5; 64 tokens behind up to
// 32,000, D = 256, 24 pages each 12.1 + 10.8 + 19.6 + 4.0; 1500 tokens behind 60,000, D =
// 128, 32 of 1922 pages each 27.9 + 26.8 + 74.3.
#include "moe_kv4_sparse.h"

#include "moe_kv4_device.h"
#include "moe_kv4_write.h"

namespace moe {

// ---- bounds

constexpr int kBoundWaves = 4;

// Pages of new tokens: a workgroup looks at `run` token rows (a lane each, every
// wavefront all of them), and for each that is the first of the call in its page it
// goes over the page's keys, up to the sequence's last. D / 8 lanes take a key, 8
// channels each, and 64 keys are loaded at once. Bound by a chain of four loads
// (offsets, page, codes, and the sums' way through LDS): us 5.6 for 64 single tokens, 2
// heads of 256, pages of 64; 9.0 for all pages of 60,000 tokens, D = 128 (9.6 MB).
template <int D>
__global__ __launch_bounds__(kBoundWaves *kWave) void kv4_bounds_kernel(Kv4Dims dm, Kv4Plane kc, Kv4Batch bt,
                                                                        uint16_t *__restrict__ bounds, int run) {
  constexpr int kLanes = D / 8, kKeys = kWave / kLanes, kLoads = 64 / (kBoundWaves * kKeys);
  __shared__ float part[kBoundWaves][2][D];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const long long row = (long long)blockIdx.x * run + lane;
  const int head = blockIdx.y;
  // the last sequence that begins at or before this lane's row
  int page = -1, keys = 0;
  if (lane < run && row < bt.T) {
    int lo = 0, hi = dm.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (bt.cu[mid] <= row) lo = mid; else hi = mid;
    }
    const Kv4Span sp = kv4_seq_span(bt, lo);
    const long long pos = sp.first + (row - sp.begin);
    if (row >= sp.begin && row < sp.begin + sp.n && pos >= 0 && pos < kv4_capacity(dm)) {
      const int slot = (int)(pos & (dm.page - 1));
      if (slot == 0 || row == sp.begin) {
        const int p = bt.table[(long long)lo * dm.max_pages + (int)(pos >> dm.page_shift)];
        if (kv4_page_ok(dm, p)) page = p;
        const long long left = sp.len - (pos - slot);
        keys = (int)(left < dm.page ? left : dm.page);
      }
    }
  }
  const int at = (lane % kLanes) * 8;
  for (uint64_t todo = __builtin_amdgcn_ballot_w64(page >= 0); todo != 0; todo &= todo - 1) {
    const int w = __builtin_ctzll(todo);
    const int pg = __builtin_amdgcn_readlane(page, w), n = __builtin_amdgcn_readlane(keys, w);
    const long long base = kv4_row(dm, pg, head, 0);
    float mn[8], mx[8];
    uint32_t nan = 0;  // channels that hold one
#pragma unroll
    for (int i = 0; i < 8; ++i) mn[i] = __builtin_huge_valf(), mx[i] = kNegInf;
    for (int k0 = 0; k0 < n; k0 += 64) {
      uint32_t word[kLoads], sb[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        // keys past the last repeat it
        const long long r = base + min(k0 + (u * kBoundWaves + wave) * kKeys + lane / kLanes, n - 1);
        word[u] = *(const uint32_t *)(kc.codes + r * (D / 2) + at / 2);
        const long long g = r * (D / kGroup) + at / kGroup;
        sb[u] = kc.scales[g] | (uint32_t)kc.biases[g] << 16;
      }
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const float s = __uint_as_float(sb[u] << 16), b = __uint_as_float(sb[u] & 0xFFFF0000u);
        float any = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = fmaf(s, (float)((word[u] >> (4 * i)) & 15u), b);
          mn[i] = fminf(mn[i], v);
          mx[i] = fmaxf(mx[i], v);
          any = fmaf(v, 0.f, any);
        }
        if (any != any) {  // an infinity or a NaN
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float v = fmaf(s, (float)((word[u] >> (4 * i)) & 15u), b);
            nan |= (uint32_t)(v != v) << i;
          }
        }
      }
    }
#pragma unroll
    for (int off = kLanes; off < kWave; off *= 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        mn[i] = fminf(mn[i], __shfl_xor(mn[i], off, kWave));
        mx[i] = fmaxf(mx[i], __shfl_xor(mx[i], off, kWave));
      }
      nan |= (uint32_t)__shfl_xor((int)nan, off, kWave);
    }
    if (lane < kLanes) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        part[wave][0][at + i] = nan >> i & 1 ? __uint_as_float(0x7FC00000u) : mn[i];
        part[wave][1][at + i] = mx[i];
      }
    }
    __syncthreads();
    uint16_t *out = bounds + ((long long)pg * dm.Hkv + head) * 2 * D;
    for (int c = threadIdx.x; c < D / 2; c += kBoundWaves * kWave) {
      float lo[2], hi[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        lo[e] = __builtin_huge_valf(), hi[e] = kNegInf;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kBoundWaves; ++i) {
          const float v = part[i][0][2 * c + e];
          bad |= v != v;
          lo[e] = fminf(lo[e], v);
          hi[e] = fmaxf(hi[e], part[i][1][2 * c + e]);
        }
        // adding 0 makes a zero +0
        lo[e] = bad ? __uint_as_float(0x7FC00000u) : lo[e] + 0.f;
        hi[e] = bad ? __uint_as_float(0x7FC00000u) : hi[e] + 0.f;
      }
      *(uint32_t *)(out + 2 * c) = pack_bf16x2(lo[0], lo[1]);
      *(uint32_t *)(out + D + 2 * c) = pack_bf16x2(hi[0], hi[1]);
    }
    __syncthreads();
  }
}

// ---- scores

constexpr int kScoreWaves = 4, kScoreTile = 16;

// The scores of a part of the call, rows row0 .. row0 + rows - 1, as
// order-preserving keys (logit_key; 0: the page does not exist), and for each
// row and head the largest sum of magnitudes that each wavefront saw (as bits; an
// infinity or a NaN where a score may not be finite).
struct ScorePart {
  uint32_t *keys;  // [rows][Hkv][pitch]
  uint32_t *most;  // [rows][Hkv][chunks * kScoreWaves]
  int row0, rows;
  int pitch, chunks, steps;  // a chunk is `steps` tiles of 16 pages for each wavefront
  int tiles;                 // token tiles of a sequence
  void *queries;             // prompts: QueryTile [slots][Hkv]; null otherwise
};

// What a score may be off by, over the sum of its terms' magnitudes, in units of
// 2^-23 (whichever way the matrix cores round): 32 for the fp32 sum of a step's
// products; 2 for the steps' sums, added in pairs; 2 D / 256 <= 2 for those of the
// second part of q and less for the third's; G / 2 for the sum of G heads; 1 for the
// parts' end and the last sums; 4 for the rounding of two scores to fp32, with room to
// spare; 2% for the magnitudes' own sum, of values rounded to 8 bits. And apart from
// that, what is flushed below 2^-126 (score_operand keeps q where its three parts
// are normal numbers).
__device__ __forceinline__ float score_error(int G) { return (48.0f + 0.5f * (float)G) * 0x1p-23f * 1.02f; }
constexpr float kScoreFlushed = 0x1p-55f;

// v as three bf16 that add up to it, NaN where the bound above would not hold.
__device__ __forceinline__ void score_operand(float v, uint16_t (&part)[3]) {
  const uint32_t a = __float_as_uint(v) & 0x7FFFFFFFu;  // 0, or 2^-90 .. 2^60
  if (a != 0 && a - 0x12800000u > 0x5D800000u - 0x12800000u) v = __uint_as_float(0x7FC00000u);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    part[i] = to_bf16(v);
    v -= bf16_to_f32(part[i]);
  }
}

// A token tile's q- and q+ as the matrix instruction takes them: part p of terms 32 m +
// 8 (l / 16) .. + 7 of token l % 16 for lane l in step m, the first half of the steps
// being q-'s.
template <int D>
struct QueryTile {
  static constexpr int kSteps = 2 * D / 32;
  uint4 v[3][kSteps][kWave];
};

// The tile of `tokens` rows from q on (rows of a head, D channels of G heads), by all
// threads, two channels at a time. Columns without a token are left as they are.
template <int D>
__device__ __forceinline__ void fill_queries(QueryTile<D> &t, const uint16_t *rows, long long stride, int tokens, int G) {
  for (int at = threadIdx.x; at < tokens * (D / 2); at += blockDim.x) {
    const int j = at / (D / 2), c2 = at % (D / 2);
    const uint16_t *q = rows + j * stride + c2 * 2;
    float neg[2] = {0.f, 0.f}, pos[2] = {0.f, 0.f};
#pragma unroll 8
    for (int g = 0; g < G; ++g) {
      const uint32_t u = *(const uint32_t *)(q + g * D);
      const float x[2] = {__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u)};
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // a NaN goes to neg, an infinity makes one there
        const float up = fmaxf(x[e], 0.f);
        pos[e] += up;
        neg[e] += x[e] - up;
      }
    }
    uint16_t a[2][3], b[2][3];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      score_operand(neg[e], a[e]);
      score_operand(pos[e], b[e]);
    }
    const int m = c2 / 16, l = (c2 / 4 % 4) * 16 + j;
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      ((uint32_t *)&t.v[p][m][l])[c2 % 4] = a[0][p] | (uint32_t)a[1][p] << 16;
      ((uint32_t *)&t.v[p][D / 32 + m][l])[c2 % 4] = b[0][p] | (uint32_t)b[1][p] << 16;
    }
  }
}

// The bounds of 16 pages as they are loaded: lane l has 16 bytes of each 64 of page l /
// 4, so that four lanes' addresses follow on each other. They change lanes in LDS.
// Which 16 bytes: swapped by l / 16, so that no banks collide there. A page that does
// not exist reads page 0: its scores are not looked at.
template <int D>
__device__ __forceinline__ const uint16_t *page_bounds(const Kv4Dims &dm, const uint16_t *bounds, int entry, int head,
                                                       int lane) {
  return bounds + ((long long)(kv4_page_ok(dm, entry) ? entry : 0) * dm.Hkv + head) * 2 * D +
         ((lane & 3) ^ (lane >> 4)) * 8;
}

// (Copied as a struct, an array of these would go to scratch memory.)
__device__ __forceinline__ uint4 load16(const uint16_t *p) {
  typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
  const u32x4_t v = *(const u32x4_t *)p;
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Where lane l finds terms 8 (l / 16) .. + 7 of page l % 16 among the 64 lanes' loads.
__device__ __forceinline__ int turned_lane(int lane) { return (lane & 15) * 4 + ((lane >> 4) ^ (lane >> 2 & 3)); }

// Sums of a page tile by a token tile: register r is page 4 (l / 16) + r, token l % 16.
struct ScoreSums {
  f32x4_t score, rest[2], most;  // rest: of the second and third parts; most: of magnitudes
};

__device__ __forceinline__ f32x4_t mfma_bf16(const uint4 &a, const uint4 &b, const f32x4_t &c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}

// One step, whose sum of products is returned. q- is negative and q+ is not: with q's
// sign the bounds' magnitudes make all terms positive.
__device__ __forceinline__ f32x4_t score_step(ScoreSums &s, const uint4 &b, const uint4 (&q)[3], bool negative) {
  const uint4 mag = negative ? make_uint4(b.x | 0x80008000u, b.y | 0x80008000u, b.z | 0x80008000u, b.w | 0x80008000u)
                             : make_uint4(b.x & 0x7FFF7FFFu, b.y & 0x7FFF7FFFu, b.z & 0x7FFF7FFFu, b.w & 0x7FFF7FFFu);
  s.most = mfma_bf16(mag, q[0], s.most);
  s.rest[0] = mfma_bf16(b, q[1], s.rest[0]);
  s.rest[1] = mfma_bf16(b, q[2], s.rest[1]);
  return mfma_bf16(b, q[0], f32x4_t{0.f, 0.f, 0.f, 0.f});
}

// Keys of the tile's pages cb .. cb + 15 for this lane's token (out: its keys; null: none),
// and the largest sum of magnitudes so far. valid: bit BIT i, page i exists.
template <int BIT>
__device__ __forceinline__ void put_scores(const ScoreSums &s, uint64_t valid, int lane, uint32_t *out, uint32_t &most) {
  const uint32_t mine = (uint32_t)(valid >> (4 * BIT * (lane >> 4)));
  uint32_t key[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const bool there = mine >> (BIT * r) & 1;
    const uint32_t k = logit_key(s.score[r] + (s.rest[0][r] + s.rest[1][r]));
    key[r] = there ? k : 0u;
    most = max(most, there ? __float_as_uint(s.most[r]) & 0x7FFFFFFFu : 0u);
  }
  if (out != nullptr) *(uint4 *)(out + 4 * (lane >> 4)) = make_uint4(key[0], key[1], key[2], key[3]);
}

// The token tile and the pages c0 .. c0 + span - 1 of a workgroup.
struct ScoreTile {
  Kv4Span sp;
  Kv4Scored sc;  // of the tile's last token
  int i0, last;  // its tokens in the sequence
};

// False where there is nothing to score. kTokens: of a workgroup.
template <int kTokens>
__device__ __forceinline__ bool score_tile(const Kv4Dims &dm, const Kv4Batch &bt, const Kv4Select &sel,
                                           const ScorePart &part, int seq, int tile, int c0, int span, ScoreTile &t) {
  t.sp = kv4_seq_span(bt, seq);
  const int n = min(t.sp.n, sel.max_new);
  t.i0 = tile * kTokens;
  t.last = min(t.i0 + kTokens, n) - 1;
  if (t.i0 >= n || t.sp.begin + t.last < part.row0 || t.sp.begin + t.i0 >= part.row0 + part.rows) return false;
  t.sc = kv4_scored(dm, t.sp.first + t.last, sel.first, sel.recent);
  return c0 <= t.sc.hi && c0 + span > t.sc.lo;
}

// Few tokens a sequence. Grid: x = sequence, y = cache head, z = token tile + tiles *
// chunk of pages (chunks that shorter sequences do not have come last: 64 sequences of
// up to 32,000 tokens, D = 256, 24 us with them in between, 12.6 without). 16 pages by
// 16 tokens a wavefront at a time; as a chunk of four loads goes to LDS to change
// lanes, the next tile's takes its registers. Bound by the chain offsets - table -
// bounds.
template <int D>
__device__ __forceinline__ void score_pages(const Kv4Dims &dm, const Kv4Batch &bt, const Kv4Select &sel,
                                            const ScorePart &part, int chunk, int tile, QueryTile<D> &sq,
                                            uint4 (&turned)[kScoreWaves][4][kWave]) {
  constexpr int kSteps = QueryTile<D>::kSteps;
  const int head = blockIdx.y, seq = blockIdx.x;
  const int span = part.steps * kScoreWaves * kScoreTile, c0 = chunk * span;
  ScoreTile t;
  if (!score_tile<kScoreTile>(dm, bt, sel, part, seq, tile, c0, span, t)) return;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int G = dm.Hq / dm.Hkv;
  const int32_t *table = bt.table + (long long)seq * dm.max_pages;
  // this lane's page in the wavefront's tile st (hi is inside the table)
  const auto entry_of = [&](int st) {
    const int c = c0 + (st * kScoreWaves + wave) * kScoreTile + (lane >> 2);
    return st < part.steps && c <= t.sc.hi ? table[c] : -1;
  };
  int entry = entry_of(0), next_entry = entry_of(1);
  uint4 raw[kSteps];
  const uint16_t *page = page_bounds<D>(dm, sel.bounds, entry, head, lane);
#pragma unroll
  for (int m = 0; m < kSteps; ++m) raw[m] = load16(page + m * 32);
  fill_queries<D>(sq, sel.q + (long long)(t.sp.begin + t.i0) * sel.q_stride + (long long)head * G * D, sel.q_stride,
                  t.last - t.i0 + 1, G);
  __syncthreads();

  const int j = lane & 15;
  const int row = t.sp.begin + t.i0 + j - part.row0;
  const bool mine = t.i0 + j <= t.last && row >= 0 && row < part.rows;
  const long long item = (long long)row * dm.Hkv + head;
  uint32_t most = 0;
  for (int st = 0; st < part.steps; ++st) {
    const int cb = c0 + (st * kScoreWaves + wave) * kScoreTile;
    if (cb > t.sc.hi) break;
    const uint64_t valid = __builtin_amdgcn_ballot_w64(kv4_page_ok(dm, entry));
    entry = next_entry;
    page = page_bounds<D>(dm, sel.bounds, entry, head, lane);
    next_entry = entry_of(st + 2);
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    ScoreSums s{zero, {zero, zero}, zero};
    f32x4_t four[kSteps / 4];
#pragma unroll
    for (int k = 0; k < kSteps / 4; ++k) {
      wave_lds_sync();  // what was there has been read
#pragma unroll
      for (int i = 0; i < 4; ++i) turned[wave][i][lane] = raw[4 * k + i];
      wave_lds_sync();
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[4 * k + i] = load16(page + (4 * k + i) * 32);
      f32x4_t one[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = 4 * k + i;
        const uint4 q[3] = {sq.v[0][m][lane], sq.v[1][m][lane], sq.v[2][m][lane]};
        one[i] = score_step(s, turned[wave][i][turned_lane(lane)], q, m < kSteps / 2);
      }
      four[k] = (one[0] + one[1]) + (one[2] + one[3]);
    }
    s.score = four[0];
    if constexpr (kSteps == 8) s.score = four[0] + four[1];
    if constexpr (kSteps == 16) s.score = (four[0] + four[1]) + (four[2] + four[3]);
    put_scores<4>(s, valid, lane, mine ? part.keys + item * part.pitch + cb : nullptr, most);
  }
  most = max(most, (uint32_t)__shfl_xor((int)most, 16, kWave));
  most = max(most, (uint32_t)__shfl_xor((int)most, 32, kWave));
  if (mine && lane < 16) part.most[item * part.chunks * kScoreWaves + chunk * kScoreWaves + wave] = most;
}

template <int D>
__global__ __launch_bounds__(kScoreWaves *kWave) void kv4_score_kernel(Kv4Dims dm, Kv4Batch bt, Kv4Select sel,
                                                                       ScorePart part) {
  __shared__ QueryTile<D> sq;
  __shared__ uint4 turned[kScoreWaves][4][kWave];
  const long long all = (long long)part.tiles * part.chunks;
  for (long long z = blockIdx.z; z < all; z += gridDim.z) {
    const int chunk = (int)(z / part.tiles);
    score_pages<D>(dm, bt, sel, part, chunk, (int)(z - (long long)chunk * part.tiles), sq, turned);
    if (z + gridDim.z < all) __syncthreads();  // the queries have been read
  }
}

// Prompts: the token tiles' operands are worked out once, for all pages, and lie in
// memory; tile `tile` of a sequence in slot query_slot.
__device__ __forceinline__ long long query_slot(const Kv4Span &sp, const ScorePart &part, int seq, int tile) {
  return (long long)(sp.begin >> 4) + tile + seq - (part.row0 >> 4) + 2;
}

template <int D>
__global__ __launch_bounds__(1024) void kv4_query_kernel(Kv4Dims dm, Kv4Batch bt, Kv4Select sel, ScorePart part) {
  __shared__ QueryTile<D> sq;
  const int head = blockIdx.y, seq = blockIdx.z, tile = blockIdx.x, G = dm.Hq / dm.Hkv;
  ScoreTile t;
  if (!score_tile<kScoreTile>(dm, bt, sel, part, seq, tile, 0, 0x7FFFFFFF, t)) return;
  uint4 *all = &sq.v[0][0][0];
  constexpr int kAll = sizeof(sq) / 16;
  if (t.last - t.i0 + 1 < kScoreTile) {  // columns without a token
    for (int i = threadIdx.x; i < kAll; i += blockDim.x) all[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  fill_queries<D>(sq, sel.q + (long long)(t.sp.begin + t.i0) * sel.q_stride + (long long)head * G * D, sel.q_stride,
                  t.last - t.i0 + 1, G);
  __syncthreads();
  uint4 *out = (uint4 *)part.queries + (query_slot(t.sp, part, seq, tile) * dm.Hkv + head) * kAll;
  for (int i = threadIdx.x; i < kAll; i += blockDim.x) out[i] = all[i];
}

// 64 pages by 64 tokens a workgroup at a time: each wavefront loads 16 of the pages
// and has 16 of the tokens, whose operands stay in registers. Grid: x = token tile of 64
// * chunks + chunk of pages, y = cache head, z = sequence.
template <int D>
__global__ __launch_bounds__(kScoreWaves *kWave) void kv4_score_prompt_kernel(Kv4Dims dm, Kv4Batch bt, Kv4Select sel,
                                                                              ScorePart part) {
  constexpr int kSteps = QueryTile<D>::kSteps, kTokens = kScoreWaves * kScoreTile;
  __shared__ uint4 turned[kScoreWaves][kSteps][kWave];
  const int head = blockIdx.y, seq = blockIdx.z;
  const int tile = blockIdx.x / part.chunks, chunk = blockIdx.x - tile * part.chunks;
  const int span = part.steps * kScoreWaves * kScoreTile, c0 = chunk * span;
  ScoreTile t;
  if (!score_tile<kTokens>(dm, bt, sel, part, seq, tile, c0, span, t)) return;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int32_t *table = bt.table + (long long)seq * dm.max_pages;
  const auto entry_of = [&](int st) {
    const int c = c0 + (st * kScoreWaves + wave) * kScoreTile + (lane >> 2);
    return st < part.steps && c <= t.sc.hi ? table[c] : -1;
  };
  const auto entry_at = [&](int st) {  // lane's page of the 64
    const int c = c0 + st * kScoreWaves * kScoreTile + lane;
    return st < part.steps && c <= t.sc.hi ? table[c] : -1;
  };
  int all_entry = entry_at(0);
  int next_entry = entry_of(1);
  uint4 raw[kSteps];
  const uint16_t *page = page_bounds<D>(dm, sel.bounds, entry_of(0), head, lane);
#pragma unroll
  for (int m = 0; m < kSteps; ++m) raw[m] = load16(page + m * 32);
  // this wavefront's tokens; a tile without any takes the first one's operands and stores nothing
  const int i0 = t.i0 + wave * kScoreTile, j = lane & 15;
  const int at = i0 <= t.last && t.sp.begin + min(i0 + kScoreTile - 1, t.last) >= part.row0 &&
                         t.sp.begin + i0 < part.row0 + part.rows ? tile * kScoreWaves + wave : -1;
  uint4 q[kSteps][3];
  {
    // some tile of the workgroup is inside the part: its last token is not before it, its first not behind
    const int inside = at >= 0 ? at : max(tile * kScoreWaves, (part.row0 - t.sp.begin) >> 4);
    const QueryTile<D> *qt = (const QueryTile<D> *)part.queries + query_slot(t.sp, part, seq, inside) * dm.Hkv + head;
#pragma unroll
    for (int m = 0; m < kSteps; ++m)
#pragma unroll
      for (int p = 0; p < 3; ++p) q[m][p] = qt->v[p][m][lane];
  }
  const int row = t.sp.begin + i0 + j - part.row0;
  const bool mine = at >= 0 && i0 + j <= t.last && row >= 0 && row < part.rows;
  const long long item = (long long)row * dm.Hkv + head;
  uint32_t most = 0;
  for (int st = 0; st < part.steps; ++st) {
    const int cb = c0 + st * kScoreWaves * kScoreTile;
    if (cb > t.sc.hi) break;
    const uint64_t valid = __builtin_amdgcn_ballot_w64(kv4_page_ok(dm, all_entry));  // of the 64 pages
    lds_barrier();  // the tiles before have been read
#pragma unroll
    for (int m = 0; m < kSteps; ++m) turned[wave][m][lane] = raw[m];
    lds_barrier();
    page = page_bounds<D>(dm, sel.bounds, next_entry, head, lane);
#pragma unroll
    for (int m = 0; m < kSteps; ++m) raw[m] = load16(page + m * 32);
    next_entry = entry_of(st + 2);
    all_entry = entry_at(st + 1);
#pragma unroll  // not a loop: hipcc would wait for the loads above before it
    for (int w = 0; w < kScoreWaves; ++w) {
      if (cb + w * kScoreTile > t.sc.hi) break;
      const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
      ScoreSums s{zero, {zero, zero}, zero};
      f32x4_t four[kSteps / 4];
#pragma unroll
      for (int k = 0; k < kSteps / 4; ++k) {
        f32x4_t one[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = 4 * k + i;
          one[i] = score_step(s, turned[w][m][turned_lane(lane)], q[m], m < kSteps / 2);
        }
        four[k] = (one[0] + one[1]) + (one[2] + one[3]);
      }
      s.score = four[0];
      if constexpr (kSteps == 8) s.score = four[0] + four[1];
      if constexpr (kSteps == 16) s.score = (four[0] + four[1]) + (four[2] + four[3]);
      put_scores<1>(s, valid >> (16 * w), lane, mine ? part.keys + item * part.pitch + cb + w * kScoreTile : nullptr, most);
    }
  }
  most = max(most, (uint32_t)__shfl_xor((int)most, 16, kWave));
  most = max(most, (uint32_t)__shfl_xor((int)most, 32, kWave));
  if (mine && lane < 16)
    *(uint4 *)(part.most + (item * part.chunks + chunk) * kScoreWaves) = make_uint4(most, most, most, most);
}

// ---- selection

constexpr int kSelectMostWaves = 16;
constexpr uint32_t kTaken = 0xFFFFFFFFu;  // key of a page that is taken whatever the others are

// Sum over the first 16 lanes (the others hold 0), wave-uniform.
__device__ __forceinline__ int first16_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0xb1, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x4e, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x140, 0xf, 0xf, false);
  return __builtin_amdgcn_readfirstlane(v);
}

// What the selection leaves for the attention.
struct SelectOut {
  int32_t *table;  // [rows][Hkv][width]
  int32_t *len;    // [rows]
  int width;       // no list is longer
};

// v plus the value a DPP lane pattern brings in (see wave_sum_dpp).
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_add64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROW_MASK, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROW_MASK, 0xf, false);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// A lane's 64-bit terms of a page's score, summed, as the score's key; wave-uniform.
__device__ __forceinline__ uint32_t score_key(double s) {
  s = dpp_add64<0xb1, 0xf>(s);
  s = dpp_add64<0x4e, 0xf>(s);
  s = dpp_add64<0x141, 0xf>(s);
  s = dpp_add64<0x140, 0xf>(s);
  s = dpp_add64<0x142, 0xa>(s);
  s = dpp_add64<0x143, 0xc>(s);
  return __builtin_amdgcn_readlane(logit_key((float)s), kWave - 1);
}

// True (wave-uniform) where one of n words of two bf16 holds an infinity or a NaN.
__device__ __forceinline__ bool any_not_finite(const uint32_t *words, int n, int lane) {
  bool any = false;
  for (int i = lane; i < n; i += kWave)
    any |= (words[i] & 0x7F80u) == 0x7F80u || (words[i] & 0x7F800000u) == 0x7F800000u;
  return __builtin_amdgcn_ballot_w64(any) != 0;
}

// A wavefront's terms of a page's score in 64 bits: lane l has D / 32 channels, of
// the smallest keys in the lower half, of the largest in the upper.
template <int D>
struct ExactScore {
  static constexpr int N = D / 32;
  double q[N];

  // N bf16 from p on, as 32-bit words.
  __device__ __forceinline__ static void words(const uint16_t *p, uint32_t (&w)[N / 2]) {
    if constexpr (N == 2) {
      w[0] = *(const uint32_t *)p;
    } else if constexpr (N == 4) {
      const uint2 x = *(const uint2 *)p;
      w[0] = x.x, w[1] = x.y;
    } else {
      const uint4 x = *(const uint4 *)p;
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    }
  }

  // From the queries of G heads in LDS.
  __device__ __forceinline__ void load(const uint16_t *queries, int G, int lane) {
#pragma unroll
    for (int e = 0; e < N; ++e) q[e] = 0.0;
    for (int g = 0; g < G; ++g) {
      uint32_t w[N / 2];
      words(queries + g * D + (lane & 31) * N, w);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float x = (e & 1) ? __uint_as_float(w[e / 2] & 0xFFFF0000u) : __uint_as_float(w[e / 2] << 16);
        q[e] += (lane < 32 ? x >= 0.f : x <= 0.f) ? 0.0 : (double)x;
      }
    }
  }

  // The score's key, of a page's words; wave-uniform.
  __device__ __forceinline__ uint32_t key(const uint32_t (&w)[N / 2]) const {
    double s = 0.0;
#pragma unroll
    for (int e = 0; e < N; ++e)
      s = fma((double)((e & 1) ? __uint_as_float(w[e / 2] & 0xFFFF0000u) : __uint_as_float(w[e / 2] << 16)), q[e], s);
    return score_key(s);
  }

  // The same by the formula itself: an infinite bound counts where it is the larger product
  // only, and 0 times it is NaN, neither of which q- . lo + q+ . hi knows.
  __device__ __forceinline__ static uint32_t by_heads(const uint16_t *page, const uint16_t *queries, int G, int lane) {
    double s = 0.0;
    for (int c = lane; c < D; c += kWave) {
      const double lo = bf16_to_f32(page[c]), hi = bf16_to_f32(page[D + c]);
      for (int g = 0; g < G; ++g) {
        const double x = bf16_to_f32(queries[g * D + c]), a = x * lo, b = x * hi;
        s += a != a || a > b ? a : b;  // NaN where either is
      }
    }
    return score_key(s);
  }
};

// One workgroup for a token and cache head. A page that is always taken has the
// largest key, one that does not exist 0. The key of the last one taken, but for its
// last 8 bits or fewer, is found 8 bits at a time from the first bit on in which keys
// differ, with counts in LDS. Pages above those bits and their error are taken, those below are not, and if
// that leaves a choice the ones between are scored again in 64 bits: up to 64 are
// ranked at once, for more the search is repeated to the last bit. Then each wavefront
// lists what it takes of its own pages.
// Bound by latency (three rounds of loads, then barriers) for few lists, by vector
// instructions for many. R: pages of a lane, their keys and places held in registers,
// so that a workgroup of W wavefronts takes 64 R W pages; 0: any number, read each
// time from the scores.
template <int D, int R>
__global__ __launch_bounds__(kSelectMostWaves *kWave) void kv4_select_kernel(Kv4Dims dm, Kv4Batch bt, Kv4Select sel,
                                                                             ScorePart part, SelectOut out) {
  extern __shared__ __attribute__((aligned(16))) uint4 queries[];  // the heads' D channels
  __shared__ __attribute__((aligned(16))) uint32_t hist[256];
  __shared__ uint32_t found[2];
  __shared__ int listed, list_page[kWave], list_place[kWave];
  __shared__ uint32_t list_key[kWave];
  __shared__ __attribute__((aligned(16))) uint4 shared[kSelectMostWaves];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), waves = blockDim.x / kWave;
  const int r = blockIdx.x, tok = part.row0 + r, head = blockIdx.y, G = dm.Hq / dm.Hkv;
  int seq;
  long long pos;
  bool here = find_token(dm, bt, tok, &seq, &pos);
  if (here) here = tok - kv4_seq_span(bt, seq).begin < sel.max_new;
  if (!here) {
    if (head == 0 && threadIdx.x == 0) out.len[r] = -1;
    return;
  }
  const Kv4Scored sc = kv4_scored(dm, pos, sel.first, sel.recent);
  const int pages = sc.own + 1;
  const int32_t *table = bt.table + (long long)seq * dm.max_pages;
  const long long item = (long long)r * dm.Hkv + head;
  uint32_t *keys = part.keys + item * part.pitch;
  // this wavefront's pages begin .. end - 1, a multiple of 64 but for the last
  const int seg = R > 0 ? R * kWave : ((pages + waves - 1) / waves + kWave - 1) / kWave * kWave;
  const int begin = min(wave * seg, pages), end = min(begin + seg, pages);

  const auto first_key = [&](int c, int entry) -> uint32_t {
    if (c >= end) return 0u;
    if (c >= sc.lo && c <= sc.hi) return sel.top > 0 ? keys[c] : 0u;
    return kv4_page_ok(dm, entry) ? kTaken : 0u;
  };
  uint32_t held[R > 0 ? R : 1];
  int place[R > 0 ? R : 1];
  if constexpr (R > 0) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = begin + i * kWave + lane;
      place[i] = c < end ? table[c] : -1;
      held[i] = first_key(c, place[i]);
    }
  }
  uint32_t most = 0;  // the largest sum of magnitudes of the scored pages
  if (sel.top > 0) {
    // in case scores have to be worked out again
    const uint16_t *q = sel.q + tok * sel.q_stride + (long long)head * G * D;
    for (int i = threadIdx.x; i < G * (D / 8); i += blockDim.x) queries[i] = *(const uint4 *)(q + i * 8);
    if (sc.hi >= sc.lo) {
      const int span = part.steps * kScoreWaves * kScoreTile;
      const uint32_t *m = part.most + item * part.chunks * kScoreWaves;
      for (int i = sc.lo / span * kScoreWaves + lane; i < (sc.hi / span + 1) * kScoreWaves; i += kWave)
        most = max(most, m[i]);
    }
  }
  // f(page, its place, key) for this wavefront's pages, 64 at a time; keys past its last are 0
  const auto each = [&](auto &&f) {
    if constexpr (R > 0) {
#pragma unroll
      for (int i = 0; i < R; ++i) f(begin + i * kWave + lane, place[i], held[i]);
    } else {
      for (int c0 = begin; c0 < end; c0 += kWave) {
        const int c = c0 + lane, entry = c < end ? table[c] : -1;
        uint32_t k = first_key(c, entry);
        f(c, entry, k);
      }
    }
  };
  const auto count_of = [](bool b) { return (int)__builtin_popcountll(__builtin_amdgcn_ballot_w64(b)); };

  // pages there are, those always taken, and the range of the others' keys
  int all = 0, certain = 0;
  uint32_t hi = 0, lo = 0xFFFFFFFFu;
  const auto range = [&]() {
    all = certain = 0;
    hi = 0;
    lo = 0xFFFFFFFFu;
    each([&](int, int, uint32_t k) {
      all += count_of(k != 0);
      certain += count_of(k == kTaken);
      hi = max(hi, k == kTaken ? 0u : k);
      lo = min(lo, k == 0 ? 0xFFFFFFFFu : k);
    });
    hi = wave_max_u32(hi);
    lo = wave_max_u32(~lo);
    __syncthreads();  // what was there has been read
    if (lane == 0) shared[wave] = make_uint4(all, certain, hi, lo);
    for (int i = threadIdx.x; i < 256; i += blockDim.x) hist[i] = 0;
    if (threadIdx.x == 0) listed = 0;
    __syncthreads();
    const uint4 x = lane < waves ? shared[lane] : make_uint4(0, 0, 0, 0);
    all = first16_sum((int)x.x);
    certain = first16_sum((int)x.y);
    hi = wave_max_u32(x.z);
    lo = ~wave_max_u32(x.w);
  };
  range();
  const int want = sel.top + certain;

  // taken: keys above `least`, and the first `ties` of those equal to it
  uint32_t least = 0;
  int ties = 0;
  // The left-th largest key that is not kTaken: its `prefix` but for the last `rest` bits or
  // fewer, and how many of the keys that share it are among the left largest.
  uint32_t prefix;
  int left, bits;
  const auto search = [&](int rest) {
    left = want - certain;
    // one bit at least, which spares a choice that hipcc 7.2 compiles to a vector
    // compare and a scalar select on another condition
    bits = 32 - __builtin_clz((hi ^ lo) | 1u);
    prefix = 0;  // of all keys up to that bit
    bool first = true;
    do {
      const int take = min(bits, 8), shift = bits - take;
      const uint32_t mask = (1u << take) - 1;
      each([&](int, int, uint32_t k) {
        if (k - 1 < kTaken - 1 && (first || k >> bits == prefix)) atomicAdd(&hist[k >> shift & mask], 1u);
      });
      __syncthreads();
      if (wave == 0) {
        // lane l: digits 255 - 4 l down to 252 - 4 l
        const uint4 x = *(const uint4 *)&hist[252 - 4 * lane];
        const uint32_t h[4] = {x.w, x.z, x.y, x.x}, sum = x.x + x.y + x.z + x.w;
        uint32_t before = (uint32_t)wave_scan((int)sum) - sum;
        if (before < (uint32_t)left && before + sum >= (uint32_t)left) {
          int i = 0;
#pragma unroll
          for (int k = 0; k < 3; ++k)
            if (i == k && before + h[k] < (uint32_t)left) before += h[k], ++i;
          found[0] = 255 - 4 * lane - i;
          found[1] = before;
        }
        *(uint4 *)&hist[252 - 4 * lane] = make_uint4(0, 0, 0, 0);
      }
      __syncthreads();
      // the digits above the first one looked at are the largest key's
      if (first) prefix = bits < 32 ? hi >> bits : 0u;
      prefix = prefix << take | __builtin_amdgcn_readfirstlane(found[0]);
      left -= (int)__builtin_amdgcn_readfirstlane(found[1]);
      bits = shift;
      first = false;
    } while (bits > rest);
  };

  int more = 0, same = 0;  // of this wavefront: keys above least, and equal to it
  bool counted = false;
  if (want == 0) {
    least = kTaken;
  } else if (all > want) {
    search(8);
    most = wave_max_u32(most);
    const float off = 2.0f * (score_error(G) * __uint_as_float(most) + kScoreFlushed);
    // the keys of border + off and border - off, rounded away; all scored pages where sums may not be finite
    const float top = key_logit(prefix << bits | ((1u << bits) - 1)), bottom = key_logit(prefix << bits);
    const float x = top + off, y = bottom - off;
    uint32_t above = logit_key(x * (1.0f + (x > 0.f ? 0x1p-22f : -0x1p-22f)));
    uint32_t below = logit_key(y * (1.0f - (y > 0.f ? 0x1p-22f : -0x1p-22f)));
    if (most >= 0x7E800000u) above = kTaken - 1, below = 1;  // 2^126: sums may overflow
    int sure = 0, near = 0;
    each([&](int, int, uint32_t k) {
      sure += count_of(k > above);
      near += count_of(k >= below && k <= above);
    });
    more = sure + near;
    __syncthreads();
    if (lane == 0) shared[wave] = make_uint4(sure, near, 0, 0);
    __syncthreads();
    const uint4 n = lane < waves ? shared[lane] : make_uint4(0, 0, 0, 0);
    sure = first16_sum((int)n.x);
    near = first16_sum((int)n.y);
    if (sure + near == want) {
      least = below - 1;
      counted = true;
    } else {
      ExactScore<D> score;
      uint32_t words[D / 64];
      // an infinity or a NaN among the bounds or queries shows in the sums of magnitudes
      const bool wild = most >= 0x7F800000u;
      const bool odd = wild && any_not_finite((const uint32_t *)queries, G * D / 2, lane);
      const auto exact = [&](const uint16_t *page) {
        if (wild && (odd || any_not_finite((const uint32_t *)page, D, lane)))
          return score.by_heads(page, (const uint16_t *)queries, G, lane);
        return score.key(words);
      };
      if (near <= kWave) {
        each([&](int c, int entry, uint32_t k) {
          if (k >= below && k <= above) {
            const int i = atomicAdd(&listed, 1);
            list_page[i] = c;
            list_place[i] = entry;  // it has a key, so it exists
          }
        });
        __syncthreads();
        for (int i = wave; i < near; i += waves) {
          const uint16_t *page =
              sel.bounds + ((long long)__builtin_amdgcn_readfirstlane(list_place[i]) * dm.Hkv + head) * 2 * D;
          score.words(page + lane * (D / 32), words);
          if (i == wave) score.load((const uint16_t *)queries, G, lane);
          const uint32_t k = exact(page);
          if (lane == 0) list_key[i] = k;
        }
        __syncthreads();
        const uint32_t lk = lane < near ? list_key[lane] : 0u;
        const int lc = lane < near ? list_page[lane] : 0;
        // how many of the listed come before lane's
        int rank = 0;
        for (int i = 0; i < near; ++i) {
          const uint32_t k = __builtin_amdgcn_readlane(lk, i);
          const int c = __builtin_amdgcn_readlane(lc, i);
          rank += k > lk || (k == lk && c < lc);
        }
        const uint64_t taken = __builtin_amdgcn_ballot_w64(lane < near && rank < want - sure);
        each([&](int c, int, uint32_t &k) {
          bool take = k > above;
          for (uint64_t todo = taken; todo != 0; todo &= todo - 1)
            take |= c == __builtin_amdgcn_readlane(lc, __builtin_ctzll(todo));
          k = take ? kTaken : 0u;
          if constexpr (R == 0) {
            if (c < end && c >= sc.lo && c <= sc.hi) keys[c] = k;
          }
        });
      } else {
        score.load((const uint16_t *)queries, G, lane);
        each([&](int c, int entry, uint32_t &k) {
          uint64_t todo = __builtin_amdgcn_ballot_w64(k >= below && k <= above);
          k = k > above ? kTaken : 0u;
          while (todo != 0) {
            const int w = __builtin_ctzll(todo);
            todo &= todo - 1;
            const uint16_t *page =
                sel.bounds + ((long long)__builtin_amdgcn_readlane(entry, w) * dm.Hkv + head) * 2 * D;
            score.words(page + lane * (D / 32), words);
            const uint32_t e = exact(page);
            k = lane == w ? e : k;
          }
          if constexpr (R == 0) {
            if (c < end && c >= sc.lo && c <= sc.hi) keys[c] = k;
          }
        });
        range();
        search(0);
        least = prefix;
        ties = left;
      }
    }
  }

  if (!counted) {
    more = same = 0;
    each([&](int, int, uint32_t k) {
      more += count_of(k > least);
      same += count_of(k != 0 && k == least);
    });
  }
  __syncthreads();
  if (lane == 0) shared[wave] = make_uint4(more, same, 0, 0);
  __syncthreads();
  // of all wavefronts up to lane's: keys equal to least, and taken
  const uint4 n = lane < waves ? shared[lane] : make_uint4(0, 0, 0, 0);
  const int seen_upto = wave_scan((int)n.y);
  const int at_upto = wave_scan((int)n.x + min((int)n.y, max(ties - (seen_upto - (int)n.y), 0)));
  int seen = wave > 0 ? __builtin_amdgcn_readlane(seen_upto, wave > 0 ? wave - 1 : 0) : 0;  // ties before this one's
  int at = wave > 0 ? __builtin_amdgcn_readlane(at_upto, wave > 0 ? wave - 1 : 0) : 0;      // its first place
  const int total = __builtin_amdgcn_readlane(at_upto, kWave - 1);
  const long long row = item * out.width;
  const int size = sel.top + sel.first + sel.recent;
  int32_t *blocks = sel.blocks == nullptr ? nullptr : sel.blocks + ((long long)tok * dm.Hkv + head) * size;
  const uint64_t lower = (1ull << lane) - 1;
  each([&](int c, int entry, uint32_t k) {
    const bool tie = k != 0 && k == least;
    const uint64_t tied = __builtin_amdgcn_ballot_w64(tie);
    const bool take = k > least || (tie && seen + __builtin_popcountll(tied & lower) < ties);
    const uint64_t taken = __builtin_amdgcn_ballot_w64(take);
    const int to = at + __builtin_popcountll(taken & lower);
    if (take && to < out.width) {
      out.table[row + to] = entry;
      if (blocks != nullptr) blocks[to] = c;
    }
    at += __builtin_popcountll(taken);
    seen += __builtin_popcountll(tied);
  });
  if (blocks != nullptr)
    for (int i = total + threadIdx.x; i < size; i += blockDim.x) blocks[i] = -1;
  if (head == 0 && threadIdx.x == 0) {
    // whole pages, but for the token's own, which ends with it (and is the last)
    const long long cap = kv4_capacity(dm);
    const bool cut = sc.own >= 0 && pos < cap && kv4_page_ok(dm, table[sc.own]);
    out.len[r] = (total << dm.page_shift) - (cut ? dm.page - 1 - (int)(pos & (dm.page - 1)) : 0);
  }
}

// ---- launchers

// Workspace of a call: for a part of its rows the score keys, the page lists and
// their lengths, and what the attention over them needs.
struct SparseWs {
  int rows;  // of a part
  int pitch, chunks, steps, tiles;  // of the scores
  bool prompt;
  size_t keys, most, queries, table, len, attention, bytes;
};

// Score keys of a part, while it has more than one row (its lists are no wider); prompts'
// query operands have up to the same again.
constexpr size_t kPartBytes = 256u << 20;

static size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Pages that a list has room for: no more are taken than the sequence's table holds.
static int list_width(const Kv4Dims &dm, const Kv4Select &sel) {
  const int size = sel.top + sel.first + sel.recent;
  return size < dm.max_pages ? size : dm.max_pages;
}

static Kv4Dims selected_dims(const Kv4Dims &dm, int rows, int width) {
  Kv4Dims d = dm;
  d.B = rows;
  d.max_pages = width;
  return d;
}

static SparseWs sparse_ws(const Kv4Dims &dm, int T, const Kv4Select &sel) {
  SparseWs w;
  const int width = list_width(dm, sel);
  w.pitch = (dm.max_pages + kScoreTile - 1) / kScoreTile * kScoreTile;
  // The prompt's kernels need 64 tokens a sequence and rows for its token tiles (us for
  // the scores of 1500 tokens behind 60,000, D = 128: 5.3 + 22.9 us with, 39 without).
  const size_t slot = (size_t)dm.Hkv * 3 * 2 * dm.D * 16 * 2;
  w.prompt = sel.top > 0 && sel.max_new >= 64 && sel.max_new <= 1 << 20 && (long long)dm.B * 16 <= T &&
             dm.B * slot <= kPartBytes / 2;
  const int tokens = w.prompt ? kScoreWaves * kScoreTile : kScoreTile;
  w.tiles = (int)(((long long)sel.max_new + tokens - 1) / tokens);
  // a workgroup's tokens are brought to it once for all its pages: no more workgroups
  // than the card holds at once (two a CU)
  const long long all = (w.pitch + kScoreWaves * kScoreTile - 1) / (kScoreWaves * kScoreTile);
  long long steps = ((long long)w.tiles * dm.B * dm.Hkv * all + 511) / 512;
  if (!w.prompt && steps > 16) steps = 16;
  if (steps > all) steps = all;
  if (steps < 1) steps = 1;
  while (w.prompt && steps < all && w.tiles * ((all + steps - 1) / steps) >= 1 << 24) steps *= 2;  // a grid's x
  w.steps = (int)steps;
  w.chunks = (int)((all + steps - 1) / steps);
  const size_t row = (size_t)dm.Hkv * w.pitch * 4;
  size_t rows = kPartBytes / row;
  if (rows > 32768) rows = 32768;
  if (w.prompt && rows > kPartBytes / 2 / (slot / 16)) rows = kPartBytes / 2 / (slot / 16);
  if (rows < 1) rows = 1;
  w.rows = rows < (size_t)T ? (int)rows : T;
  const size_t full = kv4_attention_ws(selected_dims(dm, w.rows, width), w.rows, 1, 0, true);
  const int rest = T % w.rows;
  const size_t last = rest ? kv4_attention_ws(selected_dims(dm, rest, width), rest, 1, 0, true) : 0;
  w.keys = 0;
  w.most = align256(w.keys + w.rows * row);
  w.queries = align256(w.most + (size_t)w.rows * dm.Hkv * w.chunks * kScoreWaves * 4);
  w.table = align256(w.queries + (w.prompt ? slot * (w.rows / 16 + 4 + dm.B) : 0));
  w.len = align256(w.table + (size_t)w.rows * dm.Hkv * width * 4);
  w.attention = align256(w.len + (size_t)w.rows * 4);
  w.bytes = w.attention + (full > last ? full : last);
  return w;
}

size_t kv4_sparse_ws(const Kv4Dims &dm, int T, const Kv4Select &sel) { return sparse_ws(dm, T, sel).bytes; }

template <int D>
static hipError_t launch_score(const Kv4Dims &dm, const Kv4Batch &bt, const Kv4Select &sel, const ScorePart &part,
                               hipStream_t s) {
  if (part.queries == nullptr) {
    const long long z = (long long)part.tiles * part.chunks;
    kv4_score_kernel<D><<<dim3(dm.B, dm.Hkv, z < 65535 ? (unsigned)z : 65535), kScoreWaves * kWave, 0, s>>>(dm, bt, sel,
                                                                                                            part);
    return hipGetLastError();
  }
  const int tiles = (sel.max_new + kScoreTile - 1) / kScoreTile;
  kv4_query_kernel<D><<<dim3(tiles, dm.Hkv, dm.B), 1024, 0, s>>>(dm, bt, sel, part);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  kv4_score_prompt_kernel<D><<<dim3(part.tiles * part.chunks, dm.Hkv, dm.B), kScoreWaves * kWave, 0, s>>>(dm, bt, sel,
                                                                                                          part);
  return hipGetLastError();
}

template <int D>
static hipError_t launch_selection(const Kv4Dims &dm, const Kv4Batch &bt, const Kv4Select &sel, const ScorePart &part,
                                   const SelectOut &so, hipStream_t s) {
  if (sel.top > 0) {
    const hipError_t e = launch_score<D>(dm, bt, sel, part, s);
    if (e != hipSuccess) return e;
  }
  // Few lists: two pages a lane of as many wavefronts as that takes, for the shortest
  // chain. Many: eight a lane of a quarter as many wavefronts, for fewer barriers. us with
  // two / eight, D = 128: tables of 2000 pages 6.8 / 7.7 for 2 lists, 10.9 / 12.7 for 256,
  // 16.8 / 12.6 for 400, 22.7 / 14.0 for 640, 82 / 30 for 3000. (Of 512 pages, four
  // wavefronts either way, two stays ahead: 9.4 / 12.5 for 400, 18.2 / 26.6 for 3000.) With
  // eight / any number: 4000 pages 9.0 / 12.2 for 2 lists, 25 / 60 for 1024; 8000 pages
  // 12.3 / 19.8 and 51 / 95.
  const long long lists = (long long)part.rows * dm.Hkv;
  const int per = dm.max_pages <= 2 * kSelectMostWaves * kWave && lists < 512 ? 2
                  : dm.max_pages <= 8 * kSelectMostWaves * kWave              ? 8
                                                                              : 0;
  auto *select = per == 2 ? kv4_select_kernel<D, 2> : per == 8 ? kv4_select_kernel<D, 8> : kv4_select_kernel<D, 0>;
  int waves = per > 0 ? (dm.max_pages + per * kWave - 1) / (per * kWave) : kSelectMostWaves;
  if (waves < 4) waves = 4;
  const int queries = sel.top > 0 ? dm.Hq / dm.Hkv * D * 2 : 0;
  select<<<dim3(part.rows, dm.Hkv), waves * kWave, queries, s>>>(dm, bt, sel, part, so);
  return hipGetLastError();
}

hipError_t launch_kv4_sparse(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc, const Kv4Batch &bt,
                             const Kv4Select &sel, uint16_t *out, long long out_stride, float scale, void *ws,
                             hipStream_t s) {
  const int width = list_width(dm, sel);
  const SparseWs w = sparse_ws(dm, bt.T, sel);
  const SelectOut so{(int32_t *)((char *)ws + w.table), (int32_t *)((char *)ws + w.len), width};
  for (int row0 = 0; row0 < bt.T; row0 += w.rows) {
    const ScorePart part{(uint32_t *)((char *)ws + w.keys), (uint32_t *)((char *)ws + w.most), row0,
                         bt.T - row0 < w.rows ? bt.T - row0 : w.rows, w.pitch, w.chunks, w.steps, w.tiles,
                         w.prompt ? (char *)ws + w.queries : nullptr};
    hipError_t e = dm.D == 64    ? launch_selection<64>(dm, bt, sel, part, so, s)
                   : dm.D == 128 ? launch_selection<128>(dm, bt, sel, part, so, s)
                                 : launch_selection<256>(dm, bt, sel, part, so, s);
    if (e != hipSuccess) return e;
    const Kv4Batch rows{so.table, nullptr, so.len, part.rows, true};
    const Kv4Attn at{sel.q + (long long)row0 * sel.q_stride, out + (long long)row0 * out_stride, sel.q_stride,
                     out_stride, 1, scale, false, 0, 0, 0, 0, 0};
    e = launch_kv4_attention(selected_dims(dm, part.rows, width), kc, vc, rows, at, (char *)ws + w.attention, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_kv4_bounds(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Batch &bt, uint16_t *bounds,
                             hipStream_t s) {
  // rows a workgroup looks at: one while the card holds that many workgroups
  int run = 1;
  while (run < kWave && (long long)bt.T * dm.Hkv / run > 2048) run *= 2;
  const dim3 grid((unsigned)(((long long)bt.T + run - 1) / run), dm.Hkv);
  auto *kernel = dm.D == 64 ? kv4_bounds_kernel<64> : dm.D == 128 ? kv4_bounds_kernel<128> : kv4_bounds_kernel<256>;
  kernel<<<grid, kBoundWaves * kWave, 0, s>>>(dm, kc, bt, bounds, run);
  return hipGetLastError();
}

}  // namespace moe
