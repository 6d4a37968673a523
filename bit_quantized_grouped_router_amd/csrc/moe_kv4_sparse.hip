// Attention of each new token over the cache pages that a score selects for it.
//
//   bounds   per page, cache head and channel the smallest and largest key lo, hi
//   score    of a page for a token and cache head: sum over the group's query
//            heads and the channels of max(q lo, q hi), the most that any key of
//            the page could score, summed over the heads. With q+ = sum over the
//            heads of max(q, 0) and q- = sum of min(q, 0) it is q- . lo + q+ . hi
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
#include "moe_kv4_sparse.h"

#include "moe_kv4_device.h"
#include "moe_kv4_write.h"

namespace moe {

// ---- bounds

constexpr int kBoundWaves = 4;

// Pages of new tokens: one wavefront looks at `run` token rows, and for each that
// is the first of the call in its page it goes over the page's keys, up to the
// sequence's last. D / 8 lanes take a key, 8 channels each.
template <int D>
__global__ __launch_bounds__(kBoundWaves *kWave) void kv4_bounds_kernel(Kv4Dims dm, Kv4Plane kc, Kv4Batch bt,
                                                                        uint16_t *__restrict__ bounds, int run) {
  constexpr int kLanes = D / 8, kKeys = kWave / kLanes;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const long long r0 = ((long long)blockIdx.x * kBoundWaves + wave) * run;
  if (r0 >= bt.T) return;
  const int head = blockIdx.y;
  // this lane's row: the last sequence that begins at or before it
  int page = -1, keys = 0;
  const long long row = r0 + lane;
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
  uint64_t todo = __builtin_amdgcn_ballot_w64(page >= 0);
  while (todo != 0) {
    const int w = __builtin_ctzll(todo);
    todo &= todo - 1;
    const int pg = __builtin_amdgcn_readlane(page, w), n = __builtin_amdgcn_readlane(keys, w);
    const long long base = kv4_row(dm, pg, head, 0);
    float mn[8], mx[8];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) mn[i] = __builtin_huge_valf(), mx[i] = kNegInf;
    const int at = (lane % kLanes) * 8;
    for (int k0 = 0; k0 < n; k0 += 4 * kKeys) {
      uint32_t word[4], sb[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        // keys past the last repeat it
        const long long r = base + min(k0 + u * kKeys + lane / kLanes, n - 1);
        word[u] = *(const uint32_t *)(kc.codes + r * (D / 2) + at / 2);
        const long long g = r * (D / kGroup) + at / kGroup;
        sb[u] = kc.scales[g] | (uint32_t)kc.biases[g] << 16;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float s = __uint_as_float(sb[u] << 16), b = __uint_as_float(sb[u] & 0xFFFF0000u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = fmaf(s, (float)((word[u] >> (4 * i)) & 15u), b);
          mn[i] = fminf(mn[i], v);
          mx[i] = fmaxf(mx[i], v);
          bad |= v != v;
        }
      }
    }
    // a channel that holds a NaN has NaN bounds; the lane looks again at which
    uint32_t nan = 0;
    if (__builtin_amdgcn_ballot_w64(bad) != 0) {
      for (int k = lane / kLanes; k < n; k += kKeys) {
        const long long r = base + k;
        const uint32_t word = *(const uint32_t *)(kc.codes + r * (D / 2) + at / 2);
        const long long g = r * (D / kGroup) + at / kGroup;
        const float s = bf16_to_f32(kc.scales[g]), b = bf16_to_f32(kc.biases[g]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = fmaf(s, (float)((word >> (4 * i)) & 15u), b);
          nan |= (uint32_t)(v != v) << i;
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
      for (int i = 0; i < 8; ++i)
        if (nan >> i & 1) mn[i] = mx[i] = __uint_as_float(0x7FC00000u);
      uint16_t *o = bounds + ((long long)pg * dm.Hkv + head) * 2 * D + at;
      // adding 0 makes a zero +0
      *(uint4 *)o = make_uint4(pack_bf16x2(mn[0] + 0.f, mn[1] + 0.f), pack_bf16x2(mn[2] + 0.f, mn[3] + 0.f),
                               pack_bf16x2(mn[4] + 0.f, mn[5] + 0.f), pack_bf16x2(mn[6] + 0.f, mn[7] + 0.f));
      *(uint4 *)(o + D) = make_uint4(pack_bf16x2(mx[0] + 0.f, mx[1] + 0.f), pack_bf16x2(mx[2] + 0.f, mx[3] + 0.f),
                                     pack_bf16x2(mx[4] + 0.f, mx[5] + 0.f), pack_bf16x2(mx[6] + 0.f, mx[7] + 0.f));
    }
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

// The bounds of 16 pages as they are loaded: lane l has 16 bytes of each 64 of page l /
// 4, so that four lanes' addresses follow on each other (with a page a lane, as the
// matrix instruction wants them, the L1 cache takes 16 bytes at a time: 46 us, not
// 20, for 1500 tokens behind 60,000). They change lanes through LDS, 4 KB at a time.
// Which 16 bytes: swapped by l / 16, so that no banks collide there.
template <int D>
struct PageBounds {
  static constexpr int kLoads = 2 * D / 32;
  uint4 v[kLoads];
};

template <int D>
__device__ __forceinline__ void load_bounds(const Kv4Dims &dm, const uint16_t *bounds, int entry, int head, int lane,
                                            PageBounds<D> &b) {
  const bool ok = kv4_page_ok(dm, entry);
  const uint16_t *p = bounds + ((long long)(ok ? entry : 0) * dm.Hkv + head) * 2 * D + ((lane & 3) ^ (lane >> 4)) * 8;
#pragma unroll
  for (int m = 0; m < PageBounds<D>::kLoads; ++m) {
    b.v[m] = make_uint4(0, 0, 0, 0);
    if (ok) b.v[m] = *(const uint4 *)(p + m * 32);
  }
}

// Grid: x = token tile * chunks + chunk of pages, y = cache head, z = sequence.
// 16 pages by 16 tokens a wavefront at a time; the tokens' q- and q+ lie in LDS as
// the matrix instruction takes them. What bounds it: for few tokens the chain
// offsets - table - bounds, for many the bounds' way from the L2.
template <int D>
__global__ __launch_bounds__(kScoreWaves *kWave) void kv4_score_kernel(Kv4Dims dm, Kv4Batch bt, Kv4Select sel,
                                                                       ScorePart part) {
  constexpr int kSteps = 2 * D / 32;
  __shared__ uint4 sq[3][kSteps][kWave];
  __shared__ uint4 turned[kScoreWaves][4][kWave];
  const int head = blockIdx.y, seq = blockIdx.z;
  const int tile = blockIdx.x / part.chunks, chunk = blockIdx.x - tile * part.chunks;
  const Kv4Span sp = kv4_seq_span(bt, seq);
  const int n = min(sp.n, sel.max_new), i0 = tile * kScoreTile;
  if (i0 >= n) return;
  const int last = min(i0 + kScoreTile, n) - 1;
  if (sp.begin + last < part.row0 || sp.begin + i0 >= part.row0 + part.rows) return;
  const Kv4Scored sc = kv4_scored(dm, sp.first + last, sel.first, sel.recent);
  const int span = part.steps * kScoreWaves * kScoreTile, c0 = chunk * span;
  if (c0 > sc.hi || c0 + span <= sc.lo) return;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int G = dm.Hq / dm.Hkv;
  const int32_t *table = bt.table + (long long)seq * dm.max_pages;
  // page of this lane in the wavefront's tile st (hi is inside the table)
  const auto entry_of = [&](int st) {
    const int c = c0 + (st * kScoreWaves + wave) * kScoreTile + (lane >> 2);
    return st < part.steps && c <= sc.hi ? table[c] : -1;
  };
  int entry = entry_of(0), next_entry = entry_of(1);
  PageBounds<D> here;
  load_bounds<D>(dm, sel.bounds, entry, head, lane, here);

  // q- and q+ of the tile's tokens, two channels at a time: terms 32 m + 8 (l / 16) .. + 7
  // of token l % 16 for lane l in step m. Columns without a token are not looked at.
  for (int at = threadIdx.x; at < (last - i0 + 1) * (D / 2); at += kScoreWaves * kWave) {
    const int j = at / (D / 2), c2 = at % (D / 2);
    const uint16_t *q = sel.q + (long long)(sp.begin + i0 + j) * sel.q_stride + (long long)head * G * D + c2 * 2;
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
      ((uint32_t *)&sq[p][m][l])[c2 % 4] = a[0][p] | (uint32_t)a[1][p] << 16;
      ((uint32_t *)&sq[p][D / 32 + m][l])[c2 % 4] = b[0][p] | (uint32_t)b[1][p] << 16;
    }
  }
  __syncthreads();

  const int j = lane & 15;
  const int row = sp.begin + i0 + j - part.row0;
  const bool mine = i0 + j <= last && row >= 0 && row < part.rows;
  uint32_t *out = part.keys + ((long long)row * dm.Hkv + head) * part.pitch;
  uint32_t most = 0;
  for (int st = 0; st < part.steps; ++st) {
    const int cb = c0 + (st * kScoreWaves + wave) * kScoreTile;
    if (cb > sc.hi) break;
    const uint64_t valid = __builtin_amdgcn_ballot_w64(kv4_page_ok(dm, entry));  // bit 4 i: page i of the tile
    PageBounds<D> now = here;
    entry = next_entry;
    load_bounds<D>(dm, sel.bounds, entry, head, lane, here);
    next_entry = entry_of(st + 2);
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    f32x4_t step[kSteps], rest[2] = {zero, zero}, sum = zero;
#pragma unroll
    for (int m = 0; m < kSteps; ++m) {
      if (m % 4 == 0) {
        wave_lds_sync();  // what was there has been read
#pragma unroll
        for (int i = 0; i < 4; ++i) turned[wave][i][lane] = now.v[m + i];
        wave_lds_sync();
#pragma unroll
        for (int i = 0; i < 4; ++i) now.v[m + i] = turned[wave][i][(lane & 15) * 4 + ((lane >> 4) ^ (lane >> 2 & 3))];
      }
      const bf16x8_t b = __builtin_bit_cast(bf16x8_t, now.v[m]);
      // q- is negative and q+ is not: with the sign of q the bounds' magnitudes make all terms positive
      const uint4 mag = m < kSteps / 2 ? make_uint4(now.v[m].x | 0x80008000u, now.v[m].y | 0x80008000u,
                                                    now.v[m].z | 0x80008000u, now.v[m].w | 0x80008000u)
                                       : make_uint4(now.v[m].x & 0x7FFF7FFFu, now.v[m].y & 0x7FFF7FFFu,
                                                    now.v[m].z & 0x7FFF7FFFu, now.v[m].w & 0x7FFF7FFFu);
      const bf16x8_t q = __builtin_bit_cast(bf16x8_t, sq[0][m][lane]);
      step[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, q, zero, 0, 0, 0);
      sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, mag), q, sum, 0, 0, 0);
#pragma unroll
      for (int p = 0; p < 2; ++p)
        rest[p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, __builtin_bit_cast(bf16x8_t, sq[p + 1][m][lane]), rest[p],
                                                          0, 0, 0);
    }
#pragma unroll
    for (int w = 1; w < kSteps; w *= 2)
#pragma unroll
      for (int m = 0; m + w < kSteps; m += 2 * w) step[m] += step[m + w];
    step[0] += rest[0] + rest[1];
    // register r: page 4 (l / 16) + r, token l % 16
    uint32_t key[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      key[r] = (valid >> (4 * (4 * (lane >> 4) + r)) & 1) ? logit_key(step[0][r]) : 0u;
      most = max(most, __float_as_uint(sum[r]) & 0x7FFFFFFFu);
    }
    if (mine) *(uint4 *)(out + cb + 4 * (lane >> 4)) = make_uint4(key[0], key[1], key[2], key[3]);
  }
  most = max(most, (uint32_t)__shfl_xor((int)most, 16, kWave));
  most = max(most, (uint32_t)__shfl_xor((int)most, 32, kWave));
  if (mine && lane < 16)
    part.most[((long long)row * dm.Hkv + head) * part.chunks * kScoreWaves + chunk * kScoreWaves + wave] = most;
}

// ---- selection

constexpr int kSelectMostWaves = 16;

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
  int32_t *table;  // [rows][Hkv][size]
  int32_t *len;    // [rows]
  int size;
};

// v plus the value a DPP lane pattern brings in (see wave_sum_dpp).
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_add64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROW_MASK, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROW_MASK, 0xf, false);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
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
    s = dpp_add64<0xb1, 0xf>(s);
    s = dpp_add64<0x4e, 0xf>(s);
    s = dpp_add64<0x141, 0xf>(s);
    s = dpp_add64<0x140, 0xf>(s);
    s = dpp_add64<0x142, 0xa>(s);
    s = dpp_add64<0x143, 0xc>(s);
    return __builtin_amdgcn_readlane(logit_key((float)s), kWave - 1);
  }
};

// One workgroup for a token and cache head. A page that is always taken has the
// largest key, one that does not exist 0. The key of the last one taken is found 8
// bits at a time, from the first bit on in which keys differ; pages whose scores
// lie within their error of it are scored again in 64 bits: up to 64 of them are
// ranked at once, for more the search is repeated. Each wavefront then lists what it takes of its own pages.
// Bound by latency: three rounds of loads, then barriers. R: pages of a lane, their
// keys and places held in registers, so that a workgroup of W wavefronts takes 64 R W
// pages; 0: any number, read each time from the scores.
template <int D, int R>
__global__ __launch_bounds__(kSelectMostWaves *kWave) void kv4_select_kernel(Kv4Dims dm, Kv4Batch bt, Kv4Select sel,
                                                                             ScorePart part, SelectOut out) {
  extern __shared__ __attribute__((aligned(16))) uint4 queries[];  // the heads' D channels
  __shared__ __attribute__((aligned(16))) uint32_t hist[256];
  __shared__ uint32_t found[2];
  __shared__ int listed, list_page[kWave], list_place[kWave];
  __shared__ uint32_t list_key[kWave];
  __shared__ uint32_t shared[kSelectMostWaves][2];
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

  if (threadIdx.x == 0) listed = 0;
  if (sel.top > 0) {  // in case scores have to be worked out again
    const uint16_t *q = sel.q + tok * sel.q_stride + (long long)head * G * D;
    for (int i = threadIdx.x; i < G * (D / 8); i += blockDim.x) queries[i] = *(const uint4 *)(q + i * 8);
  }
  // the largest sum of magnitudes of the scored pages
  uint32_t most = 0;
  if (sel.top > 0 && sc.hi >= sc.lo) {
    const int span = part.steps * kScoreWaves * kScoreTile;
    const uint32_t *m = part.most + item * part.chunks * kScoreWaves;
    for (int i = sc.lo / span * kScoreWaves + lane; i < (sc.hi / span + 1) * kScoreWaves; i += kWave)
      most = max(most, m[i]);
  }
  const auto first_key = [&](int c, int entry) -> uint32_t {
    if (c >= end) return 0u;
    if (c >= sc.lo && c <= sc.hi) return sel.top > 0 ? keys[c] : 0u;
    return kv4_page_ok(dm, entry) ? 0xFFFFFFFFu : 0u;
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
  // sums over the workgroup of two wave-uniform counts
  const auto add_up = [&](int &a, int &b) {
    __syncthreads();
    if (lane == 0) shared[wave][0] = a, shared[wave][1] = b;
    __syncthreads();
    a = lane < waves ? shared[lane][0] : 0;
    b = lane < waves ? shared[lane][1] : 0;
    a = first16_sum(a);
    b = first16_sum(b);
  };

  int all = 0, always = 0;  // pages there are; those always taken
  each([&](int, int, uint32_t k) {
    all += __builtin_popcountll(__builtin_amdgcn_ballot_w64(k != 0));
    always += __builtin_popcountll(__builtin_amdgcn_ballot_w64(k == 0xFFFFFFFFu));
  });
  add_up(all, always);
  const int want = sel.top + always;

  // taken: keys above `least`, and the first `ties` of those equal to it
  uint32_t least = 0;
  int ties = 0;
  if (want == 0) {
    least = 0xFFFFFFFFu;
  } else if (all > want) {
    int certain = always;  // keys 0xFFFFFFFF: taken whatever the others are
    for (int exact = 0; exact < 2; ++exact) {
      // of the others the (want - certain)-th largest
      uint32_t hi = 0, lo = 0xFFFFFFFFu;
      each([&](int, int, uint32_t k) {
        if (k != 0 && k != 0xFFFFFFFFu) hi = max(hi, k), lo = min(lo, k);
      });
      hi = wave_max_u32(hi);
      lo = ~wave_max_u32(~lo);
      __syncthreads();
      if (lane == 0) shared[wave][0] = hi, shared[wave][1] = ~lo;
      if (threadIdx.x < 256) hist[threadIdx.x] = 0;
      __syncthreads();
      hi = wave_max_u32(lane < waves ? shared[lane][0] : 0u);
      lo = ~wave_max_u32(lane < waves ? shared[lane][1] : 0u);
      // bits not known yet: one at least, which spares a choice that hipcc 7.2 compiles
      // to a vector compare and a scalar select on another condition
      int left = want - certain, bits = 32 - __builtin_clz((hi ^ lo) | 1u);
      uint64_t prefix = (uint64_t)hi >> bits;
      while (true) {
        const int take = min(bits, 8);
        each([&](int, int, uint32_t k) {
          if (k != 0 && k != 0xFFFFFFFFu && (uint64_t)k >> bits == prefix)
            atomicAdd(&hist[k >> (bits - take) & ((1u << take) - 1)], 1u);
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
        bits -= take;
        prefix = prefix << take | __builtin_amdgcn_readfirstlane(found[0]);
        left -= (int)__builtin_amdgcn_readfirstlane(found[1]);
        if (bits == 0) break;
      }
      least = (uint32_t)prefix;
      ties = left;
      if (exact) break;

      // scores that may be on the other side of the border
      most = wave_max_u32(most);
      const bool finite = most < 0x7F800000u;
      const float off = 2.0f * (score_error(G) * __uint_as_float(most) + kScoreFlushed);
      const float border = key_logit(least);
      const float above = (border + off) * (1.0f + 0x1p-22f * (border + off > 0.f ? 1.f : -1.f));
      const float below = (border - off) * (1.0f - 0x1p-22f * (border - off > 0.f ? 1.f : -1.f));
      const auto surely = [&](uint32_t k) { return k == 0xFFFFFFFFu || (k != 0 && finite && key_logit(k) > above); };
      const auto maybe = [&](uint32_t k) { return k != 0 && !surely(k) && !(finite && key_logit(k) < below); };
      int near = 0;
      certain = 0;
      each([&](int, int, uint32_t k) {
        certain += __builtin_popcountll(__builtin_amdgcn_ballot_w64(surely(k)));
        near += __builtin_popcountll(__builtin_amdgcn_ballot_w64(maybe(k)));
      });
      add_up(certain, near);
      if (finite && certain + near == want) break;  // all of those near it are taken: keys from least on
      ExactScore<D> score;
      uint32_t words[D / 64];
      if (near <= kWave) {
        each([&](int c, int entry, uint32_t k) {
          if (maybe(k)) {
            const int i = atomicAdd(&listed, 1);
            list_page[i] = c;
            list_place[i] = entry;
          }
        });
        __syncthreads();
        for (int i = wave; i < near; i += waves) {
          const long long page = (long long)__builtin_amdgcn_readfirstlane(list_place[i]) * dm.Hkv + head;
          score.words(sel.bounds + page * 2 * D + lane * (D / 32), words);
          if (i == wave) score.load((const uint16_t *)queries, G, lane);
          const uint32_t k = score.key(words);
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
        const uint64_t taken = __builtin_amdgcn_ballot_w64(lane < near && rank < want - certain);
        each([&](int c, int, uint32_t &k) {
          bool take = surely(k);
          for (uint64_t todo = taken; todo != 0; todo &= todo - 1)
            take |= c == __builtin_amdgcn_readlane(lc, __builtin_ctzll(todo));
          k = take ? 0xFFFFFFFFu : 0u;
          if constexpr (R == 0) {
            if (c < end && c >= sc.lo && c <= sc.hi) keys[c] = k;
          }
        });
        least = 0xFFFFFFFEu;
        ties = 0;
        break;
      }
      score.load((const uint16_t *)queries, G, lane);
      each([&](int c, int entry, uint32_t &k) {
        uint64_t todo = __builtin_amdgcn_ballot_w64(maybe(k));
        k = surely(k) ? 0xFFFFFFFFu : 0u;
        while (todo != 0) {
          const int w = __builtin_ctzll(todo);
          todo &= todo - 1;
          const int pg = __builtin_amdgcn_readlane(entry, w);  // it has a key, so it exists
          score.words(sel.bounds + ((long long)pg * dm.Hkv + head) * 2 * D + lane * (D / 32), words);
          const uint32_t e = score.key(words);
          k = lane == w ? e : k;
        }
        if constexpr (R == 0) {
          if (c < end && c >= sc.lo && c <= sc.hi) keys[c] = k;
        }
      });
    }
  }

  int more = 0, same = 0;
  each([&](int, int, uint32_t k) {
    more += __builtin_popcountll(__builtin_amdgcn_ballot_w64(k > least));
    same += __builtin_popcountll(__builtin_amdgcn_ballot_w64(k != 0 && k == least));
  });
  __syncthreads();  // what was there has been read
  if (lane == 0) shared[wave][0] = more, shared[wave][1] = same;
  __syncthreads();
  // of all wavefronts up to lane's: keys taken above least, and equal to it
  more = lane < waves ? (int)shared[lane][0] : 0;
  same = lane < waves ? (int)shared[lane][1] : 0;
  const int seen_upto = wave_scan(same), at_upto = wave_scan(more + min(same, max(ties - (seen_upto - same), 0)));
  int seen = wave > 0 ? __builtin_amdgcn_readlane(seen_upto, wave > 0 ? wave - 1 : 0) : 0;  // ties before this one's
  int at = wave > 0 ? __builtin_amdgcn_readlane(at_upto, wave > 0 ? wave - 1 : 0) : 0;      // its first place
  const int total = __builtin_amdgcn_readlane(at_upto, kWave - 1);
  const long long row = item * out.size;
  int32_t *blocks = sel.blocks == nullptr ? nullptr : sel.blocks + ((long long)tok * dm.Hkv + head) * out.size;
  const uint64_t lower = (1ull << lane) - 1;
  each([&](int c, int entry, uint32_t k) {
    const bool tie = k != 0 && k == least;
    const uint64_t tied = __builtin_amdgcn_ballot_w64(tie);
    const bool take = k > least || (tie && seen + __builtin_popcountll(tied & lower) < ties);
    const uint64_t taken = __builtin_amdgcn_ballot_w64(take);
    const int to = at + __builtin_popcountll(taken & lower);
    if (take && to < out.size) {
      out.table[row + to] = entry;
      if (blocks != nullptr) blocks[to] = c;
    }
    at += __builtin_popcountll(taken);
    seen += __builtin_popcountll(tied);
  });
  if (blocks != nullptr)
    for (int i = total + threadIdx.x; i < out.size; i += blockDim.x) blocks[i] = -1;
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
  int pitch, chunks, steps;  // of the scores
  size_t keys, most, table, len, attention, bytes;
};

constexpr size_t kKeysBytes = 256u << 20;  // score keys of a part, while it has more than one row

static size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

static Kv4Dims selected_dims(const Kv4Dims &dm, int rows, int size) {
  Kv4Dims d = dm;
  d.B = rows;
  d.max_pages = size;
  return d;
}

static SparseWs sparse_ws(const Kv4Dims &dm, int T, const Kv4Select &sel) {
  SparseWs w;
  const int size = sel.top + sel.first + sel.recent;
  w.pitch = (dm.max_pages + kScoreTile - 1) / kScoreTile * kScoreTile;
  // the queries are brought to LDS once for a workgroup's pages: few workgroups
  // where there are enough of them for the card
  const long long tiles = ((long long)sel.max_new + kScoreTile - 1) / kScoreTile;
  const long long all = (w.pitch + kScoreWaves * kScoreTile - 1) / (kScoreWaves * kScoreTile);
  long long steps = tiles * dm.B * dm.Hkv * all / 768;
  if (steps > 16) steps = 16;
  if (steps < 1) steps = 1;
  while (steps < all && tiles * ((all + steps - 1) / steps) >= 1 << 24) steps *= 2;
  w.steps = (int)steps;
  w.chunks = (int)((all + steps - 1) / steps);
  const size_t row = (size_t)dm.Hkv * w.pitch * 4;
  size_t rows = kKeysBytes / row;
  if (rows > 32768) rows = 32768;
  if (rows < 1) rows = 1;
  w.rows = rows < (size_t)T ? (int)rows : T;
  const size_t full = kv4_attention_ws(selected_dims(dm, w.rows, size), w.rows, 1, 0);
  const int rest = T % w.rows;
  const size_t last = rest ? kv4_attention_ws(selected_dims(dm, rest, size), rest, 1, 0) : 0;
  w.keys = 0;
  w.most = align256(w.keys + w.rows * row);
  w.table = align256(w.most + (size_t)w.rows * dm.Hkv * w.chunks * kScoreWaves * 4);
  w.len = align256(w.table + (size_t)w.rows * dm.Hkv * size * 4);
  w.attention = align256(w.len + (size_t)w.rows * 4);
  w.bytes = w.attention + (full > last ? full : last);
  return w;
}

size_t kv4_sparse_ws(const Kv4Dims &dm, int T, const Kv4Select &sel) { return sparse_ws(dm, T, sel).bytes; }

template <int D>
static hipError_t launch_selection(const Kv4Dims &dm, const Kv4Batch &bt, const Kv4Select &sel, const ScorePart &part,
                                   const SelectOut &so, hipStream_t s) {
  const long long tiles = ((long long)sel.max_new + kScoreTile - 1) / kScoreTile;
  if (sel.top > 0) {
    kv4_score_kernel<D><<<dim3((unsigned)(tiles * part.chunks), dm.Hkv, dm.B), kScoreWaves * kWave, 0, s>>>(dm, bt, sel,
                                                                                                            part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // Few lists: two pages a lane of as many wavefronts as that takes, for the shortest
  // chain. Many: eight a lane of a quarter as many wavefronts, for fewer barriers.
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
  const int size = sel.top + sel.first + sel.recent;
  const SparseWs w = sparse_ws(dm, bt.T, sel);
  const SelectOut so{(int32_t *)((char *)ws + w.table), (int32_t *)((char *)ws + w.len), size};
  for (int row0 = 0; row0 < bt.T; row0 += w.rows) {
    const ScorePart part{(uint32_t *)((char *)ws + w.keys), (uint32_t *)((char *)ws + w.most), row0,
                         bt.T - row0 < w.rows ? bt.T - row0 : w.rows, w.pitch, w.chunks, w.steps};
    hipError_t e = dm.D == 64    ? launch_selection<64>(dm, bt, sel, part, so, s)
                   : dm.D == 128 ? launch_selection<128>(dm, bt, sel, part, so, s)
                                 : launch_selection<256>(dm, bt, sel, part, so, s);
    if (e != hipSuccess) return e;
    const Kv4Batch rows{so.table, nullptr, so.len, part.rows, true};
    const Kv4Attn at{sel.q + (long long)row0 * sel.q_stride, out + (long long)row0 * out_stride, sel.q_stride,
                     out_stride, 1, scale, false, 0, 0, 0, 0};
    e = launch_kv4_attention(selected_dims(dm, part.rows, size), kc, vc, rows, at, (char *)ws + w.attention, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_kv4_bounds(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Batch &bt, uint16_t *bounds,
                             hipStream_t s) {
  // rows a wavefront looks at: one while that many wavefronts fit the card
  int run = 1;
  while (run < kWave && (long long)bt.T * dm.Hkv / run > 8192) run *= 2;
  const long long per = (long long)run * kBoundWaves;
  const dim3 grid((unsigned)((bt.T + per - 1) / per), dm.Hkv);
  auto *kernel = dm.D == 64 ? kv4_bounds_kernel<64> : dm.D == 128 ? kv4_bounds_kernel<128> : kv4_bounds_kernel<256>;
  kernel<<<grid, kBoundWaves * kWave, 0, s>>>(dm, kc, bt, bounds, run);
  return hipGetLastError();
}

}  // namespace moe
