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
// Scores are summed in 64 bits and rounded once to fp32: which page is taken is
// a jump, and so it does not depend on the order of a sum or on what else is in
// the batch. The fp64 matrix instruction does it (16 pages by 16 tokens, 4 of
// the 2 D terms at a time), at the rate of the vector unit's fp64 FMAs but
// without sums across lanes.
//
// The selected pages become page tables of their own, one for each token and
// cache head, and the attention kernel for few query rows runs over those.
#include "moe_kv4_sparse.h"

#include "moe_kv4_device.h"
#include "moe_kv4_write.h"

namespace moe {

typedef double f64x4_t __attribute__((ext_vector_type(4)));

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

// Where the scores of a part of the call go: rows row0 .. row0 + rows - 1, as
// order-preserving keys (logit_key; 0: the page does not exist).
struct ScorePart {
  uint32_t *keys;  // [rows][Hkv][max_pages]
  int row0, rows;
};

// Grid: x = token tile * chunks + chunk of pages, y = cache head, z = sequence.
// A chunk is `steps` tiles of 16 pages for each wavefront.
template <int D>
__global__ __launch_bounds__(kScoreWaves *kWave) void kv4_score_kernel(Kv4Dims dm, Kv4Batch bt, Kv4Select sel,
                                                                       ScorePart part, int chunks, int steps) {
  constexpr int kLoads = 2 * D / 32;  // 16-byte loads of a lane for a page's 2 D bounds
  __shared__ double sq[2 * D / 4][kWave];
  const int head = blockIdx.y, seq = blockIdx.z;
  const int tile = blockIdx.x / chunks, chunk = blockIdx.x - tile * chunks;
  const Kv4Span sp = kv4_seq_span(bt, seq);
  const int n = min(sp.n, sel.max_new), i0 = tile * kScoreTile;
  if (i0 >= n) return;
  const int last = min(i0 + kScoreTile, n) - 1;
  if (sp.begin + last < part.row0 || sp.begin + i0 >= part.row0 + part.rows) return;
  const Kv4Scored sc = kv4_scored(dm, sp.first + last, sel.first, sel.recent);
  const int c0 = chunk * steps * kScoreWaves * kScoreTile;
  if (c0 > sc.hi || c0 + steps * kScoreWaves * kScoreTile <= sc.lo) return;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int G = dm.Hq / dm.Hkv;

  // q- and q+ of the tile's tokens as the matrix instruction's operand: terms
  // 32 m + 8 (l / 16) + e of token l % 16 in step 8 m + e, lane l
  for (int at = threadIdx.x; at < kScoreTile * (D / 8); at += kScoreWaves * kWave) {
    const int j = at % kScoreTile, c8 = at / kScoreTile;
    double neg[8], pos[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) neg[e] = pos[e] = 0.0;
    const uint16_t *q = sel.q + (long long)(sp.begin + min(i0 + j, last)) * sel.q_stride + (long long)head * G * D + c8 * 8;
    for (int g = 0; g < G; ++g) {
      float x[8];
      load8<false>(q, (long long)g * D, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {  // a NaN goes to both
        neg[e] += x[e] >= 0.f ? 0.0 : (double)x[e];
        pos[e] += x[e] <= 0.f ? 0.0 : (double)x[e];
      }
    }
    const int m = c8 / 4, l = (c8 % 4) * 16 + j;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sq[m * 8 + e][l] = neg[e];
      sq[D / 4 + m * 8 + e][l] = pos[e];
    }
  }
  __syncthreads();

  const int32_t *table = bt.table + (long long)seq * dm.max_pages;
  for (int st = 0; st < steps; ++st) {
    const int cb = c0 + (st * kScoreWaves + wave) * kScoreTile;
    if (cb > sc.hi) break;
    const int c = cb + (lane & 15);
    const int entry = c <= sc.hi ? table[c] : -1;  // hi is inside the table
    const bool ok = kv4_page_ok(dm, entry);
    const uint16_t *b = sel.bounds + ((long long)(ok ? entry : 0) * dm.Hkv + head) * 2 * D + (lane >> 4) * 8;
    uint4 raw[kLoads];
#pragma unroll
    for (int m = 0; m < kLoads; ++m) raw[m] = *(const uint4 *)(b + m * 32);
    f64x4_t acc[2] = {{0., 0., 0., 0.}, {0., 0., 0., 0.}};
#pragma unroll
    for (int m = 0; m < kLoads; ++m) {
      const uint32_t u[4] = {raw[m].x, raw[m].y, raw[m].z, raw[m].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = (e & 1) ? __uint_as_float(u[e / 2] & 0xFFFF0000u) : __uint_as_float(u[e / 2] << 16);
        acc[e & 1] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)v, sq[m * 8 + e][lane], acc[e & 1], 0, 0, 0);
      }
    }
    const uint64_t valid = __builtin_amdgcn_ballot_w64(ok);  // bits 0 .. 15: the tile's pages
    // lane l, register r: page l / 16 + 4 r, token l % 16
    const int j = lane & 15;
    const int row = sp.begin + i0 + j - part.row0;
    if (i0 + j <= last && row >= 0 && row < part.rows) {
      uint32_t *out = part.keys + ((long long)row * dm.Hkv + head) * dm.max_pages;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = (lane >> 4) + 4 * r;
        const float v = (float)(acc[0][r] + acc[1][r]);
        if (cb + i <= sc.hi) out[cb + i] = (valid >> i & 1) ? logit_key(v) : 0u;
      }
    }
  }
}

// ---- selection

constexpr int kSelectWaves = 4;

// What the selection leaves for the attention.
struct SelectOut {
  int32_t *table;  // [rows][Hkv][size]
  int32_t *len;    // [rows]
  int size;
};

// One workgroup for a token and cache head. A page that is always taken has the
// largest key, one that does not exist 0. The `want`-th largest key is found 8
// bits at a time; each wavefront then lists what it takes of its own quarter.
__global__ __launch_bounds__(kSelectWaves *kWave) void kv4_select_kernel(Kv4Dims dm, Kv4Batch bt, Kv4Select sel,
                                                                         ScorePart part, SelectOut out) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t found[2];
  __shared__ int count[kSelectWaves][2];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = blockIdx.x, tok = part.row0 + r, head = blockIdx.y;
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
  const uint32_t *keys = part.keys + ((long long)r * dm.Hkv + head) * dm.max_pages;
  const auto key_of = [&](int c) -> uint32_t {
    if (c >= sc.lo && c <= sc.hi) return sel.top > 0 ? keys[c] : 0u;
    return kv4_page_ok(dm, table[c]) ? 0xFFFFFFFFu : 0u;
  };
  // this wavefront's pages begin .. end - 1
  const int seg = ((pages + kSelectWaves - 1) / kSelectWaves + kWave - 1) / kWave * kWave;
  const int begin = min(wave * seg, pages), end = min(begin + seg, pages);

  // pages there are, and those always taken
  int all = 0, always = 0;
  for (int c = begin + lane; c - lane < end; c += kWave) {
    const uint32_t k = c < end ? key_of(c) : 0u;
    all += __builtin_popcountll(__builtin_amdgcn_ballot_w64(k != 0));
    always += __builtin_popcountll(__builtin_amdgcn_ballot_w64(k == 0xFFFFFFFFu));
  }
  if (lane == 0) count[wave][0] = all, count[wave][1] = always;
  __syncthreads();
  all = always = 0;
#pragma unroll
  for (int w = 0; w < kSelectWaves; ++w) all += count[w][0], always += count[w][1];
  const int want = sel.top + always;

  // taken: keys above `least`, and the first `ties` of those equal to it
  uint32_t least = 0;
  int ties = 0;
  if (want == 0) {
    least = 0xFFFFFFFFu;
  } else if (all > want) {
    int left = want;
    for (int shift = 24; shift >= 0; shift -= 8) {
      hist[threadIdx.x] = 0;
      __syncthreads();
      for (int c = begin + lane; c < end; c += kWave) {
        const uint32_t k = key_of(c);
        if (k != 0 && (shift == 24 || k >> (shift + 8) == least)) atomicAdd(&hist[k >> shift & 255u], 1u);
      }
      __syncthreads();
      if (wave == 0) {
        // lane l: digits 255 - 4 l down to 252 - 4 l
        uint32_t h[4], sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += h[i] = hist[255 - 4 * lane - i];
        uint32_t before = (uint32_t)wave_scan((int)sum) - sum;
        if (before < (uint32_t)left && before + sum >= (uint32_t)left) {
          int i = 0;
#pragma unroll
          for (int k = 0; k < 3; ++k)
            if (i == k && before + h[k] < (uint32_t)left) before += h[k], ++i;
          found[0] = 255 - 4 * lane - i;
          found[1] = before;
        }
      }
      __syncthreads();
      least = least << 8 | found[0];
      left -= (int)found[1];
    }
    ties = left;
  }

  int more = 0, same = 0;
  for (int c0 = begin; c0 < end; c0 += kWave) {
    const uint32_t k = c0 + lane < end ? key_of(c0 + lane) : 0u;
    more += __builtin_popcountll(__builtin_amdgcn_ballot_w64(k > least));
    same += __builtin_popcountll(__builtin_amdgcn_ballot_w64(k != 0 && k == least));
  }
  __syncthreads();  // the counts above have been read
  if (lane == 0) count[wave][0] = more, count[wave][1] = same;
  __syncthreads();
  int at = 0, seen = 0, total = 0, equal = 0;  // at: this wavefront's first place; seen: ties before it
#pragma unroll
  for (int w = 0; w < kSelectWaves; ++w) {
    if (w == wave) at = total, seen = equal;
    total += count[w][0] + min(count[w][1], max(ties - equal, 0));
    equal += count[w][1];
  }
  const long long row = ((long long)r * dm.Hkv + head) * out.size;
  int32_t *blocks = sel.blocks == nullptr ? nullptr : sel.blocks + ((long long)tok * dm.Hkv + head) * out.size;
  const uint64_t lower = (1ull << lane) - 1;
  for (int c0 = begin; c0 < end; c0 += kWave) {
    const int c = c0 + lane;
    const uint32_t k = c < end ? key_of(c) : 0u;
    const bool tie = k != 0 && k == least;
    const uint64_t tied = __builtin_amdgcn_ballot_w64(tie);
    const bool take = k > least || (tie && seen + __builtin_popcountll(tied & lower) < ties);
    const uint64_t taken = __builtin_amdgcn_ballot_w64(take);
    if (take) {
      const int to = at + __builtin_popcountll(taken & lower);
      out.table[row + to] = table[c];
      if (blocks != nullptr) blocks[to] = c;
    }
    at += __builtin_popcountll(taken);
    seen += __builtin_popcountll(tied);
  }
  if (blocks != nullptr)
    for (int i = total + threadIdx.x; i < out.size; i += kSelectWaves * kWave) blocks[i] = -1;
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
  size_t keys, table, len, attention, bytes;
};

constexpr size_t kKeysBytes = 256u << 20;  // score keys of a part, while it has more than one row

static size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

static Kv4Dims selected_dims(const Kv4Dims &dm, int rows, int size) {
  Kv4Dims d = dm;
  d.B = rows;
  d.max_pages = size;
  return d;
}

static SparseWs sparse_ws(const Kv4Dims &dm, int T, int size) {
  SparseWs w;
  const size_t row = (size_t)dm.Hkv * dm.max_pages * 4;
  size_t rows = kKeysBytes / row;
  if (rows > 32768) rows = 32768;
  if (rows < 1) rows = 1;
  w.rows = rows < (size_t)T ? (int)rows : T;
  const size_t full = kv4_attention_ws(selected_dims(dm, w.rows, size), w.rows, 1, 0);
  const int rest = T % w.rows;
  const size_t last = rest ? kv4_attention_ws(selected_dims(dm, rest, size), rest, 1, 0) : 0;
  w.keys = 0;
  w.table = align256(w.keys + w.rows * row);
  w.len = align256(w.table + (size_t)w.rows * dm.Hkv * size * 4);
  w.attention = align256(w.len + (size_t)w.rows * 4);
  w.bytes = w.attention + (full > last ? full : last);
  return w;
}

size_t kv4_sparse_ws(const Kv4Dims &dm, int T, const Kv4Select &sel) {
  return sparse_ws(dm, T, sel.top + sel.first + sel.recent).bytes;
}

template <int D>
static hipError_t launch_score(const Kv4Dims &dm, const Kv4Batch &bt, const Kv4Select &sel, const ScorePart &part,
                               hipStream_t s) {
  constexpr int kPages = kScoreWaves * kScoreTile;
  const long long tiles = ((long long)sel.max_new + kScoreTile - 1) / kScoreTile;
  const long long all = (dm.max_pages + kPages - 1) / kPages;
  // the queries are brought to LDS once for a workgroup's pages: few workgroups
  // where there are enough of them for the card
  long long steps = tiles * dm.B * dm.Hkv * all / 2048;
  if (steps > 16) steps = 16;
  if (steps < 1) steps = 1;
  while (steps < all && tiles * ((all + steps - 1) / steps) >= 1 << 24) steps *= 2;
  const long long chunks = (all + steps - 1) / steps;
  kv4_score_kernel<D><<<dim3((unsigned)(tiles * chunks), dm.Hkv, dm.B), kScoreWaves * kWave, 0, s>>>(
      dm, bt, sel, part, (int)chunks, (int)steps);
  return hipGetLastError();
}

hipError_t launch_kv4_sparse(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc, const Kv4Batch &bt,
                             const Kv4Select &sel, uint16_t *out, long long out_stride, float scale, void *ws,
                             hipStream_t s) {
  const int size = sel.top + sel.first + sel.recent;
  const SparseWs w = sparse_ws(dm, bt.T, size);
  const SelectOut so{(int32_t *)((char *)ws + w.table), (int32_t *)((char *)ws + w.len), size};
  for (int row0 = 0; row0 < bt.T; row0 += w.rows) {
    const ScorePart part{(uint32_t *)((char *)ws + w.keys), row0, bt.T - row0 < w.rows ? bt.T - row0 : w.rows};
    hipError_t e = hipSuccess;
    if (sel.top > 0)
      e = dm.D == 64 ? launch_score<64>(dm, bt, sel, part, s)
                     : dm.D == 128 ? launch_score<128>(dm, bt, sel, part, s) : launch_score<256>(dm, bt, sel, part, s);
    if (e != hipSuccess) return e;
    kv4_select_kernel<<<dim3(part.rows, dm.Hkv), kSelectWaves * kWave, 0, s>>>(dm, bt, sel, part, so);
    e = hipGetLastError();
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
