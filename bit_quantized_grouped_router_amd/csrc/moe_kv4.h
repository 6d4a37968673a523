// The paged int4-g64 key/value cache: its shape, where a token lives in it,
// and the launchers of the kernels that write, read and attend to it.
//
// The index arithmetic is plain C++ (no HIP types), so that it can be checked
// on the host; every index that comes from device memory (sequence offsets,
// lengths, page numbers) is brought into range here before it is used.
#pragma once

#include <stddef.h>
#include <stdint.h>

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

struct Kv4Dims {
  int B, Hq, Hkv, D;
  int page, page_shift;  // tokens per page, its log2
  int num_pages, max_pages;
};

struct Kv4Plane {
  uint8_t *codes;
  uint16_t *scales, *biases;
};

// Per-sequence metadata in device memory, and the rows T of the token tensors.
struct Kv4Batch {
  const int32_t *table;  // [B][max_pages] page numbers
  const int32_t *cu;     // [B+1] first row of each sequence's new tokens
  const int32_t *len;    // [B] tokens of each sequence, the new ones included
  int T;
  // Each row is a sequence of its own (B = T, cu unused): table is [T][Hkv][max_pages], a
  // list of pages for each cache head, and len[t] the keys in them; negative: left out.
  bool rows;
};

// The new tokens of one sequence: rows begin .. begin + n - 1 of the token
// tensors, at positions first .. first + n - 1 of the sequence (first may be
// negative when the caller's lengths do not fit: such positions hold nothing).
struct Kv4Span {
  int begin, n;
  long long first, len;
};

MOE_HD Kv4Span kv4_span(int cu0, int cu1, int len, int T) {
  Kv4Span s;
  s.begin = cu0 < 0 ? 0 : (cu0 > T ? T : cu0);
  const int end = cu1 > T ? T : cu1;
  s.n = end > s.begin ? end - s.begin : 0;
  s.len = len < 0 ? 0 : len;
  s.first = s.len - s.n;
  return s;
}

// A row that is a sequence of its own.
MOE_HD Kv4Span kv4_row_span(int row, int len) {
  Kv4Span s;
  s.begin = row;
  s.n = len < 0 ? 0 : 1;
  s.len = len < 0 ? 0 : len;
  s.first = s.len - s.n;
  return s;
}

MOE_HD Kv4Span kv4_seq_span(const Kv4Batch &bt, int seq) {
  return bt.rows ? kv4_row_span(seq, bt.len[seq]) : kv4_span(bt.cu[seq], bt.cu[seq + 1], bt.len[seq], bt.T);
}

// Positions a sequence's page table row covers.
MOE_HD long long kv4_capacity(const Kv4Dims &dm) { return (long long)dm.max_pages << dm.page_shift; }

MOE_HD bool kv4_page_ok(const Kv4Dims &dm, int page) { return page >= 0 && page < dm.num_pages; }

// Cache row (of D/2 bytes of codes) of a slot of a page and a head.
MOE_HD long long kv4_row(const Kv4Dims &dm, int page, int head, int slot) {
  return (((long long)page * dm.Hkv + head) << dm.page_shift) + slot;
}

// Keys a block of query rows at positions p0 .. p1 (p0 <= p1) can see: lo ..
// hi - 1, empty when hi <= lo.
struct Kv4Range {
  long long lo, hi;
};

MOE_HD Kv4Range kv4_range(const Kv4Dims &dm, long long p0, long long p1, long long len, bool causal,
                          int window) {
  const long long cap = kv4_capacity(dm);
  Kv4Range r;
  r.hi = len < cap ? len : cap;
  if (causal && p1 + 1 < r.hi) r.hi = p1 + 1;
  r.lo = window > 0 && p0 - window + 1 > 0 ? p0 - window + 1 : 0;
  return r;
}

constexpr int kKvTile = 32;  // keys a wavefront takes at a time (two 16-key halves, one page each)

MOE_HD int kv4_tiles(const Kv4Range &r) {
  return r.hi > r.lo ? (int)((r.hi + kKvTile - 1) / kKvTile - r.lo / kKvTile) : 0;
}

// The share of one of `splits` workgroups that take a range's tiles `per` at a
// time: tiles begin .. end - 1 of the sequence; `used` splits have any. per is
// raised to what leaves no tile over.
struct Kv4Share {
  int begin, end, used;
};

MOE_HD Kv4Share kv4_share(const Kv4Range &r, int per, int splits, int split) {
  const int t0 = (int)(r.lo / kKvTile), n = kv4_tiles(r);
  const int least = n / splits + (n % splits != 0);
  if (per < least) per = least;
  if (per < 1) per = 1;
  Kv4Share s;
  s.used = n > 0 ? n / per + (n % per != 0) : 1;
  const long long b = (long long)split * per < n ? (long long)split * per : n;
  const long long e = b + per < n ? b + per : n;
  s.begin = t0 + (int)b;
  s.end = t0 + (int)e;
  return s;
}

// Row tile and (cache head, sequence) that a prompt workgroup takes: the
// workgroups are numbered x = 0 .. n - 1 of hs = 0 .. heads - 1. Every tile of
// every hs is taken exactly once. Causal calls go from the longest tile to the
// shortest; with `pair`, where all workgroups are on the card at once, two to a
// CU, so that those from number 256 on share the CUs of the first 256: tiles of
// all heads are put in one list, longest first, and its second part is turned
// round, so that the longest tile shares its CU with the shortest (us without and
// with, 16 heads on 2: 4096 tokens behind 1003, D = 128 173 and 144, D = 64 without
// earlier ones 104 and 77; 3000 tokens, D = 128 92 and 80; 1500 tokens, 32 on 8 55
// and 47).
struct Kv4Place {
  int tile;
  long long hs;
};

constexpr int kPairCus = 256;

MOE_HD Kv4Place kv4_prompt_place(int x, long long hs, int n, long long heads, bool causal, bool pair) {
  if (!causal) return Kv4Place{x, hs};
  if (!pair || n > 2 * kPairCus || heads > 2 * kPairCus || n * heads > 2 * kPairCus) return Kv4Place{n - 1 - x, hs};
  const int all = n * (int)heads, at = (int)hs * n + x;
  const int rank = at < kPairCus ? at : all - 1 - (at - kPairCus);
  return Kv4Place{n - 1 - rank / (int)heads, rank % (int)heads};
}

#ifdef __HIPCC__
// dtype: 0 bf16, 1 fp32
hipError_t launch_kv4_append(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc,
                             const Kv4Batch &bt, const void *k, const void *v, long long k_stride,
                             long long v_stride, int dtype, hipStream_t s);
hipError_t launch_kv4_read(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc,
                           const Kv4Batch &bt, void *k, void *v, long long k_stride,
                           long long v_stride, int dtype, hipStream_t s);

struct Kv4Attn {
  const uint16_t *q;
  uint16_t *out;
  long long q_stride, out_stride;  // elements between tokens
  int max_new;
  float scale;
  bool causal;
  int window;
  int above, most;  // a kernel's own sequences: those with more query rows a head than above, and at most `most`
  int room;         // partial results lie by sequence, this many tokens each; 0: by row of the call
  int per;          // tiles a workgroup takes of split keys; 0: worked out from the lengths
};

// Bytes of a call's partial results (0 when no keys are split), for T token rows
// of which no sequence has more than max_new; rows: Kv4Batch::rows.
size_t kv4_attention_ws(const Kv4Dims &dm, int T, int max_new, int window, bool rows);
bool kv4_grid_ok(const Kv4Dims &dm, int max_new);
// Sequences of many query rows (n * G), `splits` workgroups to a tile of rows;
// their partial results are joined by the other.
hipError_t launch_kv4_prefill(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc, const Kv4Batch &bt,
                              const Kv4Attn &at, int splits, float *part, hipStream_t s);
hipError_t launch_kv4_attention(const Kv4Dims &dm, const Kv4Plane &kc, const Kv4Plane &vc,
                                const Kv4Batch &bt, const Kv4Attn &at, void *ws, hipStream_t s);
#endif

}  // namespace moe
