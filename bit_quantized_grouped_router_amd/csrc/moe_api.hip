// C ABI of the int4-g64 grouped MoE layer: host-side validation, workspace
// carving and launch sequencing on the caller's stream. No allocation, no
// host synchronisation, no exceptions across the interface.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/moe_w4.h"
#include "moe_kv4.h"
#include "moe_kv4_sparse.h"
#include "moe_launch.h"
#include "moe_linear.h"
#include "moe_norm.h"
#include "moe_rope.h"

using namespace moe;

namespace {

thread_local int32_t g_last_hip_error = 0;

moe_status hip_status(hipError_t e) {
  if (e == hipSuccess) return MOE_OK;
  g_last_hip_error = (int32_t)e;
  return MOE_E_HIP;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// MOE_OK, or the first failing check of a pointer that must be present.
moe_status check_ptr(const void *p) {
  if (p == nullptr) return MOE_E_INVALID;
  if (!aligned16(p)) return MOE_E_ALIGN;
  return MOE_OK;
}

#define MOE_TRY(expr)                   \
  do {                                  \
    const moe_status st_ = (expr);      \
    if (st_ != MOE_OK) return st_;      \
  } while (0)

moe_status check_dims(const moe_dims *dm) {
  if (dm == nullptr) return MOE_E_INVALID;
  if (dm->T < 0 || dm->d <= 0 || dm->f <= 0 || dm->E <= 0 || dm->k <= 0 || dm->f_shared <= 0)
    return MOE_E_INVALID;
  if (dm->k > dm->E) return MOE_E_INVALID;
  // a shared expert of another width is a valid layer these kernels do not run
  if (dm->f_shared != dm->f) return MOE_E_UNSUPPORTED;
  if (dm->d % kGroup != 0 || dm->f % kGroup != 0) return MOE_E_UNSUPPORTED;
  if (dm->E > 1024 || dm->k > 32) return MOE_E_UNSUPPORTED;
  if (dm->d > kGemmMaxK || dm->f > kGemmMaxK) return MOE_E_UNSUPPORTED;
  const long long rows = (long long)dm->T * (dm->k + 1);
  const long long big = dm->d > 2 * dm->f ? dm->d : 2 * dm->f;
  if (rows * big >= (1ll << 31) || (long long)dm->E * 2 * dm->f * dm->d >= (1ll << 34))
    return MOE_E_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_matrix(const moe_w4_matrix &m) {
  MOE_TRY(check_ptr(m.codes));
  MOE_TRY(check_ptr(m.scales));
  MOE_TRY(check_ptr(m.biases));
  return MOE_OK;
}

moe_status check_weights(const moe_w4_weights *w, bool up, bool down) {
  if (w == nullptr) return MOE_E_INVALID;
  if (up) {
    MOE_TRY(check_matrix(w->w13));
    MOE_TRY(check_matrix(w->s13));
  }
  if (down) {
    MOE_TRY(check_matrix(w->w2));
    MOE_TRY(check_matrix(w->s2));
  }
  return MOE_OK;
}

// Shapes the router projection takes: d a multiple of 64 (one K step), E up to
// 1024, and x, Wr and the logits each under 2^31 elements.
moe_status check_router_dims(int32_t T, int32_t d, int32_t E) {
  if (T < 0 || d <= 0 || E <= 0) return MOE_E_INVALID;
  if (d % kGroup != 0 || E > 1024) return MOE_E_UNSUPPORTED;
  if ((long long)T * d >= (1ll << 31) || (long long)E * d >= (1ll << 31) ||
      (long long)T * E >= (1ll << 31))
    return MOE_E_UNSUPPORTED;
  return MOE_OK;
}

Dims to_dims(const moe_dims *dm) { return Dims{dm->T, dm->d, dm->f, dm->E, dm->k}; }

W4 to_w4(const moe_w4_matrix &m) { return W4{m.codes, m.scales, m.biases}; }

Weights to_weights(const moe_w4_weights *w) {
  return Weights{to_w4(w->w13), to_w4(w->w2), to_w4(w->s13), to_w4(w->s2)};
}

hipStream_t as_stream(void *s) { return (hipStream_t)s; }

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Carving of the layer workspace. With base == nullptr only sizes are computed.
struct LayerWs {
  int32_t *ids, *counts, *offsets, *sorted_token, *row_of, *tile_map, *num_tiles, *block_counts;
  float *wts, *o_shared, *logits;
  uint16_t *h, *o_routed;
  size_t bytes;
};

template <typename P>
P *take(char *base, size_t &off, size_t count) {
  P *p = base ? (P *)(base + off) : nullptr;
  off += align256(count * sizeof(P));
  return p;
}

LayerWs carve_layer(const Dims &dm, char *base) {
  LayerWs w{};
  size_t off = 0;
  const size_t tk = (size_t)dm.T * dm.k;
  w.ids = take<int32_t>(base, off, tk);
  w.wts = take<float>(base, off, tk);
  w.counts = take<int32_t>(base, off, dm.E);
  w.offsets = take<int32_t>(base, off, dm.E + 1);
  w.sorted_token = take<int32_t>(base, off, tk);
  w.row_of = take<int32_t>(base, off, tk);
  w.tile_map = take<int32_t>(base, off, (size_t)tile_capacity(dm) * 4);
  w.num_tiles = take<int32_t>(base, off, 4);
  w.block_counts = take<int32_t>(base, off, (size_t)perm_blocks(dm.T) * dm.E);
  w.h = take<uint16_t>(base, off, (tk + dm.T) * (size_t)dm.f);
  w.o_routed = take<uint16_t>(base, off, tk * (size_t)dm.d);
  w.o_shared = take<float>(base, off, (size_t)dm.T * dm.d);
  w.logits = take<float>(base, off, (size_t)dm.T * dm.E);  // router scores (hidden-state entry)
  w.bytes = off;
  return w;
}

// A stride between rows of `row` elements that must stay 16-byte aligned.
moe_status check_stride(int64_t stride, int64_t row) {
  if (stride < row) return MOE_E_INVALID;
  return stride % 8 != 0 ? MOE_E_UNSUPPORTED : MOE_OK;
}

moe_status check_dtype(int32_t dtype) {
  return dtype == MOE_BF16 || dtype == MOE_F32 ? MOE_OK : MOE_E_INVALID;
}

// Shapes of the 4-bit cache; Hq only matters to the attention.
moe_status check_kv4_dims(const moe_kv4_dims *dm, int32_t T, bool queries) {
  if (dm == nullptr || T < 0) return MOE_E_INVALID;
  if (dm->B <= 0 || dm->Hkv <= 0 || dm->D <= 0 || dm->page <= 0 || dm->num_pages <= 0 ||
      dm->max_pages <= 0)
    return MOE_E_INVALID;
  if (queries && (dm->Hq <= 0 || dm->Hq % dm->Hkv != 0)) return MOE_E_INVALID;
  if (dm->D != 64 && dm->D != 128 && dm->D != 256) return MOE_E_UNSUPPORTED;
  if (dm->page < 16 || dm->page > 65536 || (dm->page & (dm->page - 1)) != 0) return MOE_E_UNSUPPORTED;
  if ((long long)dm->max_pages * dm->page >= (1ll << 31)) return MOE_E_UNSUPPORTED;
  if (dm->B > 65535 || dm->Hkv > 65535 || (queries && dm->Hq > 65535)) return MOE_E_UNSUPPORTED;
  if ((long long)T * 2 * dm->Hkv * dm->D >= (1ll << 40)) return MOE_E_UNSUPPORTED;
  return MOE_OK;
}

Kv4Dims to_kv4_dims(const moe_kv4_dims *dm) {
  return Kv4Dims{dm->B, dm->Hq, dm->Hkv, dm->D, dm->page, __builtin_ctz((unsigned)dm->page),
                 dm->num_pages, dm->max_pages};
}

moe_status check_kv4_plane(const moe_kv4_plane &p) {
  MOE_TRY(check_ptr(p.codes));
  MOE_TRY(check_ptr(p.scales));
  return check_ptr(p.biases);
}

moe_status check_kv4_cache(const moe_kv4_cache *c, const moe_kv4_batch *b) {
  if (c == nullptr || b == nullptr) return MOE_E_INVALID;
  MOE_TRY(check_kv4_plane(c->k));
  MOE_TRY(check_kv4_plane(c->v));
  MOE_TRY(check_ptr(b->page_table));
  MOE_TRY(check_ptr(b->cu));
  return check_ptr(b->kv_len);
}

// An output at the address of one of the cache's planes or of the batch's arrays.
bool at_kv4_cache(const void *p, const moe_kv4_cache *c, const moe_kv4_batch *b) {
  for (const moe_kv4_plane *pl : {&c->k, &c->v})
    if (p == pl->codes || p == pl->scales || p == pl->biases) return true;
  return p == b->page_table || p == b->cu || p == b->kv_len;
}

Kv4Plane to_kv4_plane(const moe_kv4_plane &p) { return Kv4Plane{p.codes, p.scales, p.biases}; }

Kv4Batch to_kv4_batch(const moe_kv4_batch *b, int32_t T) {
  return Kv4Batch{b->page_table, b->cu, b->kv_len, T, false};
}

// max_new as the kernels take it: no sequence has more new tokens than there
// are rows.
int kv4_max_new(int32_t T, int32_t max_new) { return max_new < T ? max_new : T; }

moe_status check_kv4_attention(const moe_kv4_dims *dm, int32_t T, int32_t max_new, int32_t window) {
  MOE_TRY(check_kv4_dims(dm, T, true));
  if (max_new < 0 || (max_new == 0 && T > 0) || window < 0) return MOE_E_INVALID;
  if ((long long)T * dm->Hq >= (1ll << 31) - 64) return MOE_E_UNSUPPORTED;
  if (T > 0 && !kv4_grid_ok(to_kv4_dims(dm), kv4_max_new(T, max_new))) return MOE_E_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_rope(const moe_rope_spec *r, int32_t D) {
  if (r == nullptr || r->rot < 2 || r->rot > D || r->rot % 2 != 0) return MOE_E_INVALID;
  return check_ptr(r->freqs);
}

bool eps_ok(float eps) { return eps > 0.0f && std::isfinite(eps); }

moe_status check_head_norm(const moe_head_norm *n) {
  if (n == nullptr) return MOE_OK;
  if (!eps_ok(n->eps)) return MOE_E_INVALID;
  return check_ptr(n->weight);
}

Rope to_rope(const moe_rope_spec *r) { return Rope{r->freqs, r->rot, r->interleaved != 0, r->magnitude}; }

HeadNorm to_head_norm(const moe_head_norm *n) {
  return n == nullptr ? HeadNorm{nullptr, 1.0f, false} : HeadNorm{n->weight, n->eps, n->plus_one != 0};
}

moe_status check_kv4_sparse(const moe_kv4_dims *dm, int32_t T, int32_t max_new, const moe_kv4_pages *p) {
  MOE_TRY(check_kv4_attention(dm, T, max_new, 0));
  if (p == nullptr || p->top < 0 || p->first < 0 || p->recent < 1) return MOE_E_INVALID;
  if ((long long)p->top + p->first + p->recent > kSelectMostTaken) return MOE_E_UNSUPPORTED;
  if (dm->max_pages > kSelectMostPages || dm->Hq / dm->Hkv > 64) return MOE_E_UNSUPPORTED;
  return MOE_OK;
}

// Scratch of moe_layer_forward_noalloc: one copy per GPU, loaded with the
// library's code object and held until the process ends. Host code never uses
// the array's name as an address (on the host it is a stand-in, not device
// memory): each device's address comes from hipGetSymbolAddress, taken once
// per device with that device current, and is kept below.
static __device__ __align__(256) uint8_t scratch[MOE_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void *g_scratch_ptr[kMaxDevices] = {};

// This device's address of the scratch array (looked up on the first call).
moe_status scratch_address(void **out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_status(e);
  if (dev < 0 || dev >= kMaxDevices) return MOE_E_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_ptr[dev] == nullptr) {
    void *p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return hip_status(e);
    if (p == nullptr || ((uintptr_t)p & 255u) != 0) return MOE_E_ALIGN;
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return MOE_OK;
}

}  // namespace

extern "C" {

const char *moe_status_string(int32_t st) {
  switch (st) {
    case MOE_OK: return "ok";
    case MOE_E_INVALID: return "invalid argument";
    case MOE_E_UNSUPPORTED: return "unsupported shape";
    case MOE_E_ALIGN: return "pointer not 16-byte aligned";
    case MOE_E_WORKSPACE: return "workspace too small";
    case MOE_E_HIP: return "HIP error";
    default: return "unknown status";
  }
}

int32_t moe_last_hip_error(void) { return g_last_hip_error; }

int32_t moe_block_m(void) { return kBlockM; }

int32_t moe_tile_capacity(const moe_dims *dm) {
  if (check_dims(dm) != MOE_OK) return -1;
  return tile_capacity(to_dims(dm));
}

size_t moe_permute_workspace_bytes(const moe_dims *dm) {
  if (check_dims(dm) != MOE_OK) return 0;
  return (size_t)perm_blocks(dm->T) * dm->E * sizeof(int32_t);
}

size_t moe_layer_workspace_bytes(const moe_dims *dm) {
  if (check_dims(dm) != MOE_OK) return 0;
  return carve_layer(to_dims(dm), nullptr).bytes;
}

moe_status moe_route(const float *logits, int32_t T, int32_t E, int32_t k, int32_t *topk_ids,
                     float *topk_w, void *stream) {
  if (T < 0 || E <= 0 || k <= 0 || k > E) return MOE_E_INVALID;
  if (E > 1024 || k > 32) return MOE_E_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  MOE_TRY(check_ptr(logits));
  MOE_TRY(check_ptr(topk_ids));
  MOE_TRY(check_ptr(topk_w));
  return hip_status(launch_route(logits, T, E, k, topk_ids, topk_w, as_stream(stream)));
}

moe_status moe_permute(const moe_dims *dm, const int32_t *topk_ids, int32_t *counts,
                       int32_t *offsets, int32_t *sorted_token, int32_t *row_of,
                       int32_t *tile_map, int32_t *num_tiles, void *ws, size_t ws_bytes,
                       void *stream) {
  MOE_TRY(check_dims(dm));
  if (dm->T == 0) return MOE_OK;
  MOE_TRY(check_ptr(topk_ids));
  MOE_TRY(check_ptr(counts));
  MOE_TRY(check_ptr(offsets));
  MOE_TRY(check_ptr(sorted_token));
  MOE_TRY(check_ptr(row_of));
  MOE_TRY(check_ptr(tile_map));
  MOE_TRY(check_ptr(num_tiles));
  MOE_TRY(check_ptr(ws));
  if (ws_bytes < moe_permute_workspace_bytes(dm)) return MOE_E_WORKSPACE;
  return hip_status(launch_permute(to_dims(dm), topk_ids, counts, offsets, sorted_token, row_of,
                                   tile_map, num_tiles, (int32_t *)ws, as_stream(stream)));
}

moe_status moe_route_permute(const moe_dims *dm, const float *logits, int32_t *topk_ids,
                             float *topk_w, int32_t *counts, int32_t *offsets,
                             int32_t *sorted_token, int32_t *row_of, int32_t *tile_map,
                             int32_t *num_tiles, void *ws, size_t ws_bytes, void *stream) {
  MOE_TRY(check_dims(dm));
  if (dm->T == 0) return MOE_OK;
  MOE_TRY(check_ptr(logits));
  MOE_TRY(check_ptr(topk_ids));
  MOE_TRY(check_ptr(topk_w));
  MOE_TRY(check_ptr(counts));
  MOE_TRY(check_ptr(offsets));
  MOE_TRY(check_ptr(sorted_token));
  MOE_TRY(check_ptr(row_of));
  MOE_TRY(check_ptr(tile_map));
  MOE_TRY(check_ptr(num_tiles));
  MOE_TRY(check_ptr(ws));
  if (ws_bytes < moe_permute_workspace_bytes(dm)) return MOE_E_WORKSPACE;
  return hip_status(launch_route_permute(to_dims(dm), logits, topk_ids, topk_w, counts, offsets,
                                         sorted_token, row_of, tile_map, num_tiles,
                                         (int32_t *)ws, as_stream(stream)));
}

moe_status moe_expert_gate_up_w4(const moe_dims *dm, const uint16_t *x, const moe_w4_weights *w,
                                 const int32_t *sorted_token, const int32_t *tile_map,
                                 const int32_t *num_tiles, uint16_t *h, void *stream) {
  MOE_TRY(check_dims(dm));
  if (dm->T == 0) return MOE_OK;
  MOE_TRY(check_weights(w, true, false));
  MOE_TRY(check_ptr(x));
  MOE_TRY(check_ptr(sorted_token));
  MOE_TRY(check_ptr(tile_map));
  MOE_TRY(check_ptr(num_tiles));
  MOE_TRY(check_ptr(h));
  return hip_status(launch_gate_up(to_dims(dm), x, to_weights(w), sorted_token, tile_map,
                                   num_tiles, h, as_stream(stream)));
}

moe_status moe_expert_down_w4(const moe_dims *dm, const uint16_t *h, const moe_w4_weights *w,
                              const int32_t *tile_map, const int32_t *num_tiles,
                              uint16_t *o_routed, float *o_shared, void *stream) {
  MOE_TRY(check_dims(dm));
  if (dm->T == 0) return MOE_OK;
  MOE_TRY(check_weights(w, false, true));
  MOE_TRY(check_ptr(h));
  MOE_TRY(check_ptr(tile_map));
  MOE_TRY(check_ptr(num_tiles));
  MOE_TRY(check_ptr(o_routed));
  MOE_TRY(check_ptr(o_shared));
  return hip_status(launch_down(to_dims(dm), h, to_weights(w), tile_map, num_tiles, o_routed,
                                o_shared, as_stream(stream)));
}

moe_status moe_expert_ffn_w4(const moe_dims *dm, const uint16_t *x, const moe_w4_weights *w,
                             const int32_t *sorted_token, const int32_t *tile_map,
                             const int32_t *num_tiles, uint16_t *h, uint16_t *o_routed,
                             float *o_shared, void *stream) {
  MOE_TRY(check_dims(dm));
  if (dm->T == 0) return MOE_OK;
  MOE_TRY(check_weights(w, true, true));
  MOE_TRY(check_ptr(o_routed));
  MOE_TRY(check_ptr(o_shared));
  MOE_TRY(moe_expert_gate_up_w4(dm, x, w, sorted_token, tile_map, num_tiles, h, stream));
  return moe_expert_down_w4(dm, h, w, tile_map, num_tiles, o_routed, o_shared, stream);
}

moe_status moe_unpermute_combine(const moe_dims *dm, const uint16_t *o_routed,
                                 const float *o_shared, const float *topk_w,
                                 const int32_t *row_of, float *y, void *stream) {
  MOE_TRY(check_dims(dm));
  if (dm->T == 0) return MOE_OK;
  MOE_TRY(check_ptr(o_routed));
  MOE_TRY(check_ptr(o_shared));
  MOE_TRY(check_ptr(topk_w));
  MOE_TRY(check_ptr(row_of));
  MOE_TRY(check_ptr(y));
  return hip_status(
      launch_combine(to_dims(dm), o_routed, o_shared, topk_w, row_of, y, as_stream(stream)));
}

// The layer from logits on; arguments already validated.
static moe_status enqueue_layer(const Dims &d, const uint16_t *x, const float *logits, const Weights &W,
                         float *y, const LayerWs &L, hipStream_t s) {
  if (decode_supported(d))
    return hip_status(launch_decode(d, x, logits, W, L.ids, L.wts, L.h, y, s));
  MOE_TRY(hip_status(launch_route_permute(d, logits, L.ids, L.wts, L.counts, L.offsets,
                                          L.sorted_token, L.row_of, L.tile_map, L.num_tiles,
                                          L.block_counts, s)));
  MOE_TRY(hip_status(launch_gate_up(d, x, W, L.sorted_token, L.tile_map, L.num_tiles, L.h, s)));
  MOE_TRY(hip_status(launch_down(d, L.h, W, L.tile_map, L.num_tiles, L.o_routed, L.o_shared, s)));
  return hip_status(launch_combine(d, L.o_routed, L.o_shared, L.wts, L.row_of, y, s));
}

moe_status moe_layer_forward(const moe_dims *dm, const uint16_t *x, const float *logits,
                             const moe_w4_weights *w, float *y, void *ws, size_t ws_bytes,
                             void *stream) {
  MOE_TRY(check_dims(dm));
  if (dm->T == 0) return MOE_OK;
  MOE_TRY(check_weights(w, true, true));
  MOE_TRY(check_ptr(x));
  MOE_TRY(check_ptr(logits));
  MOE_TRY(check_ptr(y));
  MOE_TRY(check_ptr(ws));
  const Dims d = to_dims(dm);
  const LayerWs L = carve_layer(d, (char *)ws);
  if (ws_bytes < L.bytes) return MOE_E_WORKSPACE;
  return enqueue_layer(d, x, logits, to_weights(w), y, L, as_stream(stream));
}

moe_status moe_layer_forward_noalloc(const moe_dims *dm, const uint16_t *x, const float *logits,
                                     const moe_w4_weights *w, float *y, void *stream) {
  MOE_TRY(check_dims(dm));
  if (dm->T == 0) return MOE_OK;
  MOE_TRY(check_weights(w, true, true));
  MOE_TRY(check_ptr(x));
  MOE_TRY(check_ptr(logits));
  MOE_TRY(check_ptr(y));
  const Dims d = to_dims(dm);
  // the size check comes before any HIP call
  if (carve_layer(d, nullptr).bytes > (size_t)MOE_NOALLOC_SCRATCH_BYTES) return MOE_E_WORKSPACE;
  void *base = nullptr;
  MOE_TRY(scratch_address(&base));
  const LayerWs L = carve_layer(d, (char *)base);
  return enqueue_layer(d, x, logits, to_weights(w), y, L, as_stream(stream));
}

moe_status moe_router_logits(const uint16_t *x, const uint16_t *w_router, int32_t T, int32_t d,
                             int32_t E, float *logits, void *stream) {
  MOE_TRY(check_router_dims(T, d, E));
  if (T == 0) return MOE_OK;
  MOE_TRY(check_ptr(x));
  MOE_TRY(check_ptr(w_router));
  MOE_TRY(check_ptr(logits));
  return hip_status(launch_router_logits(x, w_router, T, d, E, logits, as_stream(stream)));
}

moe_status moe_layer_forward_hidden(const moe_dims *dm, const uint16_t *x,
                                    const uint16_t *w_router, const moe_w4_weights *w, float *y,
                                    void *ws, size_t ws_bytes, void *stream) {
  MOE_TRY(check_dims(dm));
  if (dm->T == 0) return MOE_OK;
  MOE_TRY(check_router_dims(dm->T, dm->d, dm->E));
  MOE_TRY(check_weights(w, true, true));
  MOE_TRY(check_ptr(x));
  MOE_TRY(check_ptr(w_router));
  MOE_TRY(check_ptr(y));
  MOE_TRY(check_ptr(ws));
  const Dims d = to_dims(dm);
  const LayerWs L = carve_layer(d, (char *)ws);
  if (ws_bytes < L.bytes) return MOE_E_WORKSPACE;
  const hipStream_t s = as_stream(stream);
  MOE_TRY(hip_status(launch_router_logits(x, w_router, d.T, d.d, d.E, L.logits, s)));
  return enqueue_layer(d, x, L.logits, to_weights(w), y, L, s);
}

moe_status moe_dequant_w4(const moe_w4_matrix *m, int32_t rows, int32_t cols, uint16_t *out,
                          void *stream) {
  if (m == nullptr || rows < 0 || cols <= 0) return MOE_E_INVALID;
  if (cols % kGroup != 0) return MOE_E_UNSUPPORTED;
  if ((long long)rows * cols >= (1ll << 34)) return MOE_E_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  MOE_TRY(check_matrix(*m));
  MOE_TRY(check_ptr(out));
  return hip_status(launch_dequant(to_w4(*m), rows, cols, out, as_stream(stream)));
}

moe_status moe_linear_w4(int32_t T, int32_t rows, int32_t cols, const uint16_t *x, int64_t x_stride,
                         const moe_w4_matrix *w, const uint16_t *bias, int32_t act,
                         const void *residual, int64_t residual_stride, void *y, int64_t y_stride,
                         int32_t dtype, void *stream) {
  if (w == nullptr || T < 0 || rows <= 0 || cols <= 0) return MOE_E_INVALID;
  if (act < MOE_ACT_NONE || act > MOE_ACT_GELU) return MOE_E_INVALID;
  MOE_TRY(check_dtype(dtype));
  if (cols % kGroup != 0 || (long long)rows * cols >= (1ll << 34)) return MOE_E_UNSUPPORTED;
  if ((long long)T * rows >= (1ll << 36) || (long long)T * cols >= (1ll << 40)) return MOE_E_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  MOE_TRY(check_stride(x_stride, cols));
  if (y_stride < rows || (residual != nullptr && residual_stride < rows)) return MOE_E_INVALID;
  MOE_TRY(check_ptr(x));
  MOE_TRY(check_matrix(*w));
  if (bias != nullptr) MOE_TRY(check_ptr(bias));
  if (residual != nullptr) MOE_TRY(check_ptr(residual));
  MOE_TRY(check_ptr(y));
  if (residual == y && residual_stride != y_stride) return MOE_E_INVALID;
  const LinearArgs a{T, rows, cols, x, x_stride, to_w4(*w), bias, act, residual, residual_stride, y, y_stride};
  if (!linear_grid_ok(a)) return MOE_E_UNSUPPORTED;
  if (x == y) return MOE_E_INVALID;  // other workgroups still read x
  return hip_status(launch_linear(a, dtype, as_stream(stream)));
}

moe_status moe_kv4_append(const moe_kv4_dims *dm, const moe_kv4_cache *cache, int32_t T,
                          const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                          int32_t dtype, const moe_kv4_batch *batch, void *stream) {
  MOE_TRY(check_kv4_dims(dm, T, false));
  MOE_TRY(check_dtype(dtype));
  if (T == 0) return MOE_OK;
  MOE_TRY(check_stride(k_stride, (int64_t)dm->Hkv * dm->D));
  MOE_TRY(check_stride(v_stride, (int64_t)dm->Hkv * dm->D));
  MOE_TRY(check_kv4_cache(cache, batch));
  MOE_TRY(check_ptr(k));
  MOE_TRY(check_ptr(v));
  return hip_status(launch_kv4_append(to_kv4_dims(dm), to_kv4_plane(cache->k), to_kv4_plane(cache->v),
                                      to_kv4_batch(batch, T), k, v, k_stride, v_stride, dtype,
                                      as_stream(stream)));
}

moe_status moe_kv4_read(const moe_kv4_dims *dm, const moe_kv4_cache *cache, int32_t T, void *k,
                        int64_t k_stride, void *v, int64_t v_stride, int32_t dtype,
                        const moe_kv4_batch *batch, void *stream) {
  MOE_TRY(check_kv4_dims(dm, T, false));
  MOE_TRY(check_dtype(dtype));
  if (T == 0) return MOE_OK;
  MOE_TRY(check_stride(k_stride, (int64_t)dm->Hkv * dm->D));
  MOE_TRY(check_stride(v_stride, (int64_t)dm->Hkv * dm->D));
  MOE_TRY(check_kv4_cache(cache, batch));
  MOE_TRY(check_ptr(k));
  MOE_TRY(check_ptr(v));
  if (k == v) return MOE_E_INVALID;  // one would be written over the other
  return hip_status(launch_kv4_read(to_kv4_dims(dm), to_kv4_plane(cache->k), to_kv4_plane(cache->v),
                                    to_kv4_batch(batch, T), k, v, k_stride, v_stride, dtype,
                                    as_stream(stream)));
}

size_t moe_kv4_attention_workspace_bytes(const moe_kv4_dims *dm, int32_t T, int32_t max_new,
                                         int32_t window) {
  if (check_kv4_attention(dm, T, max_new, window) != MOE_OK || T == 0) return 0;
  return kv4_attention_ws(to_kv4_dims(dm), T, kv4_max_new(T, max_new), window, false);
}

moe_status moe_kv4_attention(const moe_kv4_dims *dm, const moe_kv4_cache *cache, int32_t T,
                             int32_t max_new, const uint16_t *q, int64_t q_stride, uint16_t *out,
                             int64_t out_stride, const moe_kv4_batch *batch, float scale,
                             int32_t causal, int32_t window, void *ws, size_t ws_bytes,
                             void *stream) {
  MOE_TRY(check_kv4_attention(dm, T, max_new, window));
  if (!(scale > 0.0f) || !(scale <= 0x1p64f)) return MOE_E_INVALID;
  if (T == 0) return MOE_OK;
  MOE_TRY(check_stride(q_stride, (int64_t)dm->Hq * dm->D));
  MOE_TRY(check_stride(out_stride, (int64_t)dm->Hq * dm->D));
  MOE_TRY(check_kv4_cache(cache, batch));
  MOE_TRY(check_ptr(q));
  MOE_TRY(check_ptr(out));
  if (q == out && q_stride != out_stride && T > 1) return MOE_E_INVALID;  // rows would be written over others' queries
  const Kv4Dims d = to_kv4_dims(dm);
  const int n = kv4_max_new(T, max_new);
  const size_t need = kv4_attention_ws(d, T, n, window, false);
  if (need > 0) {
    if (ws_bytes < need) return MOE_E_WORKSPACE;
    MOE_TRY(check_ptr(ws));
  }
  const Kv4Attn at{q, out, q_stride, out_stride, n, scale, causal != 0, window, 0, 0, 0, 0};
  return hip_status(launch_kv4_attention(d, to_kv4_plane(cache->k), to_kv4_plane(cache->v),
                                         to_kv4_batch(batch, T), at, ws, as_stream(stream)));
}

moe_status moe_rmsnorm(int32_t T, int32_t d, const void *x, int64_t x_stride, int32_t x_dtype,
                       const void *residual, int64_t residual_stride, void *h, int64_t h_stride,
                       int32_t h_dtype, const uint16_t *weight, int32_t plus_one, float eps, void *y,
                       int64_t y_stride, int32_t y_dtype, float *scales, int32_t group, void *stream) {
  if (T < 0 || d <= 0 || !eps_ok(eps)) return MOE_E_INVALID;
  MOE_TRY(check_dtype(x_dtype));
  if (residual != nullptr) MOE_TRY(check_dtype(h_dtype));
  if (residual == nullptr && h != nullptr) return MOE_E_INVALID;
  if (y_dtype < MOE_BF16 || y_dtype > MOE_INT8) return MOE_E_INVALID;
  if (d > kNormMaxD) return MOE_E_UNSUPPORTED;
  const bool eight = y_dtype == MOE_E4M3 || y_dtype == MOE_INT8;
  if (eight && (group <= 0 || d % group != 0)) return MOE_E_INVALID;
  if (eight && group != d && group != 64 && group != 128) return MOE_E_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (x_stride < d || y_stride < d || (residual != nullptr && residual_stride < d) || (h != nullptr && h_stride < d))
    return MOE_E_INVALID;
  MOE_TRY(check_ptr(x));
  if (residual != nullptr) MOE_TRY(check_ptr(residual));
  if (h != nullptr) MOE_TRY(check_ptr(h));
  MOE_TRY(check_ptr(weight));
  MOE_TRY(check_ptr(y));
  if (eight) MOE_TRY(check_ptr(scales));
  // rows would be written over others that are still read
  if (y == x && (y_dtype != x_dtype || (y_stride != x_stride && T > 1))) return MOE_E_INVALID;
  if (h != nullptr && h == residual && h_stride != residual_stride && T > 1) return MOE_E_INVALID;
  if (y == weight || (residual != nullptr && y == residual)) return MOE_E_INVALID;
  if (h != nullptr && (h == x || h == y || h == weight)) return MOE_E_INVALID;
  if (eight && (scales == x || scales == residual || scales == h || scales == y || (const void *)scales == weight))
    return MOE_E_INVALID;
  const NormArgs a{T, d, x, x_stride, residual, residual ? residual_stride : 0, h, h ? h_stride : 0, weight, eps,
                   plus_one != 0, y, y_stride, y_dtype, eight ? scales : nullptr, eight ? group : d};
  return hip_status(launch_rmsnorm(a, x_dtype, h_dtype, as_stream(stream)));
}

moe_status moe_rope(int32_t T, int32_t H, int32_t D, const void *x, int64_t x_stride, int32_t x_dtype,
                    const int32_t *positions, const moe_rope_spec *rope, const moe_head_norm *norm,
                    void *out, int64_t out_stride, int32_t out_dtype, void *stream) {
  if (T < 0 || H <= 0 || D <= 0) return MOE_E_INVALID;
  MOE_TRY(check_dtype(x_dtype));
  MOE_TRY(check_dtype(out_dtype));
  if (D % 8 != 0 || D > kRopeMaxD || (long long)H * D >= (1ll << 31)) return MOE_E_UNSUPPORTED;
  if ((long long)T * H >= (1ll << 40) / D) return MOE_E_UNSUPPORTED;
  MOE_TRY(check_rope(rope, D));
  MOE_TRY(check_head_norm(norm));
  if (T == 0) return MOE_OK;
  MOE_TRY(check_stride(x_stride, (int64_t)H * D));
  MOE_TRY(check_stride(out_stride, (int64_t)H * D));
  MOE_TRY(check_ptr(x));
  MOE_TRY(check_ptr(positions));
  MOE_TRY(check_ptr(out));
  if (out == x && (x_dtype != out_dtype || (x_stride != out_stride && T > 1))) return MOE_E_INVALID;
  if (out == positions || out == rope->freqs || (norm != nullptr && out == norm->weight)) return MOE_E_INVALID;
  return hip_status(launch_rope(T, H, D, x, x_stride, x_dtype, positions, to_rope(rope), to_head_norm(norm), out,
                                out_stride, out_dtype, as_stream(stream)));
}

moe_status moe_kv4_rope_append(const moe_kv4_dims *dm, const moe_kv4_cache *cache, int32_t T,
                               const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                               const void *v, int64_t v_stride, int32_t dtype,
                               const moe_rope_spec *rope, const moe_head_norm *q_norm,
                               const moe_head_norm *k_norm, uint16_t *q_out, int64_t q_out_stride,
                               const moe_kv4_batch *batch, void *stream) {
  MOE_TRY(check_kv4_dims(dm, T, true));
  if ((long long)T * dm->Hq >= (1ll << 31) - 64) return MOE_E_UNSUPPORTED;
  MOE_TRY(check_dtype(dtype));
  MOE_TRY(check_rope(rope, dm->D));
  MOE_TRY(check_head_norm(q_norm));
  MOE_TRY(check_head_norm(k_norm));
  if (T == 0) return MOE_OK;
  MOE_TRY(check_stride(q_stride, (int64_t)dm->Hq * dm->D));
  MOE_TRY(check_stride(k_stride, (int64_t)dm->Hkv * dm->D));
  MOE_TRY(check_stride(v_stride, (int64_t)dm->Hkv * dm->D));
  MOE_TRY(check_stride(q_out_stride, (int64_t)dm->Hq * dm->D));
  MOE_TRY(check_kv4_cache(cache, batch));
  MOE_TRY(check_ptr(q));
  MOE_TRY(check_ptr(k));
  MOE_TRY(check_ptr(v));
  MOE_TRY(check_ptr(q_out));
  if (q == q_out && (dtype != MOE_BF16 || (q_stride != q_out_stride && T > 1))) return MOE_E_INVALID;
  // other wavefronts still read or write them
  if (q_out == k || q_out == v || (const void *)q_out == rope->freqs || (q_norm != nullptr && q_out == q_norm->weight) ||
      (k_norm != nullptr && q_out == k_norm->weight) || at_kv4_cache(q_out, cache, batch))
    return MOE_E_INVALID;
  const RopeAppend a{q, k, v, q_stride, k_stride, v_stride, q_out, q_out_stride, to_head_norm(q_norm),
                     to_head_norm(k_norm)};
  return hip_status(launch_kv4_rope_append(to_kv4_dims(dm), to_kv4_plane(cache->k), to_kv4_plane(cache->v),
                                           to_kv4_batch(batch, T), to_rope(rope), a, dtype, as_stream(stream)));
}

moe_status moe_kv4_bounds(const moe_kv4_dims *dm, const moe_kv4_cache *cache, int32_t T,
                          uint16_t *bounds, const moe_kv4_batch *batch, void *stream) {
  MOE_TRY(check_kv4_dims(dm, T, false));
  if (T == 0) return MOE_OK;
  MOE_TRY(check_kv4_cache(cache, batch));
  MOE_TRY(check_ptr(bounds));
  if (at_kv4_cache(bounds, cache, batch)) return MOE_E_INVALID;
  return hip_status(launch_kv4_bounds(to_kv4_dims(dm), to_kv4_plane(cache->k), to_kv4_batch(batch, T), bounds,
                                      as_stream(stream)));
}

size_t moe_kv4_sparse_attention_workspace_bytes(const moe_kv4_dims *dm, int32_t T, int32_t max_new,
                                                const moe_kv4_pages *pages) {
  if (check_kv4_sparse(dm, T, max_new, pages) != MOE_OK || T == 0) return 0;
  const Kv4Select sel{nullptr, nullptr, 0, kv4_max_new(T, max_new), pages->top, pages->first, pages->recent, nullptr};
  return kv4_sparse_ws(to_kv4_dims(dm), T, sel);
}

moe_status moe_kv4_sparse_attention(const moe_kv4_dims *dm, const moe_kv4_cache *cache,
                                    const uint16_t *bounds, int32_t T, int32_t max_new, const uint16_t *q,
                                    int64_t q_stride, uint16_t *out, int64_t out_stride,
                                    const moe_kv4_batch *batch, const moe_kv4_pages *pages, float scale,
                                    int32_t *blocks, void *ws, size_t ws_bytes, void *stream) {
  MOE_TRY(check_kv4_sparse(dm, T, max_new, pages));
  if (!(scale > 0.0f) || !(scale <= 0x1p64f)) return MOE_E_INVALID;
  if (T == 0) return MOE_OK;
  MOE_TRY(check_stride(q_stride, (int64_t)dm->Hq * dm->D));
  MOE_TRY(check_stride(out_stride, (int64_t)dm->Hq * dm->D));
  MOE_TRY(check_kv4_cache(cache, batch));
  MOE_TRY(check_ptr(bounds));
  MOE_TRY(check_ptr(q));
  MOE_TRY(check_ptr(out));
  if (blocks != nullptr) MOE_TRY(check_ptr(blocks));
  if (q == out && q_stride != out_stride && T > 1) return MOE_E_INVALID;  // rows would be written over others' queries
  const Kv4Select sel{bounds, q, q_stride, kv4_max_new(T, max_new), pages->top, pages->first, pages->recent, blocks};
  const Kv4Dims d = to_kv4_dims(dm);
  if (ws_bytes < kv4_sparse_ws(d, T, sel)) return MOE_E_WORKSPACE;
  MOE_TRY(check_ptr(ws));
  // one is written while others are still read
  if (out == bounds || out == ws || at_kv4_cache(out, cache, batch) || ws == q || ws == bounds ||
      at_kv4_cache(ws, cache, batch))
    return MOE_E_INVALID;
  if (blocks != nullptr && ((const void *)blocks == q || (const void *)blocks == out || (const void *)blocks == bounds ||
                            blocks == ws || at_kv4_cache(blocks, cache, batch)))
    return MOE_E_INVALID;
  return hip_status(launch_kv4_sparse(d, to_kv4_plane(cache->k), to_kv4_plane(cache->v), to_kv4_batch(batch, T), sel,
                                      out, out_stride, scale, ws, as_stream(stream)));
}

}  // extern "C"
