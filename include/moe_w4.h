/*
 * moe_w4.h - C ABI of the MI355X (gfx950) int4-g64 grouped MoE expert layer.
 *
 * The layer is the one the noticiai.com.br page on Perplexity's Lily engine
 * describes for Qwen3.6-35B-A3B:
 *   - section "O modelo em tres formatos de carga": a router scores E = 256
 *     experts and keeps k = 8 per token; one shared expert sees every token;
 *   - section "Prefill e decode: onde estao os ganhos": expert weights are
 *     4-bit affine codes in groups of 64 that share one bf16 scale and one
 *     bf16 bias; they are rebuilt to bf16 one tile at a time inside the
 *     grouped GEMM and accumulated in fp32; the routing histogram, prefix
 *     scan, scatter and block map run on the GPU with no CPU synchronisation
 *     inside the layer; at batch-1 decode the layer is bandwidth bound.
 *
 * Conventions for every entry point
 *   - Every tensor pointer is a DEVICE pointer, allocated and owned by the
 *     caller. The library never allocates, frees, copies to the host or
 *     synchronises. Scratch space comes from a caller workspace.
 *   - `stream` is a hipStream_t (NULL = the default stream). All work is
 *     enqueued on it in order and the call returns without waiting.
 *   - Arguments are validated on the host before anything is enqueued. On a
 *     failed check a negative moe_status is returned and nothing is enqueued.
 *     A failed kernel launch returns MOE_E_HIP (moe_last_hip_error() has the
 *     hipError_t). Faults inside kernels surface at the caller's next sync.
 *   - T == 0 is valid: the call returns MOE_OK and enqueues nothing.
 *   - Every pointer must be 16-byte aligned (MOE_E_ALIGN otherwise).
 *   - Outputs must not alias inputs.
 *   - No C++ exception crosses this interface. Apart from a thread-local last
 *     error and the device scratch of moe_layer_forward_noalloc (with its
 *     per-device address table), the library holds no mutable state, so calls
 *     on different streams or threads are safe when their buffers do not
 *     overlap.
 *   - bf16 tensors are passed as uint16_t bit patterns.
 *
 * Shapes (moe_dims)
 *   T tokens, d hidden size, f routed expert width, f_shared the shared
 *   expert's width, E routed experts, k experts chosen per token.
 *   Limits: T >= 0, d % 64 == 0, f % 64 == 0, d <= 6144, f <= 6144,
 *   1 <= k <= min(E, 32), 1 <= E <= 1024, T*(k+1) < 2^31 and every tensor
 *   under 2^31 elements. f_shared must equal f (a different shared width is
 *   a valid layer this version does not run: MOE_E_UNSUPPORTED; f_shared <= 0
 *   is MOE_E_INVALID).
 *
 * Weight layout (moe_w4_matrix), canonical and unshuffled
 *   codes  uint8 [n][rows][cols/2]: column c of a row is byte c>>1, in the
 *          low nibble when c is even and the high nibble when c is odd;
 *   scales bf16  [n][rows][cols/64]: group j covers columns 64j .. 64j+63;
 *   biases bf16  [n][rows][cols/64];
 *   weight w = bf16_rne( fp32( s * q + b ) ), q the unsigned code 0..15.
 *   Matrices are stored [out][in]: groups run along the input dimension.
 *
 * Permuted rows
 *   The T*k token-expert assignments are sorted by expert (stable in token
 *   order) into rows 0 .. T*k-1; the shared expert owns rows T*k .. T*k+T-1,
 *   row T*k+t holding token t. Intermediate tensors h and o are indexed by
 *   these rows.
 */
#ifndef MOE_W4_H
#define MOE_W4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_E_INVALID = -1,     /* null pointer, negative or inconsistent size */
  MOE_E_UNSUPPORTED = -2, /* a valid shape outside the limits above */
  MOE_E_ALIGN = -3,       /* a pointer is not 16-byte aligned */
  MOE_E_WORKSPACE = -4,   /* workspace smaller than the *_workspace_bytes figure */
  MOE_E_HIP = -5          /* a HIP call failed; see moe_last_hip_error() */
} moe_status;

typedef struct {
  int32_t T;        /* tokens */
  int32_t d;        /* hidden size (input of gate/up, output of down) */
  int32_t f;        /* routed expert intermediate width */
  int32_t E;        /* routed experts */
  int32_t k;        /* experts chosen per token */
  int32_t f_shared; /* shared expert intermediate width; must equal f */
} moe_dims;

typedef struct {
  const uint8_t *codes;   /* [n][rows][cols/2] packed 4-bit codes */
  const uint16_t *scales; /* [n][rows][cols/64] bf16 */
  const uint16_t *biases; /* [n][rows][cols/64] bf16 */
} moe_w4_matrix;

typedef struct {
  moe_w4_matrix w13; /* routed gate|up: n = E, rows = 2f (gate rows 0..f-1, up rows f..2f-1), cols = d */
  moe_w4_matrix w2;  /* routed down:    n = E, rows = d, cols = f */
  moe_w4_matrix s13; /* shared gate|up: n = 1, rows = 2 f_shared, cols = d */
  moe_w4_matrix s2;  /* shared down:    n = 1, rows = d, cols = f_shared */
} moe_w4_weights;

/*
 * moe_router_logits - the router's score of every expert for every token
 * (page section "O modelo em tres formatos de carga": the router scores the
 * E experts), as a bias-free projection of the hidden states:
 *   logits[t][e] = sum_c x[t][c] * w_router[e][c]
 * Products of two bf16 values are exact in fp32; they are summed in fp32, on
 * the matrix cores above 128 tokens and as dot products on the vector units
 * up to 128 (the summation order is unspecified but fixed, so results may
 * differ from another fp32 order by rounding, within d * 2^-24 * sum_c |x w|,
 * and repeat bit for bit).
 *   x         bf16 [T][d]   hidden states
 *   w_router  bf16 [E][d]   router matrix
 *   logits    fp32 [T][E]   out
 * Limits: T >= 0, d % 64 == 0, 1 <= E <= 1024, and T*d, E*d and T*E each
 * under 2^31 (MOE_E_INVALID for negative or zero sizes, MOE_E_UNSUPPORTED
 * past the limits).
 */
moe_status moe_router_logits(const uint16_t *x, const uint16_t *w_router, int32_t T, int32_t d,
                             int32_t E, float *logits, void *stream);

/*
 * moe_route - top-k selection and router weights
 * (page section "O modelo em tres formatos de carga": score E experts, keep k).
 *   logits   fp32  [T][E]  router logits
 *   topk_ids int32 [T][k]  out: chosen experts, by logit descending; equal
 *                          logits go to the lower expert index; -0 == +0
 *   topk_w   fp32  [T][k]  out: softmax over the k chosen logits
 * One wavefront per token. Preconditions (not checked on the device): no NaN
 * and at least k finite logits per token; if violated, the ids are still k
 * distinct values in [0, E) and the weights are unspecified.
 */
moe_status moe_route(const float *logits, int32_t T, int32_t E, int32_t k,
                     int32_t *topk_ids, float *topk_w, void *stream);

/* Rows per tile of the block map (the M tile height of the grouped GEMMs). */
int32_t moe_block_m(void);

/* Upper bound on the number of tiles of the block map; rows of tile_map to allocate. */
int32_t moe_tile_capacity(const moe_dims *dm);

/* Bytes of scratch workspace moe_permute needs (may be 0). */
size_t moe_permute_workspace_bytes(const moe_dims *dm);

/*
 * moe_permute - routing histogram, exclusive prefix scan, stable scatter and
 * tile block map, all on the device, no host synchronisation
 * (page section "Prefill e decode: onde estao os ganhos").
 *   topk_ids     int32 [T][k]         from moe_route
 *   counts       int32 [E]            out: rows per expert
 *   offsets      int32 [E+1]          out: exclusive scan, offsets[E] = T*k
 *   sorted_token int32 [T*k]          out: token of each permuted row
 *   row_of       int32 [T*k]          out: permuted row of assignment t*k+j
 *   tile_map     int32 [cap][4]       out: {group, row_begin, row_end, sched}
 *                                     per tile, cap = moe_tile_capacity(dm);
 *                                     groups 0..E-1 in order, then the shared
 *                                     group E (rows T*k .. T*k+T-1); each group
 *                                     split into ceil(count/BM) tiles of at most
 *                                     BM = moe_block_m() rows. sched of row i is
 *                                     the index of the i-th tile in the order
 *                                     the grouped GEMMs run them (position i
 *                                     on XCD i % 8), a permutation of
 *                                     0..num_tiles-1: first the F full tiles,
 *                                     in tile order cut into 8 runs whose
 *                                     lengths differ by at most one (longer
 *                                     runs first), the r-th tile of run x at
 *                                     position 8r + x; then the partial tiles,
 *                                     tallest first, equal heights in tile
 *                                     order. Entries past num_tiles are left
 *                                     untouched.
 *   num_tiles    int32 [1]            out: tiles written
 *   ws, ws_bytes                      scratch, >= moe_permute_workspace_bytes(dm)
 * Deterministic: the row order does not depend on scheduling.
 * Precondition: every id in [0, E) and distinct within a token (as
 * moe_route produces).
 */
moe_status moe_permute(const moe_dims *dm, const int32_t *topk_ids, int32_t *counts,
                       int32_t *offsets, int32_t *sorted_token, int32_t *row_of,
                       int32_t *tile_map, int32_t *num_tiles, void *ws, size_t ws_bytes,
                       void *stream);

/*
 * moe_route_permute - moe_route followed by moe_permute, with the same
 * outputs bit for bit. Up to 64 tokens the permutation is a single
 * one-workgroup launch (histogram, scan, block map and scatter together),
 * which removes most of the fixed cost of the routing at small batches; the
 * top-k runs in the same launch while it is short (at most 16 selection
 * rounds per wavefront, e.g. up to 32 tokens at k = 8 and E <= 256), and in
 * the moe_route kernel just before it otherwise.
 *   logits                      fp32 [T][E]
 *   topk_ids, topk_w            out, as moe_route
 *   counts .. num_tiles         out, as moe_permute
 *   ws, ws_bytes                as moe_permute
 */
moe_status moe_route_permute(const moe_dims *dm, const float *logits, int32_t *topk_ids,
                             float *topk_w, int32_t *counts, int32_t *offsets,
                             int32_t *sorted_token, int32_t *row_of, int32_t *tile_map,
                             int32_t *num_tiles, void *ws, size_t ws_bytes, void *stream);

/*
 * moe_expert_gate_up_w4 - grouped gate/up GEMM over the block map with the
 * int4-g64 dequantisation fused into the tile (the weights' bf16 MFMA
 * operands rebuilt in registers one K step at a time, fp32 accumulation; page
 * section "Prefill e decode: onde estao os ganhos"), and SiLU(gate)*up in the
 * epilogue. The block map may also be built by the caller: tiles of at most
 * moe_block_m() rows of one group, in moe_permute's layout, with a schedule
 * column that is a permutation of the tile indices.
 *   x            bf16  [T][d]
 *   sorted_token int32 [T*k], tile_map, num_tiles from moe_permute
 *   h            bf16  [T*k+T][f] out: h[p] = bf16(silu(gate_p) * up_p), with
 *                gate_p = W13_g[0:f] x_t and up_p = W13_g[f:2f] x_t for row p
 *                of group g carrying token t
 */
moe_status moe_expert_gate_up_w4(const moe_dims *dm, const uint16_t *x,
                                 const moe_w4_weights *w, const int32_t *sorted_token,
                                 const int32_t *tile_map, const int32_t *num_tiles,
                                 uint16_t *h, void *stream);

/*
 * moe_expert_down_w4 - grouped down GEMM, same fused dequantisation.
 *   h         bf16 [T*k+T][f] from moe_expert_gate_up_w4
 *   o_routed  bf16 [T*k][d]   out: W2_g h_p for the routed rows (rounded to bf16)
 *   o_shared  fp32 [T][d]     out: S2 h_p for the shared rows, row T*k+t -> t
 */
moe_status moe_expert_down_w4(const moe_dims *dm, const uint16_t *h, const moe_w4_weights *w,
                              const int32_t *tile_map, const int32_t *num_tiles,
                              uint16_t *o_routed, float *o_shared, void *stream);

/* moe_expert_ffn_w4 - moe_expert_gate_up_w4 followed by moe_expert_down_w4. */
moe_status moe_expert_ffn_w4(const moe_dims *dm, const uint16_t *x, const moe_w4_weights *w,
                             const int32_t *sorted_token, const int32_t *tile_map,
                             const int32_t *num_tiles, uint16_t *h, uint16_t *o_routed,
                             float *o_shared, void *stream);

/*
 * moe_unpermute_combine - weighted unpermute plus the shared expert
 * (page section "O modelo em tres formatos de carga": the shared expert sees
 * every token; it is added with weight 1).
 *   y[t] = o_shared[t] + sum_j topk_w[t][j] * o_routed[row_of[t*k+j]], fp32
 *   o_routed bf16 [T*k][d], o_shared fp32 [T][d], topk_w fp32 [T][k],
 *   row_of int32 [T*k], y fp32 [T][d] (out)
 */
moe_status moe_unpermute_combine(const moe_dims *dm, const uint16_t *o_routed,
                                 const float *o_shared, const float *topk_w,
                                 const int32_t *row_of, float *y, void *stream);

/* Bytes of workspace moe_layer_forward and moe_layer_forward_hidden need for
 * these dims. */
size_t moe_layer_workspace_bytes(const moe_dims *dm);

/*
 * moe_layer_forward - the whole layer on one stream with no host sync:
 * route, permute, gate/up, down, combine, or, for up to 16 tokens, the
 * decode path (two launches, one grid row per token: routing recomputed on
 * chip, each token's k + 1 experts' 4-bit weights streamed with 128-bit loads;
 * page section "Prefill e decode: onde estao os ganhos": at small batches
 * bandwidth sets the ceiling). The two paths agree within rounding; the
 * workspace's routing and permutation buffers are only written by the
 * first.
 *   x      bf16 [T][d]
 *   logits fp32 [T][E]
 *   y      fp32 [T][d] out
 *   ws     >= moe_layer_workspace_bytes(dm) bytes of device scratch
 */
moe_status moe_layer_forward(const moe_dims *dm, const uint16_t *x, const float *logits,
                             const moe_w4_weights *w, float *y, void *ws, size_t ws_bytes,
                             void *stream);

/* Bytes of the library's own device scratch array used by
 * moe_layer_forward_noalloc (one array per GPU the library runs on). */
#define MOE_NOALLOC_SCRATCH_BYTES (64u << 20)

/*
 * moe_layer_forward_noalloc - moe_layer_forward for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation): the same kernels and results, with the
 * scratch taken from a device array the library owns instead of a caller
 * workspace. The call allocates nothing.
 *   x, logits, w, y  as moe_layer_forward (the caller still owns all of them)
 * Limits: the layer's scratch (moe_layer_workspace_bytes of the dims) must fit
 * in MOE_NOALLOC_SCRATCH_BYTES = 64 MiB, otherwise MOE_E_WORKSPACE is returned
 * before any HIP call. At d = 2048, f = 512, E = 256, k = 8 that is T <= 1307
 * (every T that takes the decode path fits).
 * The array: one per GPU, loaded with the library's code object and kept until
 * the process ends; its device address is looked up (hipGetSymbolAddress) on
 * the first call on each device, with that device current, so the stream must
 * belong to the current device. Every call on a GPU shares that GPU's array and
 * leaves its contents behind; nothing in it has to start at zero (every piece
 * is written before it is read within a call). Calls that may overlap on one
 * GPU (two streams, two threads, two captured graphs replayed concurrently)
 * race on the array: order them, or use moe_layer_forward with separate
 * workspaces.
 */
moe_status moe_layer_forward_noalloc(const moe_dims *dm, const uint16_t *x, const float *logits,
                                     const moe_w4_weights *w, float *y, void *stream);

/*
 * moe_layer_forward_hidden - moe_layer_forward starting from hidden states:
 * moe_router_logits into the workspace, then the layer on those logits (the
 * same kernels, small batches included). Every argument is validated before the
 * first launch.
 *   x         bf16 [T][d]
 *   w_router  bf16 [E][d]
 *   y         fp32 [T][d] out
 *   ws        >= moe_layer_workspace_bytes(dm) bytes of device scratch
 */
moe_status moe_layer_forward_hidden(const moe_dims *dm, const uint16_t *x,
                                    const uint16_t *w_router, const moe_w4_weights *w, float *y,
                                    void *ws, size_t ws_bytes, void *stream);

/*
 * moe_dequant_w4 - rebuild one int4-g64 matrix to bf16 with the same device
 * arithmetic the GEMM tiles use (for inspection and tests).
 *   m     one matrix (n = 1) of rows x cols, cols % 64 == 0
 *   out   bf16 [rows][cols]
 */
moe_status moe_dequant_w4(const moe_w4_matrix *m, int32_t rows, int32_t cols, uint16_t *out,
                          void *stream);

/* Element types of the entry points below that take more than one. */
typedef enum { MOE_BF16 = 0, MOE_F32 = 1 } moe_dtype;

/* Activations of moe_linear_w4: z; max(z, 0); z / (1 + exp(-z));
 * z * erfc(-z / sqrt 2) / 2. */
typedef enum { MOE_ACT_NONE = 0, MOE_ACT_RELU = 1, MOE_ACT_SILU = 2, MOE_ACT_GELU = 3 } moe_act;

/*
 * moe_linear_w4 - a dense projection with int4-g64 weights and its epilogue
 * (the q, k, v and output projections around the attention below, or any
 * dense layer of the same checkpoint format):
 *   y[t][n] = act(sum_c x[t][c] * W[n][c] + bias[n]) + residual[t][n]
 * The weights are rebuilt to bf16 as in the expert GEMMs, products are exact
 * and summed in fp32 in a fixed order; the epilogue is fp32 and y is rounded
 * once.
 *   x         bf16 [T][cols], rows x_stride elements apart
 *   w         one matrix (n = 1) of rows x cols
 *   bias      bf16 [rows] or NULL
 *   residual  [T][rows] of y's type, rows residual_stride apart, or NULL; may
 *             be y itself with the same stride (updated in place)
 *   y         bf16 or fp32 (dtype) [T][rows], rows y_stride elements apart, out;
 *             overlaps neither x (MOE_E_INVALID at its address) nor, but for the
 *             above, the residual
 * Limits: T >= 0, rows >= 1, cols >= 1 (MOE_E_INVALID otherwise); cols % 64 == 0,
 * x_stride % 8 == 0, rows * cols < 2^34, T * rows < 2^36, T * cols < 2^40, T <=
 * 2^31 - 2176, and fewer than 2^23 - 8 blocks of 16 rows (T <= 16) or of 16 rows by
 * 32 tokens (x_stride or cols >= 2^23) (MOE_E_UNSUPPORTED); strides at least a row
 * long (MOE_E_INVALID).
 */
moe_status moe_linear_w4(int32_t T, int32_t rows, int32_t cols, const uint16_t *x, int64_t x_stride,
                         const moe_w4_matrix *w, const uint16_t *bias, int32_t act,
                         const void *residual, int64_t residual_stride, void *y, int64_t y_stride,
                         int32_t dtype, void *stream);

/*
 * A paged key/value cache held in int4-g64: keys and values are each a stack
 * of num_pages * Hkv matrices in the weight layout above, with `page` rows (one
 * per token slot) of D columns, i.e.
 *   codes  uint8 [num_pages][Hkv][page][D/2]
 *   scales, biases  bf16 [num_pages][Hkv][page][D/64]
 * so moe_dequant_w4 shows what a page's head holds.
 */
typedef struct {
  int32_t B;         /* sequences of the batch */
  int32_t Hq;        /* query heads, a multiple of Hkv (attention only) */
  int32_t Hkv;       /* key/value heads */
  int32_t D;         /* channels of a head: 64, 128 or 256 */
  int32_t page;      /* tokens per page: a power of two, 16 .. 65536 */
  int32_t num_pages; /* pages of the cache */
  int32_t max_pages; /* columns of the page table */
} moe_kv4_dims;

typedef struct {
  uint8_t *codes;
  uint16_t *scales;
  uint16_t *biases;
} moe_kv4_plane;

typedef struct {
  moe_kv4_plane k, v;
} moe_kv4_cache;

/*
 * The batch, in device memory and the same for append, read and attention.
 * Sequence b has kv_len[b] tokens, the last n_b = cu[b+1] - cu[b] of which are
 * rows cu[b] .. cu[b+1]-1 of the call's token tensors (T rows in all); position
 * p of the sequence lies in page page_table[b][p / page], slot p % page.
 *   page_table  int32 [B][max_pages]; entries past the sequence's pages are not used
 *   cu          int32 [B+1], ascending from 0
 *   kv_len      int32 [B]
 * Nothing a kernel reads here can make it leave its buffers: offsets are
 * clamped to 0 .. T, and a position that is negative, past the table, or on
 * a page outside 0 .. num_pages-1 has no place in the cache (not written, read
 * back as zeros, not attended to). Rows past cu[B] are not touched.
 */
typedef struct {
  const int32_t *page_table;
  const int32_t *cu;
  const int32_t *kv_len;
} moe_kv4_batch;

/*
 * Shape limits of the three calls: B, Hkv, page, num_pages, max_pages >= 1, D
 * and page as above, T >= 0 (MOE_E_INVALID for values < 1, MOE_E_UNSUPPORTED
 * for other D and page), max_pages * page < 2^31, B, Hq, Hkv <= 65535, T * Hq <
 * 2^31 - 64, max_new * Hq / Hkv < 2^28 - 128 (attention), T * 2 Hkv D < 2^40. Token strides are in elements, multiples of 8
 * (MOE_E_UNSUPPORTED) and at least a token long (MOE_E_INVALID).
 */

/*
 * moe_kv4_append - quantise the new tokens' keys and values into the cache.
 * Per group of 64 channels x: b = bf16(min x), a zero as +0; s = bf16(fp32((max x -
 * b) * fp32(1/15))) or 0 below 2^-126; code = (x - b) / s rounded to nearest, ties
 * to even, and clamped to 0 .. 15 (0 where s = 0); max x - b and x - b are
 * rounded to fp32, the quotient is not. A group that holds a NaN or an
 * infinity, or whose span or bias overflows, is stored as s = b = NaN.
 *   k, v  bf16 or fp32 (dtype) [T][Hkv][D], tokens k_stride / v_stride apart
 * Precondition: the new tokens lie in different slots (two tokens in one slot
 * leave a mixture of the two there).
 */
moe_status moe_kv4_append(const moe_kv4_dims *dm, const moe_kv4_cache *cache, int32_t T,
                          const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                          int32_t dtype, const moe_kv4_batch *batch, void *stream);

/*
 * moe_kv4_read - rebuild the same tokens' keys and values, scale * code + bias,
 * rounded to fp32 and for bf16 once more (n_b = kv_len[b] reads a whole
 * sequence).
 *   k, v  bf16 or fp32 (dtype) [T][Hkv][D], out, tokens k_stride / v_stride apart; they
 *         do not overlap (MOE_E_INVALID at one address)
 */
moe_status moe_kv4_read(const moe_kv4_dims *dm, const moe_kv4_cache *cache, int32_t T, void *k,
                        int64_t k_stride, void *v, int64_t v_stride, int32_t dtype,
                        const moe_kv4_batch *batch, void *stream);

/* Bytes of workspace moe_kv4_attention needs (may be 0; 0 for arguments out of range). */
size_t moe_kv4_attention_workspace_bytes(const moe_kv4_dims *dm, int32_t T, int32_t max_new,
                                         int32_t window);

/*
 * moe_kv4_attention - the new tokens' queries over the cache (their own keys and
 * values included, so append first).
 *   out[t][h] = sum_p softmax_p(scale * q[t][h] . k_p) v_p, with k_p, v_p =
 *   s * code + b of cache head h / (Hq / Hkv), over the positions
 *   p < kv_len that the token at position i sees: p <= i if causal, and
 *   p > i - window if window > 0. A token that sees none gets zeros (and so does one
 *   whose scores are all -infinity in fp32). Positions
 *   it does not see never reach its result, whatever the cache holds there.
 *   q       bf16 [T][Hq][D], tokens q_stride apart
 *   out     bf16 [T][Hq][D], out, tokens out_stride apart; may be q itself with the
 *           same stride (MOE_E_INVALID with another), and overlaps nothing else
 *   max_new an upper bound of every n_b; a sequence's tokens past it are not computed
 *   scale   > 0 and <= 2^64 (MOE_E_INVALID otherwise)
 *   window  >= 0 (0: none; MOE_E_INVALID when negative)
 *   ws      >= moe_kv4_attention_workspace_bytes of these dims; may be NULL when that
 *           is 0. Calls that may overlap need workspaces of their own.
 * Scores, softmax statistics and sums are fp32. What is rounded for the matrix
 * cores, by the sizes of the call:
 *   few query rows: a softmax weight times its key's scale, to bf16; keys and
 *     values enter unrounded.
 *   many (T * Hq >= 4096, T * Hq * positions of the page table or the window >=
 *     2^25, and more than 64 rows max_new * Hq / Hkv of a cache head): keys, values and
 *     weights, to fp16; to bf16 for a block of rows whose keys, values or
 *     queries fp16's range does not hold (2^15 and more, or scales below 2^-13), or
 *     whose scores times scale log2(e) pass 2^23.
 * Sums are divided at the end: while scales and biases are below 2^80 they cannot
 * overflow; larger values may come back as infinities or NaN, in their group of 64
 * channels, for the tokens that see them.
 * Results repeat bit for bit. The calls are asynchronous and may be captured.
 */
moe_status moe_kv4_attention(const moe_kv4_dims *dm, const moe_kv4_cache *cache, int32_t T,
                             int32_t max_new, const uint16_t *q, int64_t q_stride, uint16_t *out,
                             int64_t out_stride, const moe_kv4_batch *batch, float scale,
                             int32_t causal, int32_t window, void *ws, size_t ws_bytes,
                             void *stream);

/*
 * moe_rmsnorm - root-mean-square norm of rows, with the residual's addition before
 * it (a block's input norm, the norm between attention and the experts):
 *   s = x + residual;  h = s in the residual's type;
 *   y = s / sqrt(sum_c s[c]^2 / d + eps) * w,  w = weight, or 1 + weight (plus_one)
 * in fp32 (the norm is that of the unrounded sum), each output rounded once.
 * 8-bit outputs hold y / scale: for each row and `group` channels a = max |y|, scale
 * = a / 448 (MOE_E4M3, without infinities, bias 7) or a / 127 (MOE_INT8), the quotient
 * rounded to nearest, ties to even; a group of zeros has scale 0, one that holds a
 * NaN or an infinity scale NaN and codes 0.
 *   x         bf16 or fp32 (x_dtype) [T][d]
 *   residual  bf16 or fp32 (h_dtype) [T][d], or NULL
 *   h         h_dtype [T][d], out, or NULL (not stored; MOE_E_INVALID without a
 *             residual); may be the residual itself with the same stride
 *   weight    bf16 [d]
 *   y         MOE_BF16, MOE_F32, MOE_E4M3 or MOE_INT8 (y_dtype) [T][d], out; may be x
 *             itself with the same type and stride
 *   scales    fp32 [T][d / group], out, for 8-bit outputs (NULL otherwise)
 *   group     64 or 128 (d a multiple), or d: one scale a row; 8-bit outputs only
 * Other overlaps of outputs are not allowed (MOE_E_INVALID at one address). Strides
 * are in elements and at least a row long (MOE_E_INVALID); any d and any strides
 * run, multiples of 8 fast. Squares are summed in fp32: a row whose sum of squares
 * passes its range has norm infinity.
 * Limits: 1 <= d <= 32768, eps > 0 and finite (MOE_E_INVALID otherwise).
 */
typedef enum { MOE_E4M3 = 2, MOE_INT8 = 3 } moe_dtype8;

moe_status moe_rmsnorm(int32_t T, int32_t d, const void *x, int64_t x_stride, int32_t x_dtype,
                       const void *residual, int64_t residual_stride, void *h, int64_t h_stride,
                       int32_t h_dtype, const uint16_t *weight, int32_t plus_one, float eps, void *y,
                       int64_t y_stride, int32_t y_dtype, float *scales, int32_t group, void *stream);

/*
 * Rotary positions: the first rot channels of a head turn in pairs (a, b) =
 * channels (2i, 2i + 1) if interleaved, (i, i + rot / 2) otherwise, by t = position
 * * freqs[i]:  (a, b) -> magnitude * (a cos t - b sin t, a sin t + b cos t).
 * The other channels pass. t (the whole product) and its cosine and sine are taken in 64
 * bits, the rest in fp32.
 *   freqs  fp32 [rot / 2], radians a position, in device memory
 *   rot    even, 2 .. D
 */
typedef struct {
  const float *freqs;
  int32_t rot;
  int32_t interleaved;
  float magnitude;
} moe_rope_spec;

/* A norm of every head before it turns: x / sqrt(mean x^2 + eps) * w over its D channels,
 * w = weight (bf16 [D]) or 1 + weight; squares are summed in fp32, as in moe_rmsnorm. eps > 0
 * and finite. */
typedef struct {
  const uint16_t *weight;
  float eps;
  int32_t plus_one;
} moe_head_norm;

/*
 * moe_rope - norm (if norm is not NULL) and rotary positions of heads.
 *   x          bf16 or fp32 (x_dtype) [T][H][D], tokens x_stride elements apart
 *   positions  int32 [T], any values
 *   out        bf16 or fp32 (out_dtype) [T][H][D], out; may be x itself with the same
 *              type and stride (MOE_E_INVALID with another), and overlaps nothing else
 * Limits: D % 8 == 0, 8 <= D <= 512, H >= 1, H * D < 2^31, T * H * D < 2^40; strides multiples of 8
 * (MOE_E_UNSUPPORTED) and at least a token long (MOE_E_INVALID).
 */
moe_status moe_rope(int32_t T, int32_t H, int32_t D, const void *x, int64_t x_stride, int32_t x_dtype,
                    const int32_t *positions, const moe_rope_spec *rope, const moe_head_norm *norm,
                    void *out, int64_t out_stride, int32_t out_dtype, void *stream);

/*
 * moe_kv4_rope_append - moe_rope on the new tokens' queries and keys at their
 * positions in the batch's sequences, and moe_kv4_append of the turned keys and the
 * values, in one pass: what the cache holds is bit for bit what moe_kv4_append makes
 * of moe_rope's keys in fp32.
 *   q, k, v   bf16 or fp32 (dtype) [T][Hq][D], [T][Hkv][D], [T][Hkv][D]
 *   q_norm, k_norm  may be NULL
 *   q_out     bf16 [T][Hq][D], out; may be q itself if that is bf16, with the same
 *             stride (MOE_E_INVALID with another), and overlaps nothing else
 *             (MOE_E_INVALID at one address)
 * A token without a place in the cache has its queries turned and nothing written;
 * rows of no sequence are left as they are. Precondition as for moe_kv4_append.
 */
moe_status moe_kv4_rope_append(const moe_kv4_dims *dm, const moe_kv4_cache *cache, int32_t T,
                               const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                               const void *v, int64_t v_stride, int32_t dtype,
                               const moe_rope_spec *rope, const moe_head_norm *q_norm,
                               const moe_head_norm *k_norm, uint16_t *q_out, int64_t q_out_stride,
                               const moe_kv4_batch *batch, void *stream);

/*
 * moe_kv4_bounds - the smallest and the largest key of every channel, for each page
 * that holds one of the call's new tokens, over the page's slots up to the sequence's
 * last token; other pages' bounds are left as they are. Call it after every write (the
 * attention below relies on the bounds of full pages).
 *   bounds  bf16 [num_pages][Hkv][2][D]: smallest, then largest, of the keys as
 *           moe_kv4_read gives them in bf16 (a zero is +0); NaN where a key is. Overlaps
 *           neither cache nor batch (MOE_E_INVALID at one address)
 */
moe_status moe_kv4_bounds(const moe_kv4_dims *dm, const moe_kv4_cache *cache, int32_t T,
                          uint16_t *bounds, const moe_kv4_batch *batch, void *stream);

/* Which pages a token attends to: its own page and those before it, of which the first
 * `first`, the last `recent` (its own among them) and, of the others, the `top` with the
 * best scores. first, top >= 0, recent >= 1 (MOE_E_INVALID otherwise), together at most
 * 4096 (MOE_E_UNSUPPORTED). */
typedef struct {
  int32_t top, first, recent;
} moe_kv4_pages;

/* Bytes of workspace moe_kv4_sparse_attention needs (0 for arguments out of range). */
size_t moe_kv4_sparse_attention_workspace_bytes(const moe_kv4_dims *dm, int32_t T, int32_t max_new,
                                                const moe_kv4_pages *pages);

/*
 * moe_kv4_sparse_attention - causal attention of the new tokens' queries over the pages
 * that each token and cache head selects. The score of a page is the most that any
 * key inside its bounds could score, summed over the query heads of the cache head:
 *   sum_h sum_c max(q[t][h][c] * lo[c], q[t][h][c] * hi[c])
 * summed in 64 bits and rounded to fp32; ties go to the lower page of the sequence, a
 * NaN ranks below every number. 0 times an infinity is NaN, and so is a maximum of which
 * one side is; an infinite bound on the side that is not the larger does not count. Pages
 * that do not exist are not taken.
 *   out[t][h] = moe_kv4_attention's, over the keys of those pages at positions up to the
 *   token's own. Where nothing is left out it is causal attention without a window.
 *   bounds  as moe_kv4_bounds leaves them
 *   blocks  int32 [T][Hkv][first + recent + top], out, or NULL: the pages taken, as their
 *           numbers 0, 1, .. in the sequence, ascending, -1 behind them
 *   other arguments as for moe_kv4_attention; a token past max_new of its sequence, or of
 *   no sequence, is left out (its rows of out and blocks stay as they are). out (unless it
 *   is q), blocks and ws overlap nothing (MOE_E_INVALID at one address)
 * Limits, besides moe_kv4_attention's: max_pages <= 2^20, Hq / Hkv <= 64
 * (MOE_E_UNSUPPORTED).
 */
moe_status moe_kv4_sparse_attention(const moe_kv4_dims *dm, const moe_kv4_cache *cache,
                                    const uint16_t *bounds, int32_t T, int32_t max_new, const uint16_t *q,
                                    int64_t q_stride, uint16_t *out, int64_t out_stride,
                                    const moe_kv4_batch *batch, const moe_kv4_pages *pages, float scale,
                                    int32_t *blocks, void *ws, size_t ws_bytes, void *stream);

const char *moe_status_string(int32_t status);

/* hipError_t of the last MOE_E_HIP on this thread (0 if none). */
int32_t moe_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_W4_H */
