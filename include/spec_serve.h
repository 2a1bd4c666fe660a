/*
 * spec_serve.h — C ABI of the operators of libspecverify.so that stand beside
 * the drafted-tree ones of spec_tree.h, in the same loop:
 *
 *   spec_norm_rotate         norms the heads of queries and keys and rotates
 *                            them to their positions, what every drafted token
 *                            needs before its attention;
 *   spec_window_attention    spec_tree_attention with a sliding window and a
 *                            few first tokens (sinks) that stay visible;
 *   spec_cache8_attention    spec_tree_attention over a cache held in 8 bits
 *                            with a scale for each block of tokens and head,
 *                            with or without a window;
 *   spec_cache8_commit       writes the accepted path's (or a prompt's) keys
 *                            and values to such a cache.
 *
 * The conventions of spec_tree.h hold; an 8-bit cache's scales are among what
 * results that overlap it are refused for.
 */
#ifndef SPEC_SERVE_H
#define SPEC_SERVE_H

#include "spec_tree.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------- norms and positions
 * For every row r and head h of q and of k,
 *
 *   y_d = x_d / sqrt(mean_d(x_d^2) + eps) * weight_d,
 *
 * and the first `rot` channels turn by pairs (a, b), pair i < rot / 2 by the
 * angle positions[r] * inv_freq[i]:
 *
 *   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin),
 *
 * a = i and b = i + rot / 2, or with `interleaved` a = 2 i and b = 2 i + 1.
 * The others stay as normed.  Everything is fp32 and rounded once; angles are
 * reduced exactly (64-bit fractions of a turn), within 2^-24 of a turn beside
 * the rounding of the result for positions below 2^28 and frequencies below 2^20
 * in size.  An infinite or NaN frequency makes its pairs NaN.
 *
 * q or k may have 0 heads.  A result may take the place of its own input (the
 * same pointer and strides); other overlaps of results are refused, and so are
 * results whose own rows or heads overlap (a stride of 0 over several, say: inputs
 * may have it). */
typedef struct {
  int32_t rows;
  int32_t heads_q, heads_k;
  int32_t dim;             /* 64, 96, 128, 192 or 256                        */
  int32_t rot;             /* channels that turn, a multiple of 8, <= dim    */
  int32_t interleaved;
  int32_t dtype;           /* SPEC_BF16 or SPEC_F16, of q, k, weights and results */
  float eps;               /* >= 0                                           */
  const void *q;           /* [rows, heads_q, dim]                           */
  int64_t sq_row, sq_head; /* strides in elements, multiples of 8            */
  const void *k;           /* [rows, heads_k, dim]                           */
  int64_t sk_row, sk_head;
  const void *q_weight, *k_weight; /* [dim], on 16 bytes; NULL: ones         */
  const int32_t *positions;        /* [rows]                                 */
  const float *inv_freq;           /* [rot / 2], radians                     */
} spec_rotate_args;

int spec_norm_rotate(const spec_rotate_args *args, void *out_q, int64_t oq_row, int64_t oq_head, void *out_k,
                     int64_t ok_row, int64_t ok_head, spec_stream_t stream);

/* ------------------------------------------------- a window with sinks
 * What a node sees under spec_tree_attention, the cached tokens and after them
 * the drafted ones that its mask has, in order, is its own text.  Here it sees
 * the first `sinks` and the last `window` tokens of that text only.
 *
 * Of a request's cache the first `sinks` tokens and those from ctx_len - window
 * on may be read; the pages that hold none of these, and their entries of the
 * table, are not.  All else is as in spec_tree_attention. */
typedef struct {
  spec_tree_args tree;
  int32_t window; /* >= 1                                                    */
  int32_t sinks;  /* >= 0                                                    */
} spec_window_args;

size_t spec_window_workspace_bytes(const spec_window_args *args);

int spec_window_attention(const spec_window_args *args, void *out, int64_t so_node, int64_t so_head, float *out_lse,
                          int32_t *out_status, void *workspace, size_t ws_bytes, spec_stream_t stream);

/* ------------------------------------------------------ an 8-bit cache
 * Keys and values are e4m3 bytes, addressed as in spec_cache by strides in
 * bytes (multiples of 16, buffers on 16 bytes).  Token slot t of page p has
 * for layer l and head h the scale at
 *
 *   l*c_layer + p*c_page + (t / block)*c_block + h*c_head
 *
 * of k_scale and of v_scale (strides in elements); its key is the bytes'
 * values times that scale.  Scales are not negative and at most 2^60; a
 * value's scale below 2^-60 counts as 0, and bytes of NaN are NaN under any.
 * Slots past a request's length, and scales of blocks past it, may hold
 * anything. */
typedef struct {
  void *k;
  void *v;
  float *k_scale;
  float *v_scale;
  int32_t layers;    /* >= 1                                                 */
  int32_t num_pages; /* >= 1                                                 */
  int32_t page_size; /* >= 1                                                 */
  int32_t heads;     /* key/value heads, >= 1                                */
  int32_t dim;       /* 64, 96, 128, 192 or 256                              */
  int32_t block;     /* tokens per scale, divides page_size                  */
  int64_t s_layer, s_page, s_slot, s_head;
  int64_t c_layer, c_page, c_block, c_head;
} spec_cache8;

/* spec_tree_attention (window 0) or spec_window_attention over such a cache.
 * Queries, drafted keys and values and results are of `dtype`.
 *
 * Heads of 64 and 128 channels, with pages and blocks of a multiple of 16 tokens
 * and a positive scale, go to the tensor-memory kernel, all else to warp tiles,
 * which read the keys anew for every 16 query rows of a key head: 64 requests of
 * up to 9 nodes over up to 8192 tokens, 28 / 4 heads of 128, take 467 us with
 * blocks of 8 tokens and 116 with blocks of 16.
 *
 * Products run on fp16 operands that hold the bytes' values, and queries and
 * drafted keys and values, exactly: bf16 rows are scaled by powers of two
 * first, and what is below 2^-31 of a query row's largest finite size, or of that
 * of 16 drafted keys or values, is rounded within 2^-39 of it (of sizes below
 * 2^-46, within 2^-85).  Weights, times
 * the scale of their values, are rounded to fp16 relative to the row's largest
 * such product (at least 2^6 of 2^16, smallest step 2^-24), so with p_j =
 * exp(s_j - lse) an output is off by at most 2^-11 (1 + 2^-19) sum_j p_j |v_j|
 * and half a step of its own rounding, beside what fp32 sums and exponentials
 * add and 2^-31 of the largest p_j vs_j for every key.  Keys whose p_j vs_j (a
 * scale that counts as 0: 2^-60) is below 2^-118 of the row's largest may be left
 * out of the sum and of lse as well.  An infinity whose weight is that small gives
 * the row an infinity or NaN. */
typedef struct {
  int32_t B;
  int32_t total_nodes; /* cu_nodes[B]                                        */
  int32_t max_nodes;   /* <= SPEC_MAX_TREE                                   */
  int32_t heads_q;     /* a multiple of cache.heads                          */
  int32_t layer;
  float scale;
  int32_t dtype;       /* SPEC_BF16 or SPEC_F16                              */
  int32_t window;      /* 0: none                                            */
  int32_t sinks;       /* 0 without a window                                 */
  int32_t mask_words;
  const int32_t *cu_nodes;                        /* [B+1]                   */
  const void *q;                                  /* [total_nodes, heads_q, dim] */
  int64_t sq_node, sq_head;
  const void *k_new, *v_new;                      /* [total_nodes, heads, dim]   */
  int64_t sn_node, sn_head;
  const uint32_t *tree_mask;                      /* [total_nodes, mask_words] or NULL */
  spec_cache8 cache;
  const int32_t *block_table;                     /* [B, ld_table]           */
  const int32_t *ctx_len;                         /* [B]                     */
  int32_t ld_table;
  int32_t pad;
} spec_cache8_args;

size_t spec_cache8_workspace_bytes(const spec_cache8_args *args);

int spec_cache8_attention(const spec_cache8_args *args, void *out, int64_t so_node, int64_t so_head, float *out_lse,
                          int32_t *out_status, void *workspace, size_t ws_bytes, spec_stream_t stream);

/* Writes node path[b, i] of request b (i < path_len[b] <= ld_path) to token
 * ctx_len[b] + i of every layer; out_len[b] = ctx_len[b] + path_len[b] (out_len
 * may be ctx_len itself).  A path may be a prompt: nodes 0 .. n - 1.
 *
 * For every block of tokens and head that gets new ones, for keys and for
 * values alike: `need` is the smallest power of two, from 2^-126 on, whose
 * 448-fold reaches the largest finite size of the new tokens' channels (0 where
 * these are all 0; above 2^60, which attention's bounds end at, for sizes above
 * 448 2^60).  A block that holds tokens before ctx_len keeps its scale s
 * unless need > s; then `need` is its scale, and the bytes of its earlier
 * tokens become e4m3(value * s * (1 / need)).  In other blocks the scale is
 * `need`.  New bytes are e4m3(x * (1 / scale)), to nearest, ties to even (0 for
 * a scale below 2^-126, under which all new ones are 0); infinities and NaN
 * become NaN.  Slots of other tokens keep their bytes.
 *
 * A page that gets tokens belongs to one request.  A request with a bad
 * length, a node outside its tree or a bad page gets its status and out_len -1,
 * and nothing of it is written. */
typedef struct {
  int32_t B;
  int32_t total_nodes;
  int32_t dtype;                     /* of k_new and v_new                   */
  int32_t ld_path;
  const int32_t *cu_nodes;           /* [B+1]                                */
  const void *k_new, *v_new;         /* [layers, total_nodes, heads, dim]    */
  int64_t sn_layer, sn_node, sn_head;
  const int32_t *path;               /* [B, ld_path]                         */
  const int32_t *path_len;           /* [B]                                  */
  spec_cache8 cache;
  const int32_t *block_table;        /* [B, ld_table]                        */
  const int32_t *ctx_len;            /* [B]                                  */
  int32_t ld_table;
  int32_t pad;
} spec_cache8_commit_args;

int spec_cache8_commit(const spec_cache8_commit_args *args, int32_t *out_len, int32_t *out_status,
                       spec_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SPEC_SERVE_H */
