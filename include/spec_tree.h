/*
 * spec_tree.h — C ABI of the drafted-tree operators of libspecverify.so.
 *
 * spec_verify.h turns logits into emitted tokens.  These entry points are
 * the steps around it in the same loop, over a paged key/value cache:
 *
 *   spec_beam_select        grows the drafted tree: the best continuations
 *   spec_beam_reorder       over beams and vocabulary, and the beams' states
 *                           in their new order;
 *   spec_tree_attention     attention of the drafted tokens over the cache
 *                           and over their own ancestors;
 *   spec_cache_commit       writes the accepted path's keys and values to
 *                           the cache;
 *   spec_attention_weights  accumulates the attention weight that each
 *                           cached token received;
 *   spec_cache_evict        keeps the tokens of largest weight.
 *
 * The conventions of spec_verify.h hold: pointers are caller-owned DEVICE
 * memory except the host argument structs; nothing is allocated, freed or
 * synchronised; work is enqueued on `stream`; a negative SPEC_ERR_* return
 * enqueues nothing; data errors found on the device go to out_status [B]
 * (may be NULL) as an OR of SPEC_STATUS_* and never trap.  A captured call
 * replays with the contents that its buffers then have.
 *
 * A call's results overlap nothing that it reads, and one another neither,
 * except where an entry point says so: its CTAs do not begin together, and one
 * could find another's results for its arguments.  Scores, lengths, tables and
 * weights that results overlap are refused with SPEC_ERR_SHAPE.
 */
#ifndef SPEC_TREE_H
#define SPEC_TREE_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A third element type: keys, values and queries are SPEC_BF16 or SPEC_F16
   (logits SPEC_F32 or SPEC_BF16). */
enum { SPEC_F16 = 2 };

/* out_status bits beside those of spec_verify.h */
enum {
  SPEC_STATUS_BAD_PAGE = 32, /* a page of the block table outside the cache  */
  SPEC_STATUS_BAD_LEN = 64   /* a length or count below 0, over its bound, or
                                offsets that do not ascend                   */
};

#define SPEC_MAX_TREE 256 /* drafted tokens per request                      */
#define SPEC_MAX_BEAMS 64 /* beams per request, and beams kept               */

/* A paged cache.  Element (layer l, page p, slot t, head h, channel d) of
 * keys and values is at l*s_layer + p*s_page + t*s_slot + h*s_head + d
 * (strides in elements, any order of axes).  Token j of request b is in page
 * block_table[b*ld_table + j / page_size], slot j % page_size.  Both buffers
 * start on 16 bytes, strides are multiples of 8 elements, dim is 64, 96,
 * 128, 192 or 256.  Slots past a request's length may hold anything. */
typedef struct {
  void *k;
  void *v;
  int32_t dtype;     /* SPEC_BF16 or SPEC_F16                                */
  int32_t layers;    /* >= 1                                                 */
  int32_t num_pages; /* >= 1                                                 */
  int32_t page_size; /* >= 1                                                 */
  int32_t heads;     /* key/value heads, >= 1                                */
  int32_t dim;
  int64_t s_layer, s_page, s_slot, s_head;
} spec_cache;

/* -------------------------------------------------------- tree attention
 * Request b drafts n_b = cu_nodes[b+1] - cu_nodes[b] tokens (0 <= n_b <=
 * max_nodes) over ctx_len[b] cached ones.  For node i and query head h, with
 * the key/value head h / (heads_q / cache.heads),
 *
 *   s_j  = scale * q_i . k_j   over the cached keys j and over those drafted
 *                              keys j of the request that node i sees
 *   lse  = log sum_j exp(s_j),   out = sum_j exp(s_j - lse) v_j.
 *
 * A node sees drafted key j where bit j % 32 of word j / 32 of its row of
 * tree_mask is set (its ancestors and itself, as a rule); without a mask, the
 * nodes form a chain and see j <= i.  A row that sees nothing gives out 0
 * and lse -inf.  What a row does not see never reaches it, NaN and
 * infinities included.  Statistics and sums are fp32; the weights are rounded
 * to the cache's type for their product with the values (unnormalised, the
 * row's running maximum between 1 and 2^8; with SPEC_F16 weights below 2^-14
 * round to multiples of 2^-24), the result once more.  The divisor may hold the
 * largest weight of every 64 keys as rounded.  So with p_j = exp(s_j - lse) an
 * output is off by at most half a step of sum_j p_j |v_j| + 2 |out|, beside what
 * fp32 sums and exponentials add.
 *
 * A request with a bad length or page gets its status, and NaN in its rows
 * of out and lse. */
typedef struct {
  int32_t B;
  int32_t total_nodes; /* cu_nodes[B]                                        */
  int32_t max_nodes;   /* <= SPEC_MAX_TREE                                   */
  int32_t heads_q;     /* a multiple of cache.heads                          */
  int32_t layer;       /* the layer of the cache that is read                */
  float scale;
  const int32_t *cu_nodes;                      /* [B+1]                     */
  const void *q;                                /* [total_nodes, heads_q, dim] */
  int64_t sq_node, sq_head;
  const void *k_new, *v_new;                    /* [total_nodes, heads, dim]   */
  int64_t sn_node, sn_head;
  const uint32_t *tree_mask;                    /* [total_nodes, mask_words] or NULL */
  int32_t mask_words;                           /* >= ceil(max_nodes / 32)   */
  int32_t ld_table;                             /* pages per row of the table */
  spec_cache cache;
  const int32_t *block_table;                   /* [B, ld_table]             */
  const int32_t *ctx_len;                       /* [B], <= ld_table * page_size */
} spec_tree_args;

/* Workspace of spec_tree_attention (256-byte aligned, any contents; calls
   that share one are ordered).  0 for arguments that the call refuses. */
size_t spec_tree_workspace_bytes(const spec_tree_args *args);

/* out [total_nodes, heads_q, dim] of the cache's type through its strides,
   out_lse [total_nodes, heads_q] fp32 or NULL. */
int spec_tree_attention(const spec_tree_args *args, void *out, int64_t so_node, int64_t so_head, float *out_lse,
                        int32_t *out_status, void *workspace, size_t ws_bytes, spec_stream_t stream);

/* ----------------------------------------------------- attention weights
 * The rows are the last n_b = cu_rows[b+1] - cu_rows[b] tokens of a cache of
 * kv_len[b] tokens: row i sees keys j <= kv_len[b] - n_b + i.  With their
 * lse (as spec_tree_attention gave it; a row whose lse is infinite, -inf where
 * it saw nothing, adds nothing),
 *
 *   out[b, h, j] = before[b, h, j] + sum over rows i and the query heads of
 *                  key head h of exp(scale * q_i . k_j - lse_i),
 *
 * for j < kv_len[b], and 0 from there to ld - 1.  `before` may be NULL (0)
 * or `out` itself.  Sums are fp32 in a fixed order.  A request with a bad
 * length (n_b over its length, the length over ld or the table) gets its
 * status, and NaN in all of out[b]; one with a bad page its status, and NaN
 * for the keys of that page. */
typedef struct {
  int32_t B;
  int32_t total_rows;
  int32_t max_rows;   /* bound on every n_b                                  */
  int32_t heads_q;
  int32_t layer;
  float scale;
  const int32_t *cu_rows;  /* [B+1]                                          */
  const void *q;           /* [total_rows, heads_q, dim]                     */
  int64_t sq_row, sq_head;
  const float *lse;        /* [total_rows, heads_q]                          */
  spec_cache cache;        /* its values are not read                        */
  const int32_t *block_table;
  const int32_t *kv_len;   /* [B]                                            */
  int32_t ld_table;
  int32_t ld;              /* row length of before and out, [B, heads, ld]   */
} spec_weigh_args;

int spec_attention_weights(const spec_weigh_args *args, const float *before, float *out, int32_t *out_status,
                           spec_stream_t stream);

/* -------------------------------------------------------------- eviction
 * Per request and key/value head, keeps m_b = min(kv_len[b], keep) tokens of
 * a layer: the first `sink`, the last `recent`, and of the others those of
 * largest weight (ties to the lowest position; NaN below everything), and
 * moves their keys and values, in their order, to positions 0 .. m_b - 1 of
 * the pages in to_table.  These pages belong to the same cache and to no
 * token that is still to be read.
 *
 * out_index [B, heads, keep]: the kept positions ascending, then -1;
 * out_kept [B, heads, keep] (may be NULL): their weights, then 0; out_len
 * [B] = m_b (may be kv_len itself).  A request with a bad length or page gets
 * its status and out_len -1, index -1, kept 0, and nothing of it is moved. */
typedef struct {
  int32_t B;
  int32_t keep;   /* >= sink + recent, >= 1                                  */
  int32_t sink;
  int32_t recent;
  int32_t layer;
  int32_t ld;     /* row length of weights [B, heads, ld]                    */
  const float *weights;
  const int32_t *kv_len;      /* [B], <= ld                                  */
  spec_cache cache;
  const int32_t *block_table; /* [B, ld_table]                               */
  const int32_t *to_table;    /* [B, ld_to]                                  */
  int32_t ld_table;
  int32_t ld_to;              /* ld_to * page_size >= keep                   */
} spec_evict_args;

int spec_cache_evict(const spec_evict_args *args, int32_t *out_index, float *out_kept, int32_t *out_len,
                     int32_t *out_status, spec_stream_t stream);

/* ---------------------------------------------------- the accepted path
 * Writes node path[b, i] of request b (i < path_len[b] <= ld_path) to token
 * ctx_len[b] + i of every layer of the cache; out_len[b] = ctx_len[b] +
 * path_len[b] (out_len may be ctx_len itself).  A request with a bad length, a
 * node outside its tree or a bad page gets its status and out_len -1, and
 * nothing of it is written. */
typedef struct {
  int32_t B;
  int32_t total_nodes;
  const int32_t *cu_nodes;           /* [B+1]                                */
  const void *k_new, *v_new;         /* [layers, total_nodes, heads, dim]    */
  int64_t sn_layer, sn_node, sn_head;
  const int32_t *path;               /* [B, ld_path]                         */
  const int32_t *path_len;           /* [B]                                  */
  spec_cache cache;
  const int32_t *block_table;        /* [B, ld_table]                        */
  const int32_t *ctx_len;            /* [B]                                  */
  int32_t ld_path;
  int32_t ld_table;
} spec_commit_args;

int spec_cache_commit(const spec_commit_args *args, int32_t *out_len, int32_t *out_status, spec_stream_t stream);

/* ------------------------------------------------------------- the beams
 * Beam w of request b has logits row b*W + w and score scores[b, w].  Its
 * continuation by token v has the score
 *
 *   scores[b, w] + z_v - log sum_u exp(z_u);
 *
 * an ended beam (finished[b, w] != 0) has one continuation, end_token, with
 * its own score.  The logits of an ended beam, and of one of score -inf, are
 * not read.  Kept are the `keep` best continuations of a request, best first,
 * ties to the lowest w*V + v.  Where there are fewer (a score of -inf, logits of
 * -inf), the rest has score -inf, parent -1 and token -1.  Scores are compared
 * in 64 bits (row sums of fp32 exponentials, within 2^-21 of the score), so
 * continuations of different beams whose scores are nearer than that, or equal,
 * may take either order, and rounded once.  The only finite logit of a row, or
 * one that all others leave no bit of, leaves the beam's score as it is.  A NaN or +inf logit that is read, or
 * such a score, gives the request SPEC_STATUS_BAD_LOGITS, scores -inf, parents
 * and tokens -1; a logit from 2.3e38 on, which leaves fp32 once scaled by
 * log2(e), counts as +inf. */
typedef struct {
  int32_t B;
  int32_t W;           /* beams, 1 .. SPEC_MAX_BEAMS                         */
  int32_t keep;        /* 1 .. SPEC_MAX_BEAMS                                */
  int32_t V;
  int32_t dtype;       /* SPEC_F32 or SPEC_BF16                              */
  int32_t end_token;   /* in [0, V) where finished is given                  */
  const void *logits;  /* [B*W, ld], as in spec_verify.h                     */
  int64_t ld;
  const float *scores;       /* [B, W]                                       */
  const int32_t *finished;   /* [B, W] or NULL                               */
} spec_beam_args;

size_t spec_beam_workspace_bytes(const spec_beam_args *args);

int spec_beam_select(const spec_beam_args *args, float *out_scores, int32_t *out_parents, int32_t *out_tokens,
                     int32_t *out_status, void *workspace, size_t ws_bytes, spec_stream_t stream);

/* One state of the beams: `outer` blocks (layers; 1 as a rule) of [B, W]
   rows of row_bytes.  Strides in bytes. */
typedef struct {
  const void *src;
  void *dst;
  int64_t row_bytes;
  int64_t src_outer, src_batch, src_beam;
  int64_t dst_outer, dst_batch, dst_beam;
  int32_t outer;
  int32_t pad;
} spec_beam_state;

#define SPEC_MAX_STATES 8

/* dst[o, b, j] = src[o, b, parents[b, j]] for every state, in one launch;
   rows whose parent is outside [0, W) become zero.  A dst overlaps no src. */
int spec_beam_reorder(int32_t B, int32_t W, int32_t keep, const int32_t *parents, const spec_beam_state *states,
                      int32_t num_states, spec_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SPEC_TREE_H */
