// Parameter blocks and workspace layout of the drafted-tree operators,
// shared by their entry points (tree_ops.cu) and kernels.
#pragma once

#include <cstddef>
#include <cstdint>

namespace sv {

constexpr int kStatusBadPage = 32;
constexpr int kStatusBadLen = 64;

// ---------------------------------------------------------- tree attention
// An item is one key/value head of one request with one block of `rows` of
// its query rows (row r: node r / group, head r % group of the group).  Its
// keys are cut into tiles of `kt`, first the cached ones, then the drafted
// ones.  All tiles of all items in order are cut evenly over the CTAs, so a
// CTA's range may begin and end inside an item.
struct TreeParams {
  const int32_t* cu;
  const int32_t* ctx;
  const int32_t* table;
  const uint32_t* mask;
  const void* q;
  const void* k_new;
  const void* v_new;
  const void* k;   // of the layer
  const void* v;
  long long sq_node, sq_head, sn_node, sn_head, so_node, so_head;
  long long s_page, s_slot, s_head;
  void* out;
  float* lse;      // or null
  int32_t* status; // or null
  float* part_o;   // [2 * grid][dim / 4][rows][4] unnormalised outputs of split items
  float4* part_ml; // [2 * grid][rows] their reference (log2 units), sum of weights, and of weights as rounded
  int32_t* failed; // [grid] whether a wait of a CTA ran out, or null
  long long* start;  // [B + 1] first tile of each request (main kernel to combine)
  float scale_log2;  // scale * log2(e)
  int B, total, max_nodes, mask_words, ld_table;
  int num_pages, page_size, heads, group, dim;
  int grid;        // CTAs of the main kernel
  int rows;        // query rows per item
  int kt;          // keys per tile
  int weigh;       // the rows are the last of the cached tokens: no drafted keys, all rows in one block,
                   // and a request has at most `ld` tokens
  int ld;
};

struct TreeWorkspace {
  size_t off_start, off_failed, off_ml, off_o, total;
};

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

inline TreeWorkspace make_tree_workspace(int B, int grid, int rows, int dim) {
  TreeWorkspace w;
  w.off_start = 0;
  w.off_failed = up256((size_t)(B + 1) * sizeof(long long));
  w.off_ml = w.off_failed + up256((size_t)grid * sizeof(int32_t));
  w.off_o = w.off_ml + up256((size_t)2 * grid * rows * 4 * sizeof(float));
  w.total = w.off_o + up256((size_t)2 * grid * rows * dim * sizeof(float));
  return w;
}

// How a call is run: the kernel, its grid, its rows per item and keys per tile.
struct TreePlan {
  int kernel;   // 0: warp tiles (tree_attn.cu), 1: tensor memory (tree_tc.cu)
  int grid, rows, kt;
};

// ------------------------------------------------------- attention weights
struct WeighParams {
  const int32_t* cu;
  const int32_t* len;
  const int32_t* table;
  const void* q;
  const void* k;
  const float* lse;
  const float* before;
  float* out;
  int32_t* status;
  long long sq_row, sq_head, s_page, s_slot, s_head;
  float scale_log2;
  int B, total, max_rows, ld_table, ld;
  int num_pages, page_size, heads, group, dim;
};

// ------------------------------------------------------ eviction, the path
struct EvictParams {
  const float* weights;
  const int32_t* len;
  const int32_t* table;
  const int32_t* to;
  void* k;
  void* v;
  long long s_page, s_slot, s_head;
  int32_t* index;
  float* kept;      // or null
  int32_t* new_len; // may be len
  int32_t* status;  // or null
  int B, keep, sink, recent, ld, ld_table, ld_to;
  int num_pages, page_size, heads, dim;
};

struct CommitParams {
  const int32_t* cu;
  const int32_t* path;
  const int32_t* path_len;
  const int32_t* table;
  const int32_t* ctx;
  const void* k_new;
  const void* v_new;
  void* k;
  void* v;
  long long sn_layer, sn_node, sn_head, s_layer, s_page, s_slot, s_head;
  int32_t* new_len;  // may be ctx
  int32_t* status;
  int B, total, layers, ld_path, ld_table;
  int num_pages, page_size, heads, dim;
};

// ----------------------------------------------------------------- beams
constexpr int kBeamMax = 64;      // beams per request, and beams kept

struct BeamParams {
  const void* logits;
  long long ld;
  const float* scores;
  const int32_t* finished;
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  int32_t* status;
  unsigned long long* counters;  // [B] arrivals, call-tagged
  unsigned long long tag;
  float4* stat;                  // [grid * spans] (reference, sum, flags, largest logit)
  float* maxima;                 // [B * W][chunks]
  int B, W, keep, V, end_token;
  int grid, spans, chunks;       // CTAs, the most pieces of rows in one, chunks of a row
};

struct BeamWorkspace {
  size_t off_counters, off_stat, off_maxima, total;
};

inline BeamWorkspace make_beam_workspace(int B, int W, int grid, int spans, int chunks) {
  BeamWorkspace w;
  w.off_counters = 0;
  w.off_stat = up256((size_t)B * 8);
  w.off_maxima = w.off_stat + up256((size_t)grid * spans * 16);
  w.total = w.off_maxima + up256((size_t)B * W * chunks * 4);
  return w;
}

constexpr int kMaxStates = 8;

struct BeamState {
  const unsigned char* src;
  unsigned char* dst;
  long long row_bytes, src_outer, src_batch, src_beam, dst_outer, dst_batch, dst_beam;
  int outer;
  int unit;          // bytes per access, a power of two
  long long first;   // first work block of this state
  int blocks;        // work blocks per row
};

struct ReorderParams {
  const int32_t* parents;
  int B, W, keep, num;
  BeamState s[kMaxStates];
};

}  // namespace sv
