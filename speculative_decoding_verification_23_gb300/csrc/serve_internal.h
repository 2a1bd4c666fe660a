// Parameter blocks of the operators beside the drafted tree, shared by their
// entry points (serve_ops.cu) and kernels.
#pragma once

#include "tree_internal.h"

namespace sv {

// ---------------------------------------------------- norms and positions
struct RotateSide {
  const void* x;
  void* y;
  const void* weight;  // or null
  long long sx_row, sx_head, sy_row, sy_head;
  int heads;
};

struct RotateParams {
  RotateSide side[2];  // queries, keys
  const int32_t* positions;
  const float* inv_freq;
  float eps;
  int rows, dim, rot, interleaved;
  int steps;           // heads of a row, by the number that a warp takes at once
  int parts;           // warps that share a row
};

// ----------------------------------------------------- attention, 8 bits
// `t.k` and `t.v` are bytes, and so are the strides of the cache.
struct Cache8Params {
  TreeParams t;
  const float* ks;  // of the layer
  const float* vs;
  long long c_page, c_block, c_head;
  int block;
};

struct Commit8Params {
  const int32_t* cu;
  const int32_t* path;
  const int32_t* path_len;
  const int32_t* table;
  const int32_t* ctx;
  const void* x[2];        // new keys, new values
  uint8_t* held[2];
  float* scale[2];
  long long sn_layer, sn_node, sn_head, s_layer, s_page, s_slot, s_head, c_layer, c_page, c_block, c_head;
  int32_t* new_len;        // may be ctx
  int32_t* status;         // or null
  int B, total, layers, ld_path, ld_table;
  int num_pages, page_size, heads, dim, block;
  int warps;               // warps that share a unit
};

}  // namespace sv
