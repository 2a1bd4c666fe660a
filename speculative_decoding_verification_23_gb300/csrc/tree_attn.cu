// Attention of drafted trees over a paged cache on warp tiles, and the joining of
// split items.
#include "tree_join.cuh"
#include "tree_warp.cuh"

namespace sv {

TreePlan plan_tree_warp(int dim, int num_sms) {
  TreePlan p;
  p.kernel = 0;
  p.rows = 16;
  p.kt = kWtKeys;
  p.grid = num_sms * (dim <= 128 ? 2 : 1);
  return p;
}

int launch_tree_warp(const TreeParams& P, bool bf16, cudaStream_t s) {
  return bf16 ? launch_warp_dim<__nv_bfloat16, false>(P, s) : launch_warp_dim<__half, false>(P, s);
}

int launch_tree_join(const TreeParams& P, bool bf16, int num_sms, cudaStream_t s) {
  return bf16 ? launch_join_dim<__nv_bfloat16, false>(P, num_sms, s) : launch_join_dim<__half, false>(P, num_sms, s);
}

}  // namespace sv
