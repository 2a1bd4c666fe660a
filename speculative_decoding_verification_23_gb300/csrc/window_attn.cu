// Attention of drafted trees with a sliding window and sinks on warp tiles, and
// the joining of split items.
#include "tree_join.cuh"
#include "tree_warp.cuh"

namespace sv {

int launch_window_warp(const TreeParams& P, bool bf16, cudaStream_t s) {
  return bf16 ? launch_warp_dim<__nv_bfloat16, true>(P, s) : launch_warp_dim<__half, true>(P, s);
}

int launch_window_join(const TreeParams& P, bool bf16, int num_sms, cudaStream_t s) {
  return bf16 ? launch_join_dim<__nv_bfloat16, true>(P, num_sms, s) : launch_join_dim<__half, true>(P, num_sms, s);
}

}  // namespace sv
