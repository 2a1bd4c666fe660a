// Attention of drafted trees with a sliding window and sinks on the
// 5th-generation tensor cores.
#include "tree_tc.cuh"

namespace sv {

int launch_window_tc(const TreeParams& P, bool bf16, cudaStream_t s) { return launch_tc_maps<true>(P, bf16, s); }

}  // namespace sv
