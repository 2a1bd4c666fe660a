// Attention of drafted trees with a sliding window and sinks on the
// 5th-generation tensor cores: the kernel of the drafted trees, whose tiles are
// those of the sinks and of the last `window` tokens and the drafted ones.  Only
// tiles that some rows see and others do not are masked key by key.
//
// 64 ragged requests of up to 9 nodes, 28 / 4 heads, a window of 4096 in up to
// 16384 tokens: 101 us with the joining kernel, 4.8 TB/s, 71 % of the copy rate.
// Trees of up to 64 nodes, 32 / 8 heads, a window of 2000 and 64 sinks: 57 us, where
// the bytes would take 22: 128 items of some 17 tiles for 152 CTAs, so that nearly
// every CTA loads queries twice and leaves partial results, and in each item the
// sinks', the window's first and the drafted tile are masked.
#include "tree_tc.cuh"

namespace sv {

int launch_window_tc(const TreeParams& P, bool bf16, cudaStream_t s) { return launch_tc_maps<true>(P, bf16, s); }

}  // namespace sv
