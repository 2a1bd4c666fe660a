// Attention of drafted trees over a paged cache on the 5th-generation tensor cores.
#include "tree_tc.cuh"

namespace sv {

// Heads of 64 or 128 channels, pages of a multiple of 8 slots (a box of a
// TMA copy fills whole swizzle patterns of 8 rows).
bool tree_tc_fits(int dim, int page_size) { return (dim == 64 || dim == 128) && page_size % 8 == 0; }

TreePlan plan_tree_tc(int rows, int num_sms) {
  TreePlan p;
  p.kernel = 1;
  p.grid = num_sms;
  // Two row tiles where there are more rows than one has: 256 rows of 16
  // requests 89 us against 118 with one (which reads the cache twice), 160
  // rows 76 against 93; 63 rows of 64 requests 76 us against 72 with one.
  p.rows = rows > kTcRows ? 2 * kTcRows : kTcRows;
  p.kt = kTcKeys;
  return p;
}

int launch_tree_tc(const TreeParams& P, bool bf16, cudaStream_t s) { return launch_tc_maps<false>(P, bf16, s); }

}  // namespace sv
