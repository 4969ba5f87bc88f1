// Instantiations of the streaming kernel for new tokens against a cache with a sliding window and sinks,
// up to 32 query rows a key head, head dim 64.
#include "fa_tree_launch.cuh"

namespace fa {

cudaError_t launch_tree_window_d64(const TreeLaunch& a, int rows, int mod) {
  return launch_tree_rows<64, kModSink>(a, rows, mod);
}

}  // namespace fa
