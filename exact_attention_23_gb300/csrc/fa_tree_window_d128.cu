// Instantiations of the streaming kernel for new tokens against a cache with a sliding window and sinks,
// up to 32 query rows a key head, head dim 128.
#include "fa_tree_launch.cuh"

namespace fa {

cudaError_t launch_tree_window_d128(const TreeLaunch& a, int rows, int mod) {
  return launch_tree_rows<128, kModSink>(a, rows, mod);
}

}  // namespace fa
