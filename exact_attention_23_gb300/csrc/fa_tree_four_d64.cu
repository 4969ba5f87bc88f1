// Instantiations of the streaming kernel for new tokens against a cache held in 4 bits, head dim 64.
#include "fa_tree_launch.cuh"

namespace fa {

cudaError_t launch_tree_four_d64(const TreeLaunch& a, int rows, int mod) {
  return launch_tree_rows<64, kModSink | kModFour>(a, rows, mod);
}

}  // namespace fa
