// Instantiations of the streaming kernel for new tokens against a cache held in 4 bits, head dim 128.
#include "fa_tree_launch.cuh"

namespace fa {

cudaError_t launch_tree_four_d128(const TreeLaunch& a, int rows, int mod) {
  return launch_tree_rows<128, kModSink | kModFour>(a, rows, mod);
}

}  // namespace fa
