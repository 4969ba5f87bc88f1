// Instantiations of the kernel for new tokens against a cache held in 4 bits, head dim 128.
#include "fa_tree_launch.cuh"

namespace fa {

cudaError_t launch_tree4_d128(const Tree4Launch& a, int rows, int mod) {
  return rows == 8 ? launch_tree4_mod<128, 1>(a, mod) : launch_tree4_mod<128, 2>(a, mod);
}

}  // namespace fa
