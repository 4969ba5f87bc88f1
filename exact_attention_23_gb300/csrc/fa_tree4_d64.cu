// Instantiations of the kernel for new tokens against a cache held in 4 bits, head dim 64.
#include "fa_tree_launch.cuh"

namespace fa {

cudaError_t launch_tree4_d64(const Tree4Launch& a, int rows, int mod) {
  return rows == 8 ? launch_tree4_mod<64, 1>(a, mod) : launch_tree4_mod<64, 2>(a, mod);
}

}  // namespace fa
