// Instantiations of the backward with modified scores for head dim 64: with and without a
// tanh cap and a distance bias.
#include "fa_mod_launch.cuh"

namespace fa {

cudaError_t launch_bwd_mod_d64(const BwdLaunch& a, int mod, int q_heads) {
  switch (mod) {
    case kModOn: return launch_bwd_mod<64, kModOn>(a, q_heads);
    case kModOn | kModCap: return launch_bwd_mod<64, kModOn | kModCap>(a, q_heads);
    case kModOn | kModBias: return launch_bwd_mod<64, kModOn | kModBias>(a, q_heads);
    case kModOn | kModCap | kModBias:
      return launch_bwd_mod<64, kModOn | kModCap | kModBias>(a, q_heads);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa
