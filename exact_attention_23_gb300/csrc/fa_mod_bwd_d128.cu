// Instantiations of the backward with modified scores for head dim 128: with and without a
// tanh cap and a distance bias.
#include "fa_mod_launch.cuh"

namespace fa {

cudaError_t launch_bwd_mod_d128(const BwdLaunch& a, int mod, int q_heads) {
  switch (mod) {
    case kModOn: return launch_bwd_mod<128, kModOn>(a, q_heads);
    case kModOn | kModCap: return launch_bwd_mod<128, kModOn | kModCap>(a, q_heads);
    case kModOn | kModBias: return launch_bwd_mod<128, kModOn | kModBias>(a, q_heads);
    case kModOn | kModCap | kModBias:
      return launch_bwd_mod<128, kModOn | kModCap | kModBias>(a, q_heads);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa
