// Instantiations of the one-tile forward with modified scores for head dim 64: with and
// without a tanh cap and a distance bias.
#include "fa_mod_launch.cuh"

namespace fa {

cudaError_t launch_fwd_mod_d64(const FwdLaunch& a, int mod) {
  switch (mod) {
    case kModOn:
    case kModOn | kModRest: return launch_fwd_mod<64, kModOn>(a);
    case kModOn | kModCap: return launch_fwd_mod<64, kModOn | kModCap>(a);
    case kModOn | kModCap | kModRef: return launch_fwd_mod<64, kModOn | kModCap | kModRef>(a);
    case kModOn | kModCap | kModRef | kModRest:
      return launch_fwd_mod<64, kModOn | kModCap | kModRef | kModRest>(a);
    case kModOn | kModBias: return launch_fwd_mod<64, kModOn | kModBias>(a);
    case kModOn | kModCap | kModBias: return launch_fwd_mod<64, kModOn | kModCap | kModBias>(a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa
