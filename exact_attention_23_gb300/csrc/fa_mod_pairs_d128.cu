// Instantiations of the two-tile forward with modified scores for head dim 128 (documents and
// prefixes, a cap of up to 60).
#include "fa_mod_launch.cuh"

namespace fa {

cudaError_t launch_fwd_mod_pairs_d128(const FwdLaunch& a, int mod) {
  switch (mod) {
    case kModOn: return launch_fwd_mod_pairs<128, kModOn>(a);
    case kModOn | kModRest: return launch_fwd_mod_pairs<128, kModOn | kModRest>(a);
    case kModOn | kModCap | kModRef: return launch_fwd_mod_pairs<128, kModOn | kModCap | kModRef>(a);
    case kModOn | kModCap | kModRef | kModRest:
      return launch_fwd_mod_pairs<128, kModOn | kModCap | kModRef | kModRest>(a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa
