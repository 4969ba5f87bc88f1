// Instantiations of the two-tile forward with modified scores for head dim 64 (documents and
// prefixes, a cap of up to 60).
#include "fa_mod_launch.cuh"

namespace fa {

cudaError_t launch_fwd_mod_pairs_d64(const FwdLaunch& a, int mod) {
  switch (mod) {
    case kModOn: return launch_fwd_mod_pairs<64, kModOn>(a);
    case kModOn | kModRest: return launch_fwd_mod_pairs<64, kModOn | kModRest>(a);
    case kModOn | kModCap | kModRef: return launch_fwd_mod_pairs<64, kModOn | kModCap | kModRef>(a);
    case kModOn | kModCap | kModRef | kModTight:
      return launch_fwd_mod_pairs<64, kModOn | kModCap | kModRef | kModTight>(a);
    case kModOn | kModCap | kModRef | kModRest:
      return launch_fwd_mod_pairs<64, kModOn | kModCap | kModRef | kModRest>(a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa
