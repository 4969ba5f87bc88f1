// Instantiations of the one-tile forward for new tokens against a cache with more than 32 query
// rows a key head, head dim 128.
#include "fa_mod_launch.cuh"

namespace fa {

cudaError_t launch_fwd_tree_d128(const FwdLaunch& a, int mod) {
  switch (mod) {
    case kModOn: return launch_fwd_mod<128, kModTree | kModOn>(a);
    case kModOn | kModCap: return launch_fwd_mod<128, kModTree | kModOn | kModCap>(a);
    case kModOn | kModCap | kModRef: return launch_fwd_mod<128, kModTree | kModOn | kModCap | kModRef>(a);
    case kModOn | kModBias: return launch_fwd_mod<128, kModTree | kModOn | kModBias>(a);
    case kModOn | kModCap | kModBias: return launch_fwd_mod<128, kModTree | kModOn | kModCap | kModBias>(a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa
