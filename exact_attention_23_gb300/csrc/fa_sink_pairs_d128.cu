// Instantiations of the two-tile forward with sinks in front of a sliding window for head dim 128 (plain
// scores, a cap of up to 60).
#include "fa_mod_launch.cuh"

namespace fa {

cudaError_t launch_fwd_sink_pairs_d128(const FwdLaunch& a, int mod) {
  switch (mod) {
    case kModOn: return launch_fwd_mod_pairs<128, kModSink | kModOn>(a);
    case kModOn | kModRest: return launch_fwd_mod_pairs<128, kModSink | kModOn | kModRest>(a);
    case kModOn | kModCap | kModRef: return launch_fwd_mod_pairs<128, kModSink | kModOn | kModCap | kModRef>(a);
    case kModOn | kModCap | kModRef | kModRest:
      return launch_fwd_mod_pairs<128, kModSink | kModOn | kModCap | kModRef | kModRest>(a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa
