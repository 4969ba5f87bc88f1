// Instantiations of the one-tile forward with sinks in front of a sliding window for head dim 64: with
// and without a tanh cap and a distance bias.
#include "fa_mod_launch.cuh"

namespace fa {

cudaError_t launch_fwd_sink_d64(const FwdLaunch& a, int mod) {
  switch (mod) {
    case kModOn:
    case kModOn | kModRest: return launch_fwd_mod<64, kModSink | kModOn>(a);
    case kModOn | kModCap: return launch_fwd_mod<64, kModSink | kModOn | kModCap>(a);
    case kModOn | kModCap | kModRef: return launch_fwd_mod<64, kModSink | kModOn | kModCap | kModRef>(a);
    case kModOn | kModCap | kModRef | kModRest:
      return launch_fwd_mod<64, kModSink | kModOn | kModCap | kModRef | kModRest>(a);
    case kModOn | kModBias: return launch_fwd_mod<64, kModSink | kModOn | kModBias>(a);
    case kModOn | kModCap | kModBias: return launch_fwd_mod<64, kModSink | kModOn | kModCap | kModBias>(a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa
