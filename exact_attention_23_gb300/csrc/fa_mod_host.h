// Host helpers of the entry points with modified scores. Internal; not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cmath>

#include "fa_mod.cuh"
#include "fa_pdl.h"

namespace fa {

// The shared-memory opt-in is a per-device attribute: set it once per device and kernel.
template <typename Fn>
cudaError_t smem_opt_in(Fn* fn, int smem, std::atomic<uint64_t>* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  const uint64_t bit = 1ull << (dev % 64);
  if (done[dev / 64].load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done[dev / 64].fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

namespace host {

constexpr double kLog2e = 1.4426950408889634074;

// The cap's factors; false when the arguments cannot be used.
inline bool cap_factors(float scale, float softcap, fa::CapFactors* k) {
  *k = fa::CapFactors{0.f, 0.f, 0.f, 0.f};
  if (!std::isfinite(softcap) || softcap < 0.0f) return false;
  if (softcap == 0.0f) return true;
  const double u = static_cast<double>(scale) / softcap;
  k->in = static_cast<float>(u);
  k->in_exp = static_cast<float>(2.0 * kLog2e * u);
  k->out = static_cast<float>(softcap * kLog2e);
  k->limit = static_cast<float>(fa::kCapBend / std::fabs(u));
  return std::isfinite(k->in_exp) && std::isfinite(k->out);
}

inline int mod_bits(float softcap, const float* slopes) {
  return fa::kModOn | (softcap > 0.0f ? fa::kModCap : 0) | (slopes ? fa::kModBias : 0);
}

}  // namespace host
}  // namespace fa
