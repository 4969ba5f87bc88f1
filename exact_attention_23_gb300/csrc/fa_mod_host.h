// Host helpers of the entry points with modified scores. Internal; not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
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
  *k = fa::CapFactors{};
  if (!std::isfinite(softcap) || softcap < 0.0f) return false;
  if (softcap == 0.0f) return true;
  const double u = static_cast<double>(scale) / softcap;
  double power = static_cast<double>(scale) * kLog2e;
  for (int i = 0; i < 5; ++i, power *= u * u) k->c[i] = static_cast<float>(fa::kCapPoly[i] * power);
  k->in_exp = static_cast<float>(2.0 * kLog2e * u);
  k->out = static_cast<float>(softcap * kLog2e);
  k->bend = static_cast<float>(-1.0 / (softcap * kLog2e * softcap * kLog2e));
  // (squares of raw scores up to 10¹⁸ stay finite)
  k->limit = static_cast<float>(std::min(fa::kCapBend / std::fabs(u), 1e18));
  for (float c : k->c)
    if (!std::isfinite(c)) return false;
  return std::isfinite(k->in_exp) && std::isfinite(k->out) && std::isfinite(k->bend);
}

inline int mod_bits(float softcap, const float* slopes) {
  return fa::kModOn | (softcap > 0.0f ? fa::kModCap : 0) | (slopes ? fa::kModBias : 0);
}

// The forward's: a small enough cap alone takes the softmax against 0.
inline int fwd_mod_bits(float softcap, const float* slopes, const void* rest) {
  const int mod = mod_bits(softcap, slopes);
  if (mod == fa::kModOn) return mod | (rest ? fa::kModRest : 0);
  if (mod != (fa::kModOn | fa::kModCap) || softcap * kLog2e > fa::kCapRef) return mod;
  return mod | fa::kModRef | (rest ? fa::kModRest : 0);
}

}  // namespace host
}  // namespace fa
