// Launches of the streaming kernel for new tokens against a cache, shared by its instantiation files.
// Internal.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "fa_mod_host.h"
#include "fa_pdl.h"
#include "fa_tree_kernel.cuh"

namespace fa {

struct TreeLaunch {
  CUtensorMap tm_k, tm_v;
  TreeParams p;
  unsigned grid;
  cudaStream_t stream;
};

template <int D, int RG, int MOD>
cudaError_t launch_tree(const TreeLaunch& a) {
  auto* fn = &fa_tree_kernel<D, RG, MOD>;
  const int smem = TreeCfg<D, (MOD & kModFour) != 0>::kSmemBytes;
  static std::atomic<uint64_t> done[kMaxDevices / 64 + 1];
  cudaError_t e = smem_opt_in(fn, smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(fn, a.grid, kTreeBlock, smem, a.stream, a.tm_k, a.tm_v, a.p);
}

// EXTRA: kModSink, kModSink | kModFour or nothing.
template <int D, int RG, int EXTRA>
cudaError_t launch_tree_mod(const TreeLaunch& a, int mod) {
  switch (mod) {
    case kModOn: return launch_tree<D, RG, EXTRA | kModOn>(a);
    case kModOn | kModCap: return launch_tree<D, RG, EXTRA | kModOn | kModCap>(a);
    case kModOn | kModBias: return launch_tree<D, RG, EXTRA | kModOn | kModBias>(a);
    default: return launch_tree<D, RG, EXTRA | kModOn | kModCap | kModBias>(a);
  }
}

template <int D, int EXTRA>
cudaError_t launch_tree_rows(const TreeLaunch& a, int rows, int mod) {
  return rows == 16 ? launch_tree_mod<D, 1, EXTRA>(a, mod)
                    : launch_tree_mod<D, 2, EXTRA>(a, mod);
}

// With a sliding window and sinks (fa_tree_window.cu).
cudaError_t launch_tree_window_d64(const TreeLaunch& a, int rows, int mod);
cudaError_t launch_tree_window_d128(const TreeLaunch& a, int rows, int mod);
// Over a cache held in 4 bits (fa_tree_four_d….cu; a window of INT_MAX is none).
cudaError_t launch_tree_four_d64(const TreeLaunch& a, int rows, int mod);
cudaError_t launch_tree_four_d128(const TreeLaunch& a, int rows, int mod);

}  // namespace fa
