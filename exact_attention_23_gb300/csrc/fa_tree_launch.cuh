// Launches of the streaming kernel for new tokens against a cache, shared by its instantiation files.
// Internal.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "fa_mod_host.h"
#include "fa_pdl.h"
#include "fa_tree4_kernel.cuh"
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
  const int smem = TreeCfg<D>::kSmemBytes;
  static std::atomic<uint64_t> done[kMaxDevices / 64 + 1];
  cudaError_t e = smem_opt_in(fn, smem, done);
  if (e != cudaSuccess) return e;
  const unsigned cluster = (MOD & kModSink) != 0 ? std::max(a.p.list.solo, 1) : 1;
  return launch_pdl_clusters(fn, a.grid, cluster, kTreeBlock, smem, a.stream, a.tm_k, a.tm_v, a.p);
}

// EXTRA: kModSink or nothing.
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

// Over a cache held in 4 bits, `rows` (8 or 16) query rows an entry. a.p holds no tensor maps.
struct Tree4Launch {
  Tree4Params p;
  unsigned grid;
  cudaStream_t stream;
};

template <int D, int NB, int MOD>
cudaError_t launch_tree4(const Tree4Launch& a) {
  auto* fn = &fa_tree4_kernel<D, NB, MOD>;
  const int smem = Tree4Cfg<D, NB>::kSmemBytes;
  static std::atomic<uint64_t> done[kMaxDevices / 64 + 1];
  const cudaError_t e = smem_opt_in(fn, smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl_clusters(fn, a.grid, static_cast<unsigned>(std::max(a.p.t.list.solo, 1)), kTreeBlock, smem, a.stream, a.p);
}

template <int D, int NB>
cudaError_t launch_tree4_mod(const Tree4Launch& a, int mod) {
  switch (mod) {
    case kModOn: return launch_tree4<D, NB, kModOn>(a);
    case kModOn | kModCap: return launch_tree4<D, NB, kModOn | kModCap>(a);
    case kModOn | kModBias: return launch_tree4<D, NB, kModOn | kModBias>(a);
    default: return launch_tree4<D, NB, kModOn | kModCap | kModBias>(a);
  }
}

cudaError_t launch_tree4_d64(const Tree4Launch& a, int rows, int mod);
cudaError_t launch_tree4_d128(const Tree4Launch& a, int rows, int mod);

// With a sliding window and sinks (fa_tree_window_d….cu).
cudaError_t launch_tree_window_d64(const TreeLaunch& a, int rows, int mod);
cudaError_t launch_tree_window_d128(const TreeLaunch& a, int rows, int mod);

}  // namespace fa
