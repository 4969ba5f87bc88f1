// Launches of the MOD kernels (modified scores), shared by their instantiation files. Internal.
#pragma once

#include <atomic>

#include "fa_launch.h"
#include "fa_mod_host.h"

namespace fa {

template <int D, int MOD>
cudaError_t launch_fwd_mod(const FwdLaunch& a) {
  auto* fn = &fa_fwd1_kernel<D, false, true, MOD>;
  static std::atomic<uint64_t> done[kMaxDevices / 64 + 1];
  using C = Cfg1<D, (MOD & kModRef) != 0>;
  const int smem = C::kSmemBytes;
  const cudaError_t e = smem_opt_in(fn, smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(fn, a.grid, C::kThreads, smem, a.stream, a.tm_q, a.tm_k, a.tm_v, a.tm_o, a.p);
}

// The same on the pair kernel (two query tiles a CTA; a.p.tiles_per_cta = 2).
template <int D, int MOD>
cudaError_t launch_fwd_mod_pairs(const FwdLaunch& a) {
  auto* fn = &fa_fwd_kernel<D, false, true, false, MOD>;
  static std::atomic<uint64_t> done[kMaxDevices / 64 + 1];
  const int smem = Cfg<D>::kSmemBytes;
  const cudaError_t e = smem_opt_in(fn, smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(fn, a.grid, kThreads, smem, a.stream, a.tm_q, a.tm_k, a.tm_v, a.tm_o, a.p);
}

// a.p.BH counts key heads' parts; q_heads = B·H.
template <int D, int MOD>
cudaError_t launch_bwd_mod(const BwdLaunch& a, int q_heads) {
  using C = BwdCfg<D, MOD>;
  auto* fn = &fa_bwd_main_kernel<D, false, MOD>;
  static std::atomic<uint64_t> done[kMaxDevices / 64 + 1];
  cudaError_t e = smem_opt_in(fn, C::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(fa_bwd_prep_kernel<D, true>, a.grid_prep, 256, 0, a.stream, a.o, a.dout, a.lse, a.lse2,
                 a.dvec, a.p.dq_acc, a.p.T, a.p.T_pad, q_heads, a.rest);
  if (e != cudaSuccess) return e;
  e = launch_pdl(fn, a.grid_main, C::kThreads, C::kSmemBytes, a.stream, a.tm_q, a.tm_k, a.tm_v, a.tm_do,
                 a.p);
  if (e != cudaSuccess) return e;
  if (a.p.mod.parts > 1) {
    const size_t rows = static_cast<size_t>(a.p.BH / a.p.mod.parts) * a.p.T;
    const float* part_out = a.p.mod.part_out;
    e = launch_pdl(fa_bwd_sum_kernel<D>, a.grid_dq, 256, 0, a.stream, part_out, a.p.dk, a.p.dv, rows, a.p.mod.parts);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(fa_bwd_dq_kernel<D>, a.grid_dq, 256, 0, a.stream, a.p.dq_acc, a.dq, a.p.T, a.p.n_qt,
                    q_heads, a.p.scale);
}

}  // namespace fa
