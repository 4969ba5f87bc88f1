// Internal interface between the host API (fa_api.cu) and the kernel instantiations
// (fa_fwd_d64.cu, fa_fwd_d128.cu, fa_bwd_d64.cu). Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "fa_bwd_kernel.cuh"
#include "fa_decode_kernel.cuh"
#include "fa_fwd_kernel.cuh"
#include "fa_fwd1_kernel.cuh"
#include "fa_fwd_pair_kernel.cuh"
#include "fa_pdl.h"

namespace fa {

struct FwdLaunch {
  CUtensorMap tm_q, tm_k, tm_v;
  CUtensorMap tm_o;  // the output, boxes of 64 columns × 32 rows (one warp's rows)
  FwdParams p;
  unsigned grid;
  cudaStream_t stream;
};

// Each returns the CUDA error of the launch (cudaSuccess when enqueued).
cudaError_t launch_fwd_d64(const FwdLaunch& a, bool causal);
cudaError_t launch_fwd_d128(const FwdLaunch& a, bool causal);
// Q and K as e4m3 codes (tensor maps over bytes), d ∈ {64, 128}.
cudaError_t launch_fwd_fp8(const FwdLaunch& a, int d, bool causal);
// One 128-row Q tile per CTA with double-buffered S and P (fa_fwd1_kernel.cuh); a.p holds one
// tile per unit (tiles_per_cta = 1), d ∈ {64, 128}.
cudaError_t launch_fwd1(const FwdLaunch& a, int d, bool causal);
// The general form (queries against a longer key sequence, key ranges, block mask) on the
// one-tile kernel (tiles_per_cta = 1), then the merge when the key range is split.
cudaError_t launch_fwd1_gen(const FwdLaunch& a, int d, bool causal, unsigned combine_grid);
// Head dim 64 on CTA pairs (fa_fwd_pair_kernel.cuh): a.grid is even (clusters of two), a.p holds
// groups of four Q tiles per unit, tm_k has 64-row boxes and tm_v 32-column × 128-row boxes
// with the 64-byte swizzle.
cudaError_t launch_fwd_pair_d64(const FwdLaunch& a, bool causal);

// General form (Tq ≠ Tk, bottom-right causal, block masks, key ranges): the forward kernel
// with GEN = true, then, when a.p.n_splits > 1, the merge of the partial results.
cudaError_t launch_fwd_gen_d64(const FwdLaunch& a, bool causal, unsigned combine_grid);
cudaError_t launch_fwd_gen_d128(const FwdLaunch& a, bool causal, unsigned combine_grid);

// Decode (Tq = 1) on the CUDA cores: grid B·H × n_splits, then the merge when split.
cudaError_t launch_decode(const DecodeParams& p, int d, unsigned combine_grid,
                          cudaStream_t stream);
// Two query rows per head (Tq = kDecMultiMaxRows) on the CUDA cores, two warps per row: grid
// B·H × n_splits, then the merge when split. (From three rows on, the one-tile tensor-core
// kernel is faster.)
constexpr int kDecMultiMaxRows = 2;
cudaError_t launch_decode_multi(const DecodeParams& p, int d, unsigned combine_grid,
                                cudaStream_t stream);

// Modified scores (fa_mod.cuh) on the one-tile kernel, mod the kMod… bits.
cudaError_t launch_fwd_mod_d64(const FwdLaunch& a, int mod);
cudaError_t launch_fwd_mod_d128(const FwdLaunch& a, int mod);
// On the pair kernel, two query tiles a unit (a.p.tiles_per_cta = 2): kModOn, or with
// kModRef.
cudaError_t launch_fwd_mod_pairs_d64(const FwdLaunch& a, int mod);
cudaError_t launch_fwd_mod_pairs_d128(const FwdLaunch& a, int mod);
// New tokens against a cache on the same kernel (a.p.T the rows a key head, a.grid the stretches).
cudaError_t launch_fwd_tree_d64(const FwdLaunch& a, int mod);
cudaError_t launch_fwd_tree_d128(const FwdLaunch& a, int mod);

struct BwdLaunch {
  CUtensorMap tm_q, tm_k, tm_v, tm_do;
  BwdParams p;
  const __nv_bfloat16* o;
  const __nv_bfloat16* dout;
  const __nv_bfloat16* rest;  // modified scores: what o's rounding left out, or null
  const float* lse;
  float* lse2;
  float* dvec;
  __nv_bfloat16* dq;
  unsigned grid_main, grid_prep, grid_dq;
  cudaStream_t stream;
};

// Enqueues the three backward kernels (prep, main, dQ conversion) on a.stream.
cudaError_t launch_bwd_d64(const BwdLaunch& a, bool causal);
cudaError_t launch_bwd_d128(const BwdLaunch& a, bool causal);
// The same with modified scores; a.p.BH counts key heads' parts, q_heads = B·H.
cudaError_t launch_bwd_mod_d64(const BwdLaunch& a, int mod, int q_heads);
cudaError_t launch_bwd_mod_d128(const BwdLaunch& a, int mod, int q_heads);

}  // namespace fa
