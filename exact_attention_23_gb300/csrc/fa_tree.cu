// Host side of attention of new tokens against a cache (include/fa.h: fa_fwd_tree) and the
// instantiations of its kernels.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "fa.h"
#include "fa_host.h"
#include "fa_mod_host.h"
#include "fa_pdl.h"
#include "fa_tree_kernel.cuh"

using namespace fa::host;

namespace fa {

namespace {

struct TreeLaunch {
  CUtensorMap tm_k, tm_v;
  TreeParams p;
  unsigned grid, combine_grid;
  cudaStream_t stream;
};

template <int D, int RG, int MOD>
cudaError_t launch_tree(const TreeLaunch& a) {
  auto* fn = &fa_tree_kernel<D, RG, MOD>;
  const int smem = TreeCfg<D>::kSmemBytes;
  static std::atomic<uint64_t> done[kMaxDevices / 64 + 1];
  cudaError_t e = smem_opt_in(fn, smem, done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(fn, a.grid, kTreeBlock, smem, a.stream, a.tm_k, a.tm_v, a.p);
  if (e != cudaSuccess) return e;
  return launch_pdl(fa_tree_combine_kernel<D, RG * 16>, a.combine_grid, 256, 0, a.stream, a.p,
                    static_cast<int>(a.grid));
}

template <int D, int RG>
cudaError_t launch_tree_mod(const TreeLaunch& a, int mod) {
  switch (mod) {
    case kModOn: return launch_tree<D, RG, kModOn>(a);
    case kModOn | kModCap: return launch_tree<D, RG, kModOn | kModCap>(a);
    case kModOn | kModBias: return launch_tree<D, RG, kModOn | kModBias>(a);
    default: return launch_tree<D, RG, kModOn | kModCap | kModBias>(a);
  }
}

template <int D>
cudaError_t launch_tree_rows(const TreeLaunch& a, int rows, int mod) {
  return rows == 16 ? launch_tree_mod<D, 1>(a, mod)
                    : rows == 32 ? launch_tree_mod<D, 2>(a, mod) : launch_tree_mod<D, 4>(a, mod);
}

// Rows a block: the fewest of 16, 32, 64 that hold all R, so that the keys are read once; more
// rows than 64 go in blocks of 64, whose later ones find the keys in L2.
int block_rows(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : 64; }

// Chunks a stretch has at least: under two the merge costs more than the parallelism gives.
constexpr int kMinPer = 2;

struct TreeSizes {
  int R, rows, row_blocks;
  long long entries, grid, slots;
  size_t lse_off, bytes;
};

bool tree_sizes(int B, int H, int Hkv, int Tq, int Tmax, int d, int sms, TreeSizes* z) {
  if (B <= 0 || H <= 0 || Hkv <= 0 || Tq <= 0 || Tmax <= 0 || H % Hkv != 0 || (d != 64 && d != 128))
    return false;
  const long long R = static_cast<long long>(H / Hkv) * Tq, BHkv = static_cast<long long>(B) * Hkv;
  if (static_cast<long long>(B) * H > INT32_MAX || R > (1 << 24) || Tmax > (1 << 30)) return false;
  z->R = static_cast<int>(R);
  z->rows = block_rows(z->R);
  z->row_blocks = (z->R + z->rows - 1) / z->rows;
  z->entries = BHkv * z->row_blocks;
  if (z->entries > (1 << 28) || BHkv * R > (1LL << 40) || BHkv > (1LL << 60) / d / Tmax) return false;
  const long long chunks = (static_cast<long long>(Tmax) + kTreeKeys - 1) / kTreeKeys;
  if (z->entries * chunks > INT32_MAX - 64) return false;  // (the kernel numbers them with an int)
  const long long most = (z->entries * chunks + kMinPer - 1) / kMinPer;
  const long long fit = static_cast<long long>(sms) * (d == 64 ? TreeCfg<64>::kCtasPerSm : TreeCfg<128>::kCtasPerSm);
  z->grid = std::max<long long>(1, std::min(fit, most));
  z->slots = z->grid + z->entries;
  auto up = [](size_t x) { return (x + 255u) / 256u * 256u; };
  z->lse_off = up(static_cast<size_t>(z->slots) * z->rows * d * 4);
  z->bytes = z->lse_off + up(static_cast<size_t>(z->slots) * z->rows * 4);
  return true;
}

}  // namespace

}  // namespace fa

extern "C" {

size_t fa_fwd_tree_workspace_size(int B, int H, int Hkv, int Tq, int Tmax, int d) {
  fa::TreeSizes z;
  if (!fa::tree_sizes(B, H, Hkv, Tq, Tmax, d, 1, &z)) return 0;
  int dev = -1, sms = 0;
  if (check_device(&dev, &sms) != FA_OK) return 0;
  return fa::tree_sizes(B, H, Hkv, Tq, Tmax, d, sms, &z) ? z.bytes : 0;
}

int fa_fwd_tree(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                const int* ctx_len, const unsigned char* tree, int tree_per_batch, const int* depths,
                int depths_per_batch, float softcap, const float* slopes, int B, int H, int Hkv, int Tq,
                int Tmax, int d, float scale, void* workspace, size_t workspace_bytes, int* status,
                unsigned long long timeout_ns, void* stream) {
  if (!q || !k_cache || !v_cache || !o || !lse || !ctx_len || !workspace) return FA_ERR_INVALID_ARG;
  fa::TreeSizes z;
  fa::CapFactors cap;
  if (!fa::tree_sizes(B, H, Hkv, Tq, Tmax, d, 1, &z) || !scale_ok(scale) || !cap_factors(scale, softcap, &cap))
    return FA_ERR_INVALID_ARG;
  const uintptr_t words = reinterpret_cast<uintptr_t>(ctx_len) | reinterpret_cast<uintptr_t>(depths) |
                          reinterpret_cast<uintptr_t>(slopes);
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned16(lse) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) || (words & 3u))
    return FA_ERR_MISALIGNED;
  int dev = -1, sms = 0;
  const size_t qb = static_cast<size_t>(B) * H * Tq * d * 2, cb = static_cast<size_t>(B) * Hkv * Tmax * d * 2;
  const size_t lb = static_cast<size_t>(B) * H * Tq * 4;
  const size_t tb = static_cast<size_t>(tree_per_batch ? B : 1) * Tq * Tq;
  const size_t db = static_cast<size_t>(depths_per_batch ? B : 1) * Tq * 4;
  const int dst = check_device(&dev, &sms);
  if (dst == FA_OK && !fa::tree_sizes(B, H, Hkv, Tq, Tmax, d, sms, &z)) return FA_ERR_INVALID_ARG;
  if (workspace_bytes < z.bytes) return FA_ERR_INVALID_ARG;
  const void* ins[7] = {q, k_cache, v_cache, ctx_len, tree, depths, slopes};
  const size_t in_bytes[7] = {qb, cb, cb, static_cast<size_t>(B) * 4, tb, db, static_cast<size_t>(H) * 4};
  const void* outs[3] = {o, lse, workspace};
  const size_t out_bytes[3] = {qb, lb, z.bytes};
  for (int x = 0; x < 3; ++x) {
    for (int y = 0; y < 7; ++y)
      if (ins[y] && overlaps(outs[x], out_bytes[x], ins[y], in_bytes[y])) return FA_ERR_INVALID_ARG;
    for (int y = x + 1; y < 3; ++y)
      if (overlaps(outs[x], out_bytes[x], outs[y], out_bytes[y])) return FA_ERR_INVALID_ARG;
  }
  if (dst != FA_OK) return dst;
  EncodeTiledFn enc = encode_fn();
  if (!enc) return FA_ERR_LAUNCH;
  fa::TreeLaunch a;
  if (!encode_map(enc, &a.tm_k, k_cache, Tmax, d, B * Hkv, fa::kTreeKeys) ||
      !encode_map(enc, &a.tm_v, v_cache, Tmax, d, B * Hkv, fa::kTreeKeys))
    return FA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.p = fa::TreeParams{};
  a.p.q = static_cast<const __nv_bfloat16*>(q);
  a.p.o = static_cast<__nv_bfloat16*>(o);
  a.p.lse = lse;
  a.p.o_part = reinterpret_cast<float*>(ws);
  a.p.lse_part = reinterpret_cast<float*>(ws + z.lse_off);
  a.p.ctx_len = ctx_len;
  a.p.tree = tree;
  a.p.depths = depths;
  a.p.slopes = slopes;
  a.p.status = status;
  a.p.timeout_ns = timeout_ns ? timeout_ns : 2000000000ull;
  a.p.div_tq = fa::FastDiv::make(static_cast<uint32_t>(Tq));
  a.p.cap = cap;
  a.p.scale_log2 = static_cast<float>(static_cast<double>(scale) * kLog2e);
  a.p.tree_per_batch = tree_per_batch != 0;
  a.p.depths_per_batch = depths_per_batch != 0;
  a.p.B = B;
  a.p.Hkv = Hkv;
  a.p.R = z.R;
  a.p.Tq = Tq;
  a.p.Tmax = Tmax;
  a.p.row_blocks = z.row_blocks;
  a.p.min_per = fa::kMinPer;
  a.grid = static_cast<unsigned>(z.grid);
  const long long rows = static_cast<long long>(B) * Hkv * z.R;
  a.combine_grid = static_cast<unsigned>(std::min<long long>((rows + 7) / 8, static_cast<long long>(sms) * 8));
  a.stream = static_cast<cudaStream_t>(stream);
  const int mod = mod_bits(softcap, slopes);
  const cudaError_t e = (d == 64) ? fa::launch_tree_rows<64>(a, z.rows, mod) : fa::launch_tree_rows<128>(a, z.rows, mod);
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
