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
#include "fa_launch.h"
#include "fa_mod_host.h"
#include "fa_pdl.h"
#include "fa_tree_kernel.cuh"

using namespace fa::host;

namespace fa {

namespace {

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
  return launch_pdl(fn, a.grid, kTreeBlock, smem, a.stream, a.tm_k, a.tm_v, a.p);
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
                    : launch_tree_mod<D, 2>(a, mod);
}

// Up to 32 rows of a key head: the streaming kernel, in one block of 16 or 32 rows, so that the
// keys are read once. More: blocks of 128 rows on the one-tile tensor-core kernel (B4 H16 Hkv4,
// 16 tokens, 64 rows, up to 16384 keys, d = 128: 35 µs against 57 with 64 rows on mma.sync,
// whose products then take longer than the keys' bytes).
bool wide(int R) { return R > 32; }
int block_rows_log2(int R) { return R <= 16 ? 4 : R <= 32 ? 5 : 7; }

// Chunks a stretch has at least.
constexpr int kMinPer = 2, kMinPerWide = 1;

// Entries that fit the GPU at once go without stretches, a CTA each, where a CTA then walks at most
// join_chunks more chunks than its stretch would have: what the partials' way through memory and the
// second kernel are worth. By GPU time, with every context full (µs in stretches / whole, at 64-key
// chunks, wide 128; cap 30):
//   one token, d64 (join 7)    8 entries, 6 chunks 6.7 / 6.1, 10 chunks 6.8 / 8.3;  96 entries, 10 chunks
//                              10.7 / 8.6, 18 chunks 11.6 / 13.2;  456 entries, 24 chunks 35.4 / 30.6
//   d128 (5)                   8, 4: 8.1 / 7.1, 8: 8.2 / 10.6;  96, 8: 13.8 / 10.9, 12: 11.6 / 14.4;
//                              304, 24: 43.8 / 40.2
//   wide, d64, 256 rows (5)    8, 4: 9.4 / 8.5, 8: 9.9 / 12.4;  32, 6: 13.7 / 10.9, 12: 14.6 / 16.9;  128, 12: 29.4 / 17.8
//   d128, 64 rows (4)          4, 4: 9.9 / 9.8, 6: 9.9 / 12.2;  64, 8: 18.3 / 15.3, 16 entries, 8: 12.9 / 14.9
// Not beyond the chunks measured: stretches share out unequal contexts, a CTA an entry does not.
int join_chunks(bool wide_rows, int d) { return wide_rows ? (d == 64 ? 5 : 4) : d == 64 ? 7 : 5; }
constexpr int kSoloChunks = 24, kSoloChunksWide = 12;

struct TreeSizes {
  int R, rows_log2, row_blocks, chunk_log2, min_per;
  bool solo;
  long long entries, grid, slots;
  size_t lse_off, parts_off, bytes;
};

bool tree_sizes(int B, int H, int Hkv, int Tq, int Tmax, int d, int sms, TreeSizes* z) {
  if (B <= 0 || H <= 0 || Hkv <= 0 || Tq <= 0 || Tmax <= 0 || H % Hkv != 0 || (d != 64 && d != 128))
    return false;
  const long long R = static_cast<long long>(H / Hkv) * Tq, BHkv = static_cast<long long>(B) * Hkv;
  if (static_cast<long long>(B) * H > INT32_MAX || R > (1 << 24) || Tmax > (1 << 30)) return false;
  z->R = static_cast<int>(R);
  z->rows_log2 = block_rows_log2(z->R);
  z->row_blocks = (z->R + (1 << z->rows_log2) - 1) >> z->rows_log2;
  z->chunk_log2 = wide(z->R) ? 7 : 6;
  z->min_per = wide(z->R) ? kMinPerWide : kMinPer;
  z->entries = BHkv * z->row_blocks;
  if (z->entries > (1 << 28) || BHkv * R > (1LL << 40) || BHkv > (1LL << 60) / d / Tmax) return false;
  const long long chunks = (static_cast<long long>(Tmax) + (1 << z->chunk_log2) - 1) >> z->chunk_log2;
  if (z->entries * chunks > INT32_MAX - 128) return false;  // (the kernels number them with an int)
  if (z->entries << (z->rows_log2 - 3) > INT32_MAX) return false;
  const long long most = (z->entries * chunks + z->min_per - 1) / z->min_per;
  const long long fit = static_cast<long long>(sms) *
                        (wide(z->R) ? 1 : d == 64 ? TreeCfg<64>::kCtasPerSm : TreeCfg<128>::kCtasPerSm);
  const long long per = std::max<long long>(z->min_per, (z->entries * chunks + fit - 1) / fit);  // a stretch's
  z->solo = z->entries <= fit && chunks <= per + join_chunks(wide(z->R), d) &&
            chunks <= (wide(z->R) ? kSoloChunksWide : kSoloChunks);
  if (z->solo) {
    z->grid = z->entries;
    z->slots = 0;
    z->lse_off = z->parts_off = 0;
    z->bytes = 1;  // none needed
    return true;
  }
  z->grid = std::max<long long>(1, std::min(fit, most));
  z->slots = z->grid + z->entries;
  auto up = [](size_t x) { return (x + 255u) / 256u * 256u; };
  z->lse_off = up((static_cast<size_t>(z->slots) << z->rows_log2) * d * 4);
  z->parts_off = z->lse_off + up((static_cast<size_t>(z->slots) << z->rows_log2) * 4);
  z->bytes = z->parts_off + up(static_cast<size_t>(z->entries) * 8);
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
  if (!q || !k_cache || !v_cache || !o || !lse || !ctx_len) return FA_ERR_INVALID_ARG;
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
  if (!z.solo && (!workspace || workspace_bytes < z.bytes)) return FA_ERR_INVALID_ARG;
  const void* ins[7] = {q, k_cache, v_cache, ctx_len, tree, depths, slopes};
  const size_t in_bytes[7] = {qb, cb, cb, static_cast<size_t>(B) * 4, tb, db, static_cast<size_t>(H) * 4};
  const void* outs[3] = {o, lse, workspace};
  const size_t out_bytes[3] = {qb, lb, z.bytes};
  const int n_outs = z.solo ? 2 : 3;
  for (int x = 0; x < n_outs; ++x) {
    for (int y = 0; y < 7; ++y)
      if (ins[y] && overlaps(outs[x], out_bytes[x], ins[y], in_bytes[y])) return FA_ERR_INVALID_ARG;
    for (int y = x + 1; y < n_outs; ++y)
      if (overlaps(outs[x], out_bytes[x], outs[y], out_bytes[y])) return FA_ERR_INVALID_ARG;
  }
  if (dst != FA_OK) return dst;
  EncodeTiledFn enc = encode_fn();
  if (!enc) return FA_ERR_LAUNCH;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  fa::TreeLaunch a;
  a.p = fa::TreeParams{};
  a.p.q = static_cast<const __nv_bfloat16*>(q);
  a.p.o = static_cast<__nv_bfloat16*>(o);
  a.p.lse = lse;
  if (!z.solo) {
    a.p.o_part = reinterpret_cast<float*>(ws);
    a.p.lse_part = reinterpret_cast<float*>(ws + z.lse_off);
  }
  a.p.slopes = slopes;
  a.p.status = status;
  a.p.timeout_ns = timeout_ns ? timeout_ns : 2000000000ull;
  a.p.list = fa::TreeList{ctx_len, B, Hkv, Tq, Tmax, z.row_blocks, z.min_per, z.chunk_log2, z.solo ? 1 : 0,
                          z.solo ? nullptr : reinterpret_cast<int2*>(ws + z.parts_off)};
  a.p.mask = fa::TreeMask{tree, depths, fa::FastDiv::make(static_cast<uint32_t>(Tq)), tree_per_batch != 0,
                          depths_per_batch != 0};
  a.p.cap = cap;
  a.p.scale_log2 = static_cast<float>(static_cast<double>(scale) * kLog2e);
  a.p.R = z.R;
  a.grid = static_cast<unsigned>(z.grid);
  a.stream = static_cast<cudaStream_t>(stream);
  const int mod = mod_bits(softcap, slopes), BHkv = B * Hkv;
  const int box = 1 << z.chunk_log2;
  if (!encode_map(enc, &a.tm_k, k_cache, Tmax, d, BHkv, box) || !encode_map(enc, &a.tm_v, v_cache, Tmax, d, BHkv, box))
    return FA_ERR_INVALID_ARG;
  cudaError_t e;
  if (fa::wide(z.R)) {
    fa::FwdLaunch f;
    f.p = fa::FwdParams{};
    f.tm_k = a.tm_k;
    f.tm_v = a.tm_v;
    if (!encode_map(enc, &f.tm_q, q, z.R, d, BHkv) || !encode_map(enc, &f.tm_o, o, z.R, d, BHkv, 32))
      return FA_ERR_INVALID_ARG;
    f.p.o = a.p.o;
    f.p.lse = lse;
    f.p.o_part = a.p.o_part;
    f.p.lse_part = a.p.lse_part;
    f.p.status = status;
    f.p.timeout_ns = a.p.timeout_ns;
    f.p.T = z.R;
    f.p.BH = BHkv;
    f.p.tiles_per_cta = 1;
    f.p.div_bh = fa::FastDiv::make(1u);
    f.p.div_splits = fa::FastDiv::make(1u);
    f.p.scale_log2 = mod == fa::kModOn ? exponent_factor(static_cast<double>(scale) * kLog2e, &f.p.s_negate)
                                       : a.p.scale_log2;
    f.p.Tk = Tmax;
    f.p.n_qt = z.row_blocks;
    f.p.n_kv = (Tmax + 127) / 128;
    f.p.n_splits = 1;
    f.p.bmask_heads = 1;
    f.p.mod.slopes = slopes;
    f.p.mod.H = H;
    f.p.mod.div_h = fa::FastDiv::make(1u);
    f.p.mod.div_g = fa::FastDiv::make(1u);
    f.p.mod.cap = cap;
    f.p.mod.list = a.p.list;
    f.p.mod.mask = a.p.mask;
    f.grid = a.grid;
    f.stream = a.stream;
    const int fm = fwd_mod_bits(softcap, slopes, nullptr);
    if ((fm & fa::kModRef) && scale < 0.0f) {  // (as in fa_fwd_mod)
      f.p.s_negate = fa::kIdescNegateA;
      cap_factors(-scale, softcap, &f.p.mod.cap);
    }
    e = (d == 64) ? fa::launch_fwd_tree_d64(f, fm) : fa::launch_fwd_tree_d128(f, fm);
  } else {
    e = (d == 64) ? fa::launch_tree_rows<64>(a, 1 << z.rows_log2, mod) : fa::launch_tree_rows<128>(a, 1 << z.rows_log2, mod);
  }
  if (e != cudaSuccess) return FA_ERR_LAUNCH;
  if (z.solo) return FA_OK;
  const long long groups = z.entries << (z.rows_log2 - 3);  // of eight rows
  const unsigned cg = static_cast<unsigned>(std::min<long long>(groups, static_cast<long long>(sms) * 8));
  auto* combine = d == 64 ? &fa::fa_tree_combine_kernel<64> : &fa::fa_tree_combine_kernel<128>;
  e = fa::launch_pdl(combine, cg, 256, 0, a.stream, a.p, z.rows_log2, static_cast<int>(a.grid),
                     static_cast<unsigned>(groups));
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
