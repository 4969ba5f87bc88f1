// Host side of attention of new tokens against a cache (include/fa.h: fa_fwd_tree,
// fa_fwd_tree_window, fa_fwd_tree4) and the instantiations of its kernels without a window.
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
#include "fa_tree_launch.cuh"

using namespace fa::host;

namespace fa {

namespace {

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
//   a window, d64 (10)         192, 18: 19.2 / 17.0, 10: 12.3 / 11.4;  48, 18: 9.4 / 14.1;  384, 18: 27.6 / 23.4
//                              (its contexts are as unequal, but what is left of them is not)
//   4 bits, 128-key chunks     d64: 48, 4: 7.2 / 6.0, 8: 7.5 / 8.7;  192, 8: 13.1 / 9.9;  d128: 128, 6: 10.9 / 9.2
// With a window or in 4 bits, such an entry is taken by a cluster of CTAs, which join their parts through shared memory:
// as many as fit the GPU at once. (Clusters that do not all fit wait: of 152 places, one an SM, pairs find 152, threes
// 138, fours 144, sixes 138, eights 120, of 304 304, 291, 296, 276, 288; 152 entries in fours on 608 places 19.2 ->
// 23.9 µs, 16 in eights on 152 21.6 -> 28.9.) µs in stretches / in clusters, the chunks of a CTA in these in brackets,
// every context full:
//   a window, d64              8, 18: 7.8 / 6.3 (3), 66: 10.3 / 9.3 (9);  40, 34: 12.1 / 9.4 (5);  96, 18: 12.9 / 9.7 (5);
//                              200, 66: 48.4 / 39.0 (33)
//   d128                       8, 18: 9.6 / 8.6 (3), 66: 12.5 / 13.8 (9);  24, 34: 14.7 / 11.8 (5);  104, 34: 29.1 / 25.6 (17)
//   wide, d64, 128 rows        4, 34: 17.4 / 11.3 (5);  32, 16: 15.5 / 12.2 (4), 66: 28.6 / 23.3 (17);  64, 34: 30.6 / 23.7 (17)
//   d128, 64 rows              4, 34: 18.4 / 13.9 (5), 66: 19.4 / 18.1 (9);  32, 34: 27.0 / 23.2 (9);  64, 66: 60.5 / 58.1 (33)
//   4 bits, full / contexts from none to full (there it is the longest that counts)
//   d64, to 8 rows             24, 32: 9.3 / 7.8 (4), 8.8 / 7.3;  40, 64: 15.2 / 15.8 (8), 12.3 / 12.2;  104, 64: 24.6 / 24.1
//                              (13), 17.8 / 19.3
//   d64, 16 rows               64, 32: 17.1 / 13.4 (8), 18.5 / 12.5;  104, 64: 32.6 / 37.3 (32), 31.7 / 33.5
//   d128, to 8 rows            40, 32: 13.3 / 11.6 (4), 11.3 / 10.5, 64: 19.6 / 19.4 (8), 13.8 / 16.2
//   d128, 16 rows              24, 32: 17.4 / 14.0 (4), 16.6 / 13.2;  96, 64: 50.0 / 45.2 (22), 46.1 / 43.7

// What the new tokens go against: a window (0: none) with sinks, a cache in 4 bits.
struct TreeForm {
  int window, sinks;
  bool four;
};

int join_chunks(bool wide_rows, int d, const TreeForm& form) {
  if (form.four) return d == 64 ? 3 : 2;
  if (form.window > 0) return wide_rows ? 7 : d == 64 ? 10 : 5;
  return wide_rows ? (d == 64 ? 5 : 4) : d == 64 ? 7 : 5;
}
int solo_chunks(bool wide_rows, int d, int rows_log2, const TreeForm& form) {
  if (form.four) return rows_log2 > 3 ? 24 : d == 64 ? 8 : 6;
  return form.window > 0 ? 34 : wide_rows ? 12 : 24;
}
// CTAs a cluster, where `fit` fit the GPU: the most that leave every cluster a place at once. (Few chunks are one CTA's:
// 128 entries of two in 4 bits 4.9 µs, by twos 5.5; 8 of four 6.0, by fours 4.9; wide, d128, 64 entries of four 11.2,
// by twos 12.5; 4 of four 10.2, by fours 8.9.)
int cluster_ctas(bool wide_rows, long long entries, long long chunks, long long fit) {
  if (chunks < (wide_rows && entries > 16 ? 8 : 4)) return 1;
  // (and the places that they find, in sixteenths)
  const int most[5][2] = {{8, wide_rows ? 12 : 14}, {6, 14}, {4, 15}, {3, 14}, {2, 16}};
  for (const auto& m : most)
    if (m[0] <= chunks && entries * m[0] <= fit * m[1] / 16) return m[0];
  return 1;
}

struct TreeSizes {
  int R, rows_log2, row_blocks, chunk_log2, min_per;
  int solo;  // CTAs an entry without stretches, 0: stretches
  long long entries, grid, slots;
  size_t lse_off, parts_off, bytes;
};

// CTAs of the streaming kernels an SM holds.
int tree_ctas(int d) { return d == 64 ? TreeCfg<64>::kCtasPerSm : TreeCfg<128>::kCtasPerSm; }
int tree4_ctas(int d, int rows) {
  return rows == 8 ? (d == 64 ? Tree4Cfg<64, 1>::kCtasPerSm : Tree4Cfg<128, 1>::kCtasPerSm)
                   : (d == 64 ? Tree4Cfg<64, 2>::kCtasPerSm : Tree4Cfg<128, 2>::kCtasPerSm);
}

bool tree_sizes(int B, int H, int Hkv, int Tq, int Tmax, int d, const TreeForm& form, int sms, TreeSizes* z) {
  if (B <= 0 || H <= 0 || Hkv <= 0 || Tq <= 0 || Tmax <= 0 || H % Hkv != 0 || (d != 64 && d != 128))
    return false;
  const long long R = static_cast<long long>(H / Hkv) * Tq, BHkv = static_cast<long long>(B) * Hkv;
  if (static_cast<long long>(B) * H > INT32_MAX || R > (1 << 24) || Tmax > (1 << 30)) return false;
  z->R = static_cast<int>(R);
  // (4 bits: blocks of 8 or 16 rows, the tensor-core kernel's operands being bf16 in shared memory)
  const bool is_wide = wide(z->R) && !form.four;
  z->rows_log2 = form.four ? (z->R <= 8 ? 3 : 4) : block_rows_log2(z->R);
  z->row_blocks = (z->R + (1 << z->rows_log2) - 1) >> z->rows_log2;
  z->chunk_log2 = is_wide || form.four ? 7 : 6;
  z->min_per = is_wide || form.four ? kMinPerWide : kMinPer;
  z->entries = BHkv * z->row_blocks;
  if (z->entries > (1 << 28) || BHkv * R > (1LL << 40) || BHkv > (1LL << 60) / d / Tmax) return false;
  auto chunks_of = [&](long long keys) { return (keys + (1 << z->chunk_log2) - 1) >> z->chunk_log2; };
  long long chunks = chunks_of(Tmax);
  if (form.window > 0)  // those with sinks, and those that a window and the new tokens can reach into
    chunks = std::min(chunks, chunks_of(std::min(form.sinks, Tmax)) + chunks_of(static_cast<long long>(form.window) - 1 + Tq) + 1);
  if (z->entries * chunks > INT32_MAX - 128) return false;  // (the kernels number them with an int)
  if (z->entries << (z->rows_log2 - 3) > INT32_MAX) return false;
  const long long most = (z->entries * chunks + z->min_per - 1) / z->min_per;
  const long long fit = static_cast<long long>(sms) * (is_wide ? 1 : form.four ? tree4_ctas(d, 1 << z->rows_log2) : tree_ctas(d));
  const long long per = std::max<long long>(z->min_per, (z->entries * chunks + fit - 1) / fit);  // a stretch's
  const int ctas = form.four || form.window > 0 ? cluster_ctas(is_wide, z->entries, chunks, fit) : 1;
  const long long most_chunks = (chunks + ctas - 1) / ctas;  // a CTA's
  const bool whole = z->entries <= fit && most_chunks <= per + join_chunks(is_wide, d, form) &&
                     most_chunks <= solo_chunks(is_wide, d, z->rows_log2, form);
  z->solo = whole ? ctas : 0;
  if (z->solo) {
    z->grid = z->entries * z->solo;
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

namespace {

size_t tree_workspace(int B, int H, int Hkv, int Tq, int Tmax, int d, const fa::TreeForm& form) {
  fa::TreeSizes z;
  if (!fa::tree_sizes(B, H, Hkv, Tq, Tmax, d, form, 1, &z)) return 0;
  int dev = -1, sms = 0;
  if (check_device(&dev, &sms) != FA_OK) return 0;
  return fa::tree_sizes(B, H, Hkv, Tq, Tmax, d, form, sms, &z) ? z.bytes : 0;
}

bool tree_window_ok(int window, int sinks) { return window >= 1 && sinks >= 0; }
// (a cache in 4 bits may go without a window)
bool four_ok(int Tmax, int window, int sinks) {
  return Tmax % 8 == 0 && (tree_window_ok(window, sinks) || (window == 0 && sinks == 0));
}

// fa_fwd_tree, fa_fwd_tree_window and fa_fwd_tree4 (whose caches are codes, with scales).
int fwd_tree(const void* q, const void* k_cache, const void* v_cache, const void* k_scales, const void* v_scales,
             void* o, float* lse, const int* ctx_len, const unsigned char* tree, int tree_per_batch,
             const int* depths, int depths_per_batch, const fa::TreeForm& form, float softcap, const float* slopes,
             int B, int H, int Hkv, int Tq, int Tmax, int d, float scale, void* workspace, size_t workspace_bytes,
             int* status, unsigned long long timeout_ns, void* stream) {
  if (!q || !k_cache || !v_cache || !o || !lse || !ctx_len) return FA_ERR_INVALID_ARG;
  if (form.four && (!k_scales || !v_scales)) return FA_ERR_INVALID_ARG;
  fa::TreeSizes z;
  fa::CapFactors cap;
  if (!fa::tree_sizes(B, H, Hkv, Tq, Tmax, d, form, 1, &z) || !scale_ok(scale) || !cap_factors(scale, softcap, &cap))
    return FA_ERR_INVALID_ARG;
  const uintptr_t words = reinterpret_cast<uintptr_t>(ctx_len) | reinterpret_cast<uintptr_t>(depths) |
                          reinterpret_cast<uintptr_t>(slopes);
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scales) || !aligned16(v_scales) ||
      !aligned16(o) || !aligned16(lse) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) || (words & 3u))
    return FA_ERR_MISALIGNED;
  int dev = -1, sms = 0;
  const size_t qb = static_cast<size_t>(B) * H * Tq * d * 2, cb = static_cast<size_t>(B) * Hkv * Tmax * (form.four ? d / 2 : d * 2);
  const size_t sb = static_cast<size_t>(B) * Hkv * Tmax * (d / 16);
  const size_t lb = static_cast<size_t>(B) * H * Tq * 4;
  const size_t tb = static_cast<size_t>(tree_per_batch ? B : 1) * Tq * Tq;
  const size_t db = static_cast<size_t>(depths_per_batch ? B : 1) * Tq * 4;
  const int dst = check_device(&dev, &sms);
  if (dst == FA_OK && !fa::tree_sizes(B, H, Hkv, Tq, Tmax, d, form, sms, &z)) return FA_ERR_INVALID_ARG;
  if (!z.solo && (!workspace || workspace_bytes < z.bytes)) return FA_ERR_INVALID_ARG;
  const void* ins[9] = {q, k_cache, v_cache, ctx_len, tree, depths, slopes, k_scales, v_scales};
  const size_t in_bytes[9] = {qb, cb, cb, static_cast<size_t>(B) * 4, tb, db, static_cast<size_t>(H) * 4, sb, sb};
  const void* outs[3] = {o, lse, workspace};
  const size_t out_bytes[3] = {qb, lb, z.bytes};
  const int n_outs = z.solo ? 2 : 3;
  for (int x = 0; x < n_outs; ++x) {
    for (int y = 0; y < 9; ++y)
      if (ins[y] && overlaps(outs[x], out_bytes[x], ins[y], in_bytes[y])) return FA_ERR_INVALID_ARG;
    for (int y = x + 1; y < n_outs; ++y)
      if (overlaps(outs[x], out_bytes[x], outs[y], out_bytes[y])) return FA_ERR_INVALID_ARG;
  }
  if (dst != FA_OK) return dst;
  EncodeTiledFn enc = form.four ? nullptr : encode_fn();
  if (!enc && !form.four) return FA_ERR_LAUNCH;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  fa::TreeLaunch a{};
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
  a.p.list = fa::TreeList{ctx_len, B, Hkv, Tq, Tmax, z.row_blocks, z.min_per, z.chunk_log2, z.solo,
                          z.solo ? nullptr : reinterpret_cast<int2*>(ws + z.parts_off)};
  a.p.reach = fa::TreeReach{form.four && form.window == 0 ? INT32_MAX : form.window, form.sinks};
  a.p.mask = fa::TreeMask{tree, depths, fa::FastDiv::make(static_cast<uint32_t>(Tq)), tree_per_batch != 0,
                          depths_per_batch != 0};
  a.p.cap = cap;
  a.p.scale_log2 = static_cast<float>(static_cast<double>(scale) * kLog2e);
  a.p.R = z.R;
  a.grid = static_cast<unsigned>(z.grid);
  a.stream = static_cast<cudaStream_t>(stream);
  const int mod = mod_bits(softcap, slopes), BHkv = B * Hkv;
  const int box = 1 << z.chunk_log2;
  if (!form.four && (!encode_map(enc, &a.tm_k, k_cache, Tmax, d, BHkv, box) || !encode_map(enc, &a.tm_v, v_cache, Tmax, d, BHkv, box)))
    return FA_ERR_INVALID_ARG;
  cudaError_t e;
  if (form.four) {
    const fa::Tree4Launch f{{a.p, static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache),
                             static_cast<const __nv_bfloat16*>(k_scales), static_cast<const __nv_bfloat16*>(v_scales)},
                            a.grid, a.stream};
    e = (d == 64) ? fa::launch_tree4_d64(f, 1 << z.rows_log2, mod) : fa::launch_tree4_d128(f, 1 << z.rows_log2, mod);
  } else if (fa::wide(z.R)) {
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
    f.p.mod.reach = a.p.reach;
    f.grid = a.grid;
    f.stream = a.stream;
    const int fm = fwd_mod_bits(softcap, slopes, nullptr);
    if ((fm & fa::kModRef) && scale < 0.0f) {  // (as in fa_fwd_mod)
      f.p.s_negate = fa::kIdescNegateA;
      cap_factors(-scale, softcap, &f.p.mod.cap);
    }
    if (form.window > 0) e = (d == 64) ? fa::launch_fwd_tree_window_d64(f, fm) : fa::launch_fwd_tree_window_d128(f, fm);
    else e = (d == 64) ? fa::launch_fwd_tree_d64(f, fm) : fa::launch_fwd_tree_d128(f, fm);
  } else if (form.window > 0) {
    e = (d == 64) ? fa::launch_tree_window_d64(a, 1 << z.rows_log2, mod) : fa::launch_tree_window_d128(a, 1 << z.rows_log2, mod);
  } else {
    e = (d == 64) ? fa::launch_tree_rows<64, 0>(a, 1 << z.rows_log2, mod) : fa::launch_tree_rows<128, 0>(a, 1 << z.rows_log2, mod);
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

}  // namespace

extern "C" {

size_t fa_fwd_tree_workspace_size(int B, int H, int Hkv, int Tq, int Tmax, int d) {
  return tree_workspace(B, H, Hkv, Tq, Tmax, d, {0, 0, false});
}

int fa_fwd_tree(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                const int* ctx_len, const unsigned char* tree, int tree_per_batch, const int* depths,
                int depths_per_batch, float softcap, const float* slopes, int B, int H, int Hkv, int Tq,
                int Tmax, int d, float scale, void* workspace, size_t workspace_bytes, int* status,
                unsigned long long timeout_ns, void* stream) {
  return fwd_tree(q, k_cache, v_cache, nullptr, nullptr, o, lse, ctx_len, tree, tree_per_batch, depths, depths_per_batch,
                  {0, 0, false}, softcap, slopes, B, H, Hkv, Tq, Tmax, d, scale, workspace, workspace_bytes, status, timeout_ns, stream);
}

size_t fa_fwd_tree_window_workspace_size(int B, int H, int Hkv, int Tq, int Tmax, int d, int window, int sinks) {
  return tree_window_ok(window, sinks) ? tree_workspace(B, H, Hkv, Tq, Tmax, d, {window, sinks, false}) : 0;
}

int fa_fwd_tree_window(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                       const int* ctx_len, const unsigned char* tree, int tree_per_batch, const int* depths,
                       int depths_per_batch, int window, int sinks, float softcap, const float* slopes, int B, int H,
                       int Hkv, int Tq, int Tmax, int d, float scale, void* workspace, size_t workspace_bytes,
                       int* status, unsigned long long timeout_ns, void* stream) {
  if (!tree_window_ok(window, sinks)) return FA_ERR_INVALID_ARG;
  return fwd_tree(q, k_cache, v_cache, nullptr, nullptr, o, lse, ctx_len, tree, tree_per_batch, depths, depths_per_batch,
                  {window, sinks, false}, softcap, slopes, B, H, Hkv, Tq, Tmax, d, scale, workspace, workspace_bytes, status, timeout_ns, stream);
}

size_t fa_fwd_tree4_workspace_size(int B, int H, int Hkv, int Tq, int Tmax, int d, int window, int sinks) {
  return four_ok(Tmax, window, sinks) ? tree_workspace(B, H, Hkv, Tq, Tmax, d, {window, sinks, true}) : 0;
}

int fa_fwd_tree4(const void* q, const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                 void* o, float* lse, const int* ctx_len, const unsigned char* tree, int tree_per_batch,
                 const int* depths, int depths_per_batch, int window, int sinks, float softcap, const float* slopes,
                 int B, int H, int Hkv, int Tq, int Tmax, int d, float scale, void* workspace, size_t workspace_bytes,
                 int* status, unsigned long long timeout_ns, void* stream) {
  if (!four_ok(Tmax, window, sinks)) return FA_ERR_INVALID_ARG;
  return fwd_tree(q, k_codes, v_codes, k_scales, v_scales, o, lse, ctx_len, tree, tree_per_batch, depths, depths_per_batch,
                  {window, sinks, true}, softcap, slopes, B, H, Hkv, Tq, Tmax, d, scale, workspace, workspace_bytes, status,
                  timeout_ns, stream);
}

}  // extern "C"
