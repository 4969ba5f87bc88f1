// Into a cache held in 4 bits and out of it (include/fa.h: fa_append4, fa_read4; the format: fa_four.cuh).
//
// Both move bytes: a row of d values is read once as bf16 (2d bytes) and written as d/2 + d/16, or the
// other way. d/8 neighbouring lanes take a row, 16 bytes of bf16 each; a group's largest magnitude goes
// through its four lanes in two shuffles, and the lanes' eight codes, one word, are brought into the order
// of the format by one shuffle (keys: halves of words) or three (values: 8 × 8 codes transposed), so
// that whole words are written. kFourFlight rows a thread are in flight. 98304 rows of d = 64 in and out again (57 MB):
// 15.4 µs for both, 3.7 TB/s (36 with divisions for the quotients and the rows' numbers; instructions, 74 % of what
// an SM can issue, are what is left); one token of eight sequences: 3.7, two launches.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "fa.h"
#include "fa_four.cuh"
#include "fa_host.h"
#include "fa_pdl.h"
#include "fa_rope.cuh"
#include "sm103.cuh"

namespace fa {

struct FourParams {
  RopeSrc k, v;                  // append: the new rows
  __nv_bfloat16 *k_out, *v_out;  // read: [B][Hkv][n][d]
  uint8_t* codes[2];             // keys', values': [B][Hkv][Tmax][d/2]
  __nv_bfloat16* scales[2];      // [B][Hkv][Tmax][d/32]
  const int* start;              // [B]: the first of the n rows; < 0: none
  unsigned blocks;               // blocks a head
  int B, Hkv, n, Tmax;
};

constexpr int kFourThreads = 256;
constexpr int kFourFlight = 4;

// The rows of a block, all of one head: kFourFlight times the rows its threads take at once.
struct FourBlock {
  int kv, b, h, t0;
  size_t head;  // b·Hkv + h
};
__device__ __forceinline__ FourBlock four_block(const FourParams& p, int rows) {
  const unsigned x = blockIdx.x / p.blocks, heads = static_cast<unsigned>(p.B) * p.Hkv;
  FourBlock f;
  f.t0 = static_cast<int>(blockIdx.x - x * p.blocks) * rows;
  f.kv = x >= heads;
  const unsigned bh = x - (f.kv ? heads : 0u);
  f.head = bh;
  f.b = static_cast<int>(bh / static_cast<unsigned>(p.Hkv));
  f.h = static_cast<int>(bh - static_cast<unsigned>(f.b) * p.Hkv);
  return f;
}

// Which word of a row lane x (of d/8) holds, in the keys' or the values' order.
template <int D>
__device__ __forceinline__ int four_word(int kv, int x) {
  return kv ? x : four_key_word(x) * (D / 32) + (x >> 2);
}

template <int D>
__global__ void __launch_bounds__(kFourThreads) fa_append4_kernel(const FourParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kLanes = D / 8, kRows = kFourThreads / kLanes;  // rows a block takes at once
  const FourBlock f = four_block(p, kRows * kFourFlight);
  const int x = threadIdx.x % kLanes, t0 = f.t0 + threadIdx.x / kLanes;
  const int start = p.start[f.b];
  const RopeSrc s = f.kv ? p.v : p.k;
  const __nv_bfloat16* src = s.p + f.b * s.sb + f.h * s.sh + x * 8;
  uint4 in[kFourFlight];  // (read whether or not the cache has the row: no load waits for the length)
#pragma unroll
  for (int i = 0; i < kFourFlight; ++i) {
    const int t = t0 + i * kRows;
    in[i] = t < p.n ? *reinterpret_cast<const uint4*>(src + t * s.st) : make_uint4(0u, 0u, 0u, 0u);
  }
  // (rows behind `end` have no place in the cache, or are none)
  const int end = start < 0 ? 0 : static_cast<int>(min(static_cast<long long>(p.n), static_cast<long long>(p.Tmax) - start));
  const size_t at = f.head * p.Tmax + static_cast<size_t>(max(start, 0)) + t0;
  uint8_t* codes = p.codes[f.kv] + at * (D / 2) + four_word<D>(f.kv, x) * 4;
  __nv_bfloat16* scales = p.scales[f.kv] + at * (D / 32) + (x >> 2);
#pragma unroll
  for (int i = 0; i < kFourFlight; ++i) {
    float v[8];
    unpack8(in[i], v);
    const float sc = four_scale_of(four_top(in[i]));
    uint32_t w = 0x88888888u;  // (zeros, and groups that are no numbers)
    if (sc > 0.f) w = four_codes(v, sc);
    w = f.kv ? four_transpose(w, x & 7) : four_to_key(w, x);
    const int t = t0 + i * kRows;
    if (t >= end) continue;
    *reinterpret_cast<uint32_t*>(codes + i * kRows * (D / 2)) = w;
    if ((x & 3) == 0) scales[i * kRows * (D / 32)] = __float2bfloat16_rn(sc);
  }
}

template <int D>
__global__ void __launch_bounds__(kFourThreads) fa_read4_kernel(const FourParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kLanes = D / 8, kRows = kFourThreads / kLanes;
  const FourBlock f = four_block(p, kRows * kFourFlight);
  const int x = threadIdx.x % kLanes, t0 = f.t0 + threadIdx.x / kLanes;
  const int start = p.start[f.b];
  const int end = start < 0 ? 0 : static_cast<int>(min(static_cast<long long>(p.n), static_cast<long long>(p.Tmax) - start));
  const size_t at = f.head * p.Tmax + static_cast<size_t>(max(start, 0)) + t0;
  const uint8_t* codes = p.codes[f.kv] + at * (D / 2) + four_word<D>(f.kv, x) * 4;
  const unsigned short* scales = reinterpret_cast<const unsigned short*>(p.scales[f.kv]) + at * (D / 32) + (x >> 2);
  uint32_t w[kFourFlight], s[kFourFlight];  // (a scale twice in a word)
#pragma unroll
  for (int i = 0; i < kFourFlight; ++i) {
    w[i] = 0u;
    s[i] = 0u;
    if (t0 + i * kRows >= end) continue;
    w[i] = *reinterpret_cast<const uint32_t*>(codes + i * kRows * (D / 2));
    s[i] = scales[i * kRows * (D / 32)] * 0x10001u;
  }
  __nv_bfloat16* out = (f.kv ? p.v_out : p.k_out) + f.head * p.n * D + x * 8;
#pragma unroll
  for (int i = 0; i < kFourFlight; ++i) {
    const int t = t0 + i * kRows;
    const uint32_t c = f.kv ? four_transpose(w[i], x & 7) : four_from_key(w[i], x);
    if (t >= p.n) continue;
    // (with a scale of 0 where no row was read: zeros, of either sign as they come)
    const FourScale g = four_scale(s[i]);
    const uint32_t x0 = four_pair<0>(c, g), x1 = four_pair<1>(c, g), x2 = four_pair<2>(c, g), x3 = four_pair<3>(c, g);
    *reinterpret_cast<uint4*>(out + static_cast<size_t>(t) * D) =
        make_uint4(__byte_perm(x0, x1, 0x5410), __byte_perm(x2, x3, 0x5410), __byte_perm(x0, x1, 0x7632),
                   __byte_perm(x2, x3, 0x7632));
  }
}

namespace {

using namespace fa::host;

bool four_sizes(int B, int Hkv, int n, int Tmax, int d) {
  if (B <= 0 || Hkv <= 0 || n <= 0 || Tmax <= 0 || Tmax % 8 != 0 || (d != 64 && d != 128)) return false;
  if (n > (1 << 30)) return false;  // (rows behind the last of a block fit an int)
  const long long heads = static_cast<long long>(B) * Hkv;
  if (heads > (1 << 30) || heads > (1LL << 60) / d / Tmax || heads > (1LL << 38) / n) return false;
  // (a block takes at least 64 rows of a head)
  return 2 * heads * ((static_cast<long long>(n) + 63) / 64) < INT32_MAX;
}

// Sizes, pointers and overlaps of both calls: `rows` are the bf16 rows of keys and values.
int four_check(const FourParams& p, int d, const void* const rows[2], const size_t row_bytes[2], bool append) {
  const size_t heads = static_cast<size_t>(p.B) * p.Hkv, cb = heads * p.Tmax * d / 2, sb = heads * p.Tmax * (d / 16);
  const void* cache[4] = {p.codes[0], p.codes[1], p.scales[0], p.scales[1]};
  const size_t cache_bytes[4] = {cb, cb, sb, sb};
  const size_t start_bytes = static_cast<size_t>(p.B) * 4;
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 2; ++j)
      if (overlaps(cache[i], cache_bytes[i], rows[j], row_bytes[j])) return FA_ERR_INVALID_ARG;
    if (append) {
      if (overlaps(cache[i], cache_bytes[i], p.start, start_bytes)) return FA_ERR_INVALID_ARG;
      for (int j = i + 1; j < 4; ++j)
        if (overlaps(cache[i], cache_bytes[i], cache[j], cache_bytes[j])) return FA_ERR_INVALID_ARG;
    }
  }
  if (!append) {
    for (int j = 0; j < 2; ++j)
      if (overlaps(rows[j], row_bytes[j], p.start, start_bytes)) return FA_ERR_INVALID_ARG;
    if (overlaps(rows[0], row_bytes[0], rows[1], row_bytes[1])) return FA_ERR_INVALID_ARG;
  }
  int dev = -1, sms = 0;
  return check_device(&dev, &sms);
}

template <typename Fn>
int four_launch(Fn* fn, FourParams& p, int d, void* stream) {
  const unsigned per = kFourThreads / (static_cast<unsigned>(d) / 8) * kFourFlight;
  p.blocks = (static_cast<unsigned>(p.n) + per - 1) / per;
  const unsigned grid = 2u * static_cast<unsigned>(p.B) * p.Hkv * p.blocks;
  return launch_pdl(fn, grid, kFourThreads, 0, static_cast<cudaStream_t>(stream), p) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

bool four_misaligned(const FourParams& p) {
  return !aligned16(p.codes[0]) || !aligned16(p.codes[1]) || !aligned16(p.scales[0]) || !aligned16(p.scales[1]) ||
         (reinterpret_cast<uintptr_t>(p.start) & 3u);
}

}  // namespace

}  // namespace fa

using namespace fa;
using namespace fa::host;

extern "C" {

int fa_append4(const void* k, long long k_sb, long long k_sh, long long k_st, const void* v, long long v_sb,
               long long v_sh, long long v_st, void* k_codes, void* k_scales, void* v_codes, void* v_scales,
               const int* ctx_len, int B, int Hkv, int Tq, int Tmax, int d, void* stream) {
  if (!k || !v || !k_codes || !k_scales || !v_codes || !v_scales || !ctx_len || !four_sizes(B, Hkv, Tq, Tmax, d))
    return FA_ERR_INVALID_ARG;
  FourParams p{};
  p.k = {static_cast<const __nv_bfloat16*>(k), k_sb, k_sh, k_st};
  p.v = {static_cast<const __nv_bfloat16*>(v), v_sb, v_sh, v_st};
  p.codes[0] = static_cast<uint8_t*>(k_codes);
  p.codes[1] = static_cast<uint8_t*>(v_codes);
  p.scales[0] = static_cast<__nv_bfloat16*>(k_scales);
  p.scales[1] = static_cast<__nv_bfloat16*>(v_scales);
  p.start = ctx_len;
  p.B = B; p.Hkv = Hkv; p.n = Tq; p.Tmax = Tmax;
  if (!aligned16(k) || !aligned16(v) || four_misaligned(p)) return FA_ERR_MISALIGNED;
  const void* rows[2] = {k, v};
  const size_t row_bytes[2] = {span_bytes(p.k, B, Hkv, Tq, d), span_bytes(p.v, B, Hkv, Tq, d)};
  if (row_bytes[0] == 0 || row_bytes[1] == 0) return FA_ERR_INVALID_ARG;
  const int st = four_check(p, d, rows, row_bytes, true);
  if (st != FA_OK) return st;
  return four_launch(d == 64 ? &fa_append4_kernel<64> : &fa_append4_kernel<128>, p, d, stream);
}

int fa_read4(const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales, const int* start,
             void* k_out, void* v_out, int B, int Hkv, int n, int Tmax, int d, void* stream) {
  if (!k_codes || !k_scales || !v_codes || !v_scales || !start || !k_out || !v_out || !four_sizes(B, Hkv, n, Tmax, d))
    return FA_ERR_INVALID_ARG;
  FourParams p{};
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.codes[0] = static_cast<uint8_t*>(const_cast<void*>(k_codes));
  p.codes[1] = static_cast<uint8_t*>(const_cast<void*>(v_codes));
  p.scales[0] = static_cast<__nv_bfloat16*>(const_cast<void*>(k_scales));
  p.scales[1] = static_cast<__nv_bfloat16*>(const_cast<void*>(v_scales));
  p.start = start;
  p.B = B; p.Hkv = Hkv; p.n = n; p.Tmax = Tmax;
  if (!aligned16(k_out) || !aligned16(v_out) || four_misaligned(p)) return FA_ERR_MISALIGNED;
  const void* rows[2] = {k_out, v_out};
  const size_t bytes = static_cast<size_t>(B) * Hkv * n * d * 2, row_bytes[2] = {bytes, bytes};
  const int st = four_check(p, d, rows, row_bytes, false);
  if (st != FA_OK) return st;
  return four_launch(d == 64 ? &fa_read4_kernel<64> : &fa_read4_kernel<128>, p, d, stream);
}

}  // extern "C"
