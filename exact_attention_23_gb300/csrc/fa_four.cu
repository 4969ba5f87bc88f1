// Into a cache held in 4 bits and out of it (include/fa.h: fa_append4, fa_read4; the format: fa_four.cuh).
//
// Both move bytes: a row of d values is read once as bf16 (2d bytes) and written as d/2 + d/16, or the
// other way. d/8 neighbouring lanes take a row, 16 bytes of bf16 each; a group's largest magnitude goes
// through its four lanes in two shuffles, and the lanes' eight codes, one word, are brought into the order
// of the format by one shuffle (keys: halves of words) or three (values: 8 × 8 codes transposed), so
// that whole words are written. kFourFlight rows a thread are in flight.
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
  long long rows;                // 2 · B · Hkv · n
  int B, Hkv, n, Tmax;
};

constexpr int kFourThreads = 256;
constexpr int kFourFlight = 4;

// The row that a number stands for.
struct FourRow {
  int kv, b, h, t;
  size_t at;      // row of the cache
  bool in, held;  // the number is one; the cache has the row
};
__device__ __forceinline__ FourRow four_row(const FourParams& p, long long r) {
  FourRow x;
  x.in = r < p.rows;
  const long long y = x.in ? r / p.n : 0;
  x.t = static_cast<int>((x.in ? r : 0) - y * p.n);
  const int heads = p.B * p.Hkv, z = static_cast<int>(y);
  x.kv = z >= heads;
  const int bh = z - x.kv * heads;
  x.b = bh / p.Hkv;
  x.h = bh - x.b * p.Hkv;
  const int start = p.start[x.b];
  const long long row = static_cast<long long>(start) + x.t;
  x.held = x.in && start >= 0 && row < p.Tmax;
  x.at = static_cast<size_t>(bh) * p.Tmax + static_cast<size_t>(x.held ? row : 0);
  return x;
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
  const int x = threadIdx.x % kLanes;
  const long long r0 = static_cast<long long>(blockIdx.x) * (kRows * kFourFlight) + threadIdx.x / kLanes;
  FourRow row[kFourFlight];
  uint4 in[kFourFlight];
#pragma unroll
  for (int i = 0; i < kFourFlight; ++i) {
    row[i] = four_row(p, r0 + i * kRows);
    const RopeSrc s = row[i].kv ? p.v : p.k;
    in[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row[i].held)
      in[i] = *reinterpret_cast<const uint4*>(s.p + row[i].b * s.sb + row[i].h * s.sh + row[i].t * s.st + x * 8);
  }
#pragma unroll
  for (int i = 0; i < kFourFlight; ++i) {
    float v[8];
    unpack8(in[i], v);
    uint32_t top = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float s = four_scale_of(top);
    uint32_t w = 0x88888888u;  // (zeros, and groups that are no numbers)
    if (s > 0.f) {
      const float inv = __frcp_rn(s);
      w = 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) w |= four_code(v[e], s, inv) << (4 * e);
    }
    // (the lanes of a warp hold rows of both kinds where the keys end)
    const uint32_t wk = four_to_key(w, x), wv = four_transpose(w, x & 7);
    if (!row[i].held) continue;
    const int kv = row[i].kv;
    *reinterpret_cast<uint32_t*>(p.codes[kv] + row[i].at * (D / 2) + four_word<D>(kv, x) * 4) = kv ? wv : wk;
    if ((x & 3) == 0) p.scales[kv][row[i].at * (D / 32) + (x >> 2)] = __float2bfloat16_rn(s);
  }
}

template <int D>
__global__ void __launch_bounds__(kFourThreads) fa_read4_kernel(const FourParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kLanes = D / 8, kRows = kFourThreads / kLanes;
  const int x = threadIdx.x % kLanes;
  const long long r0 = static_cast<long long>(blockIdx.x) * (kRows * kFourFlight) + threadIdx.x / kLanes;
  FourRow row[kFourFlight];
  uint32_t w[kFourFlight];
  float s[kFourFlight];
#pragma unroll
  for (int i = 0; i < kFourFlight; ++i) {
    row[i] = four_row(p, r0 + i * kRows);
    const int kv = row[i].kv;
    w[i] = 0u;
    s[i] = 0.f;
    if (row[i].held) {
      w[i] = *reinterpret_cast<const uint32_t*>(p.codes[kv] + row[i].at * (D / 2) + four_word<D>(kv, x) * 4);
      s[i] = __bfloat162float(p.scales[kv][row[i].at * (D / 32) + (x >> 2)]);
    }
  }
#pragma unroll
  for (int i = 0; i < kFourFlight; ++i) {
    const uint32_t a = four_from_key(w[i], x), b = four_transpose(w[i], x & 7);
    const uint32_t c = row[i].kv ? b : a;
    if (!row[i].in) continue;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = row[i].held ? static_cast<float>(static_cast<int>((c >> (4 * e)) & 15u) - 8) * s[i] : 0.f;
    __nv_bfloat16* out = row[i].kv ? p.v_out : p.k_out;
    *reinterpret_cast<uint4*>(out + ((static_cast<size_t>(row[i].b) * p.Hkv + row[i].h) * p.n + row[i].t) * D + x * 8) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

namespace {

using namespace fa::host;

bool four_sizes(int B, int Hkv, int n, int Tmax, int d) {
  if (B <= 0 || Hkv <= 0 || n <= 0 || Tmax <= 0 || Tmax % 8 != 0 || (d != 64 && d != 128)) return false;
  const long long heads = static_cast<long long>(B) * Hkv;
  if (heads > (1 << 30) || heads > (1LL << 60) / d / Tmax || heads > (1LL << 38) / n) return false;
  // (blocks of at least 64 rows)
  return 2 * heads * n / 64 < INT32_MAX;
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
int four_launch(Fn* fn, const FourParams& p, int d, void* stream) {
  const long long per = static_cast<long long>(kFourThreads) / (d / 8) * kFourFlight;
  const unsigned grid = static_cast<unsigned>((p.rows + per - 1) / per);
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
  p.rows = 2LL * B * Hkv * Tq;
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
  p.rows = 2LL * B * Hkv * n;
  p.B = B; p.Hkv = Hkv; p.n = n; p.Tmax = Tmax;
  if (!aligned16(k_out) || !aligned16(v_out) || four_misaligned(p)) return FA_ERR_MISALIGNED;
  const void* rows[2] = {k_out, v_out};
  const size_t bytes = static_cast<size_t>(B) * Hkv * n * d * 2, row_bytes[2] = {bytes, bytes};
  const int st = four_check(p, d, rows, row_bytes, false);
  if (st != FA_OK) return st;
  return four_launch(d == 64 ? &fa_read4_kernel<64> : &fa_read4_kernel<128>, p, d, stream);
}

}  // extern "C"
