// Host side of attention with modified scores (include/fa.h: fa_visible, fa_fwd_mod, fa_bwd_mod)
// and the kernel that makes a batch's visibility.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "fa.h"
#include "fa_host.h"
#include "fa_launch.h"
#include "fa_mod_host.h"

using namespace fa::host;

namespace fa {

// What fa_visible writes (one buffer, sections on 256-byte boundaries):
//   rows   int2 [B][T_pad]  visible keys [lo, hi) of each query row ((0, 0): none; padding too)
//   fwd    int4 [B][n_t]    query tiles, most K tiles first: (tile, first K tile, past the last,
//                           first tile with padding or n_t)
//   pairs  int4 [B][n_p][2] pairs of neighbouring query tiles, n_p = ceil(n_t / 2), the longest walk
//                           first: (first tile, first tile with padding, its first K tile, past its last), (the
//                           second tile's first K tile and past its last, 0, 0)
//   bwd    int4 [B][n_t]    key tiles, most query tiles first: (tile, first query tile, past the
//                           last, 2 · first tile with padding + whether this key tile has any)
//   whole  int2 [B][n_t]    (largest lo, smallest hi) over a tile's rows: hi is 0 with padding, and only then
//   span   int2 [B][n_t]    (smallest lo, largest hi) over the rows that see a key
//   seen   int2 [B][n_t]    (first, past the last) query tile that sees a key tile
struct VisibleLayout {
  size_t rows, fwd, pairs, bwd, whole, span, seen, bytes;
};

static VisibleLayout visible_layout(int B, int T) {
  auto up = [](size_t x) { return (x + 255u) / 256u * 256u; };
  const size_t n_t = (static_cast<size_t>(T) + 127) / 128, b = static_cast<size_t>(B);
  VisibleLayout l;
  l.rows = 0;
  l.fwd = up(b * n_t * 128 * 8);
  l.pairs = l.fwd + up(b * n_t * 16);
  l.bwd = l.pairs + up(b * ((n_t + 1) / 2) * 32);
  l.whole = l.bwd + up(b * n_t * 16);
  l.span = l.whole + up(b * n_t * 8);
  l.seen = l.span + up(b * n_t * 8);
  l.bytes = l.seen + up(b * n_t * 8);
  return l;
}

struct VisibleParams {
  const int* ids;     // [B][T] or null
  const int* prefix;  // [B] or [B][T] or null
  int prefix_per_token, causal, T, n_t;
  int2* rows;
  int4 *fwd, *pairs, *bwd;
  int2 *whole, *span, *seen;
};

constexpr int kVisThreads = 1024;
constexpr int kVisTiles = 1024;

// The document starts and the paddings among 32 rows from i0 on, as bits (rows past `end`: 0).
// Eight loads stand together, so a group costs four round trips.
__device__ __forceinline__ void doc_bits(const int* ids, int i0, int end, uint32_t* starts, uint32_t* pads) {
  uint32_t st = 0u, pad = 0u;
  if (!ids) {
    *starts = i0 == 0 && end > 0 ? 1u : 0u;
    *pads = 0u;
    return;
  }
  int prev = i0 > 0 && i0 < end ? ids[i0 - 1] : 0;
#pragma unroll 1
  for (int o = 0; o < 32 && i0 + o < end; o += 8) {
    int id[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) id[e] = ids[min(i0 + o + e, end - 1)];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = i0 + o + e;
      if (i < end) {
        if (i == 0 || id[e] != prev) st |= 1u << (o + e);
        if (id[e] < 0) pad |= 1u << (o + e);
      }
      prev = id[e];
    }
  }
  *starts = st;
  *pads = pad;
}

// One block a sequence. A document is a maximal run of equal ids, so a row's document starts at
// the last change of id at or before it and ends at the next one after it: a running maximum and
// a running minimum, each thread taking one stretch of rows (as bits, 32 rows at a time) and the
// block joining the stretches. Then a warp a tile: its rows' extremes, the query tiles that see
// it, and its place among the tiles by the number it has to walk (a count of the tiles before it:
// n_t² comparisons, which at 16384 tokens are 4 a lane and tile). Latency is all it costs; the
// tiles' extremes are kept in shared memory up to kVisTiles of them.
__global__ void __launch_bounds__(kVisThreads) fa_visible_kernel(const VisibleParams p) {
  __shared__ int s_last[kVisThreads / 32], s_first[kVisThreads / 32];
  __shared__ int s_pad;
  __shared__ int2 s_span[kVisTiles], s_seen[kVisTiles];
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kVisThreads / 32;
  const int T = p.T, n_t = p.n_t;
  const long long T_pad = static_cast<long long>(n_t) * 128;
  const int* ids = p.ids ? p.ids + static_cast<size_t>(b) * T : nullptr;
  int2* rows = p.rows + static_cast<size_t>(b) * T_pad;
  int2* span = n_t <= kVisTiles ? s_span : p.span + static_cast<size_t>(b) * n_t;
  int2* seen = n_t <= kVisTiles ? s_seen : p.seen + static_cast<size_t>(b) * n_t;
  if (tid == 0) s_pad = n_t;
  const long long seg = (T_pad + kVisThreads - 1) / kVisThreads;
  const int a0 = static_cast<int>(min(static_cast<long long>(T), tid * seg));
  const int a1 = static_cast<int>(min(static_cast<long long>(T), (tid + 1) * seg));
  uint32_t starts = 0u, pads = 0u;
  int last = -1, first = T;  // this stretch's last and first document starts
  for (int g0 = a0; g0 < a1; g0 += 32) {
    doc_bits(ids, g0, a1, &starts, &pads);
    if (starts) {
      last = g0 + 31 - __clz(starts);
      if (first == T) first = g0 + __ffs(starts) - 1;
    }
  }
  // inclusive scans over the block's stretches: maximum from the left, minimum from the right
  int mx = last, mn = first;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, mx, off), c = __shfl_down_sync(0xffffffffu, mn, off);
    if (lane >= off) mx = max(mx, a);
    if (lane + off < 32) mn = min(mn, c);
  }
  if (lane == 31) s_last[warp] = mx;
  if (lane == 0) s_first[warp] = mn;
  __syncthreads();
  int cur = __shfl_up_sync(0xffffffffu, mx, 1), end = __shfl_down_sync(0xffffffffu, mn, 1);
  if (lane == 0) cur = -1;
  if (lane == 31) end = T;
  {
    // the warps before and after, a lane each
    const int l = lane < warp ? s_last[lane] : -1, f = lane > warp ? s_first[lane] : T;
    cur = max(max(cur, __reduce_max_sync(0xffffffffu, l)), 0);
    end = min(end, __reduce_min_sync(0xffffffffu, f));
  }
  const bool one = a1 - a0 <= 32;  // the stretch's bits are still in registers
  if (!one) {  // the rows' starts, front to back, for the pass below
    int c = cur;
    for (int g0 = a0; g0 < a1; g0 += 32) {
      doc_bits(ids, g0, a1, &starts, &pads);
      for (int o = 0; o < min(32, a1 - g0); ++o) {
        if ((starts >> o) & 1u) c = g0 + o;
        rows[g0 + o].x = c;
      }
    }
  }
  int padded = n_t;  // the first tile with padding
  const int* pre_at = nullptr;
  int pre_all = 0;
  if (p.prefix && p.causal) {
    if (p.prefix_per_token) pre_at = p.prefix + static_cast<size_t>(b) * T;
    else pre_all = max(0, p.prefix[b]);
  }
  for (int g0 = a0 + max(0, (a1 - a0 - 1)) / 32 * 32; g0 >= a0 && a1 > a0; g0 -= 32) {
    if (!one) doc_bits(ids, g0, a1, &starts, &pads);
    for (int o = min(32, a1 - g0) - 1; o >= 0; --o) {
      const int i = g0 + o;
      int lo;
      if (one) {
        const uint32_t at = starts & ((2u << o) - 1u);
        lo = at ? g0 + 31 - __clz(at) : cur;
      } else {
        lo = rows[i].x;
      }
      int2 r = make_int2(lo, end);
      if ((pads >> o) & 1u) {
        r = make_int2(0, 0);
        padded = i >> 7;  // (from the back)
      } else {
        if (p.causal) {
          const int pre = pre_at ? max(0, pre_at[i]) : pre_all;
          r.y = max(i + 1, pre > end - lo ? end : lo + pre);
        }
      }
      rows[i] = r;
      if (lo == i) end = i;
    }
  }
  for (long long i = T + tid; i < T_pad; i += kVisThreads) rows[i] = make_int2(0, 0);
  padded = __reduce_min_sync(0xffffffffu, padded);
  if (lane == 0) atomicMin(&s_pad, padded);
  __syncthreads();
  const size_t t0 = static_cast<size_t>(b) * n_t;
  for (int t = warp; t < n_t; t += kWarps) {
    int lo_min = T, hi_max = 0, lo_max = 0, hi_min = T;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = t * 128 + lane + 32 * k;
      if (i >= T) continue;
      const int2 r = rows[i];
      lo_max = max(lo_max, r.x);
      hi_min = min(hi_min, r.y);
      if (r.y > r.x) {
        lo_min = min(lo_min, r.x);
        hi_max = max(hi_max, r.y);
      }
    }
    lo_min = __reduce_min_sync(0xffffffffu, lo_min);
    hi_min = __reduce_min_sync(0xffffffffu, hi_min);
    lo_max = __reduce_max_sync(0xffffffffu, lo_max);
    hi_max = __reduce_max_sync(0xffffffffu, hi_max);
    if (lane == 0) {
      p.whole[t0 + t] = make_int2(lo_max, hi_min);
      span[t] = hi_max > lo_min ? make_int2(lo_min, hi_max) : make_int2(0, 0);
    }
  }
  __syncthreads();
  padded = s_pad;
  for (int t = warp; t < n_t; t += kWarps) {
    // the query tiles whose rows see a key of this tile
    int f = n_t, l = 0;
    const int k0 = t * 128;
    for (int q = lane; q < n_t; q += 32) {
      const int2 s = span[q];
      if (s.y > k0 && s.x < k0 + 128) {
        f = min(f, q);
        l = max(l, q + 1);
      }
    }
    f = __reduce_min_sync(0xffffffffu, f);
    l = __reduce_max_sync(0xffffffffu, l);
    if (lane == 0) seen[t] = l > f ? make_int2(f, l) : make_int2(0, 0);
  }
  __syncthreads();
  for (int t = warp; t < n_t; t += kWarps) {
    const int2 s = span[t], k = seen[t];
    const int kb = s.x >> 7, ke = (s.y + 127) >> 7;
    int rf = 0, rb = 0;
    for (int q = lane; q < n_t; q += 32) {
      const int2 os = span[q], ok = seen[q];
      const int on = ((os.y + 127) >> 7) - (os.x >> 7), on2 = ok.y - ok.x;
      rf += on > ke - kb || (on == ke - kb && q < t);
      rb += on2 > k.y - k.x || (on2 == k.y - k.x && q < t);
    }
    rf = __reduce_add_sync(0xffffffffu, rf);
    rb = __reduce_add_sync(0xffffffffu, rb);
    if (lane == 0) {
      p.fwd[t0 + rf] = make_int4(t, kb, ke, padded);
      p.bwd[t0 + rb] = make_int4(t, k.x, k.y, 2 * padded + (p.whole[t0 + t].y == 0 ? 1 : 0));
    }
  }
  // Pairs of query tiles, by the length of their union's walk.
  const int n_p = (n_t + 1) / 2;
  auto walk = [&](int t) {  // first K tile and past the last; (0, 0): none
    const int2 s = t < n_t ? span[t] : make_int2(0, 0);
    return make_int2(s.x >> 7, (s.y + 127) >> 7);
  };
  auto steps = [&](int2 a, int2 c) {
    if (a.y <= a.x) return c.y - c.x;
    if (c.y <= c.x) return a.y - a.x;
    return max(a.y, c.y) - min(a.x, c.x);
  };
  for (int t = warp; t < n_p; t += kWarps) {
    const int2 a = walk(2 * t), c = walk(2 * t + 1);
    const int n = steps(a, c);
    int r = 0;
    for (int q = lane; q < n_p; q += 32) {
      const int m = steps(walk(2 * q), walk(2 * q + 1));
      r += m > n || (m == n && q < t);
    }
    r = __reduce_add_sync(0xffffffffu, r);
    if (lane == 0) {
      int4* out = p.pairs + (static_cast<size_t>(b) * n_p + r) * 2;
      out[0] = make_int4(2 * t, padded, a.x, a.y);
      out[1] = make_int4(c.x, c.y, 0, 0);
    }
  }
}

}  // namespace fa

namespace {

bool mod_sizes(int B, int H, int Hkv, int T, int d) {
  if (B <= 0 || H <= 0 || Hkv <= 0 || T <= 0 || H % Hkv != 0 || (d != 64 && d != 128)) return false;
  const long long BH = static_cast<long long>(B) * H, n_t = (static_cast<long long>(T) + 127) / 128;
  // (the kernels keep tile · 128 in an int, and the unit lists count with one)
  return BH <= INT32_MAX && n_t * 128 <= INT32_MAX && BH * n_t <= INT32_MAX &&
         static_cast<long long>(T) * d * 2 < (1LL << 40) && BH * T * d < (1LL << 61);
}

// Parts that a key head's query heads are cut into in the backward (a divisor of them): the fewest
// that give at least kMinCtas CTAs, three for each of a GB300's SMs, so that their unequal walks can
// be shared out (H16 Hkv4 T8192 d128 capped, five documents: 559 µs with the 256 CTAs of whole
// groups, 475 in two parts, 519 in four; B2 T4096 causal, whose walks are even: 403, 411 and
// 455). Independent of the device, so that a workspace fits wherever it is made.
int bwd_parts(int B, int H, int Hkv, int T) {
  constexpr long long kMinCtas = 456;
  const int group = H / Hkv;
  const long long ctas = static_cast<long long>(B) * Hkv * ((static_cast<long long>(T) + 127) / 128);
  int parts = 1;
  while (parts < group && (group % parts != 0 || ctas * parts < kMinCtas)) ++parts;
  return parts;
}

// CTAs of the backward up to which all heads' units go out together (fa_bwd_mod). In L2-sized groups ->
// together, µs, five and two documents and causal: 512 CTAs (H16 Hkv4 T8192 d128) 361 -> 297, 608 -> 458, 651
// -> 649; 1280 (H20 T8192 d128) 394 -> 363, 632 -> 548, 792 -> 786, (H10 T16384 d64, cap 30) 401 -> 369, 737
// -> 665, 1077 -> 1064; 1408 (H22) 402 -> 406, 640 -> 606, 875 -> 864, (H11) 404 -> 405, 743 -> 731, 1188 -> 1167;
// 1536 (B2 H12) 433 -> 448, 656 -> 659, 944 -> 940; 2048 (B2 H16) 569 -> 613, 866 -> 881, 1250 -> 1252.
constexpr long long kFewCtas = 1400;

bool any_misaligned(std::initializer_list<const void*> ps) {
  for (const void* x : ps)
    if (!aligned16(x)) return true;
  return false;
}

}  // namespace

extern "C" {

size_t fa_visible_size(int B, int T) {
  if (B <= 0 || T <= 0) return 0;
  const long long n_t = (static_cast<long long>(T) + 127) / 128;
  if (n_t * 128 > INT32_MAX || n_t * B > INT32_MAX) return 0;
  return fa::visible_layout(B, T).bytes;
}

int fa_visible(const int* doc_ids, const int* prefix_len, int prefix_per_token, int causal,
               void* visible, size_t visible_bytes, int B, int T, void* stream) {
  if (!visible) return FA_ERR_INVALID_ARG;
  const size_t need = fa_visible_size(B, T);
  if (need == 0 || visible_bytes < need) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(visible) & 255u) || (reinterpret_cast<uintptr_t>(doc_ids) & 3u) ||
      (reinterpret_cast<uintptr_t>(prefix_len) & 3u))
    return FA_ERR_MISALIGNED;
  const size_t bt = static_cast<size_t>(B) * T * 4;
  if ((doc_ids && overlaps(visible, need, doc_ids, bt)) ||
      (prefix_len && overlaps(visible, need, prefix_len, prefix_per_token ? bt : static_cast<size_t>(B) * 4)))
    return FA_ERR_INVALID_ARG;
  int dev = -1, sms = 0;
  const int st = check_device(&dev, &sms);
  if (st != FA_OK) return st;
  const fa::VisibleLayout l = fa::visible_layout(B, T);
  uint8_t* base = static_cast<uint8_t*>(visible);
  fa::VisibleParams p{};
  p.ids = doc_ids;
  p.prefix = prefix_len;
  p.prefix_per_token = prefix_per_token != 0;
  p.causal = causal != 0;
  p.T = T;
  p.n_t = static_cast<int>((static_cast<long long>(T) + 127) / 128);
  p.rows = reinterpret_cast<int2*>(base + l.rows);
  p.fwd = reinterpret_cast<int4*>(base + l.fwd);
  p.pairs = reinterpret_cast<int4*>(base + l.pairs);
  p.bwd = reinterpret_cast<int4*>(base + l.bwd);
  p.whole = reinterpret_cast<int2*>(base + l.whole);
  p.span = reinterpret_cast<int2*>(base + l.span);
  p.seen = reinterpret_cast<int2*>(base + l.seen);
  const cudaError_t e = fa::launch_pdl(fa::fa_visible_kernel, static_cast<unsigned>(B), fa::kVisThreads, 0,
                                       static_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

int fa_fwd_mod(const void* q, const void* k, const void* v, void* o, float* lse, void* rest,
               const void* visible, int causal, float softcap, const float* slopes, int B, int H, int Hkv, int T, int d,
               float scale, int* status, unsigned long long timeout_ns, void* stream) {
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  fa::CapFactors cap;
  if (!mod_sizes(B, H, Hkv, T, d) || !scale_ok(scale) || !cap_factors(scale, softcap, &cap))
    return FA_ERR_INVALID_ARG;
  if (any_misaligned({q, k, v, o, lse, rest}) || (reinterpret_cast<uintptr_t>(visible) & 255u) ||
      (reinterpret_cast<uintptr_t>(slopes) & 3u))
    return FA_ERR_MISALIGNED;
  const int BH = B * H;
  const size_t qb = static_cast<size_t>(BH) * T * d * 2, kb = static_cast<size_t>(B) * Hkv * T * d * 2;
  const size_t lb = static_cast<size_t>(BH) * T * 4;
  const void* ins[5] = {q, k, v, visible, slopes};
  const size_t in_bytes[5] = {qb, kb, kb, fa_visible_size(B, T), static_cast<size_t>(H) * 4};
  for (int i = 0; i < 5; ++i)
    if (ins[i] && (overlaps(o, qb, ins[i], in_bytes[i]) || overlaps(lse, lb, ins[i], in_bytes[i]) ||
                   (rest && overlaps(rest, qb, ins[i], in_bytes[i]))))
      return FA_ERR_INVALID_ARG;
  if (overlaps(o, qb, lse, lb) || (rest && (overlaps(rest, qb, o, qb) || overlaps(rest, qb, lse, lb))))
    return FA_ERR_INVALID_ARG;
  int dev = -1, sms = 0;
  const int st = check_device(&dev, &sms);
  if (st != FA_OK) return st;
  EncodeTiledFn enc = encode_fn();
  if (!enc) return FA_ERR_LAUNCH;
  fa::FwdLaunch a;
  a.p = fa::FwdParams{};
  if (!encode_map(enc, &a.tm_q, q, T, d, BH) || !encode_map(enc, &a.tm_k, k, T, d, B * Hkv) ||
      !encode_map(enc, &a.tm_v, v, T, d, B * Hkv) || !encode_map(enc, &a.tm_o, o, T, d, BH, 32))
    return FA_ERR_INVALID_ARG;
  const int n_t = (T + 127) / 128;
  a.p.o = static_cast<__nv_bfloat16*>(o);
  a.p.lse = lse;
  a.p.status = status;
  a.p.T = T;
  a.p.BH = BH;
  const int mod = fwd_mod_bits(softcap, slopes, rest);
  if ((mod & fa::kModRef) && scale < 0.0f) {  // (the largest weight is that of the largest raw score)
    a.p.s_negate = fa::kIdescNegateA;
    cap_factors(-scale, softcap, &cap);
  }
  // Two query tiles a CTA, as in the dense forward, where every SM gets 1.5 such units (one tile ->
  // two tiles in µs; d64 H12, d128 H16 Hkv4; causal, eight documents, a prefix of a third):
  //   plain   d64 B3 T2048 (1.9 units an SM) 34 -> 30, 14.7 -> 12.9, 37 -> 34; d128 B1 T4096 (1.7) 76 -> 55,
  //           22 -> 20, 89 -> 65; below, d64 B2 T2048 (1.3) 26 -> 25, 11.3 -> 12.8, 29 -> 25, B1 T4096 (1.3) 42
  //           -> 44, 13.4 -> 12.8, 47 -> 44, d128 T2048 (0.8) 24 -> 31, 11.6 -> 10.0, 29 -> 30
  //   capped  d64 B3 T2048 46 -> 40, 17.5 -> 15.4, 50 -> 47; d128 B1 T4096 86 -> 73, 25 -> 23, 100 -> 85, T8192
  //           (3.4) with o's rest 328 -> 282, 78 -> 64, 367 -> 334; below, d64 B1 T4096 56 -> 61, 16.5 ->
  //           15.3, 63 -> 62, d128 T2048 27 -> 40, 12.9 -> 11.3, 33 -> 40
  // Not with a bias (d64 T4096 204 -> 204, d128 T8192 328 -> 448) or a cap above 60, whose in-place
  // scores do not fit its registers.
  const bool plain = (mod & ~fa::kModRest) == fa::kModOn;
  const bool pairs = static_cast<long long>((n_t + 1) / 2) * BH * 2 >= 3ll * sms && (plain || (mod & fa::kModRef));
  a.p.n_units = pairs ? (n_t + 1) / 2 : n_t;
  a.p.total_units = a.p.n_units * BH;
  a.p.n_kv = n_t;
  a.p.tiles_per_cta = pairs ? 2 : 1;
  a.p.div_bh = fa::FastDiv::make(static_cast<uint32_t>(BH));
  a.p.div_splits = fa::FastDiv::make(1u);
  // Unmodified scores take their maximum before the factor, as the dense kernels; others the
  // plain factor.
  a.p.scale_log2 = plain ? exponent_factor(static_cast<double>(scale) * kLog2e, &a.p.s_negate)
                                     : static_cast<float>(static_cast<double>(scale) * kLog2e);
  a.p.timeout_ns = timeout_ns ? timeout_ns : 2000000000ull;
  a.p.Tk = T;
  a.p.n_qt = n_t;
  a.p.n_splits = 1;
  a.p.kt_per_split = n_t;
  a.p.bmask_heads = 1;
  if (visible) {
    const fa::VisibleLayout l = fa::visible_layout(B, T);
    const uint8_t* base = static_cast<const uint8_t*>(visible);
    a.p.mod.rows = reinterpret_cast<const int2*>(base + l.rows);
    a.p.mod.units = reinterpret_cast<const int4*>(base + l.fwd);
    a.p.mod.pairs = reinterpret_cast<const int4*>(base + l.pairs);
  }
  a.p.mod.slopes = slopes;
  a.p.mod.rest = static_cast<__nv_bfloat16*>(rest);
  a.p.mod.T_pad = n_t * 128;
  a.p.mod.H = H;
  a.p.mod.div_h = fa::FastDiv::make(static_cast<uint32_t>(H));
  a.p.mod.div_g = fa::FastDiv::make(static_cast<uint32_t>(H / Hkv));
  a.p.mod.cap = cap;
  a.p.mod.causal = causal != 0;
  a.grid = static_cast<unsigned>(std::min(a.p.total_units, sms));
  a.stream = static_cast<cudaStream_t>(stream);
  // Steps of the other forms, far or masked, are common where the cap is small (the scores of unit
  // normal rows have deviation 1) or walks are short: the step that stands them better
  // (fa_fwd_kernel.cuh; H12 d64, µs: eight documents, cap 30, B4 T2048 48 -> 43; causal, B3 T2048 45 -> 40,
  // B4 T4096 174 -> 170, B2 T6144 182 -> 182, T8192 165 -> 173; no mask, B3 T2048 58 -> 63).
  const bool short_walks = visible || (causal && T <= 4096);
  const int tight = d == 64 && mod == (fa::kModOn | fa::kModCap | fa::kModRef) && (short_walks || softcap < 25.0f)
                        ? fa::kModTight : 0;
  const cudaError_t e = pairs ? (d == 64 ? fa::launch_fwd_mod_pairs_d64(a, mod | tight) : fa::launch_fwd_mod_pairs_d128(a, mod))
                              : (d == 64 ? fa::launch_fwd_mod_d64(a, mod) : fa::launch_fwd_mod_d128(a, mod));
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

size_t fa_bwd_mod_workspace_size(int B, int H, int Hkv, int T, int d) {
  if (!mod_sizes(B, H, Hkv, T, d)) return 0;
  const size_t base = fa_bwd_workspace_size(B, H, T, d);  // a multiple of 256
  const int parts = bwd_parts(B, H, Hkv, T);
  if (base == 0 || parts == 1) return base;
  return base + static_cast<size_t>(2) * parts * B * Hkv * T * d * 4;
}

int fa_bwd_mod(const void* q, const void* k, const void* v, const void* o, const void* dout,
               const float* lse, const void* rest, void* dq, void* dk, void* dv, void* workspace,
               size_t workspace_bytes, const void* visible, int causal, float softcap, const float* slopes, int B, int H,
               int Hkv, int T, int d, float scale, int* status, unsigned long long timeout_ns,
               void* stream) {
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace)
    return FA_ERR_INVALID_ARG;
  fa::CapFactors cap;
  if (!mod_sizes(B, H, Hkv, T, d) || !scale_ok(scale) || !cap_factors(scale, softcap, &cap))
    return FA_ERR_INVALID_ARG;
  const size_t need = fa_bwd_mod_workspace_size(B, H, Hkv, T, d);
  if (need == 0 || workspace_bytes < need) return FA_ERR_INVALID_ARG;
  if (any_misaligned({q, k, v, o, dout, lse, rest, dq, dk, dv}) || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      (reinterpret_cast<uintptr_t>(visible) & 255u) || (reinterpret_cast<uintptr_t>(slopes) & 3u))
    return FA_ERR_MISALIGNED;
  const int BH = B * H, BHkv = B * Hkv;
  const size_t qb = static_cast<size_t>(BH) * T * d * 2, kb = static_cast<size_t>(BHkv) * T * d * 2;
  const void* ins[9] = {q, k, v, o, dout, lse, visible, slopes, rest};
  const size_t in_bytes[9] = {qb, kb, kb, qb, qb, static_cast<size_t>(BH) * T * 4, fa_visible_size(B, T),
                              static_cast<size_t>(H) * 4, qb};
  const void* outs[4] = {dq, dk, dv, workspace};
  const size_t out_bytes[4] = {qb, kb, kb, need};
  for (int x = 0; x < 4; ++x) {
    for (int y = 0; y < 9; ++y)
      if (ins[y] && overlaps(outs[x], out_bytes[x], ins[y], in_bytes[y])) return FA_ERR_INVALID_ARG;
    for (int y = x + 1; y < 4; ++y)
      if (overlaps(outs[x], out_bytes[x], outs[y], out_bytes[y])) return FA_ERR_INVALID_ARG;
  }
  int dev = -1, sms = 0;
  const int st = check_device(&dev, &sms);
  if (st != FA_OK) return st;
  EncodeTiledFn enc = encode_fn();
  if (!enc) return FA_ERR_LAUNCH;
  const int bq = (d == 64) ? 128 : 64;
  fa::BwdLaunch a;
  if (!encode_map(enc, &a.tm_q, q, T, d, BH, bq) || !encode_map(enc, &a.tm_k, k, T, d, BHkv) ||
      !encode_map(enc, &a.tm_v, v, T, d, BHkv) || !encode_map(enc, &a.tm_do, dout, T, d, BH, bq))
    return FA_ERR_INVALID_ARG;
  const int n_t = (T + 127) / 128, T_pad = n_t * 128;
  auto up = [](size_t x) { return (x + 255u) / 256u * 256u; };
  const size_t rows = static_cast<size_t>(BH) * T_pad;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.p = fa::BwdParams{};
  a.lse2 = reinterpret_cast<float*>(ws);
  a.dvec = reinterpret_cast<float*>(ws + up(rows * 4));
  a.p.dq_acc = reinterpret_cast<float*>(ws + 2 * up(rows * 4));
  a.p.lse2 = a.lse2;
  a.p.dvec = a.dvec;
  a.p.dk = static_cast<__nv_bfloat16*>(dk);
  a.p.dv = static_cast<__nv_bfloat16*>(dv);
  a.p.status = status;
  a.p.T = T;
  a.p.T_pad = T_pad;
  const int parts = bwd_parts(B, H, Hkv, T);
  a.p.BH = BHkv * parts;
  a.p.n_qt = T_pad / bq;
  a.p.n_kt = n_t;
  // Heads whose units go out together, the longest walks first: with few CTAs all of them, since
  // a long walk that starts late is the call's tail; otherwise as many as keep their Q and dO (bf16)
  // and dQ accumulator (fp32) in half the L2, 64 MB.
  const long long per_head = 8LL * T_pad * d * (H / Hkv / parts);
  const long long in_l2 = std::max<long long>(1, (64LL << 20) / per_head);
  const bool few = static_cast<long long>(n_t) * a.p.BH <= kFewCtas;
  a.p.head_group = static_cast<int>(std::min<long long>(a.p.BH, few ? a.p.BH : in_l2));
  a.p.scale = scale;
  a.p.scale_log2 = static_cast<float>(static_cast<double>(scale) * kLog2e);
  a.p.timeout_ns = timeout_ns ? timeout_ns : 2000000000ull;
  if (visible) {
    const fa::VisibleLayout l = fa::visible_layout(B, T);
    const uint8_t* base = static_cast<const uint8_t*>(visible);
    a.p.mod.rows = reinterpret_cast<const int2*>(base + l.rows);
    a.p.mod.units = reinterpret_cast<const int4*>(base + l.bwd);
    a.p.mod.whole = reinterpret_cast<const int2*>(base + l.whole);
  }
  a.p.mod.slopes = slopes;
  a.p.mod.Hkv = Hkv;
  a.p.mod.group = H / Hkv;
  a.p.mod.parts = parts;
  a.p.mod.part_out = reinterpret_cast<float*>(ws + fa_bwd_workspace_size(B, H, T, d));
  a.p.mod.cap = cap;
  a.p.mod.causal = causal != 0;
  a.o = static_cast<const __nv_bfloat16*>(o);
  a.dout = static_cast<const __nv_bfloat16*>(dout);
  a.rest = static_cast<const __nv_bfloat16*>(rest);
  a.lse = lse;
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.grid_main = static_cast<unsigned>(static_cast<long long>(n_t) * a.p.BH);
  a.grid_prep = static_cast<unsigned>(sms) * 8u;
  a.grid_dq = static_cast<unsigned>(sms) * 8u;
  a.stream = static_cast<cudaStream_t>(stream);
  const int mod = mod_bits(softcap, slopes);
  const cudaError_t e = (d == 64) ? fa::launch_bwd_mod_d64(a, mod, BH) : fa::launch_bwd_mod_d128(a, mod, BH);
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
