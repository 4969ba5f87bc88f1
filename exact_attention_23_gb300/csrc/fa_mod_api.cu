// Host side of attention with modified scores (include/fa.h: fa_visible, fa_fwd_mod, fa_bwd_mod, and
// their forms with a window) and the kernel that makes a batch's visibility.
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

// What fa_visible_window adds behind it where there are sinks:
//   sink_rows   int2 [B][T_pad]   the sinks that a row sees beside its window, an interval before lo
//   sink_units  int2 [B][n_t]     their K tiles for each of fwd, all before its first
//   sink_pairs  int4 [B][n_p]     the same for both tiles of each of pairs
//   pieces      int4 [B][n_rec][2]  takes the place of bwd: a key tile with sinks is seen by query tiles up
//                 to its document's end, and such a walk is cut into pieces of at most `piece` query
//                 tiles, most first: (tile, first query tile, past the last, as in bwd), (the slot of a cut
//                 tile's piece or −1, whether the tile has sinks beyond a window, 0, 0); tile n_t: no piece
//   cuts        int4 [B][n_cut]   the cut key tiles: (tile, first slot, slots, 0); no slots: none
//   far, near   per tile, where a sequence has more than kVisTiles
struct WindowLayout {
  VisibleLayout base;
  size_t sink_rows, sink_units, sink_pairs, pieces, cuts, far, near, bytes;
  int piece, n_rec, n_cut, n_slots;
};

constexpr int kMaxSinks = 1024;
constexpr int kVisThreads = 1024;
constexpr int kVisTiles = 1024;  // whose extremes a CTA keeps in shared memory
constexpr int kVisFew = 32;

static WindowLayout window_layout(int B, int T, int window, int sinks) {
  auto up = [](size_t x) { return (x + 255u) / 256u * 256u; };
  WindowLayout l{};
  l.base = visible_layout(B, T);
  l.bytes = l.base.bytes;
  const size_t b = static_cast<size_t>(B);
  const long long n_t = (static_cast<long long>(T) + 127) / 128;
  l.n_rec = static_cast<int>(n_t);
  if (sinks == 0) return l;
  // A key tile without sinks is seen by at most (window + 126) / 128 + 1 query tiles: it is never cut.
  l.piece = static_cast<int>(std::max<long long>(8, std::min<long long>(window, T) / 128 + 2));
  // Pieces beyond one a tile. A walk of n > piece ≥ 8 query tiles leaves at most (n − 1) / piece of them, and
  // it is that of a document of 128·(n − 2) tokens and more, so n − 1 ≤ 8/7 of its length in tiles (n ≥ 9);
  // at most (sinks + 126) / 128 + 1 tiles hold a document's sinks, and documents do not overlap.
  const long long holds = (sinks + 126) / 128 + 1;
  const long long extra = n_t <= l.piece ? 0 : (n_t * holds * 8 + 7 * l.piece - 1) / (7 * l.piece);
  l.n_rec = static_cast<int>(n_t + extra);
  l.n_cut = static_cast<int>(std::min(extra, n_t));
  l.n_slots = static_cast<int>(extra + l.n_cut);
  l.sink_rows = l.bytes;
  l.sink_units = l.sink_rows + up(b * n_t * 128 * 8);
  l.sink_pairs = l.sink_units + up(b * n_t * 8);
  l.pieces = l.sink_pairs + up(b * ((n_t + 1) / 2) * 16);
  l.cuts = l.pieces + up(b * l.n_rec * 32);
  l.far = l.cuts + up(b * l.n_cut * 16);
  const size_t apart = n_t > kVisTiles ? b * n_t : 0;
  l.near = l.far + up(apart * 4);
  l.bytes = l.near + up(apart * 8);
  return l;
}

struct VisibleParams {
  const int* ids;     // [B][T] or null
  const int* prefix;  // [B] or [B][T] or null
  int prefix_per_token, causal, T, n_t;
  uint32_t by_seg;    // ⌈2³² / seg⌉, seg the rows a thread's stretch has: ⌊i / seg⌋ is the upper half of its product with i < 2¹⁵, seg > 1
  int2* rows;
  int4 *fwd, *pairs, *bwd;
  int2 *whole, *span, *seen;
  // a sliding window and sinks
  int window, sinks, piece, n_rec, n_cut;
  int2 *sink_rows, *sink_units, *near;
  int4 *sink_pairs, *pieces, *cuts;
  int* far;
};


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

// The same for a warp's stretches of seg ≤ 32 rows (`base`: its first row): ids side by side, 32 a load, as words
// of bits, of which each lane takes its stretch. (From stretches of more than 8 rows on: documents of 700 with a window and sinks,
// a thread reading its own rows -> side by side, T 32768 25.8 -> 14.2 µs, 16384 11.4 -> 9.6, 8192 7.6 -> 7.7, 4500 6.9 -> 7.8.)
__device__ __forceinline__ void warp_doc_bits(const int* ids, int base, int seg, int T, uint32_t* starts, uint32_t* pads) {
  const int lane = threadIdx.x & 31;
  uint32_t st = 0u, pad = 0u;  // lane k's: of rows base + 32k …
  int prev = base > 0 && base < T ? ids[base - 1] : 0;
#pragma unroll 1
  for (int k = 0; k < seg && base + 32 * k < T; k += 8) {
    int id[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) id[e] = ids[min(base + 32 * (k + e) + lane, T - 1)];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = base + 32 * (k + e) + lane;
      int before = __shfl_up_sync(0xffffffffu, id[e], 1);
      if (lane == 0) before = prev;
      prev = __shfl_sync(0xffffffffu, id[e], 31);
      const uint32_t s = __ballot_sync(0xffffffffu, i < T && (i == 0 || id[e] != before));
      const uint32_t p = __ballot_sync(0xffffffffu, i < T && id[e] < 0);
      if (lane == k + e && k + e < seg) {
        st = s;
        pad = p;
      }
    }
  }
  const int at = lane * seg, word = at >> 5, next = min(word + 1, 31);
  const uint32_t s0 = __shfl_sync(0xffffffffu, st, word), s1 = __shfl_sync(0xffffffffu, st, next);
  const uint32_t p0 = __shfl_sync(0xffffffffu, pad, word), p1 = __shfl_sync(0xffffffffu, pad, next);
  *starts = __funnelshift_r(s0, s1, at & 31) & bits_below(seg);
  *pads = __funnelshift_r(p0, p1, at & 31) & bits_below(seg);
}

// One block a sequence. A document is a maximal run of equal ids, so a row's document starts at
// the last change of id at or before it and ends at the next one after it: a running maximum and
// a running minimum, each thread taking one stretch of rows (as bits, 32 rows at a time) and the
// block joining the stretches. Then a warp a tile: its rows (from their stretch's bits, where a stretch
// has at most 32, so that rows are written side by side: T 16384
// 17.3 -> 12.0 µs on one CTA, with sinks 42.6 -> 16.1, half of that the lengths below being made once) and their extremes, the query tiles
// that see it, and its place among the tiles by the number it has to walk (a count of the tiles before
// it: n_t² comparisons, which at 16384 tokens are 4 a lane and tile). The
// tiles' extremes are kept in shared memory up to kVisTiles of them. WINDOW: rows see the last
// `window` keys at most; SINK: and the first `sinks` of their document (fa_visible_window).
// Long sequences of a small batch go to a cluster of CTAs a sequence, each with every `ctas`-th tile: all find the
// documents, and tell one another of their tiles through shared memory.
// FEW: at most 32 tiles on one CTA, a warp each, without what more tiles and clusters need. (One instantiation for all ->
// this, causal, documents of 700, and with a window and sinks: B4 T1024 4.2 -> 3.6 µs, 4.8 -> 4.3, 5.4 -> 4.8; B1 T4096 5.0
// -> 4.3, 5.9 -> 5.3, 7.5 -> 6.9; and with the forward behind it B4 H16 Hkv4 T62 d128 11.2 -> 9.9.)
template <bool WINDOW, bool SINK, bool FEW>
__global__ void __launch_bounds__(kVisThreads) fa_visible_kernel(const VisibleParams p) {
  constexpr int kTiles = FEW ? kVisFew : kVisTiles;
  __shared__ int s_last[kVisThreads / 32], s_first[kVisThreads / 32];
  __shared__ int s_pad;
  __shared__ int2 s_span[kTiles], s_seen[kTiles];
  __shared__ int s_far[SINK ? kTiles : 1];   // past the last query tile that sees a key tile's sinks, 0: none beyond a window
  __shared__ int2 s_near[SINK ? kTiles : 1]; // a query tile's K tiles with sinks, before its first
  // A stretch's document starts and paddings as bits, the document it starts in and the next one's start; then
  // a tile's steps in the forward, those of a piece of its walk in the backward and the pieces, and a pair's steps.
  static_assert(kVisThreads == kVisTiles, "one array for both");
  __shared__ int4 s_four[kVisThreads];
  pdl_wait();
  pdl_launch_dependents();
  const int ctas = FEW ? 1 : static_cast<int>(cluster_ctas()), rank = FEW ? 0 : static_cast<int>(cluster_ctarank());
  const int b = static_cast<int>(FEW ? blockIdx.x : cluster_id()), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int step = ctas * (kVisThreads / 32), tile0 = rank + ctas * warp;  // a warp's tiles
  const int T = p.T, n_t = p.n_t;
  const long long T_pad = static_cast<long long>(n_t) * 128;
  const int* ids = p.ids ? p.ids + static_cast<size_t>(b) * T : nullptr;
  int2* rows = p.rows + static_cast<size_t>(b) * T_pad;
  int2* span = FEW || n_t <= kVisTiles ? s_span : p.span + static_cast<size_t>(b) * n_t;
  int2* seen = FEW || n_t <= kVisTiles ? s_seen : p.seen + static_cast<size_t>(b) * n_t;
  int* far = nullptr;
  int2 *near = nullptr, *sink_rows = nullptr;
  if constexpr (SINK) {
    far = FEW || n_t <= kVisTiles ? s_far : p.far + static_cast<size_t>(b) * n_t;
    near = FEW || n_t <= kVisTiles ? s_near : p.near + static_cast<size_t>(b) * n_t;
    sink_rows = p.sink_rows + static_cast<size_t>(b) * T_pad;
    for (int t = rank + ctas * tid; t < n_t; t += ctas * kVisThreads) far[t] = 0;
  }
  if (tid == 0) s_pad = n_t;
  if (ctas > 1) {  // (no word from another CTA before its places are ready)
    __syncwarp();
    cluster_arrive_all();
  }
  auto sync_all = [&]() {
    if (ctas > 1) {
      __syncwarp();
      cluster_sync_all();
    } else {
      __syncthreads();
    }
  };
  const long long seg = (T_pad + kVisThreads - 1) / kVisThreads;
  const int a0 = static_cast<int>(min(static_cast<long long>(T), tid * seg));
  const int a1 = static_cast<int>(min(static_cast<long long>(T), (tid + 1) * seg));
  uint32_t starts = 0u, pads = 0u;
  int last = -1, first = T;  // this stretch's last and first document starts
  const bool one = FEW || seg <= 32;  // a stretch is one group of bits
  const bool side_by_side = !FEW && one && seg > 8 && ids;
  if (side_by_side) warp_doc_bits(ids, static_cast<int>(min(static_cast<long long>(T), warp * 32 * seg)), static_cast<int>(seg), T, &starts, &pads);
  for (int g0 = a0; g0 < a1; g0 += 32) {
    if (!side_by_side) doc_bits(ids, g0, a1, &starts, &pads);
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
  const int* pre_at = nullptr;
  int pre_all = 0;
  if (p.prefix && p.causal) {
    if (p.prefix_per_token) pre_at = p.prefix + static_cast<size_t>(b) * T;
    else pre_all = max(0, p.prefix[b]);
  }
  // Row i's keys, its document being [lo, end); SINK: and its sinks, and who sees it as one.
  auto row_of = [&](int i, int lo, int end, bool pad, int2* sink) {
    *sink = make_int2(0, 0);
    if (pad) return make_int2(0, 0);
    int2 r = make_int2(lo, end);
    if constexpr (WINDOW) {
      r = make_int2(max(lo, i + 1 - p.window), i + 1);
      if constexpr (SINK) {
        if (lo < r.x) *sink = make_int2(lo, min(lo + p.sinks, r.x));
        if (i - lo < p.sinks && end - i > p.window) atomicMax(far + (i >> 7), (end + 127) >> 7);  // seen from beyond the window
      }
    } else if (p.causal) {
      const int pre = pre_at ? max(0, pre_at[i]) : pre_all;
      r.y = max(i + 1, pre > end - lo ? end : lo + pre);
    }
    return r;
  };
  if (one) {
    s_four[tid] = make_int4(static_cast<int>(starts), static_cast<int>(pads), cur, end);
  } else {
    // The rows' document starts, front to back, then the rows from the back.
    int c = cur;
    for (int g0 = a0; g0 < a1; g0 += 32) {
      doc_bits(ids, g0, a1, &starts, &pads);
      for (int o = 0; o < min(32, a1 - g0); ++o) {
        if ((starts >> o) & 1u) c = g0 + o;
        rows[g0 + o].x = c;
      }
    }
    int padded = n_t;
    for (int g0 = a0 + max(0, (a1 - a0 - 1)) / 32 * 32; g0 >= a0 && a1 > a0; g0 -= 32) {
      doc_bits(ids, g0, a1, &starts, &pads);
      for (int o = min(32, a1 - g0) - 1; o >= 0; --o) {
        const int i = g0 + o, lo = rows[i].x;
        const bool pad = (pads >> o) & 1u;
        if (pad) padded = i >> 7;  // (from the back)
        int2 sink;
        rows[i] = row_of(i, lo, end, pad, &sink);
        if constexpr (SINK) sink_rows[i] = sink;
        if (lo == i) end = i;
      }
    }
    padded = __reduce_min_sync(0xffffffffu, padded);
    if (lane == 0) atomicMin(&s_pad, padded);
  }
  for (long long i = T + tid; i < T_pad; i += kVisThreads) {
    rows[i] = make_int2(0, 0);
    if constexpr (SINK) sink_rows[i] = make_int2(0, 0);
  }
  __syncthreads();
  if (ctas > 1) cluster_wait_all();
  const size_t t0 = static_cast<size_t>(b) * n_t;
  for (int t = tile0; t < n_t; t += step) {
    int lo_min = T, hi_max = 0, lo_max = 0, hi_min = T;
    int2 sinks[4];
    bool pads_here = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = t * 128 + lane + 32 * k;
      sinks[k] = make_int2(0, 0);
      if (i >= T) continue;
      int2 r;
      if (one) {
        const int s = seg == 1 ? i : static_cast<int>(__umulhi(p.by_seg, static_cast<uint32_t>(i)));
        const int4 f = s_four[s];
        const int o = i - s * static_cast<int>(seg);
        const uint32_t st = static_cast<uint32_t>(f.x), at = st & ((2u << o) - 1u), after = st & ~((2u << o) - 1u);
        const bool pad = (static_cast<uint32_t>(f.y) >> o) & 1u;
        pads_here |= pad;
        r = row_of(i, at ? i - o + 31 - __clz(at) : f.z, after ? i - o + __ffs(after) - 1 : f.w, pad, &sinks[k]);
        rows[i] = r;
        if constexpr (SINK) sink_rows[i] = sinks[k];
      } else {
        r = rows[i];
        if constexpr (SINK) sinks[k] = sink_rows[i];
      }
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
    if (__any_sync(0xffffffffu, pads_here) && lane < ctas) red_min_cluster(mapa_shared(&s_pad, lane), t);
    const int2 sp = hi_max > lo_min ? make_int2(lo_min, hi_max) : make_int2(0, 0);
    if (lane == 0) {
      p.whole[t0 + t] = make_int2(lo_max, hi_min);
      span[t] = sp;
    }
    if (lane < ctas && lane != rank) st_cluster2(mapa_shared(s_span + t, lane), sp);
    if constexpr (SINK) {
      // The tiles with sinks before the walk's first. (Documents that start within it have theirs in the walk.)
      const int kb = lo_min >> 7;
      int first_sink = T, past = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int2 s = sinks[k];
        if (s.y > s.x && s.x >> 7 < kb) {
          first_sink = min(first_sink, s.x);
          past = max(past, s.y);
        }
      }
      first_sink = __reduce_min_sync(0xffffffffu, first_sink);
      past = __reduce_max_sync(0xffffffffu, past);
      const int2 nr = past > 0 ? make_int2(first_sink >> 7, min((past + 127) >> 7, kb)) : make_int2(0, 0);
      if (lane == 0) near[t] = nr;
      __syncwarp();
      if (lane < ctas && lane != rank) {
        st_cluster2(mapa_shared(s_near + t, lane), nr);
        st_cluster1(mapa_shared(s_far + t, lane), far[t]);
      }
    }
  }
  sync_all();
  const int padded = s_pad;
  for (int t = tile0; t < n_t; t += step) {
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
    if constexpr (SINK) {
      if (far[t] > 0) {
        f = min(f, t);
        l = max(l, far[t]);
      }
    }
    if (lane == 0) seen[t] = l > f ? make_int2(f, l) : make_int2(0, 0);
  }
  __syncthreads();
  // What tiles are sorted by: a query tile's steps, a key tile's (SINK: its pieces, and the length of the
  // longest), and a pair's, the length of its union's walk.
  const int n_p = (n_t + 1) / 2;
  auto walk = [&](int t) {  // first K tile and past the last; (0, 0): none
    const int2 s = t < n_t ? span[t] : make_int2(0, 0);
    return make_int2(s.x >> 7, (s.y + 127) >> 7);
  };
  auto lengths_of = [&](int t) {
    const int2 s = walk(t);
    int4 x = make_int4(s.y - s.x, seen[t].y - seen[t].x, 1, 0);
    if constexpr (SINK) {
      x.x += near[t].y - near[t].x;
      if (far[t] > 0 && x.y > p.piece) {
        x.z = (x.y + p.piece - 1) / p.piece;
        x.y = (x.y + x.z - 1) / x.z;
      }
    }
    if (t < n_p) {
      const int2 a = walk(2 * t), c = walk(2 * t + 1);
      x.w = a.y <= a.x ? c.y - c.x : c.y <= c.x ? a.y - a.x : max(a.y, c.y) - min(a.x, c.x);
    }
    return x;
  };
  const bool kept = !FEW && n_t > kVisFew && n_t <= kVisTiles;  // (few: made where they are looked at, one a lane)
  if (kept) {
    const int t = rank + ctas * tid;
    if (t < n_t) {
      const int4 x = lengths_of(t);
      s_four[t] = x;
      for (int c = 0; c < ctas; ++c)
        if (c != rank) st_cluster4(mapa_shared(s_four + t, c), x);
    }
    sync_all();
  }
  auto lengths = [&](int t) { return kept ? s_four[t] : lengths_of(t); };
  int n_pieces = 0, n_cuts = 0;
  for (int t = tile0; t < n_t; t += step) {
    const int2 s = span[t], k = seen[t];
    const int kb = s.x >> 7, ke = (s.y + 127) >> 7;
    const int4 me = lengths(t);
    if constexpr (SINK) {
      const int2 sk = near[t];
      const int pc = me.z, m = k.y - k.x, len = me.y;
      int rf = 0, rb = 0, slot = 0, cut = 0, all = 0, cuts = 0;
      for (int q = lane; q < n_t; q += 32) {
        const int4 o = lengths(q);
        rf += o.x > me.x || (o.x == me.x && q < t);
        if (o.y > len || (o.y == len && q < t)) rb += o.z;
        if (o.z > 1 && q < t) {
          slot += o.z;
          ++cut;
        }
        all += o.z;
        cuts += o.z > 1;
      }
      rf = __reduce_add_sync(0xffffffffu, rf);
      rb = __reduce_add_sync(0xffffffffu, rb);
      slot = __reduce_add_sync(0xffffffffu, slot);
      cut = __reduce_add_sync(0xffffffffu, cut);
      n_pieces = __reduce_add_sync(0xffffffffu, all);
      n_cuts = __reduce_add_sync(0xffffffffu, cuts);
      if (lane == 0) {
        p.fwd[t0 + rf] = make_int4(t, kb, ke, padded);
        p.sink_units[t0 + rf] = sk;
        if (pc > 1 && cut < p.n_cut) p.cuts[static_cast<size_t>(b) * p.n_cut + cut] = make_int4(t, slot, pc, 0);
      }
      // pieces of len or len − 1 query tiles
      const int longer = m - (len - 1) * pc;
      for (int i = lane; i < pc && rb + i < p.n_rec; i += 32) {
        const int q0 = k.x + i * (len - 1) + min(i, longer);
        int4* out = p.pieces + (static_cast<size_t>(b) * p.n_rec + rb + i) * 2;
        out[0] = make_int4(t, q0, q0 + len - (i < longer ? 0 : 1), 2 * padded + (p.whole[t0 + t].y == 0 ? 1 : 0));
        out[1] = make_int4(pc > 1 ? slot + i : -1, far[t] > 0, 0, 0);
      }
    } else {
      int rf = 0, rb = 0;
      for (int q = lane; q < n_t; q += 32) {
        const int4 o = lengths(q);
        rf += o.x > me.x || (o.x == me.x && q < t);
        rb += o.y > me.y || (o.y == me.y && q < t);
      }
      rf = __reduce_add_sync(0xffffffffu, rf);
      rb = __reduce_add_sync(0xffffffffu, rb);
      if (lane == 0) {
        p.fwd[t0 + rf] = make_int4(t, kb, ke, padded);
        p.bwd[t0 + rb] = make_int4(t, k.x, k.y, 2 * padded + (p.whole[t0 + t].y == 0 ? 1 : 0));
      }
    }
  }
  if constexpr (SINK) {
    if (tile0 == 0) {  // (it has had one)
      for (int i = n_pieces + lane; i < p.n_rec; i += 32) {
        int4* out = p.pieces + (static_cast<size_t>(b) * p.n_rec + i) * 2;
        out[0] = make_int4(n_t, 0, 0, 2 * n_t);
        out[1] = make_int4(-1, 0, 0, 0);
      }
      for (int i = n_cuts + lane; i < p.n_cut; i += 32) p.cuts[static_cast<size_t>(b) * p.n_cut + i] = make_int4(0, 0, 0, 0);
    }
  }
  for (int t = tile0; t < n_p; t += step) {
    const int2 a = walk(2 * t), c = walk(2 * t + 1);
    const int n = lengths(t).w;
    int r = 0;
    for (int q = lane; q < n_p; q += 32) {
      const int m = lengths(q).w;
      r += m > n || (m == n && q < t);
    }
    r = __reduce_add_sync(0xffffffffu, r);
    if (lane == 0) {
      int4* out = p.pairs + (static_cast<size_t>(b) * n_p + r) * 2;
      out[0] = make_int4(2 * t, padded, a.x, a.y);
      out[1] = make_int4(c.x, c.y, 0, 0);
      if constexpr (SINK) {
        const int2 k0 = near[2 * t], k1 = 2 * t + 1 < n_t ? near[2 * t + 1] : make_int2(0, 0);
        p.sink_pairs[static_cast<size_t>(b) * n_p + r] = make_int4(k0.x, k0.y, k1.x, k1.y);
      }
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

bool window_ok(int window, int sinks) { return window >= 1 && sinks >= 0 && sinks <= fa::kMaxSinks; }

size_t up256(size_t x) { return (x + 255u) / 256u * 256u; }

// fa_visible and fa_visible_window (window > 0), whose buffer has `need` bytes.
int make_visible(const int* doc_ids, const int* prefix_len, int prefix_per_token, int causal, int window, int sinks,
                 void* visible, size_t visible_bytes, size_t need, int B, int T, void* stream) {
  if (!visible) return FA_ERR_INVALID_ARG;
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
  const uint64_t seg = (static_cast<uint64_t>(p.n_t) * 128 + fa::kVisThreads - 1) / fa::kVisThreads;
  p.by_seg = static_cast<uint32_t>((0xFFFFFFFFull + seg) / seg);
  p.rows = reinterpret_cast<int2*>(base + l.rows);
  p.fwd = reinterpret_cast<int4*>(base + l.fwd);
  p.pairs = reinterpret_cast<int4*>(base + l.pairs);
  p.bwd = reinterpret_cast<int4*>(base + l.bwd);
  p.whole = reinterpret_cast<int2*>(base + l.whole);
  p.span = reinterpret_cast<int2*>(base + l.span);
  p.seen = reinterpret_cast<int2*>(base + l.seen);
  const bool few = p.n_t <= fa::kVisFew;
  auto* fn = few ? &fa::fa_visible_kernel<false, false, true> : &fa::fa_visible_kernel<false, false, false>;
  if (window > 0) {
    p.window = window;
    p.sinks = sinks;
    fn = few ? &fa::fa_visible_kernel<true, false, true> : &fa::fa_visible_kernel<true, false, false>;
    if (sinks > 0) {
      const fa::WindowLayout wl = fa::window_layout(B, T, window, sinks);
      p.piece = wl.piece;
      p.n_rec = wl.n_rec;
      p.n_cut = wl.n_cut;
      p.sink_rows = reinterpret_cast<int2*>(base + wl.sink_rows);
      p.sink_units = reinterpret_cast<int2*>(base + wl.sink_units);
      p.sink_pairs = reinterpret_cast<int4*>(base + wl.sink_pairs);
      p.pieces = reinterpret_cast<int4*>(base + wl.pieces);
      p.cuts = reinterpret_cast<int4*>(base + wl.cuts);
      p.far = reinterpret_cast<int*>(base + wl.far);
      p.near = reinterpret_cast<int2*>(base + wl.near);
      fn = few ? &fa::fa_visible_kernel<true, true, true> : &fa::fa_visible_kernel<true, true, false>;
    }
  }
  // A cluster a sequence from 4097 to 32768 tokens, of as many CTAs as leave every cluster a place (sms SMs: pairs
  // find them all, fours 144 of 152, eights 120; 16 eights 6.8 -> 13 µs). One CTA -> eight, µs: causal T8192 7.6 ->
  // 5.3, T16384 12.5 -> 5.6, T32768 24.7 -> 7.0; a window and sinks 10.0 -> 6.3, 17.1 -> 6.8, 34.9 -> 8.8; documents of
  // 700 (which all CTAs look for) 9.2 -> 6.9, 17.3 -> 10.3, now 8.5, 41.6 -> 24.1, now 12.5.
  unsigned ctas = 1;
  if (seg <= 32 && !few)
    for (const unsigned c : {2u, 4u, 8u})
      if (B <= sms * (c == 2 ? 16 : c == 4 ? 15 : 12) / 16 / static_cast<int>(c)) ctas = c;
  const cudaError_t e = fa::launch_pdl_clusters(fn, static_cast<unsigned>(B) * ctas, ctas, fa::kVisThreads, 0,
                                                static_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

// fa_fwd_mod and fa_fwd_window (window > 0), whose visibility has visible_bytes.
int fwd_mod(const void* q, const void* k, const void* v, void* o, float* lse, void* rest, const void* visible,
            size_t visible_bytes, int causal, int window, int sinks, float softcap, const float* slopes, int B, int H,
            int Hkv, int T, int d, float scale, int* status, unsigned long long timeout_ns, void* stream) {
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
  const size_t in_bytes[5] = {qb, kb, kb, visible_bytes, static_cast<size_t>(H) * 4};
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
  // Nor at d = 64 with a short window, whose walks are mostly edges (B1 H12 T16384, visibility and forward, one tile ->
  // two: window 256 49.5 -> 51.7, with four sinks 61.5 -> 65.3; 512 61.5 -> 61.5, 74.1 -> 77.8; 1024 89.8 -> 84.7, 102
  // -> 102; 4096 237 -> 211, 247 -> 233; d128 H16 Hkv4 T8192 with sinks 512 81.4 -> 76.9, 1024 105 -> 95.7).
  const bool pairs = static_cast<long long>((n_t + 1) / 2) * BH * 2 >= 3ll * sms && (plain || (mod & fa::kModRef)) &&
                     (window == 0 || d == 128 || window > 512);
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
    if (sinks > 0) {
      const fa::WindowLayout wl = fa::window_layout(B, T, window, sinks);
      a.p.mod.sink_rows = reinterpret_cast<const int2*>(base + wl.sink_rows);
      a.p.mod.sink_units = reinterpret_cast<const int2*>(base + wl.sink_units);
      a.p.mod.sink_pairs = reinterpret_cast<const int4*>(base + wl.sink_pairs);
    }
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
  // (a window without sinks: the two-tile kernel has its intervals; the one-tile kernel with sinks skips the
  // columns that none of a warp's rows sees, T16384 H12 d64 window 256 53.4 -> 49.5 µs)
  if (window > 0 && (sinks > 0 || !pairs)) {
    const cudaError_t e = pairs ? (d == 64 ? fa::launch_fwd_sink_pairs_d64(a, mod) : fa::launch_fwd_sink_pairs_d128(a, mod))
                                : (d == 64 ? fa::launch_fwd_sink_d64(a, mod) : fa::launch_fwd_sink_d128(a, mod));
    return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
  }
  const cudaError_t e = pairs ? (d == 64 ? fa::launch_fwd_mod_pairs_d64(a, mod | tight) : fa::launch_fwd_mod_pairs_d128(a, mod))
                              : (d == 64 ? fa::launch_fwd_mod_d64(a, mod) : fa::launch_fwd_mod_d128(a, mod));
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

// fa_bwd_mod and fa_bwd_window, with a workspace of `need` bytes.
int bwd_mod(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
            const void* rest, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, size_t need,
            const void* visible, size_t visible_bytes, int causal, int window, int sinks, float softcap, const float* slopes,
            int B, int H, int Hkv, int T, int d, float scale, int* status, unsigned long long timeout_ns, void* stream) {
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace)
    return FA_ERR_INVALID_ARG;
  fa::CapFactors cap;
  if (!mod_sizes(B, H, Hkv, T, d) || !scale_ok(scale) || !cap_factors(scale, softcap, &cap))
    return FA_ERR_INVALID_ARG;
  if (need == 0 || workspace_bytes < need) return FA_ERR_INVALID_ARG;
  if (any_misaligned({q, k, v, o, dout, lse, rest, dq, dk, dv}) || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      (reinterpret_cast<uintptr_t>(visible) & 255u) || (reinterpret_cast<uintptr_t>(slopes) & 3u))
    return FA_ERR_MISALIGNED;
  const int BH = B * H, BHkv = B * Hkv;
  const size_t qb = static_cast<size_t>(BH) * T * d * 2, kb = static_cast<size_t>(BHkv) * T * d * 2;
  const void* ins[9] = {q, k, v, o, dout, lse, visible, slopes, rest};
  const size_t in_bytes[9] = {qb, kb, kb, qb, qb, static_cast<size_t>(BH) * T * 4, visible_bytes,
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
  int n_rec = n_t;  // walks a key head's part
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
    if (sinks > 0) {
      const fa::WindowLayout wl = fa::window_layout(B, T, window, sinks);
      a.p.mod.units = reinterpret_cast<const int4*>(base + wl.pieces);
      a.p.mod.sink_rows = reinterpret_cast<const int2*>(base + wl.sink_rows);
      a.p.mod.cuts = reinterpret_cast<const int4*>(base + wl.cuts);
      a.p.mod.piece_out = reinterpret_cast<float*>(ws + up256(fa_bwd_mod_workspace_size(B, H, Hkv, T, d)));
      a.p.mod.n_cut = wl.n_cut;
      a.p.mod.n_slots = wl.n_slots;
      n_rec = wl.n_rec;
    }
  }
  a.p.mod.n_rec = n_rec;
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
  a.grid_main = static_cast<unsigned>(static_cast<long long>(n_rec) * a.p.BH);
  a.grid_prep = static_cast<unsigned>(sms) * 8u;
  a.grid_dq = static_cast<unsigned>(sms) * 8u;
  a.stream = static_cast<cudaStream_t>(stream);
  const int mod = mod_bits(softcap, slopes);
  const cudaError_t e = sinks > 0 ? (d == 64 ? fa::launch_bwd_sink_d64(a, mod, BH) : fa::launch_bwd_sink_d128(a, mod, BH))
                                  : (d == 64) ? fa::launch_bwd_mod_d64(a, mod, BH) : fa::launch_bwd_mod_d128(a, mod, BH);
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
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
  return make_visible(doc_ids, prefix_len, prefix_per_token, causal, 0, 0, visible, visible_bytes,
                      fa_visible_size(B, T), B, T, stream);
}

size_t fa_visible_window_size(int B, int T, int window, int sinks) {
  if (fa_visible_size(B, T) == 0 || !window_ok(window, sinks)) return 0;
  const fa::WindowLayout l = fa::window_layout(B, T, window, sinks);
  return static_cast<long long>(l.n_rec) * B > INT32_MAX ? 0 : l.bytes;
}

int fa_visible_window(const int* doc_ids, int window, int sinks, void* visible, size_t visible_bytes, int B,
                      int T, void* stream) {
  return make_visible(doc_ids, nullptr, 0, 1, window, sinks, visible, visible_bytes,
                      fa_visible_window_size(B, T, window, sinks), B, T, stream);
}

int fa_fwd_mod(const void* q, const void* k, const void* v, void* o, float* lse, void* rest,
               const void* visible, int causal, float softcap, const float* slopes, int B, int H, int Hkv, int T, int d,
               float scale, int* status, unsigned long long timeout_ns, void* stream) {
  return fwd_mod(q, k, v, o, lse, rest, visible, fa_visible_size(B, T), causal, 0, 0, softcap, slopes, B, H, Hkv, T, d,
                 scale, status, timeout_ns, stream);
}

int fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, void* rest,
                  const void* visible, int window, int sinks, float softcap, const float* slopes, int B, int H, int Hkv,
                  int T, int d, float scale, int* status, unsigned long long timeout_ns, void* stream) {
  const size_t vb = fa_visible_window_size(B, T, window, sinks);
  if (!visible || vb == 0) return FA_ERR_INVALID_ARG;
  return fwd_mod(q, k, v, o, lse, rest, visible, vb, 1, window, sinks, softcap, slopes, B, H, Hkv, T, d, scale, status,
                 timeout_ns, stream);
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
  return bwd_mod(q, k, v, o, dout, lse, rest, dq, dk, dv, workspace, workspace_bytes,
                 fa_bwd_mod_workspace_size(B, H, Hkv, T, d), visible, fa_visible_size(B, T), causal, 0, 0, softcap, slopes,
                 B, H, Hkv, T, d, scale, status, timeout_ns, stream);
}

size_t fa_bwd_window_workspace_size(int B, int H, int Hkv, int T, int d, int window, int sinks) {
  const size_t base = fa_bwd_mod_workspace_size(B, H, Hkv, T, d);
  if (base == 0 || fa_visible_window_size(B, T, window, sinks) == 0) return 0;
  if (sinks == 0) return base;
  const fa::WindowLayout l = fa::window_layout(B, T, window, sinks);
  if (static_cast<long long>(l.n_rec) * B * Hkv * bwd_parts(B, H, Hkv, T) > INT32_MAX) return 0;
  return up256(base) + static_cast<size_t>(2) * bwd_parts(B, H, Hkv, T) * B * Hkv * l.n_slots * 128 * d * 4;
}

int fa_bwd_window(const void* q, const void* k, const void* v, const void* o, const void* dout,
                  const float* lse, const void* rest, void* dq, void* dk, void* dv, void* workspace,
                  size_t workspace_bytes, const void* visible, int window, int sinks, float softcap, const float* slopes,
                  int B, int H, int Hkv, int T, int d, float scale, int* status, unsigned long long timeout_ns,
                  void* stream) {
  const size_t vb = fa_visible_window_size(B, T, window, sinks);
  if (!visible || vb == 0) return FA_ERR_INVALID_ARG;
  return bwd_mod(q, k, v, o, dout, lse, rest, dq, dk, dv, workspace, workspace_bytes,
                 fa_bwd_window_workspace_size(B, H, Hkv, T, d, window, sinks), visible, vb, 1, window, sinks, softcap, slopes,
                 B, H, Hkv, T, d, scale, status, timeout_ns, stream);
}

}  // extern "C"
