// How attention of new tokens against a cache (fa_fwd_tree) shares out its work, and its mask.
//
// The list: for each sequence b with keys, its Hkv key heads times row blocks (the query rows that
// read the same keys, R = (H / Hkv)·Tq of them, in blocks), each entry with the chunks of the
// sequence's min(ctx_b + Tq, Tmax) keys.
//
// Work is cut by keys, not by sequences: all chunks of all (sequence, key head, row block) are
// numbered in a row, and CTA c takes the c-th of equal stretches, whatever the lengths are (they
// live on the device). A stretch crosses sequences in segments; a sequence that lies in several
// stretches leaves one partial (normalised fp32 rows and LSE) per stretch for
// fa_tree_combine_kernel. (Caches short enough for one CTA an entry, with a window
// or in 4 bits a cluster of them, go without: solo.) Stretch c's segment of list entry e has slot c + e: from one segment to
// the next c or e grows, so slots never meet.
#pragma once

#include "fa_mod.cuh"
#include "sm103.cuh"

namespace fa {

struct TreeList {
  const int* ctx_len;  // [B], < 0: inactive
  int B, Hkv, Tq, Tmax;
  int row_blocks;      // row blocks a key head
  int min_per;         // chunks a stretch has at least
  int chunk_log2;      // keys a chunk: 1 << chunk_log2
  int solo;            // CTA c takes entry c whole: no partials, no second kernel (WINDOW: cluster c, of `solo` CTAs)
  int2* parts;         // [entries] the first stretch that an entry lies in, and their number
};

struct TreeReach {
  int window, sinks;   // WINDOW: see tree_window
};

struct TreeMask {
  const uint8_t* tree;  // [Tq][Tq] or [B][Tq][Tq], or null (chain)
  const int* depths;    // [Tq] or [B][Tq], or null (0, 1, 2, …); BIAS
  FastDiv div_tq;       // row / Tq = query head within the key head's group
  int tree_per_batch, depths_per_batch;

  // Row t's flags, and a sequence's depths.
  __device__ __forceinline__ const uint8_t* row(int b, int t, int Tq) const {
    return tree + ((tree_per_batch ? static_cast<size_t>(b) * Tq : 0) + t) * Tq;
  }
  __device__ __forceinline__ const int* depths_of(int b, int Tq) const {
    return depths + (depths_per_batch ? static_cast<size_t>(b) * Tq : 0);
  }
};

__device__ __forceinline__ int tree_keys(const TreeList& p, int ctx) {
  return static_cast<int>(min(static_cast<long long>(ctx) + p.Tq, static_cast<long long>(p.Tmax)));
}

// WINDOW. A token at position ctx + depth (depths below 0 count as 0) sees the context's keys behind
// position ctx + depth − window and those before `sinks`, and of the new tokens that it sees otherwise
// those whose positions are such. So a sequence's list holds the chunks with sinks and those from the
// first window's start on: list chunk c is chunk c of the cache up to sc and chunk c + gap from there.
__device__ __forceinline__ int tree_depth(int depth) { return max(depth, 0); }
// The first row of the context in a token's window, and in any token's.
__device__ __forceinline__ int tree_row_start(const TreeList& p, const TreeReach& w, int ctx, int depth) {
  const long long lo = static_cast<long long>(ctx) + depth - w.window + 1;
  return static_cast<int>(min(max(lo, 0ll), static_cast<long long>(p.Tmax)));
}
__device__ __forceinline__ int tree_window_start(const TreeList& p, const TreeReach& w, int ctx) {
  return tree_row_start(p, w, ctx, 0);
}
// (One chunk stays, whatever is left of the window, so that a sequence with a context has an entry.)
__device__ __forceinline__ int tree_window(const TreeList& p, const TreeReach& w, int ctx, int* sc, int* gap) {
  const int size = 1 << p.chunk_log2, keys = tree_keys(p, ctx);
  const int total = (keys + size - 1) >> p.chunk_log2;
  const int first = min(tree_window_start(p, w, ctx) >> p.chunk_log2, total - 1);
  *sc = (min(w.sinks, keys) + size - 1) >> p.chunk_log2;
  *gap = max(0, first - *sc);
  return total - *gap;
}

template <bool WINDOW>
__device__ __forceinline__ int tree_chunks(const TreeList& p, const TreeReach& w, int b) {
  const int ctx = p.ctx_len[b];
  if (ctx < 0) return 0;
  if constexpr (WINDOW) {
    int sc, gap;
    return tree_window(p, w, ctx, &sc, &gap);
  }
  const long long keys = static_cast<long long>(ctx) + p.Tq;
  return static_cast<int>((min(keys, static_cast<long long>(p.Tmax)) + (1 << p.chunk_log2) - 1) >> p.chunk_log2);
}

// Of the 32 sequences from b0: this lane's chunks (of one list entry), and the positions up to and
// with this lane's sequence; whole warp. (Positions fit an int: the host refuses longer lists.)
template <bool WINDOW>
__device__ __forceinline__ void tree_scan(const TreeList& p, const TreeReach& w, int b0, int* chunks, int* incl) {
  const int lane = threadIdx.x & 31;
  *chunks = b0 + lane < p.B ? tree_chunks<WINDOW>(p, w, b0 + lane) : 0;
  int x = *chunks * p.Hkv * p.row_blocks;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  *incl = x;
}

// The list's length; the scan of its last 32 sequences stays in chunks and incl. Whole warp.
template <bool WINDOW>
__device__ __forceinline__ int tree_total(const TreeList& p, const TreeReach& w, int* chunks, int* incl) {
  int run = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    tree_scan<WINDOW>(p, w, b0, chunks, incl);
    run += __shfl_sync(0xffffffffu, *incl, 31);
  }
  return run;
}

// A stretch's segments in order.
template <bool WINDOW>
struct TreeSegments {
  struct {
    int b, chunks;               // sequence, its chunks
    int entry0;                  // list entry of the sequence's first (key head, row block)
    int start;                   // position of its first chunk
  } at;
  int pos, end;                  // next position, past the stretch's last
  int per;                       // chunks a stretch
  // the current segment
  int b, hk, rb, entry, c0, c1;  // sequence, key head, row block, list entry, chunks [c0, c1)
  bool whole;                    // it covers its entry
  __device__ __forceinline__ void begin(const TreeList& p, const TreeReach& reach) {
    if (p.solo) {
      const int entries = p.Hkv * p.row_blocks;
      at.b = static_cast<int>(WINDOW ? cluster_id() : blockIdx.x) / entries;
      at.entry0 = at.b * entries;
      at.chunks = tree_chunks<WINDOW>(p, reach, at.b);
      pos = 0;
      end = 1;
      return;
    }
    int n, incl;
    const int total = tree_total<WINDOW>(p, reach, &n, &incl);
    per = max(static_cast<int>((total + gridDim.x - 1u) / gridDim.x), p.min_per);
    // (a list shorter than grid · min_per leaves later CTAs nothing)
    pos = static_cast<int>(min(static_cast<long long>(per) * blockIdx.x, static_cast<long long>(total)));
    end = min(total - pos, per) + pos;
    if (pos >= end) return;
    // The sequence that pos lies in: up to 32 sequences from the scan at hand (a second one, with
    // its loads, cost every CTA 0.4 µs before its first key), else block by block.
    int run = 0, b0 = 0;
    if (p.B > 32) {
      for (; b0 < p.B; b0 += 32) {
        tree_scan<WINDOW>(p, reach, b0, &n, &incl);
        const int sum = __shfl_sync(0xffffffffu, incl, 31);
        if (pos < run + sum) break;
        run += sum;
      }
    }
    const int w = __ffs(__ballot_sync(0xffffffffu, run + incl > pos)) - 1;
    at.b = b0 + w;
    at.chunks = __shfl_sync(0xffffffffu, n, w);
    at.entry0 = at.b * p.Hkv * p.row_blocks;
    at.start = run + __shfl_sync(0xffffffffu, incl, w) - at.chunks * p.Hkv * p.row_blocks;
  }
  __device__ __forceinline__ bool next(const TreeList& p, const TreeReach& reach) {
    if (pos >= end) return false;
    if (p.solo) {  // (a sequence without keys has an empty segment, whose rows it writes)
      pos = 1;
      b = at.b;
      entry = static_cast<int>(WINDOW ? cluster_id() : blockIdx.x);
      hk = (entry - at.entry0) / p.row_blocks;
      rb = entry - at.entry0 - hk * p.row_blocks;
      c0 = 0;
      c1 = at.chunks;
      whole = true;
      if constexpr (WINDOW) {  // (a list has fewer than 2²⁴ chunks an entry, a cluster at most 8 CTAs)
        const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(cluster_ctas());
        c0 = at.chunks * rank / ctas;
        c1 = at.chunks * (rank + 1) / ctas;
      }
      return true;
    }
    const int entries = p.Hkv * p.row_blocks;
    int y = pos - at.start;
    while (y >= at.chunks * entries) {  // the next sequence with chunks
      at.start += at.chunks * entries;
      at.entry0 += entries;
      y = pos - at.start;
      ++at.b;
      at.chunks = tree_chunks<WINDOW>(p, reach, at.b);
    }
    const int e = y / at.chunks;
    b = at.b;
    hk = e / p.row_blocks;
    rb = e - hk * p.row_blocks;
    entry = at.entry0 + e;
    c0 = y - e * at.chunks;
    c1 = min(at.chunks, c0 + (end - pos));
    whole = c0 == 0 && c1 == at.chunks;
    pos += c1 - c0;
    return true;
  }
  // For fa_tree_combine_kernel: the CTA with an entry's first chunk says where its partials lie.
  // (One thread, in every segment. The combine finding this by itself, from all the lengths, took
  // it three more trips to memory and two divisions a row.)
  __device__ __forceinline__ void note_parts(const TreeList& p) const {
    if (p.solo || c0 != 0) return;
    const int c = static_cast<int>(blockIdx.x);
    p.parts[entry] = make_int2(c, whole ? 1 : (pos - c1 + at.chunks - 1) / per - c + 1);
  }
};

}  // namespace fa
