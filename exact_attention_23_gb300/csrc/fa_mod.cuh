// Modified attention scores: what a MOD kernel does to a raw score q·k before the softmax.
//
//   z  = scale · q·k
//   z  = cap · tanh(z / cap)            (CAP)
//   z −= slope_h · |i − j|              (BIAS, i and j the query's and the key's positions)
//   key j is visible to query i iff lo_i ≤ j < hi_i
//
// Every mask here is one interval of keys per query row: causal [0, i + 1), a prompt that sees
// itself [0, max(i + 1, prefix)), a packed document [start, ...), a sliding window [i + 1 − window, …)
// and their combinations; sinks (kModSink), the first tokens of a document that stay visible behind
// the window, are a second one in front of it. So a row needs two integers (or four), a tile of rows walks one contiguous range of K tiles, and only tiles that
// an interval's end crosses compare element by element. fa_visible_kernel makes the intervals
// and the walks once for a batch; every layer's forward and backward reads them.
#pragma once

#include "sm103.cuh"

namespace fa {

// Division of 32-bit unsigned numerators by a fixed divisor d ≥ 1 without a divide: with
// m = ⌈2⁶⁴ / d⌉, ⌊n / d⌋ = ⌊m·n / 2⁶⁴⌋ for every n < 2³² (Lemire, Kaser and Kurz, "Faster
// remainder by direct computation", 2019, theorem 1). d = 1 is taken apart (m would not fit).
struct FastDiv {
  uint64_t m;
  uint32_t d;
  static FastDiv make(uint32_t d) { return FastDiv{d > 1u ? ~0ull / d + 1ull : 0ull, d}; }
  __host__ __device__ __forceinline__ uint32_t div(uint32_t n) const {
#ifdef __CUDA_ARCH__
    return d == 1u ? n : static_cast<uint32_t>(__umul64hi(m, n));
#else
    return d == 1u ? n : static_cast<uint32_t>((static_cast<unsigned __int128>(m) * n) >> 64);
#endif
  }
};

constexpr int kModOn = 1;    // modified scores with row intervals
constexpr int kModCap = 2;   // tanh cap
constexpr int kModBias = 4;  // distance bias
constexpr int kModRef = 16;  // with a cap alone, small enough: the softmax's reference is 0 (below)
constexpr int kModRest = 32; // o's rest is written (two tiles; one tile: kModRef only, others look at the pointer)
constexpr int kModTight = 64; // kModRef on two tiles, d = 64, without rest: masked or far steps are common
constexpr int kModTree = 8;  // new tokens against a cache (fa_tree_walk.cuh)
constexpr int kModSink = 128;  // a second interval of keys a row, in front of the first (TREE: a window and sinks)

// The cap. With u = z / cap = in · s (s the raw score), the capped score in base 2 is
//   |u| ≤ 0.8:  s · (c0 + c1·s² + … + c4·s⁸): tanh(u)/u ≈ P(u²), P of degree 4 fitted by
//               iteratively reweighted least squares to a relative error of 1.0·10⁻⁶, with
//               scale·log2(e) and the powers of `in` multiplied into its coefficients on the host.
//               A relative error, so a large cap leaves small scores as they are.
//   beyond:     out · ±(1 − 2 / (1 + 2^(2·log2(e)·|u|))), which saturates by itself (2^y → ∞)
// (tanh.approx.f32 has a relative error of 2⁻¹¹: 0.02 of a score at a cap of 50.) The polynomial
// takes six packed operations a pair of scores and none of the MUFU's, which the softmax's own
// exponentials fill (8 cycles a warp and score); the exponential form takes two MUFU operations a
// score more. A warp takes it, for the columns that it decides for at once (32, or a step's), where
// one of its scores needs it. How often goes by the scores and the cap: with scores of deviation 4
// never at caps of 30 and 50, at 20 in 12 % of the 32s and 38 % of the 128s, at 10 always (forward,
// B1 H12 T16384 d64, 575, 827 and 2187 µs; backward, B2 H16 T4096 d128, 422, 457 and 446).
//
// Capped scores are bounded, so a cap of up to 60 needs no running maximum (kModRef): 2^x for
// |x| ≤ kCapRef is at most 2⁸⁸ and at least 2⁻⁸⁸, and neither sums of 2²⁰ such terms times bf16
// values of ordinary size nor their inverses leave fp32's range; bf16 has the same exponents, so P
// keeps its relative precision. The softmax is then taken against 0: no maximum, no rescaling, and no
// dependency between the capping of a step's last score and the exponential of its first, so
// that FMA and MUFU work overlap (B1 H12 T16384 d64 causal: 885 -> 712 µs, and 575
// on the two-tile kernel).
// Against a row's maximum the weight of a key that outweighs the others is 1, unrounded; against 0
// it is rounded like any other, and a row of one key would not get that key's value. O is therefore
// divided by the weights' sum with the largest one taken as rounded (top_rounded), not by the sum
// that the LSE takes: then an outweighing key's share is 1 again (o's error with scores of deviation
// 4, cap 30: 2.3e-3 -> 2.0e-3 of its norm, its own rounding being 1.66e-3). The largest weight is
// that of the largest raw score, whose capped value is made again at the row's end, but for masked
// and far columns, whose weights are looked at as they are made. (Looking at every weight: 609 µs for
// the 575. A second sum, over all the rounded weights, is no more exact where it matters and cost a
// third of the kernel's time.) A negative scale turns the products' sign on the tensor cores.
constexpr float kCapRef = 88.0f;
constexpr float kCapBend = 0.8f;
constexpr double kCapPoly[5] = {0.9999989943572278, -0.3332537198003981, 0.1323056561802812,
                                -0.04918014254491106, 0.012100138637293043};

// Padding may hold anything. Its P (and dS) are 0, but 0 · NaN must not reach a product, so whoever
// issues the first product of a tile zeroes its padded rows (those of an empty interval) in shared
// memory: `boxes` boxes of [rows][64] bf16, box_bytes apart. Whole warp.
__device__ __forceinline__ void zero_padding(uint32_t tile, int boxes, int box_bytes, int rows,
                                             const int2* intervals) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t m = 0u;  // bit k: row 32·k + lane
#pragma unroll 4
  for (int k = 0; k < rows / 32; ++k) {
    const int2 v = intervals[32 * k + lane];
    if (v.y <= v.x) m |= 1u << k;
  }
  for (; m != 0u; m &= m - 1u) {
    const uint32_t row = tile + (32 * (__ffs(m) - 1) + lane) * 128;
    for (int x = 0; x < boxes; ++x)
#pragma unroll
      for (int c = 0; c < 8; ++c)  // (neighbouring rows at other pieces: no bank conflicts)
        st_shared_v4(row + x * box_bytes + ((c + lane) & 7) * 16, 0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}
// The same, called: inlined into the forward's P·V issuer it costs plain scores 2 % without any padding
// (B1 H12 T16384 d64 421 -> 431 µs); called from the backward, 7 % (B1 H16 Hkv4 T8192 d128 649 -> 695).
static __device__ __noinline__ void zero_padding_called(uint32_t tile, int boxes, int box_bytes, int rows,
                                                        const int2* intervals) {
  zero_padding(tile, boxes, box_bytes, rows, intervals);
}

struct CapFactors {
  float c[5];      // kCapPoly[k] · in^2k · scale · log2(e)
  float in_exp;    // 2·log2(e)·scale / cap
  float out;       // cap · log2(e)
  float bend;      // −1 / out²: 1 − tanh² = 1 + bend · (capped score)²
  float limit;     // raw scores up to this are |u| ≤ kCapBend
};

// The bits [lo, hi) of a word, as far as it has them.
__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; }
__device__ __forceinline__ uint32_t bits_of(int lo, int hi) { return bits_below(hi) & ~bits_below(lo); }

// The sum l of a row's weights with its largest one, w, rounded to bf16.
__device__ __forceinline__ float top_rounded(float l, float w) {
  return l + (__uint_as_float(pack_bf16x2(w, w) & 0xFFFF0000u) - w);
}

__device__ __forceinline__ uint64_t f2_splat(float x) { return f2_pack(x, x); }

// A pair of raw scores to capped ones in base 2; FAR: some score of the warp is beyond the polynomial.
__device__ __forceinline__ float cap_exp(float s, const CapFactors& k) {
  const float y = s * k.in_exp;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + ex2_approx(fabsf(y))));
  return copysignf(fmaf(-2.0f * k.out, r, k.out), y);
}
template <bool FAR>
__device__ __forceinline__ uint64_t cap2(uint64_t s, const CapFactors& k) {
  if constexpr (FAR) {
    float s0, s1;
    f2_unpack(s, s0, s1);
    return f2_pack(cap_exp(s0, k), cap_exp(s1, k));
  } else {
    const uint64_t w = f2_mul(s, s);
    uint64_t r = f2_fma(f2_splat(k.c[4]), w, f2_splat(k.c[3]));
    r = f2_fma(r, w, f2_splat(k.c[2]));
    r = f2_fma(r, w, f2_splat(k.c[1]));
    r = f2_fma(r, w, f2_splat(k.c[0]));
    return f2_mul(s, r);
  }
}

// A row's largest weight (kModRef): top, of those noted as weights, or that of the raw score `raw`,
// the largest of the columns that the polynomial made (−∞: none).
__device__ __forceinline__ float top_weight(float top, float raw, const CapFactors& k) {
  float x, y;
  f2_unpack(cap2<false>(f2_splat(raw), k), x, y);
  return fmaxf(top, raw > -INFINITY ? ex2_approx(x) : 0.0f);
}

}  // namespace fa
