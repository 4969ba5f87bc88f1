// Modified attention scores: what a MOD kernel does to a raw score q·k before the softmax.
//
//   z  = scale · q·k
//   z  = cap · tanh(z / cap)            (CAP)
//   z −= slope_h · |i − j|              (BIAS, i and j the query's and the key's positions)
//   key j is visible to query i iff lo_i ≤ j < hi_i
//
// Every mask here is one interval of keys per query row: causal [0, i + 1), a prompt that sees
// itself [0, max(i + 1, prefix)), a packed document [start, ...) and their combinations. So a row
// needs two integers, a tile of rows walks one contiguous range of K tiles, and only tiles that
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
constexpr int kModTree = 8;  // new tokens against a cache (fa_tree_walk.cuh)

// The cap. With u = z / cap, tanh(u) is
//   |u| ≤ 0.8:  u · P(u²), P of degree 5, fitted to tanh(u)/u by iteratively reweighted least
//               squares: relative error 6·10⁻⁸, so a large cap leaves small scores as they are
//   beyond:     ±(1 − 2 / (1 + 2^(2·log2(e)·|u|))), which saturates by itself (2^y → ∞)
// (tanh.approx.f32 has a relative error of 2⁻¹¹: 0.02 of a score at a cap of 50.) The
// polynomial takes 3.5 issue slots a score on fp32 pairs and no MUFU operation; the exponential
// form takes two MUFU operations beside the softmax's own, and MUFU bounds these kernels at
// head dim 64. So a warp takes the second form only in a step where one of its scores needs it.
constexpr float kCapBend = 0.8f;

struct CapFactors {
  float in;      // scale / cap: u per raw score
  float in_exp;  // 2·log2(e)·scale / cap
  float out;     // cap · log2(e)
  float limit;   // raw scores up to this have |u| ≤ kCapBend
};

__device__ __forceinline__ uint64_t f2_splat(float x) { return f2_pack(x, x); }

// tanh(u)/u from w = u² on fp32 pairs.
__device__ __forceinline__ uint64_t tanh_ratio2(uint64_t w) {
  uint64_t r = f2_fma(f2_splat(-0.00435529975220561f), w, f2_splat(0.01909330114722252f));
  r = f2_fma(r, w, f2_splat(-0.05311431735754013f));
  r = f2_fma(r, w, f2_splat(0.13321048021316528f));
  r = f2_fma(r, w, f2_splat(-0.3333267569541931f));
  return f2_fma(r, w, f2_splat(0.9999999403953552f));
}

// tanh(u) for |u| > kCapBend, from y = 2·log2(e)·u.
__device__ __forceinline__ float tanh_far(float y) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + ex2_approx(fabsf(y))));
  return copysignf(fmaf(-2.0f, r, 1.0f), y);
}

// Whether any of a warp's n raw scores lies beyond the polynomial's range (warp-uniform).
template <int N>
__device__ __forceinline__ bool cap_far(const uint32_t* s, float limit) {
  float m = 0.0f;
#pragma unroll
  for (int t = 0; t < N; t += 2)
    m = fmax3(m, fabsf(__uint_as_float(s[t])), fabsf(__uint_as_float(s[t + 1])));
  return __any_sync(0xffffffffu, m > limit);
}

// tanh(u) of a pair of raw scores; `far` as cap_far.
__device__ __forceinline__ uint64_t cap_tanh2(float s0, float s1, const CapFactors& k, bool far) {
  const uint64_t u = f2_mul(f2_pack(s0, s1), f2_splat(k.in));
  uint64_t t = f2_mul(u, tanh_ratio2(f2_mul(u, u)));
  if (far) {
    float t0, t1;
    f2_unpack(t, t0, t1);
    if (fabsf(s0) > k.limit) t0 = tanh_far(s0 * k.in_exp);
    if (fabsf(s1) > k.limit) t1 = tanh_far(s1 * k.in_exp);
    t = f2_pack(t0, t1);
  }
  return t;
}

}  // namespace fa
