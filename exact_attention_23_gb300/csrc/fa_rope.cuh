// What the kernels that turn rows by their positions share (fa_rope.cu, fa_norm.cu): strided
// sources, fixed-point angles, and the checks of their arguments. Internal.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <cmath>

#include "fa_host.h"

namespace fa {

struct RopeSrc {
  const __nv_bfloat16* p;
  long long sb, sh, st;  // strides in elements
};

__device__ __forceinline__ void unpack8(const uint4& w, float* f) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(u[e] << 16);
    f[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
  }
}

// A frequency (radians a position) as a fraction of a turn in 2⁻⁶⁴, and the angle of a position
// within ±π (fa_rope.cu).
__device__ __forceinline__ unsigned long long turns_of(double inv_freq) {
  const double f = inv_freq * 0.15915494309189533577;  // 1 / 2π
  return __double2ull_rn((f - floor(f)) * 18446744073709551616.0);
}
__device__ __forceinline__ float angle_of(unsigned long long turns, long long pos) {
  const unsigned long long a = turns * static_cast<unsigned long long>(pos);
  return static_cast<float>(static_cast<int>(a >> 32)) * 1.4629180792671596e-9f;  // 2π·2⁻³²
}

namespace host {

// The bytes a strided [B, heads, T, d] source spans, or 0 when its strides are not usable
// (negative, or rows that a 16-byte vector cannot read).
inline size_t span_bytes(const RopeSrc& s, int B, int heads, int T, int d) {
  if (s.sb < 0 || s.sh < 0 || s.st < 0 || (s.sb & 7) || (s.sh & 7) || (s.st & 7)) return 0;
  constexpr long long kMax = 1LL << 60;
  if ((B > 1 && s.sb > kMax / B) || (heads > 1 && s.sh > kMax / heads) || (T > 1 && s.st > kMax / T))
    return 0;
  return static_cast<size_t>((B - 1) * s.sb + (heads - 1) * s.sh + (T - 1) * s.st + d) * 2;
}

inline bool contiguous(const RopeSrc& s, int B, int heads, int T, int d) {
  return (T == 1 || s.st == d) && (heads == 1 || s.sh == static_cast<long long>(T) * d) &&
         (B == 1 || s.sb == static_cast<long long>(heads) * T * d);
}

// Whether an output lies over one of the small inputs.
inline bool over_tables(const void* out, size_t bytes, const int* positions, int per_batch, const double* inv_freq,
                 int rot_dim, const int* ctx_len, int B, int T) {
  const size_t pb = static_cast<size_t>(per_batch ? B : 1) * T * 4;
  return (positions && overlaps(out, bytes, positions, pb)) ||
         overlaps(out, bytes, inv_freq, static_cast<size_t>(rot_dim) * 4) ||
         (ctx_len && overlaps(out, bytes, ctx_len, static_cast<size_t>(B) * 4));
}

inline bool sizes_ok(int B, int H, int Hkv, int T, int d, int rot_dim, float mscale) {
  if (B <= 0 || H <= 0 || Hkv < 0 || T <= 0 || (d != 64 && d != 128)) return false;
  if (rot_dim <= 0 || rot_dim > d || (rot_dim & 15)) return false;
  if (!std::isfinite(mscale)) return false;
  const long long rows = static_cast<long long>(B) * T;
  return rows < (1LL << 40) && H <= (1 << 20) && Hkv <= (1 << 20);
}

}  // namespace host
}  // namespace fa
