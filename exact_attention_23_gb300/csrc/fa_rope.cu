// Rotary positions (include/fa.h: fa_rope, fa_rope_append): pairs (a, b) of a head's first
// rot_dim dimensions are turned by the angle position · inv_freq[pair],
//
//   a' = m·(a·cos − b·sin),   b' = m·(a·sin + b·cos)      (inverse: sin → −sin, the gradient)
//
// the pair being dimensions (i, i + rot/2) in the half layout and (2i, 2i + 1) interleaved.
//
// The angle. A float product of a far position and a frequency loses the angle itself (at
// position 10⁶ an fp32 step is 0.06 rad), so it is kept as a fixed-point fraction of a turn:
// frequency / 2π in units of 2⁻⁶⁴ turns, multiplied by the integer position modulo 2⁶⁴, which
// drops whole turns exactly. The top 32 bits are the angle within ±π, where __cosf and __sinf are
// within 2⁻²¹. That is absolute: a result is within 2⁻²⁰·m·(|a| + |b|) before its rounding to bf16,
// beside which the slower functions would show only where a·cos − b·sin cancels to less than
// 2⁻¹¹·(|a| + |b|).
// Each block makes the fixed-point frequencies once, in shared memory: five fp64 operations a
// pair, of which an SM does two lanes a clock (every thread making its own took 13 of the 20 µs
// of B4 H12+12 T1024 d64).
//
// The kernel moves bytes: each row is read and written once (2 + 2 bytes an element against
// three multiply-adds a dimension). A thread owns 8 pairs (two 16-byte vectors) of one (batch,
// position) and walks several heads with them, so the angles' 64-bit products, sines and cosines
// are paid once for all its heads; four heads' loads are in flight together. Reading
// with the caller's strides lets a packed projection [B, T, heads, d] be turned straight into
// the contiguous [B, H, T, d] that attention reads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "fa.h"
#include "fa_host.h"
#include "fa_pdl.h"
#include "sm103.cuh"

namespace fa {

struct RopeSrc {
  const __nv_bfloat16* p;
  long long sb, sh, st;  // strides in elements
};

struct RopeParams {
  RopeSrc q, k, v;
  __nv_bfloat16 *q_out, *k_out, *v_out;  // [B][heads][rows][d], rows: T (rope) or Tmax (caches)
  const int* positions;                  // [T] or [B][T]; null: t, or context + t
  const int* ctx_len;                    // append: [B]
  const double* inv_freq;
  long long n_items;                     // B · T · d / 16
  unsigned n_blocks;                     // blocks per head chunk
  int pos_per_batch;
  int B, H, Hkv, T, Tmax, d_units, rot_units, log2_units;
  int heads, chunk;                      // q + k (+ v) heads; heads a thread walks
  float mscale, sign;
};

// 128 threads at 64 registers, eight blocks an SM: B1 H16+4 T16384 d128 (168 MB) 29.9 µs, 5.6 TB/s;
// B4 H12+12 T1024 d64 (25 MB) 7.9. (256 threads at 72 registers 32.1 and 8.4; two heads in
// flight at 48 registers 31.5 and 7.5; 42 registers, which spill, 40.7 and 10.3.)
constexpr int kRopeThreads = 128;
constexpr int kRopeBlocks = 8;
constexpr int kRopeFlight = 4;  // heads whose loads a thread keeps in flight

__device__ __forceinline__ void unpack8(const uint4& w, float* f) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(u[e] << 16);
    f[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
  }
}

template <bool INTER, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) fa_rope_kernel(const RopeParams p) {
  __shared__ unsigned long long turns[64];  // turns a position, in 2⁻⁶⁴
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x < 8 * p.rot_units) {
    const double f = p.inv_freq[threadIdx.x] * 0.15915494309189533577;  // 1 / 2π
    turns[threadIdx.x] = __double2ull_rn((f - floor(f)) * 18446744073709551616.0);
  }
  __syncthreads();
  const unsigned ch = blockIdx.x / p.n_blocks;
  const long long item = static_cast<long long>(blockIdx.x - ch * p.n_blocks) * kRopeThreads + threadIdx.x;
  if (item >= p.n_items) return;
  const int u = static_cast<int>(item & (p.d_units - 1));
  const long long row = item >> p.log2_units;
  const int b = static_cast<int>(row / p.T);
  const int t = static_cast<int>(row - static_cast<long long>(b) * p.T);
  const int D = p.d_units * 16;
  const bool turn = u < p.rot_units;
  // The two 16-byte vectors of this unit: (i, i + rot/2) or neighbours.
  const int c0 = (turn && !INTER) ? u * 8 : u * 16;
  const int c1 = (turn && !INTER) ? (p.rot_units + u) * 8 : u * 16 + 8;

  const int h0 = static_cast<int>(ch) * p.chunk, h1 = min(p.heads, h0 + p.chunk);
  int ctx = 0;
  bool live = true;    // append: an active sequence
  bool stored = true;  // append: the row exists in the caches
  if constexpr (APPEND) {
    ctx = p.ctx_len[b];
    live = ctx >= 0;
    stored = live && static_cast<long long>(ctx) + t < p.Tmax;
  }
  float cs[8], sn[8];
  if (turn && live && h0 < p.H + p.Hkv) {
    const long long pos = p.positions ? p.positions[p.pos_per_batch ? row : t] : static_cast<long long>(ctx) + t;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const unsigned long long a = turns[u * 8 + e] * static_cast<unsigned long long>(pos);
      const float x = static_cast<float>(static_cast<int>(a >> 32)) * 1.4629180792671596e-9f;  // 2π·2⁻³²
      cs[e] = __cosf(x) * p.mscale;
      sn[e] = __sinf(x) * (p.mscale * p.sign);
    }
  }
  for (int hb = h0; hb < h1; hb += kRopeFlight) {
    uint4 x0[kRopeFlight], x1[kRopeFlight];
#pragma unroll
    for (int i = 0; i < kRopeFlight; ++i) {
      const int h = hb + i;
      if (h >= h1 || !live) continue;
      const bool is_q = h < p.H, is_k = !is_q && h < p.H + p.Hkv;
      const RopeSrc s = is_q ? p.q : (is_k ? p.k : p.v);
      const int hh = is_q ? h : (is_k ? h - p.H : h - p.H - p.Hkv);
      const __nv_bfloat16* src = s.p + b * s.sb + hh * s.sh + t * s.st;
      x0[i] = *reinterpret_cast<const uint4*>(src + c0);
      x1[i] = *reinterpret_cast<const uint4*>(src + c1);
    }
#pragma unroll
    for (int i = 0; i < kRopeFlight; ++i) {
      const int h = hb + i;
      if (h >= h1) continue;
      const bool is_q = h < p.H, is_k = !is_q && h < p.H + p.Hkv;
      uint4 y0 = x0[i], y1 = x1[i];
      if (!live) {
        y0 = y1 = make_uint4(0u, 0u, 0u, 0u);
      } else if (turn && (is_q || is_k)) {
        float v[16];
        unpack8(x0[i], v);
        unpack8(x1[i], v + 8);
        float w[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int ia = INTER ? 2 * e : e, ib = INTER ? 2 * e + 1 : e + 8;
          w[ia] = fmaf(v[ia], cs[e], -v[ib] * sn[e]);
          w[ib] = fmaf(v[ia], sn[e], v[ib] * cs[e]);
        }
        y0 = make_uint4(pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]), pack_bf16x2(w[4], w[5]),
                        pack_bf16x2(w[6], w[7]));
        y1 = make_uint4(pack_bf16x2(w[8], w[9]), pack_bf16x2(w[10], w[11]),
                        pack_bf16x2(w[12], w[13]), pack_bf16x2(w[14], w[15]));
      }
      __nv_bfloat16* dst;
      if (is_q) {
        dst = p.q_out + ((static_cast<size_t>(b) * p.H + h) * p.T + t) * D;
      } else {
        if (APPEND && !stored) continue;
        const int hh = is_k ? h - p.H : h - p.H - p.Hkv;
        __nv_bfloat16* base = is_k ? p.k_out : p.v_out;
        const size_t rows = APPEND ? p.Tmax : p.T;
        dst = base + ((static_cast<size_t>(b) * p.Hkv + hh) * rows + (APPEND ? ctx + t : t)) * D;
      }
      *reinterpret_cast<uint4*>(dst + c0) = y0;
      *reinterpret_cast<uint4*>(dst + c1) = y1;
    }
  }
}

namespace {

using namespace fa::host;

// The bytes a strided [B, heads, T, d] source spans, or 0 when its strides are not usable
// (negative, or rows that a 16-byte vector cannot read).
size_t span_bytes(const RopeSrc& s, int B, int heads, int T, int d) {
  if (s.sb < 0 || s.sh < 0 || s.st < 0 || (s.sb & 7) || (s.sh & 7) || (s.st & 7)) return 0;
  constexpr long long kMax = 1LL << 60;
  if ((B > 1 && s.sb > kMax / B) || (heads > 1 && s.sh > kMax / heads) || (T > 1 && s.st > kMax / T))
    return 0;
  return static_cast<size_t>((B - 1) * s.sb + (heads - 1) * s.sh + (T - 1) * s.st + d) * 2;
}

bool contiguous(const RopeSrc& s, int B, int heads, int T, int d) {
  return (T == 1 || s.st == d) && (heads == 1 || s.sh == static_cast<long long>(T) * d) &&
         (B == 1 || s.sb == static_cast<long long>(heads) * T * d);
}

int rope_launch(RopeParams& p, bool append, int interleaved, int d, void* stream) {
  int dev = -1, sms = 0;
  const int st = check_device(&dev, &sms);
  if (st != FA_OK) return st;
  p.d_units = d / 16;
  p.log2_units = d == 64 ? 2 : 3;
  p.heads = p.H + p.Hkv * (append ? 2 : 1);
  p.n_items = static_cast<long long>(p.B) * p.T * p.d_units;
  const long long blocks = (p.n_items + kRopeThreads - 1) / kRopeThreads;
  // Heads a thread walks: as many as leave every SM its eight blocks, so that the angles are shared
  // widely on long sequences and a short call spreads over the GPU.
  long long chunk = p.heads;
  while (chunk > 1 && blocks * ((p.heads + chunk - 1) / chunk) < static_cast<long long>(kRopeBlocks) * sms) chunk = (chunk + 1) / 2;
  p.chunk = static_cast<int>(chunk);
  const long long grid = blocks * ((p.heads + chunk - 1) / chunk);
  if (grid > INT32_MAX) return FA_ERR_INVALID_ARG;
  p.n_blocks = static_cast<unsigned>(blocks);
  auto s = static_cast<cudaStream_t>(stream);
  auto* fn = append ? (interleaved ? &fa_rope_kernel<true, true> : &fa_rope_kernel<false, true>)
                    : (interleaved ? &fa_rope_kernel<true, false> : &fa_rope_kernel<false, false>);
  return launch_pdl(fn, static_cast<unsigned>(grid), kRopeThreads, 0, s, p) == cudaSuccess
             ? FA_OK : FA_ERR_LAUNCH;
}

// Whether an output lies over one of the small inputs.
bool over_tables(const void* out, size_t bytes, const int* positions, int per_batch, const double* inv_freq,
                 int rot_dim, const int* ctx_len, int B, int T) {
  const size_t pb = static_cast<size_t>(per_batch ? B : 1) * T * 4;
  return (positions && overlaps(out, bytes, positions, pb)) ||
         overlaps(out, bytes, inv_freq, static_cast<size_t>(rot_dim) * 4) ||
         (ctx_len && overlaps(out, bytes, ctx_len, static_cast<size_t>(B) * 4));
}

bool sizes_ok(int B, int H, int Hkv, int T, int d, int rot_dim, float mscale) {
  if (B <= 0 || H <= 0 || Hkv < 0 || T <= 0 || (d != 64 && d != 128)) return false;
  if (rot_dim <= 0 || rot_dim > d || (rot_dim & 15)) return false;
  if (!std::isfinite(mscale)) return false;
  const long long rows = static_cast<long long>(B) * T;
  return rows < (1LL << 40) && H <= (1 << 20) && Hkv <= (1 << 20);
}

}  // namespace

}  // namespace fa

using namespace fa;
using namespace fa::host;

extern "C" {

int fa_rope(const void* q, long long q_sb, long long q_sh, long long q_st, void* q_out,
            const void* k, long long k_sb, long long k_sh, long long k_st, void* k_out,
            const int* positions, int positions_per_batch, const double* inv_freq, int rot_dim,
            int interleaved, int inverse, float mscale, int B, int H, int Hkv, int T, int d,
            void* stream) {
  if (!q || !q_out || !inv_freq || !sizes_ok(B, H, Hkv, T, d, rot_dim, mscale))
    return FA_ERR_INVALID_ARG;
  if ((Hkv > 0) != (k != nullptr) || (Hkv > 0) != (k_out != nullptr)) return FA_ERR_INVALID_ARG;
  RopeParams p{};
  p.q = {static_cast<const __nv_bfloat16*>(q), q_sb, q_sh, q_st};
  p.k = {static_cast<const __nv_bfloat16*>(k), k_sb, k_sh, k_st};
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(k_out) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u) || (reinterpret_cast<uintptr_t>(inv_freq) & 7u))
    return FA_ERR_MISALIGNED;
  const size_t qs = span_bytes(p.q, B, H, T, d), ks = k ? span_bytes(p.k, B, Hkv, T, d) : 1;
  if (qs == 0 || ks == 0) return FA_ERR_INVALID_ARG;
  // An output may be its own input where that is contiguous (each thread reads what it writes);
  // any other overlap is refused.
  const size_t qo = static_cast<size_t>(B) * H * T * d * 2, ko = static_cast<size_t>(B) * Hkv * T * d * 2;
  const bool q_in_place = q == q_out && contiguous(p.q, B, H, T, d);
  const bool k_in_place = k && k == k_out && contiguous(p.k, B, Hkv, T, d);
  if (!q_in_place && overlaps(q_out, qo, q, qs)) return FA_ERR_INVALID_ARG;
  if (k && ((!k_in_place && overlaps(k_out, ko, k, ks)) || overlaps(q_out, qo, k, ks) ||
            overlaps(k_out, ko, q, qs) || overlaps(q_out, qo, k_out, ko)))
    return FA_ERR_INVALID_ARG;
  if (over_tables(q_out, qo, positions, positions_per_batch, inv_freq, rot_dim, nullptr, B, T) ||
      (k && over_tables(k_out, ko, positions, positions_per_batch, inv_freq, rot_dim, nullptr, B, T)))
    return FA_ERR_INVALID_ARG;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.positions = positions;
  p.pos_per_batch = positions_per_batch != 0;
  p.inv_freq = inv_freq;
  p.rot_units = rot_dim / 16;
  p.B = B; p.H = H; p.Hkv = Hkv; p.T = T; p.Tmax = T;
  p.mscale = mscale;
  p.sign = inverse ? -1.0f : 1.0f;
  return rope_launch(p, false, interleaved, d, stream);
}

int fa_rope_append(const void* q, long long q_sb, long long q_sh, long long q_st, void* q_out,
                   const void* k, long long k_sb, long long k_sh, long long k_st, const void* v,
                   long long v_sb, long long v_sh, long long v_st, void* k_cache, void* v_cache,
                   const int* ctx_len, const int* positions, int positions_per_batch,
                   const double* inv_freq, int rot_dim, int interleaved, float mscale, int B, int H,
                   int Hkv, int Tq, int Tmax, int d, void* stream) {
  if (!q || !q_out || !k || !v || !k_cache || !v_cache || !ctx_len || !inv_freq ||
      !sizes_ok(B, H, Hkv, Tq, d, rot_dim, mscale) || Hkv <= 0 || Tmax <= 0)
    return FA_ERR_INVALID_ARG;
  RopeParams p{};
  p.q = {static_cast<const __nv_bfloat16*>(q), q_sb, q_sh, q_st};
  p.k = {static_cast<const __nv_bfloat16*>(k), k_sb, k_sh, k_st};
  p.v = {static_cast<const __nv_bfloat16*>(v), v_sb, v_sh, v_st};
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(v) || !aligned16(k_cache) ||
      !aligned16(v_cache) || (reinterpret_cast<uintptr_t>(positions) & 3u) ||
      (reinterpret_cast<uintptr_t>(ctx_len) & 3u) || (reinterpret_cast<uintptr_t>(inv_freq) & 7u))
    return FA_ERR_MISALIGNED;
  const size_t qs = span_bytes(p.q, B, H, Tq, d), ks = span_bytes(p.k, B, Hkv, Tq, d);
  const size_t vs = span_bytes(p.v, B, Hkv, Tq, d);
  if (qs == 0 || ks == 0 || vs == 0) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * Hkv > (1LL << 60) / d / Tmax) return FA_ERR_INVALID_ARG;
  const size_t qo = static_cast<size_t>(B) * H * Tq * d * 2;
  const size_t cb = static_cast<size_t>(B) * Hkv * Tmax * d * 2;
  const bool q_in_place = q == q_out && contiguous(p.q, B, H, Tq, d);
  const void* outs[3] = {q_out, k_cache, v_cache};
  const size_t out_bytes[3] = {qo, cb, cb};
  const void* ins[3] = {q, k, v};
  const size_t in_bytes[3] = {qs, ks, vs};
  for (int a = 0; a < 3; ++a) {
    if (over_tables(outs[a], out_bytes[a], positions, positions_per_batch, inv_freq, rot_dim, ctx_len, B, Tq))
      return FA_ERR_INVALID_ARG;
    for (int b = 0; b < 3; ++b)
      if (!(a == 0 && b == 0 && q_in_place) && overlaps(outs[a], out_bytes[a], ins[b], in_bytes[b]))
        return FA_ERR_INVALID_ARG;
    for (int b = a + 1; b < 3; ++b)
      if (overlaps(outs[a], out_bytes[a], outs[b], out_bytes[b])) return FA_ERR_INVALID_ARG;
  }
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_cache);
  p.v_out = static_cast<__nv_bfloat16*>(v_cache);
  p.positions = positions;
  p.pos_per_batch = positions_per_batch != 0;
  p.ctx_len = ctx_len;
  p.inv_freq = inv_freq;
  p.rot_units = rot_dim / 16;
  p.B = B; p.H = H; p.Hkv = Hkv; p.T = Tq; p.Tmax = Tmax;
  p.mscale = mscale;
  p.sign = 1.0f;
  return rope_launch(p, true, interleaved, d, stream);
}

}  // extern "C"
