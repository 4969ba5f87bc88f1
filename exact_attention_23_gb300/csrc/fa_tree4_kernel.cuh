// New tokens against a cache held in 4 bits (fa_four.cuh): what fa_tree_kernel.cuh computes, over the same
// list of work and with the same masks, a sliding window among them (INT_MAX: none).
//
// A key's K and V row are d + d/8 bytes, a quarter of bf16's, and each of its 2d codes has to become a
// bf16 operand: a shift, a mask and a fused multiply-add a pair. That, not the memory, is what most
// instructions are for, so a code is made into an operand once for as many query rows as there are:
// keys and dimensions stand on the 16-row side of the products, Sᵀ = K·Qᵀ and Oᵀ = Vᵀ·Pᵀ, and the query rows
// on the side of 8. NB = 1 or 2 blocks of 8 rows share the operands (and a decoded token's 4 or 8 heads
// pay for no row that is not there, as 16 rows would). P goes from the layout of a result to that of an
// operand by movmatrix. More rows than 16 are further entries of the list.
//
// Measured: B8 H16 Hkv4, one token, contexts to 16384, d128 (59 MB) 24.0 µs, to 60000 (217 MB) 56.1, 3.9 TB/s (41 with
// operands left unmade: shifts, masks and multiply-adds are what it spends on top of streaming); B4 12 heads,
// 8 drafts, to 4000, d64 10.6 (in clusters of eight CTAs; 13.5 in stretches). With the query rows on the 16 side and 16 of them always: 36.4 and 17.4.
// Three CTAs an SM, four at d = 64, and four tiles a ring for 8 rows (16384 keys to 60000: three 24.0 and 56.1, two
// 23.5 and 59.2); two CTAs for 16. Five warps a CTA put three of two CTAs' ten on one quarter of the SM, so these have 168
// registers a thread, and at d = 128 spill 280 to 312 bytes all the same (at d = 64 up to 20).
//
// P is rounded to bf16, as an operand beside V's values must be, and l sums it before that: o is off by 2.3e-3 of its norm
// where its own rounding is 1.69e-3 (64 bits with P so rounded: 2.3e-3 too).
//
// A CTA's four compute warps take 32 keys each of a chunk of 128, with a running maximum, sum and O of
// their own, behind a producer warp that copies the chunk's codes and scales, two contiguous pieces each
// of K and V, into a ring; the warps' parts meet in shared memory at a segment's end.
#pragma once

#include "fa_four.cuh"
#include "fa_mod.cuh"
#include "fa_tree_kernel.cuh"

namespace fa {

struct Tree4Params {
  TreeParams t;
  const uint8_t *k, *v;          // [BHkv][Tmax][D/2] codes
  const __nv_bfloat16 *ks, *vs;  // [BHkv][Tmax][D/32] scales
};

template <int D, int NB>
struct Tree4Cfg {
  static constexpr int kKeys = 128;                        // keys per chunk
  static constexpr int kCodes = kKeys * D / 2;             // a tile's codes, in front of its scales
  static constexpr int kTile = kCodes + kKeys * D / 16;    // K or V of a chunk
  static constexpr int kStages = 4;                        // K or V tiles in flight
  static constexpr int kCtasPerSm = NB == 2 ? 2 : D == 64 ? 4 : 3;
  static constexpr int kRows = NB * 8;
  static constexpr int kRowStride = D + 8;                 // (floats; rows of the merge without bank conflicts)
  static constexpr int kMergeOff = kStages * kTile;
  static constexpr int kSmemBytes = kMergeOff + 4 * kRows * kRowStride * 4 + 128;  // + alignment slack
};

// N = 1, 2 or 4 words of shared memory.
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* at, uint32_t (&r)[N]) {
  if constexpr (N == 1) {
    r[0] = *reinterpret_cast<const uint32_t*>(at);
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(at);
    r[0] = x.x;
    r[1] = x.y;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(at);
    r[0] = x.x;
    r[1] = x.y;
    r[2] = x.z;
    r[3] = x.w;
  }
}
// An 8 × 8 matrix of 16-bit numbers, a row a quad, transposed.
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, int NB, int MOD>
__global__ void __launch_bounds__(kTreeBlock, Tree4Cfg<D, NB>::kCtasPerSm) fa_tree4_kernel(const Tree4Params pp) {
  using C = Tree4Cfg<D, NB>;
  constexpr int kW = D / 32;               // words of a key that a thread reads
  constexpr int kS = D / 64;               // words of a row's scales
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  __shared__ uint64_t full[C::kStages], empty[C::kStages];
  __shared__ uint32_t abort_flag;
  __shared__ float xm[4][C::kRows], xl[4][C::kRows];
  __shared__ float2 ml[C::kRows];  // (solo in a cluster)
  const TreeParams& p = pp.t;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);
    }
    abort_flag = 0u;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const WaitCtl wc{&abort_flag, p.status, p.timeout_ns};
  TreeSegments<true> sg;
  sg.begin(p.list, p.reach);

  if (warp == 4) {
    // ---------------------------------------------------------------- producer
    int n = 0;
    bool ok = true;
    while (ok && sg.next(p.list, p.reach)) {
      const size_t head = static_cast<size_t>(sg.b) * p.list.Hkv + sg.hk;
      int sc, gap;
      tree_window(p.list, p.reach, p.list.ctx_len[sg.b], &sc, &gap);
      for (int u = 2 * sg.c0; ok && u < 2 * sg.c1; ++u, ++n) {  // K and V tiles in turn
        const int st = n % C::kStages;
        if (n >= C::kStages && !mbar_wait_warp(&empty[st], ((n / C::kStages) - 1) & 1, wc)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          uint8_t* dst = sm + st * C::kTile;
          const int key0 = ((u >> 1) + ((u >> 1) < sc ? 0 : gap)) * C::kKeys;
          // (Tmax is a multiple of 8: sizes and addresses are multiples of 16 bytes)
          const int rows = min(C::kKeys, p.list.Tmax - key0);
          const size_t at = head * p.list.Tmax + key0;
          mbar_arrive_expect_tx(&full[st], rows * (D / 2 + D / 16));
          bulk_load(dst, ((u & 1) ? pp.v : pp.k) + at * (D / 2), rows * (D / 2), &full[st]);
          bulk_load(dst + C::kCodes, ((u & 1) ? pp.vs : pp.ks) + at * (D / 32), rows * (D / 16), &full[st]);
        }
        __syncwarp();
      }
    }
    // every copy issued must have landed before the CTA may exit
    const WaitCtl drain = drain_ctl(p.timeout_ns);
    for (int x = n > C::kStages ? n - C::kStages : 0; x < n; ++x)
      mbar_wait_warp(&full[x % C::kStages], (x / C::kStages) & 1, drain);
    return;
  }

  // ------------------------------------------------------------------ compute
  // A result's element e of key tile mt and row block nb: key mt·16 + qr + 8·(e / 2) of the warp's 32, query
  // row nb·8 + qc + e % 2. O's: dimension 16·tile + qr + 8·(e / 2).
  const int qr = lane >> 2, qc = (lane & 3) * 2;
  // This thread's first words within a tile: of key qr of the warp's 32 (K), and of key qc (V)
  const uint8_t* const k_words = sm + (warp * 32 + qr) * (D / 2) + qc * (D / 16);
  const uint8_t* const k_scales = sm + C::kCodes + (warp * 32 + qr) * (D / 16);
  const uint8_t* const v_words = sm + (warp * 32 + qc) * (D / 2) + qr * 4;
  const uint8_t* const v_scales = sm + C::kCodes + (warp * 32 + qc) * (D / 16);
  float* const xo = reinterpret_cast<float*>(sm + C::kMergeOff);  // [4][rows][D + 8]
  const float nan = __uint_as_float(0x7FC00000u);
  int st = 0, ph = 0;  // the ring's next slot, and its phase
  bool ok = true;
  while (sg.next(p.list, p.reach)) {
    const int bh = sg.b * p.list.Hkv + sg.hk;
    if (threadIdx.x == 0) sg.note_parts(p.list);
    const int ctx = p.list.ctx_len[sg.b], Tq = p.list.Tq;
    const int keys = tree_keys(p.list, ctx);
    int sc, gap;
    tree_window(p.list, p.reach, ctx, &sc, &gap);
    const int lo_all = tree_window_start(p.list, p.reach, ctx);
    int tok[2 * NB], dep[2 * NB], lo[2 * NB];  // token, depth (as the window takes it), first context key
    float nsl[2 * NB], at[2 * NB];             // (at: positions from the end of the context)
    int lo_max = 0;
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) {
      const int r = min(sg.rb * C::kRows + (i >> 1) * 8 + qc + (i & 1), p.R - 1);
      const int g = static_cast<int>(p.mask.div_tq.div(static_cast<uint32_t>(r)));
      tok[i] = r - g * Tq;
      const int d = p.mask.depths ? p.mask.depths_of(sg.b, Tq)[tok[i]] : tok[i];
      dep[i] = tree_depth(d);
      lo[i] = tree_row_start(p.list, p.reach, ctx, dep[i]);
      lo_max = max(lo_max, lo[i]);
      if constexpr ((MOD & kModBias) != 0) {
        at[i] = static_cast<float>(d);
        nsl[i] = p.slopes[sg.hk * (p.R / Tq) + g] * -1.4426950408889634f;
      }
    }
    lo_max = __reduce_max_sync(0xffffffffu, lo_max);
    // Q's fragments, the 16 dimensions of a product in the order that the keys' words have them in
    uint32_t qf[NB][D / 16][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = sg.rb * C::kRows + nb * 8 + qr;
      const uint2* q = reinterpret_cast<const uint2*>(p.q + (static_cast<size_t>(bh) * p.R + r) * D + 2 * qc);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint2 x = r < p.R ? q[k * 4] : make_uint2(0u, 0u);
        qf[nb][k][0] = x.x;
        qf[nb][k][1] = x.y;
      }
    }
    float m[2 * NB], l[2 * NB];
    float o[D / 16][NB][4];
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
#pragma unroll
    for (int x = 0; x < D / 16; ++x)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) o[x][nb][0] = o[x][nb][1] = o[x][nb][2] = o[x][nb][3] = 0.f;

    static_assert(C::kStages % 2 == 0, "a chunk's K and V have neighbouring slots");
    for (int c = sg.c0; c < sg.c1 && ok; ++c) {  // (a failed warp walks on: the merges below are joined by all)
      if (!mbar_wait_warp(&full[st], ph, wc)) {
        ok = false;
        break;
      }
      const int kt = st * C::kTile, vt = kt + C::kTile;
      const int key0 = (c + (c < sc ? 0 : gap)) * C::kKeys + warp * 32;  // this warp's first key
      // ---- Sᵀ = K·Qᵀ
      float s[2][NB][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t wa[kW], wb[kW], sa[kS], sb[kS];  // keys qr and qr + 8 of the tile
        lds_words(k_words + kt + mt * 16 * (D / 2), wa);
        lds_words(k_words + kt + (mt * 16 + 8) * (D / 2), wb);
        lds_words(k_scales + kt + mt * 16 * (D / 16), sa);
        lds_words(k_scales + kt + (mt * 16 + 8) * (D / 16), sb);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) s[mt][nb][0] = s[mt][nb][1] = s[mt][nb][2] = s[mt][nb][3] = 0.f;
#pragma unroll
        for (int x = 0; x < kW; ++x) {
          const FourScale fa = four_scale(__byte_perm(sa[x / 2], 0u, x & 1 ? 0x3232 : 0x1010));
          const FourScale fb = four_scale(__byte_perm(sb[x / 2], 0u, x & 1 ? 0x3232 : 0x1010));
          const uint32_t a0[4] = {four_pair<0>(wa[x], fa), four_pair<0>(wb[x], fb), four_pair<1>(wa[x], fa), four_pair<1>(wb[x], fb)};
          const uint32_t a1[4] = {four_pair<2>(wa[x], fa), four_pair<2>(wb[x], fb), four_pair<3>(wa[x], fa), four_pair<3>(wb[x], fb)};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma16816(s[mt][nb], a0, qf[nb][2 * x][0], qf[nb][2 * x][1]);
            mma16816(s[mt][nb], a1, qf[nb][2 * x + 1][0], qf[nb][2 * x + 1][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      // ---- scores to base-2 exponents
      // (BIAS: distances from the end of the context; positions past 2²⁴ are no fp32 numbers)
      const float behind = static_cast<float>(ctx - key0 - qr);
      auto to_exponents = [&]<bool FAR>() {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint64_t s2 = f2_pack(s[mt][nb][2 * h], s[mt][nb][2 * h + 1]);
              uint64_t x2;
              if constexpr ((MOD & kModCap) != 0) x2 = cap2<FAR>(s2, p.cap);
              else x2 = f2_mul(s2, f2_splat(p.scale_log2));
              if constexpr ((MOD & kModBias) != 0) {
                const float d0 = behind - static_cast<float>(mt * 16 + h * 8);
                x2 = f2_add(x2, f2_pack(nsl[2 * nb] * fabsf(at[2 * nb] + d0), nsl[2 * nb + 1] * fabsf(at[2 * nb + 1] + d0)));
              }
              f2_unpack(x2, s[mt][nb][2 * h], s[mt][nb][2 * h + 1]);
            }
      };
      bool far = false;
      if constexpr ((MOD & kModCap) != 0) {
        float a = 0.f;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            a = fmax3(fmax3(a, fabsf(s[mt][nb][0]), fabsf(s[mt][nb][1])), fabsf(s[mt][nb][2]), fabsf(s[mt][nb][3]));
        far = __any_sync(0xffffffffu, a > p.cap.limit);
      }
      if (far) to_exponents.template operator()<true>();
      else to_exponents.template operator()<false>();
      // ---- context keys before a row's window
      if (key0 < lo_max) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = key0 + mt * 16 + h * 8 + qr;
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i)
              if (key >= p.reach.sinks && key < min(lo[i], ctx)) s[mt][i >> 1][2 * h + (i & 1)] = -INFINITY;
          }
      }
      // ---- the new tokens' keys: the tree, and their depths in the bias and the window
      if (key0 + 32 > min(ctx, keys)) {  // (a context may fill the cache)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          // (a tile's flags and depths are loaded at once, from clamped places)
          int see[2][2 * NB], place[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int d = key0 + mt * 16 + h * 8 + qr - ctx, dc = min(max(d, 0), Tq - 1);
            place[h] = p.mask.depths ? p.mask.depths_of(sg.b, Tq)[dc] : dc;
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i)
              see[h][i] = p.mask.tree ? p.mask.row(sg.b, tok[i], Tq)[dc] : (d <= tok[i] ? 1 : 0);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = key0 + mt * 16 + h * 8 + qr, d = key - ctx, there = tree_depth(place[h]);
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) {
              float& x = s[mt][i >> 1][2 * h + (i & 1)];
              if constexpr ((MOD & kModBias) != 0) {  // from the key's index to its position
                if (d >= 0)
                  x += nsl[i] * (fabsf(at[i] - static_cast<float>(place[h])) - fabsf(at[i] - static_cast<float>(d)));
              }
              if (d >= 0 && (see[h][i] == 0 || (dep[i] - there >= p.reach.window && there >= p.reach.sinks - ctx))) x = -INFINITY;
              if (key >= keys) x = -INFINITY;
            }
          }
        }
      }
      // ---- online softmax with a lazy reference, as in fa_tree_kernel
      float mx[2 * NB];
      bool passed = false;
#pragma unroll
      for (int i = 0; i < 2 * NB; ++i) {
        const int nb = i >> 1, e = i & 1;
        mx[i] = fmaxf(fmaxf(s[0][nb][e], s[0][nb][2 + e]), fmaxf(s[1][nb][e], s[1][nb][2 + e]));
        passed = passed || mx[i] > m[i] + kTreeTau;
      }
      if (__any_sync(0xffffffffu, passed)) {
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) {
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 4));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 8));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 16));
          if (mx[i] > m[i] + kTreeTau) {
            const float a = ex2_approx(m[i] - mx[i]);  // 0 while m = −∞
            m[i] = mx[i];
            l[i] *= a;
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
              o[x][i >> 1][i & 1] *= a;
              o[x][i >> 1][2 + (i & 1)] *= a;
            }
          }
        }
      }
      uint32_t pf[2][NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float m0 = m[2 * nb] == -INFINITY ? 0.f : m[2 * nb], m1 = m[2 * nb + 1] == -INFINITY ? 0.f : m[2 * nb + 1];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float p0 = ex2_approx(s[mt][nb][2 * h] - m0), p1 = ex2_approx(s[mt][nb][2 * h + 1] - m1);
            l[2 * nb] += p0;
            l[2 * nb + 1] += p1;
            pf[mt][nb][h] = movmatrix_t(pack_bf16x2(p0, p1));
          }
      }
      // ---- Oᵀ += Vᵀ·Pᵀ
      if (!mbar_wait_warp(&full[st + 1], ph, wc)) {
        ok = false;
        break;
      }
      // Rows behind the last key, and those before every token's window, may hold anything: with a scale of 0
      // they are 0.
      const bool cut = key0 + 32 > keys || (key0 < lo_all && key0 + 32 > p.reach.sinks);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        // this thread's keys: qc, qc + 1, qc + 8, qc + 9 of the tile
        uint32_t sv[4][kS];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = mt * 16 + (e & 1) + (e >> 1) * 8;
          lds_words(v_scales + vt + key * (D / 16), sv[e]);
          if (cut) {
            const int k = key0 + key + qc;
            if (k >= keys || (k >= p.reach.sinks && k < lo_all)) {
#pragma unroll
              for (int h = 0; h < kS; ++h) sv[e][h] = 0u;
            }
          }
        }
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          uint32_t w[4][1];
#pragma unroll
          for (int e = 0; e < 4; ++e) lds_words(v_words + vt + (mt * 16 + (e & 1) + (e >> 1) * 8) * (D / 2) + 32 * h, w[e]);
#pragma unroll
          for (int g = 0; g < 2; ++g) {  // dimensions 64h + 32g …
            const uint32_t half = g ? 0x7632 : 0x5410;
            const uint32_t u0 = __byte_perm(w[0][0], w[1][0], half), u1 = __byte_perm(w[2][0], w[3][0], half);
            const FourScale f0 = four_scale(__byte_perm(sv[0][h], sv[1][h], half));
            const FourScale f1 = four_scale(__byte_perm(sv[2][h], sv[3][h], half));
            const uint32_t a0[4] = {four_pair<0>(u0, f0), four_pair<1>(u0, f0), four_pair<0>(u1, f1), four_pair<1>(u1, f1)};
            const uint32_t a1[4] = {four_pair<2>(u0, f0), four_pair<3>(u0, f0), four_pair<2>(u1, f1), four_pair<3>(u1, f1)};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              mma16816(o[4 * h + 2 * g][nb], a0, pf[mt][nb][0], pf[mt][nb][1]);
              mma16816(o[4 * h + 2 * g + 1][nb], a1, pf[mt][nb][0], pf[mt][nb][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st + 1]);
      st += 2;
      if (st == C::kStages) {
        st = 0;
        ph ^= 1;
      }
    }

    // ---- the segment's end: the warps' parts in shared memory, then rows over all threads
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 4);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 8);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 16);
      const int r = (i >> 1) * 8 + qc + (i & 1);
      if (qr == 0) {
        xm[warp][r] = m[i];
        xl[warp][r] = l[i];
      }
      float* dst = xo + (warp * C::kRows + r) * C::kRowStride + qr;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        dst[x * 16] = o[x][i >> 1][i & 1];
        dst[x * 16 + 8] = o[x][i >> 1][2 + (i & 1)];
      }
    }
    if (!ok && lane == 0) *static_cast<volatile uint32_t*>(&abort_flag) = 1u;
    asm volatile("bar.sync 1, %0;" ::"n"(kTreeThreads) : "memory");
    const bool failed = *static_cast<volatile uint32_t*>(&abort_flag) != 0u;
    constexpr int kPer = D / 8;  // threads a row
    for (int x = threadIdx.x; x < C::kRows * kPer; x += kTreeThreads) {
      const int rr = x / kPer, col = x % kPer * 8, r = sg.rb * C::kRows + rr;
      if (r >= p.R) continue;
      float M = xm[0][rr], L = 0.f, acc[8];
#pragma unroll
      for (int w = 1; w < 4; ++w) M = fmaxf(M, xm[w][rr]);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float mw = xm[w][rr], f = mw == -INFINITY ? 0.f : ex2_approx(mw - M);
        L = fmaf(f, xl[w][rr], L);
        const float4* src = reinterpret_cast<const float4*>(xo + (w * C::kRows + rr) * C::kRowStride + col);
        const float4 a = src[0], b = src[1];
        acc[0] = fmaf(f, a.x, acc[0]);
        acc[1] = fmaf(f, a.y, acc[1]);
        acc[2] = fmaf(f, a.z, acc[2]);
        acc[3] = fmaf(f, a.w, acc[3]);
        acc[4] = fmaf(f, b.x, acc[4]);
        acc[5] = fmaf(f, b.y, acc[5]);
        acc[6] = fmaf(f, b.z, acc[6]);
        acc[7] = fmaf(f, b.w, acc[7]);
      }
      if (p.list.solo > 1) {  // (into the places of the first part, which this thread has read)
        float4* dst = reinterpret_cast<float4*>(xo + rr * C::kRowStride + col);
        dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (col == 0) ml[rr] = make_float2(M, failed ? nan : L);
        continue;
      }
      const bool none = L == 0.f;
      const float inv = failed ? nan : (none ? 0.f : 1.f / L);
      const float ls = failed ? nan : (none ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] *= inv;
      if (sg.whole) {
        const size_t row = static_cast<size_t>(bh) * p.R + r;
        *reinterpret_cast<uint4*>(p.o + row * D + col) =
            make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
                       pack_bf16x2(acc[6], acc[7]));
        if (col == 0) p.lse[row] = ls;
      } else {
        const size_t row = (static_cast<size_t>(blockIdx.x) + sg.entry) * C::kRows + rr;
        float4* dst = reinterpret_cast<float4*>(p.o_part + row * D + col);
        dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (col == 0) p.lse_part[row] = ls;
      }
    }
    if (p.list.solo > 1) {
      tree_cluster_join<D>(p, xo, C::kRowStride, ml, C::kRows, bh, sg.rb);
      return;
    }
    // the merge area may be rewritten once every row has been read
    asm volatile("bar.sync 1, %0;" ::"n"(kTreeThreads) : "memory");
  }
}

}  // namespace fa
