// New tokens against a cache: attention of Tq tokens a sequence (one, a chain, or the nodes of a
// tree of drafts) over a K/V cache of [B, Hkv, Tmax, D] whose sequence b holds ctx_b tokens and,
// behind them, the Tq new ones:
//
//   token t sees key j  iff  j < ctx_b,  or  j = ctx_b + s and tree[t][s] ≠ 0 (chain: s ≤ t)
//
// with fa_mod.cuh's cap and bias. The query heads of a key head read the same keys, so a key
// head's work is R = (H / Hkv)·Tq query rows against its sequence: q, o and lse, [B, H, Tq, D] in
// memory, are [B·Hkv, R, D] as they stand.
//
// Here: key heads of up to 32 rows, in one row block of 16 or 32 (more go to the tensor-core kernel).
//
// Bound: the keys are read once, 4·R FLOP a byte: memory bandwidth. So the kernel is a streaming
// kernel: per CTA a TMA producer warp runs a ring of tiles, the K and then the V of each chunk of 64
// keys, completed on mbarriers, in front of four compute warps, and two or three CTAs share an SM.
//
// Products on mma.sync m16n8k16: a tcgen05 product has at least 64 rows on tensor memory lanes that
// only the same quarter of the warps can read, so at 16 rows its softmax would run on 16 lanes of
// one warp. Here a warp owns 16 rows and their state in registers: RG = 1 or 2 row groups times
// KG = 4 / RG key groups, a key group taking its quarter or half of each chunk with a running maximum,
// sum and O of its own, merged once per segment through shared memory. K is read as B fragments by
// ldmatrix, V by ldmatrix.trans, both conflict-free out of the 128-byte-swizzled boxes that TMA
// writes.
#pragma once

#include "fa_fwd_kernel.cuh"
#include "fa_mod.cuh"
#include "fa_tree_walk.cuh"
#include "sm103.cuh"

namespace fa {

struct TreeParams {
  const __nv_bfloat16* q;  // [BHkv][R][D]
  __nv_bfloat16* o;
  float* lse;              // [BHkv][R]
  float* o_part;           // [slots][rows][D]
  float* lse_part;         // [slots][rows]
  const float* slopes;     // [H]; BIAS
  int* status;
  uint64_t timeout_ns;
  TreeList list;
  TreeMask mask;
  CapFactors cap;
  float scale_log2;
  int R;                   // query rows a key head: (H / Hkv) · Tq
  TreeReach reach;         // WINDOW
};

constexpr int kTreeKeys = 64;        // keys per chunk
constexpr int kTreeThreads = 128;    // compute threads
constexpr int kTreeBlock = kTreeThreads + 32;
constexpr float kTreeTau = 8.0f;     // lazy rescale, as the other forward kernels

template <int D>
struct TreeCfg {
  static constexpr int kBoxBytes = kTreeKeys * 128;        // 64 keys × 64 columns
  static constexpr int kTile = kBoxBytes * (D / 64);       // K or V of a chunk
  static constexpr int kStages = (D == 64) ? 7 : 5;        // K or V tiles in flight
  static constexpr int kCtasPerSm = (D == 64) ? 3 : 2;
  // the key groups' merge: three 16-row fp32 O blocks at most
  static constexpr int kMergeOff = kStages * kTile;
  static constexpr int kSmemBytes = kMergeOff + 3 * 16 * D * 4 + 1024;  // + alignment slack
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An entry in a cluster of CTAs (solo > 1): each has left its keys' part of the rows in its shared memory, fp32
// sums `part` [rows][stride] and `ml`, a row's reference and sum of weights (a NaN where the CTA failed), and
// takes a share of rows × 4 columns to join over all.
template <int D>
__device__ __forceinline__ void tree_cluster_join(const TreeParams& p, const float* part, int stride, const float2* ml,
                                                  int rows, int bh, int rb) {
  constexpr int kMost = 8, kPer = D / 4;  // CTAs; threads a row
  __syncwarp();
  cluster_sync_all();
  const uint32_t ctas = cluster_ctas();
  for (uint32_t x = cluster_ctarank() * kTreeThreads + threadIdx.x; x < static_cast<uint32_t>(rows) * kPer; x += ctas * kTreeThreads) {
    const int rr = static_cast<int>(x) / kPer, col = static_cast<int>(x) % kPer * 4, r = rb * rows + rr;
    if (r >= p.R) break;
    float2 w[kMost];
    float4 y[kMost];
    float M = -INFINITY, L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < kMost; ++s) {
      w[s] = make_float2(-INFINITY, 0.f);
      y[s] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < ctas) {
        w[s] = ld_cluster2(mapa_shared(ml + rr, s));
        y[s] = ld_cluster4(mapa_shared(part + rr * stride + col, s));
      }
    }
#pragma unroll
    for (int s = 0; s < kMost; ++s) M = fmaxf(M, w[s].x);
#pragma unroll
    for (int s = 0; s < kMost; ++s) {
      const float f = w[s].x == -INFINITY ? 0.f : ex2_approx(w[s].x - M);
      L = fmaf(f, w[s].y, L);
      acc[0] = fmaf(f, y[s].x, acc[0]);
      acc[1] = fmaf(f, y[s].y, acc[1]);
      acc[2] = fmaf(f, y[s].z, acc[2]);
      acc[3] = fmaf(f, y[s].w, acc[3]);
    }
    const bool none = L == 0.f;
    const float inv = none ? 0.f : 1.f / L;
    const size_t row = static_cast<size_t>(bh) * p.R + r;
    *reinterpret_cast<uint2*>(p.o + row * D + col) =
        make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
    if (col == 0) p.lse[row] = none ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
  }
  __syncwarp();
  cluster_sync_all();  // no CTA leaves before its part has been read
}

template <int D, int RG, int MOD>
__global__ void __launch_bounds__(kTreeBlock, TreeCfg<D>::kCtasPerSm)
    fa_tree_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const TreeParams p) {
  using C = TreeCfg<D>;
  constexpr int KG = 4 / RG;               // key groups
  constexpr int NK = kTreeKeys / KG;       // keys of a chunk a warp takes
  constexpr int NT = NK / 8;               // score tiles of 16 rows × 8 keys
  constexpr int kRows = RG * 16;
  constexpr int kDT = D / 8;               // output tiles of 16 rows × 8 columns
  constexpr bool kWin = (MOD & kModSink) != 0;  // a window and sinks
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[C::kStages], empty[C::kStages];
  __shared__ uint32_t abort_flag;
  __shared__ float xm[3][16], xl[3][16];
  __shared__ float2 ml[kWin ? kRows : 1];  // (solo in a cluster)
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
  TreeSegments<kWin> sg;
  sg.begin(p.list, p.reach);

  if (warp == 4) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    int n = 0;
    bool ok = true;
    while (ok && sg.next(p.list, p.reach)) {
      const int bh = sg.b * p.list.Hkv + sg.hk;
      int sc = 0, gap = 0;
      if constexpr (kWin) tree_window(p.list, p.reach, p.list.ctx_len[sg.b], &sc, &gap);
      for (int u = 2 * sg.c0; ok && u < 2 * sg.c1; ++u, ++n) {  // K and V tiles in turn
        const int st = n % C::kStages;
        if (n >= C::kStages && !mbar_wait_warp(&empty[st], ((n / C::kStages) - 1) & 1, wc)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          uint8_t* dst = sm + st * C::kTile;
          mbar_arrive_expect_tx(&full[st], C::kTile);
#pragma unroll
          for (int x = 0; x < D / 64; ++x)
            tma_load_3d(dst + x * C::kBoxBytes, (u & 1) ? &tm_v : &tm_k, &full[st], x * 64,
                        ((u >> 1) + ((u >> 1) < sc ? 0 : gap)) * kTreeKeys, bh);
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
  const int rg = warp / KG, kg = warp % KG;
  const int qr = lane >> 2, qc = (lane & 3) * 2;   // fragment row and column of this thread
  const uint32_t ring = smem_u32(sm);
  float* const xo = reinterpret_cast<float*>(sm + C::kMergeOff);  // [3][16][D]
  const float nan = __uint_as_float(0x7FC00000u);
  int n = 0;
  bool ok = true;
  while (sg.next(p.list, p.reach)) {
    const int bh = sg.b * p.list.Hkv + sg.hk;
    if (threadIdx.x == 0) sg.note_parts(p.list);
    const int ctx = p.list.ctx_len[sg.b], Tq = p.list.Tq;
    const int keys = tree_keys(p.list, ctx);
    const int r0 = sg.rb * kRows + rg * 16 + qr;    // this thread's rows: r0 and r0 + 8
    int tok[2];
    int dep[2] = {0, 0}, lo[2] = {0, 0};  // WINDOW: the rows' depths, and their first context keys
    int sc = 0, gap = 0, lo_all = 0;
    if constexpr (kWin) {
      tree_window(p.list, p.reach, ctx, &sc, &gap);
      lo_all = tree_window_start(p.list, p.reach, ctx);
    }
    bool live[2];
    float nsl[2] = {0.f, 0.f}, at[2] = {0.f, 0.f};  // (at: positions from the end of the context)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 8 * i;
      live[i] = r < p.R;
      const int g = static_cast<int>(p.mask.div_tq.div(static_cast<uint32_t>(live[i] ? r : 0)));
      tok[i] = (live[i] ? r : 0) - g * Tq;
      if constexpr (kWin) {
        dep[i] = p.mask.depths ? tree_depth(p.mask.depths_of(sg.b, Tq)[tok[i]]) : tok[i];
        lo[i] = tree_row_start(p.list, p.reach, ctx, dep[i]);
      }
      if constexpr ((MOD & kModBias) != 0) {
        at[i] = static_cast<float>(p.mask.depths ? p.mask.depths_of(sg.b, Tq)[tok[i]] : tok[i]);
        nsl[i] = p.slopes[sg.hk * (p.R / Tq) + g] * -1.4426950408889634f;
      }
    }
    uint32_t qf[D / 16][4];
    {
      const __nv_bfloat16* q0 = p.q + (static_cast<size_t>(bh) * p.R + r0) * D + qc;
      const __nv_bfloat16* q1 = q0 + 8 * D;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][0] = live[0] ? *reinterpret_cast<const uint32_t*>(q0 + k * 16) : 0u;
        qf[k][1] = live[1] ? *reinterpret_cast<const uint32_t*>(q1 + k * 16) : 0u;
        qf[k][2] = live[0] ? *reinterpret_cast<const uint32_t*>(q0 + k * 16 + 8) : 0u;
        qf[k][3] = live[1] ? *reinterpret_cast<const uint32_t*>(q1 + k * 16 + 8) : 0u;
      }
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[kDT][4];
#pragma unroll
    for (int i = 0; i < kDT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    for (int c = sg.c0; c < sg.c1; ++c, n += 2) {
      const int stk = n % C::kStages, stv = (n + 1) % C::kStages;
      if (ok && !mbar_wait_warp(&full[stk], (n / C::kStages) & 1, wc)) ok = false;
      if (!ok) continue;  // (walk on: the merges below are joined by every warp)
      const uint32_t kt = ring + stk * C::kTile, vt = ring + stv * C::kTile;
      const int key0 = (c + (!kWin || c < sc ? 0 : gap)) * kTreeKeys + kg * NK;  // this warp's first key
      // ---- S = Q·Kᵀ
      // (32 dimensions of every key at a time: the fragments' loads stand together in front of
      // products that do not wait for one another)
      float s[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        uint32_t b[NT][4];
        const int ch = (k & 1) * 4 + (lane >> 3);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int row = kg * NK + j * 8 + (lane & 7);
          ldsm4(kt + (k >> 1) * C::kBoxBytes + row * 128 + ((ch ^ (row & 7)) << 4), b[j]);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) mma16816(s[j], qf[2 * k], b[j][0], b[j][1]);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma16816(s[j], qf[2 * k + 1], b[j][2], b[j][3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stk]);
      // ---- scores to base-2 exponents
      // (BIAS: distances from the end of the context; positions past 2²⁴ are no fp32 numbers)
      const float behind = static_cast<float>(ctx - key0);
      auto to_exponents = [&]<bool FAR>() {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint64_t s2 = f2_pack(s[j][2 * i], s[j][2 * i + 1]);
            uint64_t x2;
            if constexpr ((MOD & kModCap) != 0) x2 = cap2<FAR>(s2, p.cap);
            else x2 = f2_mul(s2, f2_splat(p.scale_log2));
            if constexpr ((MOD & kModBias) != 0) {
              const float d0 = at[i] + (behind - static_cast<float>(j * 8 + qc));
              x2 = f2_add(x2, f2_pack(nsl[i] * fabsf(d0), nsl[i] * fabsf(d0 - 1.0f)));
            }
            f2_unpack(x2, s[j][2 * i], s[j][2 * i + 1]);
          }
      };
      bool far = false;
      if constexpr ((MOD & kModCap) != 0) {
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
          a = fmax3(fmax3(a, fabsf(s[j][0]), fabsf(s[j][1])), fabsf(s[j][2]), fabsf(s[j][3]));
        far = __any_sync(0xffffffffu, a > p.cap.limit);
      }
      if (far) to_exponents.template operator()<true>();
      else to_exponents.template operator()<false>();
      if constexpr (kWin) {
        if (__any_sync(0xffffffffu, key0 < max(lo[0], lo[1]))) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = key0 + j * 8 + qc + e;
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (key >= p.reach.sinks && key < min(lo[i], ctx)) s[j][2 * i + e] = -INFINITY;
            }
        }
      }
      // ---- the new tokens' keys: the tree, and their depths in the bias and the window
      const bool tail = key0 + NK > min(ctx, keys);  // (a context may fill the cache)
      if (tail) {
        // Flags and depths are loaded for a pair of tiles at once, from clamped places, so that no
        // load waits for another.
#pragma unroll
        for (int j0 = 0; j0 < NT; j0 += 2) {
          int see[2][2][2], place[2][2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int d = key0 + (j0 + j) * 8 + qc + e - ctx, dc = min(max(d, 0), Tq - 1);
#pragma unroll
              for (int i = 0; i < 2; ++i)
                see[j][e][i] = p.mask.tree ? p.mask.row(sg.b, tok[i], Tq)[dc] : (d <= tok[i] ? 1 : 0);
              if constexpr ((MOD & (kModBias | kModSink)) != 0)
                place[j][e] = p.mask.depths ? p.mask.depths_of(sg.b, Tq)[dc] : dc;
            }
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = key0 + (j0 + j) * 8 + qc + e, d = key - ctx;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float& x = s[j0 + j][2 * i + e];
                if constexpr ((MOD & kModBias) != 0) {  // from the key's index to its position
                  if (d >= 0)
                    x += nsl[i] * (fabsf(at[i] - static_cast<float>(place[j][e])) - fabsf(at[i] - static_cast<float>(d)));
                }
                if constexpr (kWin) {
                  const int there = tree_depth(place[j][e]);
                  if (d >= 0 && dep[i] - there >= p.reach.window && there >= p.reach.sinks - ctx) x = -INFINITY;
                }
                if (key >= keys || (d >= 0 && see[j][e][i] == 0)) x = -INFINITY;
              }
            }
        }
      }
      // ---- online softmax with a lazy reference: in the common step no row's maximum passes its
      // reference by more than τ, and no lane needs another's scores
      float mx[2] = {s[0][0], s[0][2]};
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mx[0] = fmax3(mx[0], s[j][0], s[j][1]);
        mx[1] = fmax3(mx[1], s[j][2], s[j][3]);
      }
      if (__any_sync(0xffffffffu, mx[0] > m[0] + kTreeTau || mx[1] > m[1] + kTreeTau)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
          if (mx[i] > m[i] + kTreeTau) {
            const float a = ex2_approx(m[i] - mx[i]);  // 0 while m = −∞
            m[i] = mx[i];
            l[i] *= a;
#pragma unroll
            for (int x = 0; x < kDT; ++x) {
              o[x][2 * i] *= a;
              o[x][2 * i + 1] *= a;
            }
          }
        }
      }
      const float mu[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
      uint32_t pf[NT / 2][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float p0 = ex2_approx(s[j][2 * i] - mu[i]), p1 = ex2_approx(s[j][2 * i + 1] - mu[i]);
          l[i] += p0 + p1;  // (in fp32; P goes on in bf16, as an operand beside V must: o is off by 2.3e-3 of its norm,
                            // as 64 bits with P so rounded are; o's own rounding is 1.66e-3)
          pf[j / 2][(j & 1) * 2 + i] = pack_bf16x2(p0, p1);
        }
      }
      // ---- O += P·V
      if (!mbar_wait_warp(&full[stv], ((n + 1) / C::kStages) & 1, wc)) {
        ok = false;
        continue;
      }
      // rows behind the last key may hold anything: taken as 0 (WINDOW: and those before every token's)
      const bool cut = key0 + NK > keys || (kWin && key0 < lo_all && key0 + NK > p.reach.sinks);
#pragma unroll
      for (int k = 0; k < NT / 2; ++k) {
        const int row = kg * NK + k * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
        uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
        if (cut) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = key0 + k * 16 + h * 8 + qc;
            auto used = [&](int k) { return k < keys && !(kWin && k >= p.reach.sinks && k < lo_all); };
            keep[h] = (used(key) ? 0x0000FFFFu : 0u) | (used(key + 1) ? 0xFFFF0000u : 0u);
          }
        }
#pragma unroll
        for (int x0 = 0; x0 < D / 16; x0 += 4) {
          uint32_t b[4][4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int ch = x * 2 + (lane >> 4);
            ldsm4_t(vt + (x0 >> 2) * C::kBoxBytes + row * 128 + ((ch ^ (row & 7)) << 4), b[x]);
            if (cut) {
              b[x][0] &= keep[0];
              b[x][1] &= keep[1];
              b[x][2] &= keep[0];
              b[x][3] &= keep[1];
            }
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            mma16816(o[2 * (x0 + x)], pf[k], b[x][0], b[x][1]);
            mma16816(o[2 * (x0 + x) + 1], pf[k], b[x][2], b[x][3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stv]);
    }

    // ---- the segment's end: sums over the quad, then over the key groups
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    if constexpr (KG > 1) {
      const int slot = rg * (KG - 1) + kg - 1;
      if (kg > 0) {
        if ((lane & 3) == 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            xm[slot][qr + 8 * i] = m[i];
            xl[slot][qr + 8 * i] = l[i];
          }
        }
#pragma unroll
        for (int x = 0; x < kDT; ++x)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float2*>(xo + (slot * 16 + qr + 8 * i) * D + x * 8 + qc) =
                make_float2(o[x][2 * i], o[x][2 * i + 1]);
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kTreeThreads) : "memory");
      if (kg == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float M = m[i];
#pragma unroll
          for (int g = 0; g < KG - 1; ++g) M = fmaxf(M, xm[rg * (KG - 1) + g][qr + 8 * i]);
          const float f0 = m[i] == -INFINITY ? 0.f : ex2_approx(m[i] - M);
          float L = l[i] * f0;
#pragma unroll
          for (int x = 0; x < kDT; ++x) {
            o[x][2 * i] *= f0;
            o[x][2 * i + 1] *= f0;
          }
#pragma unroll
          for (int g = 0; g < KG - 1; ++g) {
            const int sl = rg * (KG - 1) + g;
            const float mg = xm[sl][qr + 8 * i];
            const float f = mg == -INFINITY ? 0.f : ex2_approx(mg - M);
            L = fmaf(f, xl[sl][qr + 8 * i], L);
#pragma unroll
            for (int x = 0; x < kDT; ++x) {
              const float2 y = *reinterpret_cast<const float2*>(xo + (sl * 16 + qr + 8 * i) * D + x * 8 + qc);
              o[x][2 * i] = fmaf(f, y.x, o[x][2 * i]);
              o[x][2 * i + 1] = fmaf(f, y.y, o[x][2 * i + 1]);
            }
          }
          m[i] = M;
          l[i] = L;
        }
      }
    }
    const bool failed = !ok || *static_cast<volatile uint32_t*>(&abort_flag) != 0u;
    if constexpr (kWin) {
      if (p.list.solo > 1) {
        if (kg == 0) {  // (into the places of the first part, which this thread has read)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int rr = rg * 16 + qr + 8 * i;
            if ((lane & 3) == 0) ml[rr] = make_float2(m[i], failed ? nan : l[i]);
#pragma unroll
            for (int x = 0; x < kDT; ++x)
              *reinterpret_cast<float2*>(xo + (rg * (KG - 1) * 16 + qr + 8 * i) * D + x * 8 + qc) =
                  make_float2(o[x][2 * i], o[x][2 * i + 1]);
          }
        }
        static_assert(RG == 1 || KG == 2, "row rr lies at rr · D");
        tree_cluster_join<D>(p, xo, D, ml, kRows, bh, sg.rb);
        return;
      }
    }
    if (kg == 0) {
      const size_t slot = static_cast<size_t>(blockIdx.x) + sg.entry;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!live[i]) continue;
        const bool none = l[i] == 0.f;
        const float inv = failed ? nan : (none ? 0.f : 1.f / l[i]);
        const float ls = failed ? nan : (none ? -INFINITY : (m[i] + log2f(l[i])) * 0.69314718055994530942f);
        const int r = r0 + 8 * i;
        if (sg.whole) {
          const size_t row = static_cast<size_t>(bh) * p.R + r;
          uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D + qc);
#pragma unroll
          for (int x = 0; x < kDT; ++x) dst[x * 4] = pack_bf16x2(o[x][2 * i] * inv, o[x][2 * i + 1] * inv);
          if ((lane & 3) == 0) p.lse[row] = ls;
        } else {
          const size_t row = slot * kRows + (r - sg.rb * kRows);
          float* dst = p.o_part + row * D + qc;
#pragma unroll
          for (int x = 0; x < kDT; ++x)
            *reinterpret_cast<float2*>(dst + x * 8) = make_float2(o[x][2 * i] * inv, o[x][2 * i + 1] * inv);
          if ((lane & 3) == 0) p.lse_part[row] = ls;
        }
      }
    }
    // the merge area may be rewritten once every row group has read it
    if constexpr (KG > 1) asm volatile("bar.sync 1, %0;" ::"n"(kTreeThreads) : "memory");
  }
}

// Joins the partials of the rows whose keys lie in several stretches (of `stretches`, the grid of
// the kernel before), and writes the rows of sequences without keys. A warp a row, a block eight rows
// of one list entry: its lanes read the partials' LSEs side by side, and kFlight partial rows are
// loaded before the first is used.
template <int D>
__global__ void __launch_bounds__(256, D == 64 ? 5 : 3)
    fa_tree_combine_kernel(const TreeParams p, int rows_log2, int stretches, unsigned groups) {
  constexpr int kV = D / 32;  // columns a lane
  constexpr int kFlight = 8;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const unsigned entries = static_cast<unsigned>(p.list.Hkv) * p.list.row_blocks;  // a sequence's
  for (unsigned x0 = blockIdx.x; x0 < groups; x0 += gridDim.x) {
    const unsigned entry = x0 >> (rows_log2 - 3);
    const int b = static_cast<int>(entry / entries);
    const unsigned rem = entry - b * entries, hk = rem / static_cast<unsigned>(p.list.row_blocks);
    const int in_block = static_cast<int>((x0 << 3) & ((1u << rows_log2) - 1u)) + (threadIdx.x >> 5);
    const int r = (static_cast<int>(rem - hk * p.list.row_blocks) << rows_log2) + in_block;
    if (r >= p.R) continue;
    const long long row = (static_cast<long long>(b) * p.list.Hkv + hk) * p.R + r;
    const int ctx = p.list.ctx_len[b];
    const int2 parts = p.list.parts[entry];
    __nv_bfloat16* dst = p.o + row * D + lane * kV;
    if (ctx < 0) {  // (no keys)
#pragma unroll
      for (int x = 0; x < kV; x += 2) *reinterpret_cast<uint32_t*>(dst + x) = 0u;
      if (lane == 0) p.lse[row] = -INFINITY;
      continue;
    }
    const int n = parts.y;
    if (n <= 1 || parts.x < 0 || n > stretches - parts.x) continue;  // (one part: written already)
    const size_t first = ((static_cast<size_t>(parts.x) + entry) << rows_log2) + in_block;
    float M = -INFINITY, L = 0.f, acc[kV];
#pragma unroll
    for (int x = 0; x < kV; ++x) acc[x] = 0.f;
    for (int c32 = 0; c32 < n; c32 += 32) {
      const int end = min(n, c32 + 32);
      const float ls = c32 + lane < n ? p.lse_part[first + (static_cast<size_t>(c32 + lane) << rows_log2)] : -INFINITY;
      float w = 0.f;
      for (int c = c32; c < end; c += kFlight) {
        float2 y[kFlight][kV / 2];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          const float* src = p.o_part + (first + (static_cast<size_t>(min(c + i, n - 1)) << rows_log2)) * D + lane * kV;
#pragma unroll
          for (int x = 0; x < kV / 2; ++x) y[i][x] = *reinterpret_cast<const float2*>(src + 2 * x);
        }
        if (c == c32) {  // (the first rows are on their way while the weights are made)
          float m = ls;
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
          m = fmaxf(m, M);
          const float mu = m == -INFINITY ? 0.f : m;
          const float f = ex2_approx((M - mu) * 1.4426950408889634f);  // 0 before the first
          w = ex2_approx((ls - mu) * 1.4426950408889634f);
          L *= f;
#pragma unroll
          for (int x = 0; x < kV; ++x) acc[x] *= f;
          M = m;
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          const float wi = __shfl_sync(0xffffffffu, w, (c + i) & 31);
          if (c + i >= n) continue;
          L += wi;
#pragma unroll
          for (int x = 0; x < kV / 2; ++x) {
            acc[2 * x] = fmaf(wi, y[i][x].x, acc[2 * x]);
            acc[2 * x + 1] = fmaf(wi, y[i][x].y, acc[2 * x + 1]);
          }
        }
      }
    }
    const float mu = M == -INFINITY ? 0.f : M;
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int x = 0; x < kV; x += 2)
      *reinterpret_cast<uint32_t*>(dst + x) = pack_bf16x2(acc[x] * inv, acc[x + 1] * inv);
    if (lane == 0) p.lse[row] = L == 0.f ? -INFINITY : mu + log2f(L) * 0.69314718055994530942f;
  }
}

}  // namespace fa
