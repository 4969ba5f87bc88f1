// Exact attention backward for GB300 (sm_103a): the gradients dQ, dK, dV of
// O = softmax(scale·QKᵀ [+causal mask])·V for an upstream gradient dO.
//
// The forward keeps only the row logsumexp LSE; the backward recomputes the scores and
// probabilities block by block from it instead of storing the T×T matrix, as step ④ of
// "手写 FlashAttention" (Hand-written FlashAttention, learn-llm.fim.ai ch. 19) and §2.2 of
// "FlashAttention 核心思路解析" (FlashAttention core ideas, ijyty.com: recompute per block,
// sum the per-block query gradients into the global gradient with atomic adds) describe.
// With D_i = Σ_c dO_ic·O_ic, for a query tile i and key tile j:
//
//   Pᵀ  = exp2(log2(e)·scale·K_j·Q_iᵀ − log2(e)·LSE_i)   (keys on TMEM lanes)
//   dPᵀ = V_j·dO_iᵀ
//   dSᵀ = Pᵀ ∘ (dPᵀ − D_i)
//   dV_j += Pᵀ·dO_i      dK_j += dSᵀ·Q_i      dQ_i += dS·K_j   (dK, dQ × scale at the end)
//
// Three kernels per call:
//   fa_bwd_prep_kernel   D_i, log2(e)·LSE_i (+∞ on padding rows, so their P is 0) and a
//                        zeroed fp32 dQ accumulator, all in the caller's workspace;
//   fa_bwd_main_kernel   one CTA per (128-key tile j, batch·head), walking the query tiles
//                        the mask leaves visible; dK_j, dV_j stay in TMEM for the whole walk,
//                        dQ_i partials are added to the accumulator;
//   fa_bwd_dq_kernel     accumulator × scale → bf16 dQ.
//
// Main kernel: kCWG compute warpgroups (4 at d = 64: 23 warps, 736 threads; 2 at d = 128:
// 16 warps, 512 threads), then:
//   warps 0 .. 4·kCWG−1   compute: warpgroup g owns query columns 32·g .. 32·g+31 of each
//                         tile (thread = key row); no exchange between warpgroups is needed,
//                         since P comes from the saved LSE, column by column
//   next 4 warps          dQ drain: TMEM → registers → shared memory → bulk reduce-adds
//                         into the fp32 accumulator by the TMA engine
//   next warp             score issuer: Sᵀ and dPᵀ MMAs (one elected thread); TMEM owner
//   next warp             gradient issuer: dV, dK and dQ MMAs (one elected thread); at
//                         d = 128 dV and dK only
//   next warp             TMA producer
//   last warp (d = 128)   dQ issuer: the dQᵀ MMAs, from the fourth sub-partition (measured
//                         4 % faster there; at d = 64 a separate dQ issuer was 2 % slower)
// (More compute warps hide more of the latency of each tile's chain of TMEM loads and
// stores; at d = 64 four warpgroups of 32 columns measured 4 % faster than two of 64.)
// Two issuers, because MMAs into different accumulators are not ordered with one another
// and a single issuer blocked on one barrier would hold back independent work: the score
// issuer starts Sᵀ of the next tile as soon as the compute warps have read the current
// one into registers, while the gradient issuer is still waiting for this tile's Pᵀ/dSᵀ.
// Pᵀ and dSᵀ are rounded to bf16, as operands beside dO, Q and K must be; P and dP − D are fp32 until then (windows of
// 200 on documents, d = 64: dq, dk, dv off by 2.40e-3, 2.37e-3 and 2.28e-3 of their norms, where 64 bits with these two
// roundings and the results' are by 2.36e-3, 2.34e-3 and 2.28e-3, and with the results' alone by 1.65e-3).
// Pᵀ goes to tensor memory (bf16 pairs, the A operand of the dV MMA). dSᵀ is written to
// shared memory as bf16 in the 128-byte-swizzled layout a TMA load would produce
// ([key row][64 query columns] boxes, double-buffered). The same bytes serve as the
// K-major A operand of dK (rows = keys) and the MN-major A operand of dQ (queries on M),
// so no transpose is ever materialised.
// Tensor memory (D = 64): [0,128) Sᵀ, [128,256) dPᵀ, [256,320) dV, [320,384) dK,
// [384,448) dQ, [448,512) Pᵀ (bf16 pairs).
#pragma once

#include "fa_mod.cuh"
#include "sm103.cuh"

// Timeline hooks: compiled out unless a tracing build defines FA_TRACE(tag, step).
#ifndef FA_TRACE
#define FA_TRACE(tag, step) ((void)0)
#endif

namespace fa {


// Tile shapes. Keys are always in 128-row tiles (the TMEM lanes of Sᵀ, dPᵀ, dV and dK).
// Query tiles have kBQ rows: 128 at d = 64; 64 at d = 128, where 128-column Sᵀ, dPᵀ, dV and
// dK would already fill the 512 TMEM columns. With 64-query tiles every product keeps
// M = 128: dQ is then made transposed, dQᵀ = Kᵀ·dSᵀ (head dims on TMEM lanes, N = 64).
template <int D, int MOD = 0>
struct BwdCfg {
  static_assert(D == 64 || D == 128, "head dim");
  static constexpr int kBQ = (D == 64) ? 128 : 64;    // query rows per tile
  // Compute warpgroups, each owning kNC query columns of a tile (32 at either head dim).
  // (4 at d = 128, 16 columns each: 3 to 5 % slower; but where scores are capped, whose
  // arithmetic two warpgroups cannot hide, faster: B2 H16 T4096 d128 causal, cap 30, 430 -> 410 µs,
  // with a distance bias too 495 -> 440; the bias alone 392 -> 395)
  static constexpr int kCWG = (D == 64 || (MOD & kModCap) != 0) ? 4 : 2;
  static constexpr int kNC = kBQ / kCWG;
  static constexpr int kComputeWarps = 4 * kCWG;
  // Warp roles after the compute warps: 4 dQ drain warps, score issuer, gradient issuer,
  // TMA producer.
  static constexpr int kDrainWarp0 = kComputeWarps;
  static constexpr int kScoreWarp = kDrainWarp0 + 4;
  static constexpr int kGradWarp = kScoreWarp + 1;
  static constexpr int kLoadWarp = kScoreWarp + 2;
  static constexpr bool kSplitQ = (D == 128);  // dQ products issued by a warp of their own
  static constexpr int kGradQWarp = kScoreWarp + 3;
  static constexpr int kThreads = (kSplitQ ? kGradQWarp + 1 : kLoadWarp + 1) * 32;
  static constexpr int kBox = 128 * 64 * 2;           // 128 rows × 64 bf16 columns = 16 KB
  static constexpr int kQBox = kBQ * 64 * 2;          // kBQ rows × 64 columns
  static constexpr int kKVTile = 128 * D * 2;         // a K or V tile
  static constexpr int kQTile = kBQ * D * 2;          // a Q or dO tile
  static constexpr int kK = 0;
  static constexpr int kV = kK + kKVTile;
  static constexpr int kStages = 3;                   // (Q_i, dO_i) ring depth
  static constexpr int kStage0 = kV + kKVTile;        // stage s: Q at +0, dO at +kQTile
  static constexpr int kStageBytes = 2 * kQTile;
  static constexpr int kDS = kStage0 + kStages * kStageBytes;  // dSᵀ: 2 buffers
  static constexpr int kDSBytes = 128 * kBQ * 2;      // [128 keys][kBQ queries] bf16, 64-col boxes
  // per stage: −lse2[kBQ] then D[kBQ], and (MOD) the rows' visible intervals [lo, hi)
  static constexpr int kVecBytes = (MOD ? 4 : 2) * kBQ * 4;
  static constexpr int kVec = kDS + 2 * kDSBytes;
  // Each dQ drain warp stages 16 of its TMEM columns for its 32 lanes (2 KB) for a bulk
  // reduce-add, two buffers per warp.
  static constexpr int kDQChunk = 32 * 16 * 4;
  static constexpr int kDQStage = kVec + kStages * kVecBytes;
  static constexpr int kBar = kDQStage + 4 * 2 * kDQChunk;
  static constexpr int kSmemBytes = kBar + 256 + 1024;  // barriers + 1 KB alignment slack
  // Tensor memory: Sᵀ, dPᵀ (kBQ columns each), dV, dK (D each), dQ (D columns at d = 64,
  // dQᵀ with kBQ columns at d = 128), Pᵀ as bf16 pairs (kBQ/2 columns).
  static constexpr uint32_t kColS = 0, kColDP = kBQ, kColDV = 2 * kBQ, kColDK = 2 * kBQ + D;
  static constexpr uint32_t kColDQ = 2 * kBQ + 2 * D;
  static constexpr uint32_t kColP = kColDQ + ((D == 64) ? D : kBQ);
  static_assert(kColP + kBQ / 2 <= 512, "tensor memory");
  static_assert(kSmemBytes <= 232448, "shared memory");
};

struct BwdBars {
  uint64_t kv_full;     // K_j, V_j landed
  uint64_t q_full[3];   // Q_i, dO_i, lse2_i, D_i landed in a stage
  uint64_t q_empty[3];  // both issuers' MMAs reading that stage are done (2 arrivals)
  uint64_t s_full;      // Sᵀ in TMEM
  uint64_t s_free;      // Sᵀ read into registers (8 compute warps)
  uint64_t dp_full;     // dPᵀ in TMEM
  uint64_t dp_free;     // dPᵀ read into registers (8 compute warps)
  uint64_t p_full;      // Pᵀ stored in TMEM (8 compute warps)
  uint64_t p_free;      // dV MMA done with Pᵀ
  uint64_t ds_full[2];  // dSᵀ buffer in shared memory (8 compute warps)
  uint64_t ds_free[2];  // dK and dQ MMAs done with that buffer
  uint64_t dq_full;     // a dQ partial in TMEM
  uint64_t dq_free;     // drained (4 drain warps)
  uint64_t score_done;  // every MMA of the score issuer done
  uint64_t grad_done;   // every MMA of the gradient issuer done: dK, dV final
  uint32_t tmem_base;
  uint32_t abort;
  uint32_t whole[3];    // MOD: 1: the stage's rows all see every key of this CTA's tile; 2: some are padding
};
static_assert(sizeof(BwdBars) <= 256, "barrier block");

// Modified scores (MOD instantiations; see fa_mod.cuh). K, V, dK and dV then have one head for
// every `group` query heads: the CTA of a key tile walks the query tiles of all of them, so a
// shared head's gradient is summed in its accumulators, with no second pass. Where that leaves too
// few CTAs to share out evenly, a group is cut into `parts`, each part's sum goes out in fp32, and
// fa_bwd_sum_kernel adds the parts in order (no atomics: the same bits every time).
struct BwdModParams {
  const int2* rows;     // [B][T_pad] visible key interval of each query row, or null
  const int4* units;    // [B][n_kt] (key tile, first 128-row query tile, past the last,
                        //   2 · first tile with padding + whether the key tile has any)
  const int2* whole;    // [B][n_kt] (largest lo, smallest hi) over a tile's 128 rows: hi is 0 with padding
  const float* slopes;  // [H]
  float* part_out;      // parts > 1: [2][parts][B·Hkv][T][D], dK (scaled) then dV
  int Hkv;              // key heads
  int group;            // query heads per key head
  int parts;            // parts of a group (BH then counts B·Hkv·parts)
  CapFactors cap;       // (CAP)
  int causal;           // without rows
  // SINK: `units` are [B][n_rec][2], the second (slot of a cut walk's piece or −1, whether the key tile has
  // sinks beyond a window, 0, 0); the pieces' sums go to slots and fa_bwd_pieces_kernel adds them in order.
  const int2* sink_rows;  // [B][T_pad] a row's visible sinks, an interval in front of its rows entry
  const int4* cuts;     // [B][n_cut] the cut key tiles: (tile, first slot, slots, 0)
  float* piece_out;     // [2][B·Hkv·parts][n_slots][128][D], dK (scaled) then dV
  int n_rec;            // walks a key head's part (n_kt, or with pieces)
  int n_cut, n_slots;
};

struct BwdParams {
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  const float* lse2;   // [BH][T_pad] −log2(e)·LSE, −∞ on padding rows
  const float* dvec;   // [BH][T_pad] D_i, 0 on padding rows
  float* dq_acc;       // fp32 dQ accumulator (unscaled), layout of dq_acc_offset
  int* status;
  int T;
  int T_pad;           // ceil(T / 128) · 128
  int BH;
  int n_qt;            // T_pad / kBQ query tiles
  int n_kt;            // T_pad / 128 key tiles
  int head_group;      // heads whose units are interleaved (see the unit order)
  float scale;
  float scale_log2;    // scale · log2(e)
  uint64_t timeout_ns;
  uint32_t flags;
  BwdModParams mod;    // MOD kernels only (BH then counts B·Hkv)
};

constexpr uint32_t kBwdFlagStarveQ = 1u;  // FA_FLAG_TEST_STARVE_Q

// dQ accumulator layouts.
// d = 64 (thread = query row r of a 128-row tile): [bh][tile][r/32][d/4][32 rows][4 columns],
//   so the 32 rows of one drain warp and 16 consecutive columns are 2 KB in one piece (one
//   bulk reduce-add); dq_acc_offset(bh, i, n_qt, c4, r, d) is query row r, columns
//   4·c4 .. 4·c4+3.
// d = 128 (dQᵀ: thread = head dim c of a 64-query tile): [bh][tile][c/32][16][32 dims][4 rows],
//   so the 32 dims of one drain warp and 16 consecutive query rows are 2 KB in one piece;
//   dq_acc_offset_t(bh, i, n_qt, g, c) is head dim c of query rows 4·g .. 4·g+3.
// tmem_load_cols (below), and the largest magnitude among the N (16 or 32) columns.
template <int N>
__device__ __forceinline__ float tmem_load_cols_absmax(uint32_t taddr, uint32_t* r) {
  static_assert(N == 16 || N == 32, "one load");
  float m;
  if constexpr (N == 16) tmem_ld16_absmax(taddr, r, &m);
  else tmem_ld32_max<true>(taddr, r, &m);
  tmem_ld_wait();
  if constexpr (N == 16) reg_fence16(r);
  else reg_fence32(r);
  asm volatile("" : "+f"(m));
  return m;
}
// N consecutive TMEM columns (N = 16 or a multiple of 32) of the warp's 32 lanes into r,
// with one wait for all of them.
template <int N>
__device__ __forceinline__ void tmem_load_cols(uint32_t taddr, uint32_t* r) {
  if constexpr (N == 16) {
    tmem_ld16(taddr, r);
    tmem_ld_wait();
    reg_fence16(r);
  } else {
#pragma unroll
    for (int h = 0; h < N / 32; ++h) tmem_ld32(taddr + h * 32, r + h * 32);
    tmem_ld_wait();
#pragma unroll
    for (int h = 0; h < N / 32; ++h) reg_fence32(r + h * 32);
  }
}

__host__ __device__ __forceinline__ size_t dq_acc_offset(int bh, int i, int n_qt, int c4, int r,
                                                         int d) {
  return (((((size_t)bh * n_qt + i) * 4u + (unsigned)(r >> 5)) * (size_t)(d / 4) + c4) * 32u +
          (unsigned)(r & 31)) * 4u;
}
__host__ __device__ __forceinline__ size_t dq_acc_offset_t(int bh, int i, int n_qt, int g, int c) {
  return (((((size_t)bh * n_qt + i) * 4u + (unsigned)(c >> 5)) * 16u + g) * 32u +
          (unsigned)(c & 31)) * 4u;
}

// ------------------------------------------------------------------------------------
// Preprocessing: D_i = Σ_c dO_ic·O_ic, lse2_i = −log2(e)·LSE_i (negated: the main kernel adds
// it in a packed fp32x2 FMA); zero the dQ accumulator.
// D/8 consecutive lanes share a row, each reading 8 columns (16 bytes) of O and dO.
// ------------------------------------------------------------------------------------
// MOD: a row that saw no key (lse = −∞) gets −∞ and D = 0, so that its P and dS are 0 whatever
// its o and dO hold; D takes o and, where it is given, what o's rounding left out.
template <int D, bool MOD = false>
__global__ void __launch_bounds__(256) fa_bwd_prep_kernel(const __nv_bfloat16* __restrict__ o,
                                                          const __nv_bfloat16* __restrict__ dout,
                                                          const float* __restrict__ lse,
                                                          float* __restrict__ lse2,
                                                          float* __restrict__ dvec,
                                                          float* __restrict__ dq_acc, int T,
                                                          int T_pad, int BH,
                                                          const __nv_bfloat16* __restrict__ rest = nullptr) {
  constexpr int L = D / 8;
  pdl_wait();  // launched as a programmatic dependent (o, dO and lse may come from the previous kernel)
  pdl_launch_dependents();
  const size_t nrows = (size_t)BH * T_pad;
  const size_t tid = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  const size_t stride = (size_t)gridDim.x * blockDim.x;
  // T_pad is a multiple of 128, so nrows·L is a multiple of 32 and every lane of a warp
  // runs the same number of iterations (the shuffles below need the whole warp).
  for (size_t idx = tid; idx < nrows * L; idx += stride) {
    const size_t row = idx / L;
    const int c = static_cast<int>(idx % L);
    const int bh = static_cast<int>(row / T_pad);
    const int t = static_cast<int>(row % T_pad);
    float acc = 0.f;
    if (t < T) {
      const size_t off = ((size_t)bh * T + t) * D + (size_t)c * 8;
      const uint4 a = *reinterpret_cast<const uint4*>(o + off);
      const uint4 b = *reinterpret_cast<const uint4*>(dout + off);
      const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 fa2 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&av[e]));
        const float2 fb2 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&bv[e]));
        acc = fmaf(fa2.x, fb2.x, acc);
        acc = fmaf(fa2.y, fb2.y, acc);
      }
      if (MOD && rest) {
        const uint4 r = *reinterpret_cast<const uint4*>(rest + off);
        const uint32_t rv[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 fr2 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&rv[e]));
          const float2 fb2 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&bv[e]));
          acc = fmaf(fr2.x, fb2.x, acc);
          acc = fmaf(fr2.y, fb2.y, acc);
        }
      }
    }
#pragma unroll
    for (int w = L / 2; w > 0; w >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, w);
    if (MOD) {
      if (c == 0) {
        const float ls = (t < T) ? lse[(size_t)bh * T + t] : __int_as_float(0xff800000);
        const bool none = ls == __int_as_float(0xff800000);
        dvec[row] = none ? 0.f : acc;
        lse2[row] = none ? ls : ls * -1.4426950408889634f;
      }
    } else if (c == 0) {
      dvec[row] = (t < T) ? acc : 0.f;
      lse2[row] = (t < T) ? lse[(size_t)bh * T + t] * -1.4426950408889634f : __int_as_float(0xff800000);
    }
  }
  float4* acc4 = reinterpret_cast<float4*>(dq_acc);
  const size_t n4 = nrows * (D / 4);
  for (size_t x = tid; x < n4; x += stride) acc4[x] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// ------------------------------------------------------------------------------------
// dQ = scale · accumulator, as bf16 rows.
// d = 64: one thread per (tile, 8 columns, row). d = 128: one thread per (64-row tile,
// group of 4 rows, 8 head dims), writing 4 rows × 8 columns.
// ------------------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) fa_bwd_dq_kernel(const float* __restrict__ dq_acc,
                                                        __nv_bfloat16* __restrict__ dq, int T,
                                                        int n_qt, int BH, float scale) {
  constexpr int C8 = D / 8;
  pdl_wait();  // launched as a programmatic dependent of the main kernel (dq_acc)
  pdl_launch_dependents();
  const size_t stride = (size_t)gridDim.x * blockDim.x;
  if constexpr (D == 64) {
    const size_t total = (size_t)BH * n_qt * C8 * 128;
    for (size_t idx = (size_t)blockIdx.x * blockDim.x + threadIdx.x; idx < total; idx += stride) {
      const int r = static_cast<int>(idx % 128);
      const size_t rest = idx / 128;
      const int c8 = static_cast<int>(rest % C8);
      const size_t tile = rest / C8;  // bh · n_qt + i
      const int i = static_cast<int>(tile % n_qt);
      const int bh = static_cast<int>(tile / n_qt);
      const int t = i * 128 + r;
      if (t >= T) continue;
      const float4 a = *reinterpret_cast<const float4*>(dq_acc + dq_acc_offset(bh, i, n_qt, 2 * c8, r, D));
      const float4 b = *reinterpret_cast<const float4*>(dq_acc + dq_acc_offset(bh, i, n_qt, 2 * c8 + 1, r, D));
      uint4 out;
      out.x = pack_bf16x2(a.x * scale, a.y * scale);
      out.y = pack_bf16x2(a.z * scale, a.w * scale);
      out.z = pack_bf16x2(b.x * scale, b.y * scale);
      out.w = pack_bf16x2(b.z * scale, b.w * scale);
      *reinterpret_cast<uint4*>(dq + ((size_t)bh * T + t) * D + (size_t)c8 * 8) = out;
    }
  } else {
    const size_t total = (size_t)BH * n_qt * 16 * C8;
    for (size_t idx = (size_t)blockIdx.x * blockDim.x + threadIdx.x; idx < total; idx += stride) {
      const int c8 = static_cast<int>(idx % C8);
      const size_t rest = idx / C8;
      const int g = static_cast<int>(rest % 16);
      const size_t tile = rest / 16;
      const int i = static_cast<int>(tile % n_qt);
      const int bh = static_cast<int>(tile / n_qt);
      float4 col[8];  // head dims c8·8 .. c8·8+7, each holding rows 4g .. 4g+3
#pragma unroll
      for (int e = 0; e < 8; ++e)
        col[e] = *reinterpret_cast<const float4*>(dq_acc + dq_acc_offset_t(bh, i, n_qt, g, c8 * 8 + e));
#pragma unroll
      for (int rr = 0; rr < 4; ++rr) {
        const int t = i * 64 + 4 * g + rr;
        if (t >= T) break;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 cv = col[e];
          y[e] = (rr == 0 ? cv.x : rr == 1 ? cv.y : rr == 2 ? cv.z : cv.w) * scale;
        }
        uint4 out;
        out.x = pack_bf16x2(y[0], y[1]);
        out.y = pack_bf16x2(y[2], y[3]);
        out.z = pack_bf16x2(y[4], y[5]);
        out.w = pack_bf16x2(y[6], y[7]);
        *reinterpret_cast<uint4*>(dq + ((size_t)bh * T + t) * D + (size_t)c8 * 8) = out;
      }
    }
  }
}

// dK and dV = the sums of their parts' fp32 rows, as bf16: part_out is [2][parts][rows][D], 8 values
// a thread and step. (A template, so that only the files that launch it hold it.)
template <int D>
__global__ void __launch_bounds__(256) fa_bwd_sum_kernel(const float* __restrict__ part_out,
                                                         __nv_bfloat16* __restrict__ dk,
                                                         __nv_bfloat16* __restrict__ dv, size_t rows, int parts) {
  pdl_wait();
  pdl_launch_dependents();
  const size_t n = rows * D;
  const size_t stride = (size_t)gridDim.x * blockDim.x * 8;
  for (size_t x = ((size_t)blockIdx.x * blockDim.x + threadIdx.x) * 8; x < 2 * n; x += stride) {
    const bool is_dv = x >= n;
    const size_t e = is_dv ? x - n : x;
    const float* src = part_out + (is_dv ? (size_t)parts * n : 0) + e;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
      const float4 u = *reinterpret_cast<const float4*>(src + (size_t)s * n);
      const float4 v = *reinterpret_cast<const float4*>(src + (size_t)s * n + 4);
      a.x += u.x; a.y += u.y; a.z += u.z; a.w += u.w;
      b.x += v.x; b.y += v.y; b.z += v.z; b.w += v.w;
    }
    *reinterpret_cast<uint4*>((is_dv ? dv : dk) + e) =
        make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w));
  }
}

// dK and dV of the key tiles whose walks were cut: their pieces' fp32 rows, of every part in order, as
// bf16. A block takes kPieceRows rows of a cut tile of a key head, a thread 8 values of one of its rows
// (blockIdx.x = (key head · n_cut + cut) · 128 / kPieceRows + which rows): the pieces are read one
// behind the other, so what counts is that no thread has more than one such chain.
template <int D>
constexpr int kPieceRows = 2048 / D / 2;  // (dK and dV, 256 threads of 8 values)
template <int D>
__global__ void __launch_bounds__(256) fa_bwd_pieces_kernel(const float* __restrict__ piece_out,
                                                            const int4* __restrict__ cuts,
                                                            __nv_bfloat16* __restrict__ dk,
                                                            __nv_bfloat16* __restrict__ dv, int Hkv, int BHkv, int T,
                                                            int n_cut, int n_slots, int parts) {
  constexpr int kBlocks = 128 / kPieceRows<D>;
  pdl_wait();
  pdl_launch_dependents();
  const int x = static_cast<int>(blockIdx.x / kBlocks), bh = x / n_cut;
  const int4 cut = cuts[(size_t)(bh / Hkv) * n_cut + (x - bh * n_cut)];
  const bool is_dv = threadIdx.x >= 128;
  const int e = threadIdx.x & 127, c = e % (D / 8) * 8;
  const int r = static_cast<int>(blockIdx.x % kBlocks) * kPieceRows<D> + e / (D / 8), key = cut.x * 128 + r;
  if (cut.z == 0 || key >= T) return;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
  for (int s = 0; s < parts; ++s) {
    const float* src = piece_out +
        ((((is_dv ? (size_t)BHkv * parts : 0) + (size_t)bh * parts + s) * n_slots + cut.y) * 128 + r) * D + c;
#pragma unroll 8
    for (int i = 0; i < cut.z; ++i) {
      const float4 u = *reinterpret_cast<const float4*>(src + (size_t)i * 128 * D);
      const float4 v = *reinterpret_cast<const float4*>(src + (size_t)i * 128 * D + 4);
      a.x += u.x; a.y += u.y; a.z += u.z; a.w += u.w;
      b.x += v.x; b.y += v.y; b.z += v.z; b.w += v.w;
    }
  }
  *reinterpret_cast<uint4*>((is_dv ? dv : dk) + ((size_t)bh * T + key) * D + c) =
      make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w));
}

// ------------------------------------------------------------------------------------
// Main kernel.
// ------------------------------------------------------------------------------------
// Stores 8 fp32 values of one row as bf16 into a 128-byte-swizzled box: 16-byte chunk
// `ch` of row `r` sits at chunk position ch ^ (r mod 8), as a TMA load would place it.
__device__ __forceinline__ void st_row_chunk_sw128(uint32_t box, int r, int ch, const float* x) {
  st_shared_v4(box + static_cast<uint32_t>(r) * 128u + (static_cast<uint32_t>(ch ^ (r & 7)) << 4),
               pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
               pack_bf16x2(x[6], x[7]));
}

// What a CTA walks: key tile j of key head bh, against the query tiles i0 … i0 + n_i − 1 of each of
// its query heads (b·h numbers from q0h on), n steps in all.
struct BwdWalk {
  int j, bh, i0, n;
  int n_i, q0h;  // MOD (dense: n and bh)
  int h0;        // the first query head's number within its sequence
  int part;      // which part of the key head's query heads
  int pad0;      // the first query tile with padding
  bool key_pad;  // the key tile has padding
  int slot;      // SINK: where a piece's sums go, or −1
  bool sinks;    // SINK: the key tile has sinks that are seen from beyond a window
};

// pos, head: the CTA's place in the unit order.
template <int D, bool CAUSAL, int MOD>
__device__ __forceinline__ BwdWalk bwd_walk(const BwdParams& p, int pos, int head) {
  constexpr int kBQ = BwdCfg<D, MOD>::kBQ, kPer = 128 / kBQ;  // query tiles in 128 rows
  BwdWalk w;
  w.j = pos;
  w.bh = w.q0h = head;
  w.i0 = CAUSAL ? (w.j * 128) / kBQ : 0;
  w.n = w.n_i = p.n_qt - w.i0;
  w.h0 = w.part = 0;
  w.pad0 = p.n_qt;
  w.key_pad = false;
  w.slot = -1;
  w.sinks = false;
  if constexpr (MOD != 0) {
    const int heads = p.mod.group / p.mod.parts;
    w.bh = head / p.mod.parts;
    w.part = head - w.bh * p.mod.parts;
    const int b = w.bh / p.mod.Hkv;
    w.h0 = (w.bh - b * p.mod.Hkv) * p.mod.group + w.part * heads;
    w.q0h = w.bh * p.mod.group + w.part * heads;
    if (p.mod.units) {
      constexpr bool kSink = (MOD & kModSink) != 0;
      const int4* at = p.mod.units + (kSink ? ((size_t)b * p.mod.n_rec + pos) * 2 : (size_t)b * p.n_kt + pos);
      const int4 rec = __ldg(at);
      if constexpr (kSink) {
        const int4 more = __ldg(at + 1);
        w.slot = more.x;
        w.sinks = more.y != 0;
      }
      w.j = rec.x;
      w.i0 = rec.y * kPer;
      w.n_i = max(0, rec.z * kPer - w.i0);
      w.pad0 = (rec.w >> 1) * kPer;
      w.key_pad = (rec.w & 1) != 0;
    } else if (p.mod.causal) {
      w.i0 = pos * kPer;
      w.n_i = p.n_qt - w.i0;
    }
    w.n = w.n_i * heads;
  }
  return w;
}

// The roles' waits. MOD calls the slow path instead of having it at every wait: the steps are longer
// there, and the instructions of all roles together no longer fit where they are fetched from without
// a pause (B2 H16 T4096 d128: plain 452 -> 377 µs, capped 506 -> 424; d64 H12 capped 228 -> 202).
template <int MOD>
__device__ __forceinline__ bool bwd_wait(uint64_t* bar, uint32_t parity, const WaitCtl& w) {
  if constexpr (MOD != 0) return mbar_wait_warp(bar, parity, w);
  else return mbar_wait_warp_inl(bar, parity, w);
}

// RAGGED (dense, not causal): T is no multiple of 128, and the last key tile's keys behind the end are
// masked: their rows are loaded as zeros, and a score of 0 may be so far above every other of a query
// that its P is infinite. (Causal masks them with the diagonal, MOD with the intervals' ends. A kernel
// of its own, since the branch costs the step 3 %, B2 H16 T4000 d128 641 -> 664 µs; B2 H12 d64 346 -> 349.)
template <int D, bool CAUSAL, int MOD = 0, bool RAGGED = false>
__global__ void __launch_bounds__(BwdCfg<D, MOD>::kThreads, 1)
    fa_bwd_main_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                       const BwdParams p) {
  using C = BwdCfg<D, MOD>;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  BwdBars* bars = reinterpret_cast<BwdBars*>(sm + C::kBar);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // Unit order: heads in groups of head_group, small enough that a group's Q, dO and dQ
  // accumulator stay in L2 while its CTAs run; within a group, heaviest units first (under
  // the causal mask key tile j sees the query tiles from the one holding query 128·j on),
  // all heads at one j together.
  constexpr bool kSink = (MOD & kModSink) != 0;
  const int per_group = p.head_group * (kSink ? p.mod.n_rec : p.n_kt);
  const int grp = blockIdx.x / per_group;
  const int within = blockIdx.x - grp * per_group;
  const int gsize = min(p.head_group, p.BH - grp * p.head_group);
  const int u_pos = within / gsize, u_head = grp * p.head_group + within % gsize;
  // (MOD reads its walk from memory, after the wait for the kernel before)
  const BwdWalk dense = bwd_walk<D, CAUSAL, 0>(p, u_pos, u_head);

  if (threadIdx.x == 0) {
    mbar_init(&bars->kv_full, 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bars->q_full[s], 1);
      mbar_init(&bars->q_empty[s], 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->ds_full[s], C::kComputeWarps);
      mbar_init(&bars->ds_free[s], C::kSplitQ ? 2 : 1);  // after dK (and dQ, if split)
    }
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->s_free, C::kComputeWarps);
    mbar_init(&bars->dp_full, 1);
    mbar_init(&bars->dp_free, C::kComputeWarps);
    mbar_init(&bars->p_full, C::kComputeWarps);
    mbar_init(&bars->p_free, 1);
    mbar_init(&bars->dq_full, 1);
    mbar_init(&bars->dq_free, 4);
    mbar_init(&bars->score_done, 1);
    mbar_init(&bars->grad_done, C::kSplitQ ? 2 : 1);
    bars->abort = 0u;
    fence_mbar_init();
  }
  if (warp == C::kScoreWarp) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  // Launched as a programmatic dependent of the prep kernel: the set-up above overlapped its
  // tail; its outputs (D, log2e·LSE, the zeroed dQ accumulator) are read only after this.
  // (No early trigger for the dQ conversion: letting it be scheduled during this grid's
  // last wave measured 5 % slower at d = 128.)
  pdl_wait();
  const BwdWalk wk = MOD != 0 ? bwd_walk<D, CAUSAL, MOD>(p, u_pos, u_head) : dense;
  const int j = wk.j, bh = wk.bh, i0 = wk.i0, n = wk.n;
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl wc{&bars->abort, p.status, p.timeout_ns};
  const WaitCtl drain_wc = drain_ctl(p.timeout_ns);
  const uint32_t sbase = smem_u32(sm);
  auto q_s = [&](int st) { return sbase + C::kStage0 + st * C::kStageBytes; };
  auto do_s = [&](int st) { return q_s(st) + C::kQTile; };
  // Operand steps: K-major, 16 columns = 32 bytes inside a 64-column box, next box `box`
  // bytes on; MN-major, 16 rows = 2 KB, boxes along M/N `box` bytes apart (leading byte
  // offset). K/V tiles and dSᵀ have 128-row boxes (16 KB); Q/dO tiles kBQ-row boxes.
  auto kmaj = [&](uint32_t base, int kk, uint32_t box) {
    return sdesc_sw128(base + (kk >> 2) * box + (kk & 3) * 32, 16, 1024);
  };
  auto mnmaj = [&](uint32_t base, int kk, uint32_t box) {
    return sdesc_sw128(base + kk * 2048, box, 1024);
  };
  // End of every role (each calls it last, so that no code is shared between warpgroups
  // that run with different register budgets). Nothing may be in flight on the tensor
  // core when TMEM is released.
  auto teardown = [&]() {
    if (warp == C::kScoreWarp) {
      bwd_wait<MOD>(&bars->score_done, 0, drain_wc);
      bwd_wait<MOD>(&bars->grad_done, 0, drain_wc);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == C::kScoreWarp) {
      tc_fence_after_sync();
      tmem_dealloc(tmem, 512);
    }
  };

  if (warp >= C::kScoreWarp) {
  if (warp == C::kLoadWarp) {
    // ---------------------------------------------------------------- TMA producer
    int last_t[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) last_t[s] = -1;
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_do);
      mbar_arrive_expect_tx(&bars->kv_full, 2 * C::kKVTile);
#pragma unroll
      for (int b = 0; b < D / 64; ++b) {
        tma_load_3d(sm + C::kK + b * C::kBox, &tm_k, &bars->kv_full, b * 64, j * 128, bh);
        tma_load_3d(sm + C::kV + b * C::kBox, &tm_v, &bars->kv_full, b * 64, j * 128, bh);
      }
    }
    __syncwarp();
    const bool starve = (p.flags & kBwdFlagStarveQ) != 0u;
    int ti = 0, hg = 0;  // MOD: the step's query tile within the walk, its head within the group
    for (int t = 0, st = 0, ph = 0; t < n && !starve; ++t) {
      if (t >= NS && !bwd_wait<MOD>(&bars->q_empty[st], ph ^ 1, wc)) break;
      FA_TRACE(30, t);
      int i = i0 + t, bq = bh;  // query tile and (b·h) of this step
      if constexpr (MOD != 0) {
        i = i0 + ti;
        bq = wk.q0h + hg;
        if (++ti == wk.n_i) {
          ti = 0;
          ++hg;
        }
      }
      if (lane == 0) {
        uint8_t* stage = sm + C::kStage0 + st * C::kStageBytes;
        float* vec = reinterpret_cast<float*>(sm + C::kVec + st * C::kVecBytes);
        if constexpr (MOD != 0) {
          uint32_t vec_bytes = C::kVecBytes / 2;
          if (p.mod.rows) {
            const int b = bh / p.mod.Hkv;
            const int2 w = __ldg(p.mod.whole + (size_t)b * p.n_kt + i * C::kBQ / 128);
            bars->whole[st] = (w.x <= j * 128 && w.y >= j * 128 + 128) ? 1u : w.y == 0 ? 2u : 0u;
            vec_bytes = C::kVecBytes;
          }
          mbar_arrive_expect_tx(&bars->q_full[st], 2 * C::kQTile + vec_bytes);
          if (p.mod.rows)
            bulk_load(vec + 2 * C::kBQ,
                      p.mod.rows + (size_t)(bh / p.mod.Hkv) * p.T_pad + (size_t)i * C::kBQ,
                      C::kBQ * 8, &bars->q_full[st]);
        } else {
          mbar_arrive_expect_tx(&bars->q_full[st], 2 * C::kQTile + C::kVecBytes);
        }
#pragma unroll
        for (int b = 0; b < D / 64; ++b) {
          tma_load_3d(stage + b * C::kQBox, &tm_q, &bars->q_full[st], b * 64, i * C::kBQ, bq);
          tma_load_3d(stage + C::kQTile + b * C::kQBox, &tm_do, &bars->q_full[st], b * 64,
                      i * C::kBQ, bq);
        }
        const size_t row0 = (size_t)bq * p.T_pad + (size_t)i * C::kBQ;
        bulk_load(vec, p.lse2 + row0, C::kBQ * 4, &bars->q_full[st]);
        bulk_load(vec + C::kBQ, p.dvec + row0, C::kBQ * 4, &bars->q_full[st]);
      }
      last_t[st] = t;
      __syncwarp();
      if (++st == NS) { st = 0; ph ^= 1; }
    }
    // No copy may still be in flight when the CTA exits.
    bwd_wait<MOD>(&bars->kv_full, 0, drain_wc);
#pragma unroll
    for (int s = 0; s < NS; ++s)
      if (last_t[s] >= 0) bwd_wait<MOD>(&bars->q_full[s], (last_t[s] / NS) & 1, drain_wc);
  } else if (warp == C::kScoreWarp) {
    // ---------------------------------------------------------------- score issuer
    constexpr uint32_t kIdS = idesc_bf16(128, C::kBQ, false);  // Sᵀ = K·Qᵀ, dPᵀ = V·dOᵀ
    const uint32_t k_s = sbase + C::kK, v_s = sbase + C::kV;
    // MOD: rows of padding are zeroed in K, V, Q and dO here, before the first product that reads
    // them (every other reader comes after it).
    bool ok = bwd_wait<MOD>(&bars->kv_full, 0, wc);
    if constexpr (MOD != 0) {
      if (ok && wk.key_pad) {
        const int2* iv = p.mod.rows + (size_t)(bh / p.mod.Hkv) * p.T_pad + (size_t)j * 128;
        zero_padding(k_s, 2 * (D / 64), C::kBox, 128, iv);  // (K, and V behind it)
      }
    }
    int ti = 0;  // MOD: the step's query tile within the walk
    for (int t = 0, st = 0, ph = 0; t < n && ok; ++t) {
      if (!(ok = bwd_wait<MOD>(&bars->q_full[st], ph, wc))) break;
      if constexpr (MOD != 0) {
        const int i = i0 + ti;
        if (++ti == wk.n_i) ti = 0;
        if (i >= wk.pad0 && bars->whole[st] == 2u) {
          const int2* iv = reinterpret_cast<const int2*>(sm + C::kVec + st * C::kVecBytes + 2 * C::kBQ * 4);
          zero_padding(q_s(st), 2 * (D / 64), C::kQBox, C::kBQ, iv);  // (Q, and dO behind it)
        }
      }
      if (t > 0 && !(ok = bwd_wait<MOD>(&bars->s_free, (t - 1) & 1, wc))) break;
      FA_TRACE(1, t);
      tc_fence_after_sync();
      if (lane == 0) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + C::kColS, kmaj(k_s, kk, C::kBox), kmaj(q_s(st), kk, C::kQBox), kIdS,
                 kk > 0);
        mma_commit(&bars->s_full);
      }
      __syncwarp();
      if (t > 0 && !(ok = bwd_wait<MOD>(&bars->dp_free, (t - 1) & 1, wc))) break;
      FA_TRACE(2, t);
      tc_fence_after_sync();
      if (lane == 0) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + C::kColDP, kmaj(v_s, kk, C::kBox), kmaj(do_s(st), kk, C::kQBox), kIdS,
                 kk > 0);
        mma_commit(&bars->dp_full);
        mma_commit(&bars->q_empty[st]);
      }
      __syncwarp();
      if (++st == NS) { st = 0; ph ^= 1; }
    }
    if (lane == 0) mma_commit(&bars->score_done);
    __syncwarp();
  } else if (warp == C::kGradWarp) {
    // ---------------------------------------------------------------- gradient issuer
    constexpr uint32_t kIdV = idesc_bf16(128, D, true);             // dV: A in TMEM, B MN-major
    constexpr uint32_t kIdK = idesc_bf16_ab(128, D, false, true);   // dK: A K-major, B MN-major
    // dQ (d = 64: dS·K, M = queries) or dQᵀ (d = 128: Kᵀ·dSᵀ, M = head dims): both operands
    // MN-major, N = D or kBQ.
    constexpr uint32_t kIdQ = idesc_bf16_ab(128, (D == 64) ? D : C::kBQ, true, true);
    const uint32_t k_s = sbase + C::kK;
    bool ok = true;
    for (int t = 0, st = 0; t < n && ok; ++t) {
      // dV += Pᵀ·dO_i (Pᵀ from TMEM)
      if (!(ok = bwd_wait<MOD>(&bars->p_full, t & 1, wc))) break;
      FA_TRACE(3, t);
      tc_fence_after_sync();
      if (lane == 0) {
#pragma unroll
        for (int kk = 0; kk < C::kBQ / 16; ++kk)
          mma_ts(tmem + C::kColDV, tmem + C::kColP + kk * 8, mnmaj(do_s(st), kk, C::kQBox), kIdV,
                 (t > 0 || kk > 0));
        mma_commit(&bars->p_free);
      }
      __syncwarp();
      // dK += dSᵀ·Q_i, then dQ_i = dS·K_j (d = 64) or dQ_iᵀ = K_jᵀ·dSᵀ (d = 128)
      const int b = t & 1;
      const uint32_t ds_s = sbase + C::kDS + b * C::kDSBytes;
      if (!(ok = bwd_wait<MOD>(&bars->ds_full[b], (t >> 1) & 1, wc))) break;
      if (!C::kSplitQ && t > 0 && !(ok = bwd_wait<MOD>(&bars->dq_free, (t - 1) & 1, wc))) break;
      FA_TRACE(4, t);
      tc_fence_after_sync();
      if (lane == 0) {
#pragma unroll
        for (int kk = 0; kk < C::kBQ / 16; ++kk)
          mma_ss(tmem + C::kColDK, kmaj(ds_s, kk, C::kBox), mnmaj(q_s(st), kk, C::kQBox), kIdK,
                 (t > 0 || kk > 0));
#pragma unroll
        for (int kk = 0; kk < (C::kSplitQ ? 0 : 8); ++kk) {  // K = 128 keys
          if constexpr (D == 64)
            mma_ss(tmem + C::kColDQ, mnmaj(ds_s, kk, C::kBox), mnmaj(k_s, kk, C::kBox), kIdQ, kk > 0);
          else
            mma_ss(tmem + C::kColDQ, mnmaj(k_s, kk, C::kBox), mnmaj(ds_s, kk, C::kBox), kIdQ, kk > 0);
        }
        if constexpr (!C::kSplitQ) mma_commit(&bars->dq_full);
        mma_commit(&bars->ds_free[b]);
        mma_commit(&bars->q_empty[st]);
      }
      __syncwarp();
      if (++st == NS) st = 0;
    }
    if (lane == 0) mma_commit(&bars->grad_done);
    __syncwarp();
  } else if (C::kSplitQ && warp == C::kGradQWarp) {
    // ---------------------------------------------------------------- dQ issuer (d = 128)
    // dQ_iᵀ = K_jᵀ·dSᵀ once this tile's dSᵀ is stored and the previous dQ has been drained.
    constexpr uint32_t kIdQ = idesc_bf16_ab(128, (D == 64) ? D : C::kBQ, true, true);
    const uint32_t k_s = sbase + C::kK;
    bool ok = true;
    for (int t = 0; t < n && ok; ++t) {
      const int b = t & 1;
      const uint32_t ds_s = sbase + C::kDS + b * C::kDSBytes;
      if (!(ok = bwd_wait<MOD>(&bars->ds_full[b], (t >> 1) & 1, wc))) break;
      if (t > 0 && !(ok = bwd_wait<MOD>(&bars->dq_free, (t - 1) & 1, wc))) break;
      tc_fence_after_sync();
      if (lane == 0) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {  // K = 128 keys
          if constexpr (D == 64)
            mma_ss(tmem + C::kColDQ, mnmaj(ds_s, kk, C::kBox), mnmaj(k_s, kk, C::kBox), kIdQ, kk > 0);
          else
            mma_ss(tmem + C::kColDQ, mnmaj(k_s, kk, C::kBox), mnmaj(ds_s, kk, C::kBox), kIdQ, kk > 0);
        }
        mma_commit(&bars->dq_full);
        mma_commit(&bars->ds_free[b]);
      }
      __syncwarp();
    }
    if (lane == 0) mma_commit(&bars->grad_done);
    __syncwarp();
  }
  teardown();
  } else if (warp >= C::kDrainWarp0) {
    // ---------------------------------------------------------------- dQ drain
    const int qd = warp & 3;
    // TMEM lane = query row (d = 64, dQ) or head dim (d = 128, dQᵀ); either way 64 columns.
    const int r = qd * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(qd * 32) << 16;
    int t = 0;
    bool ok = true;
    // 16 TMEM columns at a time through this warp's two 2 KB staging buffers, each handed to
    // the TMA engine as one bulk reduce-add (the warp's 32 lanes × 16 columns are contiguous
    // in the accumulator: 32 query rows × 16 dims at d = 64, 32 dims × 16 query rows at
    // d = 128); before a buffer is rewritten, the reduction issued from it two chunks
    // earlier must have read it.
    const uint32_t stage0 = sbase + C::kDQStage + qd * 2 * C::kDQChunk;
    int nchunk = 0;
    int ti = 0, hg = 0;  // MOD: as in the producer
    for (; t < n; ++t) {
      if (!(ok = bwd_wait<MOD>(&bars->dq_full, t & 1, wc))) break;
      FA_TRACE(20, t);
      int it = i0 + t, bq = bh;
      if constexpr (MOD != 0) {
        it = i0 + ti;
        bq = wk.q0h + hg;
        if (++ti == wk.n_i) {
          ti = 0;
          ++hg;
        }
      }
      tc_fence_after_sync();
      // 32 columns at a time; the buffer is released once the last columns are in registers.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t x[32];
        tmem_ld32(tmem + lane_off + C::kColDQ + h * 32, x);
        tmem_ld_wait();
        reg_fence32(x);
        if (h == 1) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->dq_free);
          FA_TRACE(21, t);
        }
        {
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2, ++nchunk) {
            const uint32_t buf = stage0 + (nchunk & 1) * C::kDQChunk;
            if (nchunk >= 2) {
              if (lane == 0) bulk_wait_group_read1();
              __syncwarp();
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
              st_shared_v4(buf + (c * 32 + lane) * 16, x[16 * k2 + 4 * c], x[16 * k2 + 4 * c + 1],
                           x[16 * k2 + 4 * c + 2], x[16 * k2 + 4 * c + 3]);
            fence_proxy_async_smem();  // the staged values, visible to the TMA engine
            __syncwarp();
            if (lane == 0) {
              // TMEM columns 32h + 16k2 …: column group 8h + 4k2 of lanes 32·qd …
              const int cg = 8 * h + 4 * k2;
              bulk_reduce_add_f32(p.dq_acc + ((D == 64) ? dq_acc_offset(bq, it, p.n_qt, cg, qd * 32, D)
                                                        : dq_acc_offset_t(bq, it, p.n_qt, cg, qd * 32)),
                                  buf, C::kDQChunk);
              bulk_commit_group();
            }
          }
        }
      }
    }
    if (!ok) {
      // Abandoned tiles: poison their dQ rows so that the failure cannot go unseen.
      const float nan = __int_as_float(0x7fc00000);
      for (; t < n; ++t) {
        int it = i0 + t, bq = bh;
        if constexpr (MOD != 0) {
          it = i0 + t % wk.n_i;
          bq = wk.q0h + t / wk.n_i;
        }
        for (int c4 = 0; c4 < 16; ++c4) {
          float* dst = p.dq_acc + ((D == 64) ? dq_acc_offset(bq, it, p.n_qt, c4, r, D)
                                             : dq_acc_offset_t(bq, it, p.n_qt, c4, r));
          red_add_v4(dst, nan, nan, nan, nan);
        }
      }
    }
    // The bulk reductions must be complete (and their sources read) before the CTA exits.
    if (lane == 0) bulk_wait_group0();
    __syncwarp();
    teardown();
  } else {
    // ---------------------------------------------------------------- compute (warps 0-7)
    constexpr int NC = C::kNC;        // query columns of this warpgroup per tile (32)
    const int g = warp >> 2;          // columns NC·g .. NC·g + NC − 1 of each tile
    const int qd = warp & 3;
    const int r = qd * 32 + lane;     // key row within the tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(qd * 32) << 16;
    // dSᵀ columns of this warpgroup: box (NC·g)/64, 16-byte chunks from ((NC·g) mod 64)/8
    const int ds_box_idx = (NC * g) / 64, ds_chunk0 = ((NC * g) % 64) / 8;
    bool ok = true;
    int hg = 0, ti = 0;  // MOD: the step's query head within the group, and its tile within the walk
    float nslope = 0.f;
    for (int t = 0, st = 0, ph = 0; t < n && ok; ++t) {
      const int i = MOD != 0 ? i0 + ti : i0 + t;
      if constexpr ((MOD & kModBias) != 0) {
        if (ti == 0) nslope = __ldg(p.mod.slopes + wk.h0 + hg) * -1.4426950408889634f;
      }
      const float* vec = reinterpret_cast<const float*>(sm + C::kVec + st * C::kVecBytes);
      if (!(ok = bwd_wait<MOD>(&bars->q_full[st], ph, wc))) break;
      if (!(ok = bwd_wait<MOD>(&bars->s_full, t & 1, wc))) break;
      FA_TRACE(10, t);
      tc_fence_after_sync();
      uint32_t s[NC];
      float top_s = 0.f;  // (CAP: the largest |S|)
      if constexpr ((MOD & kModCap) != 0) top_s = tmem_load_cols_absmax<NC>(tmem + lane_off + C::kColS + g * NC, s);
      else tmem_load_cols<NC>(tmem + lane_off + C::kColS + g * NC, s);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->s_free);
      // Pᵀ = exp2(S·scale·log2e − log2e·LSE_q), zero where the key comes after the query
      // (the argument on fp32 pairs; the workspace holds −log2e·LSE)
      float pr[NC];
      // MOD: Pᵀ's pairs, packed as they are made (CAP needs both, P and what dS multiplies; plain d64
      // is faster without, B2 H12 T4096 182 -> 178 µs, but d128, B2 H16 T4096, 377 -> 387)
      constexpr bool kTwo = MOD != 0 && !(D == 64 && (MOD & ~kModSink) == kModOn);
      uint32_t pkm[kTwo ? NC / 2 : 1];
      const float4* l4 = reinterpret_cast<const float4*>(vec + g * NC);
      const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
      if constexpr (MOD != 0) {
        // The modified scores' P, packed at once; pr keeps P · (1 − tanh²), what dS multiplies.
        const int q0 = i * C::kBQ + g * NC, key = j * 128 + r;
        bool part;  // some row of the stage does not see every key of the tile
        if (p.mod.rows) part = bars->whole[st] != 1u;
        else part = j * 128 + 127 >= (p.mod.causal ? min(i * C::kBQ + 1, p.T) : p.T);
        const bool left = j * 128 + qd * 32 + 31 <= q0;
        const float dist0 = static_cast<float>(q0 - key);
        const float base = nslope * dist0;
        const float2* l2 = reinterpret_cast<const float2*>(vec + g * NC);
        const int2* iv = reinterpret_cast<const int2*>(vec + 2 * C::kBQ) + g * NC;
        auto probabilities = [&]<bool FAR, bool LEFT>() {
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            const float2 l = l2[c / 2];
            uint64_t x2 = f2_pack(l.x, l.y), bend = 0ull;
            const uint64_t s2 = f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
            if constexpr ((MOD & kModBias) != 0) {
              const float c0 = static_cast<float>(c), c1 = static_cast<float>(c + 1);
              x2 = f2_add(x2, LEFT ? f2_pack(fmaf(nslope, c0, base), fmaf(nslope, c1, base))
                                   : f2_pack(nslope * fabsf(dist0 + c0), nslope * fabsf(dist0 + c1)));
            }
            if constexpr ((MOD & kModCap) != 0) {
              const uint64_t z2 = cap2<FAR>(s2, p.mod.cap);
              x2 = f2_add(z2, x2);
              bend = f2_fma(f2_mul(z2, z2), f2_splat(p.mod.cap.bend), f2_splat(1.0f));  // 1 − tanh²
            } else {
              x2 = f2_fma(s2, c2, x2);
            }
            float x[2];
            f2_unpack(x2, x[0], x[1]);
            pr[c] = ex2_approx(x[0]);
            pr[c + 1] = ex2_approx(x[1]);
            if constexpr (kTwo) pkm[c / 2] = pack_bf16x2(pr[c], pr[c + 1]);
            if constexpr ((MOD & kModCap) != 0)
              f2_unpack(f2_mul(f2_pack(pr[c], pr[c + 1]), bend), pr[c], pr[c + 1]);
          }
        };
        bool far = false;
        if constexpr ((MOD & kModCap) != 0) far = __any_sync(0xffffffffu, top_s > p.mod.cap.limit);
        if (far) probabilities.template operator()<true, false>();
        else if ((MOD & kModBias) != 0 && !left) probabilities.template operator()<false, false>();
        else probabilities.template operator()<false, true>();
        // A crossed tile, too, has warps whose 32 keys every one of their queries sees (the causal
        // diagonal: 6 of 16).
        if (part) {
          if (p.mod.rows) {
            const int2 v = iv[lane & (NC - 1)];
            part = __reduce_max_sync(0xffffffffu, v.x) > key - lane || __reduce_min_sync(0xffffffffu, v.y) <= key - lane + 31;
          } else {
            part = (p.mod.causal && !left) || key - lane + 31 >= p.T;
          }
        }
        if (part) {  // masked pairs to zero, whatever their exponentials were
          // Which queries see this thread's key, as bits (kBits; c: query q0 + c), or asked of each
          // query: bits, B2 H12 T4096 d64 182 -> 178 µs, capped 216 -> 202; but d128, B2 H16 T4096 capped,
          // 412 -> 423.
          constexpr bool kBits = D == 64 || kSink;
          uint32_t seen = 0u;
          // without rows: queries from q0 + rel on see the key; none sees one behind the end, whose
          // score of 0 (its row is loaded as zeros) may be far above every other of a query
          const int rel = key >= p.T ? NC : p.mod.causal ? key - q0 : 0;
          if (kBits && p.mod.rows) {
            const int2 v = iv[lane & (NC - 1)];
            const int lo = min(max(v.x - (key - lane), 0), 32), hi = min(max(v.y - (key - lane), 0), 32);
            const uint32_t below = hi >= 32 ? 0xFFFFFFFFu : (1u << hi) - 1u;
            seen = lo >= 32 ? 0u : (below >> lo) << lo;
            if constexpr (kSink) {
              if (wk.sinks) {  // (few walks have any)
                const int2 k = __ldg(p.mod.sink_rows + (size_t)(bh / p.mod.Hkv) * p.T_pad + q0 + (lane & (NC - 1)));
                seen |= bits_of(k.x - (key - lane), k.y - (key - lane));
              }
            }
            // bits of keys, a lane a query -> bits of queries, a lane a key: 32 x 32 bits transposed
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) {
              const uint32_t m = x == 16 ? 0x0000FFFFu : x == 8 ? 0x00FF00FFu : x == 4 ? 0x0F0F0F0Fu : x == 2 ? 0x33333333u : 0x55555555u;
              const uint32_t y = __shfl_xor_sync(0xffffffffu, seen, x);
              seen = (lane & x) ? ((seen & ~m) | ((y >> x) & m)) : ((seen & m) | ((y << x) & ~m));
            }
          } else if (kBits) {
            seen = rel <= 0 ? 0xFFFFFFFFu : rel >= 32 ? 0u : 0xFFFFFFFFu << rel;
          }
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            bool out0, out1;
            if (kBits) {
              out0 = !((seen >> c) & 1u);
              out1 = !((seen >> (c + 1)) & 1u);
            } else if (p.mod.rows) {
              const int2 v0 = iv[c], v1 = iv[c + 1];
              out0 = key < v0.x || key >= v0.y;
              out1 = key < v1.x || key >= v1.y;
            } else {
              out0 = rel > c;
              out1 = rel > c + 1;
            }
            if (out0) {
              pr[c] = 0.f;
              if constexpr (kTwo) pkm[c / 2] &= 0xFFFF0000u;
            }
            if (out1) {
              pr[c + 1] = 0.f;
              if constexpr (kTwo) pkm[c / 2] &= 0x0000FFFFu;
            }
          }
        }
        if (++ti == wk.n_i) {
          ti = 0;
          ++hg;
        }
      } else {
#pragma unroll
      for (int c = 0; c < NC; c += 4) {
        const float4 l = l4[c / 4];
        float x0, x1, x2, x3;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), c2,
                         f2_pack(l.x, l.y)), x0, x1);
        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), c2,
                         f2_pack(l.z, l.w)), x2, x3);
        pr[c] = ex2_approx(x0);
        pr[c + 1] = ex2_approx(x1);
        pr[c + 2] = ex2_approx(x2);
        pr[c + 3] = ex2_approx(x3);
      }
      if (CAUSAL && j * 128 + 127 > i * C::kBQ) {  // a tile the diagonal crosses
        const int rel = j * 128 + r - (i * C::kBQ + g * NC);  // key − first query of the warpgroup
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (rel > c) pr[c] = 0.f;
      }
      if (RAGGED && j * 128 + r >= p.T) {
#pragma unroll
        for (int c = 0; c < NC; ++c) pr[c] = 0.f;
      }
      }
      FA_TRACE(11, t);
      if (t >= 1 && !(ok = bwd_wait<MOD>(&bars->p_free, (t - 1) & 1, wc))) break;
      FA_TRACE(12, t);
      uint32_t pk[NC / 2];
#pragma unroll
      for (int c = 0; c < NC / 2; ++c) pk[c] = kTwo ? pkm[c % (kTwo ? NC / 2 : 1)] : pack_bf16x2(pr[2 * c], pr[2 * c + 1]);
      tc_fence_after_sync();
      if constexpr (NC == 64) tmem_st32(tmem + lane_off + C::kColP + g * 32, pk);
      else if constexpr (NC == 32) tmem_st16(tmem + lane_off + C::kColP + g * 16, pk);
      else tmem_st8(tmem + lane_off + C::kColP + g * 8, pk);
      tmem_st_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->p_full);
      FA_TRACE(13, t);
      // dSᵀ = Pᵀ ∘ (dPᵀ − D_q), into shared-memory buffer t mod 2
      const int b = t & 1;
      const uint32_t ds_box = sbase + C::kDS + b * C::kDSBytes + ds_box_idx * C::kBox;
      if (!(ok = bwd_wait<MOD>(&bars->dp_full, t & 1, wc))) break;
      FA_TRACE(14, t);
      if (t >= 2 && !(ok = bwd_wait<MOD>(&bars->ds_free[b], ((t >> 1) - 1) & 1, wc))) break;
      FA_TRACE(15, t);
      tc_fence_after_sync();
      // dPᵀ for this warpgroup's columns (were a warpgroup to own NC = 64 columns: in two
      // halves, to stay within the register budget; capped at d = 64, B2 H12 T4096: 208 -> 202 µs)
      constexpr int kDPB = (NC > 32) ? 32 : (D == 64 && (MOD & kModCap) != 0) ? 16 : NC;  // columns per dPᵀ block
#pragma unroll
      for (int h = 0; h < NC / kDPB; ++h) {
        uint32_t dp[kDPB];
        tmem_load_cols<kDPB>(tmem + lane_off + C::kColDP + g * NC + h * kDPB, dp);
        if (h == NC / kDPB - 1) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->dp_free);
        }
        const float4* d4 = reinterpret_cast<const float4*>(vec + C::kBQ + g * NC + h * kDPB);
#pragma unroll
        for (int q4 = 0; q4 < kDPB / 8; ++q4) {
          const float4 da = d4[2 * q4], db = d4[2 * q4 + 1];
          const int c = h * kDPB + q4 * 8;
          const uint32_t* dq8 = dp + q4 * 8;
          // dS = P ∘ (dP − D) on fp32 pairs
          const float dd[8] = {da.x, da.y, da.z, da.w, db.x, db.y, db.z, db.w};
          float ds[8];
#pragma unroll
          for (int e = 0; e < 8; e += 2)
            f2_unpack(f2_mul(f2_pack(pr[c + e], pr[c + e + 1]),
                             f2_sub(f2_pack(__uint_as_float(dq8[e]), __uint_as_float(dq8[e + 1])),
                                    f2_pack(dd[e], dd[e + 1]))),
                      ds[e], ds[e + 1]);
          st_row_chunk_sw128(ds_box, r, ds_chunk0 + c / 8, ds);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->ds_full[b]);
      FA_TRACE(16, t);
      if (++st == NS) { st = 0; ph ^= 1; }
    }
    // ---- epilogue: warpgroup 0 writes dV_j, warpgroup 1 writes scale·dK_j (32 columns at
    // a time)
    bool done = ok && bwd_wait<MOD>(&bars->grad_done, 0, wc) && !bars->abort;
    done = __shfl_sync(0xffffffffu, done ? 1u : 0u, 0) != 0u;  // warp-uniform (TMEM loads)
    const int key = j * 128 + r;
    tc_fence_after_sync();
    // The first half of the warpgroups writes dV, the second scale·dK, each a block of
    // D / (kCWG / 2) columns.
    constexpr int kPer = C::kCWG / 2;
    const bool is_dv = g < kPer;
    const int part = g % kPer;
    const uint32_t col = is_dv ? C::kColDV : C::kColDK;
    const float mul = is_dv ? 1.f : p.scale;
    const float nan = __int_as_float(0x7fc00000);
    __nv_bfloat16* dst = (is_dv ? p.dv : p.dk) + ((size_t)bh * p.T + key) * D;
    constexpr int kH = D / 32 / kPer;  // 32-column blocks per warpgroup
#pragma unroll
    for (int hh = 0; hh < kH; ++hh) {
      const int h = part * kH + hh;
      uint32_t x[32];
      if (done) {
        tmem_ld32(tmem + lane_off + col + h * 32, x);
        tmem_ld_wait();
      }
      reg_fence32(x);
      if (key < p.T) {
#pragma unroll
        for (int c = 0; c < 32; c += 8) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = done ? __uint_as_float(x[c + e]) * mul : nan;
          if (MOD != 0 && n == 0) {  // a key tile that no query sees
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = 0.f;
          }
          if constexpr (MOD != 0) {
            if (kSink && wk.slot >= 0) {
              float* out = p.mod.piece_out +
                           ((((is_dv ? (size_t)p.BH : 0) + (size_t)bh * p.mod.parts + wk.part) * p.mod.n_slots + wk.slot) * 128 + r) * D +
                           h * 32 + c;
              reinterpret_cast<float4*>(out)[0] = make_float4(y[0], y[1], y[2], y[3]);
              reinterpret_cast<float4*>(out)[1] = make_float4(y[4], y[5], y[6], y[7]);
              continue;
            }
            if (p.mod.parts > 1) {
              const size_t rows = (size_t)(p.BH / p.mod.parts) * p.T;
              float* out = p.mod.part_out +
                           (((is_dv ? p.mod.parts : 0) + wk.part) * rows + (size_t)bh * p.T + key) * D + h * 32 + c;
              reinterpret_cast<float4*>(out)[0] = make_float4(y[0], y[1], y[2], y[3]);
              reinterpret_cast<float4*>(out)[1] = make_float4(y[4], y[5], y[6], y[7]);
              continue;
            }
          }
          uint4 v;
          v.x = pack_bf16x2(y[0], y[1]);
          v.y = pack_bf16x2(y[2], y[3]);
          v.z = pack_bf16x2(y[4], y[5]);
          v.w = pack_bf16x2(y[6], y[7]);
          *reinterpret_cast<uint4*>(dst + h * 32 + c) = v;
        }
      }
    }
    teardown();
  }
}

}  // namespace fa
