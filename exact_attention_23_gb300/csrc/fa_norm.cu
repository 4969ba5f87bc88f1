// Norms of queries and keys for each head with the rotation in the same pass (include/fa.h:
// fa_norm_rope, fa_norm_rope_append), and their gradients (fa_norm_rope_bwd):
//
//   r = 1 / √(mean(x²) + eps),   n = x · r,   y = n ∘ w, turned                (a row x of a head)
//
// and backward from g = ∂L/∂y, with h = g turned back:
//
//   dw = Σ_rows h ∘ n,   dn = h ∘ w,   dx = r · (dn − n · mean(dn ∘ n))
//      = r · (h ∘ w − x · r² · mean(h ∘ w ∘ x))
//
// so one sum a row forward (x²) and two backward (x² and h·w·x), which go through the lanes
// together. The angles are fa_rope.cu's, and so is who reads what: a thread owns 8 pairs (two 16-byte
// vectors) of one (batch, position) and walks several heads with them, the 4 or 8 neighbouring lanes
// of a row exchange its sums in 2 or 3 shuffles, and nothing but the rows goes through memory: 4
// bytes an element forward, 6 backward.
//
// What bounds them: on long batches the rows' way from memory and the wait in its middle, the lanes' sum and a root between
// a row's loads and its stores: forward B4 H12+12 T16384 d64 (403 MB) 81.2 µs, B1 H16+4 T16384 d128 (168 MB) 34.7, 4.8 to 5.0
// TB/s, where fa_rope.cu, without a sum, moves the same bytes in 67.4 and 29.6 (copying: 6.8 TB/s), and more heads in flight
// cost blocks an SM (below); backward that size (252 MB) 50.1 µs, 5.0 TB/s. On short ones the launch and one
// wave's latency, B4 H12+12 T1024 d64 7.0 µs, one token 2.5. Arithmetic is on pairs of neighbouring
// dimensions (fp32x2), weights lie in shared memory in the order that lanes read them in, and rows are
// numbered with 32 bits, whose divisions are multiplications (backward 65 -> 51 µs).
//
// dw sums over all rows. A block of the backward takes queries or keys, never both, and keeps its 16
// sums a thread in registers over all its rows (a persistent grid), so that a call leaves at most
// kNormBlocks rows of partial sums; fa_norm_dw_kernel adds them in order: the same bits every time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "fa.h"
#include "fa_host.h"
#include "fa_mod.cuh"
#include "fa_pdl.h"
#include "fa_rope.cuh"
#include "sm103.cuh"

namespace fa {

struct NormParams {
  RopeSrc q, k, v;
  RopeSrc gq, gk;                        // backward: gradients of the results
  __nv_bfloat16 *q_out, *k_out, *v_out;  // [B][heads][rows][d], rows: T or Tmax (caches)
  const float *wq, *wk;                  // [d]
  float* part;                           // backward: [gridDim.x][d] sums of h ∘ n
  const int* positions;                  // [T] or [B][T]; null: t, or context + t
  const int* ctx_len;                    // append: [B]
  const double* inv_freq;
  long long n_items;                     // B · T · d / 16
  unsigned n_blocks;                     // blocks per head chunk
  unsigned q_blocks;                     // backward: blocks that take queries
  int pos_per_batch;
  int B, H, Hkv, T, Tmax, rot_units;
  int heads, chunk;                      // q + k (+ v) heads; heads a thread walks
  FastDiv div_t, div_q, div_k;           // by T; backward: by the queries' and the keys' head chunks
  float mscale, eps;
};

// Forward: one head's loads a thread in flight and eight blocks an SM (61 registers): B4 H12+12 T1024 d64 7.0 µs,
// B1 H16+4 T16384 d128 35.7; two heads, five blocks 7.6 and 41.7; four heads, four blocks 7.7 and 37.4.
constexpr int kNormThreads = 128;
constexpr int kNormPerSm = 8;
constexpr int kNormFlight = 1;   // heads whose loads a thread keeps in flight
// Backward: one row at hand and the next on its way, 124 registers: four blocks an SM 51.4 µs, three 54.7. (Two heads
// at once without the next: 57.7. A ring of four rows in shared memory by asynchronous copies: 69.)
constexpr int kNormBackPerSm = 4;
constexpr int kNormBlocks = 608;  // of the backward, at most (the workspace's rows)

// The sum over the lanes of a row.
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = 1; off < D / 16; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// Where a thread's two 16-byte vectors lie: (i, i + rot/2) or neighbours.
struct Unit16 {
  int c0, c1;
  bool turn;
  template <bool INTER>
  static __device__ __forceinline__ Unit16 of(int u, int rot_units) {
    Unit16 x;
    x.turn = u < rot_units;
    x.c0 = (x.turn && !INTER) ? u * 8 : u * 16;
    x.c1 = (x.turn && !INTER) ? (rot_units + u) * 8 : u * 16 + 8;
    return x;
  }
};

// A thread's 16 values as pairs turned by (cs, sn).
template <bool INTER>
__device__ __forceinline__ void turn16(float* v, const float* cs, const float* sn) {
  float w[16];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int ia = INTER ? 2 * e : e, ib = INTER ? 2 * e + 1 : e + 8;
    w[ia] = fmaf(v[ia], cs[e], -v[ib] * sn[e]);
    w[ib] = fmaf(v[ia], sn[e], v[ib] * cs[e]);
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = w[e];
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// Pair e of the sixteen bf16 values of two vectors, as fp32.
__device__ __forceinline__ uint64_t pair_of(const uint4& a, const uint4& b, int e) {
  const uint4& v = e < 4 ? a : b;
  const uint32_t x = e % 4 == 0 ? v.x : e % 4 == 1 ? v.y : e % 4 == 2 ? v.z : v.w;
  return f2_pack(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}

// Where dimension c of a weight lies in shared memory: each unit's 16 values are four vectors whose
// neighbours are the next units', so that the lanes of a row read without bank conflicts.
template <int D, bool INTER>
__device__ __forceinline__ int weight_at(int c, int rot_units) {
  int u = c / 16, e = c % 16;
  if (!INTER && c < 16 * rot_units) {
    const int half = c >= 8 * rot_units;
    u = c / 8 - (half ? rot_units : 0);
    e = c % 8 + 8 * half;
  }
  return ((e / 4) * (D / 16) + u) * 4 + e % 4;
}

template <int D, bool INTER, bool APPEND>
__global__ void __launch_bounds__(kNormThreads, kNormPerSm) fa_norm_kernel(const NormParams p) {
  __shared__ unsigned long long turns[64];
  __shared__ __align__(16) float weight[2][D];
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x < 8 * p.rot_units) turns[threadIdx.x] = turns_of(p.inv_freq[threadIdx.x]);
  if (threadIdx.x < D) {
    const int at = weight_at<D, INTER>(threadIdx.x, p.rot_units);
    weight[0][at] = p.wq[threadIdx.x];
    if (p.Hkv > 0) weight[1][at] = p.wk[threadIdx.x];
  }
  __syncthreads();
  constexpr int kUnits = D / 16;
  const unsigned ch = blockIdx.x / p.n_blocks;
  const long long item = static_cast<long long>(blockIdx.x - ch * p.n_blocks) * kNormThreads + threadIdx.x;
  const bool in = item < p.n_items;  // (whole rows: the lanes of a row stay together)
  const int u = static_cast<int>(item % kUnits);
  const uint32_t row = in ? static_cast<uint32_t>(item / kUnits) : 0u;
  const int b = static_cast<int>(p.div_t.div(row));
  const int t = static_cast<int>(row) - b * p.T;
  const Unit16 at = Unit16::of<INTER>(u, p.rot_units);
  const int h0 = static_cast<int>(ch) * p.chunk, h1 = min(p.heads, h0 + p.chunk);
  int ctx = 0;
  bool live = in;      // append: an active sequence
  bool stored = true;  // append: the row exists in the caches
  if constexpr (APPEND) {
    ctx = p.ctx_len[b];
    live = in && ctx >= 0;
    stored = live && static_cast<long long>(ctx) + t < p.Tmax;
  }
  float cs[8], sn[8];
  if (at.turn && live && h0 < p.H + p.Hkv) {
    const long long pos = p.positions ? p.positions[p.pos_per_batch ? row : t] : static_cast<long long>(ctx) + t;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = angle_of(turns[u * 8 + e], pos);
      cs[e] = __cosf(x) * p.mscale;
      sn[e] = __sinf(x) * p.mscale;
    }
  }
  for (int hb = h0; hb < h1; hb += kNormFlight) {
    uint4 x0[kNormFlight], x1[kNormFlight];
#pragma unroll
    for (int i = 0; i < kNormFlight; ++i) {
      const int h = hb + i;
      x0[i] = x1[i] = make_uint4(0u, 0u, 0u, 0u);
      if (h >= h1 || !live) continue;
      const bool is_q = h < p.H, is_k = !is_q && h < p.H + p.Hkv;
      const RopeSrc s = is_q ? p.q : (is_k ? p.k : p.v);
      const int hh = is_q ? h : (is_k ? h - p.H : h - p.H - p.Hkv);
      const __nv_bfloat16* src = s.p + b * s.sb + hh * s.sh + t * s.st;
      x0[i] = *reinterpret_cast<const uint4*>(src + at.c0);
      x1[i] = *reinterpret_cast<const uint4*>(src + at.c1);
    }
    // (on pairs of neighbouring dimensions)
    float r[kNormFlight];
#pragma unroll
    for (int i = 0; i < kNormFlight; ++i) {
      uint64_t ss = f2_pack(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint64_t v = pair_of(x0[i], x1[i], e);
        ss = f2_fma(v, v, ss);
      }
      float s0, s1;
      f2_unpack(ss, s0, s1);
      r[i] = s0 + s1;
    }
#pragma unroll
    for (int i = 0; i < kNormFlight; ++i)
      r[i] = rsqrtf(fmaf(row_sum<D>(r[i]), 1.0f / D, p.eps));
#pragma unroll
    for (int i = 0; i < kNormFlight; ++i) {
      const int h = hb + i;
      if (h >= h1 || !in) continue;
      const bool is_q = h < p.H, is_k = !is_q && h < p.H + p.Hkv;
      uint4 y0 = x0[i], y1 = x1[i];
      if (live && (is_q || is_k)) {
        float v[16];
        const uint64_t r2 = f2_pack(r[i], r[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 w = *reinterpret_cast<const float4*>(&weight[is_q ? 0 : 1][(j * kUnits + u) * 4]);
          f2_unpack(f2_mul(f2_mul(pair_of(x0[i], x1[i], 2 * j), r2), f2_pack(w.x, w.y)), v[4 * j], v[4 * j + 1]);
          f2_unpack(f2_mul(f2_mul(pair_of(x0[i], x1[i], 2 * j + 1), r2), f2_pack(w.z, w.w)), v[4 * j + 2], v[4 * j + 3]);
        }
        if (at.turn) turn16<INTER>(v, cs, sn);
        y0 = pack8(v);
        y1 = pack8(v + 8);
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
      *reinterpret_cast<uint4*>(dst + at.c0) = y0;
      *reinterpret_cast<uint4*>(dst + at.c1) = y1;
    }
  }
}

// Backward. Blocks up to q_blocks take the queries' rows, the others the keys', each walking its
// share of (block of items, head chunk) pairs.
template <int D, bool INTER>
__global__ void __launch_bounds__(kNormThreads, kNormBackPerSm) fa_norm_bwd_kernel(const NormParams p) {
  __shared__ unsigned long long turns[64];
  __shared__ __align__(16) float weight[D];
  __shared__ float sums[kNormThreads / 32][D];
  pdl_wait();
  pdl_launch_dependents();
  const bool is_q = blockIdx.x < p.q_blocks;
  if (threadIdx.x < 8 * p.rot_units) turns[threadIdx.x] = turns_of(p.inv_freq[threadIdx.x]);
  if (threadIdx.x < D) weight[weight_at<D, INTER>(threadIdx.x, p.rot_units)] = (is_q ? p.wq : p.wk)[threadIdx.x];
  __syncthreads();
  constexpr int kUnits = D / 16;
  const int heads = is_q ? p.H : p.Hkv;
  const RopeSrc xs = is_q ? p.q : p.k, gs = is_q ? p.gq : p.gk;
  __nv_bfloat16* const out = is_q ? p.q_out : p.k_out;
  const int u = static_cast<int>(threadIdx.x % kUnits);
  const Unit16 at = Unit16::of<INTER>(u, p.rot_units);
  const FastDiv div = is_q ? p.div_q : p.div_k;
  const uint32_t n_tasks = div.d * p.n_blocks, step = is_q ? p.q_blocks : gridDim.x - p.q_blocks;
  // A row of a task: (position, head), where its vectors lie, and its position's number.
  struct Row {
    const __nv_bfloat16 *x, *g;
    __nv_bfloat16* dst;
    int left;       // heads of the task behind it
    bool in;        // (whole rows: the lanes of a row stay together)
    int pos;
  };
  auto open = [&](uint32_t task) {
    Row r;
    const uint32_t block = div.div(task);  // (a position's chunks go out together)
    const int h0 = static_cast<int>(task - block * div.d) * p.chunk;
    r.left = min(heads, h0 + p.chunk) - h0 - 1;
    const long long item = static_cast<long long>(block) * kNormThreads + threadIdx.x;
    r.in = item < p.n_items;
    const uint32_t row = r.in ? static_cast<uint32_t>(item / kUnits) : 0u;
    const int b = static_cast<int>(p.div_t.div(row));
    const int t = static_cast<int>(row) - b * p.T;
    r.x = xs.p + b * xs.sb + t * xs.st + h0 * xs.sh;
    r.g = gs.p + b * gs.sb + t * gs.st + h0 * gs.sh;
    r.dst = out + ((static_cast<size_t>(b) * heads + h0) * p.T + t) * D;
    r.pos = p.positions ? p.positions[p.pos_per_batch ? row : t] : t;
    return r;
  };
  auto load = [&](const Row& r, uint4 (&v)[4]) {
    v[0] = v[1] = v[2] = v[3] = make_uint4(0u, 0u, 0u, 0u);
    if (!r.in) return;
    v[0] = *reinterpret_cast<const uint4*>(r.x + at.c0);
    v[1] = *reinterpret_cast<const uint4*>(r.x + at.c1);
    v[2] = *reinterpret_cast<const uint4*>(r.g + at.c0);
    v[3] = *reinterpret_cast<const uint4*>(r.g + at.c1);
  };
  uint64_t acc[8];  // pairs of neighbouring dimensions
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = f2_pack(0.f, 0.f);
  uint32_t task = is_q ? blockIdx.x : blockIdx.x - p.q_blocks;
  if (task < n_tasks) {
    float cs[8], sn[8];
    Row cur = open(task);
    uint4 v[4];
    load(cur, v);
    bool fresh = true;  // the row is its task's first
    while (true) {
      // The next row's vectors are on their way while this one's are worked on.
      Row next = cur;
      const bool same = cur.left > 0;
      bool more = true;
      if (same) {
        --next.left;
        next.x += xs.sh;
        next.g += gs.sh;
        next.dst += static_cast<size_t>(p.T) * D;
      } else {
        task += step;
        more = task < n_tasks;
        if (more) next = open(task);
      }
      uint4 nv[4];
      if (more) load(next, nv);
      if (fresh && at.turn) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = angle_of(turns[u * 8 + e], cur.pos);
          cs[e] = __cosf(x) * p.mscale;
          sn[e] = __sinf(x) * -p.mscale;
        }
      }
      float y[16];
      unpack8(v[2], y);
      unpack8(v[3], y + 8);
      if (at.turn) turn16<INTER>(y, cs, sn);
      uint64_t x2[8], y2[8], yw[8], ss = f2_pack(0.f, 0.f), sd = ss;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x2[e] = pair_of(v[0], v[1], e);
        y2[e] = f2_pack(y[2 * e], y[2 * e + 1]);
        const float2 w = *reinterpret_cast<const float2*>(weight + (e / 2 * kUnits + u) * 4 + e % 2 * 2);
        yw[e] = f2_mul(y2[e], f2_pack(w.x, w.y));
        ss = f2_fma(x2[e], x2[e], ss);
        sd = f2_fma(yw[e], x2[e], sd);
      }
      float s0, s1, d0, d1;
      f2_unpack(ss, s0, s1);
      f2_unpack(sd, d0, d1);
      const float sum_x = row_sum<D>(s0 + s1), sum_d = row_sum<D>(d0 + d1);
      const float r = rsqrtf(fmaf(sum_x, 1.0f / D, p.eps));
      float along = r * sum_d;  // Σ h·w·n  (r² may overflow)
      if (__any_sync(0xffffffffu, !(fabsf(along) < INFINITY))) {
        // Σ h·w·x passes fp32's range, or there is a NaN: the sum from n itself. (0 where Σ x² passes it too, as n is.)
        uint64_t sn2 = f2_pack(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) sn2 = f2_fma(yw[e], f2_mul(x2[e], f2_splat(r)), sn2);
        f2_unpack(sn2, d0, d1);
        const float sum_n = row_sum<D>(d0 + d1);
        if (!(fabsf(along) < INFINITY)) along = sum_n;
      }
      const uint64_t r2 = f2_pack(r, r), back = f2_splat(-r * (1.0f / D) * along);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        acc[e] = f2_fma(y2[e], f2_mul(x2[e], r2), acc[e]);
        const uint64_t z = f2_mul(f2_fma(x2[e], back, yw[e]), r2);
        f2_unpack(z, y[2 * e], y[2 * e + 1]);
      }
      if (cur.in) {
        *reinterpret_cast<uint4*>(cur.dst + at.c0) = pack8(y);
        *reinterpret_cast<uint4*>(cur.dst + at.c1) = pack8(y + 8);
      }
      if (!more) break;
      cur = next;
      fresh = !same;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = nv[e];
    }
  }
  // The block's sums: lanes with the same dimensions, then the warps.
  float a[16];
#pragma unroll
  for (int e = 0; e < 8; ++e) f2_unpack(acc[e], a[2 * e], a[2 * e + 1]);
#pragma unroll
  for (int e = 0; e < 16; ++e)
#pragma unroll
    for (int off = kUnits; off < 32; off <<= 1) a[e] += __shfl_xor_sync(0xffffffffu, a[e], off);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane < kUnits) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sums[warp][at.c0 + e] = a[e];
      sums[warp][at.c1 + e] = a[e + 8];
    }
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kNormThreads / 32; ++w) s += sums[w][threadIdx.x];
    p.part[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] = s;
  }
}

// dw from the blocks' sums, in order: a block takes 32 dimensions of the queries' or the keys', its
// warps every 32nd row.
__global__ void __launch_bounds__(1024) fa_norm_dw_kernel(const float* part, float* dwq, float* dwk, int d,
                                                          unsigned q_blocks, unsigned blocks) {
  __shared__ float s[32][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = d / 32;
  const bool is_q = blockIdx.x < groups;
  const int c = static_cast<int>(blockIdx.x % groups) * 32 + lane;
  const unsigned r0 = is_q ? 0u : q_blocks, r1 = is_q ? q_blocks : blocks;
  float a = 0.f;
#pragma unroll 4
  for (unsigned r = r0 + warp; r < r1; r += 32) a += part[static_cast<size_t>(r) * d + c];
  s[warp][lane] = a;
  __syncthreads();
  if (warp == 0) {
    a = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) a += s[w][lane];
    (is_q ? dwq : dwk)[c] = a;
  }
}

namespace {

using namespace fa::host;

bool norm_eps_ok(float eps) { return std::isfinite(eps) && eps > 0.0f; }
// (the kernels number rows with 32 bits; more than 2³¹ do not fit a GPU's memory)
bool norm_rows_ok(int B, int T) { return static_cast<long long>(B) * T <= INT32_MAX; }

int norm_launch(NormParams& p, bool append, int interleaved, int d, void* stream) {
  int dev = -1, sms = 0;
  const int st = check_device(&dev, &sms);
  if (st != FA_OK) return st;
  p.heads = p.H + p.Hkv * (append ? 2 : 1);
  p.n_items = static_cast<long long>(p.B) * p.T * (d / 16);
  const long long blocks = (p.n_items + kNormThreads - 1) / kNormThreads;
  // Heads a thread walks, as in fa_rope: as many as leave every SM its blocks.
  long long chunk = p.heads;
  while (chunk > 1 && blocks * ((p.heads + chunk - 1) / chunk) < static_cast<long long>(kNormPerSm) * sms) chunk = (chunk + 1) / 2;
  p.chunk = static_cast<int>(chunk);
  const long long grid = blocks * ((p.heads + chunk - 1) / chunk);
  if (grid > INT32_MAX) return FA_ERR_INVALID_ARG;
  p.n_blocks = static_cast<unsigned>(blocks);
  p.div_t = FastDiv::make(static_cast<uint32_t>(p.T));
  using Fn = void (*)(const NormParams);
  static constexpr Fn fns[2][2][2] = {
      {{&fa_norm_kernel<64, false, false>, &fa_norm_kernel<64, false, true>},
       {&fa_norm_kernel<64, true, false>, &fa_norm_kernel<64, true, true>}},
      {{&fa_norm_kernel<128, false, false>, &fa_norm_kernel<128, false, true>},
       {&fa_norm_kernel<128, true, false>, &fa_norm_kernel<128, true, true>}}};
  return launch_pdl(fns[d == 128][interleaved != 0][append], static_cast<unsigned>(grid), kNormThreads, 0,
                    static_cast<cudaStream_t>(stream), p) == cudaSuccess
             ? FA_OK : FA_ERR_LAUNCH;
}

bool words_misaligned(std::initializer_list<const void*> ps) {
  uintptr_t x = 0;
  for (const void* q : ps) x |= reinterpret_cast<uintptr_t>(q);
  return (x & 3u) != 0;
}

// Whether an output lies over a weight.
bool over_weights(const void* out, size_t bytes, const float* wq, const float* wk, int d) {
  return overlaps(out, bytes, wq, static_cast<size_t>(d) * 4) ||
         (wk && overlaps(out, bytes, wk, static_cast<size_t>(d) * 4));
}

}  // namespace

}  // namespace fa

using namespace fa;
using namespace fa::host;

extern "C" {

int fa_norm_rope(const void* q, long long q_sb, long long q_sh, long long q_st, void* q_out, const void* k,
                 long long k_sb, long long k_sh, long long k_st, void* k_out, const float* q_weight,
                 const float* k_weight, float eps, const int* positions, int positions_per_batch,
                 const double* inv_freq, int rot_dim, int interleaved, float mscale, int B, int H, int Hkv,
                 int T, int d, void* stream) {
  if (!q || !q_out || !inv_freq || !q_weight || !sizes_ok(B, H, Hkv, T, d, rot_dim, mscale) || !norm_eps_ok(eps) || !norm_rows_ok(B, T))
    return FA_ERR_INVALID_ARG;
  if ((Hkv > 0) != (k != nullptr) || (Hkv > 0) != (k_out != nullptr) || (Hkv > 0) != (k_weight != nullptr))
    return FA_ERR_INVALID_ARG;
  NormParams p{};
  p.q = {static_cast<const __nv_bfloat16*>(q), q_sb, q_sh, q_st};
  p.k = {static_cast<const __nv_bfloat16*>(k), k_sb, k_sh, k_st};
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(k_out) ||
      words_misaligned({positions, q_weight, k_weight}) || (reinterpret_cast<uintptr_t>(inv_freq) & 7u))
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
      over_weights(q_out, qo, q_weight, k_weight, d))
    return FA_ERR_INVALID_ARG;
  if (k && (over_tables(k_out, ko, positions, positions_per_batch, inv_freq, rot_dim, nullptr, B, T) ||
            over_weights(k_out, ko, q_weight, k_weight, d)))
    return FA_ERR_INVALID_ARG;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.wq = q_weight;
  p.wk = k_weight;
  p.positions = positions;
  p.pos_per_batch = positions_per_batch != 0;
  p.inv_freq = inv_freq;
  p.rot_units = rot_dim / 16;
  p.B = B; p.H = H; p.Hkv = Hkv; p.T = T; p.Tmax = T;
  p.mscale = mscale;
  p.eps = eps;
  return norm_launch(p, false, interleaved, d, stream);
}

int fa_norm_rope_append(const void* q, long long q_sb, long long q_sh, long long q_st, void* q_out,
                        const void* k, long long k_sb, long long k_sh, long long k_st, const void* v,
                        long long v_sb, long long v_sh, long long v_st, const float* q_weight,
                        const float* k_weight, float eps, void* k_cache, void* v_cache, const int* ctx_len,
                        const int* positions, int positions_per_batch, const double* inv_freq, int rot_dim,
                        int interleaved, float mscale, int B, int H, int Hkv, int Tq, int Tmax, int d,
                        void* stream) {
  if (!q || !q_out || !k || !v || !k_cache || !v_cache || !ctx_len || !inv_freq || !q_weight || !k_weight ||
      !sizes_ok(B, H, Hkv, Tq, d, rot_dim, mscale) || !norm_eps_ok(eps) || !norm_rows_ok(B, Tq) ||
      Hkv <= 0 || Tmax <= 0)
    return FA_ERR_INVALID_ARG;
  NormParams p{};
  p.q = {static_cast<const __nv_bfloat16*>(q), q_sb, q_sh, q_st};
  p.k = {static_cast<const __nv_bfloat16*>(k), k_sb, k_sh, k_st};
  p.v = {static_cast<const __nv_bfloat16*>(v), v_sb, v_sh, v_st};
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(v) || !aligned16(k_cache) ||
      !aligned16(v_cache) || words_misaligned({positions, ctx_len, q_weight, k_weight}) ||
      (reinterpret_cast<uintptr_t>(inv_freq) & 7u))
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
    if (over_tables(outs[a], out_bytes[a], positions, positions_per_batch, inv_freq, rot_dim, ctx_len, B, Tq) ||
        over_weights(outs[a], out_bytes[a], q_weight, k_weight, d))
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
  p.wq = q_weight;
  p.wk = k_weight;
  p.positions = positions;
  p.pos_per_batch = positions_per_batch != 0;
  p.ctx_len = ctx_len;
  p.inv_freq = inv_freq;
  p.rot_units = rot_dim / 16;
  p.B = B; p.H = H; p.Hkv = Hkv; p.T = Tq; p.Tmax = Tmax;
  p.mscale = mscale;
  p.eps = eps;
  return norm_launch(p, true, interleaved, d, stream);
}

size_t fa_norm_rope_bwd_workspace_size(int d) {
  return d == 64 || d == 128 ? static_cast<size_t>(kNormBlocks) * d * 4 : 0;
}

int fa_norm_rope_bwd(const void* gq, long long gq_sb, long long gq_sh, long long gq_st, const void* q,
                     long long q_sb, long long q_sh, long long q_st, void* dq, const void* gk,
                     long long gk_sb, long long gk_sh, long long gk_st, const void* k, long long k_sb,
                     long long k_sh, long long k_st, void* dk, const float* q_weight, const float* k_weight,
                     float* dq_weight, float* dk_weight, float eps, const int* positions,
                     int positions_per_batch, const double* inv_freq, int rot_dim, int interleaved,
                     float mscale, int B, int H, int Hkv, int T, int d, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (!gq || !q || !dq || !inv_freq || !q_weight || !dq_weight || !workspace ||
      !sizes_ok(B, H, Hkv, T, d, rot_dim, mscale) || !norm_eps_ok(eps) || !norm_rows_ok(B, T))
    return FA_ERR_INVALID_ARG;
  const bool keys = Hkv > 0;
  for (const void* x : {gk, k, static_cast<const void*>(dk), static_cast<const void*>(k_weight),
                        static_cast<const void*>(dk_weight)})
    if (keys != (x != nullptr)) return FA_ERR_INVALID_ARG;
  const size_t need = fa_norm_rope_bwd_workspace_size(d);
  if (workspace_bytes < need) return FA_ERR_INVALID_ARG;
  NormParams p{};
  p.q = {static_cast<const __nv_bfloat16*>(q), q_sb, q_sh, q_st};
  p.gq = {static_cast<const __nv_bfloat16*>(gq), gq_sb, gq_sh, gq_st};
  p.k = {static_cast<const __nv_bfloat16*>(k), k_sb, k_sh, k_st};
  p.gk = {static_cast<const __nv_bfloat16*>(gk), gk_sb, gk_sh, gk_st};
  if (!aligned16(gq) || !aligned16(q) || !aligned16(dq) || !aligned16(gk) || !aligned16(k) || !aligned16(dk) ||
      words_misaligned({positions, q_weight, k_weight, dq_weight, dk_weight}) ||
      (reinterpret_cast<uintptr_t>(inv_freq) & 7u) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return FA_ERR_MISALIGNED;
  const size_t none = 1;
  const void* ins[4] = {q, gq, k, gk};
  const size_t in_bytes[4] = {span_bytes(p.q, B, H, T, d), span_bytes(p.gq, B, H, T, d),
                              keys ? span_bytes(p.k, B, Hkv, T, d) : none,
                              keys ? span_bytes(p.gk, B, Hkv, T, d) : none};
  for (size_t x : in_bytes)
    if (x == 0) return FA_ERR_INVALID_ARG;
  // dq and dk may be the (contiguous) gradients that they are made from.
  const bool in_place[2] = {gq == dq && contiguous(p.gq, B, H, T, d), keys && gk == dk && contiguous(p.gk, B, Hkv, T, d)};
  const size_t wb = static_cast<size_t>(d) * 4;
  const void* outs[5] = {dq, dk, dq_weight, dk_weight, workspace};
  const size_t out_bytes[5] = {static_cast<size_t>(B) * H * T * d * 2, static_cast<size_t>(B) * Hkv * T * d * 2, wb, wb, need};
  for (int a = 0; a < 5; ++a) {
    if (!outs[a]) continue;
    for (int b = 0; b < 4; ++b)
      if (ins[b] && !(a < 2 && b == 2 * a + 1 && in_place[a]) && overlaps(outs[a], out_bytes[a], ins[b], in_bytes[b]))
        return FA_ERR_INVALID_ARG;
    if (over_tables(outs[a], out_bytes[a], positions, positions_per_batch, inv_freq, rot_dim, nullptr, B, T) ||
        over_weights(outs[a], out_bytes[a], q_weight, k_weight, d))
      return FA_ERR_INVALID_ARG;
    for (int b = a + 1; b < 5; ++b)
      if (outs[b] && overlaps(outs[a], out_bytes[a], outs[b], out_bytes[b])) return FA_ERR_INVALID_ARG;
  }
  int dev = -1, sms = 0;
  const int st = check_device(&dev, &sms);
  if (st != FA_OK) return st;
  p.q_out = static_cast<__nv_bfloat16*>(dq);
  p.k_out = static_cast<__nv_bfloat16*>(dk);
  p.wq = q_weight;
  p.wk = k_weight;
  p.part = static_cast<float*>(workspace);
  p.positions = positions;
  p.pos_per_batch = positions_per_batch != 0;
  p.inv_freq = inv_freq;
  p.rot_units = rot_dim / 16;
  p.B = B; p.H = H; p.Hkv = Hkv; p.T = T; p.Tmax = T;
  p.mscale = mscale;
  p.eps = eps;
  p.n_items = static_cast<long long>(B) * T * (d / 16);
  const long long blocks = (p.n_items + kNormThreads - 1) / kNormThreads;
  if (blocks > INT32_MAX) return FA_ERR_INVALID_ARG;
  p.n_blocks = static_cast<unsigned>(blocks);
  const long long most = std::min<long long>(kNormBlocks, static_cast<long long>(kNormBackPerSm) * sms);
  // Heads a thread walks: as many as leave every block of the grid eight tasks, of which the last may be
  // one too many (B1 H16+4 T16384 d128, 2.1 tasks of 16 heads a block: 56.8 µs; 8.4 of 4: 51.4).
  auto tasks = [&](int heads, long long chunk) { return (heads + chunk - 1) / chunk * blocks; };
  long long chunk = std::max(H, Hkv);
  while (chunk > 1 && tasks(H, chunk) + (keys ? tasks(Hkv, chunk) : 0) < 8 * most) chunk = (chunk + 1) / 2;
  p.chunk = static_cast<int>(chunk);
  const long long nq = tasks(H, chunk), nk = keys ? tasks(Hkv, chunk) : 0;
  if (nq > INT32_MAX || nk > INT32_MAX) return FA_ERR_INVALID_ARG;
  p.div_t = FastDiv::make(static_cast<uint32_t>(T));
  p.div_q = FastDiv::make(static_cast<uint32_t>((H + chunk - 1) / chunk));
  p.div_k = FastDiv::make(static_cast<uint32_t>(std::max<long long>(1, (Hkv + chunk - 1) / chunk)));
  const long long grid = std::max<long long>(keys ? 2 : 1, std::min(most, nq + nk));
  // Blocks shared out as the rows are.
  const long long qb = keys ? std::min(std::max<long long>(1, grid * H / (H + Hkv)), grid - 1) : grid;
  p.q_blocks = static_cast<unsigned>(qb);
  auto s = static_cast<cudaStream_t>(stream);
  auto* fn = d == 64 ? (interleaved ? &fa_norm_bwd_kernel<64, true> : &fa_norm_bwd_kernel<64, false>)
                     : (interleaved ? &fa_norm_bwd_kernel<128, true> : &fa_norm_bwd_kernel<128, false>);
  if (launch_pdl(fn, static_cast<unsigned>(grid), kNormThreads, 0, s, p) != cudaSuccess) return FA_ERR_LAUNCH;
  const float* part = p.part;
  return launch_pdl(fa_norm_dw_kernel, static_cast<unsigned>((keys ? 2 : 1) * (d / 32)), 1024, 0, s, part, dq_weight,
                    dk_weight, d, p.q_blocks, static_cast<unsigned>(grid)) == cudaSuccess
             ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
