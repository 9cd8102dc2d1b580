// fa_decode_scored.cu -- single-query attention over a padded cache with capped scores, a bias by
// distance, a window and a first key per batch row.
//
// Bound by HBM.  Keys and values come through a ring of 128-key stages by TMA; each of 8 warps takes 16
// keys of a stage for up to 16 query heads of the KV head, with both products on mma.sync (m16n8k16, the heads
// are the rows): the plain decode's dot products on the CUDA cores (fa_decode.cu) leave its warps 20%
// of headroom at HBM's pace, which the cap's arithmetic more than takes.  tcgen05 wants 64 rows or more,
// of which there are at most 16 here.
//
// Weights enter the second product as two bf16 terms (w = hi + lo, 16 bits), so that nothing is lost
// beside the fp32 sums.
//
// The stages of all items (a batch row's KV head with up to 16 of its query heads) form one line, and
// every CTA takes an equal stretch of it: a window makes items short, and splits of a fixed length then
// either leave SMs without work or pay the start of the pipeline too often.  The producer warp runs on
// into the next item while the others write the last one's state away, so the ring never drains.
//
// Measured (GB300, graph, d = 128): 32 requests of 8 KV heads with 4 query heads each, windows of 4096 keys
// 84 to 85 us (6.2 TB/s, 93% of the measured copy; the CUDA cores in splits of 512 keys took 164, in
// equal stretches 107), the same without a window, 1k to 32k keys, 330 us (6.9 TB/s; fa_decode 355); 8 query heads a KV
// head 101 us (fa_decode 239).
//
// Where items are short and at most two per SM (kDirectItems), each is one CTA's, which writes the results
// itself: one launch, no workspace and no line to sum up (16 requests of 512 keys with 8 KV heads 7.8 us
// against 14.3).
//
// The state of an item's stretch goes to slot (CTA + item), which no other stretch has: along the
// line one of the two grows with every stretch.  The join adds an item's states by the rescale rule.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "fa_internal.h"
#include "fa_score.cuh"
#include "fa_scored.h"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kComputeWarps = 8;
constexpr int kThreads = (kComputeWarps + 1) * 32;  // + 1 producer warp
// Keys of a stage: 32 KB each of keys and values.
template <int D>
constexpr int kStageKeys = D == 128 ? 128 : 256;
constexpr int kStages = 3;
constexpr int kMaxHeads = 16;

enum : unsigned int { kSiteFull = 1, kSiteEmpty = 2, kSiteDrain = 3 };

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

template <int D>
struct Smem {
  static constexpr int NB = 2;          // boxes of a stage: column blocks (d = 128) or row blocks
  static constexpr int kBox = 128 * 64;  // elements of a 128-row x 64-column box
  __nv_bfloat16 k[kStages][NB][kBox];           // 128-byte swizzle
  __nv_bfloat16 v[kStages][NB][kBox];
  float red_o[kComputeWarps][8][D];
  float red_m[kComputeWarps][kMaxHeads];
  float red_l[kComputeWarps][kMaxHeads];
  uint64_t full[kStages];
  uint64_t empty[kStages];
  long long scan[kComputeWarps + 1];
  long long before;  // stages of the line before the CTA's first batch row
  int first_b;
  int abort_flag;
};

// Byte offset of 16-byte chunk c of row r in a tile of boxes (128-byte swizzle).
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  const int box = D == 128 ? c >> 3 : r >> 7;
  return static_cast<uint32_t>(box * (Smem<D>::kBox * 2) + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void ldsm4(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

// c += a b: a 16 x 16 (rows: heads), b 16 x 8.
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Visible keys [x, y) of batch row b.
__device__ __forceinline__ int2 visible_keys(const ScoredDecodeParams& p, int b) {
  const int n = max(0, min(p.seqlens[b], p.Sk_max));
  int first = p.k_start ? max(0, p.k_start[b]) : 0;
  if (p.window > 0) first = max(first, n - p.window);
  return make_int2(min(first, n), n);
}

template <int D>
__device__ __forceinline__ int stages_of(int2 seen) {
  return static_cast<int>((static_cast<unsigned>(seen.y - seen.x) + kStageKeys<D> - 1) / kStageKeys<D>);
}

// A place in the line: batch row, item within it, stage within the item.
struct Walk {
  int b, sub, stage, n_stages;  // n_stages: of the item
  int2 seen;
  long long left;               // stages of the CTA's stretch from here on
};

template <int D>
__device__ __forceinline__ void enter_row(const ScoredDecodeParams& p, Walk& w) {
  do {
    w.seen = visible_keys(p, w.b);
    w.n_stages = stages_of<D>(w.seen);
  } while (w.n_stages == 0 && ++w.b < p.B);
}

// To the next item behind `n` stages of this one.
template <int D>
__device__ __forceinline__ void pass(const ScoredDecodeParams& p, Walk& w, int n) {
  w.left -= n;
  w.stage += n;
  if (w.stage < w.n_stages) return;
  w.stage = 0;
  if (++w.sub == p.subs) {
    w.sub = 0;
    ++w.b;
    if (w.left > 0) enter_row<D>(p, w);
  }
}

// Query heads of an item: the first, and how many.
__device__ __forceinline__ int2 heads_of(const ScoredDecodeParams& p, const Walk& w) {
  const int n_hsub = p.subs / p.Hkv;
  const int hk = w.sub / n_hsub, h_in = (w.sub - hk * n_hsub) * p.heads;
  return make_int2(hk * p.group + h_in, min(p.heads, p.group - h_in));
}

// O = 0, LSE = -inf of an item without keys.
template <int D>
__device__ __forceinline__ void write_empty(const ScoredDecodeParams& p, const Walk& w) {
  const int2 hq = heads_of(p, w);
  const size_t row = static_cast<size_t>(w.b) * p.Hq + hq.x;
  for (int i = threadIdx.x; i < hq.y * D; i += kThreads)
    reinterpret_cast<__nv_bfloat16*>(p.o)[row * D + i] = __float2bfloat16_rn(0.f);
  if (p.lse && static_cast<int>(threadIdx.x) < hq.y) p.lse[row + threadIdx.x] = neg_inf();
}

// One vote and barrier of the compute warps.
__device__ __forceinline__ bool compute_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}

// HALVES: 1 for up to 8 heads (the lower half of the rows is empty), 2 for up to 16.
template <int D, int HALVES>
__global__ void __launch_bounds__(kThreads, 1)
    fa_decode_scored_partial(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                             const ScoredDecodeParams p) {
  constexpr int NB = Smem<D>::NB;
  constexpr uint32_t kTileBytes = NB * Smem<D>::kBox * 2;
  extern __shared__ unsigned char smem_raw[];
  Smem<D>& s = *reinterpret_cast<Smem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], kComputeWarps);
    }
    s.abort_flag = 0;
    s.first_b = p.B;
    fence_barrier_init();
  }
  Walk w;
  if (p.direct) {
    w.b = static_cast<int>(blockIdx.x) / p.subs;
    w.sub = static_cast<int>(blockIdx.x) - w.b * p.subs;
    w.seen = visible_keys(p, w.b);
    w.n_stages = stages_of<D>(w.seen);
    w.stage = 0;
    w.left = w.n_stages;
    __syncthreads();
    if (w.left == 0) {  // (CTA-uniform)
      write_empty<D>(p, w);
      return;
    }
  } else {
    // ---- the line: stages of every batch row, summed kThreads rows at a time; twice (unless the
    //      rows fit one time), since the CTA's stretch follows from the total
    long long before = 0;  // stages (of one item a row) of the rows so far
    int mine = 0;          // stages of this thread's row, and of all up to it
    long long upto = 0;
    auto sum_rows = [&](int b0) {
      const int b = b0 + static_cast<int>(threadIdx.x);
      mine = b < p.B ? stages_of<D>(visible_keys(p, b)) : 0;
      long long sum = mine;
  #pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      __syncthreads();  // the last time's sums have been read
      if (lane == 31) s.scan[warp] = sum;
      __syncthreads();
      long long base = 0, all = 0;
  #pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) base += s.scan[i];
        all += s.scan[i];
      }
      upto = before + base + sum;
      before += all;
    };
    for (int b0 = 0; b0 < p.B; b0 += kThreads) sum_rows(b0);
    const long long total = before * p.subs;
    const long long share = total / gridDim.x, extra = total - share * gridDim.x, c = blockIdx.x;
    const long long from = c * share + min(c, extra), to = from + share + (c < extra ? 1 : 0);
    if (from == to) return;  // (CTA-uniform) nothing for this CTA
    auto find = [&](int b0) {
      const long long lo = (upto - mine) * p.subs;
      if (mine > 0 && from >= lo && from < upto * p.subs) {
        s.first_b = b0 + static_cast<int>(threadIdx.x);
        s.before = lo;
      }
    };
    if (p.B <= kThreads) {
      find(0);
    } else {
      before = 0;
      for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        sum_rows(b0);
        find(b0);
      }
    }
    __syncthreads();
    w.b = s.first_b;
    w.seen = visible_keys(p, w.b);
    w.n_stages = stages_of<D>(w.seen);
    w.left = to - from;
    {
      const long long r = from - s.before;
      w.sub = static_cast<int>(r / w.n_stages);
      w.stage = static_cast<int>(r - static_cast<long long>(w.sub) * w.n_stages);
    }
  }
  volatile int* abort_flag = &s.abort_flag;
  const int n_hsub = p.subs / p.Hkv;

  if (warp == kComputeWarps) {
    // ------------------------------------------------------------ producer --
    if (lane == 0) {
      int g = 0;  // stages across items
      bool ok = true;
      while (ok && w.left > 0) {
        const int n = static_cast<int>(min(w.left, static_cast<long long>(w.n_stages - w.stage)));
        const int hk = w.sub / n_hsub;
        for (int st = w.stage; st < w.stage + n; ++st, ++g) {
          const int slot = g % kStages, use = g / kStages;
          if (use > 0 && !mbar_wait(&s.empty[slot], (use - 1) & 1, abort_flag, kSiteEmpty)) {
            ok = false;
            break;
          }
          const int key = w.seen.x + st * kStageKeys<D>;  // rows past the cache arrive as zeros
          mbar_arrive_expect_tx(&s.full[slot], 2 * kTileBytes);
          for (int i = 0; i < NB; ++i)
            tma_load_3d(s.k[slot][i], &tk, &s.full[slot], D == 128 ? i * 64 : 0,
                        D == 128 ? key : key + i * 128, w.b * p.Hkv + hk);
          for (int i = 0; i < NB; ++i)
            tma_load_3d(s.v[slot][i], &tv, &s.full[slot], D == 128 ? i * 64 : 0,
                        D == 128 ? key : key + i * 128, w.b * p.Hkv + hk);
        }
        pass<D>(p, w, n);
      }
      if (*abort_flag)
        for (int i = max(0, g - kStages); i < g; ++i)
          mbar_drain(&s.full[i % kStages], (i / kStages) & 1, kSiteDrain);
    }
    __syncwarp();
    griddep_launch_dependents();
    return;
  }
  // --------------------------------------------------------------- compute --
  const int hr = lane >> 2, kc = lane & 3;  // this lane's heads hr, hr + 8; keys 2 kc, 2 kc + 1 (+ 8)
  // Queries as the first product's rows (heads that are not there are 0) and the bias per head of an
  // item: loaded before the last item's state is written, which hides their latency.
  uint32_t qa[D / 16][4];
  float slope2[HALVES];
  auto load_queries = [&](const Walk& at) {
    const int2 hq = heads_of(p, at);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int h = hr + 8 * half;
      const uint32_t* row = reinterpret_cast<const uint32_t*>(p.q) +
                            (static_cast<size_t>(at.b) * p.Hq + hq.x + h) * (D / 2);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const bool have = half < HALVES && h < hq.y;
        qa[ks][half] = have ? __ldg(row + ks * 8 + kc) : 0u;
        qa[ks][half + 2] = have ? __ldg(row + ks * 8 + 4 + kc) : 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < HALVES; ++u)
      slope2[u] = p.sc.slopes && hr + 8 * u < hq.y
                      ? __ldg(p.sc.slopes + hq.x + hr + 8 * u) * 1.4426950408889634f : 0.f;
  };
  load_queries(w);
  int g = 0;
  bool ok = true;
  while (w.left > 0) {
    const int n = static_cast<int>(min(w.left, static_cast<long long>(w.n_stages - w.stage)));
    const int hq0 = heads_of(p, w).x, n_heads = heads_of(p, w).y;
    float m[HALVES], l[HALVES];  // per head: running max of z, denominator
#pragma unroll
    for (int u = 0; u < HALVES; ++u) {
      m[u] = neg_inf();
      l[u] = 0.f;
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

    for (int st = w.stage; ok && st < w.stage + n; ++st, ++g) {
      const int slot = g % kStages;
      if (!mbar_wait_warp(&s.full[slot], (g / kStages) & 1, abort_flag, kSiteFull)) {
        ok = false;
        break;
      }
      const uint32_t kb = smem_u32(s.k[slot][0]), vb = smem_u32(s.v[slot][0]);
#pragma unroll 1
      for (int r0 = warp * 16; r0 < kStageKeys<D>; r0 += kComputeWarps * 16) {
        const int key0 = w.seen.x + st * kStageKeys<D> + r0;
        const int n_keys = w.seen.y - key0;  // of the warp's 16
        if (n_keys < 16) {
          // what lies behind the last key may be anything, and a weight of 0 does not cancel a NaN
          for (int i = lane; i < 16 * (D / 8); i += 32) {
            const int row = i / (D / 8);
            if (row >= n_keys)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                               vb + chunk_at<D>(r0 + row, i % (D / 8))),
                           "r"(0)
                           : "memory");
          }
          fence_proxy_async_smem();  // before the stage is filled again
          __syncwarp();
        }
        // ---- scores of 16 keys: two tiles of 8 ----
        float sc[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t b[4];
            ldsm4(kb + chunk_at<D>(r0 + nt * 8 + (lane & 7), 4 * q + (lane >> 3)), b);
            mma_bf16(sc[nt], qa[2 * q], b[0], b[1]);
            mma_bf16(sc[nt], qa[2 * q + 1], b[2], b[3]);
          }
        }
        // ---- z, in units of log2(e) ----
        if (p.capped) {
          float most = 0.f;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2 * HALVES; ++e) most = fmaxf(most, fabsf(sc[nt][e]));
          if (__all_sync(0xffffffffu, most <= p.sc.small[1])) {
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < 2 * HALVES; ++e) sc[nt][e] = cap_small(sc[nt][e], p.sc);
          } else if (p.sc.wide) {
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < 2 * HALVES; ++e) sc[nt][e] = cap_wide(sc[nt][e], p.sc);
          } else {
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < 2 * HALVES; ++e) sc[nt][e] = cap_any(sc[nt][e], p.sc);
          }
        } else {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2 * HALVES; ++e) sc[nt][e] *= p.scale_log2;
        }
        float mx[HALVES];
#pragma unroll
        for (int u = 0; u < HALVES; ++u) {
          mx[u] = neg_inf();
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = nt * 8 + 2 * kc + e;
              float& z = sc[nt][2 * u + e];
              z = fmaf(slope2[u], static_cast<float>(key0 + key - (w.seen.y - 1)), z);
              if (key >= n_keys) z = neg_inf();
              mx[u] = fmaxf(mx[u], z);
            }
          mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
          mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
        }
        // ---- online softmax, per head ----
        bool grow = false;
        float alpha[HALVES];
#pragma unroll
        for (int u = 0; u < HALVES; ++u) {
          // m_new - m is formed only once m is finite: -inf - (-inf) is never evaluated
          const bool first = m[u] == neg_inf() && mx[u] != neg_inf();
          const bool up = first || (m[u] != neg_inf() && mx[u] > m[u]);
          alpha[u] = first ? 0.f : up ? ex2_approx(m[u] - mx[u]) : 1.f;
          if (up) m[u] = mx[u];
          grow = grow || up;
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int u = 0; u < HALVES; ++u) {
            l[u] *= alpha[u];
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              o[i][2 * u] *= alpha[u];
              o[i][2 * u + 1] *= alpha[u];
            }
          }
        }
        uint32_t hi[4] = {0u, 0u, 0u, 0u}, lo[4] = {0u, 0u, 0u, 0u};  // weights as the second product's rows
#pragma unroll
        for (int u = 0; u < HALVES; ++u) {
          const float mc = m[u] == neg_inf() ? 0.f : m[u];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const float p0 = ex2_approx(sc[nt][2 * u] - mc), p1 = ex2_approx(sc[nt][2 * u + 1] - mc);
            l[u] += p0 + p1;
            const uint32_t w2 = pack_bf16x2(p0, p1);
            hi[2 * nt + u] = w2;
            lo[2 * nt + u] = pack_bf16x2(p0 - __uint_as_float(w2 << 16),
                                         p1 - __uint_as_float(w2 & 0xffff0000u));
          }
        }
        // ---- O += w V ----
#pragma unroll
        for (int i = 0; i < D / 8; i += 2) {
          uint32_t b[4];
          ldsm4_t(vb + chunk_at<D>(r0 + (lane & 15), i + (lane >> 4)), b);
          mma_bf16(o[i], hi, b[0], b[1]);
          mma_bf16(o[i + 1], hi, b[2], b[3]);
          mma_bf16(o[i], lo, b[0], b[1]);
          mma_bf16(o[i + 1], lo, b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.empty[slot]);
    }
    Walk next = w;
    pass<D>(p, next, n);
    if (next.left > 0) load_queries(next);
    // ---- the warps' states, 8 heads at a time, to the stretch's slot ----
    const int item = w.b * p.subs + w.sub;
    const size_t at = static_cast<size_t>(blockIdx.x) + item;
    if (threadIdx.x == 0 && !p.direct) {
      if (w.stage == 0) p.span[item].x = blockIdx.x;
      if (w.stage + n == w.n_stages) p.span[item].y = blockIdx.x;
    }
#pragma unroll
    for (int u = 0; u < HALVES; ++u) {
      l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
      l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
      if (kc == 0) {
        s.red_m[warp][hr + 8 * u] = m[u];
        s.red_l[warp][hr + 8 * u] = l[u];
      }
    }
    bool leave = false;
#pragma unroll
    for (int u = 0; u < HALVES; ++u) {
      if (u > 0 && compute_any(false)) leave = true;  // the first half's sums have been read
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(&s.red_o[warp][hr][i * 8 + 2 * kc]) =
            make_float2(o[i][2 * u], o[i][2 * u + 1]);
      if (compute_any(!ok || *abort_flag)) leave = true;
      for (int idx = threadIdx.x; idx < min(8, n_heads - 8 * u) * D; idx += kComputeWarps * 32) {
        const int hh = idx / D, e = idx % D, h = hh + 8 * u;
        float M = neg_inf();
#pragma unroll
        for (int i = 0; i < kComputeWarps; ++i) M = fmaxf(M, s.red_m[i][h]);
        float L = 0.f, acc = 0.f;
#pragma unroll
        for (int i = 0; i < kComputeWarps; ++i) {
          const float wt = (s.red_m[i][h] == neg_inf()) ? 0.f : ex2_approx(s.red_m[i][h] - M);
          L = fmaf(wt, s.red_l[i][h], L);
          acc = fmaf(wt, s.red_o[i][hh][e], acc);
        }
        // (a NaN in a visible key makes L one, which is not 0: it reaches O and LSE)
        const float out = L != 0.f ? acc / L : 0.f, lse2 = L != 0.f ? M + __log2f(L) : neg_inf();
        if (p.direct) {
          const size_t row = static_cast<size_t>(w.b) * p.Hq + hq0 + h;
          reinterpret_cast<__nv_bfloat16*>(p.o)[row * D + e] = __float2bfloat16_rn(out);
          if (p.lse && e == 0) p.lse[row] = lse2 * 0.69314718055994530942f;
        } else {
          p.part_o[(at * p.heads + h) * D + e] = out;
          if (e == 0) p.part_lse[at * p.heads + h] = lse2;
        }
      }
    }
    if (leave) break;  // every compute warp leaves together
    w = next;
    if (w.left > 0 && compute_any(*abort_flag)) break;  // the sums have been read
  }
  griddep_launch_dependents();
}

// One CTA per (batch row, query head), one thread per output element.
template <int D>
__global__ void __launch_bounds__(D) fa_decode_scored_join(const ScoredDecodeParams p) {
  const int bh = blockIdx.x;
  const int b = bh / p.Hq, h = bh - b * p.Hq;
  const int e = threadIdx.x;
  const int hk = h / p.group, hg = h - hk * p.group;
  const int n_hsub = p.subs / p.Hkv;
  const int item = b * p.subs + hk * n_hsub + hg / p.heads;
  const int2 seen = visible_keys(p, b);
  griddep_wait();  // the partial kernel's results are complete and visible
  float M = neg_inf(), wsum = 0.f, o = 0.f;
  if (seen.y > seen.x) {
    const int2 span = p.span[item];
    const size_t row0 = (static_cast<size_t>(span.x) + item) * p.heads + hg % p.heads;
    const int n = span.y - span.x + 1;
    for (int i = 0; i < n; ++i) M = fmaxf(M, p.part_lse[row0 + static_cast<size_t>(i) * p.heads]);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const size_t row = row0 + static_cast<size_t>(i) * p.heads;
      const float ls = p.part_lse[row];
      const float wt = (ls == neg_inf()) ? 0.f : ex2_approx(ls - M);
      wsum += wt;
      o = fmaf(wt, p.part_o[row * D + e], o);
    }
  }
  const bool live = wsum != 0.f;  // (NaN is live)
  reinterpret_cast<__nv_bfloat16*>(p.o)[static_cast<size_t>(bh) * D + e] =
      __float2bfloat16_rn(live ? o / wsum : 0.f);
  if (p.lse && e == 0)
    p.lse[bh] = live ? (M + __log2f(wsum)) * 0.69314718055994530942f : neg_inf();
}

template <int D, int HALVES>
cudaError_t launch_dh(const CUtensorMap& tk, const CUtensorMap& tv, const ScoredDecodeParams& p,
                      int ctas, cudaStream_t stream) {
  constexpr size_t smem = sizeof(Smem<D>) + 1024;
  static_assert(smem <= 232448, "decode shared memory exceeds the per-CTA limit");
  // per-device kernel attribute: set on every call for the current device
  cudaError_t e = cudaFuncSetAttribute(fa_decode_scored_partial<D, HALVES>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  hook_before(stream);
  fa_decode_scored_partial<D, HALVES><<<ctas, kThreads, smem, stream>>>(tk, tv, p);
  hook_after(stream);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const CUtensorMap& tk, const CUtensorMap& tv, const ScoredDecodeParams& p,
                     int ctas, cudaStream_t stream) {
  cudaError_t e = p.heads <= 8 ? launch_dh<D, 1>(tk, tv, p, ctas, stream)
                               : launch_dh<D, 2>(tk, tv, p, ctas, stream);
  if (e != cudaSuccess || p.direct) return e;
  return launch_dependent(fa_decode_scored_join<D>, dim3(p.B * p.Hq), dim3(D), 0, stream, p);
}

constexpr int kMaxCtas = 256;  // one per SM, and what the workspace has slots for
// Items that are one CTA's each.  8 to 304 items of 1 or 2 stages took 4.4 to 10.9 us and in a line
// 6.8 to 14.7; 32 to 304 items of up to 8 stages 7 to 28 and 8 to 32; fewer items of 4 stages 7.6
// and 7.0; more items 5% more.
constexpr int kDirectItems = 304, kDirectStages = 8, kDirectFewStages = 2, kDirectMany = 32;

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

DecodeScoredPlan decode_scored_plan(int B, int Hq, int Hkv, int Sk_max, int d, int window) {
  DecodeScoredPlan r{};
  const int group = std::max(1, Hq / std::max(1, Hkv));
  r.heads = std::min(group, kMaxHeads);
  r.subs = Hkv * ((group + r.heads - 1) / r.heads);
  const long long keys = window > 0 ? std::min(window, Sk_max) : Sk_max;
  const long long items = static_cast<long long>(B) * r.subs;
  const int stage = d == 128 ? kStageKeys<128> : kStageKeys<64>;
  const long long stages = (keys + stage - 1) / stage;
  if (items <= kDirectItems && stages <= (items >= kDirectMany ? kDirectStages : kDirectFewStages)) {
    r.direct = true;
    r.ctas = static_cast<int>(items);
    return r;
  }
  const long long line = items * ((keys + 127) / 128);
  r.ctas = static_cast<int>(std::min<long long>(line, kMaxCtas));
  r.slots = static_cast<size_t>(items + r.ctas);
  r.span_bytes = up256(static_cast<size_t>(items) * sizeof(int2));
  r.o_bytes = up256(r.slots * r.heads * d * sizeof(float));
  r.lse_bytes = up256(r.slots * r.heads * sizeof(float));
  return r;
}

cudaError_t launch_decode_scored(int d, const CUtensorMap& tk, const CUtensorMap& tv,
                                 const ScoredDecodeParams& p, const DecodeScoredPlan& plan,
                                 cudaStream_t stream) {
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int ctas = plan.direct ? plan.ctas : std::min(plan.ctas, n_sm);
  return d == 128 ? launch_d<128>(tk, tv, p, ctas, stream) : launch_d<64>(tk, tv, p, ctas, stream);
}

unsigned int read_decode_scored_status(bool clear) {
  unsigned int v = 0;
  cudaMemcpyFromSymbol(&v, g_status, sizeof v);
  if (clear) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_status, &z, sizeof z);
  }
  return v;
}

}  // namespace fa
