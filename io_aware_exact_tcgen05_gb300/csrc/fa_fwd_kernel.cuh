// fa_fwd_kernel.cuh -- forward attention kernel for sm_103a (tcgen05 + TMEM + TMA), compiled for plain,
// masked and dropped weights in fa_fwd.cu and for capped and biased scores in fa_fwd_scored.cu.
//
// One CTA owns two 128-row query tiles ("slots") that share every key/value
// tile it streams: either two query heads of one KV group at the same rows
// (grouped heads: K/V tiles are fetched once per KV head for both), or two
// consecutive row blocks of one head.  Per key/value tile j:
//
//   S_t = Q_t K_j^T          tcgen05.mma, A and B from shared memory, fp32 in TMEM
//   softmax warps of slot t  tcgen05.ld S_t (one TMEM lane = one query row = one
//                            thread), mask, row max, conditional rescale of O_t,
//                            p = 2^(s*c - m*c), row sum, P_t -> bf16 into the
//                            TMEM columns of S_t
//   O_t += P_t V_j           tcgen05.mma, A (P) from TMEM, B (V) from shared memory
//
// The two slots ping-pong: while the softmax warps of one slot work, the
// tensor core runs the other slot's MMAs.  The S x S matrix never leaves
// TMEM/registers; O is divided by l once at the end and the per-row
// logsumexp is written beside it.
//
// Method: "Flash Attention" history page 1.2 (running max, denominator and
// rescaled output), 1.3 (tiles discarded on chip), 2.1 (query-sequence
// parallelism, fully masked causal tiles skipped), 2.3 (asynchronous MMA and
// skipping the rescale while the running max does not grow); FlashAttention_01
// page, online-softmax derivation (m, l, u; mask before the max; empty rows).
//
// Warp roles (320 threads): warps 0-3 softmax of slot 0, warps 4-7 softmax of
// slot 1 (a warp may only touch TMEM lanes 32*(warp%4) .. +31, which are the
// rows it owns), warp 8 TMA producer, warp 9 MMA issuer and TMEM owner.  (Scored
// modes, 384 threads: warp 10 clears values that no row sees, warp 11 lends its registers.)
//
// The kernel is persistent: one CTA per SM walks a fixed sequence of work
// units (the heavy-first list, taken in alternating directions block by
// block so heavy and light units pair up).  Barrier phases run on across
// units; the next unit's Q is loaded once the current unit's last S product
// has read Q, its first S products overlap the current epilogue, and its
// first PV into O waits only until the epilogue has read O.
#pragma once

#include <algorithm>
#include <limits>
#include <type_traits>

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <math.h>

#include "fa_internal.h"
#include "fa_philox.cuh"
#include "fa_score.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 320;
constexpr uint32_t kTmemCols = 512;

// wait-site ids reported in the status word
enum : unsigned int {
  kSiteQ = 1, kSiteKFree, kSiteVFree, kSiteKFull, kSiteVFull, kSitePFull, kSiteSFull,
  kSiteOFull, kSiteDrain, kSiteVRaw, kSitePlan
};

template <int D>
struct FwdSmem {
  static constexpr int NB = D / 64;               // 64-wide (128-byte) column blocks per row
  static constexpr int NS = FwdTiles<D>::kKvStages;  // K and V pipeline depth
  static constexpr int kBox = kTileM * 64;        // elements per 128-row x 64-col box
  __nv_bfloat16 q[2][NB][kBox];
  __nv_bfloat16 k[NS][NB][kBox];
  __nv_bfloat16 v[NS][NB][kBox];
  uint64_t bar_q;
  uint64_t q_free;             // the unit's last S product has read Q
  uint64_t k_full[NS], v_full[NS];
  // kv_free[g % NS] completes a phase when the round issuing S of tile g
  // (g counts tiles across the CTA's units) has finished.  That round also
  // finishes PV of tile g - 1, whether it belongs to the same unit or closes
  // the previous one (a commit covers every earlier MMA), so it frees K
  // stage g % NS and V stage (g - 1) % NS: one commit per tile.
  uint64_t kv_free[NS];
  uint64_t o_empty[2];          // the slot's softmax warps have read O
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t drain;  // MMA teardown after an abort
  uint64_t v_raw[NS];  // scored modes: V of an edge tile has arrived (see edge_tile)
  uint32_t tmem_base;
  int abort_flag;
};

template <int D>
constexpr size_t fwd_smem_bytes() {
  return sizeof(FwdSmem<D>) + 1024;  // + alignment slack
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
// In place of a part's LSE (which is never +inf): the row's unit was too short to split, and wrote the results.
constexpr float kWhole = std::numeric_limits<float>::infinity();

// Fast-path bound on a row's fp32 tile sum: every weight stays below 2^64,
// so P, l and O (at most 2^64 per tile per key block) stay far from fp32
// overflow while the running max is left as it is.
constexpr float kFastLimit = 18446744073709551616.0f;  // 2^64
constexpr float kFastLog2 = 56.f;  // the same for 128 weights bounded one by one, with room to spare

// Scores of keys outside [klo, khi) become -inf (weight 0).
template <int FIRST, int COUNT>
__device__ __forceinline__ void mask_scores(uint32_t (&sr)[kTileN], int c0, int klo, int khi) {
#pragma unroll
  for (int jj = FIRST; jj < FIRST + COUNT; ++jj) {
    const int key = c0 + jj;
    if (key < klo || key >= khi) sr[jj] = 0xff800000u;
  }
}

// Scores of keys whose visibility bit is clear become -inf; bit jj of the
// 128-bit word group kb stands for key c0 + jj.
template <int FIRST, int COUNT>
__device__ __forceinline__ void mask_key_bits(uint32_t (&sr)[kTileN], uint4 kb) {
  const uint32_t w[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
  for (int jj = FIRST; jj < FIRST + COUNT; ++jj)
    if (!((w[jj >> 5] >> (jj & 31)) & 1u)) sr[jj] = 0xff800000u;
}

// Weights 2^(s*c - mc) of the 64 scores sr[64*HALF, +64) (nmc2 holds -mc
// twice), rounded to bf16 pairs and stored to TMEM columns [32*HALF, +32)
// from t_p.  sum2 gathers the fp32 weights (for l); sr_lo/sr_hi gather the
// rounded ones (for lr).  With DROP, the stored words of dropped weights are
// cleared after the sums (l, lr and the LSE stay those of the undropped
// softmax); bit jj of keep[jj / 32] says whether key jj of the tile is kept.
template <int HALF, bool DROP>
__device__ __forceinline__ void softmax_half(const uint32_t (&sr)[kTileN], uint64_t c2,
                                             uint64_t nmc2, uint32_t t_p, uint64_t (&sum2)[4],
                                             float (&sr_lo)[4], float (&sr_hi)[4],
                                             const uint32_t (&keep)[4]) {
  uint32_t pk[kTileN / 4];
#pragma unroll
  for (int jq = 0; jq < kTileN / 4; ++jq) {
    const int jj = HALF * (kTileN / 4) + jq;
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[2 * jj]), __uint_as_float(sr[2 * jj + 1])), c2,
                     nmc2),
              x0, x1);
    const float p0 = ex2_approx(x0);
    const float p1 = ex2_approx(x1);
    pk[jq] = pack_bf16x2(p0, p1);
    sum2[jq & 3] = f2_add(sum2[jq & 3], f2_pack(p0, p1));
    add_bf16x2_f32(sr_lo[jq & 3], sr_hi[jq & 3], pk[jq]);
    if (DROP) {
      const int kj = HALF * (kTileN / 2) + 2 * jq;  // the pair's first key in the tile
      const uint32_t kb = keep[kj >> 5] >> (kj & 31);
      pk[jq] &= ((kb & 1u) ? 0x0000ffffu : 0u) | ((kb & 2u) ? 0xffff0000u : 0u);
    }
  }
  tmem_st32(t_p + HALF * 32, pk);
}

__device__ __forceinline__ float sum_f2x4(const uint64_t (&v)[4]) {
  float a, b;
  f2_unpack(f2_add(f2_add(v[0], v[1]), f2_add(v[2], v[3])), a, b);
  return a + b;
}

// Kernel modes: the plain path carries no mask or dropout code at all.  Scored modes (capped
// and biased scores, row intervals of a mask plan) are kModeScored, with kModeCap and kModeBias.
enum : int {
  kModePlain = 0, kModeKeyBits = 1, kModeDropout = 2,
  kModeCap = 4, kModeBias = 8, kModeScored = 16,
  kModeWide = 32  // with kModeCap: a cap above kWideCap.  (As a branch of kModeCap: 3% on documents under a cap of 30.)
};

struct ScoredFwdParams : FwdParams {
  ScoreArgs sc;
  FwdSplit split;
};
template <int MODE>
using FwdParamsOf = std::conditional_t<(MODE & kModeScored) != 0, ScoredFwdParams, FwdParams>;

// One work unit: two 128-row query tiles ("slots") and the key tiles they
// see.  Units are numbered heavy (late) row blocks first; every role of a
// CTA walks the same unit sequence, so their barrier phases stay in step.
struct Unit {
  int b, h0, h1, r0, r1;
  int sq, qb, bz;        // logical rows [0, sq) from packed row qb of tensor batch bz
  int klo, kend, off;    // visible key interval and bottom-right causal offset
  int hk, j0, n_tiles;
  bool rows, active1;    // rows: slot 0 has rows at all
};

constexpr int kPartTiles = 5;  // least tiles of a part of a split unit

// In the scored modes a slot takes part in the rounds (last tiles first) whose tile its rows see.
struct ScoredUnit : Unit {
  int part, parts;                 // of the unit's tiles (FwdSplit)
  int begin0, end0, begin1, end1;  // rounds of slots 0 and 1
  __device__ __forceinline__ int begin(int t) const { return t ? begin1 : begin0; }
  __device__ __forceinline__ int end(int t) const { return t ? end1 : end0; }
};

__device__ __forceinline__ Unit unit_at(const FwdParams& p, int U) {
  Unit u;
  const int rbu = p.n_rbu - 1 - U / p.units_per_rbu;
  const int w = U % p.units_per_rbu;
  if (p.pack_heads) {
    const int hpairs = p.Hq >> 1;
    u.b = w / hpairs;
    u.h0 = 2 * (w % hpairs);
    u.h1 = u.h0 + 1;
    u.r0 = u.r1 = rbu * kTileM;
  } else {
    u.b = w / p.Hq;
    u.h0 = u.h1 = w % p.Hq;
    u.r0 = rbu * 2 * kTileM;
    u.r1 = u.r0 + kTileM;
  }
  u.sq = p.Sq;
  u.qb = 0;
  u.bz = u.b;
  if (p.cu_q) {  // packed ragged: b is the sequence
    u.qb = max(0, min(p.cu_q[u.b], p.Sq));
    u.sq = max(0, min(p.cu_q[u.b + 1], p.Sq) - u.qb);
    u.klo = max(0, min(p.cu_k[u.b], p.Sk));
    u.kend = max(u.klo, min(p.cu_k[u.b + 1], p.Sk));
    u.off = u.kend - u.sq;  // bottom-right causal alignment within the sequence
    u.bz = 0;
  } else {
    u.klo = p.k_start ? p.k_start[u.b] : 0;
    u.kend = p.k_end ? p.k_end[u.b] : p.Sk;
    u.klo = max(0, min(u.klo, p.Sk));
    u.kend = max(0, min(u.kend, p.Sk));
    u.off = p.Sk - p.Sq;  // bottom-right causal alignment
  }
  u.rows = u.r0 < u.sq;
  u.active1 = u.r1 < u.sq;
  u.hk = u.h0 / p.group;
  int khi = u.kend;
  if (p.causal) {
    const int last_row = min((u.active1 ? u.r1 : u.r0) + kTileM - 1, u.sq - 1);
    khi = min(khi, last_row + u.off + 1);
  }
  u.j0 = 0;
  u.n_tiles = 0;
  if (u.rows && khi > u.klo) {
    u.j0 = u.klo / kTileN;
    u.n_tiles = (khi + kTileN - 1) / kTileN - u.j0;
  }
  return u;
}

// The scored modes' units: with a plan the row blocks come in the plan's order (most key tiles
// first), and a slot visits the tiles of its rows' hull.
__device__ __forceinline__ ScoredUnit unit_at(const ScoredFwdParams& p, int U) {
  ScoredUnit u;
  u.part = 0;
  u.parts = 1;
  if (p.split.n > 1) {  // parts of a unit are neighbours
    u.part = U % p.split.n;
    U /= p.split.n;
  }
  const MaskPlan& m = p.sc.plan;
  const int heads = p.pack_heads ? p.Hq >> 1 : p.Hq;  // units of a batch row and row block
  int w, rbu;
  if (m.rows) {
    const int tile = __ldg((p.pack_heads ? m.by_q1 : m.by_q2) + U / heads);
    w = U % heads;
    u.b = tile / p.n_rbu;
    rbu = tile - u.b * p.n_rbu;
  } else {
    w = U % p.units_per_rbu;
    rbu = p.n_rbu - 1 - U / p.units_per_rbu;
    u.b = w / heads;
    w -= u.b * heads;
  }
  int lo0 = 0, hi0 = p.Sk, lo1 = 0, hi1 = p.Sk;  // hulls of the slots' rows
  if (p.pack_heads) {
    u.h0 = 2 * w;
    u.h1 = u.h0 + 1;
    if (m.rows) {
      const int4 r = __ldg(m.qt + static_cast<size_t>(u.b) * m.nq + rbu);
      lo0 = lo1 = r.x;
      hi0 = hi1 = r.y;
    }
    u.r0 = u.r1 = rbu * kTileM;
  } else {
    u.h0 = u.h1 = w;
    if (m.rows) {
      const int4* qt = m.qt + static_cast<size_t>(u.b) * m.nq + 2 * rbu;
      const int4 r = __ldg(qt);
      lo0 = r.x;
      hi0 = r.y;
      if (2 * rbu + 1 < m.nq) {
        const int4 r1 = __ldg(qt + 1);
        lo1 = r1.x;
        hi1 = r1.y;
      }
    }
    u.r0 = rbu * 2 * kTileM;
    u.r1 = u.r0 + kTileM;
  }
  u.sq = p.Sq;
  u.qb = 0;
  u.bz = u.b;
  u.off = p.Sk - p.Sq;
  u.rows = u.r0 < u.sq;
  u.active1 = u.r1 < u.sq;
  u.hk = u.h0 / p.group;
  if (p.causal) {
    hi0 = min(hi0, min(u.r0 + kTileM, u.sq) + u.off);
    hi1 = min(hi1, min(u.r1 + kTileM, u.sq) + u.off);
  }
  if (hi0 <= lo0) lo0 = 0x7fffffff, hi0 = 0;
  if (hi1 <= lo1 || !u.active1) lo1 = 0x7fffffff, hi1 = 0;
  u.klo = min(lo0, lo1);
  u.kend = max(hi0, hi1);
  u.j0 = u.n_tiles = u.begin0 = u.end0 = u.begin1 = u.end1 = 0;
  if (u.kend > 0) {
    const int end = (u.kend + kTileN - 1) / kTileN;
    u.j0 = u.klo / kTileN;
    u.n_tiles = end - u.j0;
    if (hi0 > 0) {
      u.begin0 = end - (hi0 + kTileN - 1) / kTileN;
      u.end0 = end - lo0 / kTileN;
    }
    if (hi1 > 0) {
      u.begin1 = end - (hi1 + kTileN - 1) / kTileN;
      u.end1 = end - lo1 / kTileN;
    }
    if (p.split.n > 1) {
      // equal parts of the rounds, of kPartTiles or more; those that are left over are empty
      const int n = u.n_tiles;
      u.parts = max(1, min(p.split.n, n / kPartTiles));
      const int from = u.part < u.parts ? n * u.part / u.parts : 0;
      const int to = u.part < u.parts ? n * (u.part + 1) / u.parts : 0;
      u.j0 += n - to;
      u.n_tiles = to - from;
      u.begin0 = max(u.begin0 - from, 0);
      u.end0 = max(min(u.end0, to) - from, u.begin0);
      u.begin1 = max(u.begin1 - from, 0);
      u.end1 = max(min(u.end1, to) - from, u.begin1);
    }
  }
  return u;
}

// Keys of the unit's tile j (last tiles first) that no row of the unit sees may hold anything, and a weight
// of 0 does not cancel a NaN.  Mostly only a unit's first and last tile have such keys; with a plan also those
// behind the first row's position where the causal rule cuts intervals, and any where its rows' intervals
// leave keys between them out (padding between documents).  V of such a tile is loaded for a helper warp,
// which makes zeros of those keys' values and then hands the stage on.
// (In the softmax warps or in the MMA warp the mere presence of this cost 3 to 5%.)
__device__ __forceinline__ bool edge_tile(const Unit& u, int j) {
  const int c0 = (u.j0 + u.n_tiles - 1 - j) * kTileN;
  return c0 < u.klo || c0 + kTileN > u.kend;
}

// The end of the keys from klo on that are each seen by some row of the unit: kend, unless the plan or the
// causal rule leaves some out.  (Apart from unit_at: there, in every warp, it cost 1%.)
__device__ __forceinline__ int all_seen_until(const ScoredUnit& u, const ScoredFwdParams& p) {
  if (!p.sc.plan.rows) return u.kend;
  const int t = u.r0 / kTileM;
  const int4* qt = p.sc.plan.qt + static_cast<size_t>(u.b) * p.sc.plan.nq + t;
  int4 r = __ldg(qt);
  if (p.causal) r.y = min(r.y, min(u.r0 + kTileM, u.sq) + u.off);
  if (!p.pack_heads && t + 1 < p.sc.plan.nq) {
    int4 r1 = __ldg(qt + 1);
    if (p.causal) r1.y = min(r1.y, min(u.r1 + kTileM, u.sq) + u.off);
    r.z |= r1.z | (r.y > r.x && r1.y > r1.x && (r.y < r1.x || r1.y < r.x));
    r.w = max(r.w, r1.w);
  }
  if (r.z) return 0;
  // The rule hides those up to the first row's position from no row; where all rows see their own, the hull, which
  // ends at the last row's, holds none that it hides from all.
  return p.causal && r.w == 2 ? min(u.kend, u.r0 + u.off + 1) : u.kend;
}

// Which keys of the tile from key c0 any row of the unit sees: lane w (and w + 4, ..) has those of keys
// [32 w, +32).  From the extremes of the unit's rows where they tell all (hull), else from those of each tile of rows and
// its gaps, and row by row where these are many or the causal rule cuts into the tile.
__device__ __forceinline__ uint32_t keys_seen(const ScoredUnit& u, const ScoredFwdParams& p, bool hull, int c0,
                                              int lane) {
  const int at = c0 + 32 * (lane & 3);
  auto span = [&](int lo, int hi) { return bits_below(hi - at) & ~bits_below(lo - at); };
  if (hull) return span(u.klo, u.kend);
  const MaskPlan& m = p.sc.plan;
  uint32_t mine = 0u;
  bool rows = false;
#pragma unroll 1
  for (int t = u.r0 / kTileM, end = min(m.nq, t + (p.pack_heads ? 1 : 2)); t < end; ++t) {
    const size_t i = static_cast<size_t>(u.b) * m.nq + t;
    const int4 r = __ldg(m.qt + i), g = __ldg(m.gaps + i);
    const int hi = p.causal ? min(r.y, min((t + 1) * kTileM, u.sq) + u.off) : r.y;
    mine |= span(r.x, max(r.x, hi)) & ~(span(g.x, g.y) | span(g.z, g.w));
    rows = rows || r.z == 3 || (p.causal && r.w == 2 && c0 + kTileN > t * kTileM + u.off + 1);
  }
  if (!rows) return mine;
  uint32_t seen[4] = {0u, 0u, 0u, 0u};
#pragma unroll 2
  for (int k = 0; k < (p.pack_heads ? 4 : 8); ++k) {  // (slots of packed heads have the same rows)
    const int i = u.r0 + 32 * k + lane;
    const int2 r = i < u.sq ? __ldg(m.rows + static_cast<size_t>(u.b) * p.Sq + i) : make_int2(0, 0);
    const int hi = p.causal ? min(r.y, i + u.off + 1) : r.y;
    if (hi > r.x) add_span(seen, r.x - c0, hi - c0);
  }
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    seen[w] = __reduce_or_sync(0xffffffffu, seen[w]);
    if ((lane & 3) == w) mine = seen[w];
  }
  return mine;
}

template <typename Smem>
__device__ __forceinline__ void edge_warp(Smem& s, const ScoredFwdParams& p, int lane, int n_units) {
  volatile int* abort_flag = &s.abort_flag;
  int g = 0;                    // tiles before the unit, as the producer counts them
  uint32_t uses[Smem::NS] = {};  // edge tiles each stage has held
  for (int k = 0; k * static_cast<int>(gridDim.x) < n_units; ++k) {
    const int G = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
    const int U = k * G + ((k & 1) ? (G - 1 - c) : c);
    if (U >= n_units) continue;
    ScoredUnit un = unit_at(p, U);
    const int until = all_seen_until(un, p);
    const bool hull = until == un.kend;  // which klo and kend tell all of
    un.kend = until;
    for (int j = 0; j < un.n_tiles; ++j) {
      if (!edge_tile(un, j)) continue;
      const int st = (g + j) % Smem::NS;
      const int c0 = (un.j0 + un.n_tiles - 1 - j) * kTileN;
      const uint32_t seen = keys_seen(un, p, hull, c0, lane);
#pragma unroll
      for (int i = 0; i < Smem::NS; ++i)
        if (i == st) {
          if (!mbar_wait_warp(&s.v_raw[i], uses[i] & 1, abort_flag, kSiteVRaw)) return;
          ++uses[i];
        }
      const uint32_t v0 = smem_u32(s.v[st][0]);
      for (int i = lane; i < kTileN * Smem::NB; i += 32) {  // box after box of 128-byte rows, a key each
        const uint32_t word = __shfl_sync(0xffffffffu, seen, i >> 5 & 3);
        if (word >> lane & 1) continue;
#pragma unroll
        for (int ch = 0; ch < 8; ++ch)
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v0 + i * 128 + ch * 16), "r"(0)
                       : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.v_full[st]);
    }
    g += un.n_tiles;
  }
}

// Scores of 64 keys (columns [64 HALF, +64) of the tile) straight to weights, for a tile that
// every row of the warp sees whole and whose distances have one sign: with a bias the exponent
// is s * c + (slope of the sign) * jj + bm, bm = the bias of the tile's first key less the maximum.
// The bias of a pair is stepped from that of the pair four before it, in 16 steps a half: off by
// some 2^-20 of itself.
template <int HALF, bool BIAS>
__device__ __forceinline__ void scored_half(const uint32_t (&sr)[kTileN], uint64_t c2, float sg,
                                            float bm, uint32_t t_p, uint64_t (&sum2)[4],
                                            float (&sr_lo)[4], float (&sr_hi)[4]) {
  uint32_t pk[kTileN / 4];
  uint64_t add2[4];
  const uint64_t step2 = f2_pack(8.f * sg, 8.f * sg);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    add2[q] = BIAS ? f2_pack(fmaf(sg, 64.f * HALF + 2 * q, bm), fmaf(sg, 64.f * HALF + 2 * q + 1, bm))
                   : f2_pack(bm, bm);
#pragma unroll
  for (int jq = 0; jq < kTileN / 4; ++jq) {
    const int jj = HALF * (kTileN / 4) + jq;
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[2 * jj]), __uint_as_float(sr[2 * jj + 1])), c2,
                     add2[jq & 3]),
              x0, x1);
    if (BIAS) add2[jq & 3] = f2_add(add2[jq & 3], step2);
    const float p0 = ex2_approx(x0);
    const float p1 = ex2_approx(x1);
    pk[jq] = pack_bf16x2(p0, p1);
    sum2[jq & 3] = f2_add(sum2[jq & 3], f2_pack(p0, p1));
    add_bf16x2_f32(sr_lo[jq & 3], sr_hi[jq & 3], pk[jq]);
  }
  tmem_st32(t_p + HALF * 32, pk);
}

// The same for 32 capped scores (columns [32 cc, +32)); DEGREE: of the cap's polynomial, or kCapAny.
constexpr int kCapAny = -1;
template <int DEGREE, bool BIAS>
__device__ __forceinline__ void capped_chunk(const uint32_t (&r)[32], const ScoreArgs& sc, float sg,
                                             float bm, uint32_t t_p, uint64_t (&sum2)[2],
                                             float (&sr_lo)[2], float (&sr_hi)[2]) {
  uint32_t pk[16];
  uint64_t add2[4];
  const uint64_t step2 = f2_pack(8.f * sg, 8.f * sg);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    add2[q] = BIAS ? f2_pack(fmaf(sg, 2.f * q, bm), fmaf(sg, 2.f * q + 1, bm)) : f2_pack(bm, bm);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const uint64_t s2 = f2_pack(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
    float x0, x1;
    if constexpr (DEGREE == kCapAny)
      f2_unpack(f2_add(cap_any2(s2, sc), add2[e & 3]), x0, x1);
    else
      f2_unpack(f2_fma(s2, cap_small_factor<DEGREE>(s2, sc), add2[e & 3]), x0, x1);
    if (BIAS) add2[e & 3] = f2_add(add2[e & 3], step2);
    const float p0 = ex2_approx(x0);
    const float p1 = ex2_approx(x1);
    pk[e] = pack_bf16x2(p0, p1);
    sum2[e & 1] = f2_add(sum2[e & 1], f2_pack(p0, p1));
    add_bf16x2_f32(sr_lo[e & 1], sr_hi[e & 1], pk[e]);
  }
  tmem_st16(t_p, pk);
}

// A whole tile of capped scores to weights, 32 columns at a time, last columns first (the weights
// of columns [32 cc, +32) go over those of [64 + 16 cc, +16), which have been read by then).  The next
// columns are loaded while these are worked on.  Adds to l and lr.  A loop and not one stretch of
// code: warps of one CTA may be in different degrees, and three unrolled ones do not fit the
// instruction cache (2 x 16 heads x 8192 causal, d = 128, scores that need degrees 4 and kCapAny
// in turn: 976 us unrolled, 640 as loops; degree 2 alone 518 us as a loop, 481 unrolled by 2).
template <int DEGREE, bool BIAS>
__device__ __forceinline__ void capped_tile(uint32_t t_s, uint32_t t_p, const ScoreArgs& sc, float sg,
                                            float bm, float& l, float& lr) {
  uint64_t sum2[2] = {0ull, 0ull};
  float sr_lo[2] = {0.f, 0.f}, sr_hi[2] = {0.f, 0.f};
  uint32_t ra[32], rb[32];
  tmem_ld32(t_s + 96, ra);
  tmem_wait_ld();
#pragma unroll (DEGREE == 2 ? 2 : 1)
  for (int cc = 3; cc >= 0; cc -= 2) {
    tmem_ld32(t_s + cc * 32 - 32, rb);
    capped_chunk<DEGREE, BIAS>(ra, sc, sg, fmaf(sg, 32.f * cc, bm), t_p + cc * 16, sum2, sr_lo, sr_hi);
    tmem_wait_ld();
    if (cc > 1) tmem_ld32(t_s + cc * 32 - 64, ra);
    capped_chunk<DEGREE, BIAS>(rb, sc, sg, fmaf(sg, 32.f * cc - 32.f, bm), t_p + cc * 16 - 16, sum2,
                               sr_lo, sr_hi);
    tmem_wait_ld();
  }
  float a, b;
  f2_unpack(f2_add(sum2[0], sum2[1]), a, b);
  l += a + b;
  lr += (sr_lo[0] + sr_lo[1]) + (sr_hi[0] + sr_hi[1]);
}

// 32 raw scores of a row (keys from column j0 of the tile) -> z in units of log2(e), hidden keys to
// -inf; p_rel, lo_rel, hi_rel: the row's position and its interval less the tile's first key.
template <bool CAP, bool WIDE, bool BIAS>
__device__ __forceinline__ void scored_transform(uint32_t (&r)[32], const ScoreArgs& sc, float c,
                                                 bool small, float slope2, int p_rel, int lo_rel,
                                                 int hi_rel) {
  if (CAP && !small) {
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float x = __uint_as_float(r[e]);
      r[e] = __float_as_uint(WIDE ? cap_wide(x, sc) : cap_any(x, sc));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const uint64_t s2 = f2_pack(__uint_as_float(r[e]), __uint_as_float(r[e + 1]));
      uint64_t m2 = f2_pack(c, c);
      if constexpr (CAP) m2 = cap_small_factor<4>(s2, sc);
      float x0, x1;
      f2_unpack(f2_mul(s2, m2), x0, x1);
      r[e] = __float_as_uint(x0);
      r[e + 1] = __float_as_uint(x1);
    }
  }
  if (BIAS) {
    const float pf = static_cast<float>(p_rel);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      r[e] = __float_as_uint(
          fmaf(-slope2, fabsf(pf - static_cast<float>(e)), __uint_as_float(r[e])));
  }
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (e < lo_rel || e >= hi_rel) r[e] = 0xff800000u;
}

// The softmax warps of the scored modes.  Key tiles come last first: under the causal rule the
// tile that needs the mask is then the one that sets the maximum, and a bias that falls with the
// distance lets the maximum stand from there on (first tiles first, steep slopes raised it in
// every tile and took 1.7 times as long at 2 x 16 heads x 8192 causal, d = 128; now 437 us, without
// a bias 425).  As the plain ones, with the running maximum in units of log2(e) and two ways through
// a tile:
//  * fast: every row of the warp sees the whole tile and has a maximum, its distances have one
//    sign, and the tile's sum stays below kFastLimit: scores to weights in registers;
//  * general: scores -> z in place in TMEM (with the mask), 32 columns at a time, the tile's
//    maximum, rescale, weights.  Written so that it holds few registers beside the fast way's.
template <int D, int MODE, typename Smem, typename UnitIndex>
__device__ __forceinline__ void scored_softmax_warps(Smem& s, const ScoredFwdParams& p,
                                                     uint32_t tmem, int warp, int lane,
                                                     int n_units, UnitIndex unit_index) {
  constexpr bool CAP = (MODE & kModeCap) != 0, WIDE = (MODE & kModeWide) != 0, BIAS = (MODE & kModeBias) != 0;
  volatile int* abort_flag = &s.abort_flag;
  const ScoreArgs& sc = p.sc;
  const int t = warp >> 2;
  const int row_in_tile = (warp & 3) * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t t_s = tmem + t * kTileN + lane_off;
  const uint32_t t_o = tmem + 2 * kTileN + t * D + lane_off;
  const uint32_t t_p = t_s + kTileN / 2;
  const float c = p.scale_log2;
  const uint64_t c2 = f2_pack(c, c);
  int ts = 0, us = 0;
  for (int k = 0; k * static_cast<int>(gridDim.x) < n_units; ++k) {
    const int U = unit_index(k);
    if (U >= n_units) continue;
    const ScoredUnit un = unit_at(p, U);
    if (t == 1 && !un.active1) continue;
    const int first_j = un.begin(t), n_tiles = un.end(t) - first_j;
    const int i = (t == 0 ? un.r0 : un.r1) + row_in_tile;
    const int h = (t == 0) ? un.h0 : un.h1;
    const int pos = i + un.off;
    const float slope2 = BIAS ? __ldg(sc.slopes + h) * 1.4426950408889634f : 0.f;
    // Visible keys [lo, hi) of the row.  Rows without keys (and those past the end, which are
    // not stored) are computed as if they saw everything, so that they never keep their warp
    // from the fast way; what they hold is dropped at the end.
    int lo = 0, hi = p.Sk;
    if (sc.plan.rows && i < un.sq) {
      const int2 r = __ldg(sc.plan.rows + static_cast<size_t>(un.b) * p.Sq + i);
      lo = r.x;
      hi = r.y;
    }
    if (p.causal) hi = min(hi, pos + 1);
    const bool dead = hi <= lo || i >= un.sq;
    if (dead) {
      lo = 0;
      hi = 0x7fffffff;
    }
    float m = neg_inf();  // running max of z
    float l = 0.f;        // running denominator, relative to 2^m
    float lr = 0.f;       // same, over the bf16-rounded weights
    for (int j = 0; j < n_tiles; ++j) {
      if (!mbar_wait_warp(&s.s_full[t], (ts + j) & 1, abort_flag, kSiteSFull)) return;
      tc_fence_after();
      const int c0 = (un.j0 + un.n_tiles - 1 - first_j - j) * kTileN;
      const int p_rel = pos - c0;
      bool general = __any_sync(0xffffffffu, c0 < lo || c0 + kTileN > hi || m == neg_inf());
      float sg = 0.f, bm = -m;
      if (BIAS) {
        // keys at or before every row of the warp, at or after every row, or neither
        const bool before = __all_sync(0xffffffffu, p_rel >= kTileN - 1);
        const bool after = __all_sync(0xffffffffu, p_rel <= 0);
        general = general || !(before || after);
        sg = before ? slope2 : -slope2;
        bm = fmaf(-sg, static_cast<float>(p_rel), -m);
      }
      if constexpr (CAP) {
        if (!general) {
          // the largest |score| says which polynomial holds, and bounds the weights beforehand
          float most = 0.f;
          {
            uint32_t r[32];
            float part[4];
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) tmem_ld32_max_abs(t_s + cc * 32, r, part[cc]);
            tmem_wait_ld();
            most = fmaxf(max3f(part[0], part[1], part[2]), part[3]);
          }
          const float top = fmaf(most, c, fmaxf(bm, fmaf(sg, kTileN - 1.f, bm)));
          general = __any_sync(0xffffffffu, !(top < kFastLog2));
          if (!general) {
            if (__all_sync(0xffffffffu, most <= sc.small[0]))
              capped_tile<2, BIAS>(t_s, t_p, sc, sg, bm, l, lr);
            else if (__all_sync(0xffffffffu, most <= sc.small[1]))
              capped_tile<4, BIAS>(t_s, t_p, sc, sg, bm, l, lr);
            else if constexpr (WIDE)  // one by one, the general way
              general = true;
            else
              capped_tile<kCapAny, BIAS>(t_s, t_p, sc, sg, bm, l, lr);
          }
        }
      } else if (!general) {
        uint32_t sr[kTileN];
#pragma unroll
        for (int cc = 0; cc < kTileN / 32; ++cc)
          tmem_ld32(t_s + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[cc * 32]));
        tmem_wait_ld();
        uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
        float sr_lo[4] = {0.f, 0.f, 0.f, 0.f}, sr_hi[4] = {0.f, 0.f, 0.f, 0.f};
        scored_half<0, BIAS>(sr, c2, sg, bm, t_p, sum2, sr_lo, sr_hi);
        scored_half<1, BIAS>(sr, c2, sg, bm, t_p, sum2, sr_lo, sr_hi);
        const float tsum = sum_f2x4(sum2);
        general = __any_sync(0xffffffffu, !(tsum < kFastLimit));
        if (!general) {
          l += tsum;
          lr += (sr_lo[0] + sr_lo[1]) + (sr_lo[2] + sr_lo[3]) +
                ((sr_hi[0] + sr_hi[1]) + (sr_hi[2] + sr_hi[3]));
        } else {
          // scores of [0, 64) are still in TMEM; those of [64, 128) go back over the weights
          tmem_wait_st();
          tmem_st32(t_s + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
          tmem_st32(t_s + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
          tmem_wait_st();
        }
      }
      bool grow = false;
      float alpha = 1.f;
      if (general) {
        float mx = neg_inf();
#pragma unroll 1
        for (int cc = 0; cc < kTileN / 32; ++cc) {
          uint32_t r[32];
          float most = 0.f;
          if constexpr (CAP) tmem_ld32_max_abs(t_s + cc * 32, r, most);
          else tmem_ld32(t_s + cc * 32, r);
          tmem_wait_ld();
          scored_transform<CAP, WIDE, BIAS>(r, sc, c,
                                      !CAP || __all_sync(0xffffffffu, most <= sc.small[1]), slope2,
                                      p_rel - cc * 32, lo - c0 - cc * 32, hi - c0 - cc * 32);
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mx = max3f(mx, __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
          tmem_st32(t_s + cc * 32, r);
        }
        tmem_wait_st();
        const float m_new = fmaxf(m, mx);
        // as in the plain path: the first visible key always sets the max, and -inf - (-inf) is
        // never formed
        const bool first = (m == neg_inf()) && (m_new != neg_inf());
        grow = first || (m != neg_inf() && m_new - m > p.rescale_log2);
        alpha = first ? 0.f : (grow ? ex2_approx(m - m_new) : 1.f);
        if (grow) {
          l *= alpha;
          lr *= alpha;
          m = m_new;
        }
        const float nmc = (m == neg_inf()) ? 0.f : -m;
        // weights of columns [32 cc, +32) go to columns [64 + 16 cc, +16): last columns first, so
        // that no score is overwritten before it is read
#pragma unroll 1
        for (int cc = kTileN / 32 - 1; cc >= 0; --cc) {
          uint32_t r[32], pk[16];
          tmem_ld32(t_s + cc * 32, r);
          tmem_wait_ld();
          float s_lo = 0.f, s_hi = 0.f, part = 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float p0 = ex2_approx(__uint_as_float(r[2 * e]) + nmc);
            const float p1 = ex2_approx(__uint_as_float(r[2 * e + 1]) + nmc);
            pk[e] = pack_bf16x2(p0, p1);
            part += p0 + p1;
            add_bf16x2_f32(s_lo, s_hi, pk[e]);
          }
          l += part;
          lr += s_lo + s_hi;
          tmem_st16(t_p + cc * 16, pk);
        }
      }
      if (j > 0 && __any_sync(0xffffffffu, grow)) {
        // O_t is quiescent here, as in the plain path
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t orr[32];
          tmem_ld32(t_o + cc * 32, orr);
          tmem_wait_ld();
#pragma unroll
          for (int q2 = 0; q2 < 32; ++q2)
            orr[q2] = __float_as_uint(__uint_as_float(orr[q2]) * alpha);
          tmem_st32(t_o + cc * 32, orr);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.p_full[t]);
    }
    if (n_tiles > 0) {
      if (!mbar_wait_warp(&s.o_full[t], us & 1, abort_flag, kSiteOFull)) return;
      tc_fence_after();
    }
    if (warp_aborted(abort_flag)) return;
    // ---- epilogue: O = u / lr, LSE = m ln 2 + ln l; zeros and -inf without keys ----
    {
      const bool live = l != 0.f && !dead;  // (a NaN in a visible key makes l one: it reaches O and LSE)
      const float inv = live ? 1.f / lr : 0.f;
      const bool in_range = i < un.sq && (un.parts > 1 || un.part == 0);
      const size_t row = (static_cast<size_t>(un.bz) * p.Hq + h) * p.Sq + i;
      const size_t part = static_cast<size_t>(un.part) * p.B * p.Hq * p.Sq + row;
      __nv_bfloat16* orow = reinterpret_cast<__nv_bfloat16*>(p.o) + row * D;
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t orr[32];
        if (n_tiles > 0) {
          tmem_ld32(t_o + cc * 32, orr);
          tmem_wait_ld();
        }
        if (un.parts > 1) {  // a part: the join reads it where its LSE is not -inf
          if (in_range && live) {
            float4* dst = reinterpret_cast<float4*>(p.split.part_o + part * D + cc * 32);
#pragma unroll
            for (int q2 = 0; q2 < 8; ++q2)
              dst[q2] = make_float4(
                  __uint_as_float(orr[4 * q2]) * inv, __uint_as_float(orr[4 * q2 + 1]) * inv,
                  __uint_as_float(orr[4 * q2 + 2]) * inv, __uint_as_float(orr[4 * q2 + 3]) * inv);
          }
          continue;
        }
        uint32_t pk[16];
#pragma unroll
        for (int q2 = 0; q2 < 16; ++q2)
          pk[q2] = n_tiles > 0 && live ? pack_bf16x2(__uint_as_float(orr[2 * q2]) * inv,
                                                     __uint_as_float(orr[2 * q2 + 1]) * inv)
                                       : 0u;
        if (in_range) {
          uint4* dst = reinterpret_cast<uint4*>(orow + cc * 32);
#pragma unroll
          for (int q2 = 0; q2 < 4; ++q2)
            dst[q2] = make_uint4(pk[4 * q2], pk[4 * q2 + 1], pk[4 * q2 + 2], pk[4 * q2 + 3]);
        }
      }
      const float lse = live ? fmaf(m, 0.69314718055994531f, logf(l)) : neg_inf();
      if (in_range && p.split.n > 1) p.split.part_lse[part] = un.parts > 1 ? lse : kWhole;
      if (in_range && un.parts == 1 && p.lse) p.lse[row] = lse;
    }
    if (n_tiles > 0) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.o_empty[t]);
      ts += n_tiles;
      ++us;
    }
  }
}

// Threads of a mode.  The scored modes fill the third warpgroup up, so that it can hand registers
// to the softmax warps (setmaxnreg): 128 x 56 + 256 x 224 = the 384 x 168 of the launch.
template <int MODE>
constexpr int kThreadsOf = (MODE & kModeScored) != 0 ? 384 : kThreads;

template <int D, int MODE>
__global__ void __launch_bounds__(kThreadsOf<MODE>, 1)
    fa_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                  const __grid_constant__ CUtensorMap tv, const FwdParamsOf<MODE> p) {
  using Smem = FwdSmem<D>;
  constexpr bool SCORED = (MODE & kModeScored) != 0;
  constexpr bool DROP = MODE == kModeDropout;
  constexpr bool BITS = MODE == kModeKeyBits || MODE == kModeDropout;  // key visibility bits may be present
  constexpr int NB = Smem::NB;
  constexpr int NS = Smem::NS;
  constexpr uint32_t kBoxBytes = Smem::kBox * 2;
  extern __shared__ unsigned char smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                     ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  int n_units = p.n_rbu * p.units_per_rbu;
  if constexpr (SCORED) n_units *= p.split.n;
  // The k-th unit of this CTA: units run heavy to light, so blocks of
  // gridDim.x units are walked alternately forwards and backwards (the
  // heaviest unit of one block pairs with the lightest of the next).
  auto unit_index = [&](int k) {
    const int G = static_cast<int>(gridDim.x);
    const int c = static_cast<int>(blockIdx.x);
    return k * G + ((k & 1) ? (G - 1 - c) : c);
  };

  if constexpr (SCORED) {
    if (!plan_fits(p.sc.plan, p.Sq, p.Sk)) {
      if (threadIdx.x == 0 && blockIdx.x == 0) raise_status(kStatusPlan, kSitePlan);
      return;
    }
  }
  if (threadIdx.x == 0) {
    mbar_init(&s.bar_q, 1);
    mbar_init(&s.q_free, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&s.k_full[i], 1);
      mbar_init(&s.v_full[i], 1);
      mbar_init(&s.kv_free[i], 1);
      if constexpr (SCORED) mbar_init(&s.v_raw[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s.s_full[t], 1);
      mbar_init(&s.p_full[t], 4);   // one arrival per softmax warp
      mbar_init(&s.o_full[t], 1);
      mbar_init(&s.o_empty[t], 4);  // the slot's softmax warps have read O
    }
    mbar_init(&s.drain, 1);
    s.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(&s.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  volatile int* abort_flag = &s.abort_flag;
  if (warp == 8) {
    // ------------------------------------------------------ TMA producer --
    if constexpr (SCORED) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    // K/V stages follow a tile counter g that runs across the CTA's units;
    // the next unit's Q is loaded once the previous unit's last S product
    // has read Q (q_free).
    if (lane == 0) {
      tma_prefetch_desc(&tq);
      tma_prefetch_desc(&tk);
      tma_prefetch_desc(&tv);
      const uint64_t keep = policy_evict_last();
      int g = 0, uq = 0;               // tiles and Q loads issued so far
      int k_issued = 0, v_issued = 0;  // (global tile counts, for the abort drain)
      uint32_t edges = 0, raw_parity = 0;  // stages with V of an edge tile; parity after its load
      bool ok = true;
      for (int k = 0; ok && k * static_cast<int>(gridDim.x) < n_units; ++k) {
        const int U = unit_index(k);
        if (U >= n_units) continue;
        auto un = unit_at(p, U);
        if (un.n_tiles == 0) continue;
        if (uq > 0 && !mbar_wait(&s.q_free, (uq - 1) & 1, abort_flag, kSiteQ)) break;
        mbar_arrive_expect_tx(&s.bar_q, (un.active1 ? 2 : 1) * NB * kBoxBytes);
        for (int cb = 0; cb < NB; ++cb) {
          tma_load_3d(s.q[0][cb], &tq, &s.bar_q, cb * 64, un.qb + un.r0, un.bz * p.Hq + un.h0);
          if (un.active1)
            tma_load_3d(s.q[1][cb], &tq, &s.bar_q, cb * 64, un.qb + un.r1, un.bz * p.Hq + un.h1);
        }
        ++uq;
        const int zkv = un.bz * p.Hkv + un.hk;
        if constexpr (SCORED) un.kend = all_seen_until(un, p);
        for (int j = 0; j < un.n_tiles; ++j, ++g) {
          const int st = g % NS;
          const int use = g / NS;
          const int c0 = (SCORED ? un.j0 + un.n_tiles - 1 - j : un.j0 + j) * kTileN;
          // stage st last held tile g - NS: its K was freed in round g - NS,
          // its V in round g - NS + 1
          if (use > 0 && !mbar_wait(&s.kv_free[st], (use - 1) & 1, abort_flag, kSiteKFree)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&s.k_full[st], NB * kBoxBytes);
          for (int cb = 0; cb < NB; ++cb)
            tma_load_3d_hint(s.k[st][cb], &tk, &s.k_full[st], cb * 64, c0, zkv, keep);
          k_issued = g + 1;
          if (use > 0) {
            const int r = g - NS + 1;
            if (!mbar_wait(&s.kv_free[r % NS], (r / NS) & 1, abort_flag, kSiteVFree)) {
              ok = false;
              break;
            }
          }
          uint64_t* v_bar = &s.v_full[st];
          if constexpr (SCORED) {
            edges &= ~(1u << st);
            if (edge_tile(un, j)) {
              v_bar = &s.v_raw[st];
              edges |= 1u << st;
              raw_parity ^= 1u << st;
            }
          }
          mbar_arrive_expect_tx(v_bar, NB * kBoxBytes);
          for (int cb = 0; cb < NB; ++cb)
            tma_load_3d_hint(s.v[st][cb], &tv, v_bar, cb * 64, c0, zkv, keep);
          v_issued = g + 1;
        }
      }
      if (*abort_flag) {
        // let every issued copy land before shared memory is released
        if (uq > 0) mbar_drain(&s.bar_q, (uq - 1) & 1, kSiteDrain);
        for (int j = max(0, k_issued - NS); j < k_issued; ++j)
          mbar_drain(&s.k_full[j % NS], (j / NS) & 1, kSiteDrain);
        for (int j = max(0, v_issued - NS); j < v_issued; ++j) {
          const int i = j % NS;
          if (edges >> i & 1)
            mbar_drain(&s.v_raw[i], (raw_parity >> i & 1) ^ 1, kSiteDrain);
          else
            mbar_drain(&s.v_full[i], (j / NS) & 1, kSiteDrain);
        }
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------- MMA issuer --
    if constexpr (SCORED) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    // The whole warp runs this loop (warp-uniform control flow and operands);
    // one elected lane issues each MMA and commit.  Per unit, round j issues
    // PV_t(j-1) and S_t(j) for each active slot.  A unit's first S products
    // run while the softmax warps still finish the previous unit's epilogue;
    // its first PV into O_t waits until they have read O_t (o_empty).
    constexpr uint32_t idesc_qk = idesc_bf16_f32(kTileM, kTileN, false, false);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(kTileM, D, false, true);
    constexpr uint32_t kStage = NB * kBoxBytes;  // bytes per K (or V) stage
    const uint64_t qd0 = smem_desc_sw128(smem_u32(s.q[0][0]), 16, 1024);
    const uint64_t qd1 = smem_desc_sw128(smem_u32(s.q[1][0]), 16, 1024);
    const uint64_t kd0 = smem_desc_sw128(smem_u32(s.k[0][0]), 16, 1024);
    const uint64_t vd0 = smem_desc_sw128(smem_u32(s.v[0][0]), NB > 1 ? kBoxBytes : 16u, 1024);
    int g = 0, uq = 0;
    int ts[2] = {0, 0}, us[2] = {0, 0};  // per slot: tiles and units so far
    bool ok = true;
    for (int k = 0; ok && k * static_cast<int>(gridDim.x) < n_units; ++k) {
      const int U = unit_index(k);
      if (U >= n_units) continue;
      const auto un = unit_at(p, U);
      if (un.n_tiles == 0) continue;
      const int n = un.n_tiles;
      const int nslots = un.active1 ? 2 : 1;
      if (!mbar_wait_warp(&s.bar_q, uq & 1, abort_flag, kSiteQ)) break;
      ++uq;
      for (int j = 0; ok && j <= n; ++j) {
        // K and V arrive by TMA: the mbarrier wait alone orders those shared
        // memory writes before the MMAs (both sides are async-proxy accesses).
        // Only P, written by other threads' tcgen05.st, needs the tcgen05 fence.
        const int gk = g + j, gv = g + j - 1;  // this round's K tile, V tile
        if (j < n && !mbar_wait_warp(&s.k_full[gk % NS], (gk / NS) & 1, abort_flag, kSiteKFull)) {
          ok = false;
          break;
        }
        if constexpr (SCORED) {  // every V stage in turn, whichever slots take part
          if (j > 0 && !mbar_wait_warp(&s.v_full[gv % NS], (gv / NS) & 1, abort_flag, kSiteVFull)) {
            ok = false;
            break;
          }
        }
        const uint64_t kd = desc_add(kd0, static_cast<uint32_t>(gk % NS) * kStage);
        const uint64_t vd = desc_add(vd0, static_cast<uint32_t>(((gv % NS) + NS) % NS) * kStage);
        for (int t = 0; t < nslots; ++t) {
          const uint32_t t_s = tmem + t * kTileN;
          int jt = j, n_t = n;  // round of the slot, and how many it has
          if constexpr (SCORED) {
            jt = j - un.begin(t);
            n_t = un.end(t) - un.begin(t);
            if (jt < 0 || jt > n_t || n_t == 0) continue;
          }
          if (jt > 0) {
            // O_t += P_t(j-1) V_{j-1}; P_t lives in the last 64 columns of S_t
            if (!mbar_wait_warp(&s.p_full[t], (ts[t] + jt - 1) & 1, abort_flag, kSitePFull) ||
                (!SCORED && t == 0 &&
                 !mbar_wait_warp(&s.v_full[gv % NS], (gv / NS) & 1, abort_flag, kSiteVFull)) ||
                (jt == 1 && us[t] > 0 &&
                 !mbar_wait_warp(&s.o_empty[t], (us[t] - 1) & 1, abort_flag, kSiteOFull))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t t_o = tmem + 2 * kTileN + t * D;
            const uint32_t t_p = t_s + kTileN / 2;
            mma_ts_warp(t_o, t_p, vd, idesc_pv, jt > 1 ? 1u : 0u);
#pragma unroll
            for (int kk = 1; kk < kTileN / 16; ++kk)
              mma_ts_warp(t_o, t_p + kk * 8, desc_add(vd, kk * 16 * 128), idesc_pv, 1u);
          }
          if (jt < n_t) {
            // S_t = Q_t K_j^T
            const uint64_t qd = t ? qd1 : qd0;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * kBoxBytes + (kk & 3) * 32;
              mma_ss_warp(t_s, desc_add(qd, off), desc_add(kd, off), idesc_qk, kk > 0 ? 1u : 0u);
            }
            mma_commit_warp(&s.s_full[t]);
          } else {
            mma_commit_warp(&s.o_full[t]);
          }
        }
        if (!ok) break;
        if (j < n) mma_commit_warp(&s.kv_free[gk % NS]);
        if (j == n - 1) mma_commit_warp(&s.q_free);  // the unit's last S has read Q
      }
      g += n;
      for (int t = 0; t < nslots; ++t) {
        int n_t = n;
        if constexpr (SCORED) n_t = un.end(t) - un.begin(t);
        ts[t] += n_t;
        us[t] += n_t > 0;
      }
    }
    if (warp_aborted(abort_flag)) {
      // every MMA issued so far must finish before TMEM is released
      mma_commit_warp(&s.drain);
      mbar_drain(&s.drain, 0, kSiteDrain);
    }
  } else if constexpr (SCORED) {
    if (warp < 8) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
      scored_softmax_warps<D, MODE>(s, p, tmem, warp, lane, n_units, unit_index);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
      if (warp == 10) edge_warp(s, p, lane, n_units);
    }
  } else {
    // ---------------------------------------------------- softmax warps --
    const int t = warp >> 2;
    const int row_in_tile = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + t * kTileN + lane_off;
    const uint32_t t_o = tmem + 2 * kTileN + t * D + lane_off;
    const uint32_t t_p = t_s + kTileN / 2;  // P: bf16 pairs in S columns [64, 128)
    const float c = p.scale_log2;
    int ts = 0, us = 0;  // this slot's tiles and units so far
    bool ok = true;
    for (int k = 0; ok && k * static_cast<int>(gridDim.x) < n_units; ++k) {
      const int U = unit_index(k);
      if (U >= n_units) continue;
      const Unit un = unit_at(p, U);
      if (!un.rows || (t == 1 && !un.active1)) continue;
      const int n_tiles = un.n_tiles, j0 = un.j0, klo = un.klo, kend = un.kend;
      const int sq = un.sq, qb = un.qb, bz = un.bz;
      const int i = (t == 0 ? un.r0 : un.r1) + row_in_tile;
      const int h = (t == 0) ? un.h0 : un.h1;
      const uint32_t bh = static_cast<uint32_t>(bz * p.Hq + h);  // dropout counter word 2
      const uint32_t* kbits =
          p.key_bits ? p.key_bits + static_cast<size_t>(bz) * p.mask_words : nullptr;
      // keys visible to this row: [klo, khi_row)
      int khi_row = kend;
      if (p.causal) khi_row = min(khi_row, i + un.off + 1);
      float m = neg_inf();  // running max of raw scores (unscaled)
      float l = 0.f;        // running denominator, relative to 2^(m*c)
      float lr = 0.f;       // same, over the bf16-rounded weights
      // Dropout keep bits of this row for one key tile (bit jj of word jj / 32
      // = key jj of the tile kept).  They are computed one tile ahead, after
      // the row's P has been released and while the warp waits for the next
      // S, so the Philox rounds stay off the S -> P path.
      uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};
      auto keep_bits = [&](int jt) {
        const uint32_t k8 = static_cast<uint32_t>((j0 + jt) * kTileN) >> 3;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t word = 0;
#pragma unroll
          for (int g = 0; g < 4; ++g)
            word |= dropout_keep8(p.drop, k8 + 4 * w + g, static_cast<uint32_t>(i), bh) << (8 * g);
          keep[w] = word;
        }
      };
      if (DROP && n_tiles > 0) keep_bits(0);
      for (int j = 0; j < n_tiles; ++j) {
        if (!mbar_wait_warp(&s.s_full[t], (ts + j) & 1, abort_flag, kSiteSFull)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t sr[kTileN];
#pragma unroll
        for (int cc = 0; cc < kTileN / 32; ++cc)
          tmem_ld32(t_s + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[cc * 32]));
        tmem_wait_ld();
        const int c0 = (j0 + j) * kTileN;
        const bool need_mask = (c0 < klo) || (c0 + kTileN > khi_row);
        const bool masked_tile = __any_sync(0xffffffffu, need_mask);
        if (masked_tile) mask_scores<0, kTileN>(sr, c0, klo, khi_row);
        // key visibility bits of this tile (the same 128 bits for every row)
        uint4 kb = make_uint4(~0u, ~0u, ~0u, ~0u);
        if (BITS && kbits) kb = __ldg(reinterpret_cast<const uint4*>(kbits + c0 / 32));
        const bool bit_masked = BITS && (kb.x & kb.y & kb.z & kb.w) != ~0u;
        if (bit_masked) mask_key_bits<0, kTileN>(sr, kb);
        // Fast path: weights relative to the running max as it stands.  The
        // max only keeps the weights finite, and the fp32 tile sum (needed for
        // l anyway) bounds every weight of the row, so the tile is checked
        // after the fact.  A row that has no max yet, or whose tile sum
        // reaches kFastLimit (or is not finite), sends the warp to the exact
        // path, which finds the tile max, rescales and recomputes.
        bool exact = __any_sync(0xffffffffu, m == neg_inf());
        const uint64_t c2 = f2_pack(c, c);
        uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
        float sr_lo[4] = {0.f, 0.f, 0.f, 0.f}, sr_hi[4] = {0.f, 0.f, 0.f, 0.f};
        if (!exact) {
          const float mc = m * c;
          const uint64_t nmc2 = f2_pack(-mc, -mc);
          softmax_half<0, DROP>(sr, c2, nmc2, t_p, sum2, sr_lo, sr_hi, keep);
          softmax_half<1, DROP>(sr, c2, nmc2, t_p, sum2, sr_lo, sr_hi, keep);
          const float ts = sum_f2x4(sum2);
          exact = __any_sync(0xffffffffu, !(ts < kFastLimit));
          if (!exact) {
            l += ts;
            lr += (sr_lo[0] + sr_lo[1]) + (sr_lo[2] + sr_lo[3]) +
                  ((sr_hi[0] + sr_hi[1]) + (sr_hi[2] + sr_hi[3]));
          }
        }
        bool grow = false;
        float alpha = 1.f;
        if (exact) {
          // S columns [0, 64) are still in TMEM (P goes to [64, 128)); the
          // scores of [64, 128) are still in registers.
#pragma unroll
          for (int cc = 0; cc < 2; ++cc)
            tmem_ld32(t_s + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[cc * 32]));
          tmem_wait_ld();
          tmem_wait_st();  // fast-path P stores land before they are rewritten
          if (masked_tile) mask_scores<0, kTileN / 2>(sr, c0, klo, khi_row);
          if (bit_masked) mask_key_bits<0, kTileN / 2>(sr, kb);
          // row max: 8 independent chains of 3-input max
          float mx8[8];
#pragma unroll
          for (int q2 = 0; q2 < 8; ++q2)
            mx8[q2] = fmaxf(__uint_as_float(sr[q2]), __uint_as_float(sr[q2 + 8]));
#pragma unroll
          for (int jj = 16; jj < kTileN; jj += 16)
#pragma unroll
            for (int q2 = 0; q2 < 8; ++q2)
              mx8[q2] = max3f(mx8[q2], __uint_as_float(sr[jj + q2]), __uint_as_float(sr[jj + 8 + q2]));
          const float mx = max3f(max3f(mx8[0], mx8[1], mx8[2]), max3f(mx8[3], mx8[4], mx8[5]),
                                 fmaxf(mx8[6], mx8[7]));
          const float m_new = fmaxf(m, mx);
          // A row's first visible key always sets its max (also when c = 0,
          // where (m_new - m) * c would be inf * 0); nothing is accumulated
          // yet, so the rescale factor is 0.  Later the max moves only when it
          // grows by more than the threshold.  The difference m_new - m is
          // formed only once m is finite: a row that still sees no key keeps
          // m = -inf and never evaluates -inf - (-inf).
          const bool first = (m == neg_inf()) && (m_new != neg_inf());
          grow = first || (m != neg_inf() && (m_new - m) * c > p.rescale_log2);
          alpha = first ? 0.f : (grow ? ex2_approx((m - m_new) * c) : 1.f);
          if (grow) {
            l *= alpha;
            lr *= alpha;
            m = m_new;
          }
          const float mc = (m == neg_inf()) ? 0.f : m * c;
          const uint64_t nmc2 = f2_pack(-mc, -mc);
#pragma unroll
          for (int q2 = 0; q2 < 4; ++q2) {
            sum2[q2] = 0ull;
            sr_lo[q2] = 0.f;
            sr_hi[q2] = 0.f;
          }
          softmax_half<0, DROP>(sr, c2, nmc2, t_p, sum2, sr_lo, sr_hi, keep);
          softmax_half<1, DROP>(sr, c2, nmc2, t_p, sum2, sr_lo, sr_hi, keep);
          l += sum_f2x4(sum2);
          lr += (sr_lo[0] + sr_lo[1]) + (sr_lo[2] + sr_lo[3]) +
                ((sr_hi[0] + sr_hi[1]) + (sr_hi[2] + sr_hi[3]));
        }
        if (j > 0 && __any_sync(0xffffffffu, grow)) {
          // O_t is quiescent here: PV_t(j-1) completed before S_t(j) was
          // signalled, and PV_t(j) is issued only after p_full below.
#pragma unroll
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t orr[32];
            tmem_ld32(t_o + cc * 32, orr);
            tmem_wait_ld();
#pragma unroll
            for (int q2 = 0; q2 < 32; ++q2)
              orr[q2] = __float_as_uint(__uint_as_float(orr[q2]) * alpha);
            tmem_st32(t_o + cc * 32, orr);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[t]);
        if (DROP && j + 1 < n_tiles) keep_bits(j + 1);
      }
      if (!ok) break;
      if (n_tiles > 0) {
        if (!mbar_wait_warp(&s.o_full[t], us & 1, abort_flag, kSiteOFull)) break;
        tc_fence_after();
      }
      if (warp_aborted(abort_flag)) break;
      // ---- epilogue: O = u / lr, LSE = m*scale + ln l ----------------------
      {
        const bool live = l > 0.f;
        const float inv = live ? (DROP ? p.drop.scale : 1.f) / lr : 0.f;
        const bool in_range = i < sq;
        const size_t row = (static_cast<size_t>(bz) * p.Hq + h) * p.Sq + qb + i;
        __nv_bfloat16* orow = reinterpret_cast<__nv_bfloat16*>(p.o) + row * D;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t orr[32];
          if (n_tiles > 0) {
            tmem_ld32(t_o + cc * 32, orr);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int q2 = 0; q2 < 32; ++q2) orr[q2] = 0u;
          }
          uint32_t pk[16];
#pragma unroll
          for (int q2 = 0; q2 < 16; ++q2)
            pk[q2] = pack_bf16x2(__uint_as_float(orr[2 * q2]) * inv,
                                 __uint_as_float(orr[2 * q2 + 1]) * inv);
          if (in_range) {
            uint4* dst = reinterpret_cast<uint4*>(orow + cc * 32);
#pragma unroll
            for (int q2 = 0; q2 < 4; ++q2)
              dst[q2] = make_uint4(pk[4 * q2], pk[4 * q2 + 1], pk[4 * q2 + 2], pk[4 * q2 + 3]);
          }
        }
        if (in_range && p.lse) p.lse[row] = live ? fmaf(m, p.scale, logf(l)) : neg_inf();
      }
      if (n_tiles > 0) {
        // O_t has been read: the next unit's first PV may overwrite it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.o_empty[t]);
        ts += n_tiles;
        ++us;
      }
    }
  }

  // ---- teardown ----------------------------------------------------------
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace
}  // namespace fa
