// fa_scored.h -- host-side parameter blocks of the operators around the scores: row intervals
// and their tile plan (fa_mask_plan.cu), attention with capped and biased scores
// (fa_fwd_scored.cu, fa_bwd_scored.cu, fa_decode_scored.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime_api.h>

#include "fa_internal.h"

namespace fa {

// What fa_mask_plan writes, as the attention kernels read it (all in the caller's buffer).
// rows == nullptr: no plan, every key is visible.
struct MaskPlan {
  const int4* sizes; // B, Sq, Sk, kPlanMark: what the kernels know a plan of theirs by (plan_fits)
  const int4* qt;    // [B][nq]  per 128-row tile, over its rows with keys: min lo, max hi, how many stretches
                     //          of keys between them are in no row's interval (3: more than two), whether an
                     //          interval goes past its row's position (1: and every row of the tile sees
                     //          its own; 2: not) (0, 0, 0, 0 where no row has keys)
  const int4* gaps;  // [B][nq]  those stretches, first and end key each, where they are one or two (0, 0: none)
  const uint4* seen; // [B][nk]  which of the 128 keys of a tile any row of the batch row sees
  const uint4* seen_causal;  // the same under the causal rule
  const int4* kt;    // [B][nk]  first and end query tile that may see the 128-key tile; 0 where every key of
                     //          it is seen (by some row of the batch row), else kUnseen; the same
                     //          under the causal rule
  const int2* rows;  // [B][Sq]  lo, hi of each row; (0, 0) without keys
  // tiles (batch row * tiles of a row + tile) in the order of their work, most first
  const int* by_q1;    // [B * nq]  query tiles by key tiles
  const int* by_q2;    // [B * np]  pairs of query tiles, likewise
  const int* by_k;     // [B * nk]  key tiles by query tiles
  const int* by_k_row; // [B][nk]   the same within each batch row
  const int* work;     // [B * (nq + np + nk)]  what they are ordered by
  int B, nq, np, nk;
};

constexpr int kUnseen = 0x7fffffff;

constexpr int kPlanMark = 0x6d61736b;

// 32-bit words of a plan: sizes, qt, gaps, seen, seen_causal, kt, rows, by_q1, by_q2, by_k, by_k_row, work.
inline size_t mask_plan_words(long long B, long long Sq, long long Sk) {
  const long long nq = (Sq + 127) / 128, np = (nq + 1) / 2, nk = (Sk + 127) / 128;
  return static_cast<size_t>(4 + B * (8 * nq + 12 * nk + 2 * Sq + 2 * (nq + np + nk) + nk));
}

inline MaskPlan mask_plan_view(const void* base, long long B, long long Sq, long long Sk) {
  MaskPlan m{};
  if (!base) return m;
  m.B = static_cast<int>(B);
  m.nq = static_cast<int>((Sq + 127) / 128);
  m.np = (m.nq + 1) / 2;
  m.nk = static_cast<int>((Sk + 127) / 128);
  const int* w = static_cast<const int*>(base);
  m.sizes = reinterpret_cast<const int4*>(w);
  w += 4;
  m.qt = reinterpret_cast<const int4*>(w);
  w += 4 * B * m.nq;
  m.gaps = reinterpret_cast<const int4*>(w);
  w += 4 * B * m.nq;
  m.seen = reinterpret_cast<const uint4*>(w);
  w += 4 * B * m.nk;
  m.seen_causal = reinterpret_cast<const uint4*>(w);
  w += 4 * B * m.nk;
  m.kt = reinterpret_cast<const int4*>(w);
  w += 4 * B * m.nk;
  m.rows = reinterpret_cast<const int2*>(w);
  m.by_q1 = w + 2 * B * Sq;
  m.by_q2 = m.by_q1 + B * m.nq;
  m.by_k = m.by_q2 + B * m.np;
  m.by_k_row = m.by_k + B * m.nk;
  m.work = m.by_k_row + B * m.nk;
  return m;
}

struct RowBoundsParams {
  const int32_t* cu_docs;  // [n_docs + 1] or nullptr
  const int32_t* prefix;   // [n_docs], or [B] without documents, or nullptr
  int32_t* lo;             // [B][Sq]
  int32_t* hi;
  int n_docs, B, Sq, Sk, causal, window;
};

cudaError_t launch_row_bounds(const RowBoundsParams& p, cudaStream_t stream);
cudaError_t launch_mask_plan(const int32_t* lo, const int32_t* hi, int B, int Sq, int Sk,
                             const MaskPlan& plan, cudaStream_t stream);

// Scores z = t - slope * |p - j| in units of log2(e), t = cap * tanh(s * scale / cap) (see
// fa_score.cuh for the arithmetic).
constexpr float kWideCap = 256.f;
struct ScoreArgs {
  float a;             // scale / cap
  float two_a_log2e;   // 2 * a * log2(e)
  float cap_log2e;     // cap * log2(e)
  float neg_inv_cap2;  // -1 / cap_log2e^2
  float small[3];      // |s| up to which the polynomials hold (-1: never)
  int wide;            // the cap is above kWideCap: scores past the polynomials one by one (cap_wide)
  float2 poly2[3];     // z = s * (poly2[0] + poly2[1] s^2 + ...), each twice (for packed pairs)
  float2 poly4[5];
  float2 poly7[8];     // z = y * (poly7[0] + poly7[1] y^2 + ...), y = a s
  const float* slopes; // fp32 [Hq] or nullptr
  MaskPlan plan;
};

// fa_decode on such scores: sizes, inputs and outputs of DecodeParams (its split plan is not used).
struct ScoredDecodeParams : DecodeParams {
  const int32_t* k_start;  // int32 [B] or nullptr
  int window;              // last keys seen; 0: all
  bool capped;
  int heads;               // query heads of a work item (up to 16 of one KV head)
  int subs;                // work items of a batch row
  bool direct;             // a CTA per item, which writes the results
  int2* span;              // [B * subs]: first and last CTA of each item
  ScoreArgs sc;
};

// Workspace: span, then per (CTA, item) slot the partial outputs and their log2-sums.
struct DecodeScoredPlan {
  bool direct;  // needs none
  int heads, subs, ctas;
  size_t slots, span_bytes, o_bytes, lse_bytes;
};
DecodeScoredPlan decode_scored_plan(int B, int Hq, int Hkv, int Sk_max, int d, int window);
cudaError_t launch_decode_scored(int d, const CUtensorMap& tk, const CUtensorMap& tv,
                                 const ScoredDecodeParams& p, const DecodeScoredPlan& plan,
                                 cudaStream_t stream);
unsigned int read_decode_scored_status(bool clear);

// Parts that the key tiles of a unit are split into, and what holds their results.
struct FwdSplit {
  int n;            // 1: not split
  float* part_o;    // [n][B * Hq * Sq][d]  O of each part
  float* part_lse;  // [n][B * Hq * Sq]     its LSE; -inf without keys; kWhole: the row is done
};
int fwd_scored_splits(int B, int Hq, int Hkv, int Sq, int Sk);
cudaError_t launch_fwd_scored(int d, const CUtensorMap& tq, const CUtensorMap& tk,
                              const CUtensorMap& tv, const FwdParams& base, const ScoreArgs& sc,
                              const FwdSplit& split, bool cap, cudaStream_t stream);
// Parts that the query tiles of a key tile's unit (of all heads of the group) are split into.
struct BwdSplit {
  int n;        // 1: not split
  float* part;  // [n][2][B * Hkv * Sk][d]  dK and dV of each part
};
int bwd_scored_splits(int B, int Hq, int Hkv, int Sq, int Sk);
cudaError_t launch_bwd_scored(int d, const CUtensorMap& tq, const CUtensorMap& tk,
                              const CUtensorMap& tv, const CUtensorMap& tdo,
                              const CUtensorMap& tdq, const BwdParams& base, const ScoreArgs& sc,
                              const BwdSplit& split, bool cap, cudaStream_t stream);
unsigned int read_fwd_scored_status(bool clear);
unsigned int read_bwd_scored_status(bool clear);

}  // namespace fa
