// fa_bwd_scored.cu -- the backward pass (fa_bwd_kernel.cuh) for capped scores, a bias by distance and
// the row intervals of a mask plan.
#include "fa_bwd_kernel.cuh"
#include "fa_scored.h"

namespace fa {
namespace {

template <int D>
cudaError_t launch_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     const CUtensorMap& tdo, const CUtensorMap& tdq, const ScoredBwdParams& p,
                     bool cap, cudaStream_t stream) {
  if (cap && p.sc.wide)
    return p.sc.slopes
               ? launch_bwd_mode<D, kBwdScored | kBwdCap | kBwdWide | kBwdBias>(tq, tk, tv, tdo, tdq, p, stream)
               : launch_bwd_mode<D, kBwdScored | kBwdCap | kBwdWide>(tq, tk, tv, tdo, tdq, p, stream);
  if (cap && p.sc.slopes)
    return launch_bwd_mode<D, kBwdScored | kBwdCap | kBwdBias>(tq, tk, tv, tdo, tdq, p, stream);
  if (cap) return launch_bwd_mode<D, kBwdScored | kBwdCap>(tq, tk, tv, tdo, tdq, p, stream);
  if (p.sc.slopes) return launch_bwd_mode<D, kBwdScored | kBwdBias>(tq, tk, tv, tdo, tdq, p, stream);
  return launch_bwd_mode<D, kBwdScored>(tq, tk, tv, tdo, tdq, p, stream);
}

}  // namespace

// (304: two for each of GB300's SMs.  A constant, since sizes of workspaces depend on the arguments alone.)
// Units that are at most two per SM are split where they are long, into 16 parts at most: 16 query
// heads on 2 of 2048 rows 299 -> 138 us, 4 on 1 of 8192 582 -> 201, 32 on 8 of 2048 166 -> 145.  (Up
// to one per SM: 112, 324 and not; four per SM 148, 269 and 158, and two batch rows of the last one
// 190 -> 252.)
int bwd_scored_splits(int B, int Hq, int Hkv, int Sq, int Sk) {
  const long long units = (Sk + kTileN - 1LL) / kTileN * B * Hkv;
  const long long its = (Sq + kTileM - 1LL) / kTileM * (Hq / Hkv);
  return static_cast<int>(std::max(1LL, std::min({304 / units, its / kPartIts, 16LL})));
}

cudaError_t launch_bwd_scored(int d, const CUtensorMap& tq, const CUtensorMap& tk,
                              const CUtensorMap& tv, const CUtensorMap& tdo,
                              const CUtensorMap& tdq, const BwdParams& base, const ScoreArgs& sc,
                              const BwdSplit& split, bool cap, cudaStream_t stream) {
  ScoredBwdParams p;
  static_cast<BwdParams&>(p) = base;
  p.sc = sc;
  p.split = split;
  if (d == 128) return launch_d<128>(tq, tk, tv, tdo, tdq, p, cap, stream);
  return launch_d<64>(tq, tk, tv, tdo, tdq, p, cap, stream);
}

unsigned int read_bwd_scored_status(bool clear) {
  unsigned int v = 0;
  cudaMemcpyFromSymbol(&v, g_status, sizeof v);
  if (clear) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_status, &z, sizeof z);
  }
  return v;
}

}  // namespace fa
