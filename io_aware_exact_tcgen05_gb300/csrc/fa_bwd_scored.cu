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
  if (cap && p.sc.slopes)
    return launch_bwd_mode<D, kBwdScored | kBwdCap | kBwdBias>(tq, tk, tv, tdo, tdq, p, stream);
  if (cap) return launch_bwd_mode<D, kBwdScored | kBwdCap>(tq, tk, tv, tdo, tdq, p, stream);
  if (p.sc.slopes) return launch_bwd_mode<D, kBwdScored | kBwdBias>(tq, tk, tv, tdo, tdq, p, stream);
  return launch_bwd_mode<D, kBwdScored>(tq, tk, tv, tdo, tdq, p, stream);
}

}  // namespace

cudaError_t launch_bwd_scored(int d, const CUtensorMap& tq, const CUtensorMap& tk,
                              const CUtensorMap& tv, const CUtensorMap& tdo,
                              const CUtensorMap& tdq, const BwdParams& base, const ScoreArgs& sc,
                              bool cap, cudaStream_t stream) {
  ScoredBwdParams p;
  static_cast<BwdParams&>(p) = base;
  p.sc = sc;
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
