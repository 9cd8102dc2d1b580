// fa_fwd_scored.cu -- the forward kernel (fa_fwd_kernel.cuh) for capped scores, a bias by distance
// and the row intervals of a mask plan.
#include "fa_fwd_kernel.cuh"
#include "fa_scored.h"

namespace fa {
namespace {

template <int D, int MODE>
cudaError_t launch_dm(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                      const ScoredFwdParams& p, cudaStream_t stream) {
  constexpr size_t smem = fwd_smem_bytes<D>();
  cudaError_t e = cudaFuncSetAttribute(fa_fwd_kernel<D, MODE>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  int dev = 0, n_sm = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const long long units = static_cast<long long>(p.n_rbu) * p.units_per_rbu;
  const unsigned int grid = static_cast<unsigned int>(std::min<long long>(units, n_sm));
  hook_before(stream);
  fa_fwd_kernel<D, MODE><<<grid, kThreadsOf<MODE>, smem, stream>>>(tq, tk, tv, p);
  hook_after(stream);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     const ScoredFwdParams& p, bool cap, cudaStream_t stream) {
  if (cap && p.sc.slopes)
    return launch_dm<D, kModeScored | kModeCap | kModeBias>(tq, tk, tv, p, stream);
  if (cap) return launch_dm<D, kModeScored | kModeCap>(tq, tk, tv, p, stream);
  if (p.sc.slopes) return launch_dm<D, kModeScored | kModeBias>(tq, tk, tv, p, stream);
  return launch_dm<D, kModeScored>(tq, tk, tv, p, stream);
}

}  // namespace

cudaError_t launch_fwd_scored(int d, const CUtensorMap& tq, const CUtensorMap& tk,
                              const CUtensorMap& tv, const FwdParams& base, const ScoreArgs& sc,
                              bool cap, cudaStream_t stream) {
  ScoredFwdParams p;
  static_cast<FwdParams&>(p) = base;
  p.sc = sc;
  if (d == 128) return launch_d<128>(tq, tk, tv, p, cap, stream);
  return launch_d<64>(tq, tk, tv, p, cap, stream);
}

unsigned int read_fwd_scored_status(bool clear) {
  unsigned int v = 0;
  cudaMemcpyFromSymbol(&v, g_status, sizeof v);
  if (clear) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_status, &z, sizeof z);
  }
  return v;
}

}  // namespace fa
