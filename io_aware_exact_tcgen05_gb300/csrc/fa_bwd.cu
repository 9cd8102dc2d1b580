// fa_bwd.cu -- the backward pass (fa_bwd_kernel.cuh) for plain and dropped weights.
#include "fa_bwd_kernel.cuh"

namespace fa {
namespace {

template <int D>
cudaError_t launch_bwd_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                         const CUtensorMap& tdo, const CUtensorMap& tdq, const BwdParams& p,
                         cudaStream_t stream) {
  if (p.drop.on) return launch_bwd_mode<D, kBwdDropout>(tq, tk, tv, tdo, tdq, p, stream);
  return launch_bwd_mode<D, kBwdPlain>(tq, tk, tv, tdo, tdq, p, stream);
}

}  // namespace

cudaError_t launch_bwd(int d, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       const CUtensorMap& tdo, const CUtensorMap& tdq, const BwdParams& p,
                       cudaStream_t stream) {
  if (d == 128) return launch_bwd_d<128>(tq, tk, tv, tdo, tdq, p, stream);
  return launch_bwd_d<64>(tq, tk, tv, tdo, tdq, p, stream);
}

unsigned int read_bwd_status(bool clear) {
  unsigned int v = 0;
  cudaMemcpyFromSymbol(&v, g_status, sizeof v);
  if (clear) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_status, &z, sizeof z);
  }
  return v;
}

}  // namespace fa
