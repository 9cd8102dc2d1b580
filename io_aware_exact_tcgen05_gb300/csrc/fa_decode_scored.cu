// fa_decode_scored.cu -- the single-query decode (fa_decode_kernel.cuh) with capped scores, a bias by
// distance and a window.
#include "fa_decode_kernel.cuh"

namespace fa {

void decode_scored_plan(int B, int Hq, int Hkv, int Sk_max, int window, int* chunk,
                        int* n_split) {
  const int keys = window > 0 && window < Sk_max ? window : Sk_max;
  decode_plan(B, Hq, Hkv, keys, chunk, n_split);
}

cudaError_t launch_decode_scored(int d, const ScoredDecodeParams& p, cudaStream_t stream) {
  if (d == 128) return launch_decode_d<128, true>(p, stream);
  return launch_decode_d<64, true>(p, stream);
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
