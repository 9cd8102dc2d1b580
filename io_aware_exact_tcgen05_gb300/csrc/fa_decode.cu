// fa_decode.cu -- the single-query decode (fa_decode_kernel.cuh) with plain scores.
#include "fa_decode_kernel.cuh"

namespace fa {

void decode_plan(int B, int Hq, int Hkv, int Sk_max, int* chunk, int* n_split) {
  (void)B;
  (void)Hq;
  (void)Hkv;
  // 4096 keys (2 MiB of K+V at d=128) per CTA: long streams per CTA amortise
  // the start-up and the per-split merge (measured on GB300: 512-key chunks
  // reached 4.1 TB/s, 4096-key chunks 6.1 TB/s); short caches use smaller
  // chunks so that a row still spreads over several CTAs.  Multiple of the
  // 128-key stage.
  int c = DecodeTiles::kMaxChunk;
  while (c > kStageKeys && Sk_max <= 4 * c) c >>= 1;
  *chunk = c;
  *n_split = (Sk_max + c - 1) / c;
}

cudaError_t launch_decode(int d, const DecodeParams& p, cudaStream_t stream) {
  if (d == 128) return launch_decode_d<128, false>(p, stream);
  return launch_decode_d<64, false>(p, stream);
}

unsigned int read_decode_status(bool clear) {
  unsigned int v = 0;
  cudaMemcpyFromSymbol(&v, g_status, sizeof v);
  if (clear) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_status, &z, sizeof z);
  }
  return v;
}

}  // namespace fa
