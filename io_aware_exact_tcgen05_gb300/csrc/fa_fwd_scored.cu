// fa_fwd_scored.cu -- the forward kernel (fa_fwd_kernel.cuh) for capped scores, a bias by distance
// and the row intervals of a mask plan.
#include "fa_fwd_kernel.cuh"
#include "fa_scored.h"

namespace fa {
namespace {

// O and LSE of a row from the parts of its keys, by the rescale rule; a warp per row.
template <int D>
__global__ void __launch_bounds__(256) fa_fwd_join(const ScoredFwdParams p, int rows) {
  constexpr int PER = D / 32;  // elements of a lane
  const int row = static_cast<int>(blockIdx.x) * 8 + static_cast<int>(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  griddep_wait();
  if (row >= rows || p.split.part_lse[row] == kWhole) return;
  // a lane has the weights of parts lane and lane + 32
  float w[2], M = neg_inf(), sum = 0.f;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int s = lane + 32 * u;
    w[u] = s < p.split.n ? p.split.part_lse[static_cast<size_t>(s) * rows + row] : neg_inf();
    M = fmaxf(M, w[u]);
  }
#pragma unroll
  for (int x = 16; x >= 1; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    w[u] = w[u] == neg_inf() ? 0.f : expf(w[u] - M);  // (a NaN goes on)
    sum += w[u];
  }
#pragma unroll
  for (int x = 16; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  float o[PER] = {};
#pragma unroll 8
  for (int s = 0; s < p.split.n; ++s) {
    const float ws = __shfl_sync(0xffffffffu, s < 32 ? w[0] : w[1], s & 31);
    const float* part = p.split.part_o + (static_cast<size_t>(s) * rows + row) * D;
#pragma unroll
    for (int e = 0; e < PER; ++e)  // (what a part without weight holds was never written)
      o[e] = fmaf(ws, ws != 0.f ? part[e * 32 + lane] : 0.f, o[e]);
  }
  const bool live = sum != 0.f;
  const float inv = live ? 1.f / sum : 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e)
    reinterpret_cast<__nv_bfloat16*>(p.o)[static_cast<size_t>(row) * D + e * 32 + lane] =
        __float2bfloat16_rn(live ? o[e] * inv : 0.f);
  if (lane == 0 && p.lse) p.lse[row] = live ? M + logf(sum) : neg_inf();
}

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
  const long long units = static_cast<long long>(p.n_rbu) * p.units_per_rbu * p.split.n;
  const unsigned int grid = static_cast<unsigned int>(std::min<long long>(units, n_sm));
  hook_before(stream);
  fa_fwd_kernel<D, MODE><<<grid, kThreadsOf<MODE>, smem, stream>>>(tq, tk, tv, p);
  hook_after(stream);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.split.n == 1) return e;
  const int rows = p.B * p.Hq * p.Sq;
  return launch_dependent(fa_fwd_join<D>, dim3((rows + 7) / 8), dim3(256), 0, stream, p, rows);
}

template <int D>
cudaError_t launch_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     const ScoredFwdParams& p, bool cap, cudaStream_t stream) {
  if (cap && p.sc.wide)
    return p.sc.slopes
               ? launch_dm<D, kModeScored | kModeCap | kModeWide | kModeBias>(tq, tk, tv, p, stream)
               : launch_dm<D, kModeScored | kModeCap | kModeWide>(tq, tk, tv, p, stream);
  if (cap && p.sc.slopes)
    return launch_dm<D, kModeScored | kModeCap | kModeBias>(tq, tk, tv, p, stream);
  if (cap) return launch_dm<D, kModeScored | kModeCap>(tq, tk, tv, p, stream);
  if (p.sc.slopes) return launch_dm<D, kModeScored | kModeBias>(tq, tk, tv, p, stream);
  return launch_dm<D, kModeScored>(tq, tk, tv, p, stream);
}

}  // namespace

// (152: GB300's SMs.  A constant, since sizes of workspaces depend on the arguments alone.)
// Units that leave half of the SMs or more without work are split, into parts that still fit the
// SMs at once: 8 heads of 128 rows and 32768 keys 440 -> 35 us, 8 of 512 and 8192 115 -> 30.  (Up to
// twice the SMs: 128 units of 16 tiles 36 -> 48, 16 of 64 tiles 43 us.)
int fwd_scored_splits(int B, int Hq, int Hkv, int Sq, int Sk) {
  const int group = Hq / Hkv;
  const long long units = group % 2 == 0 ? 1LL * B * (Hq / 2) * ((Sq + kTileM - 1) / kTileM)
                                         : 1LL * B * Hq * ((Sq + 2 * kTileM - 1) / (2 * kTileM));
  const long long tiles = (Sk + kTileN - 1LL) / kTileN;
  return static_cast<int>(std::max(1LL, std::min({152 / units, tiles / kPartTiles, 64LL})));
}

cudaError_t launch_fwd_scored(int d, const CUtensorMap& tq, const CUtensorMap& tk,
                              const CUtensorMap& tv, const FwdParams& base, const ScoreArgs& sc,
                              const FwdSplit& split, bool cap, cudaStream_t stream) {
  ScoredFwdParams p;
  static_cast<FwdParams&>(p) = base;
  p.sc = sc;
  p.split = split;
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
