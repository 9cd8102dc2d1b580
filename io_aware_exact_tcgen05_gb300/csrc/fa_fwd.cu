// fa_fwd.cu -- launches of the forward kernel (fa_fwd_kernel.cuh) for plain, masked and dropped weights.
#include "fa_fwd_kernel.cuh"

namespace fa {
namespace {

template <int D, int MODE>
cudaError_t launch_fwd_dd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          const FwdParams& p, cudaStream_t stream) {
  constexpr size_t smem = fwd_smem_bytes<D>();
  // The shared-memory limit is a per-device attribute of the kernel: it is
  // set on every call, for whichever device is current (no process-wide
  // state, so several devices, threads and device resets need no care).
  cudaError_t e = cudaFuncSetAttribute(fa_fwd_kernel<D, MODE>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  // persistent: one CTA per SM (shared memory allows one), each walking the
  // heavy-first unit list with stride gridDim.x
  int dev = 0, n_sm = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // Packed ragged batches keep one unit per CTA: their unit costs vary with
  // the sequence lengths, which only the hardware's dynamic CTA scheduling
  // balances (with gridDim.x = units every CTA's sequence is just its own unit).
  const long long units = static_cast<long long>(p.n_rbu) * p.units_per_rbu;
  const unsigned int grid =
      static_cast<unsigned int>(p.cu_q ? units : std::min<long long>(units, n_sm));
  hook_before(stream);
  fa_fwd_kernel<D, MODE><<<grid, kThreads, smem, stream>>>(tq, tk, tv, p);
  hook_after(stream);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_fwd_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                         const FwdParams& p, cudaStream_t stream) {
  if (p.drop.on) return launch_fwd_dd<D, kModeDropout>(tq, tk, tv, p, stream);
  if (p.key_bits) return launch_fwd_dd<D, kModeKeyBits>(tq, tk, tv, p, stream);
  return launch_fwd_dd<D, kModePlain>(tq, tk, tv, p, stream);
}

}  // namespace

cudaError_t launch_fwd(int d, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       const FwdParams& p, cudaStream_t stream) {
  if (d == 128) return launch_fwd_d<128>(tq, tk, tv, p, stream);
  return launch_fwd_d<64>(tq, tk, tv, p, stream);
}

unsigned int read_fwd_status(bool clear) {
  unsigned int v = 0;
  cudaMemcpyFromSymbol(&v, g_status, sizeof v);
  if (clear) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_status, &z, sizeof z);
  }
  return v;
}

}  // namespace fa
