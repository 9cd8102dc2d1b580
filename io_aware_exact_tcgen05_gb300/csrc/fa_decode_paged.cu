// fa_decode_paged.cu -- attention of the last Sq tokens of each request over a
// paged 8-bit KV cache, over every block or over a list of chosen blocks.
//
// One CTA per (request, KV head, query row); each warp walks the keys with a
// running maximum and sum, one key at a time, and the warps' states are merged
// at the end (the rescale rule of the online softmax).
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <math.h>

#include "fa_kv.h"
#include "fa_kv_device.cuh"

namespace fa {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

template <int D>
__global__ void __launch_bounds__(kWarps * 32) fa_decode_paged_kernel(const PagedDecodeParams p) {
  constexpr int E = D / 32;  // channels per lane
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  const int item = blockIdx.y, row = blockIdx.x;
  const int b = item / p.s.Hkv, hk = item % p.s.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ps = p.s.page_size;
  const long long room = static_cast<long long>(p.max_blocks) * ps;
  const long long len = min(static_cast<long long>(max(p.seqlens[b], 0)), room);
  const long long last = len - p.Sq + row % p.Sq;  // last key this row sees
  const size_t qrow = static_cast<size_t>(item) * p.rows + row;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + qrow * D + lane * E;
  float qv[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = __bfloat162float(q[e]) * p.scale_log2;
    acc[e] = 0.f;
  }
  float m = neg_inf(), l = 0.f;
  const int n_blk = static_cast<int>((len + ps - 1) / ps);
  const int n_list = p.sel ? min(max(p.n_sel[item], 0), p.max_sel) : n_blk;
  for (int i = warp; i < n_list; i += kWarps) {
    const int blk = p.sel ? p.sel[static_cast<size_t>(item) * p.max_sel + i] : i;
    if (blk < 0 || blk >= n_blk) continue;
    const int page = p.block_table[static_cast<size_t>(b) * p.max_blocks + blk];
    if (page < 0 || page >= p.s.num_pages) continue;
    const size_t tile = static_cast<size_t>(page) * p.s.Hkv + hk;
    const float ks = p.k_scale[tile], vs = p.v_scale[tile];
    const uint8_t* kp = static_cast<const uint8_t*>(p.k_cache) + tile * ps * D + lane * E;
    const uint8_t* vp = static_cast<const uint8_t*>(p.v_cache) + tile * ps * D + lane * E;
    const int n = static_cast<int>(min(static_cast<long long>(ps), last + 1 - 1LL * blk * ps));
    for (int j = 0; j < n; ++j) {
      float s = 0.f, v[E];
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 kk =
            e4m3x2_to_f32x2(*reinterpret_cast<const uint16_t*>(kp + static_cast<size_t>(j) * D + e));
        const float2 vv =
            e4m3x2_to_f32x2(*reinterpret_cast<const uint16_t*>(vp + static_cast<size_t>(j) * D + e));
        s = fmaf(qv[e], kk.x, fmaf(qv[e + 1], kk.y, s));
        v[e] = vv.x * vs;
        v[e + 1] = vv.y * vs;
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      s *= ks;
      const float m_new = fmaxf(m, s);
      const float alpha = (m == neg_inf()) ? 0.f : exp2f(m - m_new);
      const float w = (s == neg_inf()) ? 0.f : exp2f(s - m_new);
      m = m_new;
      l = l * alpha + w;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w, v[e], acc[e] * alpha);
    }
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kWarps * 32) {
    float M = neg_inf(), L = 0.f, o = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
    for (int w = 0; w < kWarps; ++w) {
      const float wt = (s_m[w] == neg_inf()) ? 0.f : exp2f(s_m[w] - M);
      L = fmaf(wt, s_l[w], L);
      o = fmaf(wt, s_o[w][c], o);
    }
    const bool empty = L == 0.f;
    static_cast<__nv_bfloat16*>(p.o)[qrow * D + c] = __float2bfloat16_rn(empty ? 0.f : o / L);
    if (p.lse && c == 0)
      p.lse[qrow] = empty ? neg_inf() : (M + log2f(L)) * 0.69314718055994530942f;
  }
}

}  // namespace

size_t decode_paged_workspace(int B, int Hkv, int rows, int d) {
  (void)B, (void)Hkv, (void)rows, (void)d;
  return 0;
}

cudaError_t launch_decode_paged(const PagedDecodeParams& p, cudaStream_t stream) {
  const dim3 grid(p.rows, p.B * p.s.Hkv);
  if (p.s.d == 128) fa_decode_paged_kernel<128><<<grid, kWarps * 32, 0, stream>>>(p);
  else fa_decode_paged_kernel<64><<<grid, kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
