// fa_kv_select.cu -- the blocks of a paged cache that a query attends: a cheap
// upper bound of every block's scores, then the k_blocks largest per KV head.
//
//   q8_i = rint(q_i / 2^e), e the smallest with amax(q) <= 127 * 2^e
//   u    = sum_i max(q8_i * M_i, q8_i * m_i)        (M, m: the block's bounds)
//   score = max over the KV head's query rows of u * k_scale * 2^(e + 2)
//
// |q8| <= 127, |M|, |m| <= 112 and d <= 128, so u is an integer below 2^21: it is
// exact in any order of summation, and with power-of-two scales so is the
// score.  Equal scores are then truly equal and the lower block wins.
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "fa_kv.h"
#include "fa_kv_device.cuh"

namespace fa {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreBlocks = 64;  // cache blocks per CTA
constexpr int kRowTile = 16;      // query rows quantised into shared memory at a time
constexpr int kSelectThreads = 512;

// Order-preserving map of a score to an unsigned key; NaN ranks lowest.
__device__ __forceinline__ uint32_t score_key(float s) {
  if (s != s) return 0u;
  const uint32_t u = __float_as_uint(s);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int request_blocks(const SelectParams& p, int b) {
  const int ps = p.s.page_size;
  const long long n = min(static_cast<long long>(max(p.seqlens[b], 0)),
                          static_cast<long long>(p.max_blocks) * ps);
  return static_cast<int>((n + ps - 1) / ps);
}

// One row of q as 8-bit integers: positive parts in dst[0, D), negative parts in
// dst[D, 2D), so that u is one product of 2 * D values with (M, m).  One warp.
template <int D>
__device__ __forceinline__ int quantise_row(const __nv_bfloat16* q, int8_t* dst) {
  const int lane = threadIdx.x & 31;
  float v[D / 32];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const uint32_t bits = reinterpret_cast<const uint16_t*>(q)[lane + 32 * i];
    v[i] = __uint_as_float(bits << 16);
    top = max(top, bits & 0x7fffu);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  // smallest e with amax <= 127 * 2^e = (127 / 64) * 2^(e + 6): 127 / 64 is bf16's 1 + 0x7e / 128
  int e = static_cast<int>(top >> 7) - 127 - 6 + ((top & 0x7fu) > 0x7eu ? 1 : 0);
  e = min(max(e, kScaleExpMin), kScaleExpMax);
  const float inv = pow2i(-e);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int w = min(max(__float2int_rn(v[i] * inv), -127), 127);
    dst[lane + 32 * i] = static_cast<int8_t>(max(w, 0));
    dst[D + lane + 32 * i] = static_cast<int8_t>(min(w, 0));
  }
  return e;
}

template <int D>
__global__ void __launch_bounds__(kScoreThreads) fa_block_score_kernel(const SelectParams p) {
  constexpr int LPB = 2 * D / 16;               // lanes per block: 16 bytes of bounds each
  constexpr int BPW = 32 / LPB;                 // blocks per warp at a time
  constexpr int WARPS = kScoreThreads / 32;
  __shared__ __align__(16) int8_t s_q[kRowTile][2 * D];
  __shared__ float s_scale[kRowTile];
  const int item = blockIdx.y;                  // (request, KV head)
  const int b = item / p.s.Hkv, hk = item % p.s.Hkv;
  const int n = request_blocks(p, b);
  const int first = blockIdx.x * kScoreBlocks;
  if (first >= n) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = lane % LPB, sub = lane / LPB;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) +
                           static_cast<size_t>(item) * p.rows * D;
  constexpr int PER = kScoreBlocks / (WARPS * BPW);
  float best[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) best[i] = __int_as_float(0xff800000);
  for (int r0 = 0; r0 < p.rows; r0 += kRowTile) {
    const int rows = min(kRowTile, p.rows - r0);
    __syncthreads();
    for (int r = warp; r < rows; r += WARPS) {
      const int e = quantise_row<D>(q + static_cast<size_t>(r0 + r) * D, s_q[r]);
      if (lane == 0) s_scale[r] = pow2i(e + 2);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int blk = first + (i * WARPS + warp) * BPW + sub;
      const int page = blk < n ? p.block_table[static_cast<size_t>(b) * p.max_blocks + blk] : -1;
      const bool ok = page >= 0 && page < p.s.num_pages;
      int4 w = make_int4(0, 0, 0, 0);
      float ks = 0.f;
      if (ok) {
        const size_t tile = static_cast<size_t>(page) * p.s.Hkv + hk;
        w = *reinterpret_cast<const int4*>(p.k_bounds + tile * 2 * D + part * 16);
        ks = p.k_scale[tile];
      }
      for (int r = 0; r < rows; ++r) {
        const int4 a = *reinterpret_cast<const int4*>(&s_q[r][part * 16]);
        int u = __dp4a(a.x, w.x, __dp4a(a.y, w.y, __dp4a(a.z, w.z, __dp4a(a.w, w.w, 0))));
#pragma unroll
        for (int o = 1; o < LPB; o <<= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
        const float s = static_cast<float>(u) * ks * s_scale[r];
        if (ok && (s > best[i] || s != s)) best[i] = s;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int blk = first + (i * WARPS + warp) * BPW + sub;
    if (part == 0 && blk < n) {
      const bool forced = blk < p.n_first || blk >= n - p.n_last;
      p.keys[static_cast<size_t>(item) * p.max_blocks + blk] =
          forced ? 0xffffffffu : score_key(best[i]);
    }
  }
}

// The k = min(k_blocks, n) blocks with the largest keys of one (request, KV
// head), ascending; equal keys by the lower index.  The k-th largest key T is
// found bit by bit (the largest T with at least k keys >= T); the blocks above T
// and the first of those equal to T are then written in order.
__global__ void __launch_bounds__(kSelectThreads) fa_block_select_kernel(const SelectParams p) {
  __shared__ int s_count;
  __shared__ int s_warp[2][kSelectThreads / 32];
  const int item = blockIdx.x;
  const int b = item / p.s.Hkv;
  const int n = request_blocks(p, b);
  const int k = min(p.k_blocks, n);
  const uint32_t* keys = p.keys + static_cast<size_t>(item) * p.max_blocks;
  int32_t* out = p.sel + static_cast<size_t>(item) * p.k_blocks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) p.n_sel[item] = k;
  for (int i = k + tid; i < p.k_blocks; i += kSelectThreads) out[i] = -1;
  if (k == 0) return;
  uint32_t T = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t cand = T | (1u << bit);
    int c = 0;
    for (int i = tid; i < n; i += kSelectThreads) c += keys[i] >= cand;
    c = __reduce_add_sync(0xffffffffu, c);
    __syncthreads();
    if (tid == 0) s_count = 0;
    __syncthreads();
    if (lane == 0) atomicAdd(&s_count, c);
    __syncthreads();
    if (s_count >= k) T = cand;
  }
  // thread t owns blocks [t * per, (t + 1) * per)
  const int per = (n + kSelectThreads - 1) / kSelectThreads;
  const int lo = min(tid * per, n), hi = min(lo + per, n);
  int above = 0, equal = 0;
  for (int i = lo; i < hi; ++i) {
    above += keys[i] > T;
    equal += keys[i] == T;
  }
  int ia = above, ie = equal;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, ia, o), e = __shfl_up_sync(0xffffffffu, ie, o);
    if (lane >= o) {
      ia += a;
      ie += e;
    }
  }
  if (lane == 31) {
    s_warp[0][warp] = ia;
    s_warp[1][warp] = ie;
  }
  __syncthreads();
  int before_a = ia - above, before_e = ie - equal, total_a = 0;
  for (int w = 0; w < kSelectThreads / 32; ++w) {
    if (w < warp) {
      before_a += s_warp[0][w];
      before_e += s_warp[1][w];
    }
    total_a += s_warp[0][w];
  }
  const int ties = k - total_a;  // blocks equal to T that are taken
  int pos = before_a + min(before_e, ties);
  for (int i = lo; i < hi; ++i) {
    const uint32_t key = keys[i];
    if (key > T || (key == T && before_e++ < ties)) out[pos++] = i;
  }
}

}  // namespace

cudaError_t launch_select(const SelectParams& p, cudaStream_t stream) {
  const int items = p.B * p.s.Hkv;
  const dim3 grid((p.max_blocks + kScoreBlocks - 1) / kScoreBlocks, items);
  if (p.s.d == 128) fa_block_score_kernel<128><<<grid, kScoreThreads, 0, stream>>>(p);
  else fa_block_score_kernel<64><<<grid, kScoreThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  fa_block_select_kernel<<<items, kSelectThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
