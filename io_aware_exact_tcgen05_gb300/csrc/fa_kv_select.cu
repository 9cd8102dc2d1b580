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

#include "fa_internal.h"
#include "fa_kv.h"
#include "fa_kv_device.cuh"

namespace fa {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreBlocks = 64;  // cache blocks per CTA
constexpr int kRowTile = 16;      // query rows quantised into shared memory at a time
constexpr int kSelectThreads = 256;  // 512: 5.6 us against 5.0 us for ten short items
constexpr int kSelectWarps = kSelectThreads / 32;

// Order-preserving map of a score to an unsigned key; NaN ranks lowest.
__device__ __forceinline__ uint32_t score_key(float s) {
  if (s != s) return 0u;
  const uint32_t u = __float_as_uint(s);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// (Read in L2: the selection asks before its own wait, when only L2 is sure to hold what
// kernels before the scores wrote.)
__device__ __forceinline__ int request_blocks(const SelectParams& p, int b) {
  const int ps = p.s.page_size;
  const long long n = min(static_cast<long long>(max(__ldcg(p.seqlens + b), 0)),
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

// Four lanes per block, each with a quarter of its 2 * D bounds: a query row costs a
// block 3.6 instructions (sixteen lanes per block, with two more steps of
// reduction, took 8.5).  HBM would bound the kernel; the latency of its three dependent
// loads (length and table, bounds, store) does for all but the longest tables.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) fa_block_score_kernel(const SelectParams p) {
  constexpr int LPB = 4;                        // lanes per block
  constexpr int VEC = 2 * D / (16 * LPB);       // 16-byte pieces per lane
  __shared__ __align__(16) int8_t s_q[kRowTile][2 * D];
  __shared__ float s_scale[kRowTile];
  static_assert(kScoreThreads / LPB == kScoreBlocks, "one block per four lanes");
  const int item = blockIdx.y;                  // (request, KV head)
  const int b = item / p.s.Hkv, hk = item - b * p.s.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = lane % LPB;
  const int blk = blockIdx.x * kScoreBlocks + threadIdx.x / LPB;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) +
                           static_cast<size_t>(item) * p.rows * D;
  griddep_wait();
  // the table's entry and the length are read side by side
  const int entry = blk < p.max_blocks ? p.block_table[static_cast<size_t>(b) * p.max_blocks + blk] : -1;
  const int n = request_blocks(p, b);
  if (static_cast<int>(blockIdx.x) * kScoreBlocks >= n) return;
  const bool ok = blk < n && entry >= 0 && entry < p.s.num_pages;
  // the bounds are on their way while q is quantised
  int4 w[VEC];
  float ks = 0.f;
#pragma unroll
  for (int i = 0; i < VEC; ++i) w[i] = make_int4(0, 0, 0, 0);
  if (ok) {
    const size_t tile = static_cast<size_t>(entry) * p.s.Hkv + hk;
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      w[i] = __ldg(reinterpret_cast<const int4*>(p.k_bounds + tile * 2 * D + (i * LPB + part) * 16));
    ks = p.k_scale[tile];
  }
  float best = __int_as_float(0xff800000);
  for (int r0 = 0; r0 < p.rows; r0 += kRowTile) {
    const int rows = min(kRowTile, p.rows - r0);
    __syncthreads();
    for (int r = warp; r < rows; r += kScoreThreads / 32) {
      const int e = quantise_row<D>(q + static_cast<size_t>(r0 + r) * D, s_q[r]);
      if (lane == 0) s_scale[r] = pow2i(e + 2);
    }
    __syncthreads();
#pragma unroll 2
    for (int r = 0; r < rows; ++r) {
      int u = 0;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int4 a = *reinterpret_cast<const int4*>(&s_q[r][(i * LPB + part) * 16]);
        u = __dp4a(a.x, w[i].x, __dp4a(a.y, w[i].y, __dp4a(a.z, w[i].z, __dp4a(a.w, w[i].w, u))));
      }
      u += __shfl_xor_sync(0xffffffffu, u, 1);
      u += __shfl_xor_sync(0xffffffffu, u, 2);
      const float s = static_cast<float>(u) * ks * s_scale[r];
      if (s > best || s != s) best = s;
    }
  }
  if (part == 0 && blk < n) {
    const bool forced = blk < p.n_first || blk >= n - p.n_last;
    p.keys[static_cast<size_t>(item) * p.max_blocks + blk] =
        forced ? 0xffffffffu : score_key(ok ? best : __int_as_float(0xff800000));
  }
  // the selection may launch now; earlier, its CTAs would take places that this
  // grid's own still need (22.6 us against 18.7 us for 2048 blocks x 64 items)
  griddep_launch_dependents();
}

// The k = min(k_blocks, n) blocks with the largest keys of one (request, KV
// head), ascending; equal keys by the lower index.  The k-th largest key T (the
// largest T with at least k keys >= T) is found two bits at a time: each step
// counts the keys at three candidates and costs one barrier; it ends early when a
// candidate has exactly k keys at or above it.  The blocks above T and
// the first of those equal to T are then written in order.  One CTA per item;
// latency bounds it, so the keys stay in registers (thread t holds blocks t, t +
// 256, ...) unless there are more than 8192 of them.
template <int kRounds>
__device__ __forceinline__ void select_blocks(const SelectParams& p, int item, int n, int k,
                                              const uint32_t* keys) {
  __shared__ int s_count[2][3][kSelectWarps];
  __shared__ int s_warp[2][2][kSelectWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* out = p.sel + static_cast<size_t>(item) * p.k_blocks;
  constexpr bool kInRegs = kRounds > 0;
  const int rounds = kInRegs ? kRounds : (n + kSelectThreads - 1) / kSelectThreads;
  uint32_t mine[kInRegs ? kRounds : 1];
  if (kInRegs) {
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int at = i * kSelectThreads + tid;
      mine[i] = at < n ? keys[at] : 0u;  // 0 is below every candidate
    }
  }
  // The keys that are not forced agree in their upper bits: the search starts below
  // them.
  uint32_t lo = 0xffffffffu, hi = 0u;
  auto widen = [&](uint32_t key) {
    if (key != 0xffffffffu) lo = min(lo, key), hi = max(hi, key);
  };
  if (kInRegs) {
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      if (i * kSelectThreads + tid < n) widen(mine[i]);
  } else {
    for (int at = tid; at < n; at += kSelectThreads) widen(keys[at]);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    s_warp[0][0][warp] = static_cast<int>(lo);
    s_warp[0][1][warp] = static_cast<int>(hi);
  }
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, lane < kSelectWarps ? static_cast<uint32_t>(s_warp[0][0][lane])
                                                          : 0xffffffffu);
  hi = __reduce_max_sync(0xffffffffu, lane < kSelectWarps ? static_cast<uint32_t>(s_warp[0][1][lane])
                                                          : 0u);
  uint32_t T = 0;
  int bit = 0;
  if (lo > hi) {
    T = 0xffffffffu;  // every block is forced
    bit = -2;
  } else if (lo == hi) {
    T = lo;
    bit = -2;
  } else {
    bit = (31 - __clz(lo ^ hi)) & ~1;
    T = bit < 30 ? hi >> (bit + 2) << (bit + 2) : 0u;
  }
  for (; bit >= 0; bit -= 2) {
    int c1 = 0, c2 = 0, c3 = 0;
    const uint32_t t1 = T | 1u << bit, t2 = T | 2u << bit, t3 = T | 3u << bit;
    if (kInRegs) {
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        c1 += mine[i] >= t1;
        c2 += mine[i] >= t2;
        c3 += mine[i] >= t3;
      }
    } else {
      for (int at = tid; at < n; at += kSelectThreads) {
        const uint32_t key = keys[at];
        c1 += key >= t1;
        c2 += key >= t2;
        c3 += key >= t3;
      }
    }
    c1 = __reduce_add_sync(0xffffffffu, c1);
    c2 = __reduce_add_sync(0xffffffffu, c2);
    c3 = __reduce_add_sync(0xffffffffu, c3);
    const int turn = bit >> 1 & 1;  // two buffers: one barrier a step is enough
    if (lane == 0) {
      s_count[turn][0][warp] = c1;
      s_count[turn][1][warp] = c2;
      s_count[turn][2][warp] = c3;
    }
    __syncthreads();
    int x = lane < kSelectWarps ? s_count[turn][0][lane] : 0;
    int y = lane < kSelectWarps ? s_count[turn][1][lane] : 0;
    int z = lane < kSelectWarps ? s_count[turn][2][lane] : 0;
    x = __reduce_add_sync(0xffffffffu, x);
    y = __reduce_add_sync(0xffffffffu, y);
    z = __reduce_add_sync(0xffffffffu, z);
    // exactly k keys from a candidate on: they are the selection, without ties
    if (z == k || y == k || x == k) {
      T = (z == k ? t3 : y == k ? t2 : t1) - 1;
      break;
    }
    T = z >= k ? t3 : y >= k ? t2 : x >= k ? t1 : T;
  }
  __syncthreads();  // the counts of the last step have been read
  // keys above T over the whole item, then the order inside it, 256 blocks at a time
  int above = 0;
  if (kInRegs) {
#pragma unroll
    for (int i = 0; i < kRounds; ++i) above += mine[i] > T;
  } else {
    for (int at = tid; at < n; at += kSelectThreads) above += keys[at] > T;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  if (lane == 0) s_count[1][0][warp] = above;
  __syncthreads();
  above = __reduce_add_sync(0xffffffffu, lane < kSelectWarps ? s_count[1][0][lane] : 0);
  int ties = k - above;  // blocks equal to T still to be taken
  int base = 0;
#pragma unroll(kInRegs ? kRounds : 1)
  for (int i = 0; i < rounds; ++i) {
    const int at = i * kSelectThreads + tid;
    uint32_t key = 0;
    if (kInRegs) {
      key = mine[i];
    } else if (at < n) {
      key = keys[at];
    }
    const uint32_t upper = __ballot_sync(0xffffffffu, at < n && key > T);
    const uint32_t equal = __ballot_sync(0xffffffffu, at < n && key == T);
    const int turn = i & 1;
    if (lane == 0) {
      s_warp[turn][0][warp] = __popc(upper);
      s_warp[turn][1][warp] = __popc(equal);
    }
    __syncthreads();
    int u = lane < kSelectWarps ? s_warp[turn][0][lane] : 0;
    int e = lane < kSelectWarps ? s_warp[turn][1][lane] : 0;
    const int u_all = __reduce_add_sync(0xffffffffu, u), e_all = __reduce_add_sync(0xffffffffu, e);
    const int u_before = __reduce_add_sync(0xffffffffu, lane < warp ? u : 0);
    const int e_before = __reduce_add_sync(0xffffffffu, lane < warp ? e : 0);
    const uint32_t below = (1u << lane) - 1;
    const int eq_rank = e_before + __popc(equal & below);  // among this round's equal keys
    const bool take = (upper >> lane & 1u) || ((equal >> lane & 1u) && eq_rank < ties);
    if (take) out[base + u_before + __popc(upper & below) + min(eq_rank, ties)] = at;
    base += u_all + min(e_all, ties);
    ties -= min(e_all, ties);
  }
}

__global__ void __launch_bounds__(kSelectThreads) fa_block_select_kernel(const SelectParams p) {
  const int item = blockIdx.x;
  const int n = request_blocks(p, item / p.s.Hkv);
  const int k = min(p.k_blocks, n);
  int32_t* out = p.sel + static_cast<size_t>(item) * p.k_blocks;
  griddep_wait();  // the keys are complete and visible
  if (threadIdx.x == 0) p.n_sel[item] = k;
  for (int i = k + threadIdx.x; i < p.k_blocks; i += kSelectThreads) out[i] = -1;
  if (k == 0) return;
  const uint32_t* keys = p.keys + static_cast<size_t>(item) * p.max_blocks;
  // as few comparisons as the item needs: 256, 512, ... 8192 blocks
  const int rounds = (n + kSelectThreads - 1) / kSelectThreads;
  if (rounds <= 1) select_blocks<1>(p, item, n, k, keys);
  else if (rounds <= 2) select_blocks<2>(p, item, n, k, keys);
  else if (rounds <= 4) select_blocks<4>(p, item, n, k, keys);
  else if (rounds <= 8) select_blocks<8>(p, item, n, k, keys);
  else if (rounds <= 16) select_blocks<16>(p, item, n, k, keys);
  else if (rounds <= 32) select_blocks<32>(p, item, n, k, keys);
  else select_blocks<0>(p, item, n, k, keys);
}

}  // namespace

cudaError_t launch_select(const SelectParams& p, cudaStream_t stream) {
  const int items = p.B * p.s.Hkv;
  const dim3 grid((p.max_blocks + kScoreBlocks - 1) / kScoreBlocks, items);
  const cudaError_t e =
      launch_dependent(p.s.d == 128 ? fa_block_score_kernel<128> : fa_block_score_kernel<64>, grid,
                       dim3(kScoreThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_dependent(fa_block_select_kernel, dim3(items), dim3(kSelectThreads), 0, stream, p);
}

}  // namespace fa
