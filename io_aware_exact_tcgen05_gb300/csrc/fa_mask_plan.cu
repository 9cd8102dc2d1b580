// fa_mask_plan.cu -- masks as one interval of visible keys for each row (documents, prefixes,
// windows, padding), and the tile plan by which the attention kernels skip.
//
// An interval per row is all that these masks need: a document is an interval, the causal rule
// and a prefix move its end, a window moves its start.  It costs 8 bytes a row where a mask of
// bits costs Sk / 8, and the tiles to visit follow from the intervals' extremes.
//
// Every kernel here is bound by its launch and a short chain of dependent loads: the work
// is 8 bytes a row.
#include <algorithm>

#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_scored.h"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

// lo, hi of every row: the document of the row's position by binary search.
__global__ void __launch_bounds__(256) fa_row_bounds_kernel(const RowBoundsParams p) {
  const long long idx = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (idx >= static_cast<long long>(p.B) * p.Sq) return;
  const int b = static_cast<int>(idx / p.Sq);
  const int i = static_cast<int>(idx - static_cast<long long>(b) * p.Sq);
  const int pos = i + p.Sk - p.Sq;  // the row's position among the keys
  int start = 0, end = p.Sk, prefix = 0;
  bool live = true;
  if (p.cu_docs) {
    const long long row0 = static_cast<long long>(b) * p.Sk;
    const int at = static_cast<int>(row0) + pos;  // the host keeps B * Sk below 2^31
    live = pos >= 0;
    // largest d with cu_docs[d] <= at
    int d = -1, above = p.n_docs + 1;
    while (above - d > 1) {
      const int mid = (d + above) >> 1;
      if (__ldg(p.cu_docs + mid) <= at) d = mid; else above = mid;
    }
    if (d < 0 || d >= p.n_docs) {
      live = false;
    } else {
      start = static_cast<int>(max(0ll, p.cu_docs[d] - row0));
      end = static_cast<int>(max(0ll, min(static_cast<long long>(p.Sk), p.cu_docs[d + 1] - row0)));
      if (p.prefix) prefix = p.prefix[d];
    }
  } else if (p.prefix) {
    prefix = p.prefix[b];
  }
  long long lo = start, hi = end;
  if (p.causal) hi = min(hi, max(pos + 1ll, static_cast<long long>(start) + prefix));
  if (p.window > 0) {
    lo = max(lo, static_cast<long long>(pos) - p.window + 1);
    if (!p.causal) hi = min(hi, static_cast<long long>(pos) + p.window);
  }
  if (!live || prefix < 0 || hi <= lo) lo = hi = 0;
  p.lo[idx] = static_cast<int>(lo);
  p.hi[idx] = static_cast<int>(hi);
}

__device__ __forceinline__ int key_tiles(int4 r) {
  return r.y > r.x ? (r.y + 127) / 128 - r.x / 128 : 0;
}

// The intervals clamped to [0, Sk], and their extremes over each 128-row tile.
__global__ void __launch_bounds__(128)
    fa_plan_rows_kernel(const int32_t* lo, const int32_t* hi, int Sq, int Sk, const MaskPlan m) {
  __shared__ int red[4][4];
  const int b = blockIdx.y, t = blockIdx.x;
  const int i = t * 128 + threadIdx.x;
  int l = 0, h = 0;
  if (i < Sq) {
    const size_t idx = static_cast<size_t>(b) * Sq + i;
    l = max(0, lo[idx]);
    h = min(Sk, hi[idx]);
    if (h <= l) l = h = 0;
    const_cast<int2*>(m.rows)[idx] = make_int2(l, h);
  }
  const bool live = h > l;
  const int mn_l = __reduce_min_sync(0xffffffffu, live ? l : 0x7fffffff);
  const int mx_h = __reduce_max_sync(0xffffffffu, live ? h : 0);
  const int mx_l = __reduce_max_sync(0xffffffffu, live ? l : 0);
  const int mn_h = __reduce_min_sync(0xffffffffu, live ? h : 0x7fffffff);
  const int w = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    red[w][0] = mn_l;
    red[w][1] = mx_h;
    red[w][2] = mx_l;
    red[w][3] = mn_h;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int4 r = make_int4(min(min(red[0][0], red[1][0]), min(red[2][0], red[3][0])),
                       max(max(red[0][1], red[1][1]), max(red[2][1], red[3][1])),
                       max(max(red[0][2], red[1][2]), max(red[2][2], red[3][2])),
                       min(min(red[0][3], red[1][3]), min(red[2][3], red[3][3])));
    if (r.y == 0) r = make_int4(0, 0, 0, 0);
    const size_t at = static_cast<size_t>(b) * m.nq + t;
    const_cast<int4*>(m.qt)[at] = r;
    const_cast<int*>(m.work)[at] = key_tiles(r);
  }
  griddep_launch_dependents();
}

// First and end query tile whose hull of intervals meets each key tile, and the hull of theirs;
// the work of key tiles and of pairs of query tiles.  A warp per key tile.
__global__ void __launch_bounds__(256) fa_plan_keys_kernel(const MaskPlan m) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int kt = blockIdx.x * 8 + (threadIdx.x >> 5);
  griddep_wait();
  const int4* qt = m.qt + static_cast<size_t>(b) * m.nq;
  const int c0 = kt * 128;
  if (kt < m.nk) {
    int first = 0x7fffffff, end = 0, lo = 0x7fffffff, hi = 0;
#pragma unroll 4
    for (int t = lane; t < m.nq; t += 32) {
      const int4 r = qt[t];
      if (r.x < c0 + 128 && r.y > c0) {
        first = min(first, t);
        end = t + 1;
        lo = min(lo, r.x);
        hi = max(hi, r.y);
      }
    }
    first = __reduce_min_sync(0xffffffffu, first);
    end = __reduce_max_sync(0xffffffffu, end);
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (end == 0) first = 0;
    if (lane == 0) {
      const size_t at = static_cast<size_t>(b) * m.nk + kt;
      const_cast<int4*>(m.kt)[at] = make_int4(first, end, lo, hi);
      const_cast<int*>(m.work)[static_cast<size_t>(m.B) * (m.nq + m.np) + at] = end - first;
    }
  }
  if (kt < m.np && lane == 0)
    const_cast<int*>(m.work)[static_cast<size_t>(m.B) * m.nq + static_cast<size_t>(b) * m.np + kt] =
        key_tiles(qt[2 * kt]) + (2 * kt + 1 < m.nq ? key_tiles(qt[2 * kt + 1]) : 0);
  griddep_launch_dependents();
}

// The order of the tiles by rank: the number of tiles with more work (or as much, before them in
// ties).  A warp per tile.  Over all batch rows together: with an order for each, taken side by
// side, the slowest of 152 CTAs had 10% more than the mean where the rows' masks differ.  Causal
// masks give late query tiles and early key tiles more work, so ties of query tiles rank late ones
// first.  (5 us with the two kernels before at 2 x 8192 rows, 0.1 ms at 10^6; 8 tiles a warp, which
// share its loads: 6 us, 0.18 ms.)
__global__ void __launch_bounds__(256) fa_plan_order_kernel(const MaskPlan m) {
  const int kind = blockIdx.y;  // query tiles, pairs of them, key tiles, key tiles of a batch row
  const int per_row = kind == 0 ? m.nq : kind == 1 ? m.np : m.nk;
  const int n = m.B * per_row;
  const long long e = blockIdx.x * 8ll + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  griddep_wait();
  if (e >= n) return;
  const int tile = static_cast<int>(e);
  const long long skip = kind == 0 ? 0 : 1ll * m.B * (kind == 1 ? m.nq : m.nq + m.np);
  const int* work = m.work + skip;
  const int first = kind == 3 ? tile / per_row * per_row : 0, end = kind == 3 ? first + per_row : n;
  const int mine = work[tile];
  // least work that counts in front of the tile and behind it
  const int front = kind >= 2 ? mine : mine + 1, behind = kind >= 2 ? mine + 1 : mine;
  int rank = 0;
#pragma unroll 4
  for (int x = first + lane; x < tile; x += 32) rank += work[x] >= front;
#pragma unroll 4
  for (int x = tile + 1 + lane; x < end; x += 32) rank += work[x] >= behind;
  rank = __reduce_add_sync(0xffffffffu, rank);
  int* out = const_cast<int*>(kind == 0   ? m.by_q1
                              : kind == 1 ? m.by_q2
                              : kind == 2 ? m.by_k
                                          : m.by_k_row);
  if (lane == 0) out[first + rank] = tile;
}

}  // namespace

cudaError_t launch_row_bounds(const RowBoundsParams& p, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.B) * p.Sq;
  fa_row_bounds_kernel<<<static_cast<unsigned int>((rows + 255) / 256), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_mask_plan(const int32_t* lo, const int32_t* hi, int B, int Sq, int Sk,
                             const MaskPlan& m, cudaStream_t stream) {
  fa_plan_rows_kernel<<<dim3(m.nq, B), 128, 0, stream>>>(lo, hi, Sq, Sk, m);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = launch_dependent(fa_plan_keys_kernel, dim3((std::max(m.nk, m.np) + 7) / 8, B), dim3(256), 0, stream,
                         m);
  const long long most = 1ll * B * std::max(m.nq, m.nk);
  if (e == cudaSuccess)
    e = launch_dependent(fa_plan_order_kernel, dim3(static_cast<unsigned int>((most + 7) / 8), 4),
                         dim3(256), 0, stream, m);
  return e;
}

}  // namespace fa
