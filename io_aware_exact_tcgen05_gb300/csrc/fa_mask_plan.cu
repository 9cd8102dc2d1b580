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
#include "fa_score.cuh"
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

// The intervals clamped to [0, Sk], and their extremes over each 128-row tile.  Where the interval of
// every row with keys meets or touches that of the row with keys before it, as with documents, windows and
// prefixes, no key between the extremes is unseen; only else is it looked for, every row's end against
// every interval.
__global__ void __launch_bounds__(128)
    fa_plan_rows_kernel(const int32_t* lo, const int32_t* hi, int Sq, int Sk, const MaskPlan m) {
  __shared__ int2 row[128];
  __shared__ int4 red[4];       // of a warp's rows: min lo, max hi, 1 where intervals are apart | 2 where they
                                // go past their rows' positions, whether all rows see their own
  __shared__ int2 ends[4][2];   // the first and the last interval of a warp's rows
  __shared__ int part[4];
  const int b = blockIdx.y, t = blockIdx.x;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
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
  const uint32_t alive = __ballot_sync(0xffffffffu, live);
  const uint32_t before = alive & ((1u << lane) - 1);
  const int last = before ? 31 - __clz(before) : lane;
  const int pl = __shfl_sync(0xffffffffu, l, last), ph = __shfl_sync(0xffffffffu, h, last);
  const bool breaks = __any_sync(0xffffffffu, live && before && (l > ph || pl > h));
  const int p = i + (Sk - Sq);
  const bool past = __any_sync(0xffffffffu, live && h > p + 1);
  const bool own = __all_sync(0xffffffffu, i >= Sq || (live && l <= p && h > p));
  const int mn_l = __reduce_min_sync(0xffffffffu, live ? l : 0x7fffffff);
  const int mx_h = __reduce_max_sync(0xffffffffu, live ? h : 0);
  row[threadIdx.x] = make_int2(l, h);
  if (live && !before) ends[w][0] = make_int2(l, h);
  if (live && !(alive >> lane >> 1)) ends[w][1] = make_int2(l, h);
  if (lane == 0) red[w] = make_int4(mn_l, mx_h, (breaks ? 1 : 0) | (past ? 2 : 0), own);
  __syncthreads();
  int first = 0x7fffffff, end = 0, prev = -1;
  bool apart = false, beyond = false, all_own = true;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int4 r = red[k];
    all_own = all_own && r.w;
    if (r.y == 0) continue;
    if (prev >= 0 && (ends[k][0].x > ends[prev][1].y || ends[prev][1].x > ends[k][0].y)) apart = true;
    prev = k;
    first = min(first, r.x);
    end = max(end, r.y);
    apart = apart || (r.z & 1);
    beyond = beyond || (r.z & 2);
  }
  int n_gaps = 0;
  int4 gap = make_int4(0, 0, 0, 0);
  if (apart) {  // (CTA-uniform)
    // Ends of intervals that the next row neither sees nor shares are looked for in every row's; a stretch starts at one
    // that none sees and ends at the next interval's first.
    const int2 next = row[(threadIdx.x + 1) & 127];
    const uint32_t ask = __ballot_sync(0xffffffffu, live && h < end && next.y != h && !(next.x <= h && next.y > h));
    if (lane == 0) part[w] = static_cast<int>(ask);
    __syncthreads();
    int start[2] = {-1, -1}, covered = -1;
    for (int k = 0; k < 4 && n_gaps < 3; ++k)
      for (uint32_t todo = static_cast<uint32_t>(part[k]); todo && n_gaps < 3; todo &= todo - 1) {
        const int key = row[32 * k + __ffs(todo) - 1].y;
        if (key == start[0] || key == start[1] || key == covered) continue;
        if (__syncthreads_or(l <= key && h > key)) {
          covered = key;
          continue;
        }
        ++n_gaps;
        if (n_gaps == 2) start[1] = max(start[0], key);
        start[0] = n_gaps == 1 ? key : min(start[0], key);
      }
    auto first_behind = [&](int key) {  // of the intervals
      const int x = __reduce_min_sync(0xffffffffu, live && l > key ? l : 0x7fffffff);
      __syncthreads();  // what part held has been read
      if (lane == 0) part[w] = x;
      __syncthreads();
      return min(min(part[0], part[1]), min(part[2], part[3]));
    };
    if (n_gaps == 1 || n_gaps == 2) {
      gap.x = start[0];
      gap.y = first_behind(start[0]);
    }
    if (n_gaps == 2) {
      gap.z = start[1];
      gap.w = first_behind(start[1]);
    }
  }
  if (threadIdx.x == 0) {
    const int4 r = end > 0 ? make_int4(first, end, n_gaps, !beyond ? 0 : all_own ? 1 : 2) : make_int4(0, 0, 0, 0);
    const size_t at = static_cast<size_t>(b) * m.nq + t;
    const_cast<int4*>(m.qt)[at] = r;
    const_cast<int4*>(m.gaps)[at] = gap;
    const_cast<int*>(m.work)[at] = key_tiles(r);
    if (at == 0) *const_cast<int4*>(m.sizes) = make_int4(m.B, Sq, Sk, kPlanMark);
  }
  griddep_launch_dependents();
}

// The bits of all lanes together; true where they are all of those there.
__device__ __forceinline__ bool gather_bits(uint32_t (&bits)[4], const uint32_t (&there)[4]) {
  bool all = true;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    bits[w] = __reduce_or_sync(0xffffffffu, bits[w]);
    all = all && bits[w] == there[w];
  }
  return all;
}

// First and end query tile whose hull of intervals meets each key tile, and which of its keys any row sees,
// also under the causal rule; the work of key tiles and of pairs of query tiles.  A warp per key tile.  The
// rows of a query tile are looked at one by one only where no hull holds the whole tile and its own and its gaps do not
// tell: where it has more than two, or where the causal rule cuts into it.
__global__ void __launch_bounds__(256) fa_plan_keys_kernel(const MaskPlan m, int Sq, int Sk) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int kt = blockIdx.x * 8 + (threadIdx.x >> 5);
  griddep_wait();
  const int4* qt = m.qt + static_cast<size_t>(b) * m.nq;
  const int c0 = kt * 128, c1 = min(c0 + 128, Sk), off = Sk - Sq;
  if (kt < m.nk) {
    int first = 0x7fffffff, end = 0;
    bool whole = false, whole_causal = false;  // a hull without gaps holds the tile
    for (int t0 = lane; t0 - lane < m.nq; t0 += 128) {
      int4 r[4];
      bool meets[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        r[u] = t0 + 32 * u < m.nq ? qt[t0 + 32 * u] : make_int4(0, 0, 0, 0);
#pragma unroll
      for (int u = 0; u < 4; ++u) meets[u] = r[u].x < c1 && r[u].y > c0;
      // (none does mostly, where documents are many)
      if (!__any_sync(0xffffffffu, meets[0] || meets[1] || meets[2] || meets[3])) continue;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (t0 - lane + 32 * u >= m.nq) break;
        if (!meets[u]) continue;
        first = min(first, t0 + 32 * u);
        end = t0 + 32 * u + 1;
        const bool holds = r[u].x <= c0 && r[u].y >= c1 && !r[u].z;
        whole = whole || holds;
        // (the position of a row of the tile from which on the rule cuts: the first, or where rows see their own the last)
        const int p = min((t0 + 32 * u) * 128 + (r[u].w == 1 ? 127 : 0), Sq - 1) + off;
        whole_causal = whole_causal || (holds && (!r[u].w || p >= c1 - 1));
      }
    }
    first = __reduce_min_sync(0xffffffffu, first);
    end = __reduce_max_sync(0xffffffffu, end);
    if (end == 0) first = 0;
    whole = __any_sync(0xffffffffu, whole);
    whole_causal = __any_sync(0xffffffffu, whole_causal);
    const size_t at = static_cast<size_t>(b) * m.nk + kt;
    uint32_t there[4] = {0u, 0u, 0u, 0u};
    add_span(there, 0, c1 - c0);
    uint32_t any[4], causal[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      any[w] = whole ? there[w] : 0u;
      causal[w] = whole_causal ? there[w] : 0u;
    }
    for (int t0 = first & ~31; t0 < end && !(whole && whole_causal); t0 += 32) {
      const int t = t0 + lane;
      const int4 r = t < m.nq ? qt[t] : make_int4(0, 0, 0, 0);
      bool rows = false;
      if (r.x < c1 && r.y > c0) {
        // positions of the tile's first and last row
        const int p0 = t * 128 + off, p1 = min(t * 128 + 127, Sq - 1) + off;
        const bool cut = r.w == 2 && p0 < c1 - 1;
        const int to = r.w == 1 ? min(r.y, p1 + 1) : r.y;  // under the rule
        if (r.z < 3) {
          uint32_t in[4] = {0u, 0u, 0u, 0u}, ruled[4] = {0u, 0u, 0u, 0u}, out[4] = {0u, 0u, 0u, 0u};
          add_span(in, r.x - c0, r.y - c0);
          if (!cut && to > r.x) add_span(ruled, r.x - c0, to - c0);
          if (r.z > 0) {
            const int4 gap = m.gaps[static_cast<size_t>(b) * m.nq + t];
            add_span(out, gap.x - c0, gap.y - c0);
            add_span(out, gap.z - c0, gap.w - c0);
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            any[w] |= in[w] & ~out[w];
            causal[w] |= ruled[w] & ~out[w];
          }
        }
        rows = r.z == 3 || (cut && p1 >= c0);
      }
      uint32_t look = __ballot_sync(0xffffffffu, rows);
      do {
        if (look) {
          const int i0 = (t0 + __ffs(look) - 1) * 128 + lane;
          look &= look - 1;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int i = i0 + 32 * k;
            if (i >= Sq) continue;
            const int2 s = m.rows[static_cast<size_t>(b) * Sq + i];
            add_span(any, s.x - c0, s.y - c0);
            const int h = min(s.y, i + off + 1);
            if (h > s.x) add_span(causal, s.x - c0, h - c0);
          }
        }
        whole = gather_bits(any, there);
        whole_causal = gather_bits(causal, there);
      } while (look && !(whole && whole_causal));
    }
    if (lane == 0) {
      const int full = c1 == c0 + 128;  // (keys that are not there are not seen)
      const_cast<int4*>(m.kt)[at] = make_int4(first, end, whole && full ? 0 : kUnseen, whole_causal && full ? 0 : kUnseen);
      const_cast<uint4*>(m.seen)[at] = make_uint4(any[0], any[1], any[2], any[3]);
      const_cast<uint4*>(m.seen_causal)[at] = make_uint4(causal[0], causal[1], causal[2], causal[3]);
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
                         m, Sq, Sk);
  const long long most = 1ll * B * std::max(m.nq, m.nk);
  if (e == cudaSuccess)
    e = launch_dependent(fa_plan_order_kernel, dim3(static_cast<unsigned int>((most + 7) / 8), 4),
                         dim3(256), 0, stream, m);
  return e;
}

}  // namespace fa
