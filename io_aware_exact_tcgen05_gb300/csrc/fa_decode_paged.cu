// fa_decode_paged.cu -- attention of the last Sq tokens of each request over a
// paged 8-bit KV cache, over every block or over a list of chosen blocks.
//
// The cache is read once (2 bytes per key, KV head and channel), so HBM bounds
// the kernel; the arithmetic only has to stay out of the way.  The query rows
// of a KV head (Hq / Hkv * Sq of them) are the narrow side of two
// mma.sync.m16n8k16 products in f16 with fp32 accumulation, up to 8 rows
//   S^T[16 keys x 8 rows] = K Q^T,   O^T[d x 8 rows] += V^T P^T
// and from 9 rows on
//   S[16 rows x 8 keys] = Q K^T,     O[16 rows x d] += P V
// e4m3 codes become f16 exactly (one conversion per pair).  The page's K scale
// multiplies the scores in fp32, its V scale the weights in fp32.
//
// f16 and its range: a query row is multiplied by the power of two that puts
// its largest element into [2^14, 2^15), which loses nothing above 2^-38 of it.
// Every row keeps two running maxima, both in log2 units: m over its scores x, against
// which the softmax's sum l is taken, and mv over x + log2(V scale), against which the
// weights of the values are stored, as 2^(x + log2(V scale) - mv + 9) in f16.  A maximum
// may lag by 6, so a stored weight is at most 2^15, keeps f16's 11 bits down to 2^-23 of
// the largest weight * V scale that the row has met, and is rounded by at most 2^-34 of
// that below.  With a maximum of its own per row, a loud page takes nothing from the
// others where the row gives it no weight or does not see it (against the largest V scale
// met so far, a page 2^30 louder, without weight, left the others 3 bits).  In the
// end O = acc * 2^(mv - m - 9) / l.  Sums, maxima and accumulators are fp32.
//
// Operands without shared memory: the contraction index of a product may be
// permuted freely, so a lane loads 16-byte pieces of whole rows and hands their
// bytes to the products in the order they lie.  For K (rows = keys), lane (g, t)
// (g = lane / 4, t = lane % 4) loads channels [16t, 16t + 16) of keys g and g + 8;
// for V it loads channels [16g, 16g + 16) of keys 2t, 2t+1, 2t+8 and 2t+9, and one
// byte permutation pairs two keys of a channel.  The S^T accumulator becomes the
// P^T operand by movmatrix; that of S is P's operand as it lies.
//
// Work: the 16-key blocks of all (request, KV head, row block) are laid end to
// end and every CTA takes an equal stretch (the lengths are read on the device:
// the call reads nothing back and a captured graph follows new lengths).  Inside a
// stretch the four warps take blocks in turn, each with a state of its own; the
// states of one (request, KV head, row block) are merged in the CTA.  One that lies
// inside a single CTA's stretch is finished there; the others leave partial states
// that fa_decode_paged_merge joins in a fixed order.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <math.h>

#include "fa_internal.h"
#include "fa_kv.h"
#include "fa_kv_device.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kBlockKeys = 16;
constexpr int kSms = 152;
constexpr int kMinShare = 8;        // places in the line a CTA takes at least
constexpr int kSegmentCost = 24;    // places a segment's fixed cost takes in the line
constexpr float kLag = 6.f;         // how far (log2) a weight may exceed a running maximum
constexpr float kWeightLog = 9.f;   // log2 of the stored weight of a key at the maximum

// Row tiles of 8 a CTA serves, and CTAs per SM (by registers).  Up to 8 rows the
// narrow kernel; more go through the wide one, 32 at a time.
template <int NT> struct Plan;
template <> struct Plan<1> { static constexpr int kCtasPerSm = 4; };
template <> struct Plan<2> { static constexpr int kCtasPerSm = 5; };
template <> struct Plan<4> { static constexpr int kCtasPerSm = 3; };

int row_tiles(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }
int grid_ctas(int nt) {
  return kSms * (nt == 1 ? Plan<1>::kCtasPerSm : nt == 2 ? Plan<2>::kCtasPerSm
                                                         : Plan<4>::kCtasPerSm);
}

// Running maximum of a row that has seen no key yet: finite, so that differences
// with it stay defined, and below every score.
constexpr float kNoMax = -3.0e38f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// log2 of a V scale; 0 gives -inf: values without weight.  (Taken where a scale is used: where
// it is loaded, the logarithm waits for it, and 9 to 16 rows took 10% longer.)
__device__ __forceinline__ float log2_scale(float s) { return __log2f(s); }

// How far above m a score may lie before the maxima have to move: by kLag, and so that its
// stored weight, 2^(score + up), stays below 2^(kWeightLog + kLag).
__device__ __forceinline__ float most_above(float m, float up) {
  return fminf(kLag, kWeightLog + kLag - up - m);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Where kEarly, the value is read in L2: the merge asks before its own wait, when only
// L2 is sure to hold what kernels before the partial one wrote.
template <bool kEarly>
__device__ __forceinline__ int read_count(const int32_t* p) {
  return kEarly ? __ldcg(p) : *p;
}

template <bool kEarly = false>
__device__ __forceinline__ int request_len(const PagedDecodeParams& p, int b) {
  return static_cast<int>(min(static_cast<long long>(max(read_count<kEarly>(p.seqlens + b), 0)),
                              static_cast<long long>(p.max_blocks) * p.s.page_size));
}

// 16-key blocks of a (request, KV head).
template <bool kEarly = false>
__device__ __forceinline__ int item_blocks(const PagedDecodeParams& p, int item) {
  if (p.sel) return min(max(read_count<kEarly>(p.n_sel + item), 0), p.max_sel) << p.block_shift;
  return (request_len<kEarly>(p, item / p.s.Hkv) + kBlockKeys - 1) / kBlockKeys;
}

// Places of a (request, KV head) and row block in the line: its blocks behind
// kSegmentCost places without work, for what beginning and ending a segment costs (8000 to
// 10000 clocks; 32 rows of 24 ragged requests took 62 us without them where 16 took 52).  Both
// kernels use one value: 8, 12, 16, 20, 24, 32 take 24.1, 23.7, 23.6, 23.6, 23.9, 24.4 us in geometric
// mean over 19 cases of up to 32 rows, and 12, 16, 20, 24 take 9.48, 9.42, 9.50, 9.42 us over 33
// drawn ones, mostly narrow.  (A multiple of the smallest share keeps short requests on whole shares:
// 777 keys take 6.1 us with 8, 16, 24, and 6.6 to 6.8 with 12 and 20.)
__device__ __forceinline__ long long unit_places(int n_kb) {
  return n_kb > 0 ? n_kb + kSegmentCost : 0;
}

// Where the units of the items lie in the one long line: thread t of the CTA
// sums items [t * per, (t + 1) * per), prefix[t] is the start of its first one.
struct Line {
  long long prefix[kThreads + 1];
  long long warp_sum[kWarps];
};

// Returns the start of the calling thread's items.
__device__ __forceinline__ long long make_line(const PagedDecodeParams& p, int row_blocks,
                                               Line& s) {
  const int items = p.B * p.s.Hkv;
  const int per = (items + kThreads - 1) / kThreads;
  const int lo = min(static_cast<int>(threadIdx.x) * per, items), hi = min(lo + per, items);
  long long own = 0;
  for (int i = lo; i < hi; ++i) own += unit_places(item_blocks(p, i));
  own *= row_blocks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long v = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) s.warp_sum[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) v += s.warp_sum[w];
  s.prefix[threadIdx.x + 1] = v;
  if (threadIdx.x == 0) s.prefix[0] = 0;
  __syncthreads();
  return v - own;
}

// Quotient of non-negative values; nearly always both fit 32 bits, where a
// division takes a quarter of the time.
__device__ __forceinline__ long long quotient(long long a, int b) {
  return a <= 0x7fffffffll ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b))
                           : a / b;
}

// Places per CTA.  At least 8, so that a short request is not cut into pieces that
// cost more to join than to read, but no more than an item has on average, so that
// CTAs do not queue up tiny ones (208 items of one block: 54 us in eights, 22 us one by one).
__device__ __forceinline__ long long share_of(long long total, int items, int ctas) {
  const long long even = quotient(total + ctas - 1, ctas);
  const long long least = min(static_cast<long long>(kMinShare), max(quotient(total, items), 1ll));
  if (even <= 16) return max(even, least);
  return (even + 3) & ~3ll;  // a step of the wide kernel is four blocks
}

// The CTA whose stretch holds a place of the line.
__device__ __forceinline__ int cta_of(long long place, long long share) {
  return static_cast<int>(share <= 0x7fffffffll ? quotient(place, static_cast<int>(share))
                                                : place / share);
}

// Sum over the warp of values in [0, 2^47).
__device__ __forceinline__ long long warp_sum(long long v) {
  const uint32_t lo = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v) & 0xfffffu);
  const uint32_t hi = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> 20));
  return (static_cast<long long>(hi) << 20) + lo;
}

// Where an item begins in the line, and the line's length.
struct Place {
  long long before[kWarps], all[kWarps];  // of one row block, as each warp has summed them

  // The CTA's threads, before the caller's wait: lengths are read in L2.
  __device__ __forceinline__ void sum(const PagedDecodeParams& p, int item) {
    long long total = 0, front = 0;
    if (p.sel) {
      const int items = p.B * p.s.Hkv;
      for (int i = threadIdx.x; i < items; i += kThreads) {
        const long long n = unit_places(item_blocks<true>(p, i));
        total += n;
        front += i < item ? n : 0;
      }
    } else {  // the heads of a request are alike
      const int request = item / p.s.Hkv, heads = item - request * p.s.Hkv;
      for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const long long n = unit_places((request_len<true>(p, b) + kBlockKeys - 1) / kBlockKeys);
        total += n * p.s.Hkv;
        front += n * (b < request ? p.s.Hkv : b == request ? heads : 0);
      }
    }
    total = warp_sum(total);
    front = warp_sum(front);
    if ((threadIdx.x & 31) == 0) {
      all[threadIdx.x >> 5] = total;
      before[threadIdx.x >> 5] = front;
    }
  }
  static __device__ __forceinline__ long long of(const long long (&v)[kWarps]) {
    return (v[0] + v[1]) + (v[2] + v[3]);
  }
};

// A CTA walks its stretch of the line segment by segment: blocks [kb0, kb0 + n_seg)
// of one item (request, KV head) and row block.  One thread keeps the place, in
// shared memory, so that it takes no registers in the main loop.
struct Segment {
  long long at, end, in_item;  // place in the line, the stretch's end, place in the item
  size_t qrow0;
  const int32_t* table;
  int item, hk, len, n_kb, kb0, n_seg, row0, n_rows;
  bool live;

  // Called by every thread with the start of its items; the one whose items hold
  // the stretch's start fills the segment in.
  __device__ __forceinline__ void begin(const PagedDecodeParams& p, int row_blocks, int tile_rows,
                                        const Line& line, long long start) {
    const int items = p.B * p.s.Hkv;
    const long long total = line.prefix[kThreads];
    const long long share = share_of(total, items, gridDim.x);
    const long long here = share * blockIdx.x;
    if (here >= total) {
      if (threadIdx.x == 0) live = false;
    } else if (start <= here && here < line.prefix[threadIdx.x + 1]) {
      live = true;
      at = here;
      end = min(here + share, total);
      item = threadIdx.x * ((items + kThreads - 1) / kThreads);
      in_item = here - start;
      find(p, row_blocks, tile_rows);
    }
  }
  __device__ __forceinline__ void next(const PagedDecodeParams& p, int row_blocks, int tile_rows,
                                       const Line& line) {
    at += n_seg;
    in_item += n_seg;
    live = at < end;
    if (!live) return;
    if (in_item >= unit_places(n_kb) * row_blocks) {
      in_item -= unit_places(n_kb) * row_blocks;
      // Empty items may follow, in a padded batch thousands: on to the thread whose items hold
      // the place.  (One after another, 32000 took a thread 17 ms.)
      if (item_blocks(p, ++item) == 0) {
        int t = 0;
        for (int z = kThreads; z - t > 1;) {  // the last one with prefix <= at
          const int mid = (t + z) >> 1;
          if (line.prefix[mid] <= at) t = mid; else z = mid;
        }
        const int owned = t * ((p.B * p.s.Hkv + kThreads - 1) / kThreads);
        if (owned > item) {
          item = owned;
          in_item = at - line.prefix[t];
        }
      }
    }
    find(p, row_blocks, tile_rows);
  }
  // The segment at (item, in_item), which may lie behind the item's end or in
  // front of a unit's blocks.
  __device__ __forceinline__ void find(const PagedDecodeParams& p, int row_blocks, int tile_rows) {
    n_kb = item_blocks(p, item);
    while (in_item >= unit_places(n_kb) * row_blocks) {
      in_item -= unit_places(n_kb) * row_blocks;
      n_kb = item_blocks(p, ++item);
    }
    const int places = n_kb + kSegmentCost;
    const int rb = static_cast<int>(quotient(in_item, places));
    kb0 = static_cast<int>(in_item - static_cast<long long>(rb) * places) - kSegmentCost;
    if (kb0 < 0) {
      at -= kb0;
      in_item -= kb0;
      kb0 = 0;
      if (at >= end) {
        live = false;
        return;
      }
    }
    n_seg = static_cast<int>(min(static_cast<long long>(n_kb - kb0), end - at));
    const int b = item / p.s.Hkv;
    hk = item - b * p.s.Hkv;
    len = request_len(p, b);
    row0 = rb * tile_rows;
    n_rows = min(tile_rows, p.rows - row0);
    table = p.block_table + static_cast<size_t>(b) * p.max_blocks;
    qrow0 = static_cast<size_t>(item) * p.rows + row0;
  }
};

template <int D>
struct NarrowSmem {
  Line line;
  Segment seg;
  float m[kWarps][8];
  float l[kWarps][8];
  float mv[kWarps][8];
  alignas(16) float o[kWarps][8][D + 4];
};

// What a lane looks up for one of its warp's coming blocks (block i of the
// segment; a hidden one has scales of 0 and the offset kHidden).
struct BlockInfo {
  long long offset;  // bytes from the start of a cache tensor to the block's first key
  int pos;           // position of the first key; INT_MAX: the block is hidden
  float ks, vs;
};

template <int kHidden>
__device__ __forceinline__ BlockInfo look_up(const PagedDecodeParams& p, const Segment& sg, int i) {
  const int ps = p.s.page_size;
  BlockInfo r = {kHidden, 0x7fffffff, 0.f, 0.f};
  if (i >= sg.n_seg) return r;
  const int idx = (sg.kb0 + i) >> p.block_shift, sub = (sg.kb0 + i) & ((1 << p.block_shift) - 1);
  const int blk = p.sel ? p.sel[static_cast<size_t>(sg.item) * p.max_sel + idx] : idx;
  if (blk >= 0 && static_cast<long long>(blk) * ps + sub * kBlockKeys < sg.len) {
    const int page = sg.table[blk];
    if (page >= 0 && page < p.s.num_pages) {
      const size_t tile = static_cast<size_t>(page) * p.s.Hkv + sg.hk;
      r.offset = (static_cast<long long>(tile) * ps + sub * kBlockKeys) * p.s.d;
      r.pos = blk * ps + sub * kBlockKeys;
      r.ks = p.k_scale[tile];
      r.vs = p.v_scale[tile];
    }
  }
  return r;
}

// Bytes of w that are NaN codes, as a byte mask.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

// 16 bytes of a query row (8 channels) as f16 times `up`.
__device__ __forceinline__ void scale_to_f16(const uint4& w, float up, uint32_t (&h)[4]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    h[e] = pack_f16x2(__uint_as_float(x[e] << 16) * up, __uint_as_float(x[e] & 0xffff0000u) * up);
}

// The B operand of row tile row: lane (g, t) loads its channels of row g, scales
// them by a power of two and hands k-step ks to put(ks, {b0, b1}).  Returns the
// factor that turns (product * K scale) into a score in log2 units, for row g.
template <int D, typename Put>
__device__ __forceinline__ float load_q(const PagedDecodeParams& p, size_t row, bool live, int t,
                                        Put put) {
  constexpr int N = D / 32;
  uint4 w[N];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (live)
      w[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + row * D +
                                             (i / 2) * 64 + t * 16 + (i % 2) * 8);
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu),
                                 __vmaxu2(w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu)));
  }
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const int ex = max(static_cast<int>(max(top & 0xffffu, top >> 16) >> 7) - 127, -100);
  const float up = pow2i(14 - ex);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t h[4];
    scale_to_f16(w[i], up, h);
    // k-steps (i / 2) * 4 + (i % 2) * 2 + {0, 1}: four channels of the lane each
    const int ks = (i / 2) * 4 + (i % 2) * 2;
    put(ks, make_uint2(h[0], h[1]));
    put(ks + 1, make_uint2(h[2], h[3]));
  }
  return p.scale_log2 * pow2i(ex - 14);
}

// A partial state of a row: its two maxima and its sum; the accumulator beside it counts in
// units of 2^(mv - 9).
using RowState = float4;  // m, l, mv, unused
__device__ __forceinline__ RowState row_state(float m, float l, float mv) {
  return make_float4(m, l, mv, 0.f);
}

// 2^(mv - m - 9) of a finished row.  It multiplies acc / l: with scales of 2^-100 it divided by a
// large l would be subnormal.
__device__ __forceinline__ float value_unit(float m, float mv) {
  return ex2_approx(mv - m - kWeightLog);
}

// Writes one finished output vector (four channels) or partial state.
template <int D>
__device__ __forceinline__ void emit(const PagedDecodeParams& p, const Segment& sg, int tile_rows,
                                     int row, int c, float M, float L, float MV, float4 o,
                                     float* part_o, RowState* part_ml) {
  if (sg.n_seg == sg.n_kb) {
    const bool empty = L == 0.f;
    const float inv = empty ? 0.f : 1.f / L;
    const float unit = value_unit(M, MV);
    uint2 w;
    w.x = pack_bf16x2(o.x * inv * unit, o.y * inv * unit);
    w.y = pack_bf16x2(o.z * inv * unit, o.w * inv * unit);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + (sg.qrow0 + row) * D + c) = w;
    if (p.lse && c == 0)
      p.lse[sg.qrow0 + row] = empty ? neg_inf() : (M + __log2f(L)) * 0.69314718055994530942f;
  } else {
    // a CTA's first segment may begin inside an item, its last may end inside one
    const size_t at = (2 * static_cast<size_t>(blockIdx.x) + (sg.kb0 == 0 ? 1 : 0)) * tile_rows + row;
    *reinterpret_cast<float4*>(part_o + at * D + c) = o;
    if (c == 0) part_ml[at] = row_state(M, L, MV);
  }
}

// Up to 8 query rows: the warps take blocks in turn, each with its own state.
template <int D>
__global__ void __launch_bounds__(kThreads, Plan<1>::kCtasPerSm)
    fa_decode_paged_narrow(const PagedDecodeParams p, int row_blocks, float* part_o,
                           RowState* part_ml) {
  constexpr int KC = D / 64;       // 16-byte pieces of a key row per lane
  constexpr int KS = D / 16;       // k-steps of S
  constexpr int MT = D / 16;       // m-tiles of O^T
  constexpr int VW = D / 32;       // 32-bit words of a value row per lane
  extern __shared__ __align__(16) unsigned char smem_raw[];
  NarrowSmem<D>& s = *reinterpret_cast<NarrowSmem<D>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;

  // First the wait, then the signal: once the merge may launch, what this call
  // reads (lengths, lists) is complete, so the merge may read them before its own wait.
  griddep_wait();
  griddep_launch_dependents();
  const long long start = make_line(p, row_blocks, s.line);
  const Segment& sg = s.seg;
  s.seg.begin(p, row_blocks, 8, s.line, start);
  __syncthreads();
  while (sg.live) {
    uint4 kr[2][KC];
    uint32_t vr[4][VW];
    auto load_k = [&](long long off) {
      const uint8_t* base = static_cast<const uint8_t*>(p.k_cache) + off + g * D + t * 16;
#pragma unroll
      for (int i = 0; i < KC; ++i) {
        kr[0][i] = ld_stream16(base + i * 64);
        kr[1][i] = ld_stream16(base + 8 * D + i * 64);
      }
    };
    auto load_v = [&](long long off) {
      const uint8_t* base = static_cast<const uint8_t*>(p.v_cache) + off + 2 * t * D + g * (D / 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* row = base + ((i & 1) + (i >> 1) * 8) * D;
        if constexpr (D == 128) {
          const uint4 w = ld_stream16(row);
          vr[i][0] = w.x, vr[i][1] = w.y, vr[i][2] = w.z, vr[i][3] = w.w;
        } else {
          const uint2 w = ld_stream8(row);
          vr[i][0] = w.x, vr[i][1] = w.y;
        }
      }
    };
    const int mine = (sg.n_seg - warp + kWarps - 1) / kWarps;  // blocks warp + i * kWarps
    BlockInfo info = look_up<0>(p, sg, warp + lane * kWarps);
    {  // the first block is on its way while the queries are prepared
      const long long off = __shfl_sync(0xffffffffu, info.offset, 0);
      if (mine > 0) {
        load_k(off);
        load_v(off);
      }
    }

    uint2 qf[KS];
    float c_row[2];
    {
      const float c = load_q<D>(p, sg.qrow0 + g, g < sg.n_rows, t,
                                [&](int ks, uint2 v) { qf[ks] = v; });
      c_row[0] = __shfl_sync(0xffffffffu, c, 8 * t);  // rows 2t and 2t + 1
      c_row[1] = __shfl_sync(0xffffffffu, c, 8 * t + 4);
    }
    float m[2] = {kNoMax, kNoMax}, mv[2] = {kNoMax, kNoMax}, l[2] = {0.f, 0.f}, acc[MT][4];
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;

    for (int i = 0; i < mine; ++i) {
      const int src = i & 31;
      if (src == 0 && i > 0) {  // the next 32 blocks of this warp, one per lane
        info = look_up<0>(p, sg, warp + (i + lane) * kWarps);
        const long long off = __shfl_sync(0xffffffffu, info.offset, 0);
        load_k(off);
        load_v(off);
      }
      const int pos = __shfl_sync(0xffffffffu, info.pos, src);
      const float ks = __shfl_sync(0xffffffffu, info.ks, src);
      const float vl = log2_scale(__shfl_sync(0xffffffffu, info.vs, src));
      const bool more = i + 1 < mine && src != 31;
      const long long next = __shfl_sync(0xffffffffu, info.offset, (src + 1) & 31);

      // ---- S^T = K Q^T: {key g, row 2t}, {key g, row 2t+1}, {key g+8, ...} x 2 ----
      float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const uint32_t wa[4] = {kr[0][c].x, kr[0][c].y, kr[0][c].z, kr[0][c].w};
        const uint32_t wb[4] = {kr[1][c].x, kr[1][c].y, kr[1][c].z, kr[1][c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint2 q = qf[c * 4 + e];
          mma_f16(x, e4m3x2_to_f16x2(wa[e]), e4m3x2_to_f16x2(wb[e]),
                  e4m3x2_hi_to_f16x2(wa[e]), e4m3x2_hi_to_f16x2(wb[e]), q.x, q.y);
        }
      }
      if (more) load_k(next);

      // ---- weights against the running maxima ----
      const bool edge = static_cast<long long>(pos) + kBlockKeys - 1 > sg.len - p.Sq;
      float f[2] = {ks * c_row[0], ks * c_row[1]};
      if (edge) {  // scores that are not seen become -inf
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[e & 1] = fmaxf(f[e & 1], 1.1754944e-38f);  // -inf * 0 would be NaN
          const long long key = static_cast<long long>(pos) + g + (e >> 1) * 8;
          if (key > sg.len - p.Sq + (sg.row0 + 2 * t + (e & 1)) % p.Sq) x[e] = neg_inf();
        }
      }
      float arg[4];
      bool over = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        arg[r] = fmaf(x[r], f[r], -m[r]);
        arg[2 + r] = fmaf(x[2 + r], f[r], -m[r]);
        over |= fmaxf(arg[r], arg[2 + r]) > most_above(m[r], vl - mv[r] + kWeightLog);
      }
      if (__any_sync(0xffffffffu, over)) {
        // exact maxima of the block's rows; the state moves to them
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float mx = fmaxf(x[r] * f[r], x[2 + r] * f[r]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const float mxv = fmaxf(mv[r], mx + vl);
          mx = fmaxf(m[r], mx);
          l[r] *= ex2_approx(m[r] - mx);
          const float a = ex2_approx(mv[r] - mxv);
          m[r] = mx;
          mv[r] = mxv;
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            acc[j][r] *= a;
            acc[j][2 + r] *= a;
          }
          arg[r] = fmaf(x[r], f[r], -mx);
          arg[2 + r] = fmaf(x[2 + r], f[r], -mx);
        }
      }
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        l[e & 1] += ex2_approx(arg[e]);
        w[e] = ex2_approx(fmaf(x[e], f[e & 1], vl - mv[e & 1] + kWeightLog));
      }
      const uint32_t pb0 = transpose8x8(pack_f16x2(w[0], w[1]));
      const uint32_t pb1 = transpose8x8(pack_f16x2(w[2], w[3]));

      // ---- O^T += V^T P^T ----
      if (edge) {
        bool nan = false;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool dead = static_cast<long long>(pos) + 2 * t + (r & 1) + (r >> 1) * 8 >= sg.len;
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            if (dead) vr[r][e] = 0u;  // what lies behind the last key may be anything
            nan |= nan_codes(vr[r][e]) != 0;
          }
        }
        if (p.Sq > 1 && __any_sync(0xffffffffu, nan)) {
          // A NaN value must reach the rows that see its key and no others (0 * NaN is
          // NaN): the product of "code is NaN" and "row sees key" says where it goes,
          // and the code becomes 0 for the product with the weights.
          const int last = sg.len - p.Sq + (sg.row0 + g) % p.Sq - pos - 2 * t;
          const uint32_t see0 = (last >= 0 ? 0x3c00u : 0u) | (last >= 1 ? 0x3c000000u : 0u);
          const uint32_t see1 = (last >= 8 ? 0x3c00u : 0u) | (last >= 9 ? 0x3c000000u : 0u);
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
            uint32_t n[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) n[r] = nan_codes(vr[r][j >> 1]) & 0x38383838u;  // 1.0
            const uint32_t lo = __byte_perm(n[0], n[1], sel), hi = __byte_perm(n[2], n[3], sel);
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(c, e4m3x2_to_f16x2(lo), e4m3x2_hi_to_f16x2(lo), e4m3x2_to_f16x2(hi),
                    e4m3x2_hi_to_f16x2(hi), see0, see1);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (c[e] > 0.f) acc[j][e] = __int_as_float(0x7fffffff);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < VW; ++e) vr[r][e] &= ~nan_codes(vr[r][e]);
        }
      }
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
        const uint32_t lo = __byte_perm(vr[0][j >> 1], vr[1][j >> 1], sel);
        const uint32_t hi = __byte_perm(vr[2][j >> 1], vr[3][j >> 1], sel);
        mma_f16(acc[j], e4m3x2_to_f16x2(lo), e4m3x2_hi_to_f16x2(lo), e4m3x2_to_f16x2(hi),
                e4m3x2_hi_to_f16x2(hi), pb0, pb1);
      }
      if (more) load_v(next);
    }

    // ---- merge the warps' states ----
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float sum = l[r];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const int row = 2 * t + r;
      if (g == 0) {
        s.m[warp][row] = m[r];
        s.l[warp][row] = sum;
        s.mv[warp][row] = mv[r];
      }
#pragma unroll
      for (int j = 0; j < MT; ++j)
        *reinterpret_cast<float2*>(&s.o[warp][row][g * (D / 8) + 2 * j]) =
            make_float2(acc[j][r], acc[j][2 + r]);
    }
    __syncthreads();
    for (int idx = tid; idx < sg.n_rows * (D / 4); idx += kThreads) {
      const int row = idx / (D / 4), c = (idx % (D / 4)) * 4;
      float M = kNoMax, MV = kNoMax;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        M = fmaxf(M, s.m[w][row]);
        MV = fmaxf(MV, s.mv[w][row]);
      }
      float L = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float wt = ex2_approx(s.mv[w][row] - MV);
        const float4 v = *reinterpret_cast<const float4*>(&s.o[w][row][c]);
        L = fmaf(ex2_approx(s.m[w][row] - M), s.l[w][row], L);
        o.x = fmaf(wt, v.x, o.x);
        o.y = fmaf(wt, v.y, o.y);
        o.z = fmaf(wt, v.z, o.z);
        o.w = fmaf(wt, v.w, o.w);
      }
      emit<D>(p, sg, 8, row, c, M, L, MV, o, part_o, part_ml);
    }
    __syncthreads();
    if (tid == 0) s.seg.next(p, row_blocks, 8, s.line);
    __syncthreads();
  }
}

__device__ __forceinline__ void cp_async16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Four channels of keys 2t, 2t + 1, 2t + 8 and 2t + 9 as B operands, channel j in b[.][j].
__device__ __forceinline__ void pair_up(const uint32_t (&v)[4], uint32_t (&b)[2][4]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t lo = __byte_perm(v[2 * k], v[2 * k + 1], 0x5140);
    const uint32_t hi = __byte_perm(v[2 * k], v[2 * k + 1], 0x7362);
    b[k][0] = e4m3x2_to_f16x2(lo), b[k][1] = e4m3x2_hi_to_f16x2(lo);
    b[k][2] = e4m3x2_to_f16x2(hi), b[k][3] = e4m3x2_hi_to_f16x2(hi);
  }
}

// 9 to 32 query rows: the four warps work on the same four blocks (64 keys).  Each
// computes the scores of one block for all rows; the weights go through shared
// memory as A operands, and each warp adds its 32 channels of O (at d = 64 two
// warps share 32 channels and take two of the blocks each).  So the accumulators
// of a warp are 32 rows x 32 channels, a quarter of what a warp on its own would
// hold.
// Keys go to registers; values go through shared memory, copied a step ahead, one block
// per warp: loaded from global memory each warp would take 4 bytes per lane and row (64
// keys x 32 channels), and those 16 loads cost 6 us of 52.  Hidden blocks are not loaded: all
// CTAs' reads of one place in their stead cost 1 us of 12 for 200 short items.
// Latency bounds it: 11 warps per SM are there, tensor pipe 38% busy, shared memory 49%, issue
// 40%; the waits are for products and conversions (26%), shared memory (16%), global memory
// (10%).  41.6 us for 24 requests of 500 to 9000 keys, 32 rows, 4 KV heads (3.0 TB/s), of which 36
// remain without loading keys and values.  (With the keys as M side, as the narrow kernel has it,
// 45 us where this form took 43; a warp with all 32 rows to itself 68 us where this kernel's
// first form took 66.)  With a lag of 4 or 2 in place of 6 the maxima move on more steps: 42.7 and
// 45.3 us, 2% and 5% in geometric mean over 19 cases.
// The running maxima are the CTA's; the vote on moving them is the barrier that
// hands the weights over.  A segment's first step moves them without a vote.
template <int D, int NT>
struct WideSmem {
  Line line;
  Segment seg;
  float c_row[8 * NT];
  float m[8 * NT];
  float mv[8 * NT];
  float l[kWarps][8 * NT];
  float mx[kWarps][8 * NT];
  float vl[kWarps];
  alignas(16) uint32_t q[NT / 2 * (D / 16)][32][4];    // A operands of the query rows
  alignas(16) uint4 w[2][kWarps][NT / 2][32];          // P of the four blocks, double buffered
  union {
    alignas(16) uint8_t v[2][kWarps][kBlockKeys * D];  // values of the steps to come
    alignas(16) float o[128 / D][8 * NT][D + 4];       // the segment's result
  };
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Plan<NT>::kCtasPerSm)
    fa_decode_paged_wide(const PagedDecodeParams p, int row_blocks, float* part_o,
                         RowState* part_ml) {
  constexpr int KC = D / 64;           // 16-byte pieces of a key row per lane
  constexpr int KS = D / 16;           // k-steps of S
  constexpr int DW = D / 32;           // warps side by side over the channels
  constexpr int VB = DW;               // blocks whose values a warp multiplies
  constexpr int R = 8 * NT;
  constexpr int MT = NT / 2;           // row tiles of 16
  extern __shared__ __align__(16) unsigned char smem_raw[];
  WideSmem<D, NT>& s = *reinterpret_cast<WideSmem<D, NT>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int dw = warp % DW, vb0 = (warp / DW) * VB;  // channels [32 dw, ..), blocks [vb0, ..)
  // A block's values in shared memory: 16-byte pieces, moved within their row (and at
  // d = 64 rows 1 and 2 of four changed over) so that the four rows a warp reads at once
  // lie in different banks.
  constexpr int V_ODD = D == 128 ? D : 2 * D;           // from row 2t to row 2t + 1
  const int v_row = lane / (D / 16), v_piece = lane % (D / 16);  // row of 512 / D at a time
  int v_read;
  if constexpr (D == 128)
    v_read = 2 * t * D + ((dw * 2 + (g >> 2)) ^ 2 * t) * 16 + (g & 3) * 4;
  else
    v_read = ((t >> 1) * 4 + (t & 1)) * D + ((dw * 2 + (g >> 2)) ^ (t >> 1) * 2) * 16 + (g & 3) * 4;

  // First the wait, then the signal: once the merge may launch, what this call
  // reads (lengths, lists) is complete, so the merge may read them before its own wait.
  griddep_wait();
  griddep_launch_dependents();
  const long long start = make_line(p, row_blocks, s.line);
  const Segment& sg = s.seg;
  s.seg.begin(p, row_blocks, R, s.line, start);
  __syncthreads();
  while (sg.live) {
    const int steps = (sg.n_seg + kWarps - 1) / kWarps;
    uint4 kr[2][KC] = {};
    auto load_k = [&](long long off) {
      if (off < 0) return;
      const uint8_t* base = static_cast<const uint8_t*>(p.k_cache) + off + g * D + t * 16;
#pragma unroll
      for (int i = 0; i < KC; ++i) {
        kr[0][i] = ld_stream16(base + i * 64);
        kr[1][i] = ld_stream16(base + 8 * D + i * 64);
      }
    };
    // the values of this warp's block of a step, 512 bytes at a time
    auto copy_v = [&](int step, long long off) {
      if (off < 0) return;
      const uint8_t* from = static_cast<const uint8_t*>(p.v_cache) + off + lane * 16;
      uint8_t* to = s.v[step & 1][warp];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int r = i * (512 / D) + v_row;
        const int at = D == 128 ? r * D + (v_piece ^ ((r >> 1) & 3) * 2) * 16
                                : ((r & 12) | (r & 1) << 1 | (r >> 1 & 1)) * D +
                                      (v_piece ^ ((r >> 2) & 1) * 2) * 16;
        cp_async16(to + at, from + i * 512);
      }
    };
    // lane j of every warp looks block j of the coming 32 up, and of the 32 after them
    BlockInfo info = look_up<-1>(p, sg, lane), ahead = look_up<-1>(p, sg, 32 + lane);
    // blocks that some row does not see whole
    auto edges = [&] {
      return __ballot_sync(0xffffffffu, static_cast<long long>(info.pos) + kBlockKeys - 1 > sg.len - p.Sq);
    };
    uint32_t edge = edges();
    {
      const long long off = __shfl_sync(0xffffffffu, info.offset, warp);
      load_k(off);
      copy_v(0, off);
      cp_async_commit();
    }

    for (int nt = warp; nt < NT; nt += kWarps) {
      const int r = nt * 8 + g;
      const float c = load_q<D>(p, sg.qrow0 + r, r < sg.n_rows, t, [&](int ks, uint2 v) {
        s.q[nt / 2 * KS + ks][lane][nt & 1] = v.x;
        s.q[nt / 2 * KS + ks][lane][2 + (nt & 1)] = v.y;
      });
      if (t == 0) s.c_row[r] = c;
    }
    __syncthreads();
    float c_row[MT][2], m[MT][2], mv[MT][2], l[MT][2], acc[MT][4][4];  // rows g and g + 8 of a tile
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        c_row[mt][r] = s.c_row[mt * 16 + r * 8 + g];
        m[mt][r] = kNoMax;
        mv[mt][r] = kNoMax;
        l[mt][r] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[mt][j][e] = 0.f;
    }

    for (int i = 0; i < steps; ++i) {
      const int src = (i & 7) * kWarps;  // this step's blocks are lanes src .. src + 3
      if (src == 0 && i > 0) {
        info = ahead;
        ahead = look_up<-1>(p, sg, (i / 8 + 1) * 32 + lane);
        edge = edges();
      }
      const float ks = __shfl_sync(0xffffffffu, info.ks, src + warp);
      const float vl = log2_scale(__shfl_sync(0xffffffffu, info.vs, src + warp));
      const long long next = __shfl_sync(0xffffffffu, (i & 7) == 7 ? ahead.offset : info.offset,
                                         (src + kWarps + warp) & 31);

      // ---- S = Q K^T of this warp's block: {row g, key 8u + 2t}, {row g, key + 1}, {row g + 8, ..} x 2
      float x[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[mt][0][e] = x[mt][1][e] = 0.f;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const uint32_t wa[4] = {kr[0][c].x, kr[0][c].y, kr[0][c].z, kr[0][c].w};
        const uint32_t wb[4] = {kr[1][c].x, kr[1][c].y, kr[1][c].z, kr[1][c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t a0 = e4m3x2_to_f16x2(wa[e]), a1 = e4m3x2_hi_to_f16x2(wa[e]);
          const uint32_t b0 = e4m3x2_to_f16x2(wb[e]), b1 = e4m3x2_hi_to_f16x2(wb[e]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint4 q = *reinterpret_cast<const uint4*>(s.q[mt * KS + c * 4 + e][lane]);
            mma_f16(x[mt][0], q.x, q.y, q.z, q.w, a0, a1);
            mma_f16(x[mt][1], q.x, q.y, q.z, q.w, b0, b1);
          }
        }
      }
      load_k(next);

      // ---- weights against the running maxima ----
      float f[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        f[mt][0] = ks * c_row[mt][0];
        f[mt][1] = ks * c_row[mt][1];
      }
      if (edge >> (src + warp) & 1u) {  // as in the narrow kernel
        const int pos = __shfl_sync(0xffffffffu, info.pos, src + warp);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            f[mt][r] = fmaxf(f[mt][r], 1.1754944e-38f);
            const int last = sg.len - p.Sq + (sg.row0 + mt * 16 + r * 8 + g) % p.Sq;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const long long key = static_cast<long long>(pos) + 2 * t + (e >> 1) * 8 + (e & 1);
              if (key > last) x[mt][e >> 1][2 * r + (e & 1)] = neg_inf();
            }
          }
      }
      float ws[MT][2];
      auto put_weights = [&] {
        bool over = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t a[2][2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float up = vl - mv[mt][r] + kWeightLog, most = most_above(m[mt][r], up);
            float w[4], wv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float xe = x[mt][e >> 1][2 * r + (e & 1)];
              const float arg = fmaf(xe, f[mt][r], -m[mt][r]);
              over |= arg > most;
              w[e] = ex2_approx(arg);
              wv[e] = ex2_approx(fmaf(xe, f[mt][r], up));
            }
            a[0][r] = pack_f16x2(wv[0], wv[1]);
            a[1][r] = pack_f16x2(wv[2], wv[3]);
            ws[mt][r] = (w[0] + w[1]) + (w[2] + w[3]);
          }
          s.w[i & 1][warp][mt][lane] = make_uint4(a[0][0], a[0][1], a[1][0], a[1][1]);
        }
        return over;
      };
      // A segment's first step moves the maxima without a vote.  In front of the barrier that
      // hands the weights over, a thread's part of the step's values has arrived.
      bool move = i == 0;
      if (!move) {
        move = put_weights();
        cp_async_wait();
        move = __syncthreads_or(move);
      }
      if (move) {
        // exact maxima of the four blocks' rows; the CTA's state moves to them
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float mx = fmaxf(fmaxf(x[mt][0][2 * r] * f[mt][r], x[mt][0][2 * r + 1] * f[mt][r]),
                             fmaxf(x[mt][1][2 * r] * f[mt][r], x[mt][1][2 * r + 1] * f[mt][r]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            if (t == 0) s.mx[warp][mt * 16 + r * 8 + g] = mx;
          }
        if (lane == 0) s.vl[warp] = vl;
        __syncthreads();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float m_new = m[mt][r], mv_new = mv[mt][r];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              const float mx = s.mx[w][mt * 16 + r * 8 + g];
              m_new = fmaxf(m_new, mx);
              mv_new = fmaxf(mv_new, mx + s.vl[w]);
            }
            l[mt][r] *= ex2_approx(m[mt][r] - m_new);
            const float a = ex2_approx(mv[mt][r] - mv_new);
            m[mt][r] = m_new;
            mv[mt][r] = mv_new;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[mt][j][2 * r] *= a;
              acc[mt][j][2 * r + 1] *= a;
            }
          }
        put_weights();
        cp_async_wait();
        __syncthreads();
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        l[mt][0] += ws[mt][0];
        l[mt][1] += ws[mt][1];
      }

      copy_v(i + 1, next);  // to the buffer that the step before this one has read
      cp_async_commit();

      // ---- O += P V, this warp's channels (4g + j of column g in tile j) and blocks ----
      const uint8_t* v_at = s.v[i & 1][vb0] + v_read;
#pragma unroll
      for (int v = 0; v < VB; ++v) {
        uint32_t vr[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          vr[r] = *reinterpret_cast<const uint32_t*>(v_at + v * kBlockKeys * D + (r & 1) * V_ODD +
                                                     (r >> 1) * 8 * D);
        if (edge >> (src + vb0 + v) & 1u) {
          const int vpos = __shfl_sync(0xffffffffu, info.pos, src + vb0 + v);
          bool nan = false;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            // what lies behind the last key may be anything
            if (static_cast<long long>(vpos) + 2 * t + (r & 1) + (r >> 1) * 8 >= sg.len) vr[r] = 0u;
            nan |= nan_codes(vr[r]) != 0;
          }
          if (p.Sq > 1 && __any_sync(0xffffffffu, nan)) {
            // NaN values go to the rows that see their keys, and to no others (as in
            // the narrow kernel)
            uint32_t n[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              n[r] = nan_codes(vr[r]) & 0x38383838u;
              vr[r] &= ~nan_codes(vr[r]);
            }
            uint32_t b[2][4];
            pair_up(n, b);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint32_t see[2][2];
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const int last = sg.len - p.Sq + (sg.row0 + mt * 16 + r * 8 + g) % p.Sq - vpos - 2 * t;
                see[0][r] = (last >= 0 ? 0x3c00u : 0u) | (last >= 1 ? 0x3c000000u : 0u);
                see[1][r] = (last >= 8 ? 0x3c00u : 0u) | (last >= 9 ? 0x3c000000u : 0u);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(c, see[0][0], see[0][1], see[1][0], see[1][1], b[0][j], b[1][j]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (c[e] > 0.f) acc[mt][j][e] = __int_as_float(0x7fffffff);
              }
            }
          }
        }
        uint32_t b[2][4];
        pair_up(vr, b);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint4 a = s.w[i & 1][vb0 + v][mt][lane];
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_f16(acc[mt][j], a.x, a.y, a.z, a.w, b[0][j], b[1][j]);
        }
      }
    }

    // ---- the CTA's state ----
    __syncthreads();  // the values have been read: their place takes the result
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float sum = l[mt][r];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int row = mt * 16 + r * 8 + g;
        if (t == 0) {
          s.l[warp][row] = sum;
          if (warp == 0) {
            s.m[row] = m[mt][r];
            s.mv[row] = mv[mt][r];
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float4*>(&s.o[warp / DW][row][dw * 32 + 8 * t + 4 * e]) =
              make_float4(acc[mt][0][2 * r + e], acc[mt][1][2 * r + e], acc[mt][2][2 * r + e],
                          acc[mt][3][2 * r + e]);
      }
    __syncthreads();
    for (int idx = tid; idx < sg.n_rows * (D / 4); idx += kThreads) {
      const int row = idx / (D / 4), c = (idx % (D / 4)) * 4;
      float4 o = *reinterpret_cast<const float4*>(&s.o[0][row][c]);
      if constexpr (D == 64) {
        const float4 u = *reinterpret_cast<const float4*>(&s.o[1][row][c]);
        o = make_float4(o.x + u.x, o.y + u.y, o.z + u.z, o.w + u.w);
      }
      float L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) L += s.l[w][row];
      emit<D>(p, sg, R, row, c, s.m[row], L, s.mv[row], o, part_o, part_ml);
    }
    __syncthreads();
    if (tid == 0) s.seg.next(p, row_blocks, R, s.line);
    __syncthreads();
  }
}

// Joins the partial states of the units (item and row block) that lie in several CTAs' stretches,
// in their order, and writes the rows of items without any key.  A row's states go
// through kSplit warps (four when there are few rows and so, for long contexts, many states
// per row; else one); each keeps up to four states' loads in flight.
//
// A CTA takes `span` groups of kWarps / kSplit rows, one after another in the items' order.  Where
// its first item begins in the line is summed up while the partial kernel still runs: that takes
// only the lengths and lists, which were complete before that kernel let this one launch.
// From there the CTA walks.  (With the whole line built by every warp of a CTA for each
// group of rows the plan took 40% as many instructions as the attention of 512 items, and grew with
// the square of the items: 100 ms for 32000 of them, 4000 requests of 8 heads.)
template <int D, int kSplit>
__global__ void __launch_bounds__(kThreads)
    fa_decode_paged_merge(const PagedDecodeParams p, int row_blocks, int tile_rows, int ctas,
                          int span, const float* part_o, const RowState* part_ml) {
  constexpr int E = D / 32;
  constexpr int kRows = kWarps / kSplit;  // rows per group
  constexpr int kBatch = 4;
  __shared__ Place place;
  __shared__ float s_m[kWarps], s_l[kWarps], s_mv[kWarps];
  __shared__ __align__(16) float s_o[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % kSplit;
  const int items = p.B * p.s.Hkv;
  const int groups = (p.rows + kRows - 1) / kRows;  // of an item
  const int first = blockIdx.x * span;
  int item = first / groups;
  int left = min(span, items * groups - first);     // groups still to be taken
  int row = (first - item * groups) * kRows + warp / kSplit;
  place.sum(p, item);
  int n_kb = item_blocks<true>(p, item);
  __syncthreads();
  long long start = Place::of(place.before) * row_blocks;
  const long long share = share_of(Place::of(place.all) * row_blocks, items, ctas);
  int r, c0, c1;  // row of the unit, the CTAs of its first and last block
  auto locate = [&] {
    if (n_kb == 0) return;
    const int rb = row / tile_rows;
    r = row - rb * tile_rows;
    const long long at = start + rb * unit_places(n_kb) + kSegmentCost;  // the unit's first block
    c0 = cta_of(at, share);
    c1 = cta_of(at + n_kb - 1, share);
  };
  locate();
  // Every CTA waits, also one with nothing to join: what follows this kernel in
  // the stream may then rely on the partial kernel's completion as well.
  griddep_wait();
  while (true) {
    const bool real = row < p.rows;
    const size_t qrow = static_cast<size_t>(item) * p.rows + row;
    if (n_kb == 0) {  // no key: O = 0, LSE = -inf
      if (real && part == 0) {
        uint32_t* out =
            reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + qrow * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) out[e / 2] = 0u;
        if (p.lse && lane == 0) p.lse[qrow] = neg_inf();
      }
    } else if (c0 != c1) {  // else one CTA has finished the rows of the unit
      float M = kNoMax, L = 0.f, MV = kNoMax, o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = 0.f;
      auto move_to = [&](float m, float mv) {  // the state is taken against m and mv
        L *= ex2_approx(M - m);
        const float a = ex2_approx(MV - mv);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= a;
        M = m;
        MV = mv;
      };
      auto add = [&](float m, float l, float mv, auto&& acc) {  // a state below M and MV
        L = fmaf(ex2_approx(m - M), l, L);
        const float w = ex2_approx(mv - MV);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(w, acc(e), o[e]);
      };
      if (real) {
        for (int c = c0 + part; c <= c1; c += kSplit * kBatch) {
          RowState ml[kBatch];
          float v[kBatch][E];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int cc = c + i * kSplit;
            const size_t slot = (2 * static_cast<size_t>(cc) + (cc == c0 ? 1 : 0)) * tile_rows + r;
            ml[i] = row_state(kNoMax, 0.f, kNoMax);
#pragma unroll
            for (int e = 0; e < E; ++e) v[i][e] = 0.f;
            if (cc <= c1) {
              ml[i] = part_ml[slot];
              if constexpr (E == 4) {
                const float4 x = *reinterpret_cast<const float4*>(part_o + slot * D + lane * 4);
                v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
              } else {
                const float2 x = *reinterpret_cast<const float2*>(part_o + slot * D + lane * 2);
                v[i][0] = x.x, v[i][1] = x.y;
              }
            }
          }
          float m = M, mv = MV;
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            m = fmaxf(m, ml[i].x);
            mv = fmaxf(mv, ml[i].z);
          }
          move_to(m, mv);
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            add(ml[i].x, ml[i].y, ml[i].z, [&](int e) { return v[i][e]; });
        }
      }
      if constexpr (kSplit > 1) {
        if (lane == 0) {
          s_m[warp] = M;
          s_l[warp] = L;
          s_mv[warp] = MV;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
        __syncthreads();
        if (part == 0) {
          float m = M, mv = MV;
#pragma unroll
          for (int w = 1; w < kSplit; ++w) {
            m = fmaxf(m, s_m[warp + w]);
            mv = fmaxf(mv, s_mv[warp + w]);
          }
          move_to(m, mv);
#pragma unroll
          for (int w = 1; w < kSplit; ++w)
            add(s_m[warp + w], s_l[warp + w], s_mv[warp + w],
                [&](int e) { return s_o[warp + w][lane * E + e]; });
        }
      }
      if (real && part == 0) {
        const bool empty = L == 0.f;
        const float inv = empty ? 0.f : 1.f / L, unit = value_unit(M, MV);
        uint32_t* out =
            reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + qrow * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16x2(o[e] * inv * unit, o[e + 1] * inv * unit);
        if (p.lse && lane == 0)
          p.lse[qrow] = empty ? neg_inf() : (M + __log2f(L)) * 0.69314718055994530942f;
      }
    }
    if (kSplit > 1 || --left == 0) break;  // with four warps a row a CTA has one row
    row += kRows;
    if (row - warp / kSplit >= p.rows) {  // the next item
      start += unit_places(n_kb) * row_blocks;
      n_kb = item_blocks<true>(p, ++item);
      row = warp / kSplit;
    }
    locate();
  }
}

template <int D, int NT>
cudaError_t launch_nt(const PagedDecodeParams& p, cudaStream_t stream) {
  constexpr size_t smem = NT == 1 ? sizeof(NarrowSmem<D>) : sizeof(WideSmem<D, NT == 1 ? 2 : NT>);
  static_assert(smem <= 48 * 1024, "fits without an opt-in");
  const int row_blocks = (p.rows + 8 * NT - 1) / (8 * NT);
  // no more CTAs than there can be shares
  const long long list = p.sel ? p.max_sel : p.max_blocks;
  const long long most =
      ((list << p.block_shift) + kSegmentCost) * p.B * p.s.Hkv * row_blocks;
  const int ctas = static_cast<int>(min(static_cast<long long>(kSms * Plan<NT>::kCtasPerSm), most));
  float* part_o = static_cast<float*>(p.workspace);
  RowState* part_ml = reinterpret_cast<RowState*>(part_o + 2 * static_cast<size_t>(ctas) * 8 * NT * D);
  const float* c_o = part_o;
  const RowState* c_ml = part_ml;
  cudaError_t e;
  hook_before(stream);
  if constexpr (NT == 1)
    e = launch_dependent(fa_decode_paged_narrow<D>, dim3(ctas), dim3(kThreads), smem, stream, p,
                         row_blocks, part_o, part_ml);
  else
    e = launch_dependent(fa_decode_paged_wide<D, NT>, dim3(ctas), dim3(kThreads), smem, stream, p,
                         row_blocks, part_o, part_ml);
  hook_after(stream);
  if (e != cudaSuccess) return e;
  // Four warps a row while there are no more rows than the GPU holds CTAs at once (8 per SM by
  // registers), then a warp each and no more CTAs than that.  1024 rows: 24.3 us with four warps
  // each, 26.0 with one; 2304 rows: 43.5 and 40.3.  2048 CTAs of one group: 45.7 us, 1024 of two 44.1.
  const int items = p.B * p.s.Hkv;
  constexpr int kMost = 8 * kSms;
  if (1LL * p.rows * items <= kMost)
    return launch_dependent(fa_decode_paged_merge<D, kWarps>, dim3(p.rows * items), dim3(kThreads), 0,
                            stream, p, row_blocks, 8 * NT, ctas, 1, c_o, c_ml);
  const int groups = (p.rows + kWarps - 1) / kWarps * items;
  const int span = (groups + kMost - 1) / kMost;
  return launch_dependent(fa_decode_paged_merge<D, 1>, dim3((groups + span - 1) / span),
                          dim3(kThreads), 0, stream, p, row_blocks, 8 * NT, ctas, span, c_o, c_ml);
}

template <int D>
cudaError_t launch_d(const PagedDecodeParams& p, cudaStream_t stream) {
  const int nt = row_tiles(p.rows);
  if (nt == 1) return launch_nt<D, 1>(p, stream);
  if (nt == 2) return launch_nt<D, 2>(p, stream);
  return launch_nt<D, 4>(p, stream);
}

}  // namespace

size_t decode_paged_workspace(int B, int Hkv, int rows, int d) {
  (void)B, (void)Hkv;
  const int nt = row_tiles(rows);
  return 2 * static_cast<size_t>(grid_ctas(nt)) * 8 * nt * (d * sizeof(float) + sizeof(RowState));
}

cudaError_t launch_decode_paged(const PagedDecodeParams& p, cudaStream_t stream) {
  return p.s.d == 128 ? launch_d<128>(p, stream) : launch_d<64>(p, stream);
}

}  // namespace fa
