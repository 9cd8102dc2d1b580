// fa_decode_paged.cu -- attention of the last Sq tokens of each request over a
// paged 8-bit KV cache, over every block or over a list of chosen blocks.
//
// The cache is read once (2 bytes per key, KV head and channel), so HBM bounds
// the kernel; the arithmetic only has to stay out of the way.  The query rows
// of a KV head (Hq / Hkv * Sq of them) are the narrow side of two
// mma.sync.m16n8k16 products in f16 with fp32 accumulation:
//   S^T[16 keys x 8 rows] = K Q^T,   O^T[d x 8 rows] += V^T P^T
// e4m3 codes become f16 exactly (one conversion per pair).  The page's K scale
// multiplies the scores in fp32, its V scale the weights in fp32.
//
// f16 and its range: a query row is multiplied by the power of two that puts
// its largest element into [2^14, 2^15), which loses nothing above 2^-38 of it.
// Weights are taken against a running maximum m that may lag by 2 (log2 units)
// and are stored as w * 2^13 * v_scale / v_ref <= 2^15 (v_ref: the largest V scale
// so far), so a weight keeps f16's 11 bits down to 2^-27 of the largest and is
// rounded by at most 2^-38 of it below.  Sums, maxima and accumulators are fp32.
//
// Operands without shared memory: the contraction index of a product may be
// permuted freely, so a lane loads 16-byte pieces of whole rows and hands their
// bytes to the products in the order they lie.  For K (rows = keys), lane (g, t)
// (g = lane / 4, t = lane % 4) loads channels [16t, 16t + 16) of keys g and g + 8;
// for V it loads channels [16g, 16g + 16) of keys 2t, 2t+1, 2t+8 and 2t+9, and one
// byte permutation pairs two keys of a channel.  The S^T accumulator becomes the
// P^T operand by movmatrix.
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
constexpr int kMinShare = 16;       // 16-key blocks a CTA takes at least
constexpr float kLag = 2.f;         // how far (log2) a weight may exceed the running maximum
constexpr float kWeightUnit = 8192.f;

// Row tiles of 8 a CTA serves, and CTAs per SM (by registers and shared memory).
template <int NT> struct Plan;
template <> struct Plan<1> { static constexpr int kCtasPerSm = 4; };
template <> struct Plan<2> { static constexpr int kCtasPerSm = 3; };
template <> struct Plan<4> { static constexpr int kCtasPerSm = 2; };

int row_tiles(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }
int grid_ctas(int nt) {
  return kSms * (nt == 1 ? Plan<1>::kCtasPerSm : nt == 2 ? Plan<2>::kCtasPerSm
                                                         : Plan<4>::kCtasPerSm);
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
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

__device__ __forceinline__ int request_len(const PagedDecodeParams& p, int b) {
  return static_cast<int>(min(static_cast<long long>(max(p.seqlens[b], 0)),
                              static_cast<long long>(p.max_blocks) * p.s.page_size));
}

// 16-key blocks of a (request, KV head).
__device__ __forceinline__ int item_blocks(const PagedDecodeParams& p, int item) {
  if (p.sel) return min(max(p.n_sel[item], 0), p.max_sel) * (p.s.page_size / kBlockKeys);
  return (request_len(p, item / p.s.Hkv) + kBlockKeys - 1) / kBlockKeys;
}

// Where the blocks of the items lie in the one long line: thread t of the CTA
// sums items [t * per, (t + 1) * per), prefix[t] is the start of its first one.
struct Line {
  long long prefix[kThreads + 1];
  long long warp_sum[kWarps];
};

__device__ __forceinline__ void make_line(const PagedDecodeParams& p, int row_blocks, Line& s) {
  const int items = p.B * p.s.Hkv;
  const int per = (items + kThreads - 1) / kThreads;
  const int lo = min(static_cast<int>(threadIdx.x) * per, items), hi = min(lo + per, items);
  long long own = 0;
  for (int i = lo; i < hi; ++i) own += item_blocks(p, i);
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
}

__device__ __forceinline__ long long share_of(long long total, int ctas) {
  return max((total + ctas - 1) / ctas, static_cast<long long>(kMinShare));
}

template <int D, int NT>
struct DecodeSmem {
  Line line;
  float m[kWarps][8 * NT];
  float l[kWarps][8 * NT];
  alignas(16) float o[kWarps][8 * NT][D + 4];
  alignas(16) uint2 q[NT > 1 ? NT * (D / 16) * 32 : 1];  // Q fragments; registers hold them for one tile
  float c_row[8 * NT];
};

// What a lane looks up for one of its warp's coming blocks.
struct BlockInfo {
  long long offset;  // bytes from the start of a cache tensor to the block's first key
  int pos;           // position of the first key; INT_MAX: the block is hidden
  float ks, vs;
};

__device__ __forceinline__ BlockInfo look_up(const PagedDecodeParams& p, int item, int hk, int len,
                                             const int32_t* table, int kb, int d) {
  const int ps = p.s.page_size, per_page = ps / kBlockKeys;
  const int idx = kb / per_page, sub = kb % per_page;
  const int blk = p.sel ? p.sel[static_cast<size_t>(item) * p.max_sel + idx] : idx;
  BlockInfo r = {0, 0x7fffffff, 1.f, 1.f};
  if (blk >= 0 && static_cast<long long>(blk) * ps + sub * kBlockKeys < len) {
    const int page = table[blk];
    if (page >= 0 && page < p.s.num_pages) {
      const size_t tile = static_cast<size_t>(page) * p.s.Hkv + hk;
      r.offset = (static_cast<long long>(tile) * ps + sub * kBlockKeys) * d;
      r.pos = blk * ps + sub * kBlockKeys;
      r.ks = p.k_scale[tile];
      r.vs = p.v_scale[tile];
    }
  }
  return r;
}

__device__ __forceinline__ bool has_nan_code(uint32_t w) {
  return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Plan<NT>::kCtasPerSm)
    fa_decode_paged_kernel(const PagedDecodeParams p, int row_blocks, float* part_o, float2* part_ml) {
  constexpr int KC = D / 64;       // 16-byte pieces of a key row per lane
  constexpr int KS = D / 16;       // k-steps of S
  constexpr int MT = D / 16;       // m-tiles of O^T
  constexpr int VW = D / 32;       // 32-bit words of a value row per lane
  constexpr int R = 8 * NT;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  DecodeSmem<D, NT>& s = *reinterpret_cast<DecodeSmem<D, NT>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int items = p.B * p.s.Hkv;

  make_line(p, row_blocks, s.line);
  const long long total = s.line.prefix[kThreads];
  const long long share = share_of(total, gridDim.x);
  long long at = share * blockIdx.x;
  const long long end = min(at + share, total);
  if (at >= end) {
    griddep_launch_dependents();
    return;
  }
  // the item that holds position `at`, and the position inside it
  int item;
  long long in_item;
  {
    int a = 0, z = kThreads;
    while (z - a > 1) {
      const int mid = (a + z) >> 1;
      if (s.line.prefix[mid] <= at) a = mid; else z = mid;
    }
    item = a * ((items + kThreads - 1) / kThreads);
    in_item = at - s.line.prefix[a];
    while (true) {
      const long long w = static_cast<long long>(item_blocks(p, item)) * row_blocks;
      if (in_item < w) break;
      in_item -= w;
      ++item;
    }
  }

  while (at < end) {
    const int n_kb = item_blocks(p, item);
    if (n_kb == 0) {  // an item without keys takes no place in the line
      ++item;
      in_item = 0;
      continue;
    }
    const int rb = static_cast<int>(in_item / n_kb);
    const int kb0 = static_cast<int>(in_item % n_kb);
    const int n_seg = static_cast<int>(min(static_cast<long long>(n_kb - kb0), end - at));
    const int b = item / p.s.Hkv, hk = item % p.s.Hkv;
    const int len = request_len(p, b);
    const int row0 = rb * R;
    const int n_rows = min(R, p.rows - row0);
    const int32_t* table = p.block_table + static_cast<size_t>(b) * p.max_blocks;
    const size_t qrow0 = static_cast<size_t>(item) * p.rows + row0;

    // ---- queries: scaled by a power of two per row, as B operands ----
    uint2 qf[NT == 1 ? KS : 1];
    float c_row[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (NT > 1 && (nt % kWarps) != warp) continue;  // the warps share the work, through s.q
      const int r = nt * 8 + g;
      uint4 w[2 * KC];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 2 * KC; ++i) {
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < n_rows)
          w[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                 (qrow0 + r) * D + (i / 2) * 64 + t * 16 +
                                                 (i % 2) * 8);
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = __vmaxu2(top, x[e] & 0x7fff7fffu);
      }
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ex = max(static_cast<int>(max(top & 0xffffu, top >> 16) >> 7) - 127, -100);
      const float up = pow2i(14 - ex);
      const float c = p.scale_log2 * pow2i(ex - 14);
#pragma unroll
      for (int i = 0; i < 2 * KC; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          h[e] = pack_f16x2(__uint_as_float(x[e] << 16) * up,
                            __uint_as_float(x[e] & 0xffff0000u) * up);
        // k-step (i / 2) * 4 + (i % 2) * 2 + {0, 1}: four channels each
        const int ks = (i / 2) * 4 + (i % 2) * 2;
        if (NT == 1) {
          qf[ks] = make_uint2(h[0], h[1]);
          qf[ks + 1] = make_uint2(h[2], h[3]);
        } else {
          s.q[(nt * KS + ks) * 32 + lane] = make_uint2(h[0], h[1]);
          s.q[(nt * KS + ks + 1) * 32 + lane] = make_uint2(h[2], h[3]);
        }
      }
      if (NT == 1) {
        c_row[0][0] = __shfl_sync(0xffffffffu, c, 8 * t);
        c_row[0][1] = __shfl_sync(0xffffffffu, c, 8 * t + 4);
      } else if (t == 0) {
        s.c_row[r] = c;
      }
    }
    if (NT > 1) {
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        c_row[nt][0] = s.c_row[nt * 8 + 2 * t];
        c_row[nt][1] = s.c_row[nt * 8 + 2 * t + 1];
      }
    }

    float m[NT][2], l[NT][2], acc[NT][MT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = neg_inf();
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][j][e] = 0.f;
    }
    float v_ref = 0.f, v_mul = 0.f;  // v_mul = 2^13 / v_ref

    const int mine = (n_seg - warp + kWarps - 1) / kWarps;  // blocks kb0 + warp + i * kWarps
    BlockInfo info = {0, 0x7fffffff, 1.f, 1.f};
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
    // P^T (B operand) times V^T, for the value words as they stand
    auto add_pv = [&](const uint32_t (&pb)[NT][2]) {
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
        const uint32_t lo = __byte_perm(vr[0][j >> 1], vr[1][j >> 1], sel);
        const uint32_t hi = __byte_perm(vr[2][j >> 1], vr[3][j >> 1], sel);
        const uint32_t a0 = e4m3x2_to_f16x2(lo), a1 = e4m3x2_to_f16x2(lo >> 16);
        const uint32_t a2 = e4m3x2_to_f16x2(hi), a3 = e4m3x2_to_f16x2(hi >> 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_f16(acc[nt][j], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
      }
    };

    // A NaN value must reach the rows that see its key and no others (0 * NaN is
    // NaN): the product of "code is NaN" and "row sees key" says where it goes, and
    // the code becomes 0 for the product with the weights.
    auto mark_nan = [&](uint32_t hidden) {
      uint32_t see[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint32_t h = hidden >> (nt * 4);
        see[nt][0] = transpose8x8(((h & 1u) ? 0u : 0x3c00u) | ((h & 2u) ? 0u : 0x3c000000u));
        see[nt][1] = transpose8x8(((h & 4u) ? 0u : 0x3c00u) | ((h & 8u) ? 0u : 0x3c000000u));
      }
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
        uint32_t n[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)  // 0x38 is e4m3's 1.0
          n[r] = __vcmpeq4(vr[r][j >> 1] & 0x7f7f7f7fu, 0x7f7f7f7fu) & 0x38383838u;
        const uint32_t lo = __byte_perm(n[0], n[1], sel), hi = __byte_perm(n[2], n[3], sel);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float c[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16(c, e4m3x2_to_f16x2(lo), e4m3x2_to_f16x2(lo >> 16), e4m3x2_to_f16x2(hi),
                  e4m3x2_to_f16x2(hi >> 16), see[nt][0], see[nt][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c[e] > 0.f) acc[nt][j][e] = __int_as_float(0x7fffffff);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int w = 0; w < VW; ++w)
          vr[r][w] &= ~__vcmpeq4(vr[r][w] & 0x7f7f7f7fu, 0x7f7f7f7fu);
    };

    for (int i = 0; i < mine; ++i) {
      if ((i & 31) == 0) {  // the next 32 blocks of this warp, one per lane
        const int kb = i + lane < mine ? kb0 + warp + (i + lane) * kWarps : -1;
        if (kb >= 0) info = look_up(p, item, hk, len, table, kb, D);
        const long long off = __shfl_sync(0xffffffffu, info.offset, 0);
        load_k(off);
        load_v(off);
      }
      const int src = i & 31;
      const int pos = __shfl_sync(0xffffffffu, info.pos, src);
      const float ks = __shfl_sync(0xffffffffu, info.ks, src);
      const float vs = __shfl_sync(0xffffffffu, info.vs, src);
      const bool more = i + 1 < mine && src != 31;
      const long long next = __shfl_sync(0xffffffffu, info.offset, (src + 1) & 31);

      // ---- S^T = K Q^T ----
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nt][e] = 0.f;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const uint32_t wa[4] = {kr[0][c].x, kr[0][c].y, kr[0][c].z, kr[0][c].w};
        const uint32_t wb[4] = {kr[1][c].x, kr[1][c].y, kr[1][c].z, kr[1][c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t a0 = e4m3x2_to_f16x2(wa[e]), a2 = e4m3x2_to_f16x2(wa[e] >> 16);
          const uint32_t a1 = e4m3x2_to_f16x2(wb[e]), a3 = e4m3x2_to_f16x2(wb[e] >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 q = NT == 1 ? qf[NT == 1 ? c * 4 + e : 0] : s.q[(nt * KS + c * 4 + e) * 32 + lane];
            mma_f16(x[nt], a0, a1, a2, a3, q.x, q.y);
          }
        }
      }
      if (more) load_k(next);

      // ---- weights against the running maximum ----
      // x[nt]: {key g, row 2t}, {key g, row 2t+1}, {key g+8, row 2t}, {key g+8, row 2t+1}
      const bool edge = static_cast<long long>(pos) + kBlockKeys - 1 > len - p.Sq;
      float arg[NT][4];
      bool over = vs > v_ref;
      uint32_t hidden = 0;  // bit nt * 4 + e
      if (edge) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = row0 + nt * 8 + 2 * t + (e & 1);
            const long long key = static_cast<long long>(pos) + g + (e >> 1) * 8;
            if (key > len - p.Sq + row % p.Sq) hidden |= 1u << (nt * 4 + e);
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f = ks * c_row[nt][e & 1];
          arg[nt][e] = fmaf(x[nt][e], f, -m[nt][e & 1]);
          if (edge && (hidden >> (nt * 4 + e) & 1u)) arg[nt][e] = neg_inf();
          over |= arg[nt][e] > kLag;
        }
      if (__any_sync(0xffffffffu, over)) {
        // exact maximum of the block's rows; the state moves to it
        float v_down = 1.f;
        if (vs > v_ref) {
          v_down = v_ref / vs;  // 0 before the first block
          v_ref = vs;
          v_mul = kWeightUnit / vs;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float f = ks * c_row[nt][r];
            float mx = neg_inf();
            if (!(hidden >> (nt * 4 + r) & 1u)) mx = x[nt][r] * f;
            if (!(hidden >> (nt * 4 + 2 + r) & 1u)) mx = fmaxf(mx, x[nt][2 + r] * f);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float m_new = fmaxf(m[nt][r], mx);
            const float a = m[nt][r] == neg_inf() ? 0.f : ex2_approx(m[nt][r] - m_new);
            m[nt][r] = m_new;
            l[nt][r] *= a;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              acc[nt][j][r] *= a * v_down;
              acc[nt][j][2 + r] *= a * v_down;
            }
#pragma unroll
            for (int e = r; e < 4; e += 2)
              arg[nt][e] = (hidden >> (nt * 4 + e) & 1u) ? neg_inf()
                                                         : fmaf(x[nt][e], f, -m_new);
          }
      }
      const float unit = vs * v_mul;
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = ex2_approx(arg[nt][e]);
          l[nt][e & 1] += w[e];
          w[e] *= unit;
        }
        pb[nt][0] = transpose8x8(pack_f16x2(w[0], w[1]));
        pb[nt][1] = transpose8x8(pack_f16x2(w[2], w[3]));
      }

      // ---- O^T += V^T P^T ----
      if (edge) {
        bool nan = false;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool dead = static_cast<long long>(pos) + 2 * t + (r & 1) + (r >> 1) * 8 >= len;
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            if (dead) vr[r][w] = 0u;  // what lies behind the last key may be anything
            nan |= has_nan_code(vr[r][w]);
          }
        }
        if (p.Sq > 1 && __any_sync(0xffffffffu, nan)) mark_nan(hidden);
      }
      add_pv(pb);
      if (more) load_v(next);
    }

    // ---- merge the warps' states ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float sum = l[nt][r];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const int row = nt * 8 + 2 * t + r;
        if (g == 0) {
          s.m[warp][row] = m[nt][r];
          s.l[warp][row] = sum;
        }
        const float back = v_ref * (1.f / kWeightUnit);
#pragma unroll
        for (int j = 0; j < MT; ++j)
          *reinterpret_cast<float2*>(&s.o[warp][row][g * (D / 8) + 2 * j]) =
              make_float2(acc[nt][j][r] * back, acc[nt][j][2 + r] * back);
      }
    __syncthreads();
    const bool whole = n_seg == n_kb;
    const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (kb0 == 0 ? 1 : 0);
    for (int idx = tid; idx < n_rows * (D / 4); idx += kThreads) {
      const int row = idx / (D / 4), c = (idx % (D / 4)) * 4;
      float M = neg_inf();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s.m[w][row]);
      float L = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float wt = s.m[w][row] == neg_inf() ? 0.f : ex2_approx(s.m[w][row] - M);
        const float4 v = *reinterpret_cast<const float4*>(&s.o[w][row][c]);
        // a warp without a visible key has l = 0 (or NaN, which has to stay)
        L += wt == 0.f ? s.l[w][row] * 0.f : wt * s.l[w][row];
        o.x = fmaf(wt, v.x, o.x);
        o.y = fmaf(wt, v.y, o.y);
        o.z = fmaf(wt, v.z, o.z);
        o.w = fmaf(wt, v.w, o.w);
      }
      if (whole) {
        const bool empty = L == 0.f;
        const float inv = empty ? 0.f : 1.f / L;
        uint2 w;
        w.x = pack_bf16x2(o.x * inv, o.y * inv);
        w.y = pack_bf16x2(o.z * inv, o.w * inv);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + (qrow0 + row) * D + c) = w;
        if (p.lse && c == 0)
          p.lse[qrow0 + row] = empty ? neg_inf() : (M + __log2f(L)) * 0.69314718055994530942f;
      } else {
        *reinterpret_cast<float4*>(part_o + (slot * R + row) * D + c) = o;
        if (c == 0) part_ml[slot * R + row] = make_float2(M, L);
      }
    }
    __syncthreads();
    at += n_seg;
    in_item += n_seg;
    if (in_item >= static_cast<long long>(n_kb) * row_blocks) {
      ++item;
      in_item = 0;
    }
  }
  griddep_launch_dependents();
}

// One CTA per (query row, item): joins the partial states of an item that lies in
// several CTAs' stretches, and writes the rows of items without any key.
template <int D>
__global__ void __launch_bounds__(kThreads)
    fa_decode_paged_merge(const PagedDecodeParams p, int row_blocks, int tile_rows, int ctas,
                          const float* part_o, const float2* part_ml) {
  constexpr int E = D / 32;
  __shared__ Line line;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  const int row = blockIdx.x, item = blockIdx.y;
  const int n_kb = item_blocks(p, item);
  const int rb = row / tile_rows, r = row % tile_rows;
  const size_t qrow = static_cast<size_t>(item) * p.rows + row;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) + qrow * D;
  if (n_kb == 0) {
    griddep_wait();
    for (int c = threadIdx.x; c < D; c += kThreads) out[c] = __float2bfloat16_rn(0.f);
    if (p.lse && threadIdx.x == 0) p.lse[qrow] = neg_inf();
    return;
  }
  make_line(p, row_blocks, line);
  const int items = p.B * p.s.Hkv;
  const int per = (items + kThreads - 1) / kThreads;
  long long start = line.prefix[item / per];
  for (int i = item / per * per; i < item; ++i)
    start += static_cast<long long>(item_blocks(p, i)) * row_blocks;
  start += static_cast<long long>(rb) * n_kb;
  const long long share = share_of(line.prefix[kThreads], ctas);
  const int c0 = static_cast<int>(start / share);
  const int c1 = static_cast<int>((start + n_kb - 1) / share);
  // Every CTA waits, also one with nothing to join: what follows this kernel in
  // the stream may then rely on the partial kernel's completion as well.
  griddep_wait();
  if (c0 == c1) return;  // one CTA finished it
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float M = neg_inf(), L = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int c = c0 + warp; c <= c1; c += kWarps) {
    const size_t at = (2 * static_cast<size_t>(c) + (c == c0 ? 1 : 0)) * tile_rows + r;
    const float2 ml = part_ml[at];
    const float m_new = fmaxf(M, ml.x);
    const float a = M == neg_inf() ? 0.f : ex2_approx(M - m_new);
    const float w = ml.x == neg_inf() ? 0.f : ex2_approx(ml.x - m_new);
    M = m_new;
    L = L * a + (w == 0.f ? ml.y * 0.f : w * ml.y);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(w, part_o[at * D + lane * E + e], o[e] * a);
  }
  if (lane == 0) {
    s_m[warp] = M;
    s_l[warp] = L;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kThreads) {
    M = neg_inf();
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
    float sum = 0.f, v = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float wt = s_m[w] == neg_inf() ? 0.f : ex2_approx(s_m[w] - M);
      sum += wt == 0.f ? s_l[w] * 0.f : wt * s_l[w];
      v = fmaf(wt, s_o[w][c], v);
    }
    const bool empty = sum == 0.f;
    out[c] = __float2bfloat16_rn(empty ? 0.f : v / sum);
    if (p.lse && c == 0)
      p.lse[qrow] = empty ? neg_inf() : (M + __log2f(sum)) * 0.69314718055994530942f;
  }
}

template <int D, int NT>
cudaError_t launch_nt(const PagedDecodeParams& p, cudaStream_t stream) {
  const size_t smem = sizeof(DecodeSmem<D, NT>);
  cudaError_t e = cudaFuncSetAttribute(fa_decode_paged_kernel<D, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int row_blocks = (p.rows + 8 * NT - 1) / (8 * NT);
  // no more CTAs than there can be shares
  const long long list = p.sel ? p.max_sel : p.max_blocks;
  const long long most = list * (p.s.page_size / kBlockKeys) * p.B * p.s.Hkv * row_blocks;
  const int ctas = static_cast<int>(min(static_cast<long long>(kSms * Plan<NT>::kCtasPerSm),
                                        (most + kMinShare - 1) / kMinShare));
  float* part_o = static_cast<float*>(p.workspace);
  float2* part_ml = reinterpret_cast<float2*>(part_o + 2 * static_cast<size_t>(ctas) * 8 * NT * D);
  hook_before(stream);
  fa_decode_paged_kernel<D, NT><<<ctas, kThreads, smem, stream>>>(p, row_blocks, part_o, part_ml);
  hook_after(stream);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_dependent(fa_decode_paged_merge<D>, dim3(p.rows, p.B * p.s.Hkv), dim3(kThreads), 0,
                          stream, p, row_blocks, 8 * NT, ctas, static_cast<const float*>(part_o),
                          static_cast<const float2*>(part_ml));
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
  return 2 * static_cast<size_t>(grid_ctas(nt)) * 8 * nt * (d * sizeof(float) + sizeof(float2));
}

cudaError_t launch_decode_paged(const PagedDecodeParams& p, cudaStream_t stream) {
  return p.s.d == 128 ? launch_d<128>(p, stream) : launch_d<64>(p, stream);
}

}  // namespace fa
