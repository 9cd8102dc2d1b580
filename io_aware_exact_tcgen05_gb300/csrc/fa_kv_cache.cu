// fa_kv_cache.cu -- the paged 8-bit KV cache: block tables and slot maps from
// request lengths (fa_kv_assign), the quantising write (fa_kv_write_fp8) and
// the dequantising read (fa_kv_read_fp8).
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "fa_internal.h"
#include "fa_kv.h"
#include "fa_kv_device.cuh"

namespace fa {
namespace {

// ----------------------------------------------------------------- assign --
//
// Request b holds len_b tokens and gets new_b more:
//   have = ceil(len / ps), full = ceil((len + new) / ps), need = full - have,
//   end_b = sum_{i<=b} need_i; its new pages are free_pages[end_b - need_b ..).
// Token t of the packed new tokens belongs to the request with
// cu_new[b] <= t < cu_new[b+1].  A block past `have` starts with a new token, so
// the thread that holds that token also writes the block's table entry.
//
// Every CTA scans the lengths itself, 256 requests at a time (a few KB from
// L2), and then serves its own stretch of tokens: one launch, no exchange
// between CTAs.
constexpr int kAssignThreads = 256;
constexpr int kAssignTokens = 1024;  // packed tokens per CTA

__device__ __forceinline__ long long block_scan_inclusive(long long v, long long* warp_sums,
                                                          long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // warp_sums of an earlier scan have been read
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  long long before = 0, sum = 0;
  for (int w = 0; w < kAssignThreads / 32; ++w) {
    const long long x = warp_sums[w];
    if (w < warp) before += x;
    sum += x;
  }
  *total = sum;
  return v + before;
}

__device__ __forceinline__ int32_t clamp_i32(long long v) {
  return static_cast<int32_t>(v > 0x7fffffffll ? 0x7fffffffll : v);
}

__global__ void __launch_bounds__(kAssignThreads) fa_kv_assign_kernel(const KvAssignParams p) {
  __shared__ long long s_cu[kAssignThreads + 1];
  __shared__ long long s_start[kAssignThreads];
  __shared__ int s_seq[kAssignThreads], s_have[kAssignThreads];
  __shared__ bool s_live[kAssignThreads];
  __shared__ long long s_sums[kAssignThreads / 32];
  __shared__ int s_used;
  const int tid = threadIdx.x;
  const int shift = 31 - __clz(p.page_size);  // a power of two
  const long long t_lo = static_cast<long long>(blockIdx.x) * kAssignTokens;
  const long long t_hi = min(t_lo + kAssignTokens, static_cast<long long>(p.total_new));
  const bool first_cta = blockIdx.x == 0;
  long long cu0 = 0, need0 = 0, k0 = 0;  // totals of the requests before this chunk
  if (tid == 0) s_used = 0;
  griddep_wait();
  for (int base = 0; base < p.B; base += kAssignThreads) {
    const int b = base + tid;
    const bool real = b < p.B;
    const long long seq = real ? max(p.seqlens[b], 0) : 0;
    const long long add = real ? max(p.newlens[b], 0) : 0;
    long long sum_new, sum_need;
    const long long cu_end = cu0 + block_scan_inclusive(add, s_sums, &sum_new);
    const long long have = (seq + p.page_size - 1) >> shift;
    const long long full = (seq + add + p.page_size - 1) >> shift;
    const bool never = full > p.max_blocks || cu_end > p.total_new;
    const long long need = never ? 0 : full - have;
    const long long end = need0 + block_scan_inclusive(need, s_sums, &sum_need);
    const bool refused = never || (need > 0 && end > p.n_free);
    s_cu[tid] = cu_end - add;
    if (tid == kAssignThreads - 1) s_cu[kAssignThreads] = cu_end;
    s_start[tid] = end - need;
    s_seq[tid] = static_cast<int>(seq);
    s_have[tid] = static_cast<int>(min(have, static_cast<long long>(p.max_blocks)));
    s_live[tid] = real && !refused;
    if (first_cta) {
      const long long out = refused ? seq : seq + add;
      long long sum_k;
      const long long k_end = k0 + block_scan_inclusive(real ? out : 0, s_sums, &sum_k);
      if (real) {
        p.seqlens_out[b] = clamp_i32(out);
        p.cu_new[b + 1] = clamp_i32(cu_end);
        p.cu_k[b + 1] = clamp_i32(k_end);
        if (b == 0) p.cu_new[0] = p.cu_k[0] = 0;
        if (!refused && need > 0) atomicMax(&s_used, static_cast<int>(end));
      }
      k0 += sum_k;
    }
    __syncthreads();
    // this chunk's part of the CTA's tokens
    const long long lo = max(t_lo, s_cu[0]), hi = min(t_hi, s_cu[kAssignThreads]);
    for (long long t = lo + tid; t < hi; t += kAssignThreads) {
      int a = 0, z = kAssignThreads;  // last request with s_cu <= t
      while (z - a > 1) {
        const int mid = (a + z) >> 1;
        if (s_cu[mid] <= t) a = mid; else z = mid;
      }
      long long slot = -1;
      if (s_live[a]) {
        // a live request fits its table, whose positions fit 31 bits
        const int pos = s_seq[a] + static_cast<int>(t - s_cu[a]);
        const int blk = pos >> shift;
        const int off = pos & (p.page_size - 1);
        int32_t* row = p.block_table + static_cast<long long>(base + a) * p.max_blocks;
        int page;
        if (blk < s_have[a]) {
          page = row[blk];
        } else {
          page = p.free_pages[s_start[a] + (blk - s_have[a])];
          if (off == 0) row[blk] = page;
        }
        if (page >= 0) slot = static_cast<long long>(page) * p.page_size + off;
      }
      p.slot_map[t] = slot;
    }
    cu0 += sum_new;
    need0 += sum_need;
    __syncthreads();
    if (!first_cta && cu0 >= t_hi) break;
  }
  // packed rows behind the last request
  for (long long t = max(t_lo, cu0) + tid; t < t_hi; t += kAssignThreads) p.slot_map[t] = -1;
  if (first_cta && tid == 0) *p.n_used = s_used;
}

// ------------------------------------------------------------------ write --
//
// A run is the new tokens of one page.  With n tokens in the page before it,
//   s_tok = 2^e, e the smallest with amax(new) <= 448 * 2^e (finite values),
//   s = max(s_old, s_tok) if n > 0, else s_tok,
//   new code = rn_sat(x / s), held code = rn(code * s_old / s).
// With power-of-two scales both are exact but for e4m3's own rounding, so a
// page that is requantised loses nothing above its subnormals.
//
// One CTA per (stretch of packed tokens, KV head, K or V) serves the runs that
// start in its stretch.  HBM bounds long prompts: every value is read once and
// stays in registers between the maximum and the rounding, a thread's 16 pieces of
// 16 bytes all in flight at once.  (With 8 pieces and twice the threads the cost of finding
// and closing a run, some 700 instructions a warp, took more issue slots than the
// data: 88 us against 77 us for 65k tokens of 8 heads, d = 128; with the values fetched into
// L2 early 70 us, 5.9 TB/s.)

// quantise8 for a scale that is no power of two, by division.  Out of line: eight divisions at every use
// had the quantising write wait for instructions.
__device__ __noinline__ uint2 quantise8_divide(uint4 w, float s) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  uint32_t c[4];
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = i == 0 ? x[0] : i == 1 ? x[1] : i == 2 ? x[2] : x[3];
    const uint32_t q = pack_e4m3x2(__fdiv_rn(__uint_as_float(v << 16), s),
                                   __fdiv_rn(__uint_as_float(v & 0xffff0000u), s));
    if (i == 0) c[0] = q;
    if (i == 1) c[1] = q;
    if (i == 2) c[2] = q;
    if (i == 3) c[3] = q;
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

constexpr int kPieces = 16;  // 16-byte pieces a thread holds of a full page

template <int D, int PS>
struct WriteTile {
  static constexpr int kCols = D / 8;  // 16-byte pieces of a row
  static constexpr int kThreads = PS * kCols / kPieces < 32 ? 32 : PS * kCols / kPieces;
  static constexpr int kRows = kThreads / kCols;  // rows of one pass
  static constexpr int kPasses = PS / kRows;
  static constexpr int kWarps = kThreads / 32;
};

template <int D, int PS>
__global__ void __launch_bounds__(WriteTile<D, PS>::kThreads, 640 / WriteTile<D, PS>::kThreads)
    fa_kv_write_kernel(const KvWriteParams p, int stretch) {
  using T = WriteTile<D, PS>;
  __shared__ uint32_t s_max[2][T::kWarps];
  __shared__ __half2 s_hi[T::kWarps][D / 2], s_lo[T::kWarps][D / 2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the heads of one stretch are neighbours in the grid: token-major inputs hold
  // them side by side
  const int part = blockIdx.x % (2 * p.s.Hkv);
  const int h = part % p.s.Hkv;
  const bool is_v = part >= p.s.Hkv;
  const long long st_h = is_v ? p.v_stride_h : p.k_stride_h;
  const long long st_t = is_v ? p.v_stride_t : p.k_stride_t;
  const int col = tid % T::kCols, row0 = tid / T::kCols;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? p.v : p.k) + h * st_h + col * 8;
  uint8_t* cache = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache);
  float* scales = is_v ? p.v_scale : p.k_scale;
  int8_t* bounds = is_v ? nullptr : p.k_bounds;
  const long long n_slots = static_cast<long long>(p.s.num_pages) * PS;
  const int t_lo = blockIdx.x / (2 * p.s.Hkv) * stretch;
  const int t_hi = min(t_lo + stretch, p.n_tokens);
  int turn = 0;
  griddep_wait();

  // Every warp reads the slots of the stretch and of a page's length behind it at
  // once and marks the tokens that follow their predecessor in its page; runs are
  // then found without another load.
  constexpr int kWords = PS / 16;       // 2 * PS tokens in words of 32
  uint32_t follows = 0, begins = 0;     // lane w: masks of word w
  {
    long long slots[kWords];
    long long before = t_lo > 0 ? p.slot_map[t_lo - 1] : -1;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const int t = t_lo + 32 * w + lane;
      slots[w] = t < p.n_tokens ? p.slot_map[t] : -1;
    }
    // Which values the stretch reads does not depend on the slots: they come to L2 while
    // the slots come to the registers (70 us against 76 us; stretches of one to four
    // tokens gain nothing, and fetching those of the CTA 400 or 1520 further on takes 74
    // or 75 us).
    if (stretch >= 8) {
      constexpr int kLines = D / 64;
      for (int i = tid; i < (t_hi - t_lo) * kLines; i += T::kThreads) {
        const __nv_bfloat16* line = src - col * 8 + (t_lo + i / kLines) * st_t + i % kLines * 64;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(line));
      }
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      long long prev = __shfl_up_sync(0xffffffffu, slots[w], 1);
      if (lane == 0) prev = before;
      before = __shfl_sync(0xffffffffu, slots[w], 31);
      const bool in_run = slots[w] > 0 && slots[w] == prev + 1 && (slots[w] & (PS - 1)) != 0;
      const bool first = !in_run && slots[w] >= 0 && slots[w] < n_slots && t_lo + 32 * w + lane < t_hi;
      const uint32_t m = __ballot_sync(0xffffffffu, in_run), n = __ballot_sync(0xffffffffu, first);
      if (lane == w) follows = m, begins = n;
    }
  }
#pragma unroll 1
  for (int w = 0; w < (PS + 31) / 32; ++w) {
#pragma unroll 1
    for (uint32_t todo = __shfl_sync(0xffffffffu, begins, w); todo; todo &= todo - 1) {
      const int at = __ffs(todo) - 1;
      const int t = t_lo + 32 * w + at;
      const long long first = p.slot_map[t];
      const int page = static_cast<int>(first / PS), off = static_cast<int>(first & (PS - 1));
      const size_t tile = static_cast<size_t>(page) * p.s.Hkv + h;
      float s_old = off > 0 ? scales[tile] : 0.f;
      int len = 1;  // up to the first token that does not follow
      for (int u = 32 * w + at + 1; u < 32 * kWords; u = (u | 31) + 1) {
        const uint32_t stop = ~__shfl_sync(0xffffffffu, follows, u >> 5) >> (u & 31);
        len += stop ? __ffs(stop) - 1 : 32 - (u & 31);
        // (the zeros shifted in count as "follows": a set bit below them, or the word's end)
        if (stop) break;
      }
      len = min(len, PS - off);
      uint4 x[T::kPasses];
      const __nv_bfloat16* from = src + (t + row0) * st_t;
#pragma unroll
      for (int i = 0; i < T::kPasses; ++i) {
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row0 + i * T::kRows < len) x[i] = ld_stream16(from);
        from += T::kRows * st_t;
      }
      uint32_t m = 0;  // largest magnitude of the even and odd values, as bf16 bits
#pragma unroll
      for (int i = 0; i < T::kPasses; ++i)
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                 __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
      // infinities or NaN somewhere in the warp
      const bool odd_values = __any_sync(0xffffffffu, max(m & 0xffffu, m >> 16) >= 0x7f80u);
      if (odd_values) {
        m = 0;
#pragma unroll
        for (int i = 0; i < T::kPasses; ++i) m = __vmaxu2(m, max_finite_bf16x2(x[i]));
      }
      const uint32_t top = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
      if (lane == 0) s_max[turn][warp] = top;
      // all reads of the page's old scale and bounds come before this barrier,
      // all writes after it
      if (!(s_old > 0.f && s_old <= 3.4028235e38f)) s_old = 0.f;
      __half2 old_hi, old_lo;
      if (bounds && off > 0 && tid < D / 2) {
        const char2 a = reinterpret_cast<const char2*>(bounds + tile * 2 * D)[tid];
        const char2 b = reinterpret_cast<const char2*>(bounds + tile * 2 * D + D)[tid];
        old_hi = __floats2half2_rn(a.x, a.y);
        old_lo = __floats2half2_rn(b.x, b.y);
      }
      __syncthreads();
      uint32_t amax = 0;
#pragma unroll
      for (int w = 0; w < T::kWarps; ++w) amax = max(amax, s_max[turn][w]);
      turn ^= 1;
      const float s = fmaxf(s_old, block_scale(amax));
      const float ratio = off > 0 ? s_old / s : 0.f;
      uint8_t* dst = cache + tile * PS * D;
      if (off > 0 && s > s_old) {
        for (int i = tid; i < off * T::kCols; i += T::kThreads) {
          uint2* w = reinterpret_cast<uint2*>(dst) + i;
          *w = rescale_codes(*w, ratio);
        }
      }
      const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0;
      const float inv = 1.f / s;
      __half2 hi[4], lo[4];
      uint2* to = reinterpret_cast<uint2*>(dst) + (off + row0) * T::kCols + col;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        hi[e] = __float2half2_rn(-65504.f);
        lo[e] = __float2half2_rn(65504.f);
      }
#pragma unroll
      for (int i = 0; i < T::kPasses; ++i) {
        const int r = row0 + i * T::kRows;
        if (r < len) {
          uint2 c = pow2 ? quantise8(x[i], inv) : quantise8_divide(x[i], s);
          to[i * T::kRows * T::kCols] = c;
          if (bounds) {
            if (odd_values) c = zero_nan_codes(c);
            const uint32_t w[4] = {c.x, c.x >> 16, c.y, c.y >> 16};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t v = e4m3x2_to_f16x2(w[e]);
              hi[e] = __hmax2(hi[e], *reinterpret_cast<const __half2*>(&v));
              lo[e] = __hmin2(lo[e], *reinterpret_cast<const __half2*>(&v));
            }
          }
        }
      }
      if (tid == 0) scales[tile] = s;
      if (bounds) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
          for (int o = T::kCols; o < 32; o <<= 1) {
            hi[e] = __hmax2(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
            lo[e] = __hmin2(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
          }
          if (lane < T::kCols) {
            s_hi[warp][col * 4 + e] = hi[e];
            s_lo[warp][col * 4 + e] = lo[e];
          }
        }
        __syncthreads();
        for (int c = tid; c < D / 2; c += T::kThreads) {
          __half2 a = s_hi[0][c], z = s_lo[0][c];
#pragma unroll
          for (int w = 1; w < T::kWarps; ++w) {
            a = __hmax2(a, s_hi[w][c]);
            z = __hmin2(z, s_lo[w][c]);
          }
          float2 f = __half22float2(a), g = __half22float2(z);
          f = make_float2(ceilf(f.x * 0.25f), ceilf(f.y * 0.25f));
          g = make_float2(floorf(g.x * 0.25f), floorf(g.y * 0.25f));
          if (off > 0) {
            if (c != tid) {  // fewer threads than channel pairs
              const char2 u = reinterpret_cast<const char2*>(bounds + tile * 2 * D)[c];
              const char2 v = reinterpret_cast<const char2*>(bounds + tile * 2 * D + D)[c];
              old_hi = __floats2half2_rn(u.x, u.y);
              old_lo = __floats2half2_rn(v.x, v.y);
            }
            const float2 u = __half22float2(old_hi), v = __half22float2(old_lo);
            const float by = fmaxf(ratio, 1.1754944e-38f);  // a ratio of 0 would round inwards
            f = make_float2(fmaxf(f.x, ceilf(u.x * by)), fmaxf(f.y, ceilf(u.y * by)));
            g = make_float2(fminf(g.x, floorf(v.x * by)), fminf(g.y, floorf(v.y * by)));
            // A ratio that is no power of two rounds codes, some away from zero.  Rounding keeps
            // their order, so the bound rounded like a code encloses them.
            if ((__float_as_uint(ratio) & 0x7fffffu) != 0) {
              const float2 a = e4m3x2_to_f32x2(pack_e4m3x2(4.f * u.x * ratio, 4.f * u.y * ratio));
              const float2 b = e4m3x2_to_f32x2(pack_e4m3x2(4.f * v.x * ratio, 4.f * v.y * ratio));
              f = make_float2(fmaxf(f.x, ceilf(a.x * 0.25f)), fmaxf(f.y, ceilf(a.y * 0.25f)));
              g = make_float2(fminf(g.x, floorf(b.x * 0.25f)), fminf(g.y, floorf(b.y * 0.25f)));
            }
          }
          reinterpret_cast<char2*>(bounds + tile * 2 * D)[c] =
              make_char2(static_cast<signed char>(f.x), static_cast<signed char>(f.y));
          reinterpret_cast<char2*>(bounds + tile * 2 * D + D)[c] =
              make_char2(static_cast<signed char>(g.x), static_cast<signed char>(g.y));
        }
      }
    }
  }
}

// ------------------------------------------------------------------- read --
//
// Packed row r of KV head h is code * scale of the sequence's token, rounded to
// bf16 (exact for power-of-two scales: e4m3 has 4 significant bits).  HBM bounds
// it (1 byte read, 2 written per element).  A CTA takes 64 packed rows: one thread a row
// finds its sequence, page and scale, once; then a thread turns 8 codes into 16 bytes, so
// that a warp's stores are whole 512-byte pieces, with four rows' loads in flight.  (With
// every thread finding its own rows the lookups took 82% of the issue slots.)
constexpr int kReadThreads = 256;
constexpr int kReadRows = 64;

template <int D>
__global__ void __launch_bounds__(kReadThreads) fa_kv_read_kernel(const KvReadParams p) {
  constexpr int CPR = D / 8;
  constexpr int ROWS = kReadThreads / CPR;  // rows of one pass
  constexpr int PASSES = kReadRows / ROWS;
  // a row's first code, -1: zeros, -2: the row stays as it was
  __shared__ long long s_from[kReadRows];
  __shared__ float s_scale[kReadRows];
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const long long r0 = static_cast<long long>(blockIdx.x) * kReadRows;
  griddep_wait();
  if (threadIdx.x < kReadRows) {
    const long long r = r0 + threadIdx.x;
    const int ps = p.s.page_size, shift = 31 - __clz(ps);
    int a = 0;  // last sequence with cu_k <= r
    for (int z = p.nseq; z - a > 1;) {
      const int mid = (a + z) >> 1;
      if (p.cu_k[mid] <= r) a = mid; else z = mid;
    }
    const long long pos = r - p.cu_k[a];
    long long from = -2;
    float scale = 0.f;
    if (r < p.total_k && pos >= 0 && r < p.cu_k[a + 1]) {
      from = -1;
      if ((pos >> shift) < p.max_blocks) {
        const int page = p.block_table[static_cast<long long>(a) * p.max_blocks + (pos >> shift)];
        if (page >= 0 && page < p.s.num_pages) {
          const long long tile = static_cast<long long>(page) * p.s.Hkv + h;
          from = (tile * ps + (pos & (ps - 1))) * D;
          scale = (is_v ? p.v_scale : p.k_scale)[tile];
        }
      }
    }
    s_from[threadIdx.x] = from;
    s_scale[threadIdx.x] = scale;
  }
  __syncthreads();
  const int col = threadIdx.x % CPR, row = threadIdx.x / CPR;
  const uint8_t* cache = static_cast<const uint8_t*>(is_v ? p.v_cache : p.k_cache) + col * 8;
  uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? p.v : p.k) +
                                        (static_cast<size_t>(h) * p.total_k + r0) * D) + threadIdx.x;
  uint2 w[PASSES];
  long long from[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    from[i] = s_from[row + i * ROWS];
    w[i] = make_uint2(0u, 0u);
    if (from[i] >= 0) w[i] = ld_stream8(cache + from[i]);
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i)
    if (from[i] > -2) out[i * kReadThreads] = dequantise8(w[i], s_scale[row + i * ROWS]);
}

}  // namespace

cudaError_t launch_kv_assign(const KvAssignParams& p, cudaStream_t stream) {
  const int grid = max(1, (p.total_new + kAssignTokens - 1) / kAssignTokens);
  return launch_dependent(fa_kv_assign_kernel, dim3(grid), dim3(kAssignThreads), 0, stream, p);
}

namespace {

template <int D, int PS>
cudaError_t launch_write(const KvWriteParams& p, cudaStream_t stream) {
  // A stretch of a page's length has about one run in it when prompts come in;
  // single tokens are a run each, so few tokens are spread over more CTAs: the
  // longest stretch that still leaves some 16 CTAs for each of 152 SMs.
  const long long work = 2LL * p.n_tokens * p.s.Hkv;
  int stretch = 1;
  while (stretch < PS && work / (2 * stretch) >= 152 * 16) stretch *= 2;
  const dim3 grid(static_cast<unsigned int>((p.n_tokens + stretch - 1LL) / stretch * 2 * p.s.Hkv));
  return launch_dependent(fa_kv_write_kernel<D, PS>, grid, dim3(WriteTile<D, PS>::kThreads), 0,
                          stream, p, stretch);
}

template <int D>
cudaError_t launch_write_d(const KvWriteParams& p, cudaStream_t stream) {
  switch (p.s.page_size) {
    case 16: return launch_write<D, 16>(p, stream);
    case 32: return launch_write<D, 32>(p, stream);
    case 64: return launch_write<D, 64>(p, stream);
    default: return launch_write<D, 128>(p, stream);
  }
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteParams& p, cudaStream_t stream) {
  return p.s.d == 128 ? launch_write_d<128>(p, stream) : launch_write_d<64>(p, stream);
}

cudaError_t launch_kv_read(const KvReadParams& p, cudaStream_t stream) {
  const dim3 grid((p.total_k + kReadRows - 1) / kReadRows, p.s.Hkv, 2);
  return launch_dependent(p.s.d == 128 ? fa_kv_read_kernel<128> : fa_kv_read_kernel<64>, grid,
                          dim3(kReadThreads), 0, stream, p);
}

}  // namespace fa
