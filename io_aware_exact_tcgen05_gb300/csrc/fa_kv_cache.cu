// fa_kv_cache.cu -- the paged 8-bit KV cache: block tables and slot maps from
// request lengths (fa_kv_assign), the quantising write (fa_kv_write_fp8) and
// the dequantising read (fa_kv_read_fp8).
#include <cuda_runtime.h>
#include <cuda_bf16.h>

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
constexpr int kAssignTokens = 2048;  // packed tokens per CTA

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
  const long long t_lo = static_cast<long long>(blockIdx.x) * kAssignTokens;
  const long long t_hi = min(t_lo + kAssignTokens, static_cast<long long>(p.total_new));
  const bool first_cta = blockIdx.x == 0;
  long long cu0 = 0, need0 = 0, k0 = 0;  // totals of the requests before this chunk
  if (tid == 0) s_used = 0;
  for (int base = 0; base < p.B; base += kAssignThreads) {
    const int b = base + tid;
    const bool real = b < p.B;
    const long long seq = real ? max(p.seqlens[b], 0) : 0;
    const long long add = real ? max(p.newlens[b], 0) : 0;
    long long sum_new, sum_need;
    const long long cu_end = cu0 + block_scan_inclusive(add, s_sums, &sum_new);
    const long long have = (seq + p.page_size - 1) / p.page_size;
    const long long full = (seq + add + p.page_size - 1) / p.page_size;
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
        const long long pos = s_seq[a] + (t - s_cu[a]);
        const int blk = static_cast<int>(pos / p.page_size);
        const int off = static_cast<int>(pos % p.page_size);
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
// One CTA per (stretch of kWriteChunk packed tokens, KV head, K or V) serves the
// runs that start in its stretch.  A run is the new tokens of one page: with
// n tokens in the page before it,
//   s_tok = 2^e, e the smallest with amax(new) <= 448 * 2^e (finite values),
//   s = max(s_old, s_tok) if n > 0, else s_tok,
//   new code = rn_sat(x / s), held code = rn(code * s_old / s).
// With power-of-two scales both are exact but for e4m3's own rounding, so a
// page that is requantised loses nothing above its subnormals.
// The run's values stay in registers between the maximum and the rounding:
// each is read once.
constexpr int kWriteThreads = 128;

template <int D>
__global__ void __launch_bounds__(kWriteThreads) fa_kv_write_kernel(const KvWriteParams p,
                                                                    int chunk) {
  constexpr int CPR = D / 8;                   // 16-byte chunks per row
  constexpr int RPP = kWriteThreads / CPR;     // rows per pass
  constexpr int PASSES = 128 / RPP;            // a run has at most 128 rows
  __shared__ int s_len, s_max;
  __shared__ int s_hi[D], s_lo[D];
  const int tid = threadIdx.x, ps = p.s.page_size;
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? p.v : p.k);
  const long long st_h = is_v ? p.v_stride_h : p.k_stride_h;
  const long long st_t = is_v ? p.v_stride_t : p.k_stride_t;
  uint8_t* cache = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache);
  float* scales = is_v ? p.v_scale : p.k_scale;
  int8_t* bounds = is_v ? nullptr : p.k_bounds;
  const long long n_slots = static_cast<long long>(p.s.num_pages) * ps;
  const int t0 = blockIdx.x * chunk;
  const int t1 = min(t0 + chunk, p.n_tokens);
  const int col = tid % CPR, row0 = tid / CPR;

  for (int t = t0; t < t1; ++t) {
    const long long slot = p.slot_map[t];
    if (slot < 0 || slot >= n_slots) continue;  // uniform over the CTA
    const int off = static_cast<int>(slot % ps);
    if (t > 0 && off > 0 && p.slot_map[t - 1] == slot - 1) continue;  // inside a run
    const int page = static_cast<int>(slot / ps);
    const int most = min(ps - off, p.n_tokens - t);
    __syncthreads();
    if (tid == 0) {
      s_len = most;
      s_max = 0;
    }
    for (int c = tid; c < D; c += kWriteThreads) {
      s_hi[c] = -128;
      s_lo[c] = 127;
    }
    __syncthreads();
    if (tid > 0 && tid < most && p.slot_map[t + tid] != slot + tid) atomicMin(&s_len, tid);
    const size_t tile = (static_cast<size_t>(page) * p.s.Hkv + h);
    float s_old = off > 0 ? scales[tile] : 0.f;
    if (!(s_old > 0.f && s_old <= 3.4028235e38f)) s_old = 0.f;
    __syncthreads();
    const int len = s_len;
    uint4 x[PASSES];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = row0 + i * RPP;
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < len) {
        x[i] = *reinterpret_cast<const uint4*>(src + h * st_h + (t + r) * st_t + col * 8);
        m = __vmaxu2(m, max_finite_bf16x2(x[i]));
      }
    }
    const int mine = max(m & 0xffffu, m >> 16);
    const int top = __reduce_max_sync(0xffffffffu, mine);
    if ((tid & 31) == 0) atomicMax(&s_max, top);
    __syncthreads();
    const float s_tok = block_scale(static_cast<uint32_t>(s_max));
    const float s = fmaxf(s_old, s_tok);
    uint8_t* dst = cache + tile * ps * D;
    const bool grown = off > 0 && s > s_old;
    const float ratio = off > 0 ? s_old / s : 0.f;
    if (grown) {
      for (int i = tid; i < off * CPR; i += kWriteThreads) {
        uint2* w = reinterpret_cast<uint2*>(dst) + i;
        *w = rescale_codes(*w, ratio);
      }
    }
    const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0;
    const float inv = 1.f / s;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = row0 + i * RPP;
      if (r < len) {
        const uint2 c = quantise8(x[i], s, inv, pow2);
        reinterpret_cast<uint2*>(dst)[(off + r) * CPR + col] = c;
        if (bounds) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float v = code_value((e < 4 ? c.x : c.y) >> (8 * (e & 3)) & 0xffu);
            atomicMax(&s_hi[col * 8 + e], static_cast<int>(ceilf(v * 0.25f)));
            atomicMin(&s_lo[col * 8 + e], static_cast<int>(floorf(v * 0.25f)));
          }
        }
      }
    }
    __syncthreads();
    if (tid == 0) scales[tile] = s;
    if (bounds) {
      int8_t* bd = bounds + tile * 2 * D;
      for (int c = tid; c < D; c += kWriteThreads) {
        int hi = s_hi[c], lo = s_lo[c];
        if (off > 0) {
          hi = max(hi, static_cast<int>(ceilf(bd[c] * ratio)));
          lo = min(lo, static_cast<int>(floorf(bd[D + c] * ratio)));
        }
        bd[c] = static_cast<int8_t>(hi);
        bd[D + c] = static_cast<int8_t>(lo);
      }
    }
  }
}

// ------------------------------------------------------------------- read --
//
// Packed row r of KV head h is code * scale of the sequence's token, rounded to
// bf16 (exact for power-of-two scales: e4m3 has 4 significant bits).  One
// thread turns 16 codes into 32 bytes.
constexpr int kReadThreads = 256;

template <int D>
__global__ void __launch_bounds__(kReadThreads) fa_kv_read_kernel(const KvReadParams p) {
  constexpr int CPR = D / 16;
  constexpr int ROWS = kReadThreads / CPR;
  const int col = threadIdx.x % CPR;
  const long long r = static_cast<long long>(blockIdx.x) * ROWS + threadIdx.x / CPR;
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  if (r >= p.total_k) return;
  // last sequence with cu_k <= r; behind the last one the row stays as it was
  int a = 0, z = p.nseq;
  while (z - a > 1) {
    const int mid = (a + z) >> 1;
    if (p.cu_k[mid] <= r) a = mid; else z = mid;
  }
  const long long first = p.cu_k[a];
  if (r < first || r >= p.cu_k[a + 1]) return;
  const long long pos = r - first;
  const int ps = p.s.page_size;
  const long long blk = pos / ps;
  int page = -1;
  if (blk < p.max_blocks) page = p.block_table[static_cast<long long>(a) * p.max_blocks + blk];
  uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
  if (page >= 0 && page < p.s.num_pages) {
    const size_t tile = static_cast<size_t>(page) * p.s.Hkv + h;
    const float s = (is_v ? p.v_scale : p.k_scale)[tile];
    const uint8_t* c = static_cast<const uint8_t*>(is_v ? p.v_cache : p.k_cache) +
                       (tile * ps + static_cast<int>(pos % ps)) * D + col * 16;
    const uint4 w = *reinterpret_cast<const uint4*>(c);
    lo = dequantise8(make_uint2(w.x, w.y), s);
    hi = dequantise8(make_uint2(w.z, w.w), s);
  }
  uint4* out = reinterpret_cast<uint4*>(
      static_cast<__nv_bfloat16*>(is_v ? p.v : p.k) +
      (static_cast<size_t>(h) * p.total_k + r) * D + col * 16);
  out[0] = lo;
  out[1] = hi;
}

}  // namespace

cudaError_t launch_kv_assign(const KvAssignParams& p, cudaStream_t stream) {
  const int grid = max(1, (p.total_new + kAssignTokens - 1) / kAssignTokens);
  fa_kv_assign_kernel<<<grid, kAssignThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv_write(const KvWriteParams& p, cudaStream_t stream) {
  const int chunk = p.n_tokens <= 1024 ? 1 : 16;
  const dim3 grid((p.n_tokens + chunk - 1) / chunk, p.s.Hkv, 2);
  if (p.s.d == 128) fa_kv_write_kernel<128><<<grid, kWriteThreads, 0, stream>>>(p, chunk);
  else fa_kv_write_kernel<64><<<grid, kWriteThreads, 0, stream>>>(p, chunk);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvReadParams& p, cudaStream_t stream) {
  const int rows = kReadThreads / (p.s.d / 16);
  const dim3 grid((p.total_k + rows - 1) / rows, p.s.Hkv, 2);
  if (p.s.d == 128) fa_kv_read_kernel<128><<<grid, kReadThreads, 0, stream>>>(p);
  else fa_kv_read_kernel<64><<<grid, kReadThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
