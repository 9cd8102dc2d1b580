// fa_prep.cu -- from a projection's rows [token][head][channel] to what the scores are taken of:
// norms of queries and keys for each head, the position rotation, head-major tensors (or rows of
// a padded cache); and the way back for the gradients.  One pass over the data each.
//
//   u = x * r * (w + w_off), r = 1 / sqrt(mean(x^2) + eps)      (no weight: u = x)
//   y = u with its pairs (a, b) of frequency i turned:  (a c - b s, b c + a s)
//   c, s = cos, sin of position[axis_i] * inv_freq_i
// Backward, g = dy turned back:
//   dw = sum g x r;   a = g (w + w_off);   dx = r (a - x r mean(a x r))
//
// Bound by HBM: every element is read and written once (the backward reads x as well), some ten
// operations each.  D / 16 lanes share a head's vector, 16 channels a lane: two 16-byte pieces
// that hold both members of the lane's pairs, so a rotation needs no exchange; the norm is one
// reduction over the lanes.  A warp takes 32 * 16 / D heads at once and walks the heads of a token,
// for which it takes the angles once.
//
// Angles: a position times a frequency in turns, as 64-bit fixed point, of which whole turns
// fall off by themselves: exact to 2^-31 turns for any 32-bit position, without 64-bit floating
// point.  Sine and cosine of the remainder (within half a turn) are the fast ones, off by 2^-20.5 at
// most, a 2000th of what the rounding of y to bf16 may do.
//
// Sums over a head and the weights' gradients are held in fp32; a CTA adds its share of dw in a
// fixed order and a second kernel adds the CTAs' likewise: same result every time.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_prep.h"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPrepCtasPerSm = 3;
constexpr int kMaxPartialRows = 512;

// f / (2 pi) turns as a 64-bit fixed-point fraction (whole turns dropped); 1 / (2 pi) in 64 bits.
__device__ __forceinline__ uint64_t turns64(float f) {
  constexpr uint64_t kInvTwoPi = 0x28BE60DB9391054Aull;  // floor(2^64 / (2 pi))
  const uint32_t bits = __float_as_uint(f);
  const int ex = static_cast<int>((bits >> 23) & 255);
  const uint64_t mant = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int sh = (ex ? ex : 1) - 150;  // f = mant * 2^sh
  const uint64_t lo = mant * kInvTwoPi, hi = __umul64hi(mant, kInvTwoPi);
  uint64_t t;
  if (sh >= 0) t = sh < 64 ? lo << sh : 0;
  else if (sh > -64) t = (lo >> -sh) | (hi << (64 + sh));
  else t = sh > -128 ? hi >> (-sh - 64) : 0;
  return (bits >> 31) ? 0 - t : t;
}

// cos and sin of pos * t turns.
__device__ __forceinline__ void turn(uint64_t t, int pos, float& c, float& s) {
  const uint32_t lo = static_cast<uint32_t>(t), hi = static_cast<uint32_t>(t >> 32);
  const uint32_t q = static_cast<uint32_t>(pos);
  const uint32_t f = hi * q + __umulhi(lo, q) - (pos < 0 ? lo : 0u);  // bits 32..63 of t * pos
  const float x = static_cast<float>(static_cast<int>(f)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  __sincosf(x, &s, &c);
}

struct Vec {
  float a[8], b[8];
};

__device__ __forceinline__ void unpack8(const uint4 w, float (&v)[8]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(x[e] << 16);
    v[2 * e + 1] = __uint_as_float(x[e] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) {
  return __ldcs(reinterpret_cast<const uint4*>(p));
}

__device__ __forceinline__ void store16(__nv_bfloat16* p, const uint4 v) {
  *reinterpret_cast<uint4*>(p) = v;
}

// The lane's pairs turned by (c, s) (back: by -s): channels 2 i and 2 i + 1 of a piece, or the same
// channel of both pieces.
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float na = fmaf(a, c, -b * s);
  b = fmaf(b, c, a * s);
  a = na;
}

__device__ __forceinline__ void rotate(Vec& v, const float (&c)[8], const float (&s)[8],
                                       bool interleaved, bool back) {
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      turn_pair(v.a[2 * e], v.a[2 * e + 1], c[e], back ? -s[e] : s[e]);
      turn_pair(v.b[2 * e], v.b[2 * e + 1], c[4 + e], back ? -s[4 + e] : s[4 + e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) turn_pair(v.a[e], v.b[e], c[e], back ? -s[e] : s[e]);
  }
}

template <int LPH>
__device__ __forceinline__ float sum_head(float v) {
#pragma unroll
  for (int o = LPH / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int D, bool BACK>
__global__ void __launch_bounds__(kThreads, BACK ? 2 : kPrepCtasPerSm)
    fa_prep_kernel(const PrepParams p) {
  constexpr int LPH = D / 16;    // lanes per head
  constexpr int HPW = 32 / LPH;  // heads per warp and step
  __shared__ float dw_red[BACK ? kWarps : 1][BACK ? D : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int blk = blockIdx.x, ri = 0;
  while (ri < 2 && blk >= p.role[ri].blocks) blk -= p.role[ri++].blocks;
  const PrepRole& r = p.role[ri];
  const int x = lane % LPH, sub = lane / LPH;
  // the lane's two pieces of 8 channels
  const int rot_lanes = r.rotated ? p.rot / 16 : 0;
  const bool turns = x < rot_lanes;
  const int ca = turns ? 8 * x : 16 * x;
  const int cb = turns ? p.rot / 2 + 8 * x : 16 * x + 8;
  uint64_t t64[8];
  int axis[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    t64[e] = 0;
    axis[e] = 0;
    if (turns) {
      const int i = p.interleaved ? (e < 4 ? 4 * x + e : p.rot / 4 + 4 * x + e - 4) : 8 * x + e;
      axis[e] = p.freq_axis ? p.freq_axis[i] : 0;
      if (axis[e] < p.n_axes) t64[e] = turns64(p.inv_freq[i]);
      else axis[e] = 0;
    }
  }
  Vec w;
  const __nv_bfloat16* wp = static_cast<const __nv_bfloat16*>(r.w);
  if (wp) {
    unpack8(*reinterpret_cast<const uint4*>(wp + ca), w.a);
    unpack8(*reinterpret_cast<const uint4*>(wp + cb), w.b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w.a[e] += p.w_off;
      w.b[e] += p.w_off;
    }
  }
  Vec dw;
#pragma unroll
  for (int e = 0; e < 8; ++e) dw.a[e] = dw.b[e] = 0.f;
  const int n_steps = (r.heads + HPW - 1) / HPW;
  const int per_part = (n_steps + p.parts - 1) / p.parts;
  const long long items = static_cast<long long>(p.B) * p.S * p.parts;
  for (long long it = static_cast<long long>(blk) * kWarps + warp; it < items;
       it += static_cast<long long>(r.blocks) * kWarps) {
    const int part = static_cast<int>(it % p.parts);
    const long long token = it / p.parts;
    const int b = static_cast<int>(token / p.S);
    const int s = static_cast<int>(token - static_cast<long long>(b) * p.S);
    const int start = p.row_start ? p.row_start[b] : 0;
    const int row = ri == 0 ? s : start + s;
    float c[8], sn[8];
    if (turns) {
      if (p.positions && p.n_axes > 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          turn(t64[e], __ldg(p.positions + axis[e] * static_cast<long long>(p.B) * p.S + token),
               c[e], sn[e]);
      } else {
        const int pos = p.positions ? __ldg(p.positions + token) : start + s;
#pragma unroll
        for (int e = 0; e < 8; ++e) turn(t64[e], pos, c[e], sn[e]);
      }
    }
    if (row < 0 || row >= r.y_rows) continue;  // warp-uniform: no room in the cache
    const __nv_bfloat16* xt = static_cast<const __nv_bfloat16*>(r.x) + b * r.xb + s * r.xt;
    __nv_bfloat16* yt = static_cast<__nv_bfloat16*>(r.y) +
                        (static_cast<long long>(b) * r.heads * r.y_rows + row) * D;
    const int step1 = min(n_steps, (part + 1) * per_part);
#pragma unroll 2
    for (int st = part * per_part; st < step1; ++st) {
      const int h = st * HPW + sub;
      const bool live = h < r.heads;
      Vec v, g;
      uint4 va = make_uint4(0u, 0u, 0u, 0u), vb = va, ga = va, gb = va;
      __nv_bfloat16* yh = yt + static_cast<long long>(h) * r.y_rows * D;
      if (live) {
        if (!BACK || wp) {
          va = load16(xt + h * r.xh + ca);
          vb = load16(xt + h * r.xh + cb);
        }
        if (BACK) {
          ga = load16(yh + ca);
          gb = load16(yh + cb);
        }
      }
      if (!wp && !turns) {  // nothing to compute: bits as they are
        if (live) {
          __nv_bfloat16* to = BACK ? static_cast<__nv_bfloat16*>(r.dx) + b * r.db + s * r.dt + h * r.dh
                                   : yh;
          store16(to + ca, BACK ? ga : va);
          store16(to + cb, BACK ? gb : vb);
        }
        continue;
      }
      unpack8(va, v.a);
      unpack8(vb, v.b);
      float rn = 1.f;
      if (wp) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v.a[e], v.a[e], fmaf(v.b[e], v.b[e], ss));
        rn = rsqrtf(sum_head<LPH>(ss) * (1.f / D) + p.eps);
      }
      if (!BACK) {
        if (wp) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v.a[e] *= rn * w.a[e];
            v.b[e] *= rn * w.b[e];
          }
        }
        if (turns) rotate(v, c, sn, p.interleaved, false);
        if (live) {
          store16(yh + ca, pack8(v.a));
          store16(yh + cb, pack8(v.b));
        }
      } else {
        unpack8(ga, g.a);
        unpack8(gb, g.b);
        if (turns) rotate(g, c, sn, p.interleaved, true);
        if (wp) {
          float dot = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v.a[e] *= rn;
            v.b[e] *= rn;
            if (live) {
              dw.a[e] = fmaf(g.a[e], v.a[e], dw.a[e]);
              dw.b[e] = fmaf(g.b[e], v.b[e], dw.b[e]);
            }
            g.a[e] *= w.a[e];
            g.b[e] *= w.b[e];
            dot = fmaf(g.a[e], v.a[e], fmaf(g.b[e], v.b[e], dot));
          }
          dot = sum_head<LPH>(dot) * (1.f / D);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            g.a[e] = rn * fmaf(-dot, v.a[e], g.a[e]);
            g.b[e] = rn * fmaf(-dot, v.b[e], g.b[e]);
          }
        }
        if (live) {
          __nv_bfloat16* to = static_cast<__nv_bfloat16*>(r.dx) + b * r.db + s * r.dt + h * r.dh;
          store16(to + ca, pack8(g.a));
          store16(to + cb, pack8(g.b));
        }
      }
    }
  }
  if constexpr (BACK) {
    if (!r.dw) return;  // CTA-uniform
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = LPH; o < 32; o <<= 1) {
        dw.a[e] += __shfl_xor_sync(0xffffffffu, dw.a[e], o);
        dw.b[e] += __shfl_xor_sync(0xffffffffu, dw.b[e], o);
      }
      if (sub == 0) {
        dw_red[warp][ca + e] = dw.a[e];
        dw_red[warp][cb + e] = dw.b[e];
      }
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float sum = 0.f;
#pragma unroll
      for (int wi = 0; wi < kWarps; ++wi) sum += dw_red[wi][threadIdx.x];
      p.partial[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] = sum;
    }
    griddep_launch_dependents();
  }
}

// dw of queries (CTA 0) and keys (CTA 1) from the CTAs' shares, 8 interleaved sums a channel.
template <int D>
__global__ void __launch_bounds__(8 * D) fa_prep_dw_kernel(const PrepParams p) {
  __shared__ float red[8][D];
  const int ch = threadIdx.x % D, part = threadIdx.x / D;
  const PrepRole& r = p.role[blockIdx.x];
  if (!r.dw) return;
  const int first = blockIdx.x ? p.role[0].blocks : 0;
  griddep_wait();
  float sum = 0.f;
#pragma unroll 4
  for (int k = part; k < r.blocks; k += 8) sum += p.partial[static_cast<size_t>(first + k) * D + ch];
  red[part][ch] = sum;
  __syncthreads();
  if (part == 0) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) t += red[k][ch];
    r.dw[ch] = t;
  }
}

}  // namespace

int prep_partial_rows() { return kMaxPartialRows; }

// CTAs are dealt to queries, keys and values by their heads.  With few tokens several warps share
// a token's heads, as long as there are not enough warps for the device.
void prep_plan(PrepParams* p, int n_sm) {
  const int hpw = 32 / (p->d / 16);
  const long long tokens = static_cast<long long>(p->B) * p->S;
  int heads = 0, most = 0;
  for (const PrepRole& r : p->role) {
    heads += r.heads;
    most = std::max(most, (r.heads + hpw - 1) / hpw);
  }
  const long long want = static_cast<long long>(n_sm) * kWarps;
  p->parts = static_cast<int>(std::min<long long>(most, std::max(1LL, want / std::max(1LL, 3 * tokens))));
  const long long items = tokens * p->parts;
  const int total = std::min(n_sm * kPrepCtasPerSm, kMaxPartialRows - 3);
  for (PrepRole& r : p->role) {
    const long long share = std::max(1LL, static_cast<long long>(total) * r.heads / std::max(1, heads));
    r.blocks = r.heads ? static_cast<int>(std::min(share, (items + kWarps - 1) / kWarps)) : 0;
  }
}

namespace {
int grid_of(const PrepParams& p) { return p.role[0].blocks + p.role[1].blocks + p.role[2].blocks; }
}  // namespace

cudaError_t launch_prep(const PrepParams& p, cudaStream_t stream) {
  if (p.d == 128) fa_prep_kernel<128, false><<<grid_of(p), kThreads, 0, stream>>>(p);
  else fa_prep_kernel<64, false><<<grid_of(p), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_prep_bwd(const PrepParams& p, cudaStream_t stream) {
  if (p.d == 128) fa_prep_kernel<128, true><<<grid_of(p), kThreads, 0, stream>>>(p);
  else fa_prep_kernel<64, true><<<grid_of(p), kThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !(p.role[0].dw || p.role[1].dw)) return e;
  if (p.d == 128) return launch_dependent(fa_prep_dw_kernel<128>, dim3(2), dim3(1024), 0, stream, p);
  return launch_dependent(fa_prep_dw_kernel<64>, dim3(2), dim3(512), 0, stream, p);
}

}  // namespace fa
