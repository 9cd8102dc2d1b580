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
// whose angles its lanes work out together, once, in shared memory.
//
// Angles: a position times a frequency in turns, as 64-bit fixed point, of which whole turns
// fall off by themselves: exact to 2^-31 turns for any 32-bit position and any frequency below 2^24, without
// 64-bit floating point.  The remainder (within half a turn) goes to fp32, 2^-25 and 2^-26 turns for its two roundings;
// its sine and cosine are the fast ones, off by 2^-20.5 at most: 2^-19.9 together, a 2000th of what the rounding
// of y to bf16 may do.
//
// Sums over a head and the weights' gradients are held in fp32; a CTA adds its share of dw in a
// fixed order and a second kernel adds the CTAs' likewise: same result every time.
//
// The work is one line of steps, of a few heads each: a token's queries, keys and values, then the next
// token's; every warp takes an equal stretch of it.  Dealing queries, keys and values to different CTAs
// left two fifths of the time to the slowest; whole tokens left a seventh to the last round.
//
// Measured (GB300, inputs from HBM): 2 x 8192 tokens of 16 + 2 x 16 heads, d = 128 forward 71 us (5.7 TB/s,
// 85% of the measured copy); 3 x 2777 tokens of 28 + 2 x 4 heads with three axes backward 52 us (4.3 TB/s): the
// chain of two reductions a step at 16 warps per SM, which is what the registers allow, with 72 bytes of a thread
// spilled (forward: 64 registers and 44 bytes).  (A token's positions loaded a token ahead, or the sums of dw in
// shared memory, changed nothing.)
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
// CTAs per SM that the registers allow: the grid is one wave of them.
constexpr int kFwdCtasPerSm = 4;
constexpr int kBwdCtasPerSm = 2;
constexpr int kMaxPartialRows = 512;  // most CTAs of a backward pass

// f / (2 pi) turns as a 64-bit fixed-point fraction (whole turns dropped), cut off below 2^-64: 1 / (2 pi) in
// 128 bits, of which a position and a frequency up to 2^24 take 55 away.
__device__ __forceinline__ uint64_t turns64(float f) {
  constexpr uint64_t kHi = 0x28BE60DB9391054Aull, kLo = 0x7F09D5F47D4D3770ull;  // floor(2^128 / (2 pi))
  const uint32_t bits = __float_as_uint(f);
  const int ex = static_cast<int>((bits >> 23) & 255);
  const uint64_t mant = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int sh = (ex ? ex : 1) - 150;  // f = mant * 2^sh
  const uint64_t low = mant * kLo, w0 = mant * kHi, w1 = w0 + __umul64hi(mant, kLo);
  const uint64_t w2 = __umul64hi(mant, kHi) + (w1 < w0);  // mant / (2 pi) = w2 : w1 : low
  uint64_t t;
  if (sh > 0) t = sh < 64 ? (w1 << sh) | (low >> (64 - sh)) : 0;
  else if (sh == 0) t = w1;
  else if (sh > -64) t = (w1 >> -sh) | (w2 << (64 + sh));
  else t = sh > -128 ? w2 >> (-sh - 64) : 0;
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

// 16 channels of a lane as fp32 pairs: two pieces of 8.
struct Vec {
  uint64_t a[4], b[4];
};

__device__ __forceinline__ void unpack8(const uint4 w, uint64_t (&v)[4]) {
  v[0] = bf16x2_to_f2(w.x);
  v[1] = bf16x2_to_f2(w.y);
  v[2] = bf16x2_to_f2(w.z);
  v[3] = bf16x2_to_f2(w.w);
}

__device__ __forceinline__ uint32_t pack2(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return pack_bf16x2(lo, hi);
}

__device__ __forceinline__ uint4 pack8(const uint64_t (&v)[4]) {
  return make_uint4(pack2(v[0]), pack2(v[1]), pack2(v[2]), pack2(v[3]));
}

__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) {
  return __ldcs(reinterpret_cast<const uint4*>(p));
}

__device__ __forceinline__ void store16(__nv_bfloat16* p, const uint4 v) {
  *reinterpret_cast<uint4*>(p) = v;
}

__device__ __forceinline__ uint64_t f2_both(float v) { return f2_pack(v, v); }

// Cosines and sines of a token's frequencies (negative sines turn back), laid out so that the
// lanes of a head read 16 neighbouring bytes each: pairs of pieces 8 frequencies a lane, as two groups
// of four; interleaved as they come (place_of).
template <int D>
struct Angles {
  float c[D / 2], s[D / 2];
};

template <int D>
__device__ __forceinline__ int place_of(int i, bool interleaved) {
  return interleaved ? i : ((i >> 2 & 1) * (D / 16) + (i >> 3)) * 4 + (i & 3);
}

__device__ __forceinline__ void load_pairs(const float* p, uint64_t (&v)[2]) {
  const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(p);
  v[0] = x.x;
  v[1] = x.y;
}

__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The lane's pairs turned: the same channel of both pieces (a + i b times c + i s), or neighbours
// when interleaved.  fa, fb: where the lane's two groups of four are.
template <int D>
__device__ __forceinline__ void rotate(Vec& v, const Angles<D>& g, int fa, int fb, bool interleaved) {
  if (interleaved) {
    const float4 ca = *reinterpret_cast<const float4*>(g.c + fa);
    const float4 sa = *reinterpret_cast<const float4*>(g.s + fa);
    const float4 cb = *reinterpret_cast<const float4*>(g.c + fb);
    const float4 sb = *reinterpret_cast<const float4*>(g.s + fb);
    const float c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
    const float s[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint64_t& x = e < 4 ? v.a[e & 3] : v.b[e & 3];
      float lo, hi;
      f2_unpack(x, lo, hi);
      x = f2_fma(x, f2_both(c[e]), f2_mul(f2_pack(hi, lo), f2_pack(-s[e], s[e])));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      uint64_t c[2], s[2];
      load_pairs(g.c + (e ? fb : fa), c);
      load_pairs(g.s + (e ? fb : fa), s);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint64_t x = v.a[e + i], y = v.b[e + i];
        v.a[e + i] = f2_sub(f2_mul(x, c[i]), f2_mul(y, s[i]));
        v.b[e + i] = f2_fma(y, c[i], f2_mul(x, s[i]));
      }
    }
  }
}

template <int LPH>
__device__ __forceinline__ float sum_head(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  float t = lo + hi;
#pragma unroll
  for (int o = LPH / 2; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

// What the lanes of a warp need of a token besides the data.
template <int D>
struct Lane {
  const Angles<D>* angles;
  const float* weight;  // the lane's channels, with the offset: four groups of four, D / 4 apart
  int ca, cb, f_a, f_b;
  bool turns;           // the lane's channels turn
};

// One head vector's share of a lane, forward: norm and rotation.
template <int D>
__device__ __forceinline__ void forward_vec(Vec& v, const PrepParams& p, const Lane<D>& t, bool norm,
                                            bool turns) {
  if (norm) {
    uint64_t ss = f2_mul(v.a[0], v.a[0]);
    ss = f2_fma(v.b[0], v.b[0], ss);
#pragma unroll
    for (int e = 1; e < 4; ++e) ss = f2_fma(v.a[e], v.a[e], f2_fma(v.b[e], v.b[e], ss));
    const uint64_t rn2 = f2_both(rsqrtf(sum_head<D / 16>(ss) * (1.f / D) + p.eps));
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      uint64_t wa[2], wb[2];
      load_pairs(t.weight + e / 2 * (D / 4), wa);
      load_pairs(t.weight + (2 + e / 2) * (D / 4), wb);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v.a[e + i] = f2_mul(v.a[e + i], f2_mul(rn2, wa[i]));
        v.b[e + i] = f2_mul(v.b[e + i], f2_mul(rn2, wb[i]));
      }
    }
  }
  if (turns) rotate<D>(v, *t.angles, t.f_a, t.f_b, p.interleaved);
}

// The same backward: g becomes the gradient of v, dw gathers the weight's.  A lane without a head
// holds zeros (live false), of which eps = 0 would make NaN.
template <int D>
__device__ __forceinline__ void backward_vec(Vec& v, Vec& g, Vec& dw, const PrepParams& p,
                                             const Lane<D>& t, bool norm, bool turns, bool live) {
  if (turns) rotate<D>(g, *t.angles, t.f_a, t.f_b, p.interleaved);
  if (!norm) return;
  uint64_t ss = f2_mul(v.a[0], v.a[0]);
  ss = f2_fma(v.b[0], v.b[0], ss);
#pragma unroll
  for (int e = 1; e < 4; ++e) ss = f2_fma(v.a[e], v.a[e], f2_fma(v.b[e], v.b[e], ss));
  const float rn = rsqrtf(sum_head<D / 16>(ss) * (1.f / D) + p.eps);
  const uint64_t rn2 = f2_both(live ? rn : 0.f);
  uint64_t dot = 0ull;
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    uint64_t wa[2], wb[2];
    load_pairs(t.weight + e / 2 * (D / 4), wa);
    load_pairs(t.weight + (2 + e / 2) * (D / 4), wb);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v.a[e + i] = f2_mul(v.a[e + i], rn2);
      v.b[e + i] = f2_mul(v.b[e + i], rn2);
      dw.a[e + i] = f2_fma(g.a[e + i], v.a[e + i], dw.a[e + i]);
      dw.b[e + i] = f2_fma(g.b[e + i], v.b[e + i], dw.b[e + i]);
      g.a[e + i] = f2_mul(g.a[e + i], wa[i]);
      g.b[e + i] = f2_mul(g.b[e + i], wb[i]);
      dot = f2_fma(g.a[e + i], v.a[e + i], f2_fma(g.b[e + i], v.b[e + i], dot));
    }
  }
  const uint64_t nd2 = f2_both(-sum_head<D / 16>(dot) * (1.f / D));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    g.a[e] = f2_mul(rn2, f2_fma(nd2, v.a[e], g.a[e]));
    g.b[e] = f2_mul(rn2, f2_fma(nd2, v.b[e], g.b[e]));
  }
}

// Steps [st, end) of one role (0: queries, 1: keys, 2: values) for token (b, s): HPW heads a step.  A step's
// loads are issued a step ahead (in the backward two steps ahead, or three CTAs of 80 registers, were
// slower; prefetching the next token into L2 cost an eighth).
template <int D, bool BACK, int ROLE>
__device__ __forceinline__ void token_heads(const PrepParams& p, const Lane<D>& t, int b, int s, int row,
                                            int sub, int st, int end, Vec& dw) {
  constexpr int HPW = 512 / D;
  const PrepRole& r = p.role[ROLE];
  if (st >= end || row < 0 || row >= r.y_rows) return;
  const bool norm = ROLE < 2 && r.w, turns = ROLE < 2 && t.turns;
  int h = st * HPW + sub;
  const __nv_bfloat16* x =
      static_cast<const __nv_bfloat16*>(r.x) + b * r.xb + s * r.xt + h * r.xh;
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(r.y) +
                     ((static_cast<long long>(b) * r.heads + h) * r.y_rows + row) * D;
  __nv_bfloat16* dx = BACK ? static_cast<__nv_bfloat16*>(r.dx) + b * r.db + s * r.dt + h * r.dh : nullptr;
  const long long x_inc = HPW * r.xh, y_inc = static_cast<long long>(HPW) * r.y_rows * D,
                  d_inc = BACK ? HPW * r.dh : 0;
  uint4 xa, xb, ga, gb;
  auto fetch = [&](bool have) {
    xa = xb = ga = gb = make_uint4(0u, 0u, 0u, 0u);
    if (!have || h >= r.heads) return;
    if (!BACK || norm) {
      xa = load16(x + t.ca);
      xb = load16(x + t.cb);
    }
    if (BACK) {
      ga = load16(y + t.ca);
      gb = load16(y + t.cb);
    }
  };
  fetch(true);
#pragma unroll 1
  for (; st < end; ++st) {
    const bool live = h < r.heads;
    __nv_bfloat16* to = BACK ? dx : y;
    uint4 oa = BACK ? ga : xa, ob = BACK ? gb : xb;
    const uint4 va = xa, vb = xb;
    x += x_inc;
    y += y_inc;
    dx += d_inc;
    h += HPW;
    fetch(st + 1 < end);
    if (norm || turns) {
      Vec v;
      unpack8(va, v.a);
      unpack8(vb, v.b);
      if constexpr (BACK) {
        Vec g;
        unpack8(oa, g.a);
        unpack8(ob, g.b);
        backward_vec<D>(v, g, dw, p, t, norm, turns, live);
        oa = pack8(g.a);
        ob = pack8(g.b);
      } else {
        forward_vec<D>(v, p, t, norm, turns);
        oa = pack8(v.a);
        ob = pack8(v.b);
      }
    }
    if (live) {
      store16(to + t.ca, oa);
      store16(to + t.cb, ob);
    }
  }
}

template <int D, bool BACK>
__global__ void __launch_bounds__(kThreads, BACK ? kBwdCtasPerSm : kFwdCtasPerSm)
    fa_prep_kernel(const PrepParams p) {
  constexpr int LPH = D / 16;    // lanes per head
  constexpr int HPW = 32 / LPH;  // heads per warp and step
  __shared__ __align__(16) Angles<D> angles[kWarps];
  __shared__ __align__(16) float weight[2][D];  // of queries and keys, with the offset
  __shared__ float dw_red[BACK ? kWarps : 1][BACK ? 2 * D : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int x = lane % LPH, sub = lane / LPH;
  Lane<D> tq, tk;
  tq.angles = &angles[warp];
  tq.weight = weight[0] + 4 * x;
  // the lane's two pieces of 8 channels
  tq.turns = x < p.rot / 16;
  tq.ca = tq.turns ? 8 * x : 16 * x;
  tq.cb = tq.turns ? p.rot / 2 + 8 * x : 16 * x + 8;
  tq.f_a = 4 * x;
  tq.f_b = (p.interleaved ? p.rot / 4 : D / 4) + 4 * x;
  tk = tq;
  tk.weight = weight[1] + 4 * x;
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    // group k of four channels of lane xi, as the lanes' pieces are
    const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(p.role[i / D].w);
    const int k = i % D / (D / 4), xi = i % (D / 4) / 4, e = i % 4;
    const bool ti = xi < p.rot / 16;
    const int ch = (k < 2 ? (ti ? 8 * xi : 16 * xi) : (ti ? p.rot / 2 + 8 * xi : 16 * xi + 8)) +
                   4 * (k & 1) + e;
    weight[i / D][i % D] = w ? __bfloat162float(w[ch]) + p.w_off : 1.f;
  }
  // the lane's share of a token's angles: frequencies lane and lane + 32
  uint64_t t64[2];
  int axis[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = lane + 32 * e;
    t64[e] = 0;
    axis[e] = 0;
    if (i < p.rot / 2) {
      const int ax = p.freq_axis ? p.freq_axis[i] : 0;
      if (ax < p.n_axes) {
        t64[e] = turns64(p.inv_freq[i]);
        axis[e] = ax;
      }
    }
  }
  __syncthreads();
  const int steps_q = (p.role[0].heads + HPW - 1) / HPW, steps_k = (p.role[1].heads + HPW - 1) / HPW;
  const int steps_v = (p.role[2].heads + HPW - 1) / HPW;
  const int steps = steps_q + steps_k + steps_v;
  // The work is one line of steps, token by token, of which every warp takes an equal stretch.
  const long long tokens = static_cast<long long>(p.B) * p.S, line = tokens * steps;
  const long long warps = static_cast<long long>(gridDim.x) * kWarps;
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const long long share = line / warps, extra = line - share * warps;
  const long long from = w * share + min(w, extra);
  long long left = share + (w < extra ? 1 : 0);
  long long token = from / steps;
  int st = static_cast<int>(from - token * steps);
  int b = static_cast<int>(token / p.S);
  int s = static_cast<int>(token - static_cast<long long>(b) * p.S);
  Vec dwq, dwk;
#pragma unroll
  for (int e = 0; e < 4; ++e) dwq.a[e] = dwq.b[e] = dwk.a[e] = dwk.b[e] = 0ull;
  while (left > 0) {
    const int end = static_cast<int>(min(static_cast<long long>(steps), st + left));
    const int start = p.row_start ? p.row_start[b] : 0;
    if (p.rot > 0) {
      __syncwarp();  // the last token's angles have been read
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = lane + 32 * e;
        if (i < p.rot / 2) {
          const int pos = p.positions ? __ldg(p.positions + axis[e] * tokens + token) : start + s;
          float co, si;
          turn(t64[e], pos, co, si);
          const int at = place_of<D>(i, p.interleaved);
          angles[warp].c[at] = co;
          angles[warp].s[at] = BACK ? -si : si;
        }
      }
      __syncwarp();
    }
    token_heads<D, BACK, 0>(p, tq, b, s, s, sub, st, min(end, steps_q), dwq);
    token_heads<D, BACK, 1>(p, tk, b, s, start + s, sub, max(0, st - steps_q),
                            min(end - steps_q, steps_k), dwk);
    token_heads<D, BACK, 2>(p, tk, b, s, start + s, sub, max(0, st - steps_q - steps_k),
                            min(end - steps_q - steps_k, steps_v), dwk);
    left -= end - st;
    st = 0;
    ++token;
    if (++s == p.S) {
      s = 0;
      ++b;
    }
  }
  if constexpr (BACK) {
    if (!(p.role[0].dw || p.role[1].dw)) return;  // grid-uniform
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const Vec& d = k ? dwk : dwq;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v[4];
        f2_unpack(d.a[e], v[0], v[1]);
        f2_unpack(d.b[e], v[2], v[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int o = LPH; o < 32; o <<= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (sub == 0) {
          dw_red[warp][k * D + tq.ca + 2 * e] = v[0];
          dw_red[warp][k * D + tq.ca + 2 * e + 1] = v[1];
          dw_red[warp][k * D + tq.cb + 2 * e] = v[2];
          dw_red[warp][k * D + tq.cb + 2 * e + 1] = v[3];
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
      float sum = 0.f;
#pragma unroll
      for (int wi = 0; wi < kWarps; ++wi) sum += dw_red[wi][i];
      p.partial[static_cast<size_t>(blockIdx.x) * 2 * D + i] = sum;
    }
    griddep_launch_dependents();
  }
}

// dw of queries (blockIdx.y 0) and keys (1) from the CTAs' shares: 32 channels a CTA, a warp adds every 32nd
// share, and the warps' sums are added in order.  (Two CTAs of D channels with 8 sums each were a chain of
// loads of 5 us.)
__global__ void __launch_bounds__(1024) fa_prep_dw_kernel(const PrepParams p) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int ch = blockIdx.x * 32 + lane;
  float* dw = p.role[blockIdx.y].dw;
  griddep_wait();
  if (!dw) return;
  float sum = 0.f;
#pragma unroll 8
  for (int k = part; k < p.blocks; k += 32)
    sum += p.partial[static_cast<size_t>(k) * 2 * p.d + blockIdx.y * p.d + ch];
  red[part][lane] = sum;
  __syncthreads();
  if (part == 0) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += red[k][lane];
    dw[ch] = t;
  }
}

}  // namespace

int prep_partial_rows() { return kMaxPartialRows; }

void prep_plan(PrepParams* p, int n_sm, bool back) {
  const int hpw = 32 / (p->d / 16);
  long long steps = 0;
  for (const PrepRole& r : p->role) steps += (r.heads + hpw - 1) / hpw;
  steps *= static_cast<long long>(p->B) * p->S;
  const int wave = back ? std::min(n_sm * kBwdCtasPerSm, kMaxPartialRows) : n_sm * kFwdCtasPerSm;
  p->blocks = static_cast<int>(std::min<long long>(wave, (steps + kWarps - 1) / kWarps));
}

cudaError_t launch_prep(const PrepParams& p, cudaStream_t stream) {
  if (p.d == 128) fa_prep_kernel<128, false><<<p.blocks, kThreads, 0, stream>>>(p);
  else fa_prep_kernel<64, false><<<p.blocks, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_prep_bwd(const PrepParams& p, cudaStream_t stream) {
  if (p.d == 128) fa_prep_kernel<128, true><<<p.blocks, kThreads, 0, stream>>>(p);
  else fa_prep_kernel<64, true><<<p.blocks, kThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !(p.role[0].dw || p.role[1].dw)) return e;
  return launch_dependent(fa_prep_dw_kernel, dim3(p.d / 32, 2), dim3(1024), 0, stream, p);
}

}  // namespace fa
