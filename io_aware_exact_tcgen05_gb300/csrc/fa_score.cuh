// fa_score.cuh -- the arithmetic of capped and biased scores, shared by the forward, the backward
// and the decode.
//
// Scores leave the matrix product as s = <q, k>.  In units of log2(e), what the softmax sees is
//   z = cap' * tanh(a * s) - slope' * |p - j|,   a = scale / cap,  cap' = cap * log2(e)
// (without a cap: s * scale * log2(e) in place of the first term).
//
// tanh is taken two ways:
//  * |a * s| <= 1/4 or 5/8: a polynomial, tanh(x) = x * (1 + c1 x^2 + ..) up to x^4 or x^8 in the
//    brackets, fitted in the maximum norm: off by at most 4e-7 or 1e-7 of the value.  Three or five
//    packed multiply-adds for two scores and no special-function instruction.  The coefficients
//    arrive with a and cap' folded in.
//  * else 1 - 2 / (1 + 2^(2 a s log2 e)): two special-function instructions, off by about 2^-22 of
//    the cap.
// Both are far below the rounding of the weights to bf16 (2^-9 of a weight).
#pragma once

#include "fa_scored.h"
#include "sm103_ptx.cuh"

namespace fa {

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap' * tanh(a s) for any s.
__device__ __forceinline__ float cap_any(float s, const ScoreArgs& sc) {
  const float e = ex2_approx(s * sc.two_a_log2e);
  return fmaf(-2.f * sc.cap_log2e, rcp_approx(1.f + e), sc.cap_log2e);
}

__device__ __forceinline__ uint64_t cap_any2(uint64_t s2, const ScoreArgs& sc) {
  float e0, e1;
  f2_unpack(f2_mul(s2, f2_pack(sc.two_a_log2e, sc.two_a_log2e)), e0, e1);
  f2_unpack(f2_add(f2_pack(ex2_approx(e0), ex2_approx(e1)), f2_pack(1.f, 1.f)), e0, e1);
  return f2_fma(f2_pack(-2.f * sc.cap_log2e, -2.f * sc.cap_log2e),
                f2_pack(rcp_approx(e0), rcp_approx(e1)), f2_pack(sc.cap_log2e, sc.cap_log2e));
}

// The factor m with cap' * tanh(a s) = s * m, for two scores with |s| <= small[0] (degree 2) or
// small[1] (degree 4).
template <int DEGREE>
__device__ __forceinline__ uint64_t cap_small_factor(uint64_t s2, const ScoreArgs& sc) {
  const float2* c = DEGREE == 2 ? sc.poly2 : sc.poly4;
  const uint64_t u = f2_mul(s2, s2);
  uint64_t m = f2_pack(c[DEGREE].x, c[DEGREE].y);
#pragma unroll
  for (int i = DEGREE - 1; i >= 0; --i) m = f2_fma(u, m, f2_pack(c[i].x, c[i].y));
  return m;
}

// cap' * tanh(a s) of one score, by whichever way holds.
__device__ __forceinline__ float cap_one(float s, const ScoreArgs& sc) {
  const float u = s * s;
  float m = sc.poly4[4].x;
#pragma unroll
  for (int i = 3; i >= 0; --i) m = fmaf(u, m, sc.poly4[i].x);
  return fabsf(s) <= sc.small[1] ? s * m : cap_any(s, sc);
}

}  // namespace fa
