// fa_score.cuh -- the arithmetic of capped and biased scores, shared by the forward, the backward
// and the decode.
//
// Scores leave the matrix product as s = <q, k>.  In units of log2(e), what the softmax sees is
//   z = cap' * tanh(a * s) - slope' * |p - j|,   a = scale / cap,  cap' = cap * log2(e)
// (without a cap: s * scale * log2(e) in place of the first term).
//
// tanh is taken two ways:
//  * |a * s| <= 5/8: a polynomial, tanh(x) = x * (1 + c1 x^2 + .. + c4 x^8), fitted in the maximum
//    norm: off by at most 1.0e-7 of the value.  Five packed multiply-adds for two scores and no
//    special-function instruction.  The coefficients arrive with a and cap' folded in.
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

// The factor m with cap' * tanh(a s) = s * m, for two scores with |a s| <= 5/8.
__device__ __forceinline__ uint64_t cap_small_factor(uint64_t s2, const ScoreArgs& sc) {
  const uint64_t u = f2_mul(s2, s2);
  uint64_t m = f2_fma(u, f2_pack(sc.poly[4], sc.poly[4]), f2_pack(sc.poly[3], sc.poly[3]));
  m = f2_fma(u, m, f2_pack(sc.poly[2], sc.poly[2]));
  m = f2_fma(u, m, f2_pack(sc.poly[1], sc.poly[1]));
  return f2_fma(u, m, f2_pack(sc.poly[0], sc.poly[0]));
}

// cap' * tanh(a s) of one score, by whichever way holds.
__device__ __forceinline__ float cap_one(float s, const ScoreArgs& sc) {
  const float u = s * s;
  float m = fmaf(u, sc.poly[4], sc.poly[3]);
  m = fmaf(u, m, sc.poly[2]);
  m = fmaf(u, m, sc.poly[1]);
  m = fmaf(u, m, sc.poly[0]);
  return fabsf(s) <= sc.small ? s * m : cap_any(s, sc);
}

}  // namespace fa
