// fa_score.cuh -- the arithmetic of capped and biased scores, shared by the forward, the backward
// and the decode.
//
// Scores leave the matrix product as s = <q, k>.  In units of log2(e), what the softmax sees is
//   z = cap' * tanh(a * s) - slope' * |p - j|,   a = scale / cap,  cap' = cap * log2(e)
// (without a cap: s * scale * log2(e) in place of the first term).
//
// tanh is taken two ways:
//  * |a * s| <= 0.25, 0.7 or 1.4: a polynomial, tanh(x) = x * (1 + c1 x^2 + ..) of degree 2, 4 or 7 in
//    x^2, fitted to the least relative error: off by at most 4.0e-7, 3.0e-7, 3.4e-7 of the value.  Four,
//    six or ten packed multiply-adds for two scores and no special-function instruction; the
//    coefficients arrive with cap' folded in, those of degrees 2 and 4 with a as well.
//  * else 1 - 2 / (1 + 2^(2 a s log2 e)): two special-function instructions, off by about 2^-22 of
//    the cap, whatever the score.
// Both are far below the rounding of the weights to bf16 (2^-9 of a weight) while the cap is small: 6e-5 of
// an exponent at the largest cap that takes the second for every score of a tile (kWideCap; at 2^20 it
// would be a quarter of one).  Above that each score takes the way that keeps its own accuracy (cap_wide).
#pragma once

#include "fa_scored.h"
#include "sm103_ptx.cuh"

namespace fa {

// tmem_ld32_max for the maximum of the magnitudes.
__device__ __forceinline__ void tmem_ld32_max_abs(uint32_t taddr, uint32_t (&r)[32], float& mx) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.abs.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31]), "=f"(mx)
      : "r"(taddr));
}

// Whether the plan (if any) was made for these sizes.  The tiles and offsets in one of others would lead out of the
// tensors; a kernel that gets one records kStatusPlan and returns.
constexpr unsigned int kStatusPlan = 4u;
__device__ __forceinline__ bool plan_fits(const MaskPlan& m, int Sq, int Sk) {
  if (!m.rows) return true;
  const int4 s = __ldg(m.sizes);
  return s.x == m.B && s.y == Sq && s.z == Sk && s.w == kPlanMark;
}

// The n lowest bits of a word (none for n < 0, all for n > 32).
__device__ __forceinline__ uint32_t bits_below(int n) {
  return static_cast<uint32_t>((1ull << max(0, min(n, 32))) - 1);
}

// Sets bits [a, e) of 128, a <= e, of which what lies outside falls off.
__device__ __forceinline__ void add_span(uint32_t (&bits)[4], int a, int e) {
#pragma unroll
  for (int w = 0; w < 4; ++w) bits[w] |= bits_below(e - 32 * w) & ~bits_below(a - 32 * w);
}

// Two fp32 values -> f16 pair (round to nearest even), and back (exact).
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint64_t f16x2_to_f2(uint32_t w) {
  float lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(w));
  return f2_pack(lo, hi);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The smaller of two; NaN where one is.
__device__ __forceinline__ float min_or_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// cap' * tanh(a s) for any s.
__device__ __forceinline__ float cap_any(float s, const ScoreArgs& sc) {
  const float e = ex2_approx(s * sc.two_a_log2e);
  return fmaf(-2.f * sc.cap_log2e, rcp_approx(1.f + e), sc.cap_log2e);
}

// The same for two scores of one row, which share a reciprocal (1 / x = y / (x y)); at 2^60 the
// quotient is 0 beside 1.  (A NaN reaches both: not for scores of different rows.)
__device__ __forceinline__ uint64_t cap_any2(uint64_t s2, const ScoreArgs& sc) {
  float x0, x1;
  f2_unpack(f2_mul(s2, f2_pack(sc.two_a_log2e, sc.two_a_log2e)), x0, x1);
  const float e0 = ex2_approx(min_or_nan(x0, 60.f)), e1 = ex2_approx(min_or_nan(x1, 60.f));
  f2_unpack(f2_add(f2_pack(e0, e1), f2_pack(1.f, 1.f)), x0, x1);
  const float r = rcp_approx(x0 * x1);
  const uint64_t r2 = f2_mul(f2_pack(r, r), f2_pack(x1, x0));
  return f2_fma(f2_pack(-2.f * sc.cap_log2e, -2.f * sc.cap_log2e), r2,
                f2_pack(sc.cap_log2e, sc.cap_log2e));
}

// The factor m with cap' * tanh(a s) = s * m for two scores with |s| <= small[0] (degree 2) or
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

// m and y = a s with cap' * tanh(a s) = y * m for two scores with |s| <= small[2].
__device__ __forceinline__ uint64_t cap_factor7(uint64_t s2, const ScoreArgs& sc, uint64_t& y2) {
  y2 = f2_mul(s2, f2_pack(sc.a, sc.a));
  const uint64_t u = f2_mul(y2, y2);
  uint64_t m = f2_pack(sc.poly7[7].x, sc.poly7[7].y);
#pragma unroll
  for (int i = 6; i >= 0; --i) m = f2_fma(u, m, f2_pack(sc.poly7[i].x, sc.poly7[i].y));
  return m;
}

// cap' * tanh(a s) of any score under any cap, off by what its own size allows: the degree-7 form in
// y = a s, whose coefficients hold cap' alone and fit for every a; past its range cap_any (|tanh| > 0.88).
__device__ __forceinline__ float cap_wide(float s, const ScoreArgs& sc) {
  const float y = s * sc.a, u = y * y;
  float m = sc.poly7[7].x;
#pragma unroll
  for (int i = 6; i >= 0; --i) m = fmaf(u, m, sc.poly7[i].x);
  return fabsf(s) <= sc.small[2] ? y * m : cap_any(s, sc);
}

// cap' * tanh(a s) of one score with |s| <= small[1].
__device__ __forceinline__ float cap_small(float s, const ScoreArgs& sc) {
  const float u = s * s;
  float m = sc.poly4[4].x;
#pragma unroll
  for (int i = 3; i >= 0; --i) m = fmaf(u, m, sc.poly4[i].x);
  return s * m;
}

}  // namespace fa
