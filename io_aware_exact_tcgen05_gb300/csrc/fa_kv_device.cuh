// fa_kv_device.cuh -- device helpers of the paged 8-bit KV cache: the block
// scale, and e4m3 codes to and from bf16 and fp32.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sm103_ptx.cuh"

namespace fa {

constexpr int kScaleExpMin = -100;  // block scales are 2^e with e in [-100, 119]
constexpr int kScaleExpMax = 119;

// Largest magnitude of eight bf16 values as bf16 bits, in the two halves of the
// result; infinities and NaN count as 0.
__device__ __forceinline__ uint32_t max_finite_bf16x2(const uint4& w) {
  uint32_t m = 0;
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = x[i] & 0x7fff7fffu;
    m = __vmaxu2(m, a & __vcmpltu2(a, 0x7f807f80u));
  }
  return m;
}

// 2^e for whole e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// The block scale for a largest magnitude given as bf16 bits: the smallest 2^e
// with amax <= 448 * 2^e = 1.75 * 2^(e + 8), e clamped.  bf16's 0.75 is 0x60.
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7fu) > 0x60u ? 1 : 0);
  return pow2i(min(max(e, kScaleExpMin), kScaleExpMax));
}

// The two low or high e4m3 bytes of a word -> f16x2, exact.  (Taking the half
// inside the conversion costs nothing; a shift before it costs a third.)
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint32_t w) {
  const uint32_t h = e4m3x2_to_f16x2(w);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// NaN codes -> 0 (the bounds of a page leave NaN out).
__device__ __forceinline__ uint2 zero_nan_codes(const uint2& w) {
  return make_uint2(w.x & ~__vcmpeq4(w.x & 0x7f7f7f7fu, 0x7f7f7f7fu),
                    w.y & ~__vcmpeq4(w.y & 0x7f7f7f7fu, 0x7f7f7f7fu));
}

// 16 bytes that are read once: past L1.
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// Eight bf16 values -> e4m3 codes of value * inv (inv = 1 / s for a power-of-two
// scale: the product is the quotient).
__device__ __forceinline__ uint2 quantise8(const uint4& w, float inv) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = pack_e4m3x2(__uint_as_float(x[i] << 16) * inv, __uint_as_float(x[i] & 0xffff0000u) * inv);
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Codes * ratio, rounded to e4m3 again.
__device__ __forceinline__ uint2 rescale_codes(const uint2& w, float ratio) {
  uint32_t c[4] = {w.x, w.x >> 16, w.y, w.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = e4m3x2_to_f32x2(c[i]);
    c[i] = pack_e4m3x2(v.x * ratio, v.y * ratio);
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Eight codes * s -> bf16.
__device__ __forceinline__ uint4 dequantise8(const uint2& w, float s) {
  const float2 a = e4m3x2_to_f32x2(w.x), b = e4m3x2_to_f32x2(w.x >> 16);
  const float2 c = e4m3x2_to_f32x2(w.y), d = e4m3x2_to_f32x2(w.y >> 16);
  return make_uint4(pack_bf16x2(a.x * s, a.y * s), pack_bf16x2(b.x * s, b.y * s),
                    pack_bf16x2(c.x * s, c.y * s), pack_bf16x2(d.x * s, d.y * s));
}

}  // namespace fa
