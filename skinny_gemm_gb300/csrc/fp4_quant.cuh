// fp4_quant.cuh -- sixteen bf16 values at a time to e2m1 codes and block scales:
// device code of the quantiser (fp4.cu) and of the products that quantise a few
// activation rows themselves (fp4_mm.cu).
#pragma once

#include "common.cuh"
#include "fp4.cuh"

namespace w4a16 {
namespace fp4 {

// Eight values to eight codes, value i in bits 4 i.
__device__ __forceinline__ uint32_t codes8(const float* y) {
  uint32_t d;
  asm("{ .reg .b8 a, b, c, e;\n"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 e, %8, %7;\n"
      "mov.b32 %0, {a, b, c, e}; }"
      : "=r"(d)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return d;
}

// Sixteen bf16 values, 32 bytes.
struct Vec16 {
  uint4 a, b;
};
__device__ __forceinline__ Vec16 load16(const uint16_t* p) { return Vec16{ld_nc_v4(p), ld_nc_v4(p + 8)}; }
__device__ __forceinline__ Vec16 zero16() { return Vec16{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}; }

// The largest |x| of eight bf16 values as bits (bf16 magnitudes order like integers).
__device__ __forceinline__ uint32_t peak8(const uint4& v) {
  const uint32_t a = __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), b = __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu);
  const uint32_t m = __vmaxu2(a, b);
  return max(m & 0xFFFFu, m >> 16);
}

// ... of its finite values.
__device__ __forceinline__ uint32_t finite_peak8(const uint4& v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = word_of(v, i) & 0x7FFF7FFFu, lo = w & 0xFFFFu, hi = w >> 16;
    m = max(m, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
  }
  return m;
}

// 2^e for e in -149 .. 127.
__device__ __forceinline__ float exp2i(int e) {
  return e >= -126 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(1u << (e + 149));
}

// 2^e for e in -126 .. 127.
__device__ __forceinline__ float exp2n(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The nv factor's exponent from the row's largest finite |x| (bf16 bits): 2688 = 1.3125 * 2^11, and 1.3125 has
// significand bits 0x28 of 7.  Subnormal peaks are below every bound that counts.
__device__ __forceinline__ int factor_exp(uint32_t peak) {
  const int e = (int)(peak >> 7) - 127 - 11 + ((peak & 0x7Fu) > 0x28u ? 1 : 0);
  return max(e, -126);
}

__device__ __forceinline__ uint32_t peak16(const Vec16& v) { return max(peak8(v.a), peak8(v.b)); }
__device__ __forceinline__ uint32_t finite_peak16(const Vec16& v) { return max(finite_peak8(v.a), finite_peak8(v.b)); }

__device__ __forceinline__ float rcp(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// Two sums a b + c at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{ .reg .b64 a, b, c; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 a, a, b, c; mov.b64 {%0, %1}, a; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{ .reg .b64 a, b; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Sixteen values to codes and their block's scale byte; peak is the block's largest |x| (bf16 bits).
//
// nv.  The codes depend on which side of a border (a multiple of 1/4 up to 5) the quotient y = x / (s f) lies, ties
// included.  x has 8 significant bits and s 4, so that a y that is not on a border is at least 2^-10 from it.  x times an
// approximate reciprocal is off by 2^-20 at most; rounded to a multiple of 2^-12 (by adding and taking off 1.5 * 2^11) it is
// on a border where y is, and on y's side of it elsewhere.  The same for the scale: p / f / 6 against the borders of
// e4m3, 5 significant bits: at least 2^-9 of it away, or on it; kept to 2^-16 of it.
template <int FMT>
__device__ __forceinline__ uint2 block16(const Vec16& v, uint32_t peak, int e, uint32_t& byte) {
  float y[16];
  widen8(v.a, y);
  widen8(v.b, y + 8);
  if (FMT == W4A16_FP4_MX) {
    // floor(log2 peak) - 2 + 127 is the exponent field less 2; a subnormal peak gives 0
    byte = max((int)(peak >> 7) - 2, 0);
    const float s = exp2n(127 - (int)byte);
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(y[i], s);
    if (peak >= 0x7F80u) byte = 0xFFu;
  } else {
    const float p = __fmul_rn(bf16_bits_to_f32((uint16_t)peak), exp2n(-e));
    const float want = __uint_as_float((__float_as_uint(__fmul_rn(p, 1.0f / 6.0f)) + 64u) & ~127u);
    uint16_t pair;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pair) : "f"(0.0f), "f"(want));
    byte = pair & 0xFFu;
    // the scale in fp32: e4m3's bits at half the place of fp32's, times 2^120
    float s = __fmul_rn(__uint_as_float(byte << 20), exp2n(120));
    if (e < -90) {  // s f might leave fp32's normal range
      const float inv = exp2n(-e);
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(y[i], inv);
    } else {
      s = __fmul_rn(s, exp2n(e));
    }
    const float r = byte ? rcp(s) : 0.0f;
    constexpr float kRound = 1.5f * 2048.0f;
    const float2 rr = make_float2(r, r), up = make_float2(kRound, kRound), down = make_float2(-kRound, -kRound);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 q = add2(fma2(make_float2(y[i], y[i + 1]), rr, up), down);
      y[i] = q.x;
      y[i + 1] = q.y;
    }
    if (peak >= 0x7F80u) byte = 0x7Fu;
  }
  if (peak >= 0x7F80u) return make_uint2(0, 0);
  return make_uint2(codes8(y), codes8(y + 8));
}

}  // namespace fp4
}  // namespace w4a16
