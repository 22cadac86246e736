// Conversions between bf16 rows and the quantised formats of a paged K/V cache.
//
// e4m3: a floating-point format, so a scale's mantissa would buy next to nothing; a power
// of two makes the scaling exact in both directions: the only rounding is that of x 2^-e
// to e4m3's four significant bits, and c 2^e is exact in bf16. e = ceil(log2(max|x| / 448))
// comes from the bits of max|x|: 448 = 1.75 * 2^8, so with max|x| = f * 2^E, 1 <= f < 2,
// e = E - 8 (+ 1 if f > 1.75).
//
// e2m1: two significant bits, so a power of two would leave up to half of the few codes
// unused: 16 values share a scale of four significant bits. Its byte is bits 14..7 of the
// scale as fp16, so a scale is one shift, and code * scale has six significant bits: exact
// in fp16 and bf16.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/bd_paged.h"
#include "ptx.cuh"

namespace bd {

// ---- bf16 values as bits

// max|x| of 8 bf16 values as bits (the order of magnitudes is that of their bits)
__device__ __forceinline__ uint32_t absmax8(const uint4& x) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t t = __vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m));
  return max(t & 0xffffu, t >> 16);
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The power of two that takes a row of q with max|q| of bits mx to f 2^14, 1 <= f < 2, in two
// factors, and its inverse: max|q| = f 2^E, a row below 2^-110 is scaled by 2^124 only.
__device__ __forceinline__ float2 q_factors(uint32_t mx, float* inv) {
  const int E = max(int(mx >> 7) - 127, -110), E0 = min(E, 113);
  *inv = __uint_as_float(uint32_t(127 - 14 + E0) << 23) * __uint_as_float(uint32_t(127 + (E - E0)) << 23);
  return make_float2(__uint_as_float(uint32_t(127 + 14 - E0) << 23), __uint_as_float(uint32_t(127 - (E - E0)) << 23));
}

// ---- e4m3

// Exponent byte b of an e4m3 row as a factor 2^(b - 127); byte 255 marks a row
// that held an infinity or a NaN.
__device__ __forceinline__ float exp_factor(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(b << 23);
}

__device__ __forceinline__ uint32_t pack4_e4m3(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Quantises a row spread over LPR lanes (8 values each): codes, and the exponent byte.
template <int LPR>
__device__ __forceinline__ uint2 quantise8(const uint4& x, uint32_t* byte) {
  uint32_t mx = absmax8(x);
#pragma unroll
  for (int s = LPR / 2; s > 0; s >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, s));
  if (mx >= 0x7f80u) {
    *byte = 255u;
    return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
  }
  // bits of max|x|: exponent field E + 127, 7 mantissa bits (1.75 = 0x60); a value
  // below the clamp, zero and subnormals among them, takes the lowest exponent
  int e = int(mx >> 7) - 127 - 8 + ((mx & 0x7fu) > 0x60u ? 1 : 0);
  e = min(60, max(-60, e));
  *byte = uint32_t(e + 127);
  const float f = __uint_as_float(uint32_t(127 - e) << 23);
  return make_uint2(pack4_e4m3(bf16_lo(x.x) * f, bf16_hi(x.x) * f, bf16_lo(x.y) * f, bf16_hi(x.y) * f),
                    pack4_e4m3(bf16_lo(x.z) * f, bf16_hi(x.z) * f, bf16_lo(x.w) * f, bf16_hi(x.w) * f));
}

// 4 codes times f as bf16 (exact: 4 significant bits and a power of two)
__device__ __forceinline__ uint2 dequantise4(uint32_t c, float f) {
  uint32_t a, b;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(c));
  const float2 x = __half22float2(*reinterpret_cast<__half2*>(&a)), y = __half22float2(*reinterpret_cast<__half2*>(&b));
  return make_uint2(bf16_pair(x.x * f, x.y * f), bf16_pair(y.x * f, y.y * f));
}

// ---- e2m1

constexpr uint32_t kLeastScale = 8, kMostScale = 226;  // bytes that are written: 2^-14 .. 10240

// Scale bytes as fp16: of two bytes at bits 0 and 16 a pair, of one at bit 0 the same twice.
__device__ __forceinline__ uint32_t scale_pair(uint32_t b) { return b << 7; }
__device__ __forceinline__ uint32_t scale_twice(uint32_t b) { return b * 0x00800080u; }

// 8 codes as fp16 pairs, element order
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t c, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 p, q, r, s;\n\tmov.b32 {p, q, r, s}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, p;\n\tcvt.rn.f16x2.e2m1x2 %1, q;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, r;\n\tcvt.rn.f16x2.e2m1x2 %3, s;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Scale byte of 16 values with max|x| of bits mx (finite): the smallest of [8, 226] that has
// max|x| <= 6 s. max|x| has 8 significant bits and 6 s has 6, so the quotient by 6 in fp32 is
// never taken for one on the other side of an s, at worst for the one before.
__device__ __forceinline__ uint32_t scale_byte(uint32_t mx) {
  const float t = __uint_as_float(mx << 16);
  int b = int(__float_as_uint(t * (1.f / 6.f)) >> 20) - (112 << 3);
  b = min(max(b, int(kLeastScale)), int(kMostScale));
  const float s = __uint_as_float((uint32_t(b) << 20) + (112u << 23));
  return uint32_t(min(b + (6.f * s < t ? 1 : 0), int(kMostScale)));
}

// 8 values as codes of scale byte b (255: zeros). x / s is taken as x times an approximate 1 / s, off
// by less than 2^-22, and rounded to a multiple of 2^-10 (by adding and taking off 1.5 * 2^13; what
// saturates anyway may come out anyhow above 6): a quotient midway between two codes, a multiple of 1/4,
// comes out exact, and others are 2^-8 of it away from there at least (8 significant bits of x against 7 of
// the code's midpoint times s). The sign is x's, of zeros too.
__device__ __forceinline__ uint32_t quantise8_e2m1(const uint4& x, uint32_t b) {
  if (b == 255u) return 0u;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__uint_as_float((b << 20) + (112u << 23))));
  float y[8];
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = bf16_lo(w[i]), hi = bf16_hi(w[i]);
    float2 v = dev::ffma2(make_float2(lo, hi), make_float2(r, r), make_float2(12288.f, 12288.f));
    v = dev::fadd2(v, make_float2(-12288.f, -12288.f));
    y[2 * i] = copysignf(v.x, lo);
    y[2 * i + 1] = copysignf(v.y, hi);
  }
  uint32_t c;
  asm("{\n\t.reg .b8 p, q, r, s;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 r, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 s, %8, %7;\n\t"
      "mov.b32 %0, {p, q, r, s};\n\t}"
      : "=r"(c)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return c;
}

// 8 codes of scale byte b as bf16
__device__ __forceinline__ uint4 dequantise8_e2m1(uint32_t c, uint32_t b) {
  uint32_t h[4];
  e2m1x8_to_f16(c, h);
  const uint32_t s = scale_twice(b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = mul_f16x2(h[i], s);
    const float2 v = __half22float2(*reinterpret_cast<__half2*>(&h[i]));
    h[i] = bf16_pair(v.x, v.y);
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// The 16 values of scale number i of a row: codes at d, the scale's byte at e.
__device__ __forceinline__ void store_group_e2m1(const uint4& x, const uint4& y, uint32_t i, uint8_t* d, uint8_t* e) {
  const uint32_t mx = max(absmax8(x), absmax8(y)), byte = mx >= 0x7f80u ? 255u : scale_byte(mx);
  reinterpret_cast<uint2*>(d)[i] = make_uint2(quantise8_e2m1(x, byte), quantise8_e2m1(y, byte));
  e[i] = uint8_t(byte);
}

// Quantises a row spread over LPR lanes (8 values each; the whole warp takes part) and stores
// its codes at d and its exponent or scale bytes at e.
template <int LPR, int FMT>
__device__ __forceinline__ void store_quantised(const uint4& x, uint32_t sub, bool store, uint8_t* d, uint8_t* e) {
  if constexpr (FMT == BD_CACHE_E4M3) {
    uint32_t byte;
    const uint2 c = quantise8<LPR>(x, &byte);
    if (!store) return;
    reinterpret_cast<uint2*>(d)[sub] = c;
    if (sub == 0) *e = uint8_t(byte);
  } else {
    uint32_t mx = absmax8(x);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));  // of the two lanes that share a scale
    const uint32_t byte = mx >= 0x7f80u ? 255u : scale_byte(mx);
    if (!store) return;
    reinterpret_cast<uint32_t*>(d)[sub] = quantise8_e2m1(x, byte);
    if (sub % 2 == 0) e[sub / 2] = uint8_t(byte);
  }
}

}  // namespace bd
