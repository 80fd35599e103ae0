// Device side of the packed entries: groups of 16 dims, 16 codes of 4 bits (e2m1:
// 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) and one scale of 8 bits (e4m3), value = code *
// scale * 2^exp.  A code has 2 significant bits and a scale 4, so that a value has 6
// and bf16 and fp16 hold code * scale (up to 2,688, at least 2^-10) exactly.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv4.h"

namespace csa2 {

// A scale as a number: NaN for the byte 0x7f, which marks a group that held a NaN or an infinity.
CSA2_DEV __half kv4_scale(uint8_t byte) { return __half(__nv_cvt_fp8_to_halfraw(byte, __NV_E4M3)); }

// Two codes (the first in the low bits) as numbers.
CSA2_DEV __half2 kv4_pair(uint8_t byte) { return __half2(__nv_cvt_fp4x2_to_halfraw2(byte, __NV_E2M1)); }

// Eight codes of a word as four pairs.  (The bytes are named in the conversion: taken out of the word first, each cost two
// instructions more.)
CSA2_DEV void kv4_pairs(uint32_t codes, __half2 (&x)[4]) {
  uint32_t y[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const __half2*>(&y[i]);
}

// Two scales, in the low bits, as numbers.
CSA2_DEV __half2 kv4_scales(uint32_t two) {
  uint32_t y;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(y) : "r"(two));
  return *reinterpret_cast<const __half2*>(&y);
}

// Eight codes times their scale, exactly.
CSA2_DEV void kv4_eight(uint32_t codes, __half2 scale, float (&x)[8]) {
  __half2 y[4];
  kv4_pairs(codes, y);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(__hmul2(y[i], scale));
    x[2 * i] = v.x;
    x[2 * i + 1] = v.y;
  }
}

// 16 numbers as codes and a scale's byte.  The scale is the e4m3 number nearest to a sixth of the
// largest magnitude (ties to even, at least 2^-9, at most 448), a code the e2m1 number nearest to x / scale (ties to even, at
// most 6); `down` is 2^-exp, which no product here rounds by that is not 0 or saturated in the end.
// kF32: x are any fp32 numbers, whose quotients are rounded to fp32 first; that moves none onto a
// border between two codes, as the border times the scale is itself an fp32 number and its neighbours' quotients
// are more than half a step away.  Otherwise they have 8 significant bits (bf16), and a quotient that is not on a border (of 3
// bits; 5 between two scales) is 2^-8 away from it: products with reciprocals, off by 2^-22, are rounded to 11 bits (fp16,
// or fp32 bits), which puts those of borders onto them and moves no other as far.
template <bool kF32>
CSA2_DEV uint8_t kv4_quantise(const float (&x)[16], float down, uint2& codes) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(x[i])));
  top *= down;
  codes = make_uint2(0u, 0u);
  if (!(top < INFINITY)) {   // a NaN or an infinity, or 2^-exp takes numbers beyond fp32, which saturate
    float raw = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(raw) : "f"(fabsf(x[i])));
    if (!(raw < INFINITY)) return 0x7f;
  }
  const float sixth = kF32 ? __fdiv_rn(top, 6.f) : __uint_as_float((__float_as_uint(top * (1.f / 6.f)) + 0x200u) & ~0x3ffu);
  const uint8_t byte = __nv_cvt_float_to_fp8(fmaxf(sixth, 0.001953125f), __NV_SATFINITE, __NV_E4M3);
  const float scale = __half2float(kv4_scale(byte));
  float inv = 0.f;
  if (!kF32) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
  const float mul = inv * down;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float2 y;
    if (kF32) y = make_float2(__fdiv_rn(x[2 * i] * down, scale), __fdiv_rn(x[2 * i + 1] * down, scale));
    else y = __half22float2(__floats2half2_rn(x[2 * i] * mul, x[2 * i + 1] * mul));
    w[i >> 2] |= uint32_t(__nv_cvt_float2_to_fp4x2(y, __NV_E2M1, cudaRoundNearest)) << (8 * (i & 3));
  }
  codes = make_uint2(w[0], w[1]);
  return byte;
}

}  // namespace csa2
