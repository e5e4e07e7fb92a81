// kv4.cuh -- device conversions between bf16 / fp16 and the 4-bit cache format.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "kv4.h"

namespace ra {

// The scale byte of a group with largest magnitude `amax` (a finite bf16 value):
// amax / 6 rounded to nearest even with 3 mantissa bits, at most 10240.  amax
// has 8 significant bits, so amax / 6 either lies exactly on a rounding border
// (and the correctly rounded quotient is that border) or at least 2^-12 away
// from one: the fp32 quotient decides like the exact one.
// `scale` receives the byte's value.
__device__ __forceinline__ uint32_t kv4_scale_byte(float amax, float& scale) {
  const float s = fminf(__fdiv_rn(amax, 6.f), kKv4MaxScale);
  // fp16 keeps 10 mantissa bits of a normal number; 3 are wanted.  Adding
  // 1.5 * 2^(23 + e - 3) rounds s (in [2^e, 2^(e+1)), e >= -14) to a multiple
  // of 2^(e-3), half to even.
  const int e = max((int)(__float_as_uint(s) >> 23), 127 - 14);
  const float magic = __uint_as_float(((uint32_t)(e + 20) << 23) | 0x400000u);
  scale = __fadd_rn(__fadd_rn(s, magic), -magic);
  return (uint32_t)__half_as_ushort(__float2half_rn(scale)) >> 7;
}

// 16 bf16 elements (two 16-byte words) -> 8 bytes of codes, element 2b in the
// low and 2b + 1 in the high half of byte b; returns the scale byte.
__device__ __forceinline__ uint32_t kv4_round_group(const uint4 (&src)[2], uint2& codes) {
  const uint4 a = src[0], b = src[1];
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  // magnitudes as integers order like the numbers; both halves of a word at once
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
  const uint32_t top = max(m & 0xffffu, m >> 16);
  if (top >= 0x7f80u) {  // an infinity or NaN: the group reads as NaN
    codes = make_uint2(0u, 0u);
    return kKv4NanScale;
  }
  float s;
  const uint32_t byte = kv4_scale_byte(__uint_as_float(top << 16), s);
  // x / s: x has 8 significant bits and s 4, so the quotient lies either on a
  // border of the code grid (a multiple of 1/4) or at least 2^-11 from one.
  // x times the rounded reciprocal is off by less than 2^-20; adding and
  // taking away 1.5 * 2^9 rounds it to a multiple of 2^-14, which puts the
  // former exactly on the border (the conversion then ties to even) and moves
  // none of the latter across one.
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t c[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float lo = __uint_as_float(w[i] << 16) * inv, hi = __uint_as_float(w[i] & 0xffff0000u) * inv;
    lo = __fadd_rn(__fadd_rn(lo, 768.f), -768.f);
    hi = __fadd_rn(__fadd_rn(hi, 768.f), -768.f);
    uint32_t byte2;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}"
        : "=r"(byte2) : "f"(hi), "f"(lo));
    c[i >> 2] |= byte2 << (8 * (i & 3));
  }
  codes = make_uint2(c[0], c[1]);
  return byte;
}

// The four bytes of a word of codes -> eight fp16 numbers, the low code of a byte
// in the low half.
__device__ __forceinline__ void kv4_code_pairs(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Eight codes and their group's scale byte -> eight bf16 values (exact: 6
// significant bits).
__device__ __forceinline__ uint4 kv4_expand_half(uint32_t codes, uint32_t scale) {
  const float s = __half2float(__ushort_as_half((unsigned short)(scale << 7)));
  uint32_t h[4], o[4];
  kv4_code_pairs(codes, h);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    const __nv_bfloat162 v = __floats2bfloat162_rn(f.x * s, f.y * s);
    o[j] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace ra
