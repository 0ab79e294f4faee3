// Conversions between 8-bit codes and wider numbers (sm_103a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "pairs.cuh"

namespace vbs {

// Four codes to two pairs of fp16 (exact).
template <int FMT> __device__ __forceinline__ void codes4(u32 w, u32& lo, u32& hi) {
  if (FMT == VBS_I8) {
    // byte b + 128 under an exponent of 2^10: 1024 + 128 + b, less 1152
    w ^= 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    u32 a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias), y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
    lo = *reinterpret_cast<u32*>(&x);
    hi = *reinterpret_cast<u32*>(&y);
  } else {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
  }
}

// Four codes as fp32 (exact).
template <int FMT> __device__ __forceinline__ void decode4(u32 w, float2& lo, float2& hi) {
  u32 a, b;
  codes4<FMT>(w, a, b);
  lo = __half22float2(*reinterpret_cast<__half2*>(&a));
  hi = __half22float2(*reinterpret_cast<__half2*>(&b));
}

// Four values within the format's range (already scaled) to four codes, rounded to nearest, ties to even.
template <int FMT> __device__ __forceinline__ u32 encode4(float a, float b, float c, float d) {
  if (FMT == VBS_I8) {
    // adding 1.5 x 2^23 leaves the rounded integer in the low bits
    const float k = 12582912.f;
    const u32 lo = __byte_perm(__float_as_uint(a + k), __float_as_uint(b + k), 0x0040);
    const u32 hi = __byte_perm(__float_as_uint(c + k), __float_as_uint(d + k), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
  }
  u32 r;
  asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\t"
      "mov.b32 %0, {x, y};\n\t}" : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// encode4 of a 2^-e, .. with inv = (2^-e, 2^-e): the product is exact, so that it and the rounding are one fma for int8.
template <int FMT> __device__ __forceinline__ u32 encode4_scaled(float a, float b, float c, float d, u64 inv) {
  if (FMT == VBS_I8) {
    const u64 k = pair(12582912.f, 12582912.f);
    unpair(fma2(pair(a, b), inv, k), a, b);
    unpair(fma2(pair(c, d), inv, k), c, d);
    const u32 lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
    const u32 hi = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
  }
  unpair(mul2(pair(a, b), inv), a, b);
  unpair(mul2(pair(c, d), inv), c, d);
  return encode4<FMT>(a, b, c, d);
}

}  // namespace vbs
