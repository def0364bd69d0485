// cache8.cuh -- the 8-bit cache: codes, scales and their conversions.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "np_common.cuh"

namespace npk {

constexpr int kScaleMin = -60, kScaleMax = 60;  // a scale is 2^e, e in between

// e of a stored scale, whatever its bits: the exponent field, clamped
__device__ __forceinline__ int scale_exp(uint32_t bits) {
  return min(max((int)((bits >> 23) & 0xffu) - 127, kScaleMin), kScaleMax);
}
// 2^e, e in [-126, 127]
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <int FORM>
struct Form8;

template <>
struct Form8<NP_E4M3> {
  // The least e with a <= 448 2^e = 1.75 2^(8 + e), a > 0 and normal: the exponent of
  // a, less 8, and one more where its significand is above 1.75.
  __device__ __forceinline__ static int need(uint32_t a) {
    return (int)(a >> 23) - 127 - 8 + ((a & 0x7fffffu) > 0x600000u ? 1 : 0);
  }
  // two values, rounded to nearest even, at most 448 in size
  __device__ __forceinline__ static uint32_t code2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  }
  // (A NaN is all ones in both; cvt keeps its sign out.)
  // the two low codes of w as fp16, exact
  __device__ __forceinline__ static uint32_t half_lo(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
  }
  __device__ __forceinline__ static uint32_t half_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
  }
};

template <>
struct Form8<NP_INT8> {
  // 127 2^e = 1.984375 2^(6 + e)
  __device__ __forceinline__ static int need(uint32_t a) {
    return (int)(a >> 23) - 127 - 6 + ((a & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  }
  __device__ __forceinline__ static uint32_t code1(float x) {
    // (NaN: fmaxf takes the bound, so it is caught before)
    const float y = x == x ? fminf(fmaxf(x, -127.f), 127.f) : 0.f;
    return (uint32_t)__float2int_rn(y) & 0xffu;
  }
  __device__ __forceinline__ static uint32_t code2(float lo, float hi) {
    return code1(lo) | (code1(hi) << 8);
  }
  // A byte x + 128 under 0x64 is the fp16 1024 + 128 + x; less 1152 it is x.
  __device__ __forceinline__ static uint32_t half_of(uint32_t biased) {
    const uint32_t off = 0x64806480u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&biased),
                              *reinterpret_cast<const __half2*>(&off));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  __device__ __forceinline__ static uint32_t half_lo(uint32_t w) {
    return half_of(__byte_perm(w ^ 0x80808080u, 0x64646464u, 0x4140));
  }
  __device__ __forceinline__ static uint32_t half_hi(uint32_t w) {
    return half_of(__byte_perm(w ^ 0x80808080u, 0x64646464u, 0x4342));
  }
};

// four codes as fp32
template <int FORM>
__device__ __forceinline__ void widen8x4(uint32_t w, float* x) {
  const uint32_t a = Form8<FORM>::half_lo(w), b = Form8<FORM>::half_hi(w);
  const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&b));
  x[0] = lo.x;
  x[1] = lo.y;
  x[2] = hi.x;
  x[3] = hi.y;
}

}  // namespace npk
