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

// x 2^d, d <= 0: in two steps, for 2^d alone may be no number where x 2^d is one (softmax
// sums and their partials reach 2^74 per position: V's exponents are not in them, but in
// their reference).
__device__ __forceinline__ float scaled_down(float x, float d) {
  return x * ex2(fminf(d + 100.f, 0.f)) * ex2(fmaxf(d, -100.f));
}

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

// Four codes times their block's scale as bf16: exact, for a code has four (e4m3)
// or at most seven significant bits and the scale is a power of two.
template <int FORM>
struct Scaled8;

__device__ __forceinline__ uint32_t bf16_twice(int e) {  // 2^e in both halves, e in [-126, 127]
  return (uint32_t)(e + 127) * 0x00800080u;
}
__device__ __forceinline__ uint32_t bf16_mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <>
struct Scaled8<NP_E4M3> {
  // A code's exponent and mantissa as bf16's are the value times 2^-120, subnormals
  // too.  2^(120 + e) is bf16's up to e = 7; larger scales take two factors.
  uint32_t f, more;
  __device__ __forceinline__ explicit Scaled8(int e) : f(bf16_twice(min(120 + e, 127))), more(bf16_twice(max(e - 7, 0))) {}
  __device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) const {
    const uint32_t a = __byte_perm(w, 0u, 0x1404), b = __byte_perm(w, 0u, 0x3424);
    lo = bf16_mul2(((a >> 4) & 0x07f007f0u) | (a & 0x80008000u), f);
    hi = bf16_mul2(((b >> 4) & 0x07f007f0u) | (b & 0x80008000u), f);
  }
  // (the same for all of a token's codes: the caller asks once)
  __device__ __forceinline__ bool large() const { return more != 0x3f803f80u; }
  __device__ __forceinline__ void widen_large(uint32_t& lo, uint32_t& hi) const {
    lo = bf16_mul2(lo, more);
    hi = bf16_mul2(hi, more);
  }
};

template <>
struct Scaled8<NP_INT8> {
  // Under 0x43 the low seven bits are the bf16 128 + them, and the sign bit alone
  // 128 or 256: their difference is the code.
  uint32_t f;
  __device__ __forceinline__ explicit Scaled8(int e) : f(bf16_twice(e)) {}
  __device__ __forceinline__ static uint32_t code(uint32_t t) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(t & 0xff7fff7fu), "r"(t & 0xff80ff80u));
    return r;
  }
  __device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) const {
    lo = bf16_mul2(code(__byte_perm(w, 0x43434343u, 0x4140)), f);
    hi = bf16_mul2(code(__byte_perm(w, 0x43434343u, 0x4342)), f);
  }
  __device__ __forceinline__ bool large() const { return false; }
  __device__ __forceinline__ void widen_large(uint32_t&, uint32_t&) const {}
};

// Four codes as fp16, times 2^-d: exact to d = 15 (an e4m3 code is no finer than 2^-9, fp16
// than 2^-24); the caller has smaller d only.
template <int FORM>
struct Below8;

// 2^-d in both halves
__device__ __forceinline__ __half2 half_twice_below(uint32_t d) {
  return __float2half2_rn(__uint_as_float((127u - d) << 23));
}

template <>
struct Below8<NP_E4M3> {
  __half2 f;
  __device__ __forceinline__ explicit Below8(uint32_t d) : f(half_twice_below(d)) {}
  __device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) const {
    const uint32_t a = Form8<NP_E4M3>::half_lo(w), b = Form8<NP_E4M3>::half_hi(w);
    const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&a), f);
    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&b), f);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
};

template <>
struct Below8<NP_INT8> {
  // (1152 + code) 2^-d - 1152 2^-d
  __half2 f, off;
  __device__ __forceinline__ explicit Below8(uint32_t d) : f(half_twice_below(d)) {
    const uint32_t c = 0xe480e480u;  // -1152
    off = __hmul2(*reinterpret_cast<const __half2*>(&c), f);
  }
  __device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) const {
    const uint32_t t = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(t, 0x64646464u, 0x4140), b = __byte_perm(t, 0x64646464u, 0x4342);
    const __half2 x = __hfma2(*reinterpret_cast<const __half2*>(&a), f, off);
    const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&b), f, off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
};

// 16 bytes to shared memory, zeros where !live
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0)
               : "memory");
}

template <int N>
__device__ __forceinline__ void lds(uint32_t at, uint32_t* w) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(at));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
  else asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at));
}

__device__ __forceinline__ void sts4(uint32_t at, const uint32_t* w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}

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
