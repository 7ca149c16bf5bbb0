// kda_paged_e4m3.cuh -- the 8-bit cache of the paged calls: e4m3 values with a
// scale for every 16 tokens and head.
#pragma once

#include <cuda_fp8.h>

#include "kda_paged.cuh"

namespace kda {

// Scales.  Within these bounds the largest ratio of two, 2^100, times any weight that
// counts (2^-24 of the row's largest) is a normal float.
constexpr float kMinScale = 0x1p-50f, kMaxScale = 0x1p50f;
constexpr float kMaxE4m3 = 448.f;

__device__ __forceinline__ bool good_scale(float s) { return s >= kMinScale && s <= kMaxScale; }

// Four and 16 values; every e4m3 value is an fp16 value.
__device__ __forceinline__ void e4m3_to_f32(uint32_t w, float (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void e4m3_to_f32(const uint4 &w, float (&x)[16]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y[4];
    e4m3_to_f32(u[i], y);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[4 * i + j] = y[j];
  }
}
// Two values (the low 16 bits of w), and back, rounded to nearest.
__device__ __forceinline__ __half2 e4m3_to_f16(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3);
  return *reinterpret_cast<const __half2 *>(&h);
}
__device__ __forceinline__ uint32_t f16_to_e4m3(__half2 x) {
  return __nv_cvt_halfraw2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
}
// The two fp16 pairs of four values, and those of 16.
__device__ __forceinline__ void e4m3_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ void e4m3_to_f16(const uint4 &w, uint32_t (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) e4m3_to_f16(u[i], x[2 * i], x[2 * i + 1]);
}
// Four values, rounded to nearest; beyond 448 they become 448.
__device__ __forceinline__ uint32_t f32_to_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// A value that is rounded to 8 bits as the exact result is: x is it rounded to fp32, rest
// has the sign of what is missing (0: nothing).  Of the two fp32 neighbours of an inexact
// result this is the one whose last bit is 1, which is neither an e4m3 value nor half way
// between two; rounded to nearest, results beside a half would become it.  (Values outside
// these bounds become 0 or 448 either way.)
__device__ __forceinline__ float odd_neighbour(float x, float rest) {
  const uint32_t b = __float_as_uint(x);
  const bool inexact = rest != 0.f && fabsf(x) > 0x1p-12f && fabsf(x) < 1024.f;
  return !inexact || (b & 1u) ? x : __uint_as_float((rest > 0.f) == (x > 0.f) ? b + 1u : b - 1u);
}
__device__ __forceinline__ float product_for_e4m3(float a, float b) {
  const float x = a * b;
  return odd_neighbour(x, fmaf(a, b, -x));
}
__device__ __forceinline__ float quotient_for_e4m3(float a, float b) {  // b > 0
  const float x = a / b;
  return odd_neighbour(x, fmaf(-x, b, a));
}

// The smallest power of two p with amax <= 448 p (448 = 1.75 * 2^8), within the
// scales' bounds.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u);
  return __uint_as_float((uint32_t)min(max(e, 127 - 50), 127 + 50) << 23);
}

}  // namespace kda
