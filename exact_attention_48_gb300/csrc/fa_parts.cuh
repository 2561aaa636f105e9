// fa_parts.cuh -- values as the sum of two e4m3 parts, the nearest e4m3 value and
// that of what is left, and other conversions of the kernels on an 8-bit cache.
// Device code only.
#pragma once

#include <cfloat>
#include <cstdint>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace fa {

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint2 codes_to_f16(uint32_t w) {
  uint2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(w));
  return r;
}
// Four weights (two f16 pairs) as their two e4m3 parts.
__device__ __forceinline__ void parts_of(uint32_t a, uint32_t b, uint32_t *hi, uint32_t *lo) {
  asm("{\n\t.reg .b16 ha, hb, la, lb;\n\t.reg .b32 x, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 ha, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 hb, %3;\n\t"
      "mov.b32 %0, {ha, hb};\n\t"
      "cvt.rn.f16x2.e4m3x2 x, ha;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, hb;\n\t"
      "sub.rn.f16x2 x, %2, x;\n\t"
      "sub.rn.f16x2 y, %3, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 la, x;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 lb, y;\n\t"
      "mov.b32 %1, {la, lb};\n\t}"
      : "=&r"(*hi), "=&r"(*lo)
      : "r"(a), "r"(b));
}

// The greatest finite magnitude of 16 bf16 values.
__device__ __forceinline__ float greatest(const uint32_t (&w)[8]) {
  float most = 0.0f;
#pragma unroll
  for (int y = 0; y < 8; ++y) {
    const float a = fabsf(__uint_as_float(w[y] << 16)), z = fabsf(__uint_as_float(w[y] & 0xffff0000u));
    if (a <= FLT_MAX) most = fmaxf(most, a);
    if (z <= FLT_MAX) most = fmaxf(most, z);
  }
  return most;
}

// 16 bf16 values times `by` as their two parts (NaN where they are not finite).
__device__ __forceinline__ void q_parts(const uint32_t (&w)[8], float by, uint4 *hi, uint4 *lo) {
  uint32_t a[4], z[4];
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    float v[4] = {__uint_as_float(w[2 * y] << 16), __uint_as_float(w[2 * y] & 0xffff0000u),
                  __uint_as_float(w[2 * y + 1] << 16), __uint_as_float(w[2 * y + 1] & 0xffff0000u)};
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = fabsf(v[x]) <= FLT_MAX ? v[x] * by : NAN;
    a[y] = pack_e4m3x4(v[0], v[1], v[2], v[3]);
    const uint2 h = codes_to_f16(a[y]);
    const float2 h0 = __half22float2(*reinterpret_cast<const __half2 *>(&h.x));
    const float2 h1 = __half22float2(*reinterpret_cast<const __half2 *>(&h.y));
    z[y] = pack_e4m3x4(v[0] - h0.x, v[1] - h0.y, v[2] - h1.x, v[3] - h1.y);
  }
  *hi = make_uint4(a[0], a[1], a[2], a[3]);
  *lo = make_uint4(z[0], z[1], z[2], z[3]);
}

}  // namespace fa
