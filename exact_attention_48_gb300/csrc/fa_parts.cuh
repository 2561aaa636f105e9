// fa_parts.cuh -- values as the sum of two e4m3 parts, the nearest e4m3 value and
// that of what is left, and other conversions of the kernels on an 8-bit cache.
// Device code only.
#pragma once

#include <cfloat>
#include <cstdint>

#include "ptx.cuh"

namespace fa {

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^x / l, |x| up to 128 and l up to fp32's greatest: between the factors nothing leaves the range that the result is in.
__device__ __forceinline__ float quotient(float x, float l) { return ex2(0.5f * x) * (1.0f / l) * ex2(0.5f * x); }
// Four values as their two e4m3 parts.  (From fp32: the conversions of f16 pairs take several instructions each.)
__device__ __forceinline__ void parts_of(float a, float b, float c, float d, uint32_t *hi, uint32_t *lo) {
  const uint32_t h = pack_e4m3x4(a, b, c, d);
  float r0, r1, r2, r3;
  asm("{\n\t.reg .b32 n, x, y;\n\t.reg .b16 l, u, a0, a1, b0, b1;\n\t"
      "xor.b32 n, %4, 0x80808080;\n\t"
      "mov.b32 {l, u}, n;\n\t"
      "cvt.rn.f16x2.e4m3x2 x, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, u;\n\t"
      "mov.b32 {a0, a1}, x;\n\t"
      "mov.b32 {b0, b1}, y;\n\t"
      "add.rn.f32.f16 %0, a0, %5;\n\t"
      "add.rn.f32.f16 %1, a1, %6;\n\t"
      "add.rn.f32.f16 %2, b0, %7;\n\t"
      "add.rn.f32.f16 %3, b1, %8;\n\t}"
      : "=&f"(r0), "=&f"(r1), "=&f"(r2), "=&f"(r3)
      : "r"(h), "f"(a), "f"(b), "f"(c), "f"(d));
  *hi = h;
  *lo = pack_e4m3x4(r0, r1, r2, r3);
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
    parts_of(v[0], v[1], v[2], v[3], &a[y], &z[y]);
  }
  *hi = make_uint4(a[0], a[1], a[2], a[3]);
  *lo = make_uint4(z[0], z[1], z[2], z[3]);
}

// Tiles of rows of D codes, as TMA leaves them: where 16-byte piece x of row r lies, and the
// descriptor of one (K-major, or MN-major with slabs of D columns `lbo` bytes apart).
template <int D>
__device__ __forceinline__ uint32_t piece_at(int r, int x) {
  return r * D + (D == 128 ? (x ^ (r & 7)) : (x ^ ((r >> 1) & 3))) * 16;
}
template <int D>
__device__ __forceinline__ uint64_t sdesc_codes(const void *tile, uint32_t lbo = 16) {
  return D == 128 ? sdesc_sw128(smem_addr(tile), lbo, 1024) : sdesc_sw64(smem_addr(tile), lbo, 512);
}

}  // namespace fa
