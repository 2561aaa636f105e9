// fa_angles.cuh -- what the kernels that turn rows by their positions share: the
// angle of a position, bf16 pairs, and a thread's pieces of a row.  Device code
// only.
//
// Angles.  The product p * f has to be exact to about 2^-20 of a turn for
// positions in the millions, which fp32 cannot hold and fp64 (a sixty-fourth
// of the fp32 rate here) is too slow for.  Each frequency becomes a 64-bit
// fixed-point fraction of a turn per position (a 24-bit mantissa times
// 2^66 / 2 pi, shifted), and the product modulo 2^64 is the fraction of a
// turn itself: whole turns fall off the top.  Its top 32 bits go to
// sincospi as fp32.  Error, in turns: rounding to 24 bits 2^-26 near half a
// turn, the cut 2^-32, the fraction's last bits (1 + f / 4) |p| 2^-64, since
// 2^66 / 2 pi is cut too; together below 2^-25 up to f = 128.
#pragma once

#include <cstdint>

#include "fa_cache.h"

namespace fa {

// f / (2 pi) turns as a 0.64 fixed-point number, modulo one turn.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  const uint32_t bits = __float_as_uint(f);
  const int e = (bits >> 23) & 255;
  const uint64_t m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  constexpr uint64_t kInv2Pi = 0xa2f9836e4e441529ull;  // floor(2^66 / (2 pi))
  const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  const int s = 152 - (e ? e : 1);  // f / (2 pi) * 2^64 = (m * kInv2Pi) >> s
  uint64_t r;
  if (s <= 0)
    r = s > -64 ? lo << -s : 0;
  else if (s < 64)
    r = (lo >> s) | (hi << (64 - s));
  else
    r = s < 128 ? hi >> (s - 64) : 0;
  return (bits >> 31) ? 0 - r : r;
}

__device__ __forceinline__ float2 unpack2(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// The cosine and sine of the angle that a position makes with a frequency, or with its
// fraction of a turn.
__device__ __forceinline__ void angle_of(long long pos, uint64_t turns, float *cs, float *sn) {
  const uint64_t a = static_cast<uint64_t>(pos) * turns;
  const float half_turns = static_cast<float>(static_cast<int32_t>(a >> 32)) * 4.656612873077393e-10f;  // 2^-31
  sincospif(half_turns, sn, cs);
}
__device__ __forceinline__ void angle_of(long long pos, float f, float *cs, float *sn) {
  angle_of(pos, turn_fraction(f), cs, sn);
}

// A thread's two 16-byte pieces of a row.  Neighbouring threads take
// neighbouring pieces, so that a warp's accesses fill whole sectors.
struct Pieces {
  int c0, c1;      // first columns
  int p0, p1;      // pairs p0 .. p0 + 3 and p1 .. p1 + 3 (of the two pieces, or of both together)
  bool t0, t1;     // the pieces turn
};

template <bool INTERLEAVED>
__device__ __forceinline__ Pieces pieces_of(int d, int rot, int c) {
  Pieces x;
  if (INTERLEAVED) {  // a piece holds four whole pairs
    x.c0 = c * 8;
    x.c1 = d / 2 + c * 8;
    x.p0 = x.c0 / 2;
    x.p1 = x.c1 / 2;
    x.t0 = x.c0 < rot;
    x.t1 = x.c1 < rot;
  } else if (c * 16 < rot) {  // the two halves of eight pairs
    x.c0 = c * 8;
    x.c1 = rot / 2 + c * 8;
    x.p0 = c * 8;
    x.p1 = c * 8 + 4;
    x.t0 = x.t1 = true;
  } else {  // two pieces past rot
    x.c0 = rot + (c * 16 - rot) / 2;
    x.c1 = x.c0 + (d - rot) / 2;
    x.p0 = x.p1 = 0;
    x.t0 = x.t1 = false;
  }
  return x;
}

}  // namespace fa
