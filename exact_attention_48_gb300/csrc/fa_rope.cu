// fa_rope.cu -- rotary positions: rotate q and k by their positions, and, in
// the append form, put the rotated k and the plain v in their cache rows.
//
// Pair i of a row at position p turns by the angle p * f_i:
//   y1 = m (x1 cos - x2 sin),  y2 = m (x2 cos + x1 sin),
// with pairs (i, i + rot/2) or (2i, 2i+1) of the first rot columns; the
// backward pass is the transposed rotation (the angle negated).
//
// The pass reads and writes every row once and does six flops a pair, so HBM
// bounds it.  A thread owns eight pairs (16 columns) of one token and keeps
// their cosines and sines in registers over the heads it walks, so the
// angles cost once per token and head group, not once per head.
//
// Angles.  The product p * f has to be exact to about 2^-20 of a turn for
// positions in the millions, which fp32 cannot hold and fp64 (a sixty-fourth
// of the fp32 rate here) is too slow for.  Each frequency becomes a 64-bit
// fixed-point fraction of a turn per position (a 24-bit mantissa times
// 2^66 / 2 pi, shifted), and the product modulo 2^64 is the fraction of a
// turn itself: whole turns fall off the top.  Its top 32 bits go to
// sincospi.

#include <cstdint>

#include "fa_cache.h"

namespace fa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;  // heads in flight per thread

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

// Where row (b, n) of head h comes from and goes to; false if it goes nowhere.
struct RopeRow {
  const __nv_bfloat16 *src;
  __nv_bfloat16 *dst;
  bool turn;
};

template <bool APPEND>
__device__ __forceinline__ bool rope_row(const RopeParams &p, int h, int b, int n, int row, RopeRow *r) {
  if (h < p.H) {
    r->src = p.q + b * p.sq.b + h * p.sq.h + n * p.sq.n;
    r->dst = p.qo + b * p.sqo.b + h * p.sqo.h + n * p.sqo.n;
    r->turn = true;
    return true;
  }
  if (APPEND && (row < 0 || row >= p.Nk)) return false;
  h -= p.H;
  if (h < p.Hkv) {
    r->src = p.k + b * p.sk.b + h * p.sk.h + n * p.sk.n;
    r->dst = p.ko + b * p.sko.b + h * p.sko.h + row * p.sko.n;
    r->turn = true;
    return true;
  }
  h -= p.Hkv;
  r->src = p.v + b * p.sv.b + h * p.sv.h + n * p.sv.n;
  r->dst = p.vo + b * p.svo.b + h * p.svo.h + row * p.svo.n;
  r->turn = false;
  return true;
}

__device__ __forceinline__ float2 unpack2(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// grid: x = blocks of tokens, y = head groups (heads h = y, y + groups, ...)
template <bool INTERLEAVED, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_kernel(const RopeParams p) {
  const int per_row = p.d >> 4;  // threads of a row, 16 columns each
  const int c = threadIdx.x & (per_row - 1);
  const int tokens = kRopeThreads / per_row;
  const int t = blockIdx.x * tokens + static_cast<int>(threadIdx.x) / per_row;
  if (t >= p.B * p.N) return;
  const int b = t / p.N, n = t - b * p.N;
  int row = n;
  if (APPEND) row = p.cache_len[b] - p.N + n;

  // columns [c0, c0 + 8) and [c1, c1 + 8): eight pairs, or the columns past rot
  const bool turns = c * 16 < p.rot;
  const bool halves = !INTERLEAVED && turns;
  const int c0 = halves ? c * 8 : c * 16, c1 = halves ? c * 8 + (p.rot >> 1) : c * 16 + 8;

  float cs[8], sn[8];
  if (turns) {
    const long long pos = p.positions ? p.positions[b * p.pos_b + n] : row;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t a = static_cast<uint64_t>(pos) * turn_fraction(p.inv_freq[c * 8 + i]);
      const float half_turns = static_cast<float>(static_cast<int32_t>(a >> 32)) * 4.656612873077393e-10f;  // 2^-31
      sincospif(half_turns, &sn[i], &cs[i]);
      cs[i] *= p.factor;
      sn[i] *= p.factor * p.sign;
    }
  }

  for (int h0 = blockIdx.y; h0 < p.heads; h0 += kRopeUnroll * p.head_groups) {
    RopeRow r[kRopeUnroll];
    uint4 x0[kRopeUnroll], x1[kRopeUnroll];
    bool on[kRopeUnroll];
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int h = h0 + u * p.head_groups;
      on[u] = h < p.heads && rope_row<APPEND>(p, h, b, n, row, &r[u]);
      // in place, columns that do not turn stay where they are
      if (on[u] && !(turns && r[u].turn) && r[u].src == r[u].dst) on[u] = false;
      if (on[u]) {
        const int a0 = r[u].turn ? c0 : c * 16, a1 = r[u].turn ? c1 : c * 16 + 8;
        x0[u] = *reinterpret_cast<const uint4 *>(r[u].src + a0);
        x1[u] = *reinterpret_cast<const uint4 *>(r[u].src + a1);
      }
    }
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      if (!on[u]) continue;
      const int a0 = r[u].turn ? c0 : c * 16, a1 = r[u].turn ? c1 : c * 16 + 8;
      uint32_t w[8] = {x0[u].x, x0[u].y, x0[u].z, x0[u].w, x1[u].x, x1[u].y, x1[u].z, x1[u].w};
      if (turns && r[u].turn) {
        if (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 x = unpack2(w[i]);
            w[i] = pack2(x.x * cs[i] - x.y * sn[i], x.y * cs[i] + x.x * sn[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 a = unpack2(w[i]), z = unpack2(w[i + 4]);
            w[i] = pack2(a.x * cs[2 * i] - z.x * sn[2 * i], a.y * cs[2 * i + 1] - z.y * sn[2 * i + 1]);
            w[i + 4] = pack2(z.x * cs[2 * i] + a.x * sn[2 * i], z.y * cs[2 * i + 1] + a.y * sn[2 * i + 1]);
          }
        }
      }
      *reinterpret_cast<uint4 *>(r[u].dst + a0) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4 *>(r[u].dst + a1) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

}  // namespace

cudaError_t launch_rope(bool interleaved, const RopeParams &p, cudaStream_t stream) {
  const int tokens = kRopeThreads / (p.d >> 4);
  const dim3 grid((p.B * p.N + tokens - 1) / tokens, p.head_groups);
  if (p.cache_len) {
    if (interleaved)
      fa_rope_kernel<true, true><<<grid, kRopeThreads, 0, stream>>>(p);
    else
      fa_rope_kernel<false, true><<<grid, kRopeThreads, 0, stream>>>(p);
  } else {
    if (interleaved)
      fa_rope_kernel<true, false><<<grid, kRopeThreads, 0, stream>>>(p);
    else
      fa_rope_kernel<false, false><<<grid, kRopeThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace fa
