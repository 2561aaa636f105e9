// fa_rope.cu -- rotary positions: rotate q and k by their positions, and, in
// the append form, put the rotated k and the plain v in their cache rows.
//
// Pair i of a row at position p turns by the angle p * f_i:
//   y1 = m (x1 cos - x2 sin),  y2 = m (x2 cos + x1 sin),
// with pairs (i, i + rot/2) or (2i, 2i+1) of the first rot columns; the
// backward pass is the transposed rotation (the angle negated).
//
// The pass reads and writes every row once and does six flops a pair, so HBM
// bounds it.  A CTA takes a few tokens and all their heads (or, with few
// tokens, a part of the heads): its threads first share the cosines and sines
// of those tokens out among themselves through shared memory, one angle per
// token and pair and not per head (see fa_angles.cuh), then each keeps the eight pairs of its
// (token, piece) in registers over the heads it walks.  The first heads' rows
// are on their way before the angles are computed.
// Measured on the device, B4 H32 Hkv32 N4096 d128: 82 us, 6570 GB/s (0.97 of the
// copy rate); B8 H16 Hkv4 N2047 d64, 84 MB: 16.6 us.

#include <cstdint>

#include "fa_angles.cuh"
#include "fa_cache.h"

namespace fa {
namespace {

constexpr int kRopeThreads = 128;
// Heads in flight per thread, and CTAs on an SM (with CTAs of twice the threads,
// B4 H32 N4096 d128, 84 us: 4 heads and 2 CTAs 88.5, 6 and 2 84.8, 8 and 2 85.1, 3
// and 3 87, 4 and 4 104).
constexpr int kRopeUnroll = 4;
constexpr int kRopeCtas = 6;  // (80 registers: the half-split form spills one; of the append form see the kernel)

// grid: x = blocks of `tokens` tokens, y = head groups.  Thread: piece c of
// d / 16, token of the block, and first head.  The append form, with a tensor
// more to place, needs about 100 registers (at 80 it spills 15 to 30 of them) and
// has four CTAs on an SM (B4 H32
// N4096 d128, 805 MB: 149 us, 0.80 of the copy rate; the others 0.97).
template <bool INTERLEAVED, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads, APPEND ? 4 : kRopeCtas) fa_rope_kernel(const RopeParams p) {
  extern __shared__ float table[];  // cos, then sin: [tokens][rot / 2]
  const int per_row = p.d >> 4, half = p.rot >> 1;
  const int t0 = blockIdx.x * p.tokens, all = p.B * p.N;
  const int c = threadIdx.x & (per_row - 1);
  const int tl = (static_cast<int>(threadIdx.x) / per_row) & (p.tokens - 1);
  const int lanes = per_row * p.tokens;           // threads of a head
  const int heads_at_once = kRopeThreads / lanes;
  const int t = t0 + tl;
  const int b = t / p.N, n = t - b * p.N;
  const Pieces x = pieces_of<INTERLEAVED>(p.d, p.rot, c);
  // rows of the three tensors' first heads
  const __nv_bfloat16 *src[3] = {p.q + b * p.sq.b + n * p.sq.n, p.k + b * p.sk.b + n * p.sk.n, nullptr};
  __nv_bfloat16 *dst[3] = {p.qo + b * p.sqo.b + n * p.sqo.n, nullptr, nullptr};
  bool row_on = true;
  if (APPEND) {
    const long long row = t < all ? static_cast<long long>(p.cache_len[b]) - p.N + n : -1;
    row_on = row >= 0 && row < p.Nk;
    src[2] = p.v + b * p.sv.b + n * p.sv.n;
    dst[1] = p.ko + b * p.sko.b + row * p.sko.n;
    dst[2] = p.vo + b * p.svo.b + row * p.svo.n;
  } else {
    dst[1] = p.ko + b * p.sko.b + n * p.sko.n;
  }
  const int step = heads_at_once * gridDim.y;
  uint4 w0[kRopeUnroll], w1[kRopeUnroll];
  __nv_bfloat16 *to[kRopeUnroll];
  bool turn[kRopeUnroll];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      int h = h0 + u * step;
      const __nv_bfloat16 *from;
      bool on = h < p.heads && t < all;
      turn[u] = true;
      if (h < p.H) {
        from = src[0] + h * p.sq.h;
        to[u] = dst[0] + h * p.sqo.h;
      } else if (!APPEND || h < p.H + p.Hkv) {
        h -= p.H;
        on = on && row_on;
        from = src[1] + h * p.sk.h;
        to[u] = dst[1] + h * p.sko.h;
      } else {
        h -= p.H + p.Hkv;
        on = on && row_on;
        from = src[2] + h * p.sv.h;
        to[u] = dst[2] + h * p.svo.h;
        turn[u] = false;
      }
      // (in place, pieces that do not turn stay where they are)
      if (!on || (from == to[u] && !(turn[u] && (x.t0 || x.t1)))) {
        to[u] = nullptr;
        continue;
      }
      w0[u] = __ldcs(reinterpret_cast<const uint4 *>(from + x.c0));
      w1[u] = __ldcs(reinterpret_cast<const uint4 *>(from + x.c1));
    }
  };
  // the first heads are on their way while the angles are computed
  int h0 = blockIdx.y * heads_at_once + static_cast<int>(threadIdx.x) / lanes;
  load(h0);
  float *cos_t = table, *sin_t = table + p.tokens * half;
  for (int e = threadIdx.x; e < p.tokens * half; e += kRopeThreads) {
    const int te = t0 + e / half, i = e % half;
    if (te >= all) break;
    const int be = te / p.N, ne = te - be * p.N;
    const long long pos = p.positions ? p.positions[be * p.pos_b + ne]
                                      : (APPEND ? static_cast<long long>(p.cache_len[be]) - p.N + ne : ne);
    float sn, cs;
    angle_of(pos, p.inv_freq[i], &cs, &sn);
    cos_t[e] = cs * p.factor;
    sin_t[e] = sn * (p.factor * p.sign);
  }
  __syncthreads();
  if (t >= all) return;
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (x.t0) cs[i] = cos_t[tl * half + x.p0 + i], sn[i] = sin_t[tl * half + x.p0 + i];
    if (x.t1) cs[i + 4] = cos_t[tl * half + x.p1 + i], sn[i + 4] = sin_t[tl * half + x.p1 + i];
  }
  for (;;) {
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      if (!to[u]) continue;
      uint32_t w[8] = {w0[u].x, w0[u].y, w0[u].z, w0[u].w, w1[u].x, w1[u].y, w1[u].z, w1[u].w};
      if (turn[u]) {
        if (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (!(i < 4 ? x.t0 : x.t1)) continue;
            const float2 y = unpack2(w[i]);
            w[i] = pack2(y.x * cs[i] - y.y * sn[i], y.y * cs[i] + y.x * sn[i]);
          }
        } else if (x.t0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 a = unpack2(w[i]), z = unpack2(w[i + 4]);
            w[i] = pack2(a.x * cs[2 * i] - z.x * sn[2 * i], a.y * cs[2 * i + 1] - z.y * sn[2 * i + 1]);
            w[i + 4] = pack2(z.x * cs[2 * i] + a.x * sn[2 * i], z.y * cs[2 * i + 1] + a.y * sn[2 * i + 1]);
          }
        }
      }
      __stcs(reinterpret_cast<uint4 *>(to[u] + x.c0), make_uint4(w[0], w[1], w[2], w[3]));
      __stcs(reinterpret_cast<uint4 *>(to[u] + x.c1), make_uint4(w[4], w[5], w[6], w[7]));
    }
    h0 += kRopeUnroll * step;
    if (h0 >= p.heads) return;
    load(h0);
  }
}

}  // namespace

cudaError_t launch_rope(bool interleaved, const RopeParams &p, cudaStream_t stream) {
  const dim3 grid((p.B * p.N + p.tokens - 1) / p.tokens, p.head_groups);
  const size_t smem = sizeof(float) * p.tokens * p.rot;
  if (p.cache_len) {
    if (interleaved)
      fa_rope_kernel<true, true><<<grid, kRopeThreads, smem, stream>>>(p);
    else
      fa_rope_kernel<false, true><<<grid, kRopeThreads, smem, stream>>>(p);
  } else {
    if (interleaved)
      fa_rope_kernel<true, false><<<grid, kRopeThreads, smem, stream>>>(p);
    else
      fa_rope_kernel<false, false><<<grid, kRopeThreads, smem, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace fa
