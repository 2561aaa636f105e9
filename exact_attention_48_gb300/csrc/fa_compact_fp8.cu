// fa_compact_fp8.cu -- rows of a cache held in 8 bits moved together: row
// base + i becomes the old row base + kept[i], and every block of rows that is
// written the greatest scale of the blocks its rows come from.  A row whose own
// scale was smaller is rounded to it again (a shift of exponents, exact but for
// codes that fall below e4m3's normal range); one whose scale it is is moved bit
// by bit.
//
// HBM bounds both forms.  A CTA works on windows of 128 destination rows, one to
// eight blocks: it reads the rows' codes into registers and the scales of the
// blocks they come from, finds each block's greatest, and writes.  Out of place
// every window is a CTA of its own.  In place a destination row may be the source
// of an earlier destination only (kept ascends and kept[i] >= i), so one CTA takes
// a head's windows of K or V in order.

#include <cstdint>

#include "fa_cache8.h"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kWindow = 128;  // destination rows of a step, aligned: whole blocks

// One tensor of the two.
struct Side {
  const uint8_t *src;
  uint8_t *dst;
  const float *scale;
  float *scale_out;
  long long src_n, dst_n;
};
__device__ __forceinline__ Side side_of(const Compact8Params &p, int tensor, int b, int h) {
  const Strides &s = tensor ? p.sv : p.sk, &o = tensor ? p.svo : p.sko;
  const long long bh = static_cast<long long>(b) * p.Hkv + h;
  Side x;
  x.src = (tensor ? p.v : p.k) + b * s.b + h * s.h;
  x.dst = (tensor ? p.vo : p.ko) + b * o.b + h * o.h;
  x.scale = (tensor ? p.vs : p.ks) + bh * p.blocks;
  x.scale_out = (tensor ? p.vso : p.kso) + bh * p.blocks_out;
  x.src_n = s.n;
  x.dst_n = o.n;
  return x;
}

// What a thread holds of a window: a 16-byte piece of each of ITEMS rows.
template <int D>
struct Window {
  static constexpr int kPieces = D / 16, kPass = kThreads / kPieces, kItems = kWindow / kPass;
  uint4 w[kItems];
  float s[kItems];     // the row's scale before, 0: no row
  bool stays[kItems];  // it is where it belongs

  // Window rows r0 + [0, 128): the rows that move there, and rows before `base`
  // of a block that is written (they stay, and count).
  __device__ __forceinline__ void read(const Compact8Params &p, const Side &x, const int *kept, long long base,
                                       long long r0) {
    const int c = threadIdx.x % kPieces;
#pragma unroll
    for (int it = 0; it < kItems; ++it) {
      const long long dst = r0 + it * kPass + static_cast<int>(threadIdx.x) / kPieces, i = dst - base;
      s[it] = 0.0f;
      stays[it] = false;
      if (dst < 0 || dst >= p.Nout) continue;
      if (i < 0) {
        // a row before base, in a block that rows from base on share
        const long long first = base > 0 ? base : 0;
        if ((dst >> p.block_log2) != (first >> p.block_log2)) continue;
        s[it] = x.scale_out[dst >> p.block_log2];
        stays[it] = true;
        w[it] = *reinterpret_cast<const uint4 *>(x.dst + dst * x.dst_n + c * 16);
        continue;
      }
      if (i >= p.M) continue;
      const int from = kept[i];
      const long long src = base + from;
      if (from < 0 || src < 0 || src >= p.Nk) continue;
      s[it] = x.scale[src >> p.block_log2];
      stays[it] = p.in_place && src == dst;
      w[it] = __ldcs(reinterpret_cast<const uint4 *>(x.src + src * x.src_n + c * 16));
    }
  }
  // most, moved: [8] of the window's blocks, zero before.
  __device__ __forceinline__ void count(const Compact8Params &p, uint32_t *most, uint32_t *moved, long long base,
                                        long long r0) {
#pragma unroll
    for (int it = 0; it < kItems; ++it) {
      const int row = it * kPass + static_cast<int>(threadIdx.x) / kPieces;
      if (!(s[it] > 0.0f) || threadIdx.x % kPieces) continue;
      atomicMax(&most[row >> p.block_log2], __float_as_uint(s[it]));
      if (r0 + row >= base) moved[row >> p.block_log2] = 1u;
    }
  }
  __device__ __forceinline__ void write(const Compact8Params &p, const Side &x, const uint32_t *most,
                                        const uint32_t *moved, long long r0) {
    const int c = threadIdx.x % kPieces;
#pragma unroll
    for (int it = 0; it < kItems; ++it) {
      const int row = it * kPass + static_cast<int>(threadIdx.x) / kPieces, blk = row >> p.block_log2;
      if (!(s[it] > 0.0f) || !moved[blk]) continue;
      const float now = __uint_as_float(most[blk]);
      if (now == s[it] && stays[it]) continue;
      uint4 v = w[it];
      if (now != s[it]) {
        const float r = s[it] / now;
        v.x = rescale_codes(v.x, r);
        v.y = rescale_codes(v.y, r);
        v.z = rescale_codes(v.z, r);
        v.w = rescale_codes(v.w, r);
      }
      __stcs(reinterpret_cast<uint4 *>(x.dst + (r0 + row) * x.dst_n + c * 16), v);
    }
    const int blk = threadIdx.x;
    if (blk < (kWindow >> p.block_log2) && moved[blk])
      x.scale_out[(r0 >> p.block_log2) + blk] = __uint_as_float(most[blk]);
  }
};

// The first window that rows from base on lie in.
__device__ __forceinline__ long long first_window(long long base) { return base >> 7; }  // (arithmetic: floors)

// (K and V of a window in one CTA, 108 registers and two CTAs an SM: B16 Hkv16
// 16384 to 8192 rows d128 324 us.)
template <int D>
__global__ void __launch_bounds__(kThreads, 6) fa_compact_fp8_gather_kernel(const Compact8Params p, int windows) {
  __shared__ uint32_t most[8], moved[8];
  const int x = blockIdx.x >> 1, bh = x / windows, b = bh / p.Hkv, h = bh - b * p.Hkv;
  const long long base = p.base ? p.base[b] : 0;
  const long long r0 = (first_window(base) + (x - bh * windows)) * kWindow;
  const int *kept = p.kept + b * p.kept_b + h * p.kept_h;
  if (threadIdx.x < 8) most[threadIdx.x] = moved[threadIdx.x] = 0u;
  const Side side = side_of(p, blockIdx.x & 1, b, h);
  Window<D> w;
  w.read(p, side, kept, base, r0);
  __syncthreads();
  w.count(p, most, moved, base, r0);
  __syncthreads();
  w.write(p, side, most, moved, r0);
}

template <int D>
__global__ void __launch_bounds__(kThreads) fa_compact_fp8_slide_kernel(const Compact8Params p, int windows) {
  __shared__ uint32_t most[2][8], moved[2][8];
  const int tensor = blockIdx.x & 1, bh = blockIdx.x >> 1, b = bh / p.Hkv, h = bh - b * p.Hkv;
  const long long base = p.base ? p.base[b] : 0;
  const int *kept = p.kept + b * p.kept_b + h * p.kept_h;
  const Side x = side_of(p, tensor, b, h);
  if (threadIdx.x < 16) (&most[0][0])[threadIdx.x] = (&moved[0][0])[threadIdx.x] = 0u;
  for (int i = 0; i < windows; ++i) {
    const long long r0 = (first_window(base) + i) * kWindow;
    Window<D> w;
    w.read(p, x, kept, base, r0);
    __syncthreads();  // every row and scale has been read; the last window's counts are no longer needed
    w.count(p, most[i & 1], moved[i & 1], base, r0);
    if (threadIdx.x < 8) most[~i & 1][threadIdx.x] = moved[~i & 1][threadIdx.x] = 0u;
    __syncthreads();
    w.write(p, x, most[i & 1], moved[i & 1], r0);
  }
}

}  // namespace

cudaError_t launch_compact8(const Compact8Params &p, cudaStream_t stream) {
  const long long heads = static_cast<long long>(p.B) * p.Hkv;
  // windows that M rows may touch (from a window's start without a base)
  const int windows = p.base ? (p.M - 1 + kWindow - 1) / kWindow + 1 : (p.M + kWindow - 1) / kWindow;
  const unsigned grid = static_cast<unsigned>(p.in_place ? heads * 2 : heads * windows * 2);  // below 2^31: checked on entry
  if (p.in_place) {
    if (p.d == 64)
      fa_compact_fp8_slide_kernel<64><<<grid, kThreads, 0, stream>>>(p, windows);
    else
      fa_compact_fp8_slide_kernel<128><<<grid, kThreads, 0, stream>>>(p, windows);
  } else {
    if (p.d == 64)
      fa_compact_fp8_gather_kernel<64><<<grid, kThreads, 0, stream>>>(p, windows);
    else
      fa_compact_fp8_gather_kernel<128><<<grid, kThreads, 0, stream>>>(p, windows);
  }
  return cudaGetLastError();
}

}  // namespace fa
