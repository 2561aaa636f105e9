// fa_cache_compact.cu -- rows of a key/value cache (and their weights) moved
// together: row base + i becomes the old row base + kept[i].
//
// Nothing but copies: HBM bounds both forms (each moved row read and written
// once).  Out of place every row is independent: a thread moves 16-byte
// pieces of K and V, four rows at a time.  In place a destination row may be
// the source of an earlier destination only (kept ascends and kept[i] >= i),
// so one CTA takes a head's rows in order, chunk by chunk: every row of a
// chunk is read before any of it is written, and the next chunk's rows, which
// all lie at or behind that chunk's own places, are already on their way
// while this one is written.  Heads times two tensors alone may leave SMs
// idle, so a row is cut across CTAs where there are few.
// Measured, B16 Hkv16 16384 to 8192 rows d128 with weights: out of place 318 us
// (6810 GB/s, the HBM copy rate), in place 356 (6080).  One head has at most 17
// CTAs in place, each of which walks the whole list: 131072 to 65536 rows of 1,
// 2 and 8 heads take 102, 106 and 119 us, out of place 12, 23 and 82.

#include <cstdint>

#include "fa_cache.h"

namespace fa {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;     // rows in flight per thread, of K and of V

// The move of list entry i of a head: false if it is skipped.
struct Move {
  long long src, dst;
};
__device__ __forceinline__ bool move_of(const CompactParams &p, const int *kept, long long base, int i, Move *m) {
  if (i >= p.M) return false;
  const int from = kept[i];
  m->src = base + from;
  m->dst = base + i;
  return from >= 0 && m->src >= 0 && m->src < p.Nk && m->dst >= 0 && m->dst < p.Nout;
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) fa_cache_gather_kernel(const CompactParams p) {
  constexpr int kPieces = D / 8;                      // 16-byte pieces of a row
  constexpr int kPass = kMoveThreads / kPieces;       // rows of a pass over the threads
  constexpr int kBlockRows = kPass * kMoveRows;
  const int blocks = (p.M + kBlockRows - 1) / kBlockRows;
  const int bh = blockIdx.x / blocks, b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int i0 = (blockIdx.x - bh * blocks) * kBlockRows + static_cast<int>(threadIdx.x) / kPieces;
  const int c = threadIdx.x % kPieces;
  const int *kept = p.kept + b * p.kept_b + h * p.kept_h;
  const long long base = p.base ? p.base[b] : 0;
  const __nv_bfloat16 *k = p.k + b * p.sk.b + h * p.sk.h + c * 8, *v = p.v + b * p.sv.b + h * p.sv.h + c * 8;
  __nv_bfloat16 *ko = p.ko + b * p.sko.b + h * p.sko.h + c * 8, *vo = p.vo + b * p.svo.b + h * p.svo.h + c * 8;
  Move m[kMoveRows];
  bool on[kMoveRows];
  uint4 kx[kMoveRows], vx[kMoveRows];
#pragma unroll
  for (int r = 0; r < kMoveRows; ++r) on[r] = move_of(p, kept, base, i0 + r * kPass, &m[r]);
#pragma unroll
  for (int r = 0; r < kMoveRows; ++r) {
    if (!on[r]) continue;
    kx[r] = __ldcs(reinterpret_cast<const uint4 *>(k + m[r].src * p.sk.n));
    vx[r] = __ldcs(reinterpret_cast<const uint4 *>(v + m[r].src * p.sv.n));
  }
  if (p.w && c == 0) {
#pragma unroll
    for (int r = 0; r < kMoveRows; ++r)
      if (on[r])
        p.wo[static_cast<long long>(bh) * p.Nout + m[r].dst] = p.w[static_cast<long long>(bh) * p.Nk + m[r].src];
  }
#pragma unroll
  for (int r = 0; r < kMoveRows; ++r) {
    if (!on[r]) continue;
    __stcs(reinterpret_cast<uint4 *>(ko + m[r].dst * p.sko.n), kx[r]);
    __stcs(reinterpret_cast<uint4 *>(vo + m[r].dst * p.svo.n), vx[r]);
  }
}

// In place: CTA x takes slice x % slices (pieces columns wide) of tensor
// (x / slices) % (2 or 3) of head x / slices / (2 or 3); tensor 2 is the
// weights, one CTA a head.
// (threads x pieces a thread and chunk, B16 Hkv16 16384 to 8192 rows and 8 x
// 131072 to 16384, d128: 512 x 4 529 and 45 us, 512 x 2 395 and 60, 1024 x 2
// 451 and 39, 1024 x 3 356 and 36, 1024 x 4 415 and 38)
constexpr int kSlideThreads = 1024;
constexpr int kSlideRows = 3;

template <typename T>
struct Chunk {
  T x[kSlideRows];
  long long dst[kSlideRows];  // row, -1: stays
};

template <typename T>
__device__ __forceinline__ void slide(const CompactParams &p, int b, int h, const T *src, T *dst, long long row_src,
                                      long long row_dst, int pieces) {
  const int *kept = p.kept + b * p.kept_b + h * p.kept_h;
  const long long base = p.base ? p.base[b] : 0;
  const int pass = kSlideThreads / pieces, rows = pass * kSlideRows;
  const int r0 = static_cast<int>(threadIdx.x) / pieces, c = threadIdx.x % pieces;
  auto read = [&](int i0, Chunk<T> &ch) {
#pragma unroll
    for (int r = 0; r < kSlideRows; ++r) {
      Move m;
      const bool on = move_of(p, kept, base, i0 + r * pass + r0, &m) && m.src != m.dst;
      ch.dst[r] = on ? m.dst : -1;
      if (on) ch.x[r] = src[m.src * row_src + c];
    }
  };
  auto write = [&](const Chunk<T> &ch) {
#pragma unroll
    for (int r = 0; r < kSlideRows; ++r)
      if (ch.dst[r] >= 0) dst[ch.dst[r] * row_dst + c] = ch.x[r];
  };
  Chunk<T> a, z;
  read(0, a);
  for (long long i0 = 0; i0 < p.M; i0 += 2ll * rows) {
    if (i0 + rows < p.M) read(static_cast<int>(i0 + rows), z);
    __syncthreads();  // every row of the chunk has been read
    write(a);
    if (i0 + rows >= p.M) break;
    if (i0 + 2ll * rows < p.M) read(static_cast<int>(i0 + 2ll * rows), a);
    __syncthreads();
    write(z);
  }
}

__global__ void __launch_bounds__(kSlideThreads) fa_cache_slide_kernel(const CompactParams p, int slices) {
  const int tensors = p.w ? 3 : 2;
  const int x = blockIdx.x, slice = x % slices, tensor = (x / slices) % tensors, bh = x / slices / tensors;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  if (tensor == 2) {
    if (slice == 0) slide<float>(p, b, h, p.w + static_cast<long long>(bh) * p.Nk, p.wo + static_cast<long long>(bh) * p.Nout, 1, 1, 1);
    return;
  }
  const Strides &s = tensor ? p.sv : p.sk;
  const int pieces = p.d / 8 / slices;
  __nv_bfloat16 *t = (tensor ? p.vo : p.ko) + b * s.b + h * s.h + slice * pieces * 8;
  slide<uint4>(p, b, h, reinterpret_cast<const uint4 *>(t), reinterpret_cast<uint4 *>(t), s.n / 8, s.n / 8, pieces);
}

}  // namespace

cudaError_t launch_cache_compact(const CompactParams &p, cudaStream_t stream) {
  const long long heads = static_cast<long long>(p.B) * p.Hkv;
  if (p.in_place) {
    // rows cut (down to 32 bytes, a DRAM sector) until the CTAs cover the SMs twice
    int slices = 1;
    while (heads * 2 * slices < 2 * 152 && slices < p.d / 16) slices *= 2;
    fa_cache_slide_kernel<<<static_cast<unsigned>(heads * (p.w ? 3 : 2) * slices), kSlideThreads, 0, stream>>>(p,
                                                                                                                slices);
    return cudaGetLastError();
  }
  const int block_rows = kMoveThreads / (p.d / 8) * kMoveRows;
  const long long grid = heads * ((p.M + block_rows - 1) / block_rows);  // below 2^31: checked on entry
  if (p.d == 64)
    fa_cache_gather_kernel<64><<<static_cast<unsigned>(grid), kMoveThreads, 0, stream>>>(p);
  else
    fa_cache_gather_kernel<128><<<static_cast<unsigned>(grid), kMoveThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
