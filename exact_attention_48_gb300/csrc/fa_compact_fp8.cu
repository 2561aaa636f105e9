// fa_compact_fp8.cu -- rows of a cache held in 8 bits moved together: row
// base + i becomes the old row base + kept[i], and every block of rows that is
// written the greatest scale of the blocks its rows come from.  A row whose own
// scale was smaller is rounded to it again (a shift of exponents, exact but for
// codes that fall below e4m3's normal range); one whose scale it is is moved bit
// by bit.
//
// HBM bounds both forms.  Out of place a warp moves 16 rows of K or V; it looks through
// the list and the scales of its whole block by itself (up to 128 of each, which the
// block's other warps look through as well), so that no warp waits for another and
// 64 of them an SM keep loads in flight.  B16 Hkv16 16384 to 8192 rows d128 (1.1 GB) 164 us,
// 0.98 of the copy bandwidth (blocks of 128 rows: 174); a CTA a window of 128 rows with
// the blocks' greatest scales found in shared memory took 209, both tensors in a CTA 324.
// (32 registers; at d = 128 28 bytes of spills stored, 36 loaded.)
//
// In place a destination row may be the source of an earlier destination only (kept
// ascends and kept[i] >= i), so a head's windows of K or V go in order.  Columns do
// not depend on each other, only the scales do: where there are few heads, a cluster
// of up to 8 CTAs shares a head, each with its columns of longer windows; a
// cluster barrier a window lets the first of them write a window's scales only when
// all have read them.  The next window's rows and the list after it are on their way
// meanwhile (a later window's sources lie behind the rows written here).  B16 Hkv16 16384 to
// 8192 rows d128 292 us; B1 Hkv2 131072 to 65536 rows 158 us, 1214 with a CTA a head; B1
// Hkv8 328 us.  The bf16 cache's move (fa_cache_compact.cu) takes 363, 103 and 119 for twice
// the bytes: a head's slices have no scale in common there and need not meet.

#include <cstdint>

#include "fa_cache8.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kWindow = 128;  // destination rows, aligned: whole blocks

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

__device__ __forceinline__ uint4 rescale_piece(uint4 v, float r) {
  return make_uint4(rescale_codes(v.x, r), rescale_codes(v.y, r), rescale_codes(v.z, r), rescale_codes(v.w, r));
}

// Out of place.  grid: x = (window of 128 rows of a head, K or V); a warp moves 16 rows,
// and looks through the list and the scales of its whole block by itself (no exchange
// between warps but where rows before base stay).
template <int D>
__global__ void __launch_bounds__(kThreads, 8) fa_compact_fp8_gather_kernel(const Compact8Params p, int windows) {
  constexpr int kPieces = D / 16, kPass = 32 / kPieces, kItems = 16 / kPass;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int x = blockIdx.x >> 1, bh = x / windows, b = bh / p.Hkv, h = bh - b * p.Hkv;
  const long long base = p.base ? p.base[b] : 0;
  const long long w0 = ((base >> 7) + (x - bh * windows)) * kWindow;  // (arithmetic: floors)
  const long long r0 = w0 + warp * 16, b0 = (r0 >> p.block_log2) << p.block_log2;
  const int *kept = p.kept + b * p.kept_b + h * p.kept_h;
  const Side side = side_of(p, blockIdx.x & 1, b, h);
  // the block's rows, 32 at a time: the row that moves there (-1: none), its scale
  const long long shared_blk = (base > 0 ? base : 0) >> p.block_log2;  // rows before base in it stay, and count
  int from = -1;
  float scale = 0.0f, most = 0.0f;
  bool moved = false;
  for (int u = 0; u < 1 << p.block_log2; u += 32) {
    const long long dst = b0 + u + lane, i = dst - base;
    int f = -1;
    float s = 0.0f;
    if (dst >= 0 && dst < p.Nout && lane < 1 << p.block_log2) {
      if (i < 0) {
        if ((dst >> p.block_log2) == shared_blk) {
          f = static_cast<int>(dst);
          s = side.scale_out[shared_blk];
        }
      } else if (i < p.M) {
        const int k = kept[i];
        const long long src = base + k;
        if (k >= 0 && src >= 0 && src < p.Nk) {
          f = static_cast<int>(src);
          s = side.scale[src >> p.block_log2];
          moved |= s > 0.0f;
        }
      }
    }
    most = fmaxf(most, s);
    if (u == ((static_cast<int>(r0 - b0)) & ~31)) {  // this warp's own rows are among them
      from = f;
      scale = s;
    }
  }
  const int c = lane % kPieces, own = static_cast<int>(r0 - b0) & 31;
  uint4 w[kItems];
#pragma unroll
  for (int it = 0; it < kItems; ++it) {
    const int row = it * kPass + lane / kPieces, f = __shfl_sync(0xffffffffu, from, own + row);
    if (f < 0) continue;
    const uint8_t *at = r0 + row < base ? side.dst + f * side.dst_n : side.src + f * side.src_n;
    w[it] = __ldcs(reinterpret_cast<const uint4 *>(at + c * 16));
  }
  most = warp_max_f32(most);
  moved = __any_sync(0xffffffffu, moved);
  if (base > w0) __syncthreads();  // rows of the output and a scale of it that count have been read
  if (!moved) return;
#pragma unroll
  for (int it = 0; it < kItems; ++it) {
    const int row = it * kPass + lane / kPieces;
    const float s = __shfl_sync(0xffffffffu, scale, own + row);
    if (!(s > 0.0f)) continue;
    __stcs(reinterpret_cast<uint4 *>(side.dst + (r0 + row) * side.dst_n + c * 16),
           s == most ? w[it] : rescale_piece(w[it], s / most));
  }
  if (r0 == b0 && lane == 0) side.scale_out[r0 >> p.block_log2] = most;
}

__device__ __forceinline__ void meet(int log2_cluster) {
  if (log2_cluster)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  else
    __syncthreads();
}

constexpr int kSlideItems = 4;  // rows of a thread

// In place.  grid: x = (head, K or V, rank in the cluster).  A row takes t = 2^lt threads
// of a CTA, a window 4 T / t rows.
template <int D, int T>
__global__ void __launch_bounds__(T, 1024 / T) fa_compact_fp8_slide_kernel(const Compact8Params p, int windows,
                                                                           int log2_cluster) {
  constexpr int kLogPieces = D == 128 ? 3 : 2, kMostBlocks = T * kSlideItems / 16;
  __shared__ uint32_t most[3][kMostBlocks], moved[3][kMostBlocks];  // used in turn
  const int tid = threadIdx.x, lt = kLogPieces - log2_cluster, step = T >> lt, window = step * kSlideItems;
  const int rank = blockIdx.x & ((1 << log2_cluster) - 1), of = blockIdx.x >> log2_cluster;
  const int tensor = of & 1, bh = of >> 1, b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int c = (rank << lt) + (tid & ((1 << lt) - 1)), first = tid >> lt;  // column piece, row of the window
  const long long base = p.base ? p.base[b] : 0, begin = (base >> 7) * kWindow;  // (arithmetic: floors)
  const long long shared_blk = (base > 0 ? base : 0) >> p.block_log2;            // rows before base in it stay, and count
  const int *kept = p.kept + b * p.kept_b + h * p.kept_h;
  const Side x = side_of(p, tensor, b, h);
  for (int i = tid; i < kMostBlocks; i += T) most[0][i] = moved[0][i] = 0u;

  // The rows that move to the thread's rows of window i: an old row, or -1.
  int from[kSlideItems];
  auto list = [&](int i) {
#pragma unroll
    for (int it = 0; it < kSlideItems; ++it) {
      const long long dst = begin + static_cast<long long>(i) * window + it * step + first, e = dst - base;
      from[it] = -1;
      if (i >= windows || dst < 0 || dst >= p.Nk) continue;
      if (e < 0) {
        if ((dst >> p.block_log2) == shared_blk) from[it] = static_cast<int>(dst);
      } else if (e < p.M) {
        const int k = kept[e];
        const long long src = base + k;
        if (k >= 0 && src >= 0 && src < p.Nk) from[it] = static_cast<int>(src);
      }
    }
  };
  uint4 w[kSlideItems], wn[kSlideItems];
  float s[kSlideItems], sn[kSlideItems];  // the rows' scales before, 0: no row
  uint32_t stays = 0, staysn;             // rows that are where they belong, a bit each
  auto read = [&](int i) {
    staysn = 0;
#pragma unroll
    for (int it = 0; it < kSlideItems; ++it) {
      const int src = from[it];
      sn[it] = 0.0f;
      if (src < 0) continue;
      sn[it] = x.scale[src >> p.block_log2];
      wn[it] = __ldcs(reinterpret_cast<const uint4 *>(x.src + src * x.src_n + c * 16));
      if (src == begin + static_cast<long long>(i) * window + it * step + first) staysn |= 1u << it;
    }
  };
  list(0);
  read(0);
  list(1);
  int turn = 0;
  for (int i = 0; i < windows; ++i) {
    const long long r0 = begin + static_cast<long long>(i) * window;
    const int now_turn = turn, next_turn = turn == 2 ? 0 : turn + 1;
    turn = next_turn;
#pragma unroll
    for (int it = 0; it < kSlideItems; ++it) w[it] = wn[it], s[it] = sn[it];
    stays = staysn;
    __syncthreads();  // the counts are zero
    read(i + 1);
    list(i + 2);
    for (int j = tid; j < kMostBlocks; j += T) most[next_turn][j] = moved[next_turn][j] = 0u;
#pragma unroll
    for (int it = 0; it < kSlideItems; ++it) {
      const int row = it * step + first;
      if (!(s[it] > 0.0f) || (tid & ((1 << lt) - 1))) continue;
      atomicMax(&most[now_turn][row >> p.block_log2], __float_as_uint(s[it]));
      if (r0 + row >= base) moved[now_turn][row >> p.block_log2] = 1u;
    }
    meet(log2_cluster);  // every rank has read this window's rows and scales
#pragma unroll
    for (int it = 0; it < kSlideItems; ++it) {
      const int row = it * step + first, blk = row >> p.block_log2;
      if (!(s[it] > 0.0f) || !moved[now_turn][blk]) continue;
      const float now = __uint_as_float(most[now_turn][blk]);
      if (now == s[it] && ((stays >> it) & 1u)) continue;
      __stcs(reinterpret_cast<uint4 *>(x.dst + (r0 + row) * x.dst_n + c * 16),
             now == s[it] ? w[it] : rescale_piece(w[it], s[it] / now));
    }
    if (rank == 0 && tid < (window >> p.block_log2) && moved[now_turn][tid])
      x.scale_out[(r0 >> p.block_log2) + tid] = __uint_as_float(most[now_turn][tid]);
  }
}

}  // namespace

template <int D, int T>
static cudaError_t launch_slide(const Compact8Params &p, int log2_cluster, cudaStream_t stream) {
  const int window = (T * kSlideItems * 16 / D) << log2_cluster;
  const int windows = static_cast<int>((static_cast<long long>(p.M) + (p.base ? kWindow - 1 : 0) + window - 1) / window);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(p.B) * p.Hkv * 2 << log2_cluster));  // (below 2^26)
  cfg.blockDim = dim3(T);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1u << log2_cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = log2_cluster ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fa_compact_fp8_slide_kernel<D, T>, p, windows, log2_cluster);
}

// Some two CTAs an SM at most, where a window has rows for them; where that leaves SMs idle, CTAs of 1024 threads, whose
// windows are four times as long (a window takes some 4 us, whatever it holds: B1 Hkv2 131072 to 65536 rows 159 us, 246
// with 256).
template <int D>
static cudaError_t launch_slide(const Compact8Params &p, cudaStream_t stream) {
  const long long heads = static_cast<long long>(p.B) * p.Hkv * 2;
  constexpr int kWindow256 = kThreads * kSlideItems * 16 / D;
  int lc = 0;
  while ((16 << (lc + 1)) <= D && heads << (lc + 1) <= 304 && p.M > kWindow256 << lc) ++lc;
  return heads << lc <= 152 && p.M > kWindow256 << lc ? launch_slide<D, 1024>(p, lc, stream)
                                                      : launch_slide<D, kThreads>(p, lc, stream);
}

cudaError_t launch_compact8(const Compact8Params &p, cudaStream_t stream) {
  if (p.in_place) return p.d == 64 ? launch_slide<64>(p, stream) : launch_slide<128>(p, stream);
  // windows that M rows may touch (from a window's start without a base)
  const int windows = p.base ? (p.M - 1 + kWindow - 1) / kWindow + 1 : (p.M + kWindow - 1) / kWindow;
  const unsigned grid = static_cast<unsigned>(static_cast<long long>(p.B) * p.Hkv * windows * 2);  // below 2^31: checked on entry
  if (p.d == 64)
    fa_compact_fp8_gather_kernel<64><<<grid, kThreads, 0, stream>>>(p, windows);
  else
    fa_compact_fp8_gather_kernel<128><<<grid, kThreads, 0, stream>>>(p, windows);
  return cudaGetLastError();
}

}  // namespace fa
