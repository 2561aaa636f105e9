// fa_cache_select.cu -- which rows of a cache to keep: the first rows, the
// most recent rows and, of the others, those with the greatest accumulated
// weight (ties to the lower row), in ascending order.
//
// Weights are compared as 32-bit keys in the order of the numbers (both
// zeros alike, every NaN below every number).  The key of the last row kept
// is found digit by digit from the top (11, 11 and 10 bits): a histogram of
// the digit over the rows that agree with the digits found so far, then a
// search from the top.  After it every row is above the edge, on it, or below;
// a thread marks both kinds in its stretch of up to 32 rows, a prefix sum over
// the threads gives the places, and the rows above and the first few on the
// edge are put in order in shared memory and written from there (straight from
// the threads, each into its own sector, the writes took 10000 cycles).
//
// A row list is a few KB to a few hundred, so latency bounds the call, not
// bytes: a CTA keeps the keys of up to 16384 rows in shared memory through all
// passes (two CTAs to an SM), and a longer list, or a list of more than 8192 rows
// where there are few, goes to a cluster of up to 8 CTAs, which read each other's histograms and counts through distributed
// shared memory.  Lists past 8 * 16384 rows are read again (from L2) in each
// pass.  The loops over the keys are short ones: every instruction of this
// kernel comes cold from memory (unrolled with the keys in registers the
// ordered pass alone took 12000 cycles).  Weights of one cache crowd into a few
// exponents, so the histogram has four copies that a warp's lanes share out;
// in a cluster two, which the passes take in turn so that one cluster barrier
// a pass is enough.  One warp searches: 64 coarse sums, then the 32 bins of
// one of them, so that little is read from other CTAs (all bins of all CTAs
// took 4700 cycles a pass).
// Measured on the device: B16 Hkv16 16384 rows to 8192 21 us (28 with all
// weights alike), 8 lists of 131072 to 16384 18 us, of 32768 12 us, 2 of 640 to
// 256 6 us.

#include <cooperative_groups.h>
#include <cstdint>

#include "fa_cache.h"

namespace fa {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelStretch = 32;                      // rows of a thread and step, at most
constexpr int kSelStep = kSelThreads * kSelStretch;  // rows of a CTA and step
constexpr int kSelBins = 2048;
constexpr int kSelCoarse = kSelBins / 32;
constexpr int kSelCopies = 4;
constexpr int kSelOneCta = 8192;                     // rows that one CTA does as fast as a cluster

__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);  // -0 becomes +0
  return (u >> 31) ? ~u : u | 0x80000000u;
}

struct SelectShared {
  int hist[kSelCopies][kSelBins];
  int coarse[2][kSelCoarse];         // sums of 32 bins, of this CTA; the passes take them in turn
  int warp_sum[2][kSelWarps];
  int count[2];                      // this CTA's rows above and on the edge
  int digit, rest;                   // what the search found
  uint32_t key[kSelStep];            // 16-byte pieces swizzled, see place(); then the rows to write
};

// Where row i of the step lies in the key array: a thread's stretch is eight
// 16-byte pieces, and swizzled by the thread they read without conflicts.
__device__ __forceinline__ int place(int i) {
  const int c = i >> 2;
  return ((c ^ ((c >> 3) & 7)) << 2) | (i & 3);
}

// Exclusive scan over the block's threads of a pair; *total: the sums.
__device__ __forceinline__ int2 block_scan(int2 v, SelectShared &s, int2 *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 n = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, n.x, o), y = __shfl_up_sync(0xffffffffu, n.y, o);
    if (lane >= o) n.x += x, n.y += y;
  }
  __syncthreads();  // warp_sum may still be read from the last scan
  if (lane == 31) s.warp_sum[0][warp] = n.x, s.warp_sum[1][warp] = n.y;
  __syncthreads();
  int2 t = make_int2(0, 0), before = t;
  for (int w = 0; w < kSelWarps; ++w) {
    if (w == warp) before = t;
    t.x += s.warp_sum[0][w];
    t.y += s.warp_sum[1][w];
  }
  *total = t;
  return make_int2(before.x + n.x - v.x, before.y + n.y - v.y);
}

// One warp, lane l holding the count of the l-th place from the top: the first
// place at which `rest` is reached, and what is left of rest before it.
__device__ __forceinline__ int search(int count, int *rest) {
  const int lane = threadIdx.x & 31;
  int incl = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  const int at = __ffs(__ballot_sync(0xffffffffu, incl >= *rest)) - 1;
  *rest -= __shfl_sync(0xffffffffu, incl - count, at);
  return at;
}

// CLUSTER: more than one CTA a list; LONG: the list does not fit the cluster's
// shared memory.
template <bool CLUSTER, bool LONG>
__global__ void __launch_bounds__(kSelThreads, 2) fa_cache_select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  SelectShared &s = *reinterpret_cast<SelectShared *>(smem);
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = CLUSTER ? static_cast<int>(cluster.num_blocks()) : 1;
  const int rank = CLUSTER ? static_cast<int>(cluster.block_rank()) : 0;
  const int bh = blockIdx.x / ranks, b = bh / p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = cache_rows(p.cache_len, b, p.Nk);
  int *kept = p.kept + static_cast<long long>(bh) * p.keep;
  if (bh % p.Hkv == 0 && rank == 0 && tid == 0) p.new_len[b] = min(len, p.keep);
  if (len <= p.keep) {  // (the same for the whole cluster)
    for (int i = rank * kSelThreads + tid; i < p.keep; i += ranks * kSelThreads) kept[i] = i < len ? i : -1;
    return;
  }
  const float *w = p.w + static_cast<long long>(bh) * p.Nk;
  const int lo = p.first, hi = len - p.recent, need = p.keep - p.first - p.recent;

  // this CTA's part of the list, [j0, j1)
  const int n = hi - lo;
  const int per = ((n + ranks - 1) / ranks + kSelThreads - 1) / kSelThreads * kSelThreads;
  const int j0 = min(lo + static_cast<long long>(rank) * per, static_cast<long long>(hi));
  const int j1 = min(static_cast<long long>(j0) + per, static_cast<long long>(hi));
  if (!LONG && need > 0) {
#pragma unroll 8
    for (int j = j0 + tid; j < j1; j += kSelThreads) s.key[place(j - j0)] = order_key(w[j]);
  }
  for (int i = rank * kSelThreads + tid; i < lo; i += ranks * kSelThreads) kept[i] = i;
  for (int i = rank * kSelThreads + tid; i < p.recent; i += ranks * kSelThreads) kept[p.keep - p.recent + i] = hi + i;
  if (need == 0) return;

  // the key of the last row kept: `edge` under `mask`, found from the top
  uint32_t edge = 0, mask = 0;
  int rest = need;  // rows to take among those that agree with edge so far
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t bins = pass == 2 ? 1024 : 2048;
    // the copies of this pass, and this lane's
    constexpr int kCopies = CLUSTER ? kSelCopies / 2 : kSelCopies;
    const int copy0 = CLUSTER ? kCopies * (pass & 1) : 0, turn = pass & 1;
    int *mine = s.hist[copy0 + (lane & (kCopies - 1))];
    for (int i = tid; i < kCopies * kSelBins / 4; i += kSelThreads)
      reinterpret_cast<int4 *>(s.hist[copy0])[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    auto count = [&](uint32_t key) {
      if ((key & mask) == edge) atomicAdd(&mine[(key >> shift) & (bins - 1)], 1);
    };
    if (LONG) {
#pragma unroll 4
      for (int j = j0 + tid; j < j1; j += kSelThreads) count(order_key(w[j]));
    } else {
#pragma unroll 2
      for (int i = tid * 4; i < j1 - j0; i += kSelThreads * 4) {
        const uint4 k = *reinterpret_cast<const uint4 *>(&s.key[place(i)]);
        count(k.x);
        if (i + 1 < j1 - j0) count(k.y);
        if (i + 2 < j1 - j0) count(k.z);
        if (i + 3 < j1 - j0) count(k.w);
      }
    }
    __syncthreads();
    // coarse sums: a warp a bin of 32 at a time
    for (int c = warp; c < kSelCoarse; c += kSelWarps) {
      int x = 0;
#pragma unroll
      for (int y = 0; y < kCopies; ++y) x += s.hist[copy0 + y][c * 32 + lane];
      x = __reduce_add_sync(0xffffffffu, x);
      if (lane == 0) s.coarse[turn][c] = x;
    }
    if (CLUSTER)
      cluster.sync();
    else
      __syncthreads();
    if (warp == 0) {  // from the top: the first digit at which `rest` rows are reached
      int2 c = make_int2(0, 0);  // this lane's two coarse sums, the upper one in y
      for (int r = 0; r < ranks; ++r) {
        const int *h = CLUSTER ? cluster.map_shared_rank(s.coarse[turn], r) : s.coarse[turn];
        const int2 v = *reinterpret_cast<const int2 *>(h + kSelCoarse - 2 - 2 * lane);
        c.x += v.x;
        c.y += v.y;
      }
      int left = rest;
      const int pair = search(c.x + c.y, &left);
      const int upper = __shfl_sync(0xffffffffu, c.y, pair);
      int at = kSelCoarse - 1 - 2 * pair;
      if (left > upper) {
        left -= upper;
        --at;
      }
      int f = 0;
      for (int r = 0; r < ranks; ++r) {
        const int *h = CLUSTER ? cluster.map_shared_rank(s.hist[copy0], r) : s.hist[copy0];
#pragma unroll
        for (int y = 0; y < kCopies; ++y) f += h[y * kSelBins + at * 32 + 31 - lane];
      }
      const int bin = search(f, &left);
      if (lane == 0) {
        s.digit = at * 32 + 31 - bin;
        s.rest = left;
      }
    }
    __syncthreads();
    edge |= static_cast<uint32_t>(s.digit) << shift;
    mask |= (bins - 1) << shift;
    rest = s.rest;
  }

  // The rows above the edge and on it in a thread's stretch of the step at
  // `base`, as bits; *first: the stretch's first row.
  auto marks = [&](int base, int *first) {
    const int rows = min(j1 - base, kSelStep);
    const int each = (rows + 4 * kSelThreads - 1) / (4 * kSelThreads) * 4;  // whole pieces, all threads at work
    const int i0 = tid * each, i1 = min(i0 + each, rows);
    uint2 m = make_uint2(0u, 0u);
#pragma unroll 2
    for (int i = i0; i < i1; i += 4) {
      uint32_t k[4];
      if (LONG) {
#pragma unroll
        for (int y = 0; y < 4; ++y) k[y] = i + y < i1 ? order_key(w[base + i + y]) : 0u;
      } else {
        const uint4 v = *reinterpret_cast<const uint4 *>(&s.key[place(i)]);
        k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        if (i + y >= i1) break;
        m.x |= static_cast<uint32_t>(k[y] > edge) << (i - i0 + y);
        m.y |= static_cast<uint32_t>(k[y] == edge) << (i - i0 + y);
      }
    }
    *first = base + i0;
    return m;
  };

  // rows above the edge and on it in the parts before this one
  int2 seen = make_int2(0, 0);
  if (CLUSTER) {
    int2 c = make_int2(0, 0);
    for (int base = j0; base < j1; base += kSelStep) {
      int first;
      const uint2 m = marks(base, &first);
      c.x += __popc(m.x);
      c.y += __popc(m.y);
    }
    int2 total;
    block_scan(c, s, &total);
    if (tid == 0) s.count[0] = total.x, s.count[1] = total.y;
    cluster.sync();
    int2 x = make_int2(0, 0);
    if (lane < rank) {
      const int *y = cluster.map_shared_rank(s.count, lane);
      x = make_int2(y[0], y[1]);
    }
    seen.x = __reduce_add_sync(0xffffffffu, x.x);
    seen.y = __reduce_add_sync(0xffffffffu, x.y);
    cluster.sync();  // no CTA leaves while another reads its counts
  }
  // in order: row j goes to place (rows above before j) + min(rows on the edge before j, rest)
  for (int base = j0; base < j1; base += kSelStep) {
    int first;
    const uint2 m = marks(base, &first);
    int2 total;
    const int2 before = block_scan(make_int2(__popc(m.x), __popc(m.y)), s, &total);
    // (block_scan's barriers: every thread has read its keys, their array now
    // takes the rows)
    int a = before.x, o = seen.y + before.y;
    const int o0 = min(seen.y, rest);
    for (uint32_t left = m.x | m.y; left; left &= left - 1) {
      const int i = __ffs(left) - 1;
      const bool above = (m.x >> i) & 1u;
      if (above || o < rest) s.key[a + min(o, rest) - o0] = first + i;
      a += above;
      o += !above;
    }
    __syncthreads();
    const int out = total.x + min(seen.y + total.y, rest) - o0;
    int *dst = kept + lo + seen.x + o0;
    for (int i = tid; i < out; i += kSelThreads) dst[i] = static_cast<int>(s.key[i]);
    __syncthreads();
    seen.x += total.x;
    seen.y += total.y;
  }
}

template <bool CLUSTER, bool LONG>
cudaError_t launch_select(const SelectParams &p, int ranks, cudaStream_t stream) {
  auto kern = fa_cache_select_kernel<CLUSTER, LONG>;
  const int smem = static_cast<int>(sizeof(SelectShared));
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.Hkv * ranks);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_cache_select(const SelectParams &p, cudaStream_t stream) {
  // the smallest cluster whose shared memory holds the list
  const int n = p.Nk - p.first - p.recent;
  int ranks = 1;
  while (ranks < 8 && n > ranks * kSelStep) ranks *= 2;
  // and a larger one for long lists that would leave SMs idle (8 lists of 32768
  // rows in clusters of 2 18.0 us, of 8 12.2; 16 and 32 of 16384 in one CTA each
  // 13.6, in 8 and 4 11.8 and 12.0; 2 of 8192 the same in 1 and in 8, 9.9, and
  // slower in 2, 11.7)
  const long long lists = static_cast<long long>(p.B) * p.Hkv;
  while (ranks < 8 && n > kSelOneCta && lists * ranks * 2 <= 152) ranks *= 2;
  if (ranks == 1) return launch_select<false, false>(p, ranks, stream);
  return n > ranks * kSelStep ? launch_select<true, true>(p, ranks, stream)
                              : launch_select<true, false>(p, ranks, stream);
}

}  // namespace fa
