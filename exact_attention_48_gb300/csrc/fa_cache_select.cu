// fa_cache_select.cu -- which rows of a cache to keep: the first rows, the
// most recent rows and, of the others, those with the greatest accumulated
// weight (ties to the lower row), in ascending order.
//
// Weights are compared as 32-bit keys in the order of the numbers (both
// zeros alike, every NaN below every number).  The key of the last row kept
// is found digit by digit from the top (11, 11 and 10 bits): a histogram of
// the digit over the rows that agree with the digits found so far, then a
// scan from the top.  After it every row is above the edge, on it, or below;
// the rows above and the first few on the edge are written in order by
// prefix counts of both.
//
// A row list is a few KB to a few hundred, so latency bounds the call, not
// bytes: a thread keeps its keys in registers through all passes (16 of
// them, 16384 a CTA), and a longer list goes to a cluster of up to 8 CTAs,
// which add their histograms and exchange their counts through distributed
// shared memory.  Lists past 8 * 16384 rows are read again (from L2) in each
// pass.

#include <cooperative_groups.h>
#include <cstdint>

#include "fa_cache.h"

namespace fa {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelKeys = 16;                       // keys per thread and step
constexpr int kSelStep = kSelThreads * kSelKeys;   // keys per CTA and step
constexpr int kSelBins = 2048;

__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);  // -0 becomes +0
  return (u >> 31) ? ~u : u | 0x80000000u;
}

struct SelectShared {
  int hist[kSelBins];
  int sum[kSelBins];                 // cluster totals
  int above[kSelKeys * kSelWarps];   // per (step row, warp): rows above the edge, on it; then their prefixes
  int on[kSelKeys * kSelWarps];
  int warp_sum[2][kSelWarps];
  int count[2];                      // this CTA's rows above and on the edge
  int digit, rest;                   // what the scan found
};

// Inclusive scan over the block's threads of a pair; *total: the sums.
__device__ __forceinline__ int2 block_scan(int2 v, SelectShared &s, int2 *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) v.x += x, v.y += y;
  }
  __syncthreads();  // warp_sum may still be read from the last scan
  if (lane == 31) s.warp_sum[0][warp] = v.x, s.warp_sum[1][warp] = v.y;
  __syncthreads();
  int x = s.warp_sum[0][lane], y = s.warp_sum[1][lane];  // kSelWarps = 32: a lane per warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += a, y += b;
  }
  const int bx = __shfl_sync(0xffffffffu, x, warp > 0 ? warp - 1 : 0);
  const int by = __shfl_sync(0xffffffffu, y, warp > 0 ? warp - 1 : 0);
  if (warp > 0) v.x += bx, v.y += by;
  *total = make_int2(__shfl_sync(0xffffffffu, x, 31), __shfl_sync(0xffffffffu, y, 31));
  return v;
}

// LONG: the list does not fit the cluster's registers.
template <bool LONG>
__global__ void __launch_bounds__(kSelThreads, 1) fa_cache_select_kernel(const SelectParams p) {
  __shared__ SelectShared s;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
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
  for (int i = rank * kSelThreads + tid; i < lo; i += ranks * kSelThreads) kept[i] = i;
  for (int i = rank * kSelThreads + tid; i < p.recent; i += ranks * kSelThreads) kept[p.keep - p.recent + i] = hi + i;
  if (need == 0) return;

  // this CTA's part of the list, [j0, j1)
  const int n = hi - lo;
  const int per = ((n + ranks - 1) / ranks + kSelThreads - 1) / kSelThreads * kSelThreads;
  const int j0 = min(lo + static_cast<long long>(rank) * per, static_cast<long long>(hi));
  const int j1 = min(static_cast<long long>(j0) + per, static_cast<long long>(hi));
  uint32_t key[kSelKeys];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {
      const int j = base + i * kSelThreads + tid;
      key[i] = j < j1 ? order_key(w[j]) : 0u;
    }
  };
  if (!LONG) load(j0);

  // the key of the last row kept: `edge` under `mask`, found from the top
  uint32_t edge = 0, mask = 0;
  int rest = need;  // rows to take among those that agree with edge so far
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t bins = pass == 2 ? 1024 : 2048;
    for (int i = tid; i < kSelBins; i += kSelThreads) s.hist[i] = 0;
    __syncthreads();
    for (int base = j0; base < j1; base += kSelStep) {
      if (LONG) load(base);
#pragma unroll
      for (int i = 0; i < kSelKeys; ++i) {
        const int j = base + i * kSelThreads + tid;
        const bool in = j < j1 && (key[i] & mask) == edge;
        const uint32_t digit = (key[i] >> shift) & (bins - 1);
        // rows that are all alike (a cache nobody has looked at) add once per warp
        const unsigned who = __ballot_sync(0xffffffffu, in);
        if (who == 0) continue;
        const uint32_t lead = __shfl_sync(0xffffffffu, digit, __ffs(who) - 1);
        if (__all_sync(0xffffffffu, !in || digit == lead)) {
          if (lane == 0) atomicAdd(&s.hist[lead], __popc(who));
        } else if (in) {
          atomicAdd(&s.hist[digit], 1);
        }
      }
    }
    const int *sum = s.hist;
    if (ranks > 1) {
      cluster.sync();
      // each CTA adds its share of the bins and gives everyone the result
      const int share = kSelBins / ranks;
      for (int i = tid; i < share; i += kSelThreads) {
        const int bin = rank * share + i;
        int t = 0;
        for (int r = 0; r < ranks; ++r) t += cluster.map_shared_rank(s.hist, r)[bin];
        for (int r = 0; r < ranks; ++r) cluster.map_shared_rank(s.sum, r)[bin] = t;
      }
      cluster.sync();
      sum = s.sum;
    } else {
      __syncthreads();
    }
    // from the top: the first digit at which `rest` rows are reached
    const int hi_bin = kSelBins - 1 - 2 * tid;
    const int c1 = sum[hi_bin], c0 = sum[hi_bin - 1];
    int2 total;
    const int upto = block_scan(make_int2(c1 + c0, 0), s, &total).x;  // rows in this thread's bins and above
    const int before = upto - c1 - c0;
    if (before < rest && upto >= rest) {  // exactly one thread
      const bool first = before + c1 >= rest;
      s.digit = first ? hi_bin : hi_bin - 1;
      s.rest = rest - before - (first ? 0 : c1);
    }
    __syncthreads();
    edge |= static_cast<uint32_t>(s.digit) << shift;
    mask |= (bins - 1) << shift;
    rest = s.rest;
    __syncthreads();
  }

  // rows above the edge and on it in the parts before this one
  int2 seen = make_int2(0, 0);
  if (ranks > 1) {
    int2 mine = make_int2(0, 0);
    for (int base = j0; base < j1; base += kSelStep) {
      if (LONG) load(base);
#pragma unroll
      for (int i = 0; i < kSelKeys; ++i) {
        const bool in = base + i * kSelThreads + tid < j1;
        mine.x += in && key[i] > edge;
        mine.y += in && key[i] == edge;
      }
    }
    int2 total;
    block_scan(mine, s, &total);
    if (tid == 0) s.count[0] = total.x, s.count[1] = total.y;
    cluster.sync();
    for (int r = 0; r < rank; ++r) {
      const int *c = cluster.map_shared_rank(s.count, r);
      seen.x += c[0];
      seen.y += c[1];
    }
    cluster.sync();  // no CTA leaves while another reads its counts
  }
  // in order: row j goes to place (rows above before j) + min(rows on the edge before j, rest)
  for (int base = j0; base < j1; base += kSelStep) {
    if (LONG) load(base);
    unsigned ba[kSelKeys], bo[kSelKeys];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {
      const bool in = base + i * kSelThreads + tid < j1;
      ba[i] = __ballot_sync(0xffffffffu, in && key[i] > edge);
      bo[i] = __ballot_sync(0xffffffffu, in && key[i] == edge);
      if (lane == 0) {
        s.above[i * kSelWarps + warp] = __popc(ba[i]);
        s.on[i * kSelWarps + warp] = __popc(bo[i]);
      }
    }
    __syncthreads();
    constexpr int kEntries = kSelKeys * kSelWarps;  // 512, a thread each
    const int2 v = tid < kEntries ? make_int2(s.above[tid], s.on[tid]) : make_int2(0, 0);
    int2 total;
    const int2 incl = block_scan(v, s, &total);
    if (tid < kEntries) {
      s.above[tid] = incl.x - v.x;
      s.on[tid] = incl.y - v.y;
    }
    __syncthreads();
    const unsigned below = (1u << lane) - 1u;
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {
      const int a = seen.x + s.above[i * kSelWarps + warp] + __popc(ba[i] & below);
      const int o = seen.y + s.on[i * kSelWarps + warp] + __popc(bo[i] & below);
      const bool take = ((ba[i] >> lane) & 1u) || (((bo[i] >> lane) & 1u) && o < rest);
      if (take) kept[lo + a + min(o, rest)] = base + i * kSelThreads + tid;
    }
    seen.x += total.x;
    seen.y += total.y;
  }
}

template <bool LONG>
cudaError_t launch_select(const SelectParams &p, int ranks, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.Hkv * ranks);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_cache_select_kernel<LONG>, p);
}

}  // namespace

cudaError_t launch_cache_select(const SelectParams &p, cudaStream_t stream) {
  // the smallest cluster whose registers hold the list
  const int n = p.Nk - p.first - p.recent;
  int ranks = 1;
  while (ranks < 8 && n > ranks * kSelStep) ranks *= 2;
  return n > ranks * kSelStep ? launch_select<true>(p, ranks, stream) : launch_select<false>(p, ranks, stream);
}

}  // namespace fa
