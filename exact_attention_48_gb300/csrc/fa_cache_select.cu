// fa_cache_select.cu -- which rows of a cache to keep: the first rows, the
// most recent rows and, of the others, those with the greatest accumulated
// weight (ties to the lower row), in ascending order.
//
// Weights are compared as 32-bit keys in the order of the numbers (both
// zeros alike, every NaN below every number).  Plain form: one CTA per head,
// the key of the last row kept found bit by bit, then one ordered pass.

#include <cstdint>

#include "fa_cache.h"

namespace fa {
namespace {

constexpr int kSelThreads = 512;

__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);  // -0 becomes +0
  return (u >> 31) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int block_sum(int x, int *sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if (lane == 0) sh[warp] = x;
  __syncthreads();
  int s = 0;
  for (int w = 0; w < kSelThreads / 32; ++w) s += sh[w];
  return s;
}

__global__ void __launch_bounds__(kSelThreads) fa_cache_select_kernel(const SelectParams p) {
  __shared__ int sh[kSelThreads / 32], run[3];
  const int bh = blockIdx.x, b = bh / p.Hkv;
  const int len = cache_rows(p.cache_len, b, p.Nk);
  int *kept = p.kept + static_cast<long long>(bh) * p.keep;
  if (bh % p.Hkv == 0 && threadIdx.x == 0) p.new_len[b] = min(len, p.keep);
  if (len <= p.keep) {
    for (int i = threadIdx.x; i < p.keep; i += kSelThreads) kept[i] = i < len ? i : -1;
    return;
  }
  const float *w = p.w + static_cast<long long>(bh) * p.Nk;
  const int lo = p.first, hi = len - p.recent, need = p.keep - p.first - p.recent;
  for (int i = threadIdx.x; i < lo; i += kSelThreads) kept[i] = i;
  for (int i = threadIdx.x; i < p.recent; i += kSelThreads) kept[p.keep - p.recent + i] = hi + i;
  // the greatest key that at least `need` rows reach
  uint32_t edge = 0;
  for (int bit = 31; bit >= 0 && need > 0; --bit) {
    const uint32_t cand = edge | (1u << bit);
    int n = 0;
    for (int j = lo + threadIdx.x; j < hi; j += kSelThreads) n += order_key(w[j]) >= cand;
    if (block_sum(n, sh) >= need) edge = cand;
  }
  int above = 0;
  for (int j = lo + threadIdx.x; j < hi && need > 0; j += kSelThreads) above += order_key(w[j]) > edge;
  const int ties = need - block_sum(above, sh);  // rows at the edge to keep, the lowest ones
  if (threadIdx.x == 0) run[0] = run[1] = 0;
  for (int j0 = lo; j0 < hi && need > 0; j0 += 32) {  // in order, one warp
    if (threadIdx.x >= 32) break;
    __syncwarp();
    const int j = j0 + threadIdx.x;
    const uint32_t key = j < hi ? order_key(w[j]) : 0u;
    const bool tie = j < hi && key == edge;
    const unsigned mt = __ballot_sync(0xffffffffu, tie), below = (1u << threadIdx.x) - 1u;
    const bool take = j < hi && (key > edge || (tie && run[1] + __popc(mt & below) < ties));
    const unsigned mk = __ballot_sync(0xffffffffu, take);
    if (take) kept[lo + run[0] + __popc(mk & below)] = j;
    __syncwarp();
    if (threadIdx.x == 0) run[0] += __popc(mk), run[1] += __popc(mt);
  }
}

}  // namespace

cudaError_t launch_cache_select(const SelectParams &p, cudaStream_t stream) {
  fa_cache_select_kernel<<<p.B * p.Hkv, kSelThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
