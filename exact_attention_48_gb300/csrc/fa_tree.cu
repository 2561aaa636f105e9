// fa_tree.cu -- attention of a tree of drafted tokens over a key/value cache.
//
// Row i of the tree sees the cache rows before the tree, its own row and its
// ancestors' rows.  Plain form: one warp per query row walks the keys it
// sees with a running maximum and sum, a lane owns d / 32 columns.

#include <cstdint>

#include "fa_cache.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;

template <int D>
__global__ void __launch_bounds__(128) fa_tree_kernel(const TreeParams p) {
  constexpr int CPL = D / 32;
  const int lane = threadIdx.x & 31;
  const long long rows = static_cast<long long>(p.B) * p.H * p.Nt;
  const long long r = blockIdx.x * 4ll + (threadIdx.x >> 5);
  if (r >= rows) return;
  const int i = static_cast<int>(r % p.Nt), bh = static_cast<int>(r / p.Nt), b = bh / p.H, h = bh % p.H, hk = h / p.G;
  const int len = cache_rows(p.cache_len, b, p.Nk), base = len - p.Nt;
  uint32_t seen[4] = {0, 0, 0, 0};
  bool live = base + i >= 0;
  for (int x = i; live && x >= 0;) {
    seen[x >> 5] |= 1u << (x & 31);
    const int up = p.parents[b * p.par_b + x];
    live = up >= -1 && up < x && (up < 0 || base + up >= 0);
    x = up;
  }
  float q[CPL], o[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    q[c] = __bfloat162float(p.q[b * p.sq.b + h * p.sq.h + i * p.sq.n + lane * CPL + c]) * p.scale_log2;
    o[c] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  const int end = live ? len : 0;
  for (int j = 0; j < end; ++j) {
    const int node = j - base;
    if (node >= 0 && !((seen[node >> 5] >> (node & 31)) & 1u)) continue;
    const __nv_bfloat16 *kr = p.k + b * p.sk.b + hk * p.sk.h + j * p.sk.n + lane * CPL;
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < CPL; ++c) s += q[c] * __bfloat162float(kr[c]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s), a = ex2(m - mn), w = ex2(s - mn);
    l = l * a + w;
    const __nv_bfloat16 *vr = p.v + b * p.sv.b + hk * p.sv.h + j * p.sv.n + lane * CPL;
#pragma unroll
    for (int c = 0; c < CPL; ++c) o[c] = o[c] * a + w * __bfloat162float(vr[c]);
    m = mn;
  }
#pragma unroll
  for (int c = 0; c < CPL; ++c)
    p.o[b * p.so.b + h * p.so.h + i * p.so.n + lane * CPL + c] = __float2bfloat16_rn(l > 0.0f ? o[c] / l : 0.0f);
  if (lane == 0) p.lse[r] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

cudaError_t launch_tree(const TreeParams &p, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.B) * p.H * p.Nt;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  if (p.d == 64)
    fa_tree_kernel<64><<<grid, 128, 0, stream>>>(p);
  else
    fa_tree_kernel<128><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
