// fa_cache_compact.cu -- rows of a key/value cache (and their weights) moved
// together: row base + i becomes the old row base + kept[i].
//
// In place a destination row may be a source of an earlier destination only
// (kept ascends, so kept[i] >= i): one CTA per head takes the rows in order,
// a chunk at a time, and every row of a chunk is read before any is written.

#include <cstdint>

#include "fa_cache.h"

namespace fa {
namespace {

constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) fa_cache_compact_kernel(const CompactParams p) {
  const int bh = blockIdx.x, b = bh / p.Hkv, h = bh % p.Hkv;
  const int per_row = p.d / 8;  // 16-byte pieces of a row
  const int rows = kMoveThreads / per_row, c = threadIdx.x % per_row;
  const int *kept = p.kept + b * p.kept_b + h * p.kept_h;
  const long long base = p.base ? p.base[b] : 0;
  for (int i0 = 0; i0 < p.M; i0 += rows) {
    const int i = i0 + static_cast<int>(threadIdx.x) / per_row;
    const int from = i < p.M ? kept[i] : -1;
    const long long src = base + from, dst = base + i;
    const bool on = from >= 0 && src >= 0 && src < p.Nk && dst >= 0 && dst < p.Nout;
    uint4 kx, vx;
    float wx = 0.0f;
    if (on) {
      kx = *reinterpret_cast<const uint4 *>(p.k + b * p.sk.b + h * p.sk.h + src * p.sk.n + c * 8);
      vx = *reinterpret_cast<const uint4 *>(p.v + b * p.sv.b + h * p.sv.h + src * p.sv.n + c * 8);
      if (p.w && c == 0) wx = p.w[static_cast<long long>(bh) * p.Nk + src];
    }
    __syncthreads();
    if (on) {
      *reinterpret_cast<uint4 *>(p.ko + b * p.sko.b + h * p.sko.h + dst * p.sko.n + c * 8) = kx;
      *reinterpret_cast<uint4 *>(p.vo + b * p.svo.b + h * p.svo.h + dst * p.svo.n + c * 8) = vx;
      if (p.w && c == 0) p.wo[static_cast<long long>(bh) * p.Nout + dst] = wx;
    }
  }
}

}  // namespace

cudaError_t launch_cache_compact(const CompactParams &p, cudaStream_t stream) {
  fa_cache_compact_kernel<<<p.B * p.Hkv, kMoveThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
