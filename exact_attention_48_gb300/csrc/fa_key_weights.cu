// fa_key_weights.cu -- accumulated attention weight of each cached key:
//   w_j = w_in_j + sum over the query rows i (and the heads of the group)
//         that see key j of exp(scale q_i . k_j - lse_i).
// Plain form: one thread per key, the query rows broadcast from shared memory.

#include <cstdint>

#include "fa_cache.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 16;  // query rows staged at a time

template <int D>
__global__ void __launch_bounds__(128) fa_key_weights_kernel(const KeyWeightParams p) {
  __shared__ float sq[kRows][D];
  __shared__ float sl[kRows];
  const int blocks = (p.Nk + 127) / 128;
  const int bh = blockIdx.x / blocks, b = bh / p.Hkv, hk = bh % p.Hkv;
  const int j = (blockIdx.x % blocks) * 128 + threadIdx.x;
  const int len = cache_rows(p.cache_len, b, p.Nk);
  const bool on = j < len;
  uint32_t kr[D / 2];
  if (on) {
    const uint4 *src = reinterpret_cast<const uint4 *>(p.k + b * p.sk.b + hk * p.sk.h + j * p.sk.n);
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      const uint4 x = src[c];
      kr[4 * c] = x.x, kr[4 * c + 1] = x.y, kr[4 * c + 2] = x.z, kr[4 * c + 3] = x.w;
    }
  }
  float total = 0.0f;
  for (int g = 0; g < p.G; ++g) {
    const int h = hk * p.G + g;
    float head = 0.0f;
    for (int i0 = 0; i0 < p.Nq; i0 += kRows) {
      __syncthreads();
      for (int e = threadIdx.x; e < kRows * D; e += 128) {
        const int i = i0 + e / D;
        sq[e / D][e % D] =
            i < p.Nq ? __bfloat162float(p.q[b * p.sq.b + h * p.sq.h + i * p.sq.n + e % D]) * p.scale_log2 : 0.0f;
      }
      if (threadIdx.x < kRows && i0 + static_cast<int>(threadIdx.x) < p.Nq)
        sl[threadIdx.x] = p.lse[(static_cast<long long>(b) * p.H + h) * p.Nq + i0 + threadIdx.x] * kLog2e;
      __syncthreads();
      if (!on) continue;
      for (int r = 0; r < kRows && i0 + r < p.Nq; ++r) {
        if (sl[r] == -INFINITY || (p.causal && j > len - p.Nq + i0 + r)) continue;
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < D / 2; ++c) {
          s = fmaf(sq[r][2 * c], __uint_as_float(kr[c] << 16), s);
          s = fmaf(sq[r][2 * c + 1], __uint_as_float(kr[c] & 0xffff0000u), s);
        }
        head += ex2(s - sl[r]);
      }
    }
    total += head;
  }
  if (j < p.Nk) {
    const long long at = static_cast<long long>(bh) * p.Nk + j;
    const float before = p.w_in ? p.w_in[at] : 0.0f;
    p.w[at] = on ? before + total : before;
  }
}

}  // namespace

cudaError_t launch_key_weights(const KeyWeightParams &p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.B) * p.Hkv * ((p.Nk + 127) / 128);
  if (p.d == 64)
    fa_key_weights_kernel<64><<<grid, 128, 0, stream>>>(p);
  else
    fa_key_weights_kernel<128><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
