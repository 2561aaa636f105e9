// fa_tree_fp8.cu -- attention of the newest rows of each sequence, or of a tree
// of drafted tokens, over a cache held in 8 bits: the choice of a kernel
// (fa_tree_fp8_tc.cu, fa_tree_fp8_rows.cu), and the merging of what the runs' ends cut.

#include <cstdint>

#include "fa_cache8.h"
#include "fa_runs.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kModelCtas = 152;                // GB300's SMs: the grid the runs are cut for
constexpr float kLn2 = 0.69314718055994530942f;

// Merge the partial results of units cut by a run's end:
//   O = sum 2^(lse_s - M) O_s / sum 2^(lse_s - M).
// (O_s up to bf16's greatest, of at most 152 runs: added up as 2^-8 of themselves.)
// WARPS warps take one row of one cut unit, dealing the runs out among themselves
// (a run's row is one coalesced read) and adding up in a fixed order: eight where a
// unit is cut into many runs, one where it is cut into two or three (B16 H16 Nt32:
// 4864 rows, 15 us with eight).
constexpr int kMergeWarps = 8;
constexpr float kAddAs = 0.00390625f;

// +inf, the mark of padding, before NaN, and NaN before every other value.
__device__ __forceinline__ float merge_max(float a, float b) {
  const float x = fmaxf(a, b);
  return x != INFINITY && (a != a || b != b) ? NAN : x;
}

template <int D, int WARPS>
__global__ void __launch_bounds__(kMergeWarps * 32) fa_tree_fp8_merge_kernel(const Tree8Params p, int total) {
  constexpr int kCols = D / 32;
  __shared__ float sh_m[WARPS], sh_l[WARPS], sh_o[WARPS][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit_rows = p.G * p.Nt, rows = p.rows;
  const int at_row = WARPS == 1 ? blockIdx.x * kMergeWarps + warp : blockIdx.x, w0 = WARPS == 1 ? 0 : warp;
  if (at_row >= total) return;
  const int r = at_row % unit_rows, x = at_row / unit_rows;
  cudaGridDependencySynchronize();  // (launched while the main kernel still runs)
  const int4 cut = p.cuts[x];
  const int b = cut.x, hk = cut.y, first = cut.z, last = cut.w;
  // nothing was cut here (b = -1); after a timeout the entry may hold anything
  if (b < 0 || b >= p.B || hk < 0 || hk >= p.Hkv || first < 0 || first >= last || last >= p.ranges) return;
  const int group = r / rows, lr = r % rows;
  float m = -INFINITY, l = 0.0f, o[kCols];
#pragma unroll
  for (int y = 0; y < kCols; ++y) o[y] = 0.0f;
#pragma unroll 2
  for (int run = first + w0; run <= last; run += WARPS) {
    const long long at = ((static_cast<long long>(run) * p.groups + group) * 2 + (run == first ? 1 : 0)) * rows + lr;
    const float s = p.part_lse[at];
    float v[kCols];
#pragma unroll
    for (int y = 0; y < kCols; ++y) v[y] = p.part_o[at * D + y * 32 + lane];
    const float mn = merge_max(m, s);
    const float fa = m == mn ? 1.0f : (m == -INFINITY ? 0.0f : ex2(m - mn));
    const float fb = s == -INFINITY ? 0.0f : (s == mn ? 1.0f : ex2(s - mn));
    const float fo = fb * kAddAs;
    l = l * fa + fb;
#pragma unroll
    for (int y = 0; y < kCols; ++y) o[y] = o[y] * fa + v[y] * fo;
    m = mn;
  }
  const int node = r % p.Nt, h = hk * p.G + r / p.Nt;
  __nv_bfloat16 *dst = p.o + b * p.so.b + h * p.so.h + node * p.so.n;
  float *lse = p.lse + (static_cast<long long>(b) * p.H + h) * p.Nt + node;
  if constexpr (WARPS == 1) {
    const bool any = m != -INFINITY && m != INFINITY;  // +inf: padding
#pragma unroll
    for (int y = 0; y < kCols; ++y) dst[y * 32 + lane] = __float2bfloat16(any ? o[y] / l * (1.0f / kAddAs) : 0.0f);
    if (lane == 0) *lse = any ? (m + log2f(l)) * kLn2 : -INFINITY;
    return;
  }
  if (lane == 0) {
    sh_m[w0] = m;
    sh_l[w0] = l;
  }
#pragma unroll
  for (int y = 0; y < kCols; ++y) sh_o[w0][y * 32 + lane] = o[y];
  __syncthreads();
  if (threadIdx.x >= D) return;
  float M = -INFINITY;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) M = merge_max(M, sh_m[w]);
  float sum = 0.0f, out = 0.0f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const float mw = sh_m[w], f = mw == -INFINITY ? 0.0f : (mw == M ? 1.0f : ex2(mw - M));
    sum += sh_l[w] * f;
    out += sh_o[w][threadIdx.x] * f;
  }
  const bool any = M != -INFINITY && M != INFINITY;
  dst[threadIdx.x] = __float2bfloat16(any ? out / sum * (1.0f / kAddAs) : 0.0f);
  if (threadIdx.x == 0) *lse = any ? (M + log2f(sum)) * kLn2 : -INFINITY;
}

template <int D>
cudaError_t launch_merge8(const Tree8Params &p, cudaStream_t stream) {
  const long long cuts = p.cuts_by_unit ? static_cast<long long>(p.B) * p.Hkv : p.ranges;  // at most 152
  const bool many = p.ranges >= 4ll * p.B * p.Hkv;  // a unit is cut into about ranges / units + 1 runs
  const int rows = static_cast<int>(cuts * p.G * p.Nt);  // (at most 152 runs a group of rows: below 2^24)
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(many ? rows : (rows + kMergeWarps - 1) / kMergeWarps));
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return many ? cudaLaunchKernelEx(&cfg, fa_tree_fp8_merge_kernel<D, kMergeWarps>, p, rows)
              : cudaLaunchKernelEx(&cfg, fa_tree_fp8_merge_kernel<D, 1>, p, rows);
}

}  // namespace

// Short caches are not cut inside a unit: see plan_tree.
constexpr int kWholeTiles = 8;

// Rows of a group (a CTA's): 8, 16 or 32 as columns of the transposed products
// (fa_tree_fp8_tc.cu), or 128 as lanes (fa_tree_fp8_rows.cu), which cost the same
// however many are used.  The forms on the same calls, us:
//                                       columns         lanes
//   B16 H16 T1 Nk16384, d = 128             162 (8)     254
//                                           168 (16)
//                       d = 64              110 (8)     224
//                                           135 (16)
//   B2 H32 Hkv8 T5 Nk100001, d = 128         86 (32)    114
//                            d = 64          82 (32)     96
//   B16 H16 T32 Nk16384, d = 128            207 (32)    264
//                        d = 64             187 (32)    224
//   B2 H32 Hkv8 T64 Nk65536, d = 128        405 (64)    157
// Runs: as many as fill the SMs with a CTA for each of the unit's groups.  77 to 151 groups
// (9729 query rows of a cache head and more) make one run, and leave up to half of the
// SMs without a CTA; not measured.
Tree8Plan plan_tree8(int B, int H, int Hkv, int Nt, int Nk, int d) {
  Tree8Plan pl{};
  const int rows = H / Hkv * Nt;  // (below 2^31: H < 2^24, Nt <= 128)
  pl.rows = rows <= 8 ? 8 : (rows <= 16 ? 16 : (rows <= 32 ? 32 : 128));
  pl.groups = (rows + pl.rows - 1) / pl.rows;
  const int per_unit = (Nk + kKeys - 1) / kKeys;
  const long long units = static_cast<long long>(B) * Hkv;
  pl.whole = per_unit <= kWholeTiles ? 1 : 0;
  const long long pieces = pl.whole ? units : units * per_unit;
  long long ranges = kModelCtas / pl.groups;
  if (ranges < 1) ranges = 1;
  if (ranges > pieces) ranges = pieces;
  pl.ranges = static_cast<int>(ranges);
  pl.merge = ranges > 1 && !pl.whole;
  pl.part_rows = pl.merge ? static_cast<size_t>(ranges) * pl.groups * 2 * pl.rows : 0;
  return pl;
}

cudaError_t launch_tree8(const CUtensorMap &tk, const CUtensorMap &tv, const Tree8Params &p, bool merge,
                         cudaStream_t stream) {
  const cudaError_t e = p.rows <= 32 ? launch_tree8_tc(tk, tv, p, stream) : launch_tree8_rows(tk, tv, p, stream);
  if (e != cudaSuccess || !merge) return e;
  return p.d == 128 ? launch_merge8<128>(p, stream) : launch_merge8<64>(p, stream);
}

}  // namespace fa
