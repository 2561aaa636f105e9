// fa_verify.cu -- drafted tokens verified against the target's probabilities.
//
// At node n the children are tried in order.  R is what they have left of the
// target's row p_n and S its sum (R = p_n, S = 1 before the first one); child i
// with token x is accepted if u_i q(x) S < R(x), else
//     R <- max(R - S q, 0),  S <- sum R,
// with q the draft's row at n (or, without one, certainty of x).  Where no child
// is left, the next token is the first y with R(0) + .. + R(y) > u_0 sum R (of
// p_n, should R be zero).
//
// What bounds it.  The tests need single values, which all nodes' threads fetch at
// once; the sums need a row of p (and of q) where a sibling is left to try, and one
// for the next token: a few dependent passes over a row.  A sequence's row is cut
// over a cluster of CTAs, which add their sums through distributed shared memory;
// S is kept by all of them and they take the same decisions.
//
// Precision.  Which token a number falls on is decided by a sum over the whole
// vocabulary, so R and S are pairs of fp32 (hi + lo, about 48 bits): fp64 runs at
// a sixty-fourth of the fp32 rate here, and a row in it would take longer than
// its memory traffic.  The few comparisons are in fp64.

#include <cooperative_groups.h>
#include <cstdint>

#include "fa_cache8.h"

namespace cg = cooperative_groups;

namespace fa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxNodes = 128, kMaxRanks = 8;
constexpr int kUnroll = 8;
constexpr int kTile = 32 * kUnroll;   // least elements of a warp's tile
constexpr int kMaxTiles = 2048;       // tiles of a CTA's share of a row

// A number as the sum of two fp32, |lo| at most half a unit of hi's last place.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ double value(Pair a) { return static_cast<double>(a.hi) + a.lo; }
__device__ __forceinline__ Pair quick_sum(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return Pair{s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), z = __fsub_rn(s, a);
  return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return quick_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
// r - s q, or 0 if that is less.
__device__ __forceinline__ Pair less(Pair r, Pair s, float q) {
  const float ph = __fmul_rn(s.hi, q), pl = __fmaf_rn(s.hi, q, -ph);
  const Pair p = quick_sum(ph, __fmaf_rn(s.lo, q, pl));
  const Pair d = two_sum(r.hi, -p.hi);
  const Pair x = quick_sum(d.hi, __fadd_rn(d.lo, __fsub_rn(r.lo, p.lo)));
  return x.hi > 0.0f ? x : Pair{0.0f, 0.0f};
}

struct Shared {
  int parent[kMaxNodes], token[kMaxNodes];
  float u[kMaxNodes], p[kMaxNodes], q[kMaxNodes];  // the node's number, and its token's p and q at its parent
  int rejected[kMaxNodes];                         // tokens rejected at the node being worked on
  Pair sums[kMaxNodes];                            // S before the first, the second, ... child
  Pair tile[kMaxTiles];                            // this CTA's sums of R
  Pair warp[kWarps];
  Pair rank[kMaxRanks];                            // every CTA's sum
  double scan[kWarps];
  int found, last;
};

// R(y) after the first k children of a node.
__device__ __forceinline__ Pair rest(const Shared &s, int k, float p, float q, int y, bool drafted) {
  Pair r{p > 0.0f ? p : 0.0f, 0.0f};
  for (int j = 0; j < k; ++j) r = less(r, s.sums[j], drafted ? q : (y == s.rejected[j] ? 1.0f : 0.0f));
  return r;
}

__global__ void __launch_bounds__(kThreads) fa_verify_kernel(const VerifyParams p) {
  __shared__ Shared s;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = p.ranks, rank = blockIdx.x % ranks, b = blockIdx.x / ranks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool drafted = p.draft != nullptr;
  // this CTA's share of a row, and the warps' tiles in it
  const int share = (p.V + ranks - 1) / ranks;
  const int v0 = min(p.V, rank * share), v1 = min(p.V, v0 + share);
  const int per_tile = kTile * ((share + kTile * kMaxTiles - 1) / (kTile * kMaxTiles));
  const int tiles = (v1 - v0 + per_tile - 1) / per_tile;
  const float *target = p.target + b * p.tb, *draft = drafted ? p.draft + b * p.db : nullptr;

  if (tid < p.Nt) {
    const int up = p.parents[b * p.par_b + tid], x = p.tokens[b * p.tok_b + tid];
    const bool asks = tid > 0 && up >= 0 && up < tid && x >= 0 && x < p.V;
    s.parent[tid] = tid == 0 ? up : (asks ? up : -2);
    s.token[tid] = x;
    s.u[tid] = p.uniforms[b * p.uni_b + tid];
    s.p[tid] = asks ? target[up * p.tn + x] : 0.0f;
    s.q[tid] = asks ? (drafted ? draft[up * p.dn + x] : 1.0f) : 0.0f;
  }
  if (tid == 0) s.sums[0] = Pair{1.0f, 0.0f};
  __syncthreads();
  if (s.parent[0] != -1) {  // (the same for the whole cluster)
    if (rank == 0) {
      for (int i = tid; i < p.Nt; i += kThreads) p.accepted[static_cast<long long>(b) * p.Nt + i] = -1;
      if (tid == 0) p.counts[b] = 0, p.next[b] = -1;
    }
    return;
  }

  int node = 0, k = 0, have = 0, count = 1;  // the node, children tried, sums known past the first
  // sums[k]: the sum of R after k children, of all CTAs; tile sums on the way
  auto sum_rest = [&]() {
    const float *pr = target + node * p.tn, *qr = drafted ? draft + node * p.dn : nullptr;
    Pair mine{0.0f, 0.0f};
    for (int i = warp; i < tiles; i += kWarps) {
      const int at = v0 + i * per_tile, end = min(v1, at + per_tile);
      Pair acc{0.0f, 0.0f};
      for (int y0 = at + lane; y0 < end; y0 += kTile) {
        float pv[kUnroll], qv[kUnroll];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
          const int y = y0 + 32 * j;
          pv[j] = y < end ? pr[y] : 0.0f;
          qv[j] = drafted && k > 0 && y < end ? qr[y] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) acc = add(acc, rest(s, k, pv[j], qv[j], y0 + 32 * j, drafted));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1)
        acc = add(acc, Pair{__shfl_xor_sync(0xffffffffu, acc.hi, o), __shfl_xor_sync(0xffffffffu, acc.lo, o)});
      if (lane == 0) s.tile[i] = acc;
      mine = add(mine, acc);
    }
    if (lane == 0) s.warp[warp] = mine;
    __syncthreads();
    if (tid < ranks) {
      Pair all{0.0f, 0.0f};
      for (int w = 0; w < kWarps; ++w) all = add(all, s.warp[w]);
      *cluster.map_shared_rank(&s.rank[rank], tid) = all;
    }
    cluster.sync();
    Pair all{0.0f, 0.0f};
    for (int r = 0; r < ranks; ++r) all = add(all, s.rank[r]);
    return all;
  };

  if (rank == 0 && tid == 0) p.accepted[static_cast<long long>(b) * p.Nt] = 0;
  for (int i = 1; i < p.Nt; ++i) {
    if (s.parent[i] != node) continue;
    if (k > have) {
      const Pair all = sum_rest();
      if (tid == 0) s.sums[k] = all;
      cluster.sync();  // (the sums are read by all before the next ones come)
      have = k;
    }
    const Pair r = rest(s, k, s.p[i], s.q[i], s.token[i], drafted);
    const double total = k ? value(s.sums[k]) : 1.0;
    if (static_cast<double>(s.u[i]) * s.q[i] * total < value(r)) {
      if (rank == 0 && tid == 0) p.accepted[static_cast<long long>(b) * p.Nt + count] = i;
      node = i;
      k = have = 0;
      ++count;
      __syncthreads();
    } else {
      __syncthreads();
      if (tid == 0) s.rejected[k] = s.token[i];
      ++k;
      __syncthreads();
    }
  }

  // ---- the token that follows
  Pair all = sum_rest();
  if (!(all.hi > 0.0f) && k > 0) {  // nothing is left: the target's row itself
    cluster.sync();
    k = 0;
    all = sum_rest();
  }
  const double total = value(all);
  const float u0 = fminf(fmaxf(s.u[0], 0.0f), 0.99999994f);
  const double mark = static_cast<double>(u0) * total;
  double below = 0.0;
  int owner = -1, fallback = -1;
  double before = 0.0;
  for (int r = 0; r < ranks; ++r) {
    const double v = value(s.rank[r]);
    if (v > 0.0) {
      fallback = r;
      if (owner < 0 && below + v > mark) owner = r, before = below;
    }
    below += v;
  }
  if (owner < 0 && fallback >= 0) {  // rounding at the very end: the last CTA with anything
    owner = fallback;
    before = -1.0;
  }
  if (rank == 0) {
    for (int i = tid; i < p.Nt; i += kThreads)
      if (i >= count) p.accepted[static_cast<long long>(b) * p.Nt + i] = -1;
    if (tid == 0) {
      p.counts[b] = count;
      if (owner < 0) p.next[b] = -1;
    }
  }
  if (rank == owner) {
    // the tile: the first whose running sum is past the mark, or the last with anything
    if (tid == 0) s.found = -1, s.last = -1;
    __syncthreads();
    if (tid == 0) {
      double run = before < 0.0 ? 0.0 : before;
      for (int i = 0; i < tiles; ++i) {
        const double v = value(s.tile[i]);
        if (!(v > 0.0)) continue;
        s.last = i;
        if (before >= 0.0 && run + v > mark) {
          s.found = i;
          s.scan[0] = run;
          break;
        }
        run += v;
      }
    }
    __syncthreads();
    const bool exact = s.found >= 0;
    const int tile = exact ? s.found : s.last, at = v0 + tile * per_tile, end = min(v1, at + per_tile);
    double run = exact ? s.scan[0] : 0.0;
    const float *pr = target + node * p.tn, *qr = drafted ? draft + node * p.dn : nullptr;
    __syncthreads();
    if (tid == 0) s.found = p.V, s.last = -1;
    for (int y0 = at; y0 < end; y0 += kThreads) {
      __syncthreads();
      if (s.found < p.V) break;
      const int y = y0 + tid;
      const bool on = y < end;
      const Pair r = on ? rest(s, k, pr[y], drafted && k > 0 ? qr[y] : 0.0f, y, drafted) : Pair{0.0f, 0.0f};
      const double mine = value(r);
      double incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double z = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += z;
      }
      if (lane == 31) s.scan[warp] = incl;
      __syncthreads();
      double up_to = run;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) up_to += s.scan[w];
        run += s.scan[w];
      }
      if (mine > 0.0) {
        atomicMax(&s.last, y);
        if (exact && up_to + incl > mark) atomicMin(&s.found, y);
      }
      __syncthreads();
    }
    __syncthreads();
    if (tid == 0) p.next[b] = s.found < p.V ? s.found : s.last;
  }
  cluster.sync();  // no CTA leaves while another may write its shared memory
}

}  // namespace

cudaError_t launch_verify(VerifyParams p, cudaStream_t stream) {
  int ranks = 1;
  while (ranks < kMaxRanks && p.V > ranks * 4096) ranks *= 2;
  p.ranks = ranks;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_verify_kernel, p);
}

}  // namespace fa
