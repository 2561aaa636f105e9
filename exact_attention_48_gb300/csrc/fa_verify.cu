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
// for the next token: a few dependent passes over a row, each some 2 us of latency.
// A sequence's row is cut over a cluster of CTAs, which add their sums through
// distributed shared memory; all of them know every sum and take the same decisions.
// Without a draft's row a rejection changes one value of R, so that one pass a node
// gives its sums, but for those below a sixteenth of what was last added up.
//
// Precision.  Which token a number falls on is decided by a sum over the whole
// vocabulary, so R and S are pairs of fp32 (hi + lo, about 48 bits; 44 where S is a
// difference), and so are the comparisons: fp64 runs at a sixty-fourth of the fp32 rate
// here, 256 cycles for one addition of a 512-thread CTA.

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
constexpr int kMaxTiles = 1024;       // tiles of a CTA's share of a row (32 a lane of its search)

// A number as the sum of two fp32, |lo| at most half a unit of hi's last place.
struct Pair {
  float hi, lo;
};
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
__device__ __forceinline__ Pair times(Pair a, float b) {
  const float ph = __fmul_rn(a.hi, b), pl = __fmaf_rn(a.hi, b, -ph);
  return quick_sum(ph, __fmaf_rn(a.lo, b, pl));
}
__device__ __forceinline__ Pair times(Pair a, Pair b) {
  const float ph = __fmul_rn(a.hi, b.hi), pl = __fmaf_rn(a.hi, b.hi, -ph);
  return quick_sum(ph, __fadd_rn(pl, __fmaf_rn(a.hi, b.lo, __fmul_rn(a.lo, b.hi))));
}
__device__ __forceinline__ Pair minus(Pair a, Pair b) {
  const Pair d = two_sum(a.hi, -b.hi);
  return quick_sum(d.hi, __fadd_rn(d.lo, __fsub_rn(a.lo, b.lo)));
}
__device__ __forceinline__ bool below(Pair a, Pair b) { return minus(a, b).hi < 0.0f; }
// r - s q, or 0 if that is less.
__device__ __forceinline__ Pair less(Pair r, Pair s, float q) {
  const Pair x = minus(r, times(s, q));
  return x.hi > 0.0f ? x : Pair{0.0f, 0.0f};
}
__device__ __forceinline__ Pair from_lane(Pair a, int lane) {
  return Pair{__shfl_sync(0xffffffffu, a.hi, lane), __shfl_sync(0xffffffffu, a.lo, lane)};
}
// The sum over the lanes' 2^n neighbours, in all of them.
__device__ __forceinline__ Pair lanes_sum(Pair a, int width) {
  for (int o = 1; o < width; o <<= 1)
    a = add(a, Pair{__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)});
  return a;
}
// Sums over the lanes up to each one.
__device__ __forceinline__ Pair lanes_scan(Pair a) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair z{__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
    if (lane >= o) a = add(z, a);
  }
  return a;
}

struct Shared {
  int parent[kMaxNodes], token[kMaxNodes];
  float u[kMaxNodes], p[kMaxNodes], q[kMaxNodes];  // the node's number, and its token's p and q at its parent
  int rejected[kMaxNodes];                         // tokens rejected at the node being worked on
  Pair sums[kMaxNodes];                            // S before the first, the second, ... child
  Pair taken;                                      // what the last rejection took of R, without a draft's row
  Pair tile[kMaxTiles];                            // this CTA's sums of R
  Pair warp[kWarps];
  Pair rank[2][kMaxRanks];                         // every CTA's sum, of two passes in turn
};

// R(y) after the first k children of a node.
__device__ __forceinline__ Pair rest(const Shared &s, int k, float p, float q, int y, bool drafted) {
  Pair r{p > 0.0f ? p : 0.0f, 0.0f};
  if (drafted) {
    for (int j = 0; j < k; ++j) r = less(r, s.sums[j], q);
  } else {
    for (int j = 0; j < k; ++j)
      if (y == s.rejected[j]) r = less(r, s.sums[j], 1.0f);
  }
  return r;
}

// A node's rows, after its first k children.
struct Node {
  const float *p, *q;  // q: null without a draft's row
  int k;
};

// R of kUnroll elements y0, y0 + step, ... (0 from `end` on).  All are asked for before any is used, and every address
// is valid: a load behind a branch would wait for the one before it.
__device__ __forceinline__ void rests(Pair (&r)[kUnroll], const Shared &s, const Node &n, int y0, int step, int end) {
  float q[kUnroll];
#pragma unroll
  for (int e = 0; e < kUnroll; ++e) r[e] = Pair{__ldg(n.p + min(y0 + e * step, end - 1)), 0.0f};
  if (n.q && n.k > 0) {
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) q[e] = __ldg(n.q + min(y0 + e * step, end - 1));
  }
#pragma unroll
  for (int e = 0; e < kUnroll; ++e)
    if (y0 + e * step >= end || !(r[e].hi > 0.0f)) r[e].hi = 0.0f;
  if (n.q && n.k > 0) {  // the first rejection: S is 1, and p - q a pair
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
      const Pair x = two_sum(r[e].hi, -q[e]);
      r[e] = x.hi > 0.0f ? x : Pair{0.0f, 0.0f};
    }
  }
  for (int j = n.q ? 1 : 0; j < n.k; ++j) {
    const Pair S = s.sums[j];
    if (n.q) {
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) r[e] = less(r[e], S, q[e]);
    } else {
      const int x = s.rejected[j];
#pragma unroll
      for (int e = 0; e < kUnroll; ++e)
        if (y0 + e * step == x) r[e] = less(r[e], S, 1.0f);
    }
  }
}

__global__ void __launch_bounds__(kThreads, 2) fa_verify_kernel(const VerifyParams p) {
  __shared__ Shared s;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = p.ranks, rank = blockIdx.x % ranks, b = blockIdx.x / ranks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // (all of the cluster's CTAs have to have started before one writes to another's shared memory: waited for below)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;");
  const bool drafted = p.draft != nullptr;
  // this CTA's share of a row, and the warps' tiles in it
  const int share = (p.V + ranks - 1) / ranks;
  const int v0 = min(p.V, rank * share), v1 = min(p.V, v0 + share);
  const int per_tile = kTile * ((share + kTile * kMaxTiles - 1) / (kTile * kMaxTiles));
  const int tiles = (v1 - v0 + per_tile - 1) / per_tile;
  const float *target = p.target + b * p.tb, *draft = drafted ? p.draft + b * p.db : nullptr;
  int *accepted = p.accepted + static_cast<long long>(b) * p.Nt;

  if (tid < kMaxNodes) {
    int up = -2;
    if (tid < p.Nt) {
      const int x = p.tokens[b * p.tok_b + tid];
      up = p.parents[b * p.par_b + tid];
      const bool asks = tid > 0 && up >= 0 && up < tid && x >= 0 && x < p.V;
      s.token[tid] = x;
      s.u[tid] = p.uniforms[b * p.uni_b + tid];
      s.p[tid] = asks ? target[up * p.tn + x] : 0.0f;
      s.q[tid] = asks ? (drafted ? draft[up * p.dn + x] : 1.0f) : 0.0f;
      if (tid > 0 && !asks) up = -2;
    }
    s.parent[tid] = up;
  }
  if (tid == 0) s.sums[0] = Pair{1.0f, 0.0f};
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (s.parent[0] != -1) {  // (the same for the whole cluster)
    if (rank == 0) {
      for (int i = tid; i < p.Nt; i += kThreads) accepted[i] = -1;
      if (tid == 0) p.counts[b] = 0, p.next[b] = -1;
    }
    return;
  }

  // Every warp walks the tree, on the same numbers.
  int node = 0, k = 0, count = 1, pass = 0;  // the node, children tried, nodes accepted, passes made
  // the sum of R after k children, of all CTAs; tile sums on the way
  auto sum_rest = [&]() {
    const Node n{target + node * p.tn, drafted ? draft + node * p.dn : nullptr, k};
    Pair mine{0.0f, 0.0f};
    for (int i = warp; i < tiles; i += kWarps) {
      const int at = v0 + i * per_tile, end = min(v1, at + per_tile);
      float hi = 0.0f, lo = 0.0f;  // (the errors of the additions gathered in lo)
      for (int y0 = at + lane; y0 - lane < end; y0 += kTile) {
        Pair r[kUnroll];
        rests(r, s, n, y0, 32, end);
#pragma unroll
        for (int e = 0; e < kUnroll; ++e) {
          const Pair t = two_sum(hi, r[e].hi);
          hi = t.hi;
          lo = __fadd_rn(lo, __fadd_rn(t.lo, r[e].lo));
        }
      }
      const Pair sum = lanes_sum(two_sum(hi, lo), 32);
      if (lane == 0) s.tile[i] = sum;
      mine = add(mine, sum);
    }
    if (lane == 0) s.warp[warp] = mine;
    __syncthreads();
    Pair *shared_sums = s.rank[pass & 1];
    if (warp == 0) {
      const Pair all = lanes_sum(s.warp[lane % kWarps], kWarps);
      if (lane < ranks) *cluster.map_shared_rank(&shared_sums[rank], lane) = all;
    }
    cluster.sync();
    ++pass;
    return lanes_sum(lane % kMaxRanks < ranks ? shared_sums[lane % kMaxRanks] : Pair{0.0f, 0.0f}, kMaxRanks);
  };

  if (rank == 0 && tid == 0) accepted[0] = 0;
  int have = 0;        // sums[0 .. have] are known
  float added = 0.0f;  // the last of them that was added up
  for (int w = 0; w < kMaxNodes / 32; ++w) {
    // the children of the node among nodes 32 w .. 32 w + 31 (those of an accepted one come after it)
    uint32_t kids = __ballot_sync(0xffffffffu, s.parent[32 * w + lane] == node && 32 * w + lane > 0);
    while (kids) {
      const int i = 32 * w + __ffs(kids) - 1;
      kids &= kids - 1;
      if (k > have) {
        // without a draft's row the rejected token is all that has gone; what is left is added up anew where it is a small
        // part of the last sum, whose 48 bits it would not keep (or even turn negative)
        Pair all{0.0f, 0.0f};
        if (!drafted && have > 0) all = minus(s.sums[k - 1], s.taken);  // (k - 1 children were tried with a sum of this row)
        if (drafted || have == 0 || !(all.hi >= 0.0625f * added)) {
          all = sum_rest();
          added = all.hi;
        }
        if (tid == 0) s.sums[k] = all;
        __syncthreads();
        have = k;
      }
      const Pair r = rest(s, k, s.p[i], s.q[i], s.token[i], drafted);
      const Pair ask = times(times(Pair{s.u[i], 0.0f}, s.q[i]), s.sums[k]);
      if (below(ask, r)) {
        if (rank == 0 && tid == 0) accepted[count] = i;
        node = i;
        k = have = 0;
        ++count;
        kids = __ballot_sync(0xffffffffu, s.parent[32 * w + lane] == node);
      } else {
        __syncthreads();  // (the others have read what changes)
        if (tid == 0) {
          s.rejected[k] = s.token[i];
          s.taken = minus(r, less(r, s.sums[k], 1.0f));  // of R, without a draft's row
        }
        ++k;
        __syncthreads();
      }
    }
  }

  // ---- the token that follows
  Pair all = sum_rest();
  if (!(all.hi > 0.0f) && k > 0) {  // nothing is left: the target's row itself
    k = 0;
    all = sum_rest();
  }
  const float u0 = fminf(fmaxf(s.u[0], 0.0f), 0.99999994f);
  const Pair mark = times(all, u0);
  // the CTA whose share the mark falls into (or, by rounding at the very end, the last one with anything)
  const Pair own = lane < ranks ? s.rank[(pass - 1) & 1][lane] : Pair{0.0f, 0.0f};
  const Pair upto = lanes_scan(own);
  const uint32_t any = __ballot_sync(0xffffffffu, own.hi > 0.0f);
  const uint32_t past = __ballot_sync(0xffffffffu, own.hi > 0.0f && below(mark, upto));
  const int owner = past ? __ffs(past) - 1 : 31 - __clz(any);  // (-1: nothing at all)
  const Pair before = owner > 0 ? from_lane(upto, owner - 1) : Pair{0.0f, 0.0f};
  if (rank == 0) {
    for (int i = tid; i < p.Nt; i += kThreads)
      if (i >= count) accepted[i] = -1;
    if (tid == 0) {
      p.counts[b] = count;
      if (owner < 0) p.next[b] = -1;
    }
  }
  if (rank == owner && warp == 0) {
    // a warp's search: the first of its lanes' parts, in order, whose running sum is past the mark, or the last with
    // anything; `run`: what lies before
    Pair run = before;
    auto find = [&](Pair part) {
      const Pair upto_lane = lanes_scan(part);
      const uint32_t some = __ballot_sync(0xffffffffu, part.hi > 0.0f);
      const uint32_t hit = __ballot_sync(0xffffffffu, part.hi > 0.0f && below(mark, add(run, upto_lane)));
      const int at = hit ? __ffs(hit) - 1 : (some ? 31 - __clz(some) : 0);
      if (at > 0) run = add(run, from_lane(upto_lane, at - 1));
      return at;
    };
    // tiles, a run of them per lane, then one of those per lane in turn
    const int per_lane = (tiles + 31) / 32;
    Pair part{0.0f, 0.0f};
    for (int i = lane * per_lane; i < min(tiles, (lane + 1) * per_lane); ++i) part = add(part, s.tile[i]);
    int tile = find(part) * per_lane;
    part = lane < per_lane && tile + lane < tiles ? s.tile[tile + lane] : Pair{0.0f, 0.0f};
    tile += find(part);
    // the tile's elements, 256 at a time, eight a lane
    const Node n{target + node * p.tn, drafted ? draft + node * p.dn : nullptr, k};
    const int at = v0 + tile * per_tile, end = min(v1, at + per_tile);
    int last = at;  // the last element with anything so far
    for (int c = at; c < end; c += kTile) {
      Pair r[kUnroll];
      rests(r, s, n, c + lane * kUnroll, 1, end);
      part = Pair{0.0f, 0.0f};
      int mine = -1;
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) {
        part = add(part, r[e]);
        if (r[e].hi > 0.0f) mine = e;
      }
      const Pair upto_lane = lanes_scan(part);
      const uint32_t some = __ballot_sync(0xffffffffu, mine >= 0);
      const uint32_t hit = __ballot_sync(0xffffffffu, mine >= 0 && below(mark, add(run, upto_lane)));
      if (some) {
        const int l = 31 - __clz(some);
        last = c + l * kUnroll + __shfl_sync(0xffffffffu, mine, l);
      }
      if (hit) {
        const int l = __ffs(hit) - 1;
        if (l > 0) run = add(run, from_lane(upto_lane, l - 1));
        // (every lane goes through its own eight; the lane in question has the answer)
        int found = -1;
#pragma unroll
        for (int e = 0; e < kUnroll; ++e) {
          run = add(run, r[e]);
          if (found < 0 && r[e].hi > 0.0f && below(mark, run)) found = e;
        }
        if (found < 0) found = mine;  // (rounding: its last one)
        last = c + l * kUnroll + __shfl_sync(0xffffffffu, found, l);
        break;
      }
      run = add(run, from_lane(upto_lane, 31));
    }
    if (lane == 0) p.next[b] = last;
  }
  cluster.sync();  // no CTA leaves while another may write its shared memory
}

}  // namespace

cudaError_t launch_verify(VerifyParams p, cudaStream_t stream) {
  // CTAs of a sequence: enough to read its rows at once, but all of the batch's at work together (two an SM)
  int ranks = 1;
  while (ranks < kMaxRanks && p.V > ranks * 2048 && 2ll * ranks * p.B <= 2 * 152) ranks *= 2;
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
