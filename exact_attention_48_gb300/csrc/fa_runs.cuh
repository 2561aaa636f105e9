// fa_runs.cuh -- what the drafted-tree attentions share: the list of 128-key
// tiles of all (b, hk) units cut into equal runs, a CTA's walk over its run, and
// the table of which node sees which.  P is the kernel's parameter block
// (cache_len, parents, par_b, B, Hkv, Nk, Nt, ranges, whole).  Device code only.
#pragma once

#include <cstdint>

#include "fa_cache.h"

namespace fa {

constexpr int kKeys = 128;  // keys of a tile

// Node i's bit row: words 0..i/32, in a triangular table.
__device__ __forceinline__ int bit_row(int i) {
  const int g = i >> 5;
  return 16 * g * (g + 1) + (i & 31) * (g + 1);
}

// Tiles of a sequence of n rows (an empty one keeps a tile, all hidden, so
// that its rows get written).
__device__ __forceinline__ int tiles_of(int n) { return n > 0 ? (n + kKeys - 1) / kKeys : 1; }

// First tile of run c of `runs` over `total` tiles (a 64-bit division takes
// hundreds of cycles of a CTA's start: 32 bits when they do).
__device__ __forceinline__ long long run_start(long long total, long long c, long long runs) {
  const unsigned long long x = static_cast<unsigned long long>(total) * c;
  if (x >> 32) return static_cast<long long>(x / runs);
  return static_cast<uint32_t>(x) / static_cast<uint32_t>(runs);
}
__device__ __forceinline__ long long divide(long long a, long long b) {
  if ((a | b) >> 32) return a / b;
  return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

// Where a CTA's run of tiles starts and ends, in the list of all units' tiles.
struct RunStart {
  long long t, end;    // [t, end)
  long long b_start;   // first tile of batch entry b
  long long total;     // tiles of all units
  int b;
  int runs;            // runs they are cut into
};

// The segments of a run: one per unit that it touches.
template <class P>
struct Walk {
  const P &p;
  long long t, end, u0;  // next tile, end of the run, first tile of the unit
  int b, hk, len, tiles;
  int k0, k1;            // the segment's tiles within the unit
  bool tail;             // it holds the unit's last tile
  __device__ Walk(const P &pp, const RunStart &s) : p(pp), t(s.t), end(s.end), b(s.b) {
    load();
    hk = static_cast<int>(divide(t - s.b_start, tiles));
    u0 = s.b_start + static_cast<long long>(hk) * tiles;
    k1 = 0;
    tail = false;
  }
  __device__ void load() {
    len = cache_rows(p.cache_len, b, p.Nk);
    tiles = tiles_of(len);
  }
  // The next segment, false at the run's end.
  __device__ bool next() {
    if (tail) {
      u0 += tiles;
      if (++hk == p.Hkv) {
        hk = 0;
        ++b;
        if (t < end) load();
      }
      tail = false;
    }
    if (t >= end) return false;
    k0 = static_cast<int>(t - u0);
    const long long rest = end - u0;
    tail = rest >= tiles;
    k1 = tail ? tiles : static_cast<int>(rest);
    t = u0 + k1;
    return true;
  }
  __device__ int base() const { return len - p.Nt; }
  // First tile that needs the mask.
  __device__ int masked_from() const { return base() <= 0 ? 0 : base() / kKeys; }
  // The segment holds tiles that need it, so the tree's table is built for it.
  __device__ bool masked() const { return k1 > masked_from(); }
  // The whole unit in this segment: its rows are final.
  __device__ bool whole() const { return tail && k0 == 0; }
};

// The runs that `total` tiles are cut into (sequences shorter than the cache
// may leave fewer tiles than the grid has runs: no run is empty).
template <class P>
__device__ __forceinline__ long long runs_of(const P &p, long long total) {
  return total < p.ranges ? total : p.ranges;
}

// First tile of the unit that holds tile t (t >= b_start, the first tile of a
// sequence of `tiles` tiles a unit).
__device__ __forceinline__ long long unit_start(long long t, long long b_start, int tiles) {
  return b_start + divide(t - b_start, tiles) * tiles;
}

// Run c over the tiles of all units, located by the whole block (every thread
// calls it; ends with a barrier).  With p.whole a run's ends are moved back to
// their units' starts, so that no unit is cut.  False: there is no run c, or
// nothing is left of it.
template <int kThreads, class P>
__device__ __forceinline__ bool find_run(const P &p, int c, RunStart *out, long long *scan) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (!p.cache_len) {
    const int tiles = tiles_of(p.Nk);
    const long long per_b = static_cast<long long>(p.Hkv) * tiles, total = per_b * p.B;
    const long long runs = runs_of(p, total);
    if (tid == 0 && c < runs) {
      long long t = run_start(total, c, runs), end = run_start(total, c + 1, runs);
      if (p.whole) t = unit_start(t, 0, tiles), end = unit_start(end, 0, tiles);
      out->t = t;
      out->end = end;
      out->b = static_cast<int>(divide(t, per_b));
      out->b_start = out->b * per_b;
      out->total = total;
      out->runs = static_cast<int>(runs);
    }
    __syncthreads();
    return c < runs && out->t < out->end;
  }
  if (p.B <= 32) {  // a lane per sequence, by one warp
    if (warp == 0) {
      const int tiles = lane < p.B ? tiles_of(cache_rows(p.cache_len, lane, p.Nk)) : 0;
      const long long n = static_cast<long long>(p.Hkv) * tiles;
      long long incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const long long total = __shfl_sync(0xffffffffu, incl, 31), runs = runs_of(p, total);
      const long long t = run_start(total, c, runs), end = run_start(total, c + 1, runs);
      const int first = __ffs(__ballot_sync(0xffffffffu, t < incl)) - 1;  // (none past the last run)
      const int last = __ffs(__ballot_sync(0xffffffffu, end < incl)) - 1;
      if (lane == 0) {
        out->t = out->end = out->total = total;
        out->runs = static_cast<int>(runs);
      }
      __syncwarp();
      if (lane == first) {
        out->t = p.whole ? unit_start(t, incl - n, tiles) : t;
        out->b = lane;
        out->b_start = incl - n;
      }
      if (lane == last) out->end = p.whole ? unit_start(end, incl - n, tiles) : end;
    }
    __syncthreads();
    return out->t < out->end;
  }
  // each thread sums a block of batch entries, then a scan over the threads
  const int chunk = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * chunk, p.B), b1 = min(b0 + chunk, p.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += tiles_of(cache_rows(p.cache_len, b, p.Nk));
  mine *= p.Hkv;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) scan[warp] = incl;
  if (tid == 0) out->t = out->end = 0x7fffffffffffffffll;  // (past the last tile)
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const long long runs = runs_of(p, total);
  const long long ends[2] = {run_start(total, c, runs), run_start(total, c + 1, runs)};
  for (int e = 0; e < 2; ++e) {
    long long at = before + incl - mine;  // first tile of entry b0
    if (ends[e] < at || ends[e] >= at + mine) continue;  // exactly one thread goes on, none past the last tile
    for (int b = b0;; ++b) {
      const int tiles = tiles_of(cache_rows(p.cache_len, b, p.Nk));
      const long long n = static_cast<long long>(p.Hkv) * tiles;
      if (ends[e] < at + n) {
        const long long t = p.whole ? unit_start(ends[e], at, tiles) : ends[e];
        if (e == 0) {
          out->t = t;
          out->b = b;
          out->b_start = at;
        } else {
          out->end = t;
        }
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  if (tid == 0) {
    if (out->end > total) out->end = total;
    out->total = total;
    out->runs = static_cast<int>(runs);
  }
  __syncthreads();
  return out->t < out->end;
}

// The visibility table of one unit's tree, by one warp: bit rows, and the
// padding nodes (an invalid parent, or a row before the cache's start, in
// the node itself or in an ancestor).
template <class P>
__device__ __forceinline__ void build_table(const P &p, int b, int base, uint32_t *bits, uint32_t *dead,
                                            volatile int8_t *jump) {
  const int lane = threadIdx.x & 31;
  const int n = p.Nt, words = (n + 31) >> 5;
  uint32_t bad[4] = {0, 0, 0, 0};  // this lane's copy of the padding bits
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w >= words) break;
    const int i = w * 32 + lane;
    int up = -1;
    bool live = false;
    if (i < n) {
      up = p.parents ? p.parents[b * p.par_b + i] : i - 1;  // (none given: a chain)
      live = up >= -1 && up < i && base + i >= 0;
      if (!live) up = -1;
      uint32_t *r = bits + bit_row(i);
      for (int x = 0; x < w; ++x) r[x] = 0;
      r[w] = 1u << lane;
    }
    jump[i] = static_cast<int8_t>(up);
    bad[w] = __ballot_sync(0xffffffffu, !live);
  }
  __syncwarp();
  for (int round = 0; round < 7; ++round) {
    // read every node's jump target, then write (two halves keep the warp in step)
    uint32_t add[4][4];
    int to[4], next[4];
    bool any = false;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      to[w] = next[w] = -1;
#pragma unroll
      for (int x = 0; x < 4; ++x) add[w][x] = 0;
      if (w < words) to[w] = jump[w * 32 + lane];
      if (to[w] >= 0) {
        any = true;
        next[w] = jump[to[w]];
        const uint32_t *r = bits + bit_row(to[w]);
#pragma unroll
        for (int x = 0; x <= w; ++x)
          if (x <= (to[w] >> 5)) add[w][x] = r[x];
      }
    }
    if (!__any_sync(0xffffffffu, any)) break;
    __syncwarp();
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w >= words) break;
      const int i = w * 32 + lane;
      if (to[w] >= 0) {
        uint32_t *r = bits + bit_row(i);
#pragma unroll
        for (int x = 0; x <= w; ++x)
          if (x <= (to[w] >> 5)) r[x] |= add[w][x];
      }
      jump[i] = static_cast<int8_t>(next[w]);
    }
    __syncwarp();
  }
  // padding spreads to every node that has a padding node among its ancestors
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t m = 0xffffffffu;
    if (w < words) {
      const int i = w * 32 + lane;
      bool d = true;
      if (i < n) {
        const uint32_t *r = bits + bit_row(i);
        uint32_t hit = 0;
#pragma unroll
        for (int x = 0; x <= w; ++x) hit |= r[x] & bad[x];
        d = hit != 0;
      }
      m = __ballot_sync(0xffffffffu, d);
    }
    if (lane == 0) dead[w] = m;
  }
  __syncwarp();
}

// Keys 32 q .. 32 q + 31 of a tile whose first key is node n0 of the tree (or
// before it) that node i sees: rows before the tree, and its bit row.
__device__ __forceinline__ uint32_t visible(const uint32_t *bits, int i, bool live, int f) {
  if (!live || f >= 128) return 0u;
  if (f <= -32) return ~0u;  // rows before the tree
  const uint32_t *r = bits + bit_row(i);
  const int top = i >> 5;    // words 0..top; nodes past it are not seen
  if (f < 0) return (r[0] << -f) | ((1u << -f) - 1u);
  const int x = f >> 5;
  const uint32_t lo = x <= top ? r[x] : 0u, hi = x + 1 <= top ? r[x + 1] : 0u;
  return __funnelshift_r(lo, hi, f & 31);
}

// Some node sees one of 16 rows, the first of which is node f of the tree (or before it).
__device__ __forceinline__ bool slice_seen(const uint32_t *dead, int f) {
  if (f < 0) return true;
  if (f >= 128) return false;
  const int w = f >> 5;
  return (__funnelshift_r(~dead[w], w < 3 ? ~dead[w + 1] : 0u, f & 31) & 0xffffu) != 0u;
}

}  // namespace fa
