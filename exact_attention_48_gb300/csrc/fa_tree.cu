// fa_tree.cu -- attention of a tree of drafted tokens over a key/value cache.
//
// Row (g, i) of a unit (b, hk) is tree node i under query head hk * G + g.
// It sees the cache rows before the tree, its own row and its ancestors'
// rows: softmax over those with a running maximum and sum, 128 keys at a
// time, as in the forward pass.
//
// What bounds it.  Every key costs 4 d bytes of cache and 4 d flops a row, so
// up to about 280 rows (the tensor rate over the HBM rate) the cache traffic
// sets the pace: each K and V tile is read once and used for all rows of the
// unit, as A = Q (128 rows) against 128 keys on tcgen05.  The 128-key tiles
// of all units form one list that is cut into equal runs, one per CTA (one
// CTA per SM), whatever the sequences' lengths; a unit cut by a run's end
// leaves partial results that a second kernel merges.
//
// CTA (384 threads): warps 0..3 and 4..7 softmax (a row per thread), warp 8
// TMA producer (Q, and K and V tiles through one ring), warp 9 MMA issuer and
// TMEM owner, warp 10 the tree's visibility table, warp 11 idle.  With one
// row tile the two softmax warpgroups take alternate key tiles of it (each
// with its own maximum, sum and O, merged at the end of the unit); with two
// row tiles each takes its own.  TMEM columns: S_t at 128 t, O_t at 256 + d t,
// P (bf16) over S.
//
// The tree.  Only a unit's last tiles hold nodes.  Warp 10 turns parents into
// one bit row per node (its ancestors and itself) by pointer doubling, at
// most seven rounds, into shared memory while earlier tiles are worked on;
// the softmax of those tiles tests bits.  Rows behind the sequence's end and
// padding nodes' rows are set to zero in the V tile, for 0 * NaN is NaN.

#include <cstdint>

#include "fa_cache.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kRows = 128;  // query rows of a row tile
constexpr int kKeys = 128;  // keys of a tile
constexpr int kThreads = 384;
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpMask = 10;
constexpr int kModelCtas = 152;  // GB300's SMs: the grid the runs are cut for
constexpr float kRescaleThreshold = 8.0f;  // a row's maximum moves only when exceeded by more (log2 units)
constexpr float kLn2 = 0.69314718055994530942f;
constexpr uint32_t kTmemCols = 512;
// 104 registers for the control warps and 200 for the softmax: the split of
// the forward kernel, whose roles these are (128 * 104 + 256 * 200 is what
// 384 threads were launched with, 168 each).
constexpr uint32_t kRegsControl = 104, kRegsSoftmax = 200;
static_assert(128 * kRegsControl + 256 * kRegsSoftmax <= kThreads * 168, "register split");

template <int D, bool SPLIT>
struct TreeLayout {
  static constexpr int kSlabs = D / 64;
  static constexpr uint32_t kTile = kKeys * D * 2;                // a Q, K or V tile
  static constexpr int kQTiles = SPLIT ? 1 : 2;
  static constexpr int kSlots = D == 128 ? 5 : 10;                // ring of K and V tiles
  // first the small things, then (1 KB aligned) the tiles
  static constexpr uint32_t kOffBits = 0;                         // node bit rows, see bit_row()
  static constexpr uint32_t kOffDead = kOffBits + 32 * (1 + 2 + 3 + 4) * 4;
  static constexpr uint32_t kOffJump = kOffDead + 16;             // int8[128]: pointer doubling
  static constexpr uint32_t kOffRange = kOffJump + 128;           // the run's start (see RunStart)
  static constexpr uint32_t kOffScan = kOffRange + 32;            // 12 warps' sums
  static constexpr uint32_t kOffStats = kOffScan + 12 * 8;        // SPLIT: m, l, lb of both warpgroups
  static constexpr uint32_t kOffBar = kOffStats + (SPLIT ? 2 * 3 * kRows * 4 : 0);
  // full[S], empty[S], s_full[2], p_ready[2], pv_done[2], q_full, q_empty, mask_full, mask_empty, drain
  static constexpr int kNumBars = 2 * kSlots + 6 + 5;
  static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;    // TMEM address, abort flag
  static constexpr uint32_t kSmall = (kOffMisc + 16 + 15) / 16 * 16;
  static constexpr uint32_t kTiles = (kQTiles + kSlots) * kTile;
  static constexpr uint32_t kRequest = kSmall + 1008 + kTiles;    // dynamic shared memory starts 16-byte aligned
  static_assert(kOffBar % 8 == 0 && kOffRange % 8 == 0 && kOffScan % 8 == 0, "alignment");
  static_assert(kRequest <= 232448, "shared memory budget");
};

// Node i's bit row: words 0..i/32, in a triangular table.
__device__ __forceinline__ int bit_row(int i) {
  const int g = i >> 5;
  return 16 * g * (g + 1) + (i & 31) * (g + 1);
}

// Tiles of a sequence of n rows (an empty one keeps a tile, all hidden, so
// that its rows get written).
__device__ __forceinline__ int tiles_of(int n) { return n > 0 ? (n + kKeys - 1) / kKeys : 1; }

// Where a CTA's run of tiles starts and ends, in the list of all units' tiles.
struct RunStart {
  long long t, end;    // [t, end)
  long long b_start;   // first tile of batch entry b
  int b;
  int pad;
};

// The segments of a run: one per unit that it touches.
struct Walk {
  const TreeParams &p;
  long long t, end, u0;  // next tile, end of the run, first tile of the unit
  int b, hk, len, tiles;
  int k0, k1;            // the segment's tiles within the unit
  bool tail;             // it holds the unit's last tile
  __device__ Walk(const TreeParams &pp, const RunStart &s) : p(pp), t(s.t), end(s.end), b(s.b) {
    load();
    hk = static_cast<int>((t - s.b_start) / tiles);
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
__device__ __forceinline__ long long runs_of(const TreeParams &p, long long total) {
  return total < p.ranges ? total : p.ranges;
}

// Run c over the tiles of all units, located by the whole block (every thread
// calls it; ends with a barrier).  False: there is no run c.
__device__ __forceinline__ bool find_run(const TreeParams &p, int c, RunStart *out, long long *scan) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (!p.cache_len) {
    const long long per_b = static_cast<long long>(p.Hkv) * tiles_of(p.Nk), total = per_b * p.B;
    const long long runs = runs_of(p, total);
    if (tid == 0 && c < runs) {
      out->t = total * c / runs;
      out->end = total * (c + 1) / runs;
      out->b = static_cast<int>(out->t / per_b);
      out->b_start = out->b * per_b;
    }
    __syncthreads();
    return c < runs;
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
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  long long at = before + incl - mine;  // first tile of entry b0
  const long long runs = runs_of(p, total);
  const long long t = total * c / runs;
  if (c < runs && t >= at && t < at + mine) {  // exactly one thread
    for (int b = b0;; ++b) {
      const long long n = static_cast<long long>(p.Hkv) * tiles_of(cache_rows(p.cache_len, b, p.Nk));
      if (t < at + n) {
        out->t = t;
        out->end = total * (c + 1) / runs;
        out->b = b;
        out->b_start = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  return c < runs;
}

// The visibility table of one unit's tree, by one warp: bit rows, and the
// padding nodes (an invalid parent, or a row before the cache's start, in
// the node itself or in an ancestor).
__device__ __forceinline__ void build_table(const TreeParams &p, int b, int base, uint32_t *bits, uint32_t *dead,
                                            volatile int8_t *jump) {
  const int lane = threadIdx.x & 31;
  const int n = p.Nt;
  uint32_t bad[4] = {0, 0, 0, 0};  // this lane's copy of the padding bits
  for (int w = 0; w < 4; ++w) {
    const int i = w * 32 + lane;
    int up = -1;
    bool live = false;
    if (i < n) {
      up = p.parents[b * p.par_b + i];
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
      const int i = w * 32 + lane;
      to[w] = jump[i];
      next[w] = -1;
#pragma unroll
      for (int x = 0; x < 4; ++x) add[w][x] = 0;
      if (to[w] >= 0) {
        any = true;
        next[w] = jump[to[w]];
        const uint32_t *r = bits + bit_row(to[w]);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (x <= (to[w] >> 5)) add[w][x] = r[x];
      }
    }
    if (!__any_sync(0xffffffffu, any)) break;
    __syncwarp();
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int i = w * 32 + lane;
      if (to[w] >= 0) {
        uint32_t *r = bits + bit_row(i);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (x <= (to[w] >> 5)) r[x] |= add[w][x];
      }
      jump[i] = static_cast<int8_t>(next[w]);
    }
    __syncwarp();
  }
  // padding spreads to every node that has a padding node among its ancestors
  for (int w = 0; w < 4; ++w) {
    const int i = w * 32 + lane;
    bool d = true;
    if (i < n) {
      const uint32_t *r = bits + bit_row(i);
      uint32_t hit = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (x <= w) hit |= r[x] & bad[x];
      d = hit != 0;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, d);
    if (lane == 0) dead[w] = m;
  }
  __syncwarp();
}

// The state of one softmax row over a segment.
struct RowState {
  float m, l, lb;
};

struct SoftmaxArgs {
  uint64_t *s_full, *p_ready, *pv_done, *full, *mask_full;
  uint32_t tS, tO;  // this warpgroup's columns, lane base added
  uint8_t *ring;    // K and V slots
  const uint32_t *bits, *dead;
  int node;         // tree node of this thread's row, -1 if the row is unused
  int warps;        // warps of the warpgroup that hold rows
};

// One 128-key tile: scores from TMEM, running maximum and sum, P as bf16 over
// S, O rescaled when the maximum moves.  `cnt`: tiles this warpgroup has
// taken so far (barrier phases); first: its first tile of the segment;
// e_v: the V tile's place in the ring's sequence; key0: first key of the
// tile.  MASK: the tile holds nodes or rows behind the end.
template <int D, int SLOTS, bool MASK>
__device__ __forceinline__ bool softmax_tile(const SoftmaxArgs &a, const TreeParams &p, const WaitCtl &ctl,
                                             const Walk &wk, RowState &st, uint32_t cnt, bool first, uint32_t e_v,
                                             int key0) {
  const float c = p.scale_log2;
  const bool neg = p.neg != 0;
  if (!__all_sync(0xffffffffu, mbar_wait(a.s_full, cnt & 1, ctl, kSiteSFull))) return false;
  tc_fence_after();
  uint32_t s[4][32];
#pragma unroll
  for (int q = 0; q < 4; ++q) tmem_ld32(a.tS + q * 32, s[q]);
#pragma unroll
  for (int q = 0; q < 4; ++q) tmem_ld_wait(s[q]);

  uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};  // visible keys of the tile
  if (MASK) {
    const int n0 = key0 - wk.base();  // node of the tile's first key
    const int i = a.node;
    const bool live = i >= 0 && !((a.dead[i >> 5] >> (i & 31)) & 1u);
    uint32_t w[6];                    // bits of nodes -32.. 0 and 0..127, then nothing
    w[4] = w[5] = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) w[x] = live && x <= (i >> 5) ? a.bits[bit_row(i) + x] : 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int f = n0 + 32 * q;      // first node of this quarter
      uint32_t v;
      if (f <= -32) {
        v = ~0u;                      // rows before the tree
      } else if (f < 0) {
        v = (w[0] << -f) | ((1u << -f) - 1u);
      } else {
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (x == (f >> 5)) lo = w[x], hi = w[x + 1];
        }
        v = __funnelshift_r(lo, hi, f & 31);
      }
      see[q] = live ? v : 0u;
    }
    const uint32_t hide = __float_as_uint(neg ? INFINITY : -INFINITY);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int x = 0; x < 32; ++x)
        if (!((see[q] >> x) & 1u)) s[q][x] = hide;
  }

  float mx;
  {
    float mq[4];
    if (!neg) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float m0 = fmax3(__uint_as_float(s[q][0]), __uint_as_float(s[q][1]), __uint_as_float(s[q][2]));
#pragma unroll
        for (int x = 3; x < 31; x += 2) m0 = fmax3(m0, __uint_as_float(s[q][x]), __uint_as_float(s[q][x + 1]));
        mq[q] = fmaxf(m0, __uint_as_float(s[q][31]));
      }
      mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float m0 = fmin3(__uint_as_float(s[q][0]), __uint_as_float(s[q][1]), __uint_as_float(s[q][2]));
#pragma unroll
        for (int x = 3; x < 31; x += 2) m0 = fmin3(m0, __uint_as_float(s[q][x]), __uint_as_float(s[q][x + 1]));
        mq[q] = fminf(m0, __uint_as_float(s[q][31]));
      }
      mx = fminf(fminf(mq[0], mq[1]), fminf(mq[2], mq[3]));
    }
  }
  const bool hidden = MASK && (see[0] | see[1] | see[2] | see[3]) == 0u;  // (0 * -inf is NaN)
  const float cand = hidden ? -INFINITY : mx * c;
  const bool grow = cand > st.m + kRescaleThreshold;
  float alpha = 1.0f;
  if (grow) {
    alpha = ex2(st.m - cand);
    st.m = cand;
  }
  const float2 cc = make_float2(c, c), nm = make_float2(-st.m, -st.m);
  uint32_t pk[4][16];
  float2 sf = make_float2(0.f, 0.f);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float2 sq = make_float2(0.f, 0.f);
#pragma unroll
    for (int x = 0; x < 32; x += 2) {
      const float2 y = ffma2(make_float2(__uint_as_float(s[q][x]), __uint_as_float(s[q][x + 1])), cc, nm);
      float p0 = ex2(y.x), p1 = ex2(y.y);
      if (MASK) {
        p0 = (see[q] >> x) & 1u ? p0 : 0.0f;
        p1 = (see[q] >> (x + 1)) & 1u ? p1 : 0.0f;
      }
      pk[q][x / 2] = pack_bf16x2(p0, p1);
      sq = fadd2(sq, make_float2(p0, p1));
    }
    tmem_st16(a.tS + q * 16, pk[q]);
    sf = fadd2(sf, sq);
  }
  tmem_st_wait();

  if (!first && __any_sync(0xffffffffu, grow)) {
    if (!__all_sync(0xffffffffu, mbar_wait(a.pv_done, (cnt - 1) & 1, ctl, kSitePvDone))) return false;
    tc_fence_after();
#pragma unroll 1
    for (int ch = 0; ch < D / 16; ++ch) {
      uint32_t o[16];
      tmem_ld16(a.tO + ch * 16, o);
      tmem_ld_wait16(o);
#pragma unroll
      for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
      tmem_st16(a.tO + ch * 16, o);
    }
    tmem_st_wait();
  }
  if (MASK) {  // V rows that no query row sees
    if (!__all_sync(0xffffffffu, mbar_wait(&a.full[e_v % SLOTS], (e_v / SLOTS) & 1, ctl, kSiteVFull))) return false;
    uint8_t *v = a.ring + (e_v % SLOTS) * (kKeys * D * 2);
    for (int r = threadIdx.x & 127; r < kKeys; r += a.warps * 32) {
      const int node = key0 + r - wk.base();
      if (node < 0 || (node < p.Nt && !((a.dead[node >> 5] >> (node & 31)) & 1u))) continue;
#pragma unroll
      for (int sl = 0; sl < D / 64; ++sl)
#pragma unroll
        for (int x = 0; x < 8; ++x)
          *reinterpret_cast<uint4 *>(v + sl * (kKeys * 128) + r * 128 + x * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  warp_arrive(a.p_ready);

  st.l = st.l * alpha + (sf.x + sf.y);
  float2 sb = make_float2(0.f, 0.f);  // sum of the bf16 weights: what O is divided by
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float2 sq = make_float2(0.f, 0.f);
#pragma unroll
    for (int x = 0; x < 16; ++x) sq = add_bf16x2_f32(sq, pk[q][x]);
    sb = fadd2(sb, sq);
  }
  st.lb = st.lb * alpha + (sb.x + sb.y);
  return true;
}

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    fa_tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const TreeParams p) {
  using L = TreeLayout<D, SPLIT>;
  constexpr int S = L::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *small = smem_raw;
  uint8_t *tiles = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + L::kSmall + 1023) &
                                               ~uintptr_t(1023));
  uint8_t *sQ = tiles, *ring = tiles + L::kQTiles * L::kTile;
  uint32_t *bits = reinterpret_cast<uint32_t *>(small + L::kOffBits);
  uint32_t *dead = reinterpret_cast<uint32_t *>(small + L::kOffDead);
  RunStart *run = reinterpret_cast<RunStart *>(small + L::kOffRange);
  uint64_t *full = reinterpret_cast<uint64_t *>(small + L::kOffBar);
  uint64_t *empty = full + S;
  uint64_t *s_full = empty + S;    // [2 warpgroups]
  uint64_t *p_ready = s_full + 2;  // [2]
  uint64_t *pv_done = p_ready + 2;  // [2]
  uint64_t *q_full = pv_done + 2, *q_empty = q_full + 1;
  uint64_t *mask_full = q_empty + 1, *mask_empty = mask_full + 1, *drain = mask_empty + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(small + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(small + L::kOffMisc + 4);
  const WaitCtl ctl{abort_flag, p.status};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = blockIdx.x % p.groups, c = blockIdx.x / p.groups;
  // row tiles of this CTA: 2 * group and the next, if there is one
  const int tile0 = 2 * group;
  const bool two = !SPLIT && tile0 + 1 < p.row_tiles;
  const int rows_used = p.gpt * p.Nt;         // rows of a row tile
  const int warps = (rows_used + 31) / 32;    // softmax warps with rows, per warpgroup

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_ready[t], warps);
      mbar_init(&pv_done[t], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(mask_full, 1);
    mbar_init(mask_empty, SPLIT || two ? 2 * warps : warps);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (!find_run(p, c, run, reinterpret_cast<long long *>(small + L::kOffScan))) return;
  if (warp == kWarpMma) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk wk(p, *run);

  if (warp >= kWarpProducer) {
    regs_decrease<kRegsControl>();
    if (warp == kWarpProducer && lane == 0) {
      // ---------------------------------------------------------- producer
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      uint32_t e = 0, nq = 0;  // ring loads and Q loads so far
      bool ok = true;
      auto load = [&](const CUtensorMap *map, int row) -> bool {
        const uint32_t sl = e % S;
        if (!mbar_wait(&empty[sl], ((e / S) & 1) ^ 1, ctl, kSiteKvEmpty)) return false;
        mbar_arrive_expect_tx(&full[sl], L::kTile);
#pragma unroll
        for (int x = 0; x < L::kSlabs; ++x)
          tma_load_4d(ring + sl * L::kTile + x * kKeys * 128, map, &full[sl], x * 64, row, wk.hk, wk.b);
        ++e;
        return true;
      };
      while (ok && wk.next()) {
        if (!(ok = mbar_wait(q_empty, (nq & 1) ^ 1, ctl, kSiteQEmpty))) break;
        const int nt = two ? 2 : 1;
        mbar_arrive_expect_tx(q_full, nt * L::kSlabs * rows_used * 128);
        for (int t = 0; t < nt; ++t)
#pragma unroll
          for (int x = 0; x < L::kSlabs; ++x)
            tma_load_4d(sQ + t * L::kTile + x * kRows * 128, &tm_q, q_full, x * 64, 0,
                        wk.hk * p.G + (tile0 + t) * p.gpt, wk.b);
        ++nq;
        for (int j = wk.k0; ok && j < wk.k1; ++j) ok = load(&tm_k, j * kKeys) && load(&tm_v, j * kKeys);
      }
      // every copy issued lands before this thread leaves (bounded waits)
      for (uint32_t i = e > S ? e - S : 0; i < e; ++i) mbar_drain(&full[i % S], (i / S) & 1);
      if (nq) mbar_drain(q_full, (nq - 1) & 1);
    } else if (warp == kWarpMma && lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t kIdS = idesc_bf16(kRows, kKeys, false, false);
      constexpr uint32_t kIdO = idesc_bf16(kRows, D, false, true);
      const uint32_t aQ = smem_addr(sQ), aR = smem_addr(ring);
      uint32_t g = 0, nq = 0;         // tiles and Q loads so far
      uint32_t cnt[2] = {0, 0};       // P V products per warpgroup so far
      bool ok = true;
      auto full_wait = [&](uint32_t e, int site) {
        const bool r = mbar_wait(&full[e % S], (e / S) & 1, ctl, site);
        tc_fence_after();
        return r;
      };
      // S of warpgroup t = its Q tile times K of tile x (counted over the run)
      auto issue_s = [&](int t, uint32_t x) {
        const uint64_t dq = sdesc_sw128(aQ + (SPLIT ? 0 : t) * L::kTile, 16, 1024);
        const uint64_t dk = sdesc_sw128(aR + ((2 * x) % S) * L::kTile, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + t * 128, desc_add(dq, kmajor_step(kk, kRows)), desc_add(dk, kmajor_step(kk, kKeys)), kIdS,
                 kk > 0 ? 1u : 0u);
        tc_commit(&s_full[t]);
      };
      auto issue_pv = [&](int t, uint32_t x, bool first) -> bool {
        if (!mbar_wait(&p_ready[t], cnt[t] & 1, ctl, kSitePReady)) return false;
        ++cnt[t];
        tc_fence_after();
        const uint64_t dv = sdesc_sw128(aR + ((2 * x + 1) % S) * L::kTile, kKeys * 128, 1024);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          mma_ts(tmem + 256 + t * D, tmem + t * 128 + kk * 8, desc_add(dv, mnmajor_step(kk)), kIdO,
                 (!first || kk > 0) ? 1u : 0u);
        tc_commit(&pv_done[t]);
        return true;
      };
      while (ok && wk.next()) {
        const int n = wk.k1 - wk.k0;
        if (!(ok = mbar_wait(q_full, nq & 1, ctl, kSiteQFull))) break;
        tc_fence_after();
        if constexpr (SPLIT) {
          // tile x of the segment belongs to warpgroup x & 1; its S is issued
          // right after the P V product two tiles before it
          for (int x = 0; ok && x < n + 2; ++x) {
            if (x >= 2) {
              const int y = x - 2;
              ok = full_wait(2 * (g + y) + 1, kSiteVFull) && issue_pv(y & 1, g + y, y < 2);
              if (ok) tc_commit(&empty[(2 * (g + y) + 1) % S]);
            }
            if (ok && x < n) {
              if (!(ok = full_wait(2 * (g + x), kSiteKFull))) break;
              issue_s(x & 1, g + x);
              tc_commit(&empty[(2 * (g + x)) % S]);
              if (x == n - 1) tc_commit(q_empty);
            }
          }
        } else {
          for (int x = 0; ok && x <= n; ++x) {
            if (x > 0 && !(ok = full_wait(2 * (g + x - 1) + 1, kSiteVFull))) break;
            if (x > 0 && !(ok = issue_pv(0, g + x - 1, x == 1))) break;
            if (x < n) {
              if (!(ok = full_wait(2 * (g + x), kSiteKFull))) break;
              issue_s(0, g + x);
            }
            if (x > 0) {
              if (two && !(ok = issue_pv(1, g + x - 1, x == 1))) break;
              tc_commit(&empty[(2 * (g + x - 1) + 1) % S]);
            }
            if (x < n) {
              if (two) issue_s(1, g + x);
              tc_commit(&empty[(2 * (g + x)) % S]);
              if (x == n - 1) tc_commit(q_empty);
            }
          }
        }
        g += n;
        ++nq;
      }
      tc_commit(drain);
      mbar_drain(drain, 0);
    } else if (warp == kWarpMask) {
      // ---------------------------------------------------------- the tree's table
      uint32_t n = 0;
      while (wk.next()) {
        if (!wk.masked()) continue;
        if (!__all_sync(0xffffffffu, mbar_wait(mask_empty, (n & 1) ^ 1, ctl, kSiteMaskEmpty))) break;
        build_table(p, wk.b, wk.base(), bits, dead, reinterpret_cast<volatile int8_t *>(small + L::kOffJump));
        warp_arrive(mask_full);
        ++n;
      }
    }
  } else {
    regs_increase<kRegsSoftmax>();
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2, wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const int mtile = tile0 + (SPLIT ? 0 : t);
    const bool works = wq < warps && (SPLIT || t == 0 || two);
    if (works || SPLIT) {
      // this thread's row: head and node, if the tile has that many
      const int gh = mtile * p.gpt + row / p.Nt;  // head within the group
      const bool used = row < rows_used && gh < p.G;
      SoftmaxArgs a;
      a.s_full = &s_full[t];
      a.p_ready = &p_ready[t];
      a.pv_done = &pv_done[t];
      a.full = full;
      a.mask_full = mask_full;
      a.tS = tmem + t * 128 + lane_base;
      a.tO = tmem + 256 + t * D + lane_base;
      a.ring = ring;
      a.bits = bits;
      a.dead = dead;
      a.node = used ? row % p.Nt : -1;
      a.warps = warps;
      float *xm = reinterpret_cast<float *>(small + L::kOffStats);  // SPLIT: [2][128] each of m, l, lb
      float *xl = xm + 2 * kRows, *xb = xl + 2 * kRows;
      uint32_t g = 0, cnt = 0, nmask = 0;
      bool ok = true;
      while ((ok || SPLIT) && wk.next()) {
        const int n = wk.k1 - wk.k0, mfrom = wk.masked_from();
        RowState st{-INFINITY, 0.0f, 0.0f};
        if (works && ok) {
          bool have_mask = false;
          const int step = SPLIT ? 2 : 1;
          for (int x = SPLIT ? t : 0; ok && x < n; x += step) {
            const int kt = wk.k0 + x;
            const bool first = x < step;
            if (kt >= mfrom) {
              if (!have_mask) {
                ok = __all_sync(0xffffffffu, mbar_wait(mask_full, nmask & 1, ctl, kSiteMaskFull));
                have_mask = true;
                if (!ok) break;
              }
              ok = softmax_tile<D, S, true>(a, p, ctl, wk, st, cnt, first, 2 * (g + x) + 1, kt * kKeys);
            } else {
              ok = softmax_tile<D, S, false>(a, p, ctl, wk, st, cnt, first, 2 * (g + x) + 1, kt * kKeys);
            }
            ++cnt;
          }
          if (ok && wk.masked() && !have_mask)
            ok = __all_sync(0xffffffffu, mbar_wait(mask_full, nmask & 1, ctl, kSiteMaskFull));
          if (ok && cnt > 0 && n > (SPLIT ? t : 0))
            ok = __all_sync(0xffffffffu, mbar_wait(a.pv_done, (cnt - 1) & 1, ctl, kSitePvDone));
        }
        tc_fence_after();
        // ---- the segment's result
        const bool padding = wk.tail && a.node >= 0 && works && ok && ((dead[a.node >> 5] >> (a.node & 31)) & 1u);
        const int h = wk.hk * p.G + gh;
        const bool store = used && ok;
        const bool whole = wk.whole();
        // partial results: slot 2 x + 1 for a unit that starts here and goes
        // on, 2 x for one that started before
        const long long prow = (static_cast<long long>(blockIdx.x) * 2 + (wk.k0 == 0 ? 1 : 0)) * (SPLIT ? kRows : 2 * kRows) +
                               (SPLIT ? 0 : t * kRows) + row;
        if constexpr (SPLIT) {
          if (works) {
            xm[t * kRows + row] = st.m;
            xl[t * kRows + row] = st.l;
            xb[t * kRows + row] = st.lb;
          }
          tc_fence_before();
          named_barrier(1, 256);
          tc_fence_after();
          if (works && ok) {
            const float m0 = xm[row], m1 = xm[kRows + row];
            const float M = fmaxf(m0, m1);
            const float f0 = m0 == -INFINITY ? 0.0f : ex2(m0 - M), f1 = m1 == -INFINITY ? 0.0f : ex2(m1 - M);
            const float l = xl[row] * f0 + xl[kRows + row] * f1, lb = xb[row] * f0 + xb[kRows + row] * f1;
            const bool any = l > 0.0f && !padding;
            const float inv = any ? 1.0f / lb : 0.0f;
            const float g0 = f0 * inv, g1 = f1 * inv;
            const uint32_t t0 = tmem + 256 + lane_base, t1 = t0 + D;
            // each warpgroup writes half of the columns
#pragma unroll 1
            for (int ch = t * (D / 2); ch < (t + 1) * (D / 2); ch += 16) {
              uint32_t o0[16], o1[16];
              tmem_ld16(t0 + ch, o0);
              tmem_ld_wait16(o0);
              if (n > 1) {
                tmem_ld16(t1 + ch, o1);
                tmem_ld_wait16(o1);
              } else {
#pragma unroll
                for (int x = 0; x < 16; ++x) o1[x] = 0u;
              }
              float r[16];
#pragma unroll
              for (int x = 0; x < 16; ++x)
                r[x] = any ? __uint_as_float(o0[x]) * g0 + __uint_as_float(o1[x]) * g1 : 0.0f;
              if (!store) continue;
              if (whole) {
                uint4 *dst = reinterpret_cast<uint4 *>(p.o + wk.b * p.so.b + h * p.so.h + a.node * p.so.n + ch);
#pragma unroll
                for (int x = 0; x < 2; ++x)
                  dst[x] = make_uint4(pack_bf16x2(r[8 * x], r[8 * x + 1]), pack_bf16x2(r[8 * x + 2], r[8 * x + 3]),
                                      pack_bf16x2(r[8 * x + 4], r[8 * x + 5]), pack_bf16x2(r[8 * x + 6], r[8 * x + 7]));
              } else {
                float4 *dst = reinterpret_cast<float4 *>(p.part_o + prow * D + ch);
#pragma unroll
                for (int x = 0; x < 4; ++x) dst[x] = make_float4(r[4 * x], r[4 * x + 1], r[4 * x + 2], r[4 * x + 3]);
              }
            }
            if (store && t == 0) {
              const float lse2 = any ? M + log2f(l) : -INFINITY;
              if (whole)
                p.lse[(static_cast<long long>(wk.b) * p.H + h) * p.Nt + a.node] = any ? lse2 * kLn2 : -INFINITY;
              else
                p.part_lse[prow] = padding ? INFINITY : lse2;
            }
          }
          tc_fence_before();
          named_barrier(2, 256);
        } else if (ok) {
          const bool any = st.l > 0.0f && !padding;
          const float inv = any ? 1.0f / st.lb : 0.0f;
#pragma unroll 1
          for (int ch = 0; ch < D; ch += 16) {
            uint32_t o0[16];
            tmem_ld16(a.tO + ch, o0);
            tmem_ld_wait16(o0);
            float r[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) r[x] = any ? __uint_as_float(o0[x]) * inv : 0.0f;
            if (!store) continue;
            if (whole) {
              uint4 *dst = reinterpret_cast<uint4 *>(p.o + wk.b * p.so.b + h * p.so.h + a.node * p.so.n + ch);
#pragma unroll
              for (int x = 0; x < 2; ++x)
                dst[x] = make_uint4(pack_bf16x2(r[8 * x], r[8 * x + 1]), pack_bf16x2(r[8 * x + 2], r[8 * x + 3]),
                                    pack_bf16x2(r[8 * x + 4], r[8 * x + 5]), pack_bf16x2(r[8 * x + 6], r[8 * x + 7]));
            } else {
              float4 *dst = reinterpret_cast<float4 *>(p.part_o + prow * D + ch);
#pragma unroll
              for (int x = 0; x < 4; ++x) dst[x] = make_float4(r[4 * x], r[4 * x + 1], r[4 * x + 2], r[4 * x + 3]);
            }
          }
          if (store) {
            const float lse2 = any ? st.m + log2f(st.l) : -INFINITY;
            if (whole)
              p.lse[(static_cast<long long>(wk.b) * p.H + h) * p.Nt + a.node] = any ? lse2 * kLn2 : -INFINITY;
            else
              p.part_lse[prow] = padding ? INFINITY : lse2;
          }
          tc_fence_before();
        }
        if (wk.masked()) {
          if (works && ok) warp_arrive(mask_empty);
          ++nmask;
        }
        g += n;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merge the partial results of units cut by a run's end: one block per row,
// the runs dealt to its warps, a lane owns D / 32 columns.
//   O = sum 2^(lse_s - M) O_s / sum 2^(lse_s - M)
template <int D, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) fa_tree_merge_kernel(const TreeParams p) {
  constexpr int CPL = D / 32;
  __shared__ long long sums[WARPS][2];
  __shared__ float sh_m[WARPS], sh_l[WARPS], sh_o[WARPS][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads_rows = p.G * p.Nt;
  const int unit = blockIdx.x / heads_rows, r = blockIdx.x % heads_rows;
  const int b = unit / p.Hkv, hk = unit % p.Hkv, gh = r / p.Nt, node = r % p.Nt;
  // first tile of the unit and the number of all tiles
  long long before = 0, total = 0;
  if (!p.cache_len) {
    const long long per_b = static_cast<long long>(p.Hkv) * tiles_of(p.Nk);
    before = per_b * b;
    total = per_b * p.B;
  } else {
    for (int x = threadIdx.x; x < p.B; x += WARPS * 32) {
      const int n = tiles_of(cache_rows(p.cache_len, x, p.Nk));
      total += n;
      if (x < b) before += n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    if (WARPS > 1) {
      if (lane == 0) sums[warp][0] = total, sums[warp][1] = before;
      __syncthreads();
      total = before = 0;
      for (int w = 0; w < WARPS; ++w) total += sums[w][0], before += sums[w][1];
    }
    total *= p.Hkv;
    before *= p.Hkv;
  }
  const int tiles = tiles_of(cache_rows(p.cache_len, b, p.Nk));
  const long long u0 = before + static_cast<long long>(hk) * tiles, u1 = u0 + tiles - 1;
  const long long runs = runs_of(p, total);
  const int c0 = static_cast<int>(((u0 + 1) * runs - 1) / total);  // the run that holds tile u0
  const int c1 = static_cast<int>(((u1 + 1) * runs - 1) / total);
  if (c0 == c1) return;  // written by its CTA
  const int mtile = gh / p.gpt, row = (gh % p.gpt) * p.Nt + node;
  const int group = p.split ? 0 : mtile / 2;
  const int slot_rows = p.split ? kRows : 2 * kRows;
  const int in_slot = (p.split ? 0 : (mtile & 1) * kRows) + row;
  float m = -INFINITY, l = 0.0f, o[CPL];
#pragma unroll
  for (int x = 0; x < CPL; ++x) o[x] = 0.0f;
#pragma unroll 4
  for (int c = c0 + warp; c <= c1; c += WARPS) {
    const long long pr =
        (static_cast<long long>(c * p.groups + group) * 2 + (c == c0 ? 1 : 0)) * slot_rows + in_slot;
    const float s = p.part_lse[pr];
    float v[CPL];
#pragma unroll
    for (int x = 0; x < CPL; ++x) v[x] = p.part_o[pr * D + lane * CPL + x];
    const float mn = fmaxf(m, s);
    if (mn == -INFINITY) continue;
    const float fa = m == -INFINITY ? 0.0f : ex2(m - mn), fb = s == mn ? 1.0f : (s == -INFINITY ? 0.0f : ex2(s - mn));
    l = l * fa + fb;
#pragma unroll
    for (int x = 0; x < CPL; ++x) o[x] = o[x] * fa + v[x] * fb;
    m = mn;
  }
  if (WARPS > 1) {
    if (lane == 0) sh_m[warp] = m, sh_l[warp] = l;
#pragma unroll
    for (int x = 0; x < CPL; ++x) sh_o[warp][lane * CPL + x] = o[x];
    __syncthreads();
    if (warp > 0) return;
    float M = -INFINITY;
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sh_m[w]);
    l = 0.0f;
#pragma unroll
    for (int x = 0; x < CPL; ++x) o[x] = 0.0f;
    for (int w = 0; w < WARPS; ++w) {
      const float f = sh_m[w] == M ? 1.0f : (sh_m[w] == -INFINITY ? 0.0f : ex2(sh_m[w] - M));
      l += sh_l[w] * f;
#pragma unroll
      for (int x = 0; x < CPL; ++x) o[x] += sh_o[w][lane * CPL + x] * f;
    }
    m = M;
  }
  const bool any = m != -INFINITY && m != INFINITY;  // +inf: padding
  const int h = hk * p.G + gh;
  __nv_bfloat16 *dst = p.o + b * p.so.b + h * p.so.h + node * p.so.n + lane * CPL;
#pragma unroll
  for (int x = 0; x < CPL; x += 2)
    *reinterpret_cast<uint32_t *>(dst + x) = any ? pack_bf16x2(o[x] / l, o[x + 1] / l) : 0u;
  if (lane == 0)
    p.lse[(static_cast<long long>(b) * p.H + h) * p.Nt + node] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <int D, bool SPLIT>
cudaError_t launch_tree_t(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const TreeParams &p,
                          bool merge, cudaStream_t stream) {
  using L = TreeLayout<D, SPLIT>;
  auto kern = fa_tree_kernel<D, SPLIT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kRequest);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(p.ranges) * p.groups, kThreads, L::kRequest, stream>>>(tq, tk, tv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || !merge) return e;
  const unsigned rows = static_cast<unsigned>(p.B) * p.Hkv * p.G * p.Nt;
  // runs a unit may be cut into
  if (p.ranges / (p.B * p.Hkv) >= 4)
    fa_tree_merge_kernel<D, 8><<<rows, 256, 0, stream>>>(p);
  else
    fa_tree_merge_kernel<D, 1><<<rows, 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

TreePlan plan_tree(int B, int H, int Hkv, int Nt, int Nk) {
  TreePlan pl{};
  const int G = H / Hkv;
  pl.gpt = kRows / Nt < G ? kRows / Nt : G;
  pl.row_tiles = (G + pl.gpt - 1) / pl.gpt;
  pl.split = pl.row_tiles == 1 ? 1 : 0;
  pl.groups = (pl.row_tiles + 1) / 2;
  const long long tiles = static_cast<long long>(B) * Hkv * ((Nk + kKeys - 1) / kKeys);
  long long ranges = kModelCtas / pl.groups;
  if (ranges < 1) ranges = 1;
  if (ranges > tiles) ranges = tiles;
  pl.ranges = static_cast<int>(ranges);
  pl.merge = ranges > 1 && Nk > kKeys;
  pl.part_rows = pl.merge ? static_cast<size_t>(ranges) * pl.groups * 2 * (pl.split ? kRows : 2 * kRows) : 0;
  return pl;
}

cudaError_t launch_tree(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const TreeParams &p,
                        bool merge, cudaStream_t stream) {
  if (p.d == 64)
    return p.split ? launch_tree_t<64, true>(tq, tk, tv, p, merge, stream)
                   : launch_tree_t<64, false>(tq, tk, tv, p, merge, stream);
  return p.split ? launch_tree_t<128, true>(tq, tk, tv, p, merge, stream)
                 : launch_tree_t<128, false>(tq, tk, tv, p, merge, stream);
}

}  // namespace fa
