// fa_tree.cu -- attention of a tree of drafted tokens over a key/value cache.
//
// Row (g, i) of a unit (b, hk) is tree node i under query head hk * G + g.
// It sees the cache rows before the tree, its own row and its ancestors'
// rows: softmax over those with a running maximum and sum, 128 keys at a
// time, as in the forward pass.
//
// What bounds it.  Every key costs 4 d bytes of cache and 4 d flops a row, so
// up to about 280 rows (the tensor rate over the HBM rate) the floor is the
// cache traffic: each K and V tile is read once for up to two row tiles of a
// unit, as A = Q (128 rows) against 128 keys on tcgen05 (a unit of more row
// tiles is walked once by each pair of them).  The 128-key tiles of all units
// form one list that is cut into equal runs, one per CTA (one CTA per SM),
// whatever the sequences' lengths; a unit cut by a run's end leaves partial
// results that a second kernel merges.
//   One row tile at d = 128 keeps to the floor but for the runs' ends and the
// merge (device times, B2 Hkv8 Nk65536, 79 us of traffic: 1 to 128 rows 89 to 93
// us; B16 H16 Nt32, ragged up to 16384 keys: 242 to 248 against 243).  With two
// row tiles the chain of each, S, softmax and P V, sets the pace (256 rows 128
// us), and at d = 64, where a tile has half the bytes and as many exponentials,
// with one as well (60 to 68 us and 104 against 40).  Three and four row tiles
// take as long, 230 and 236 us at d = 128: a lone tile's CTAs have half the work
// and as many SMs as a pair's.
//
// CTA (384 threads): warps 0..3 and 4..7 softmax (a row per thread), warp 8
// TMA producer (Q, and K and V tiles through one ring), warp 9 MMA issuer and
// TMEM owner, warp 10 the tree's visibility table, warp 11 idle.  With one
// row tile the two softmax warpgroups take alternate key tiles of it (each
// with its own maximum, sum and O, merged at the end of the unit); with two
// row tiles each takes its own.  TMEM columns: the S buffers (two of 128, three
// at d = 64 with one row tile), P (bf16) over S, and O_0, O_1 in the last 2 d.
//
// The tree.  Only a unit's last tiles hold nodes.  Warp 10 turns parents into
// one bit row per node (its ancestors and itself) by pointer doubling, at
// most seven rounds, into shared memory while earlier tiles are worked on;
// the softmax of those tiles tests bits.  Rows behind the sequence's end and
// padding nodes' rows are set to zero in the V tile, for 0 * NaN is NaN.
//
// Rounding.  Scores, maxima, sums, O and the partial results are fp32.  The
// weights of P V are rounded to bf16, since the product with bf16 V takes bf16 on
// its other side: off by at most 2^-8 of each, and O is divided by the sum of the
// rounded ones.
//
// Scores that are not finite.  A score of -inf weighs nothing: while a row has
// seen no other its maximum stays -inf and its exponents are taken relative to 0
// (-inf less -inf would be NaN).  A NaN that a row sees makes its sum NaN, and
// with it its O and logsumexp, through the merge of the runs as well.  A sum of
// zero marks a row that nothing was added to.

#include <cstdint>

#include "fa_cache.h"
#include "fa_runs.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kRows = 128;  // query rows of a row tile
constexpr int kThreads = 384;
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpMask = 10;
constexpr int kModelCtas = 152;  // GB300's SMs: the grid the runs are cut for
constexpr float kRescaleThreshold = 8.0f;  // a row's maximum moves only when exceeded by more (log2 units)
constexpr float kLn2 = 0.69314718055994530942f;
constexpr uint32_t kTmemCols = 512;
// Register split: 384 threads launched with 168 each; no role spills at 152 for
// the control warps and 176 for the softmax.  (At 104 and 200, the forward
// kernel's split, the issuer and the producer spill: B2 H32 Hkv8 Nt64 Nk65536
// d128 139 us against 127.)
constexpr uint32_t kRegsControl = 152, kRegsSoftmax = 176;
static_assert(128 * kRegsControl + 256 * kRegsSoftmax <= kThreads * 168, "register split");

template <int D, bool SPLIT>
struct TreeLayout {
  static constexpr int kSlabs = D / 64;
  static constexpr uint32_t kTile = kKeys * D * 2;                // a Q, K or V tile
  static constexpr int kQTiles = SPLIT ? 1 : 2;
  static constexpr int kSlots = D == 128 ? 5 : 10;                // ring of K and V tiles
  // S buffers.  With one row tile the key tiles take them in turn; a third one,
  // where TMEM has room for it, lets a warpgroup's next scores be formed while
  // it still works on the last ones: with few rows and 32 KB tiles that chain
  // and not HBM would set the pace (B2 H8 Hkv8 Nt1 Nk65536 d64: 66 us with
  // two, 61.5 with three and the cheaper merge).
  static constexpr int kSBufs = SPLIT && D == 64 ? 3 : 2;
  static constexpr uint32_t kO = kTmemCols - 2 * D;               // first O column
  static_assert(kSBufs * 128 <= kTmemCols - 2 * D, "TMEM columns");
  // first the small things, then (1 KB aligned) the tiles
  static constexpr uint32_t kOffBits = 0;                         // node bit rows, see bit_row()
  static constexpr uint32_t kOffDead = kOffBits + 32 * (1 + 2 + 3 + 4) * 4;
  static constexpr uint32_t kOffJump = kOffDead + 16;             // int8[128]: pointer doubling
  static constexpr uint32_t kOffRange = kOffJump + 128;           // the run's start (see RunStart)
  static constexpr uint32_t kOffScan = kOffRange + 48;            // 12 warps' sums
  static constexpr uint32_t kOffStats = kOffScan + 12 * 8;        // SPLIT: m, l, lb of both warpgroups
  static constexpr uint32_t kOffBar = kOffStats + (SPLIT ? 2 * 3 * kRows * 4 : 0);
  // full[S], empty[S], s_full[kSBufs], p_ready[2][2], pv_done[2][2], q_full, q_empty, mask_full, mask_empty, drain
  static constexpr int kNumBars = 2 * kSlots + kSBufs + 8 + 5;
  static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;    // TMEM address, abort flag
  static constexpr uint32_t kSmall = (kOffMisc + 16 + 15) / 16 * 16;
  static constexpr uint32_t kTiles = (kQTiles + kSlots) * kTile;
  static constexpr uint32_t kRequest = kSmall + 1008 + kTiles;    // dynamic shared memory starts 16-byte aligned
  static_assert(kOffBar % 8 == 0 && kOffRange % 8 == 0 && kOffScan % 8 == 0, "alignment");
  static_assert(kRequest <= 232448, "shared memory budget");
};

// The state of one softmax row over a segment.
struct RowState {
  float m, l, lb;
};

struct SoftmaxArgs {
  uint64_t *s_full, *p_ready, *pv_done, *full;
  uint32_t s_phase;  // of the tile's S buffer
  uint32_t tS, tO;   // its columns and this warpgroup's O, lane base added
  uint8_t *ring;    // K and V slots
  const uint32_t *bits, *dead;
  int node;         // tree node of this thread's row, -1 if the row is unused
  int warps;        // warps of the warpgroup that hold rows
};

// The running maximum moves to `cand` if that exceeds it by enough; returns
// whether it did, and the factor of what was summed before.
__device__ __forceinline__ bool move_max(RowState &st, float cand, float *alpha) {
  *alpha = 1.0f;
  if (!(cand > st.m + kRescaleThreshold)) return false;
  *alpha = ex2(st.m - cand);
  st.m = cand;
  return true;
}

// The P V product of this warpgroup's tile number k.
__device__ __forceinline__ bool pv_wait(const SoftmaxArgs &a, const WaitCtl &ctl, uint32_t k) {
  return mbar_wait(a.pv_done + (k & 1), (k >> 1) & 1, ctl, kSitePvDone);
}

// What a row's exponents are taken relative to.
__device__ __forceinline__ float exponent_base(const RowState &st) { return st.m == -INFINITY ? 0.0f : st.m; }

// O rescaled where a row's maximum moved (after the P V product before it).
template <int D>
__device__ __forceinline__ bool rescale_o(const SoftmaxArgs &a, const WaitCtl &ctl, uint32_t cnt, float alpha) {
  if (!__all_sync(0xffffffffu, pv_wait(a, ctl, cnt - 1))) return false;
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
  return true;
}

__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
  float m = fmax3(__uint_as_float(s[0]), __uint_as_float(s[1]), __uint_as_float(s[2]));
#pragma unroll
  for (int x = 3; x < 31; x += 2) m = fmax3(m, __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
  return fmaxf(m, __uint_as_float(s[31]));
}
__device__ __forceinline__ float min32(const uint32_t (&s)[32]) {
  float m = fmin3(__uint_as_float(s[0]), __uint_as_float(s[1]), __uint_as_float(s[2]));
#pragma unroll
  for (int x = 3; x < 31; x += 2) m = fmin3(m, __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
  return fminf(m, __uint_as_float(s[31]));
}

// One 128-key tile: scores from TMEM, running maximum and sum, P as bf16 over
// S, O rescaled when the maximum moves.  `cnt`: tiles this warpgroup has
// taken so far (barrier phases); first: its first tile of the segment.
template <int D>
__device__ __forceinline__ bool softmax_tile(const SoftmaxArgs &a, const TreeParams &p, const WaitCtl &ctl,
                                             RowState &st, uint32_t cnt, bool first) {
  const float c = p.scale_log2;
  if (!__all_sync(0xffffffffu, mbar_wait(a.s_full, a.s_phase, ctl, kSiteSFull))) return false;
  tc_fence_after();
  uint32_t s[4][32];
#pragma unroll
  for (int q = 0; q < 4; ++q) tmem_ld32(a.tS + q * 32, s[q]);
#pragma unroll
  for (int q = 0; q < 4; ++q) tmem_ld_wait(s[q]);
  float mx;
  if (!p.neg)
    mx = fmaxf(fmaxf(max32(s[0]), max32(s[1])), fmaxf(max32(s[2]), max32(s[3])));
  else
    mx = fminf(fminf(min32(s[0]), min32(s[1])), fminf(min32(s[2]), min32(s[3])));
  float alpha;
  const bool grow = move_max(st, mx * c, &alpha);
  const float base = exponent_base(st);
  const float2 cc = make_float2(c, c), nm = make_float2(-base, -base);
  uint32_t pk[4][16];
  float2 sf = make_float2(0.f, 0.f);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float2 sq = make_float2(0.f, 0.f);
#pragma unroll
    for (int x = 0; x < 32; x += 2) {
      const float2 y = ffma2(make_float2(__uint_as_float(s[q][x]), __uint_as_float(s[q][x + 1])), cc, nm);
      const float p0 = ex2(y.x), p1 = ex2(y.y);
      pk[q][x / 2] = pack_bf16x2(p0, p1);
      sq = fadd2(sq, make_float2(p0, p1));
    }
    tmem_st16(a.tS + q * 16, pk[q]);
    sf = fadd2(sf, sq);
  }
  tmem_st_wait();
  if (!first && __any_sync(0xffffffffu, grow) && !rescale_o<D>(a, ctl, cnt, alpha)) return false;
  tc_fence_before();
  warp_arrive(a.p_ready + (cnt & 1));

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

// The same for a tile that holds nodes or rows behind the end (its first key
// is node n0), at most two or three of a unit's tiles: a loop over the
// quarters, twice over S, because code that runs once per unit comes cold
// from memory (the unrolled form took 7000 cycles, most of them waiting for
// its instructions).  e_v: the V tile's place in the ring's sequence.
template <int D, int SLOTS>
__device__ __forceinline__ bool masked_tile(const SoftmaxArgs &a, const TreeParams &p, const WaitCtl &ctl,
                                            RowState &st, uint32_t cnt, bool first, uint32_t e_v, int n0) {
  const float c = p.scale_log2;
  if (!__all_sync(0xffffffffu, mbar_wait(a.s_full, a.s_phase, ctl, kSiteSFull))) return false;
  tc_fence_after();
  const int i = a.node;
  const bool live = i >= 0 && !((a.dead[i >> 5] >> (i & 31)) & 1u);
  const uint32_t hide = __float_as_uint(p.neg ? INFINITY : -INFINITY);
  float mx = __uint_as_float(hide);
  uint32_t any = 0;
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    const uint32_t see = visible(a.bits, i, live, n0 + 32 * q);
    any |= see;
    uint32_t s[32];
    tmem_ld32(a.tS + q * 32, s);
    tmem_ld_wait(s);
#pragma unroll
    for (int x = 0; x < 32; ++x)
      if (!((see >> x) & 1u)) s[x] = hide;
    mx = p.neg ? fminf(mx, min32(s)) : fmaxf(mx, max32(s));
  }
  float alpha;
  const bool grow = move_max(st, any ? mx * c : -INFINITY, &alpha);  // (0 * -inf is NaN)
  const float base = exponent_base(st);
  float2 sf = make_float2(0.f, 0.f), sb = sf;
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {  // P's quarter q lies over S's columns 16 q .. 16 q + 15, read by then
    const uint32_t see = visible(a.bits, i, live, n0 + 32 * q);
    uint32_t s[32], pk[16];
    tmem_ld32(a.tS + q * 32, s);
    tmem_ld_wait(s);
#pragma unroll
    for (int x = 0; x < 32; x += 2) {
      const float p0 = (see >> x) & 1u ? ex2(fmaf(__uint_as_float(s[x]), c, -base)) : 0.0f;
      const float p1 = (see >> (x + 1)) & 1u ? ex2(fmaf(__uint_as_float(s[x + 1]), c, -base)) : 0.0f;
      pk[x / 2] = pack_bf16x2(p0, p1);
      sf = fadd2(sf, make_float2(p0, p1));
      sb = add_bf16x2_f32(sb, pk[x / 2]);
    }
    tmem_st16(a.tS + q * 16, pk);
  }
  tmem_st_wait();
  if (!first && __any_sync(0xffffffffu, grow) && !rescale_o<D>(a, ctl, cnt, alpha)) return false;
  // V rows that no query row sees become zeros (0 * NaN is NaN)
  if (!__all_sync(0xffffffffu, mbar_wait(&a.full[e_v % SLOTS], (e_v / SLOTS) & 1, ctl, kSiteVFull))) return false;
  uint8_t *v = a.ring + (e_v % SLOTS) * (kKeys * D * 2);
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    const int lane = threadIdx.x & 31, node = n0 + 32 * q + lane;
    const bool gone = node >= p.Nt || (node >= 0 && ((a.dead[node >> 5] >> (node & 31)) & 1u));
    const uint32_t rows = __ballot_sync(0xffffffffu, gone);
    if (rows == 0) continue;
    // 16-byte pieces, a row's eight side by side
    for (int e = threadIdx.x & 127; e < 32 * 8; e += a.warps * 32) {
      if (!((rows >> (e >> 3)) & 1u)) continue;
#pragma unroll
      for (int sl = 0; sl < D / 64; ++sl)
        *reinterpret_cast<uint4 *>(v + sl * (kKeys * 128) + q * 32 * 128 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  warp_arrive(a.p_ready + (cnt & 1));
  st.l = st.l * alpha + (sf.x + sf.y);
  st.lb = st.lb * alpha + (sb.x + sb.y);
  return true;
}

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    fa_tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const TreeParams p) {
  using L = TreeLayout<D, SPLIT>;
  constexpr int S = L::kSlots, NS = L::kSBufs;
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
  uint64_t *s_full = empty + S;          // [buffer]
  // Each warpgroup's tiles take two barriers of each kind in turn.  With a third
  // S buffer a warpgroup may be through with a tile while the product of its
  // last one is still to come (S of tile x is issued after the product of tile
  // x - 3): the issuer would find p_ready two phases on, and the warpgroup
  // pv_done a phase short, and a parity wait can tell neither from the phase it
  // wants.  On a barrier that serves every other tile the phase before is done.
  uint64_t *p_ready = s_full + NS;       // [warpgroup][2]
  uint64_t *pv_done = p_ready + 4;       // [warpgroup][2]
  uint64_t *q_full = pv_done + 4, *q_empty = q_full + 1;
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
    for (int i = 0; i < NS; ++i) mbar_init(&s_full[i], 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&p_ready[2 * t], warps);
      mbar_init(&p_ready[2 * t + 1], warps);
      mbar_init(&pv_done[2 * t], 1);
      mbar_init(&pv_done[2 * t + 1], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(mask_full, 1);
    mbar_init(mask_empty, SPLIT || two ? 2 * warps : warps);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kWarpProducer && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  const bool has_run = find_run<kThreads>(p, c, run, reinterpret_cast<long long *>(small + L::kOffScan));
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // (thread 0 writes the cuts below, when its softmax comes to them)
  if (p.cuts && !p.cuts_by_unit && group == 0 && threadIdx.x == 0) p.cuts[c] = make_int4(-1, 0, 0, 0);
  if (!has_run) {
    if (warp == kWarpMma) tmem_dealloc(tmem, kTmemCols);
    return;
  }
  Walk wk(p, *run);

  if (warp >= kWarpProducer) {
    regs_decrease<kRegsControl>();
    if (warp == kWarpProducer && lane == 0) {
      // ---------------------------------------------------------- producer
      uint32_t e = 0, nq = 0;   // ring loads and Q loads so far
      uint32_t sl = 0, ph = 0;  // the ring's next slot and its phase
      bool ok = true;
      auto load = [&](const CUtensorMap *map, int row) -> bool {
        if (!mbar_wait(&empty[sl], ph ^ 1, ctl, kSiteKvEmpty)) return false;
#ifdef FA_TEST_SKIP_FIRST_V_LOAD
        // Test builds only: the run's first V tile is never loaded, so the wait
        // for it runs out and the bounded-wait path is taken.
        if (e == 1) {
          ++e;
          ++sl;
          return true;
        }
#endif
        mbar_arrive_expect_tx(&full[sl], L::kTile);
#pragma unroll
        for (int x = 0; x < L::kSlabs; ++x)
          tma_load_4d(ring + sl * L::kTile + x * kKeys * 128, map, &full[sl], x * 64, row, wk.hk, wk.b);
        ++e;
        if (++sl == S) {
          sl = 0;
          ph ^= 1;
        }
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
      const uint64_t dQ = sdesc_sw128(smem_addr(sQ), 16, 1024);
      const uint64_t dK = sdesc_sw128(smem_addr(ring), 16, 1024);             // slot 0 as a K tile
      const uint64_t dV = sdesc_sw128(smem_addr(ring), kKeys * 128, 1024);    // and as a V tile
      // A place in the ring's sequence of loads K_0 V_0 K_1 V_1 ...: its slot
      // and phase, stepped from tile to tile without a division.
      struct Place {
        uint32_t slot, phase;
        __device__ void next_tile() {
          slot += 2;
          if (slot >= S) {
            slot -= S;
            phase ^= 1;
          }
        }
      };
      Place kp{0, 0}, vp{1, 0};
      uint32_t nq = 0;            // Q loads so far
      uint32_t cnt[2] = {0, 0};   // P V products per warpgroup so far
      uint32_t ss = 0, ps = 0;    // buffers of the next S and of the next P V product (one row tile)
      bool ok = true;
      auto full_wait = [&](const Place &x, int site) {
        const bool r = mbar_wait(&full[x.slot], x.phase, ctl, site);
        tc_fence_after();
        return r;
      };
      // S in buffer s = the warpgroup's Q tile times the K tile at x
      auto issue_s = [&](uint32_t s, const Place &x) {
        const uint64_t dq = desc_add(dQ, (SPLIT ? 0 : s) * L::kTile), dk = desc_add(dK, x.slot * L::kTile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + s * 128, desc_add(dq, kmajor_step(kk, kRows)), desc_add(dk, kmajor_step(kk, kKeys)), kIdS,
                 kk > 0 ? 1u : 0u);
        tc_commit(&s_full[s]);
      };
      // O_t += P (over S in buffer s) times the V tile at x
      auto issue_pv = [&](int t, uint32_t s, const Place &x, bool first) -> bool {
        const uint32_t bar = 2 * t + (cnt[t] & 1);
        if (!mbar_wait(&p_ready[bar], (cnt[t] >> 1) & 1, ctl, kSitePReady)) return false;
        ++cnt[t];
        tc_fence_after();
        const uint64_t dv = desc_add(dV, x.slot * L::kTile);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          mma_ts(tmem + L::kO + t * D, tmem + s * 128 + kk * 8, desc_add(dv, mnmajor_step(kk)), kIdO,
                 (!first || kk > 0) ? 1u : 0u);
        tc_commit(&pv_done[bar]);
        return true;
      };
      while (ok && wk.next()) {
        const int n = wk.k1 - wk.k0;
        if (!(ok = mbar_wait(q_full, nq & 1, ctl, kSiteQFull))) break;
        tc_fence_after();
        if constexpr (SPLIT) {
          // tile x of the segment belongs to warpgroup x & 1; its S is issued
          // right after the P V product that frees its buffer
          for (int x = 0; ok && x < n + NS; ++x) {
            const int y = x - NS;
            if (y >= 0 && y < n) {
              ok = full_wait(vp, kSiteVFull) && issue_pv(y & 1, ps, vp, y < 2);
              if (ok) tc_commit(&empty[vp.slot]);
              vp.next_tile();
              if (++ps == NS) ps = 0;
            }
            if (ok && x < n) {
              if (!(ok = full_wait(kp, kSiteKFull))) break;
              issue_s(ss, kp);
              tc_commit(&empty[kp.slot]);
              kp.next_tile();
              if (++ss == NS) ss = 0;
              if (x == n - 1) tc_commit(q_empty);
            }
          }
        } else {
          for (int x = 0; ok && x <= n; ++x) {
            if (x > 0 && !(ok = full_wait(vp, kSiteVFull))) break;
            if (x > 0 && !(ok = issue_pv(0, 0, vp, x == 1))) break;
            if (x < n) {
              if (!(ok = full_wait(kp, kSiteKFull))) break;
              issue_s(0, kp);
            }
            if (x > 0) {
              if (two && !(ok = issue_pv(1, 1, vp, x == 1))) break;
              tc_commit(&empty[vp.slot]);
              vp.next_tile();
            }
            if (x < n) {
              if (two) issue_s(1, kp);
              tc_commit(&empty[kp.slot]);
              kp.next_tile();
              if (x == n - 1) tc_commit(q_empty);
            }
          }
        }
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
      a.p_ready = &p_ready[2 * t];
      a.pv_done = &pv_done[2 * t];
      a.full = full;
      a.tS = tmem + t * 128 + lane_base;
      a.tO = tmem + L::kO + t * D + lane_base;
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
        // what the merge has to do for a unit that starts here: nothing, or its
        // runs if it goes on in the next ones
        if (threadIdx.x == 0 && group == 0 && p.cuts && wk.k0 == 0 && (!wk.tail || p.cuts_by_unit))
          p.cuts[p.cuts_by_unit ? wk.b * p.Hkv + wk.hk : c] =
              wk.tail ? make_int4(-1, 0, 0, 0)
                      : make_int4(wk.b, wk.hk, c,
                                  static_cast<int>(divide((wk.u0 + wk.tiles) * run->runs - 1, run->total)));
        RowState st{-INFINITY, 0.0f, 0.0f};
        if (works && ok) {
          bool have_mask = false;
          const int step = SPLIT ? 2 : 1;
          for (int x = SPLIT ? t : 0; ok && x < n; x += step) {
            const int kt = wk.k0 + x;
            if (SPLIT) {
              const uint32_t q = g + x, s = q % NS;
              a.s_full = &s_full[s];
              a.s_phase = (q / NS) & 1;
              a.tS = tmem + s * 128 + lane_base;
            } else {
              a.s_phase = cnt & 1;
            }
            const bool first = x < step;
            if (kt >= mfrom) {
              if (!have_mask) {
                ok = __all_sync(0xffffffffu, mbar_wait(mask_full, nmask & 1, ctl, kSiteMaskFull));
                have_mask = true;
                if (!ok) break;
              }
              ok = masked_tile<D, S>(a, p, ctl, st, cnt, first, 2 * (g + x) + 1, kt * kKeys - wk.base());
            } else {
              ok = softmax_tile<D>(a, p, ctl, st, cnt, first);
            }
            ++cnt;
          }
          if (ok && wk.masked() && !have_mask)
            ok = __all_sync(0xffffffffu, mbar_wait(mask_full, nmask & 1, ctl, kSiteMaskFull));
          if (ok && cnt > 0 && n > (SPLIT ? t : 0))
            ok = __all_sync(0xffffffffu, pv_wait(a, ctl, cnt - 1));
        }
        tc_fence_after();
        // ---- the segment's result
        const bool padding = wk.tail && a.node >= 0 && works && ok && ((dead[a.node >> 5] >> (a.node & 31)) & 1u);
        const int h = wk.hk * p.G + gh;
        const bool store = used && ok;
        const bool whole = wk.whole();
        // partial results: slot 2 x + 1 for a unit that starts here and goes
        // on, 2 x for one that started before
        constexpr int kSlotRows = SPLIT ? kRows : 2 * kRows;
        const long long slot = static_cast<long long>(blockIdx.x) * 2 + (wk.k0 == 0 ? 1 : 0);
        const int srow = (SPLIT ? 0 : t * kRows) + row;
        float *part_o = p.part_o + slot * (kSlotRows * D) + srow;  // [column][row]: a warp's rows side by side
        const long long prow = slot * kSlotRows + srow;
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
            const bool any = l != 0.0f && !padding;
            const float inv = any ? 1.0f / lb : 0.0f;
            const float g0 = f0 * inv, g1 = f1 * inv;
            const uint32_t t0 = tmem + L::kO + lane_base, t1 = t0 + D;
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
#pragma unroll
                for (int x = 0; x < 16; ++x) part_o[(ch + x) * kSlotRows] = r[x];
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
          const bool any = st.l != 0.0f && !padding;
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
#pragma unroll
              for (int x = 0; x < 16; ++x) part_o[(ch + x) * kSlotRows] = r[x];
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

// Merge the partial results of units cut by a run's end (the unit that starts
// in a run and goes on in the next ones; at most one a run):
//   O = sum 2^(lse_s - M) O_s / sum 2^(lse_s - M).
// A lane takes a row and 16 columns, a warp ROWS rows and 16 * 32 / ROWS
// columns of one unit's row tile; the block's WARPS warps deal the runs out
// among themselves and add up through shared memory, so that a unit cut into
// a hundred runs is merged in a few round trips.
constexpr int kMergeCols = 16;

// The greater of two runs' logsumexps: +inf, the mark of padding, before NaN,
// and NaN before every other value.
__device__ __forceinline__ float merge_max(float a, float b) {
  const float x = fmaxf(a, b);
  return x != INFINITY && (a != a || b != b) ? NAN : x;
}

template <int D, int ROWS, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) fa_tree_merge_kernel(const TreeParams p) {
  constexpr int kCols = kMergeCols * 32 / ROWS;  // of a block
  __shared__ float sh_m[WARPS][32], sh_l[WARPS][32], sh_o[WARPS][32][kMergeCols + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int used = p.gpt * p.Nt, row_groups = (used + ROWS - 1) / ROWS;
  int x = blockIdx.x;
  const int c0 = x % (D / kCols) * kCols + lane / ROWS * kMergeCols;
  x /= D / kCols;
  const int row = x % row_groups * ROWS + lane % ROWS;
  x /= row_groups;
  const int mtile = x % p.row_tiles;
  const int gh = mtile * p.gpt + row / p.Nt, node = row % p.Nt;
  const bool on = row < used && gh < p.G;
  cudaGridDependencySynchronize();  // (launched while the main kernel still runs)
  const int4 cut = p.cuts[x / p.row_tiles];
  const int b = cut.x, hk = cut.y, r0 = cut.z, r1 = cut.w;
  // nothing was cut here (b = -1); after a timeout the entry may hold anything
  if (b < 0 || b >= p.B || hk < 0 || hk >= p.Hkv || r0 < 0 || r0 >= r1 || r1 >= p.ranges) return;

  const int group = p.split ? 0 : mtile / 2, slot_rows = p.split ? kRows : 2 * kRows;
  const int in_slot = (p.split ? 0 : (mtile & 1) * kRows) + row;
  float m = -INFINITY, l = 0.0f, o[kMergeCols];
#pragma unroll
  for (int y = 0; y < kMergeCols; ++y) o[y] = 0.0f;
#pragma unroll 2
  for (int r = r0 + warp; r <= r1; r += WARPS) {
    const long long slot = static_cast<long long>(r * p.groups + group) * 2 + (r == r0 ? 1 : 0);
    const float s = on ? p.part_lse[slot * slot_rows + in_slot] : -INFINITY;
    const float *part = p.part_o + (slot * D + c0) * slot_rows + in_slot;
    float v[kMergeCols];
#pragma unroll
    for (int y = 0; y < kMergeCols; ++y) v[y] = on ? part[y * slot_rows] : 0.0f;
    const float mn = merge_max(m, s);
    const float fa = m == mn ? 1.0f : (m == -INFINITY ? 0.0f : ex2(m - mn));
    const float fb = s == -INFINITY ? 0.0f : (s == mn ? 1.0f : ex2(s - mn));
    l = l * fa + fb;
#pragma unroll
    for (int y = 0; y < kMergeCols; ++y) o[y] = o[y] * fa + v[y] * fb;
    m = mn;
  }
  sh_m[warp][lane] = m;
  sh_l[warp][lane] = l;
#pragma unroll
  for (int y = 0; y < kMergeCols; ++y) sh_o[warp][lane][y] = o[y];
  __syncthreads();
  if (warp > 0) return;
  float M = -INFINITY;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) M = merge_max(M, sh_m[w][lane]);
  l = 0.0f;
#pragma unroll
  for (int y = 0; y < kMergeCols; ++y) o[y] = 0.0f;
  for (int w = 0; w < WARPS; ++w) {
    const float mw = sh_m[w][lane], f = mw == -INFINITY ? 0.0f : (mw == M ? 1.0f : ex2(mw - M));
    l += sh_l[w][lane] * f;
#pragma unroll
    for (int y = 0; y < kMergeCols; ++y) o[y] += sh_o[w][lane][y] * f;
  }
  if (!on) return;
  const bool any = M != -INFINITY && M != INFINITY;  // +inf: padding
  const float inv = any ? 1.0f / l : 0.0f;
  const int h = hk * p.G + gh;
  uint4 *dst = reinterpret_cast<uint4 *>(p.o + b * p.so.b + h * p.so.h + node * p.so.n + c0);
#pragma unroll
  for (int y = 0; y < kMergeCols; y += 8)
    dst[y / 8] = any ? make_uint4(pack_bf16x2(o[y] * inv, o[y + 1] * inv), pack_bf16x2(o[y + 2] * inv, o[y + 3] * inv),
                                  pack_bf16x2(o[y + 4] * inv, o[y + 5] * inv), pack_bf16x2(o[y + 6] * inv, o[y + 7] * inv))
                     : make_uint4(0u, 0u, 0u, 0u);
  if (c0 == 0)
    p.lse[(static_cast<long long>(b) * p.H + h) * p.Nt + node] = any ? (M + log2f(l)) * kLn2 : -INFINITY;
}

// The merge is launched as a dependent of the main kernel: its launch is set up
// while that one runs.  The main kernel triggers nothing early, so the blocks of
// the merge are placed when its last CTA has left.
template <int D, int ROWS, int WARPS>
cudaError_t launch_merge(const TreeParams &p, cudaStream_t stream) {
  const long long cuts = p.cuts_by_unit ? static_cast<long long>(p.B) * p.Hkv : p.ranges;
  const long long blocks = cuts * p.row_tiles * ((p.gpt * p.Nt + ROWS - 1) / ROWS) *
                           (D / (kMergeCols * 32 / ROWS));  // (at most 152 runs per pair of row tiles)
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(WARPS * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_tree_merge_kernel<D, ROWS, WARPS>, p);
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
  // a unit is cut into about ranges / units + 1 runs
  const bool many = p.ranges >= 2ll * p.B * p.Hkv;
  if (SPLIT && p.gpt * p.Nt <= 8)
    return many ? launch_merge<D, 8, 8>(p, stream) : launch_merge<D, 8, 2>(p, stream);
  return many ? launch_merge<D, 32, 8>(p, stream) : launch_merge<D, 32, 2>(p, stream);
}

}  // namespace

// Short caches are not cut inside a unit: up to 8 tiles take about as long as
// the merge that their cutting would need (B1 H8 Hkv2 Nt7 on the device: Nk1000
// 13.7 us cut into 16 runs, 15.4 whole; Nk500 13.5 and 12.0), and without a
// workspace and a second launch the whole call goes from 29 to 24 us.
constexpr int kWholeTiles = 8;

TreePlan plan_tree(int B, int H, int Hkv, int Nt, int Nk) {
  TreePlan pl{};
  const int G = H / Hkv;
  pl.gpt = kRows / Nt < G ? kRows / Nt : G;
  pl.row_tiles = (G + pl.gpt - 1) / pl.gpt;
  pl.split = pl.row_tiles == 1 ? 1 : 0;
  pl.groups = (pl.row_tiles + 1) / 2;
  const int per_unit = (Nk + kKeys - 1) / kKeys;
  const long long units = static_cast<long long>(B) * Hkv;
  pl.whole = per_unit <= kWholeTiles ? 1 : 0;
  const long long pieces = pl.whole ? units : units * per_unit;
  long long ranges = kModelCtas / pl.groups;
  if (ranges < 1) ranges = 1;
  if (ranges > pieces) ranges = pieces;
  pl.ranges = static_cast<int>(ranges);
  pl.merge = ranges > 1 && !pl.whole;
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
