// fa_tree_fp8_tc.cu -- attention of the newest rows of each sequence, or of a tree
// of drafted tokens, over a cache held in 8 bits, up to 32 query rows of a cache
// head, on tcgen05's 8-bit form.
//
// Both products run on the cache's codes as TMA leaves them in shared memory, with
// nothing converted: S^T = K Q^T (a lane per key, a column per query row) and
// O^T = V^T P^T (a lane per column of V).  q and the weights P are each the sum of
// two e4m3 parts, the nearest value and that of what is left; the parts are columns
// of their own of one product (N = 2 C for C query rows) and are added in fp32.
//
// Scales.  A score is scale * ks * (q . codes).  A value's scale goes into its
// weight: with r_j = vs_j / (the tile's greatest vs), e_j = t_j + log2 r_j (t_j the
// score in log2 units) and m = max e_j over the tile's 128 keys,
//     P_j = 2^(e_j - m + 8),   O += 2^(m + log2 vs_max - A - 8) (P codes),
//     l  += 2^(m - M - 8) sum P_j / r_j,   o = 2^(A - M) O / l,
// with references of their own for l and O: M near the greatest m and A near the greatest
// m + log2 vs_max, so that neither sum leaves fp32's range, whatever the scales are.  A
// tile's weights always reach up to 2^8: e4m3's second part ends at 2^-10, 2^-18 of the
// tile's greatest weighted value, and a long flat tail beside one sharp key keeps its
// weight.  That takes a fresh O^T a tile, which a warpgroup adds to fp32 registers.
// vs_max is taken over the slices of 16 keys that some row sees; r_j is 2^-100 at least
// (1 / r_j has to stay in fp32).
//
// Rounding.  A row of q is divided by a power of two (2^-100 or more) so that its greatest
// value lies in (224, 448]; bf16's 8 bits are 4 + 4, so its parts are exact but where the second
// falls below e4m3's least step: off by at most 2^-10, 2^-17.8 of the row's greatest
// value.  A weight is rounded to its parts likewise: off by at most 2^-9 of itself, or
// 2^-10 with its tile's greatest at 2^8; l adds up the unrounded weights.  Scores, maxima,
// sums and O are fp32.
//
// What bounds it.  HBM, 2 d bytes a key: a 128-key tile takes an SM 1400 cycles of its
// share of the traffic at d = 128, its products some 560 (a tcgen05 instruction takes 60 or
// more whatever its N) and its softmax about 10 issue slots a row and warp.  Up to 8
// rows: B16 H16 T1 Nk16384 (1.1 GB) 162 us, 0.98 of the copy bandwidth.  32 rows: B16 H16
// T32 Nk16384 (lengths of three quarters on average, 0.8 GB) 176 us, 0.70, and B2 H32 Hkv8
// T5 Nk100001 (0.4 GB) 86 us, 0.70, where a run of 82 tiles has a start, an end and a
// second launch to pay for: 63 % of the issue slots, and the way of a tile through
// its softmax (1750 cycles a tile).  d = 64: a tile has half the bytes and takes the same
// steps, 110 us for the first (0.54 GB), 187 for the second's shape with full caches.
// Codes converted to f16 for mma.sync took 210, 470 and 170 us, 160 and 253 at d = 64.
//
// CTA: four warpgroups of softmax, a key per thread, which take the tiles in turn (32
// rows: two a tile, 16 columns each); one that adds up O^T, a column of V per thread; then
// the TMA producer, a warp that issues S^T and owns TMEM, one that issues O^T (one thread
// for both took 1950 cycles a tile, most of them in the instructions themselves), and
// one for q's parts and the tree's table.  TMEM: four S^T and four O^T of 2 C columns.
// The tiles of all units form one list that is cut into equal runs (fa_runs.cuh), and a
// CTA's products run on from unit to unit.

#include <cstdint>

#include "fa_cache8.h"
#include "fa_parts.cuh"
#include "fa_runs.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr float kMoveBy = 8.0f;   // a running maximum moves only when exceeded by more (log2 units)
constexpr float kLift = 8.0f;     // weights reach 2^kLift
constexpr float kLn2 = 0.69314718055994530942f;
// The CTA's warps: four warpgroups of softmax, then one that adds up O^T, then the
// control warps.  A softmax warpgroup takes 16 columns of a tile: with 32 columns two
// share a tile (one with all 32 would need 112 registers, and code that does not stay in
// the instruction cache: three of them took 1830 cycles a tile).  Registers: launched
// with kRegsLaunch a thread, split by setmaxnreg; that many is what the compiler keeps to
// in every role, and it spills for it: 152 to 160 bytes stored (340 to 368 loaded) with 16 and
// 32 columns, 88 to 100 (196 to 208) with 8.
constexpr int kGroups = 4, kSoftmaxWarps = 4 * kGroups, kThreads = 128 * (kGroups + 2);
constexpr int kWarpAdd = kSoftmaxWarps, kWarpProducer = kWarpAdd + 4, kWarpS = kWarpProducer + 1;
constexpr int kWarpO = kWarpProducer + 2, kWarpQ = kWarpProducer + 3;
constexpr uint32_t kRegsLaunch = 80, kRegsSoftmax = 88, kRegsAdd = 80, kRegsControl = 48;
static_assert(128 * (kGroups * kRegsSoftmax + kRegsAdd + kRegsControl) <= kThreads * kRegsLaunch, "register split");
static_assert(kRegsSoftmax >= kRegsLaunch && kRegsAdd >= kRegsLaunch && kRegsControl <= kRegsLaunch,
              "setmaxnreg goes up or down only");

template <int D, int C>
struct LayoutTc {
  static constexpr int kCols = C < 16 ? C : 16;           // of a softmax warpgroup
  static constexpr int kHalves = C / kCols, kAtWork = kGroups / kHalves;  // warpgroups of a tile, tiles at work
  static constexpr uint32_t kTile = kKeys * D;         // a K or V tile
  static constexpr int kBufs = 4;                      // of S^T, and of O^T
  // Slots of K and of V: as many as buffers, so that the barrier of a product tells of its operand's slot as well (a
  // commit of its own for that: B16 H16 T32 Nk16384, full caches, 215 us for 203).  V tiles are asked for kLag tiles
  // after their K: S^T runs about so far ahead of O^T, and a V tile that came with its K would hold its slot meanwhile.
  static constexpr int kSlots = kBufs, kLag = 3;
  static constexpr uint32_t kTmem = 2 * kBufs * 2 * C;
  static_assert(kTmem <= 512, "TMEM columns");
  // How many of what one role leaves to another are used in turn.
  // A tile's maxima: tile x + 8's are written by warpgroups that saw tile x + 4 - kAtWork added up at their tile before,
  // or a later one, so x; buffer x % kBufs of the weights is free when tile x - kBufs has been added up.
  static constexpr int kTiles = 8;
  static_assert(kBufs >= kAtWork && kTiles >= kBufs + kAtWork, "tile x's maxima have been read by then");
  // A segment's row factors: segment n + NB + 3's are written when S^T of segment n + NB + 1 is done, so that of a tile
  // beyond x + NB, x any of segment n's, and that takes tile x's scores read.
  static constexpr int kSegs = 8;
  static_assert(kSegs >= kBufs + 3, "segment n's factors have been read by then");
  static constexpr uint32_t kQ = 2 * C * D;            // q's parts (two segments' in turn)
  // first the small things, then (1 KB aligned) ring, P, q
  static constexpr uint32_t kOffBits = 0;
  static constexpr uint32_t kOffDead = kOffBits + 32 * (1 + 2 + 3 + 4) * 4;
  static constexpr uint32_t kOffJump = kOffDead + 16;
  static constexpr uint32_t kOffRange = kOffJump + 128;
  static constexpr uint32_t kOffScan = kOffRange + 48;                    // warps' sums
  static constexpr uint32_t kOffMost = kOffScan + 24 * 8;                 // [2][softmax warps][kCols] greatest e, in turn
  static constexpr uint32_t kOffBase = kOffMost + 2 * kSoftmaxWarps * kCols * 4;   // [softmax warps][2][kCols]: 8 - m, l's factor
  static constexpr uint32_t kOffTileM = kOffBase + kSoftmaxWarps * 2 * kCols * 4;  // [kTiles][C] m + log2 vs_max
  static constexpr uint32_t kOffAdd = kOffTileM + kTiles * C * 4;         // [4 warps][C]: factors of O
  static constexpr uint32_t kOffL = kOffAdd + 4 * C * 4;                  // [softmax warps][kCols] l, and [groups][kCols] its base
  static constexpr uint32_t kOffLm = kOffL + kSoftmaxWarps * kCols * 4;
  static constexpr uint32_t kOffRow = kOffLm + kGroups * kCols * 4;           // [kSegs][C] rows' factors
  static constexpr uint32_t kOffBar = kOffRow + kSegs * C * 4;
  // k_full[slots], v_full[slots], s_full[bufs], s_free[bufs], pv_done[bufs], o_empty[bufs], p_ready[bufs], q_full[2],
  // q_empty[2], mask_full, mask_empty, l_full, l_empty, drain[2]
  static constexpr int kNumBars = 2 * kSlots + 5 * kBufs + 10;
  static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;            // TMEM address, abort flag
  static constexpr uint32_t kSmall = (kOffMisc + 16 + 15) / 16 * 16;
  static constexpr uint32_t kRing = 2 * kSlots * kTile;
  static constexpr uint32_t kPTile = kKeys * 64, kP = kBufs * kPTile;  // weights: 64 bytes a key, 2 C used
  static constexpr uint32_t kRequest = kSmall + 1008 + kRing + kP + 2 * kQ;
  static_assert(kOffBar % 8 == 0 && kOffRange % 8 == 0 && kOffScan % 8 == 0 && kOffMost % 16 == 0, "alignment");
  static_assert(kRequest <= 232448, "shared memory budget");
};

// Sums over the warp's lanes of N values each: lane l gets the sum of value l % N, in a
// fixed order.
template <int N>
__device__ __forceinline__ float lane_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = N / 2; o; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int x = 0; x < o; ++x) {
      const float keep = up ? v[x + o] : v[x], send = up ? v[x] : v[x + o];
      v[x] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
#pragma unroll
  for (int o = N; o < 32; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

// N columns' two parts, of this thread's lane: hi at `at`, lo C columns on.
template <int C, int N>
__device__ __forceinline__ void tmem_parts(uint32_t at, uint32_t (&hi)[N], uint32_t (&lo)[N]) {
  if constexpr (N == 16) {
    tmem_ld16(at, hi);
    tmem_ld16(at + C, lo);
    tmem_ld_wait16(hi);
    tmem_ld_wait16(lo);
  } else {
    static_assert(N == 8 && C == 8, "side by side");
    uint32_t w[16];
    tmem_ld16(at, w);
    tmem_ld_wait16(w);
#pragma unroll
    for (int y = 0; y < 8; ++y) hi[y] = w[y], lo[y] = w[8 + y];
  }
}

template <int D, int C>
__global__ void __launch_bounds__(kThreads, 1)
    fa_tree_fp8_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          const Tree8Params p) {
  using L = LayoutTc<D, C>;
  constexpr int kCols = L::kCols;
  constexpr int kAddWarps = D / 32;  // with columns of V
  constexpr int NB = L::kBufs, kLag = L::kLag;
  // (lane l of a warp looks after column l % C where a thing is done once a column)
  extern __shared__ uint8_t smem_raw[];
  uint8_t *small = smem_raw;
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + L::kSmall + 1023) &
                                              ~uintptr_t(1023));
  uint8_t *ring_v = ring + NB * L::kTile, *sP = ring + L::kRing, *sQ = sP + L::kP;
  uint32_t *bits = reinterpret_cast<uint32_t *>(small + L::kOffBits);
  uint32_t *dead = reinterpret_cast<uint32_t *>(small + L::kOffDead);
  RunStart *run = reinterpret_cast<RunStart *>(small + L::kOffRange);
  auto floats = [&](uint32_t off) { return reinterpret_cast<float *>(small + off); };
  float *tile_m = floats(L::kOffTileM), *row_f = floats(L::kOffRow);
  float *sum_l = floats(L::kOffL), *sum_m = floats(L::kOffLm);
  uint64_t *k_full = reinterpret_cast<uint64_t *>(small + L::kOffBar), *v_full = k_full + NB;
  // Tile x of the run uses number x % NB of the buffers' barriers.  No wait can find its barrier two phases on: tile
  // x + NB's product waits for what tile x's readers arrive on, and its weights for tile x's sums.
  uint64_t *s_full = v_full + NB, *s_free = s_full + NB, *pv_done = s_free + NB, *o_empty = pv_done + NB;
  uint64_t *p_ready = o_empty + NB;
  uint64_t *q_full = p_ready + NB, *q_empty = q_full + 2, *mask_full = q_empty + 2, *mask_empty = mask_full + 1;
  uint64_t *l_full = mask_empty + 1, *l_empty = l_full + 1, *drain = l_empty + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(small + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(small + L::kOffMisc + 4);
  const WaitCtl ctl{abort_flag, p.status};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = blockIdx.x % p.groups, c = blockIdx.x / p.groups;
  const int first_row = group * C, unit_rows = p.G * p.Nt;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NB; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4 * L::kHalves);
      mbar_init(&p_ready[i], 4 * L::kHalves);
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_empty[i], kAddWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    mbar_init(mask_full, 1);
    mbar_init(mask_empty, kSoftmaxWarps + kAddWarps);
    mbar_init(l_full, kSoftmaxWarps);
    mbar_init(l_empty, kAddWarps);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpS) {
    tmem_alloc(tmem_slot, L::kTmem);
    tmem_relinquish();
  }
  if (warp == kWarpProducer && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  const bool has_run = find_run<kThreads>(p, c, run, reinterpret_cast<long long *>(small + L::kOffScan));
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // (the thread that writes the cuts below writes this one, so that the two stores have an order)
  if (p.cuts && !p.cuts_by_unit && group == 0 && threadIdx.x == kWarpAdd * 32) p.cuts[c] = make_int4(-1, 0, 0, 0);
  if (!has_run) {
    if (warp == kWarpS) tmem_dealloc(tmem, L::kTmem);
    return;
  }
  Walk<Tree8Params> wk(p, *run);
  const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;

  if (warp >= kWarpProducer) {
    regs_decrease<kRegsControl>();
    if (warp == kWarpProducer && lane == 0) {
      // ---------------------------------------------------------- producer
      const uint32_t total = static_cast<uint32_t>(wk.end - wk.t);
      uint32_t ks = 0, kph = 1, vs = 0, vph = 1;  // the next slots and their phases
      uint32_t nk = 0, nv = 0;                    // tiles asked for
      int left = 0, row = 0;
      int4 ahead[kLag];                           // where the K tiles whose V is still to come lie
      bool ok = true;
#pragma unroll
      for (int i = 0; i < kLag; ++i) ahead[i] = make_int4(0, 0, 0, 0);
      for (uint32_t y = 0; ok && y < total + kLag; ++y) {
        const int4 v = ahead[0];
#pragma unroll
        for (int i = 0; i + 1 < kLag; ++i) ahead[i] = ahead[i + 1];
        if (y < total) {
          if (left == 0) {
            wk.next();
            left = wk.k1 - wk.k0;
            row = wk.k0 * kKeys;
          }
          // (the slot's last tile has been multiplied)
          if (!(ok = mbar_wait(&s_full[ks], kph, ctl, kSiteKEmpty))) break;
          mbar_arrive_expect_tx(&k_full[ks], L::kTile);
          tma_load_4d(ring + ks * L::kTile, &tm_k, &k_full[ks], 0, row, wk.hk, wk.b);
          ++nk;
          if (++ks == NB) {
            ks = 0;
            kph ^= 1;
          }
          ahead[kLag - 1] = make_int4(row, wk.hk, wk.b, 0);
          row += kKeys;
          --left;
        }
        if (y >= kLag) {
          if (!(ok = mbar_wait(&pv_done[vs], vph, ctl, kSiteVEmpty))) break;
#ifdef FA_TEST_SKIP_FIRST_V_LOAD
          // Test builds only: the run's first V tile is never loaded, so the wait
          // for it runs out and the bounded-wait path is taken.
          if (y > kLag)
#endif
          {
            mbar_arrive_expect_tx(&v_full[vs], L::kTile);
            tma_load_4d(ring_v + vs * L::kTile, &tm_v, &v_full[vs], 0, v.x, v.y, v.z);
          }
          ++nv;
          if (++vs == NB) {
            vs = 0;
            vph ^= 1;
          }
        }
      }
      // every copy issued lands before this thread leaves (bounded waits)
      for (uint32_t i = nk > NB ? nk - NB : 0; i < nk; ++i) mbar_drain(&k_full[i % NB], (i / NB) & 1);
      for (uint32_t i = nv > NB ? nv - NB : 0; i < nv; ++i) mbar_drain(&v_full[i % NB], (i / NB) & 1);
    } else if (warp == kWarpS && lane == 0) {
      // ---------------------------------------------------------- S^T = K Q^T
      constexpr uint32_t kIdS = idesc_e4m3(kKeys, 2 * C, false, false);
      const uint64_t dQ = sdesc_codes<D>(sQ), dT = sdesc_codes<D>(ring);
      uint32_t seg = 0, buf = 0, ph = 0;  // segment, buffer and slot, their phase
      bool ok = true;
      while (ok && wk.next()) {
        const uint32_t qb = seg & 1;
        if (!(ok = mbar_wait(&q_full[qb], (seg >> 1) & 1, ctl, kSiteQFull))) break;
        ++seg;
        const uint64_t dq = desc_add(dQ, qb * L::kQ);
        for (int j = wk.k0; j < wk.k1; ++j) {
          if (!(ok = mbar_wait_both(&s_free[buf], ph ^ 1, kSiteSFree, &k_full[buf], ph, kSiteKFull, ctl))) break;
          tc_fence_after();
          const uint64_t dk = desc_add(dT, buf * L::kTile);
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            mma_ss_f8(tmem + buf * 2 * C, desc_add(dk, kk * 32), desc_add(dq, kk * 32), kIdS, kk > 0 ? 1u : 0u);
          tc_commit(&s_full[buf]);
          if (++buf == NB) {
            buf = 0;
            ph ^= 1;
          }
        }
        tc_commit(&q_empty[qb]);
      }
      tc_commit(&drain[0]);
      mbar_drain(&drain[0], 0);
    } else if (warp == kWarpO && lane == 0) {
      // ---------------------------------------------------------- O^T = V^T P^T
      // (at d = 64 rows 64.. of the product are what follows the tile in shared memory: nothing reads them)
      constexpr uint32_t kIdO = idesc_e4m3(128, 2 * C, true, true);
      const uint64_t dT = sdesc_codes<D>(ring_v, L::kTile), dP = sdesc_codes<64>(sP);
      const uint32_t total = static_cast<uint32_t>(wk.end - wk.t);
      uint32_t buf = 0, ph = 0;  // buffer and slot, their phase
      for (uint32_t y = 0; y < total; ++y) {
        // (O^T's buffer is free as well: its weights were written when tile y - NB had been added up)
        if (!mbar_wait_both(&v_full[buf], ph, kSiteVFull, &p_ready[buf], ph, kSitePReady, ctl)) break;
        tc_fence_after();
        const uint64_t dv = desc_add(dT, buf * L::kTile), dp = desc_add(dP, buf * L::kPTile);
#pragma unroll
        for (int kk = 0; kk < kKeys / 32; ++kk)
          mma_ss_f8(tmem + (NB + buf) * 2 * C, desc_add(dv, kk * 32 * D), desc_add(dp, kk * 2048), kIdO, kk > 0 ? 1u : 0u);
        tc_commit(&pv_done[buf]);
        if (++buf == NB) {
          buf = 0;
          ph ^= 1;
        }
      }
      tc_commit(&drain[1]);
      mbar_drain(&drain[1], 0);
    } else if (warp == kWarpQ) {
      // ---------------------------------------------------------- q's parts, D / 16 lanes a row, and the tree's table
      constexpr int kLanes = D / 16;
      uint32_t n = 0, nmask = 0;
      while (wk.next()) {
        const uint32_t qb = n & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&q_empty[qb], ((n >> 1) & 1) ^ 1, ctl, kSiteQEmpty))) break;
        const float sign = p.scale_log2 < 0.0f ? -1.0f : 1.0f;
#pragma unroll 2
        for (int r0 = 0; r0 < C; r0 += 32 / kLanes) {
          const int r = r0 + lane / kLanes, x = lane % kLanes, row = first_row + r;
          uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
          if (row < unit_rows) {
            const uint4 *src = reinterpret_cast<const uint4 *>(p.q + wk.b * p.sq.b + (wk.hk * p.G + row / p.Nt) * p.sq.h +
                                                               (row % p.Nt) * p.sq.n + x * 16);
            const uint4 a = src[0], z = src[1];
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
            w[4] = z.x, w[5] = z.y, w[6] = z.z, w[7] = z.w;
          }
          float most = greatest(w);
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
          const float unit = least_scale(most), by = sign / unit;
          uint4 hi, lo;
          q_parts(w, by, &hi, &lo);
          uint8_t *to = sQ + qb * L::kQ + piece_at<D>(r, x);
          *reinterpret_cast<uint4 *>(to) = hi;
          *reinterpret_cast<uint4 *>(to + C * D) = lo;
          if (x == 0) row_f[n % L::kSegs * C + r] = unit * fabsf(p.scale_log2);
        }
        fence_proxy_async_smem();
        warp_arrive(&q_full[qb]);
        ++n;
        if (!wk.masked()) continue;
        if (!__all_sync(0xffffffffu, mbar_wait(mask_empty, (nmask & 1) ^ 1, ctl, kSiteMaskEmpty))) break;
        build_table(p, wk.b, wk.base(), bits, dead, reinterpret_cast<volatile int8_t *>(small + L::kOffJump));
        warp_arrive(mask_full);
        ++nmask;
      }
    }
  } else if (warp >= kWarpAdd + kAddWarps) {
    // (the other warps of the warpgroup have no column of V)
    regs_increase<kRegsAdd>();
  } else if (warp >= kWarpAdd) {
    // ------------------------------------------------------------ O^T added up, a column of V per thread
    regs_increase<kRegsAdd>();
    const int col = (warp & 3) * 32 + lane, mine = lane & (C - 1);
    float *fac = floats(L::kOffAdd) + (warp - kWarpAdd) * C;
    uint32_t x = 0, seg = 0, nmask = 0;
    bool ok = true;
    while (wk.next()) {
      if (threadIdx.x == kWarpAdd * 32 && group == 0 && p.cuts && wk.k0 == 0 && (!wk.tail || p.cuts_by_unit))
        p.cuts[p.cuts_by_unit ? wk.b * p.Hkv + wk.hk : c] =
            wk.tail ? make_int4(-1, 0, 0, 0)
                    : make_int4(wk.b, wk.hk, c, static_cast<int>(divide((wk.u0 + wk.tiles) * run->runs - 1, run->total)));
      float o[C], A = -INFINITY;  // O is relative to 2^A
#pragma unroll
      for (int r = 0; r < C; ++r) o[r] = 0.0f;
      for (int kt = wk.k0; ok && kt < wk.k1; ++kt, ++x) {
        const uint32_t buf = x % NB;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[buf], (x / NB) & 1, ctl, kSitePvDone)))) break;
        tc_fence_after();
        // the factor of the column that this lane looks after
        const float m = tile_m[x % L::kTiles * C + mine];
        const bool move = m > A + kMoveBy;
        const float alpha = move ? ex2(A - m) : 1.0f;  // (0 at first)
        if (move) A = m;
        fac[mine] = m == -INFINITY ? 0.0f : ex2(m - A);
        __syncwarp();
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int r = 0; r < C; ++r) o[r] *= __shfl_sync(0xffffffffu, alpha, r);
        }
        const uint32_t at = tmem + (NB + buf) * 2 * C + lane_base;
#pragma unroll
        for (int r = 0; r < C; r += kCols) {
          uint32_t hi[kCols], lo[kCols];
          tmem_parts<C>(at + r, hi, lo);
#pragma unroll
          for (int y = 0; y < kCols; y += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(fac + r + y);
            o[r + y] = fmaf(__uint_as_float(hi[y]) + __uint_as_float(lo[y]), f.x, o[r + y]);
            o[r + y + 1] = fmaf(__uint_as_float(hi[y + 1]) + __uint_as_float(lo[y + 1]), f.y, o[r + y + 1]);
            o[r + y + 2] = fmaf(__uint_as_float(hi[y + 2]) + __uint_as_float(lo[y + 2]), f.z, o[r + y + 2]);
            o[r + y + 3] = fmaf(__uint_as_float(hi[y + 3]) + __uint_as_float(lo[y + 3]), f.w, o[r + y + 3]);
          }
        }
        tc_fence_before();
        warp_arrive(&o_empty[buf]);
      }
      // ---- the segment's result
      if (ok && wk.masked()) ok = __all_sync(0xffffffffu, mbar_wait(mask_full, nmask & 1, ctl, kSiteMaskFull));
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(l_full, seg & 1, ctl, kSiteLseFull));
      const bool whole = wk.whole();
      const long long slot = (static_cast<long long>(blockIdx.x) * 2 + (wk.k0 == 0 ? 1 : 0)) * C;
      if (ok) {
        const int row = first_row + mine;
        float l = 0.0f, M = -INFINITY;
#pragma unroll
        for (int w = 0; w < L::kAtWork; ++w) M = fmaxf(M, sum_m[(w * L::kHalves + mine / kCols) * kCols + mine % kCols]);
#pragma unroll
        for (int w = 0; w < 4 * L::kAtWork; ++w) {
          const int wg = (w >> 2) * L::kHalves + mine / kCols, col = mine % kCols;
          const float m = sum_m[wg * kCols + col], v = sum_l[(wg * 4 + (w & 3)) * kCols + col];
          l += m == -INFINITY ? v : v * ex2(m - M);
        }
        const int row_node = row < unit_rows ? row % p.Nt : 0;
        const bool padding = wk.tail && ((dead[row_node >> 5] >> (row_node & 31)) & 1u);
        const bool any = l != 0.0f && !padding;
        fac[mine] = any ? quotient(A - M, l) : 0.0f;
        if (warp == kWarpAdd && lane < C && row < unit_rows) {
          const float lse2 = any ? (M == -INFINITY ? 0.0f : M) - kLift + log2f(l) : -INFINITY;
          const int h = wk.hk * p.G + row / p.Nt;
          if (whole)
            p.lse[(static_cast<long long>(wk.b) * p.H + h) * p.Nt + row_node] = any ? lse2 * kLn2 : -INFINITY;
          else
            p.part_lse[slot + mine] = padding ? INFINITY : lse2;
        }
        const uint32_t none = __ballot_sync(0xffffffffu, !any);  // rows without a result: 0
        if (whole) {
          const int rows = unit_rows - first_row;
          int node = first_row % p.Nt;
          __nv_bfloat16 *head = p.o + wk.b * p.so.b + (wk.hk * p.G + first_row / p.Nt) * p.so.h + col;
#pragma unroll
          for (int r = 0; r < C; ++r) {
            if (r < rows) head[node * p.so.n] = __float2bfloat16((none >> r) & 1u ? 0.0f : o[r] * fac[r]);
            if (++node == p.Nt) {
              node = 0;
              head += p.so.h;
            }
          }
        } else {
          float *part = p.part_o + slot * D + col;
#pragma unroll
          for (int r = 0; r < C; ++r)
            if (first_row + r < unit_rows) part[r * D] = (none >> r) & 1u ? 0.0f : o[r] * fac[r];
        }
      }
      __syncwarp();
      warp_arrive(l_empty);
      if (wk.masked()) {
        warp_arrive(mask_empty);
        ++nmask;
      }
      ++seg;
    }
  } else {
    // ------------------------------------------------------------ softmax, a key per thread, 16 columns
    regs_increase<kRegsSoftmax>();
    constexpr int W = L::kAtWork;
    const int wg = warp >> 2, key = threadIdx.x & 127, mine = lane & (kCols - 1);
    const int c0 = wg % L::kHalves * kCols;  // its first column
    float *base = floats(L::kOffBase) + warp * 2 * kCols;  // 8 - m, then l's factor
    uint32_t x = 0, seg = 0, nmask = 0;  // tiles before the segment, segments, masked ones
    uint32_t y0 = wg / L::kHalves;       // this warpgroup's next tile of the run
    bool ok = true;
    while (wk.next()) {
      const int n = wk.k1 - wk.k0;
      const int from = wk.base();
      float l[kCols], lm = -INFINITY;  // l of its columns, relative to lm, which a lane has of its own
#pragma unroll
      for (int r = 0; r < kCols; ++r) l[r] = 0.0f;
      bool have_mask = false;
      // this key's scale, and the value scale of 16-key slice lane % 8 (0: behind the end)
      const float *k_scale = p.k_scale + (static_cast<long long>(wk.b) * p.Hkv + wk.hk) * p.blocks;
      const float *v_scale = p.v_scale + (static_cast<long long>(wk.b) * p.Hkv + wk.hk) * p.blocks;
      float ks = 0.0f, v8 = 0.0f;
      auto fetch = [&](int kt) {
        const int j = kt * kKeys + key, j8 = kt * kKeys + (lane & 7) * 16;
        ks = j < wk.len ? k_scale[j >> p.block_log2] : 0.0f;
        v8 = j8 < wk.len ? v_scale[j8 >> p.block_log2] : 0.0f;
      };
      if (y0 < x + n) fetch(wk.k0 + static_cast<int>(y0 - x));
      // (written before the products of this segment were issued)
      const float *rf = row_f + seg % L::kSegs * C + c0;
      for (; y0 < x + n; y0 += W) {  // (a warp that gave up still meets the others)
        const int kt = wk.k0 + static_cast<int>(y0 - x);
        const uint32_t buf = y0 % NB;
        const bool masked = kt * kKeys + kKeys > from;
        if (ok && masked && !have_mask) {
          ok = __all_sync(0xffffffffu, mbar_wait(mask_full, nmask & 1, ctl, kSiteMaskFull));
          have_mask = true;
        }
        // (scales of rows that no node sees may be anything)
        if (masked && !slice_seen(dead, kt * kKeys + (lane & 7) * 16 - from)) v8 = 0.0f;
        // log2 of this value's scale over the tile's greatest (vanishing ones count as 2^-100 of it), and its inverse
        const float kn = ks, vmax = warp_max_f32(v8), own = __shfl_sync(0xffffffffu, v8, (key >> 4) & 7);
        const float lr = own > 0.0f ? fmaxf(lg2(own) - lg2(vmax), -100.0f) : 0.0f, inv = ex2(-lr);
        if (y0 + W < x + n) fetch(kt + W);
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&s_full[buf], (y0 / NB) & 1, ctl, kSiteSFull));
        if (!ok) {
          named_barrier(1 + wg, 128);
          continue;
        }
        tc_fence_after();
        float s[kCols];
        const uint32_t at = tmem + buf * 2 * C + c0 + lane_base;
        {
          uint32_t hi[kCols], lo[kCols];
          tmem_parts<C>(at, hi, lo);
#pragma unroll
          for (int y = 0; y < kCols; y += 2) {
            const float2 f = *reinterpret_cast<const float2 *>(rf + y);
            const float2 e = ffma2(fadd2(make_float2(__uint_as_float(hi[y]), __uint_as_float(hi[y + 1])),
                                         make_float2(__uint_as_float(lo[y]), __uint_as_float(lo[y + 1]))),
                                   fmul2(f, make_float2(kn, kn)), make_float2(lr, lr));
            s[y] = e.x;
            s[y + 1] = e.y;
          }
        }
        tc_fence_before();
        warp_arrive(&s_free[buf]);
        const int node = kt * kKeys + key - from;
        if (masked) {
          // the rows that see this key (rows that are padding may: their results are replaced).  A loop, because
          // code that runs once a unit comes cold from memory.
          uint32_t rows = node < 0 ? ~0u : 0u;
          if (node >= 0 && node < p.Nt) {
            int i = (first_row + c0) % p.Nt;
#pragma unroll 1
            for (int r = 0; r < kCols; ++r) {
              if ((i >> 5) >= (node >> 5) && ((bits[bit_row(i) + (node >> 5)] >> (node & 31)) & 1u)) rows |= 1u << r;
              if (++i == p.Nt) i = 0;
            }
          }
#pragma unroll
          for (int r = 0; r < kCols; ++r)
            if (!((rows >> r) & 1u)) s[r] = -INFINITY;
        }
        // the tile's maxima: over the warp's keys, then over the four warps, whose places are used in turn (one may be a
        // tile ahead)
        float *most = floats(L::kOffMost) + ((y0 / W & 1) * kSoftmaxWarps + wg * 4) * kCols;
#pragma unroll
        for (int r = 0; r < kCols; r += 4) {
          const float4 v = make_float4(warp_max_f32(s[r]), warp_max_f32(s[r + 1]), warp_max_f32(s[r + 2]),
                                       warp_max_f32(s[r + 3]));
          if (lane == 0) *reinterpret_cast<float4 *>(most + (warp & 3) * kCols + r) = v;
        }
        named_barrier(1 + wg, 128);
        const float m = fmaxf(fmaxf(most[mine], most[kCols + mine]), fmaxf(most[2 * kCols + mine], most[3 * kCols + mine]));
        const bool move = m > lm + kMoveBy;
        const float alpha = move ? ex2(lm - m) : 1.0f;
        if (move) lm = m;
        base[mine] = kLift - (m == -INFINITY ? 0.0f : m);
        base[kCols + mine] = m == -INFINITY ? 0.0f : ex2(m - lm);
        if ((warp & 3) == 0) tile_m[y0 % L::kTiles * C + c0 + mine] = m + lg2(vmax);
        __syncwarp();
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int r = 0; r < kCols; ++r) l[r] *= __shfl_sync(0xffffffffu, alpha, r);
        }
        // the weights' buffer is free once tile y0 - NB's sums are done (see kTiles)
        if (y0 >= NB && !(ok = __all_sync(0xffffffffu, mbar_wait(&o_empty[buf], ((y0 - NB) / NB) & 1, ctl, kSiteDqEmpty))))
          continue;
        uint8_t *ptile = sP + buf * L::kPTile;
        {
          uint32_t hi[kCols / 4], lo[kCols / 4];
#pragma unroll
          for (int y = 0; y < kCols; y += 4) {
            const float4 b = *reinterpret_cast<const float4 *>(base + y);
            const float4 g = *reinterpret_cast<const float4 *>(base + kCols + y);
            const float2 e0 = fadd2(make_float2(s[y], s[y + 1]), make_float2(b.x, b.y));
            const float2 e1 = fadd2(make_float2(s[y + 2], s[y + 3]), make_float2(b.z, b.w));
            const float w0 = ex2(e0.x), w1 = ex2(e0.y), w2 = ex2(e1.x), w3 = ex2(e1.y);
            const float2 ii = make_float2(inv, inv);
            const float2 n0 = ffma2(make_float2(w0, w1), fmul2(make_float2(g.x, g.y), ii), make_float2(l[y], l[y + 1]));
            const float2 n1 =
                ffma2(make_float2(w2, w3), fmul2(make_float2(g.z, g.w), ii), make_float2(l[y + 2], l[y + 3]));
            l[y] = n0.x;
            l[y + 1] = n0.y;
            l[y + 2] = n1.x;
            l[y + 3] = n1.y;
            parts_of(w0, w1, w2, w3, &hi[y / 4], &lo[y / 4]);
          }
          if constexpr (kCols == 16) {
            *reinterpret_cast<uint4 *>(ptile + piece_at<64>(key, c0 / 16)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(ptile + piece_at<64>(key, (c0 + C) / 16)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          } else {
            *reinterpret_cast<uint4 *>(ptile + piece_at<64>(key, 0)) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
          }
        }
        if (masked) {
          // V rows that no query row sees become zeros (0 * NaN is NaN).  (The buffer's number is worked out anew here: kept
          // from above it is one more register spilled in the loop, 215 us for 203.)
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&v_full[y0 % NB], (y0 / NB) & 1, ctl, kSiteVFull)))) continue;
          if (c0 == 0 && (node >= p.Nt || (node >= 0 && ((dead[node >> 5] >> (node & 31)) & 1u)))) {
            uint4 *v = reinterpret_cast<uint4 *>(ring_v + (y0 % NB) * L::kTile + key * D);
#pragma unroll
            for (int y = 0; y < D / 16; ++y) v[y] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(&p_ready[buf]);
      }
      x += n;
      if (ok && wk.masked() && !have_mask)
        ok = __all_sync(0xffffffffu, mbar_wait(mask_full, nmask & 1, ctl, kSiteMaskFull));
      // ---- l over the warp's keys
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(l_empty, (seg & 1) ^ 1, ctl, kSiteLseEmpty));
      if (ok) {
        const float sum = lane_sums(l);
        if (lane < kCols) {
          sum_l[warp * kCols + lane] = sum;
          if ((warp & 3) == 0) sum_m[wg * kCols + lane] = lm;
        }
      }
      warp_arrive(l_full);
      if (wk.masked()) {
        warp_arrive(mask_empty);
        ++nmask;
      }
      ++seg;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpS) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmem);
  }
}

template <int D, int C>
cudaError_t launch_tc(const CUtensorMap &tk, const CUtensorMap &tv, const Tree8Params &p, cudaStream_t stream) {
  using L = LayoutTc<D, C>;
  auto kern = fa_tree_fp8_tc_kernel<D, C>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kRequest);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(p.ranges) * p.groups, kThreads, L::kRequest, stream>>>(tk, tv, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree8_tc(const CUtensorMap &tk, const CUtensorMap &tv, const Tree8Params &p, cudaStream_t stream) {
  const bool d64 = p.d == 64;
  switch (p.rows) {
    case 8: return d64 ? launch_tc<64, 8>(tk, tv, p, stream) : launch_tc<128, 8>(tk, tv, p, stream);
    case 16: return d64 ? launch_tc<64, 16>(tk, tv, p, stream) : launch_tc<128, 16>(tk, tv, p, stream);
    default: return d64 ? launch_tc<64, 32>(tk, tv, p, stream) : launch_tc<128, 32>(tk, tv, p, stream);
  }
}

}  // namespace fa
