// fa_tree_fp8_rows.cu -- attention of the newest rows of each sequence, or of a
// tree of drafted tokens, over a cache held in 8 bits, more than 32 query rows of a
// cache head, on tcgen05's 8-bit form.
//
// The mathematics and the rounding are those of fa_tree_fp8_tc.cu (q and the
// weights as two e4m3 parts, weights relative to their own tile's greatest, a fresh O
// a tile, references of their own for O and l), the other way round: a lane per query row, S = Q K^T with a column per key,
// O = P V with P from TMEM.  A row's maximum and sum are then one thread's, where
// the transposed form takes them over lanes and warps (64 rows 3300 cycles a tile
// there); up to 128 rows cost the same.
//
// What bounds it.  The products at d = 128: 16 instructions of 128 x 128 x 32 a tile, 90
// cycles each, 1440 cycles of a tile of 128 keys and 128 rows, as many as its share of
// the HBM traffic takes (1400).  A softmax takes a warp some 700 instructions.
// B2 H32 Hkv8 Nt64 Nk65536 (256 rows, two CTAs a tile): 157 us, 2100 cycles a tile, the
// way from a tile's O to the next one's start.  d = 64: 127 us (129 with two warpgroups of
// softmax and one O), the way of a tile through its S: product, softmax, product.
//
// CTA (640 threads): two warpgroups of softmax (three at d = 64), a row per thread, which
// take the tiles in turn; two (one) that add up O in registers, 64 columns of a row per
// thread (at d = 128 one alone held the next product up: 182 us for B2 H32 Hkv8 Nt64
// Nk65536), the first of them brings q's parts; warp 16 TMA producer, warp 17 issues S and owns TMEM, warp 18
// issues O, warp 19 the tree's table.  TMEM: three S of 128 columns (S of tile x + 2 is
// formed while tile x's weights, over its S, still wait for their product) and O, or two O of 64.  The
// tiles of all units form one list that is cut into equal runs (fa_runs.cuh), and a
// CTA's products run on from unit to unit.

#include <cstdint>

#include "fa_cache8.h"
#include "fa_parts.cuh"
#include "fa_runs.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kRows = 128;
constexpr int kThreads = 640;
constexpr int kWarpProducer = 16, kWarpS = 17, kWarpO = 18, kWarpMask = 19;
constexpr float kMoveBy = 8.0f;   // a running maximum moves only when exceeded by more (log2 units)
constexpr float kLift = 8.0f;     // weights reach 2^kLift
constexpr float kLn2 = 0.69314718055994530942f;
// Register split: 640 threads launched with 96 each.
// (The compiler keeps to 96 in every role: 254 to 280 bytes of spills stored, 512 to 560 loaded.)
constexpr uint32_t kRegsSoftmax = 104, kRegsAdd = 104, kRegsControl = 64;
static_assert(kRegsSoftmax == kRegsAdd && 512 * kRegsSoftmax + 128 * kRegsControl <= kThreads * 96, "register split");
static_assert(kRegsSoftmax >= 96 && kRegsAdd >= 96 && kRegsControl <= 96, "setmaxnreg goes up or down only");

template <int D>
struct LayoutRows {
  // Four warpgroups: of softmax, and to add up O, 64 columns each.
  static constexpr int kAdd = D / 64, kSoft = 4 - kAdd, kWarpAdd = 4 * kSoft;
  static constexpr uint32_t kTile = kKeys * D;         // a K or V tile, or one part of q
  // V tiles are asked for kLag tiles after their K (S runs about so far ahead of O).
  static constexpr int kLag = 2;
  static constexpr int kBufs = 3;                      // of S, and slots of K and of V
  static constexpr uint32_t kTmem = 512, kO = kBufs * 128;
  static constexpr int kOs = (kTmem - kO) / D;         // O buffers: 1, or 2 at d = 64
  // A tile's maxima are kept for 8 tiles: tile x + 8's come after S of it, so after O of tile x + 5, which waits for tile
  // x + 5 - kOs' sums, tile x's among them.
  static constexpr int kTiles = 8;
  static constexpr uint32_t kQ = 2 * kTile;            // both parts; two segments' in turn
  // first the small things, then (1 KB aligned) the ring and q
  static constexpr uint32_t kOffBits = 0;
  static constexpr uint32_t kOffDead = kOffBits + 32 * (1 + 2 + 3 + 4) * 4;
  static constexpr uint32_t kOffJump = kOffDead + 16;
  static constexpr uint32_t kOffRange = kOffJump + 128;
  static constexpr uint32_t kOffScan = kOffRange + 48;             // 20 warps' sums
  static constexpr uint32_t kOffScale = kOffScan + 20 * 8;         // [softmax warps][3][8]: a tile's scales
  static constexpr uint32_t kOffTileM = kOffScale + kWarpAdd * 24 * 4;   // [tiles][128] m + log2 vs_max
  static constexpr uint32_t kOffL = kOffTileM + kTiles * kRows * 4;      // [kSoft][128] l, [kSoft][128] its base
  static constexpr uint32_t kOffRow = kOffL + 2 * kSoft * kRows * 4;       // [3 segments][128] rows' factors
  static constexpr uint32_t kOffBar = kOffRow + 3 * kRows * 4;
  // k_full[3], v_full[3], s_full[3], p_ready[3], pv_done[3], q_full[2], o_empty[2], mask_full, mask_empty, l_full,
  // l_empty, drain[2]
  static constexpr int kNumBars = 5 * kBufs + 2 + 8;
  static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;     // TMEM address, abort flag
  static constexpr uint32_t kSmall = (kOffMisc + 16 + 15) / 16 * 16;
  static constexpr uint32_t kRing = 2 * kBufs * kTile;
  static constexpr uint32_t kRequest = kSmall + 1008 + kRing + 2 * kQ;
  static_assert(kOffBar % 8 == 0 && kOffRange % 8 == 0 && kOffScan % 8 == 0 && kOffScale % 16 == 0, "alignment");
  static_assert(kRequest <= 232448, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    fa_tree_fp8_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                            const Tree8Params p) {
  using L = LayoutRows<D>;
  constexpr int NB = L::kBufs, NO = L::kOs, kLag = L::kLag, W = L::kSoft, kWarpAdd = L::kWarpAdd;
  constexpr int kCols = 64;  // of O, a thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t *small = smem_raw;
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + L::kSmall + 1023) &
                                              ~uintptr_t(1023));
  uint8_t *ring_v = ring + NB * L::kTile, *sQ = ring + L::kRing;
  uint32_t *bits = reinterpret_cast<uint32_t *>(small + L::kOffBits);
  uint32_t *dead = reinterpret_cast<uint32_t *>(small + L::kOffDead);
  RunStart *run = reinterpret_cast<RunStart *>(small + L::kOffRange);
  auto floats = [&](uint32_t off) { return reinterpret_cast<float *>(small + off); };
  float *tile_m = floats(L::kOffTileM), *row_f = floats(L::kOffRow);
  float *sum_l = floats(L::kOffL), *sum_m = sum_l + L::kSoft * kRows;
  uint64_t *k_full = reinterpret_cast<uint64_t *>(small + L::kOffBar), *v_full = k_full + NB;
  // Tile x of the run uses slot, buffer and barrier number x % 3 of each kind (a p_ready for each warpgroup would not do:
  // a warpgroup may be through with its next tile before the issuer has looked); s_full tells that K's slot is free as
  // well, pv_done that V's and S's are.  No wait can find its barrier two phases on: what would complete the next phase
  // waits for what the waiter does after this one.
  uint64_t *s_full = v_full + NB, *p_ready = s_full + NB, *pv_done = p_ready + NB, *q_full = pv_done + NB;
  uint64_t *o_empty = q_full + 2, *mask_full = o_empty + 2, *mask_empty = mask_full + 1;
  uint64_t *l_full = mask_empty + 1, *l_empty = l_full + 1, *drain = l_empty + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(small + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(small + L::kOffMisc + 4);
  const WaitCtl ctl{abort_flag, p.status};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = blockIdx.x % p.groups, c = blockIdx.x / p.groups;
  const int first_row = group * kRows, unit_rows = p.G * p.Nt;
  const int rows = min(kRows, unit_rows - first_row), warps = (rows + 31) / 32;  // of a warpgroup, with rows

  if (threadIdx.x == 0) {
    for (int i = 0; i < NB; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&pv_done[i], 1);
      mbar_init(&p_ready[i], warps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], warps);
      mbar_init(&o_empty[i], L::kAdd * warps);
      mbar_init(&drain[i], 1);
    }
    mbar_init(mask_full, 1);
    mbar_init(mask_empty, 4 * warps);
    mbar_init(l_full, W * warps);
    mbar_init(l_empty, L::kAdd * warps);
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
      // ---------------------------------------------------------- S = Q K^T
      constexpr uint32_t kIdS = idesc_e4m3(kRows, kKeys, false, false);
      constexpr int kSteps = D / 32;
      const uint64_t dQ = sdesc_codes<D>(sQ), dT = sdesc_codes<D>(ring);
      uint32_t seg = 0, buf = 0, ph = 0;  // segment, buffer and slot, their phase
      bool ok = true;
      while (ok && wk.next()) {
        const uint32_t qb = seg & 1;
        if (!(ok = mbar_wait(&q_full[qb], (seg >> 1) & 1, ctl, kSiteQFull))) break;
        ++seg;
        const uint64_t dq = desc_add(dQ, qb * L::kQ);
        for (int j = wk.k0; j < wk.k1; ++j) {
          if (!(ok = mbar_wait_both(&pv_done[buf], ph ^ 1, kSiteSFree, &k_full[buf], ph, kSiteKFull, ctl))) break;
          tc_fence_after();
          const uint64_t dk = desc_add(dT, buf * L::kTile);
#pragma unroll
          for (int kk = 0; kk < 2 * kSteps; ++kk)  // both parts of q, one after the other
            mma_ss_f8(tmem + buf * 128, desc_add(dq, kk / kSteps * L::kTile + kk % kSteps * 32),
                      desc_add(dk, kk % kSteps * 32), kIdS, kk > 0 ? 1u : 0u);
          tc_commit(&s_full[buf]);
          if (++buf == NB) {
            buf = 0;
            ph ^= 1;
          }
        }
      }
      tc_commit(&drain[0]);
      mbar_drain(&drain[0], 0);
    } else if (warp == kWarpO && lane == 0) {
      // ---------------------------------------------------------- O = P V
      constexpr uint32_t kIdO = idesc_e4m3(kRows, D, false, true);
      const uint64_t dT = sdesc_codes<D>(ring_v);
      const uint32_t total = static_cast<uint32_t>(wk.end - wk.t);
      uint32_t buf = 0, ph = 0;  // buffer and slot, their phase
      for (uint32_t y = 0; y < total; ++y) {
        if (!(mbar_wait_both(&v_full[buf], ph, kSiteVFull, &p_ready[buf], ph, kSitePReady, ctl) &&
              mbar_wait(&o_empty[y % NO], ((y / NO) & 1) ^ 1, ctl, kSiteDqEmpty)))
          break;
        tc_fence_after();
        const uint64_t dv = desc_add(dT, buf * L::kTile);
        const uint32_t tp = tmem + buf * 128, to = tmem + L::kO + y % NO * D;
#pragma unroll
        for (int kk = 0; kk < kKeys / 32; ++kk) {
          mma_ts_f8(to, tp + kk * 16, desc_add(dv, kk * 32 * D), kIdO, kk > 0 ? 1u : 0u);
          mma_ts_f8(to, tp + kk * 16 + 8, desc_add(dv, kk * 32 * D), kIdO, 1u);
        }
        tc_commit(&pv_done[buf]);
        if (++buf == NB) {
          buf = 0;
          ph ^= 1;
        }
      }
      tc_commit(&drain[1]);
      mbar_drain(&drain[1], 0);
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
  } else if (warp >= kWarpAdd && (warp & 3) >= warps) {
    // (no rows: q's rows here stay what they are, and only rows that nothing reads come of them)
    regs_increase<kRegsAdd>();
  } else if (warp >= kWarpAdd) {
    // ------------------------------------------------------------ O added up, 64 columns of a row per thread; q's parts
    regs_increase<kRegsAdd>();
    const int r = (warp & 3) * 32 + lane, row = first_row + r;
    const bool first = warp < kWarpAdd + 4;
    const int c0 = first ? 0 : kCols;
    const bool used = r < rows;
    const int node = used ? row % p.Nt : -1, gh = used ? row / p.Nt : 0;
    // q of segment `seg`, into the buffer of the segment before the last one (whose products are all done: this
    // thread has seen their sums)
    auto load_q = [&](const Walk<Tree8Params> &w, uint32_t seg) {
      // (read twice, the second time from a cache: held, a row would take 64 registers)
      const uint4 *src = reinterpret_cast<const uint4 *>(p.q + w.b * p.sq.b + (w.hk * p.G + gh) * p.sq.h +
                                                         (used ? node : 0) * p.sq.n);
      auto piece = [&](int x, uint32_t (&v)[8]) {
        const uint4 a = used ? src[2 * x] : make_uint4(0u, 0u, 0u, 0u), z = used ? src[2 * x + 1] : make_uint4(0u, 0u, 0u, 0u);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = z.x, v[5] = z.y, v[6] = z.z, v[7] = z.w;
      };
      float most = 0.0f;
#pragma unroll 4
      for (int x = 0; x < D / 16; ++x) {
        uint32_t v[8];
        piece(x, v);
        most = fmaxf(most, greatest(v));
      }
      const float unit = least_scale(most), by = (p.scale_log2 < 0.0f ? -1.0f : 1.0f) / unit;
      uint8_t *to = sQ + (seg & 1) * L::kQ;
#pragma unroll 2
      for (int x = 0; x < D / 16; ++x) {
        uint32_t v[8];
        piece(x, v);
        uint4 hi, lo;
        q_parts(v, by, &hi, &lo);
        *reinterpret_cast<uint4 *>(to + piece_at<D>(r, x)) = hi;
        *reinterpret_cast<uint4 *>(to + L::kTile + piece_at<D>(r, x)) = lo;
      }
      row_f[seg % 3 * kRows + r] = unit * fabsf(p.scale_log2);
      fence_proxy_async_smem();
      warp_arrive(&q_full[seg & 1]);
    };
    Walk<Tree8Params> wn(p, *run);  // a segment ahead
    bool more = first && wn.next();
    if (first) load_q(wn, 0);
    uint32_t x = 0, seg = 0, nmask = 0;
    uint32_t buf = 0, ph = 0;  // tile x's, and its phase
    bool ok = true;
    while (wk.next()) {
      if (threadIdx.x == kWarpAdd * 32 && group == 0 && p.cuts && wk.k0 == 0 && (!wk.tail || p.cuts_by_unit))
        p.cuts[p.cuts_by_unit ? wk.b * p.Hkv + wk.hk : c] =
            wk.tail ? make_int4(-1, 0, 0, 0)
                    : make_int4(wk.b, wk.hk, c, static_cast<int>(divide((wk.u0 + wk.tiles) * run->runs - 1, run->total)));
      if (more && (more = wn.next())) load_q(wn, seg + 1);
      float o[kCols];
#pragma unroll
      for (int y = 0; y < kCols; ++y) o[y] = 0.0f;
      float A = -INFINITY;  // O is relative to 2^A
      for (int kt = wk.k0; ok && kt < wk.k1; ++kt, ++x) {
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[buf], ph, ctl, kSitePvDone)))) break;
        if (++buf == NB) {
          buf = 0;
          ph ^= 1;
        }
        tc_fence_after();
        const float m = tile_m[x % L::kTiles * kRows + r];
        const bool move = m > A + kMoveBy;
        if (__any_sync(0xffffffffu, move)) {
          const float a = move ? ex2(A - m) : 1.0f;  // (0 at first)
          if (move) A = m;
#pragma unroll
          for (int y = 0; y < kCols; ++y) o[y] *= a;
        }
        const float f = m == -INFINITY ? 0.0f : ex2(m - A);
        const float2 ff = make_float2(f, f);
        const uint32_t tO = tmem + L::kO + x % NO * D + lane_base + c0;
        auto gather = [&](const uint32_t (&w)[16], int q) {
#pragma unroll
          for (int y = 0; y < 16; y += 2) {
            const float2 n = ffma2(make_float2(__uint_as_float(w[y]), __uint_as_float(w[y + 1])), ff,
                                   make_float2(o[q + y], o[q + y + 1]));
            o[q + y] = n.x;
            o[q + y + 1] = n.y;
          }
        };
#pragma unroll
        for (int q = 0; q < kCols; q += 32) {
          uint32_t wa[16], wb[16];
          tmem_ld16(tO + q, wa);
          tmem_ld16(tO + q + 16, wb);
          tmem_ld_wait16(wa);
          tmem_ld_wait16(wb);
          gather(wa, q);
          gather(wb, q + 16);
        }
        tc_fence_before();
        warp_arrive(&o_empty[x % NO]);
      }
      // ---- the segment's result
      if (ok && wk.masked()) ok = __all_sync(0xffffffffu, mbar_wait(mask_full, nmask & 1, ctl, kSiteMaskFull));
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(l_full, seg & 1, ctl, kSiteLseFull));
      if (ok && used) {
        float l = 0.0f, M = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, sum_m[w * kRows + r]);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float m = sum_m[w * kRows + r], v = sum_l[w * kRows + r];
          l += m == -INFINITY ? v : v * ex2(m - M);
        }
        const bool padding = wk.tail && ((dead[node >> 5] >> (node & 31)) & 1u);
        const bool any = l != 0.0f && !padding;
        const float inv = any ? quotient(A - M, l) : 0.0f;
        const float lse2 = any ? (M == -INFINITY ? 0.0f : M) - kLift + log2f(l) : -INFINITY;
        const int h = wk.hk * p.G + gh;
        if (wk.whole()) {
          if (first) p.lse[(static_cast<long long>(wk.b) * p.H + h) * p.Nt + node] = any ? lse2 * kLn2 : -INFINITY;
          uint4 *dst = reinterpret_cast<uint4 *>(p.o + wk.b * p.so.b + h * p.so.h + node * p.so.n + c0);
#pragma unroll
          for (int y = 0; y < kCols; y += 8)
            dst[y / 8] = any ? make_uint4(pack_bf16x2(o[y] * inv, o[y + 1] * inv), pack_bf16x2(o[y + 2] * inv, o[y + 3] * inv),
                                          pack_bf16x2(o[y + 4] * inv, o[y + 5] * inv),
                                          pack_bf16x2(o[y + 6] * inv, o[y + 7] * inv))
                             : make_uint4(0u, 0u, 0u, 0u);
        } else {
          const long long at = (static_cast<long long>(blockIdx.x) * 2 + (wk.k0 == 0 ? 1 : 0)) * kRows + r;
          if (first) p.part_lse[at] = padding ? INFINITY : lse2;
          float4 *dst = reinterpret_cast<float4 *>(p.part_o + at * D + c0);
#pragma unroll
          for (int y = 0; y < kCols; y += 4)
            dst[y / 4] = any ? make_float4(o[y] * inv, o[y + 1] * inv, o[y + 2] * inv, o[y + 3] * inv)
                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
      }
      warp_arrive(l_empty);
      if (wk.masked()) {
        warp_arrive(mask_empty);
        ++nmask;
      }
      ++seg;
    }
  } else if ((warp & 3) >= warps) {
    regs_increase<kRegsSoftmax>();
  } else {
    // ------------------------------------------------------------ softmax, a row per thread
    regs_increase<kRegsSoftmax>();
    const int wg = warp >> 2, r = (warp & 3) * 32 + lane;
    const int node = r < rows ? (first_row + r) % p.Nt : -1;
    float *sc = floats(L::kOffScale) + warp * 24;  // [3][8]: K's scales, log2 of V's over the greatest, its inverse
    uint32_t x = 0, seg = 0, nmask = 0;            // tiles before the segment, segments, masked ones
    uint32_t y0 = wg;                              // this warpgroup's next tile of the run
    uint32_t buf = wg, bph = 0;                    // its S and its phase
    bool ok = true;
    while (wk.next()) {
      const int n = wk.k1 - wk.k0, from = wk.base();
      float l = 0.0f, lm = -INFINITY;
      bool have_mask = false;
      // the scales of 16-key slice lane % 8, a tile of this warpgroup ahead (0: behind the end)
      const float *k_scale = p.k_scale + (static_cast<long long>(wk.b) * p.Hkv + wk.hk) * p.blocks;
      const float *v_scale = p.v_scale + (static_cast<long long>(wk.b) * p.Hkv + wk.hk) * p.blocks;
      float ks = 0.0f, vs = 0.0f;
      auto fetch = [&](int kt) {
        const int j = kt * kKeys + (lane & 7) * 16;
        ks = j < wk.len ? k_scale[j >> p.block_log2] : 0.0f;
        vs = j < wk.len ? v_scale[j >> p.block_log2] : 0.0f;
      };
      if (y0 < x + n) fetch(wk.k0 + static_cast<int>(y0 - x));
      for (; ok && y0 < x + n; y0 += W) {
        const int kt = wk.k0 + static_cast<int>(y0 - x);
        const bool masked = kt * kKeys + kKeys > from;
        if (masked && !have_mask) {
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(mask_full, nmask & 1, ctl, kSiteMaskFull)))) break;
          have_mask = true;
        }
        // (scales of rows that no node sees may be anything)
        if (masked && !slice_seen(dead, kt * kKeys + (lane & 7) * 16 - from)) ks = vs = 0.0f;
        const float vmax = warp_max_f32(vs);
        const float lr = vs > 0.0f ? fmaxf(lg2(vs) - lg2(vmax), -100.0f) : 0.0f;
        __syncwarp();
        if (lane < 8) {
          sc[lane] = ks;
          sc[8 + lane] = lr;
          sc[16 + lane] = ex2(-lr);
        }
        __syncwarp();
        if (y0 + W < x + n) fetch(kt + W);
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&s_full[buf], bph, ctl, kSiteSFull)))) break;
        tc_fence_after();
        const float f = row_f[seg % 3 * kRows + r];  // (written before the products of this segment were issued)
        const uint32_t tS = tmem + buf * 128 + lane_base;
        const int n0 = kt * kKeys - from;
        const bool live = masked && node >= 0 && !((dead[node >> 5] >> (node & 31)) & 1u);
        // the greatest e = score + log2 r of the tile
        float m = -INFINITY;
        auto greatest_of = [&](const uint32_t (&s)[32], int q) {
          const float2 kq = *reinterpret_cast<const float2 *>(sc + 2 * q), lq = *reinterpret_cast<const float2 *>(sc + 8 + 2 * q);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float t = fmax3(__uint_as_float(s[16 * h]), __uint_as_float(s[16 * h + 1]), __uint_as_float(s[16 * h + 2]));
#pragma unroll
            for (int y = 3; y < 15; y += 2)
              t = fmax3(t, __uint_as_float(s[16 * h + y]), __uint_as_float(s[16 * h + y + 1]));
            t = fmaxf(t, __uint_as_float(s[16 * h + 15]));
            // (a factor of 0 times -inf is NaN, which fmaxf passes over)
            m = fmaxf(m, fmaf(t, f * (h ? kq.y : kq.x), h ? lq.y : lq.x));
          }
        };
        uint32_t sa[32];
        if (masked) {  // (a loop: code that runs once a unit comes cold from memory)
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            tmem_ld32(tS + q * 32, sa);
            const uint32_t see = visible(bits, node, live, n0 + 32 * q);
            tmem_ld_wait(sa);
#pragma unroll
            for (int y = 0; y < 32; ++y)
              if (!((see >> y) & 1u)) sa[y] = 0xff800000u;  // -inf
            greatest_of(sa, q);
          }
        } else {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            tmem_ld32(tS + q * 32, sa);
            tmem_ld_wait(sa);
            greatest_of(sa, q);
          }
        }
        const float b = kLift - (m == -INFINITY ? 0.0f : m);
        float lt = 0.0f;  // sum of the weights over r
        // 32 keys' weights, over scores that have been read: their two parts, 8 columns each
        auto weights = [&](const uint32_t (&s)[32], int q, auto mask_tag) {
          const float2 kq = *reinterpret_cast<const float2 *>(sc + 2 * q), lq = *reinterpret_cast<const float2 *>(sc + 8 + 2 * q);
          const float2 iq = *reinterpret_cast<const float2 *>(sc + 16 + 2 * q);
          const uint32_t see = mask_tag ? visible(bits, node, live, n0 + 32 * q) : ~0u;
          uint32_t pk[16];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float g = f * (h ? kq.y : kq.x), e = (h ? lq.y : lq.x) + b;
            const float2 gg = make_float2(g, g), ee = make_float2(e, e);
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int y = 0; y < 16; y += 4) {
              const int z = 16 * h + y;
              const float2 e0 = ffma2(make_float2(__uint_as_float(s[z]), __uint_as_float(s[z + 1])), gg, ee);
              const float2 e1 = ffma2(make_float2(__uint_as_float(s[z + 2]), __uint_as_float(s[z + 3])), gg, ee);
              float2 w0 = make_float2(ex2(e0.x), ex2(e0.y)), w1 = make_float2(ex2(e1.x), ex2(e1.y));
              if (mask_tag) {
                w0.x = (see >> z) & 1u ? w0.x : 0.0f;
                w0.y = (see >> (z + 1)) & 1u ? w0.y : 0.0f;
                w1.x = (see >> (z + 2)) & 1u ? w1.x : 0.0f;
                w1.y = (see >> (z + 3)) & 1u ? w1.y : 0.0f;
              }
              sum = fadd2(sum, fadd2(w0, w1));
              parts_of(w0.x, w0.y, w1.x, w1.y, &pk[z / 4], &pk[8 + z / 4]);
            }
            lt = fmaf(sum.x + sum.y, h ? iq.y : iq.x, lt);
          }
          tmem_st16(tS + q * 16, pk);
        };
        if (masked) {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            tmem_ld32(tS + q * 32, sa);
            tmem_ld_wait(sa);
            weights(sa, q, MaskTag<true>{});
          }
        } else {  // (a loop as well: unrolled, its code does not stay in the instruction cache, 247 us for 189)
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            tmem_ld32(tS + q * 32, sa);
            tmem_ld_wait(sa);
            weights(sa, q, MaskTag<false>{});
          }
        }
        tmem_st_wait();
        if (m > lm + kMoveBy) {
          l *= ex2(lm - m);
          lm = m;
        }
        l += lt == 0.0f ? 0.0f : lt * (m == -INFINITY ? 1.0f : ex2(m - lm));
        tile_m[y0 % L::kTiles * kRows + r] = m + lg2(vmax);
        if (masked) {
          // V rows that no query row sees become zeros (0 * NaN is NaN)
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&v_full[buf], bph, ctl, kSiteVFull)))) break;
          for (int key = r; key < kKeys; key += warps * 32) {
            const int i = n0 + key;
            if (i < p.Nt && (i < 0 || !((dead[i >> 5] >> (i & 31)) & 1u))) continue;
            uint4 *v = reinterpret_cast<uint4 *>(ring_v + buf * L::kTile + key * D);
#pragma unroll
            for (int y = 0; y < D / 16; ++y) v[y] = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        warp_arrive(&p_ready[buf]);
        buf += W;
        if (buf >= NB) {
          buf -= NB;
          bph ^= 1;
        }
      }
      if (!ok && y0 < x + n) y0 += (x + n - y0 + W - 1) / W * W;
      x += n;
      if (ok && wk.masked() && !have_mask)
        ok = __all_sync(0xffffffffu, mbar_wait(mask_full, nmask & 1, ctl, kSiteMaskFull));
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(l_empty, (seg & 1) ^ 1, ctl, kSiteLseEmpty));
      if (ok) {
        sum_l[wg * kRows + r] = l;
        sum_m[wg * kRows + r] = lm;
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

template <int D>
cudaError_t launch_rows(const CUtensorMap &tk, const CUtensorMap &tv, const Tree8Params &p, cudaStream_t stream) {
  constexpr uint32_t kBytes = LayoutRows<D>::kRequest;
  auto kern = fa_tree_fp8_rows_kernel<D>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(p.ranges) * p.groups, kThreads, kBytes, stream>>>(tk, tv, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree8_rows(const CUtensorMap &tk, const CUtensorMap &tv, const Tree8Params &p, cudaStream_t stream) {
  return p.d == 128 ? launch_rows<128>(tk, tv, p, stream) : launch_rows<64>(tk, tv, p, stream);
}

}  // namespace fa
