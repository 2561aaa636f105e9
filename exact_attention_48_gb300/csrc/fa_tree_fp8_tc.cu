// fa_tree_fp8_tc.cu -- attention of the newest rows of each sequence, or of a tree
// of drafted tokens, over a cache held in 8 bits: d = 128, on tcgen05's 8-bit form.
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
//     P_j = 2^(e_j - m + 8),   O += vs_max 2^(m - M - 8) (P codes),
//     l  += 2^(m - M - 8) sum P_j / r_j,
// so a tile's weights always reach up to 2^8, whatever the running maximum M is:
// e4m3's second part ends at 2^-10, 2^-18 of the tile's greatest weighted value,
// and a long flat tail beside one sharp key keeps its weight.  That takes a fresh
// O^T a tile, which a warpgroup adds to fp32 registers.
//
// Rounding.  A row of q is divided by a power of two so that its greatest value lies
// in (224, 448]; bf16's 8 bits are 4 + 4, so its parts are exact but where the second
// falls below e4m3's least step: off by at most 2^-10, 2^-17.8 of the row's greatest
// value.  A weight is rounded to f16 and to its parts: off by at most 2^-8 of itself,
// or 2^-9 of 2^8 at its tile's greatest.  Scores, maxima, sums and O are fp32.
//
// What bounds it.  HBM, 2 d bytes a key, up to about 64 rows: a 128-key tile takes
// an SM 1400 cycles of its share of the traffic, its products some 560 (a tcgen05
// instruction takes 60 or more whatever its N) and its softmax about 10 issue slots
// a row and warp.  More rows come in groups of 64, a CTA each, whose tiles mostly
// come from L2.
//
// CTA (512 threads): warps 0..3 and 4..7 softmax, a key per thread, alternate tiles;
// warps 8..11 add up O^T, a column of V per thread; warp 12 TMA producer, warp 13
// MMA issuer and TMEM owner, warp 14 the tree's table, warp 15 q's parts.  TMEM: two
// S^T and two O^T of 2 C columns.  The tiles of all units form one list that is cut
// into equal runs (fa_runs.cuh), and a CTA's products run on from unit to unit.

#include <cfloat>
#include <cstdint>
#include <cuda_fp16.h>

#include "fa_cache8.h"
#include "fa_runs.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kD = 128;
constexpr int kThreads = 512;
constexpr int kWarpAdd = 8, kWarpProducer = 12, kWarpMma = 13, kWarpMask = 14, kWarpQ = 15;
constexpr float kMoveBy = 8.0f;   // a running maximum moves only when exceeded by more (log2 units)
constexpr float kLift = 8.0f;     // weights reach 2^kLift
constexpr float kLn2 = 0.69314718055994530942f;
// Register split: 512 threads launched with 128 each.
constexpr uint32_t kRegsSoftmax = 160, kRegsControl = 64;  // (the sums' warps keep their 128)
static_assert(256 * kRegsSoftmax + 128 * 128 + 128 * kRegsControl <= kThreads * 128, "register split");

template <int C>
struct LayoutTc {
  static constexpr uint32_t kTile = kKeys * kD;        // a K or V tile, 16 KB
  static constexpr int kSlots = 10;
  static constexpr uint32_t kTmem = 8 * C <= 512 ? 8 * C : 512;  // S^T, S^T, O^T, O^T
  static constexpr uint32_t kQ = 2 * C * kD;           // q's parts
  // first the small things, then (1 KB aligned) ring, P, q
  static constexpr uint32_t kOffBits = 0;
  static constexpr uint32_t kOffDead = kOffBits + 32 * (1 + 2 + 3 + 4) * 4;
  static constexpr uint32_t kOffJump = kOffDead + 16;
  static constexpr uint32_t kOffRange = kOffJump + 128;
  static constexpr uint32_t kOffScan = kOffRange + 48;                    // 16 warps' sums
  static constexpr uint32_t kOffMost = kOffScan + 16 * 8;                 // [8 warps][C] greatest e
  static constexpr uint32_t kOffBase = kOffMost + 8 * C * 4;              // [8 warps][2][C]: 8 - m, l's factor
  static constexpr uint32_t kOffMove = kOffBase + 8 * 2 * C * 4;          // [8 warps][C]: l's rescale
  static constexpr uint32_t kOffTileM = kOffMove + 8 * C * 4;             // [4 tiles][C] m, for the sums' warps
  static constexpr uint32_t kOffTileV = kOffTileM + 4 * C * 4;            // [4 tiles] vs_max
  static constexpr uint32_t kOffAdd = kOffTileV + 16;                     // [4 warps][2][C]: factors of O
  static constexpr uint32_t kOffL = kOffAdd + 4 * 2 * C * 4;              // [8 warps][C] l, and [2][C] its base
  static constexpr uint32_t kOffLm = kOffL + 8 * C * 4;
  static constexpr uint32_t kOffRow = kOffLm + 2 * C * 4;                 // [4 segments][C] rows' factors
  static constexpr uint32_t kOffBar = kOffRow + 4 * C * 4;
  // full[S], empty[S], s_full[2], p_ready[2], pv_done[2], o_empty[2], q_full, q_empty, mask_full, mask_empty, l_full,
  // l_empty, drain
  static constexpr int kNumBars = 2 * kSlots + 8 + 7;
  static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;            // TMEM address, abort flag
  static constexpr uint32_t kSmall = (kOffMisc + 16 + 15) / 16 * 16;
  static constexpr uint32_t kRing = kSlots * kTile, kP = 2 * kTile;
  static constexpr uint32_t kRequest = kSmall + 1008 + kRing + kP + kQ;
  static_assert(kOffBar % 8 == 0 && kOffRange % 8 == 0 && kOffScan % 8 == 0 && kOffMost % 16 == 0, "alignment");
  static_assert(kRequest <= 232448, "shared memory budget");
};

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint2 codes_to_f16(uint32_t w) {
  uint2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(w));
  return r;
}
// Four weights (two f16 pairs) as their two e4m3 parts.
__device__ __forceinline__ void parts_of(uint32_t a, uint32_t b, uint32_t *hi, uint32_t *lo) {
  asm("{\n\t.reg .b16 ha, hb, la, lb;\n\t.reg .b32 x, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 ha, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 hb, %3;\n\t"
      "mov.b32 %0, {ha, hb};\n\t"
      "cvt.rn.f16x2.e4m3x2 x, ha;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, hb;\n\t"
      "sub.rn.f16x2 x, %2, x;\n\t"
      "sub.rn.f16x2 y, %3, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 la, x;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 lb, y;\n\t"
      "mov.b32 %1, {la, lb};\n\t}"
      : "=&r"(*hi), "=&r"(*lo)
      : "r"(a), "r"(b));
}

// 32 lanes x N consecutive columns.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&r)[N]) {
  static_assert(N % 16 == 0, "columns");
#pragma unroll
  for (int c = 0; c < N; c += 16) {
    uint32_t w[16];
    tmem_ld16(addr + c, w);
#pragma unroll
    for (int x = 0; x < 16; ++x) r[c + x] = __uint_as_float(w[x]);
  }
}

// Sums over the warp's lanes of N values each (N = 16, 32): lane l gets the sum of
// value l % N, in a fixed order.
template <int N>
__device__ __forceinline__ float lane_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int n = N;
#pragma unroll
  for (int o = N / 2; o; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int x = 0; x < N / 2; ++x) {
      if (x >= o) break;
      const float keep = up ? v[x + o] : v[x], send = up ? v[x] : v[x + o];
      v[x] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
    n >>= 1;
  }
  if (N == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
  return v[0];
}

// Whether node i sees the key that is `node` rows from the tree's start.
__device__ __forceinline__ bool sees(const uint32_t *bits, int i, bool live, int node, int Nt) {
  if (!live || node >= Nt) return false;
  if (node < 0) return true;
  if ((node >> 5) > (i >> 5)) return false;
  return (bits[bit_row(i) + (node >> 5)] >> (node & 31)) & 1u;
}

template <int C>
__global__ void __launch_bounds__(kThreads, 1)
    fa_tree_fp8_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          const Tree8Params p) {
  using L = LayoutTc<C>;
  constexpr int S = L::kSlots;
  constexpr int kLanes = C < 32 ? C : 32, kPerLane = C / kLanes;  // columns that lanes look after
  extern __shared__ uint8_t smem_raw[];
  uint8_t *small = smem_raw;
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + L::kSmall + 1023) &
                                              ~uintptr_t(1023));
  uint8_t *sP = ring + L::kRing, *sQ = sP + L::kP;
  uint32_t *bits = reinterpret_cast<uint32_t *>(small + L::kOffBits);
  uint32_t *dead = reinterpret_cast<uint32_t *>(small + L::kOffDead);
  RunStart *run = reinterpret_cast<RunStart *>(small + L::kOffRange);
  auto floats = [&](uint32_t off) { return reinterpret_cast<float *>(small + off); };
  float *tile_m = floats(L::kOffTileM), *tile_v = floats(L::kOffTileV), *row_f = floats(L::kOffRow);
  float *sum_l = floats(L::kOffL), *sum_m = floats(L::kOffLm);
  uint64_t *full = reinterpret_cast<uint64_t *>(small + L::kOffBar);
  uint64_t *empty = full + S;
  // Tile x of the run uses s_full, p_ready, pv_done and o_empty number x & 1.
  uint64_t *s_full = empty + S, *p_ready = s_full + 2, *pv_done = p_ready + 2, *o_empty = pv_done + 2;
  uint64_t *q_full = o_empty + 2, *q_empty = q_full + 1, *mask_full = q_empty + 1, *mask_empty = mask_full + 1;
  uint64_t *l_full = mask_empty + 1, *l_empty = l_full + 1, *drain = l_empty + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(small + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(small + L::kOffMisc + 4);
  const WaitCtl ctl{abort_flag, p.status};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = blockIdx.x % p.groups, c = blockIdx.x / p.groups;
  const int first_row = group * C, unit_rows = p.G * p.Nt;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_empty[i], 4);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(mask_full, 1);
    mbar_init(mask_empty, 12);
    mbar_init(l_full, 8);
    mbar_init(l_empty, 4);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
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
  if (p.cuts && !p.cuts_by_unit && group == 0 && threadIdx.x == 0) p.cuts[c] = make_int4(-1, 0, 0, 0);
  if (!has_run) {
    if (warp == kWarpMma) tmem_dealloc(tmem, L::kTmem);
    return;
  }
  Walk<Tree8Params> wk(p, *run);
  const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;

  if (warp >= kWarpProducer) {
    regs_decrease<kRegsControl>();
    if (warp == kWarpProducer && lane == 0) {
      // ---------------------------------------------------------- producer
      uint32_t e = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap *map, int row) -> bool {
        const uint32_t sl = e % S;
        if (!mbar_wait(&empty[sl], ((e / S) & 1) ^ 1, ctl, kSiteKvEmpty)) return false;
#ifdef FA_TEST_SKIP_FIRST_V_LOAD
        // Test builds only: the run's first V tile is never loaded, so the wait
        // for it runs out and the bounded-wait path is taken.
        if (e == 1) {
          ++e;
          return true;
        }
#endif
        mbar_arrive_expect_tx(&full[sl], L::kTile);
        tma_load_4d(ring + sl * L::kTile, map, &full[sl], 0, row, wk.hk, wk.b);
        ++e;
        return true;
      };
      while (ok && wk.next())
        for (int j = wk.k0; ok && j < wk.k1; ++j) ok = load(&tm_k, j * kKeys) && load(&tm_v, j * kKeys);
      // every copy issued lands before this thread leaves (bounded waits)
      for (uint32_t i = e > S ? e - S : 0; i < e; ++i) mbar_drain(&full[i % S], (i / S) & 1);
    } else if (warp == kWarpMma && lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t kIdS = idesc_e4m3(kKeys, 2 * C, false, false);
      constexpr uint32_t kIdO = idesc_e4m3(kD, 2 * C, true, true);
      const uint64_t dQ = sdesc_sw128(smem_addr(sQ), 16, 1024), dT = sdesc_sw128(smem_addr(ring), 16, 1024);
      const uint64_t dP = sdesc_sw128(smem_addr(sP), 16, 1024);
      const uint32_t total = static_cast<uint32_t>(wk.end - wk.t);
      uint32_t left = 0, seg = 0;  // tiles of the segment that S is to be formed of, segments begun
      bool ok = true;
      for (uint32_t i = 0; ok && i < total + 2; ++i) {
        if (i >= 2) {
          // O^T = V^T P^T of tile i - 2
          const uint32_t y = i - 2, buf = y & 1, ph = (y >> 1) & 1, sl = (2 * y + 1) % S;
          if (!(ok = mbar_wait(&p_ready[buf], ph, ctl, kSitePReady) &&
                     mbar_wait(&full[sl], ((2 * y + 1) / S) & 1, ctl, kSiteVFull) &&
                     mbar_wait(&o_empty[buf], ph ^ 1, ctl, kSiteSFree)))
            break;
          tc_fence_after();
          const uint64_t dv = desc_add(dT, sl * L::kTile), dp = desc_add(dP, buf * L::kTile);
#pragma unroll
          for (int kk = 0; kk < kKeys / 32; ++kk)
            mma_ss_f8(tmem + (2 + buf) * 2 * C, desc_add(dv, kk * 4096), desc_add(dp, kk * 4096), kIdO, kk > 0 ? 1u : 0u);
          tc_commit(&pv_done[buf]);
          tc_commit(&empty[sl]);
        }
        if (i < total) {
          // S^T = K Q^T of tile i (its buffer was read before tile i - 2's weights were ready)
          if (left == 0) {
            wk.next();
            left = wk.k1 - wk.k0;
            if (!(ok = mbar_wait(q_full, seg & 1, ctl, kSiteQFull))) break;
            ++seg;
          }
          const uint32_t sl = (2 * i) % S;
          if (!(ok = mbar_wait(&full[sl], ((2 * i) / S) & 1, ctl, kSiteKFull))) break;
          tc_fence_after();
          const uint64_t dk = desc_add(dT, sl * L::kTile);
#pragma unroll
          for (int kk = 0; kk < kD / 32; ++kk)
            mma_ss_f8(tmem + (i & 1) * 2 * C, desc_add(dk, kk * 32), desc_add(dQ, kk * 32), kIdS, kk > 0 ? 1u : 0u);
          tc_commit(&s_full[i & 1]);
          tc_commit(&empty[sl]);
          if (--left == 0) tc_commit(q_empty);
        }
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
    } else if (warp == kWarpQ) {
      // ---------------------------------------------------------- q's parts, eight lanes a row
      uint32_t n = 0;
      while (wk.next()) {
        if (!__all_sync(0xffffffffu, mbar_wait(q_empty, (n & 1) ^ 1, ctl, kSiteQEmpty))) break;
        const float sign = p.scale_log2 < 0.0f ? -1.0f : 1.0f;
#pragma unroll 2
        for (int r0 = 0; r0 < C; r0 += 4) {
          const int r = r0 + (lane >> 3), x = lane & 7, row = first_row + r;
          uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
          if (row < unit_rows) {
            const uint4 *src = reinterpret_cast<const uint4 *>(p.q + wk.b * p.sq.b + (wk.hk * p.G + row / p.Nt) * p.sq.h +
                                                               (row % p.Nt) * p.sq.n + x * 16);
            const uint4 a = src[0], z = src[1];
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
            w[4] = z.x, w[5] = z.y, w[6] = z.z, w[7] = z.w;
          }
          float most = 0.0f;
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const float a = fabsf(__uint_as_float(w[y] << 16)), z = fabsf(__uint_as_float(w[y] & 0xffff0000u));
            if (a <= FLT_MAX) most = fmaxf(most, a);
            if (z <= FLT_MAX) most = fmaxf(most, z);
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
          const float unit = least_scale(most), by = sign / unit;
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float v[4] = {__uint_as_float(w[2 * y] << 16), __uint_as_float(w[2 * y] & 0xffff0000u),
                          __uint_as_float(w[2 * y + 1] << 16), __uint_as_float(w[2 * y + 1] & 0xffff0000u)};
#pragma unroll
            for (int z = 0; z < 4; ++z) v[z] = fabsf(v[z]) <= FLT_MAX ? v[z] * by : NAN;
            hi[y] = pack_e4m3x4(v[0], v[1], v[2], v[3]);
            const uint2 h = codes_to_f16(hi[y]);
            const float2 h0 = __half22float2(*reinterpret_cast<const __half2 *>(&h.x));
            const float2 h1 = __half22float2(*reinterpret_cast<const __half2 *>(&h.y));
            lo[y] = pack_e4m3x4(v[0] - h0.x, v[1] - h0.y, v[2] - h1.x, v[3] - h1.y);
          }
          const uint32_t at = r * kD + ((x ^ (r & 7)) * 16);
          *reinterpret_cast<uint4 *>(sQ + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4 *>(sQ + C * kD + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          if (x == 0) row_f[(n & 3) * C + r] = unit * fabsf(p.scale_log2);
        }
        fence_proxy_async_smem();
        warp_arrive(q_full);
        ++n;
      }
    }
  } else if (warp >= kWarpAdd) {
    // ------------------------------------------------------------ O^T added up, a column of V per thread
    const int col = (warp & 3) * 32 + lane;
    float *fac = floats(L::kOffAdd) + (warp - kWarpAdd) * 2 * C;
    uint32_t x = 0, seg = 0, nmask = 0;
    bool ok = true;
    while (wk.next()) {
      if (threadIdx.x == kWarpAdd * 32 && group == 0 && p.cuts && wk.k0 == 0 && (!wk.tail || p.cuts_by_unit))
        p.cuts[p.cuts_by_unit ? wk.b * p.Hkv + wk.hk : c] =
            wk.tail ? make_int4(-1, 0, 0, 0)
                    : make_int4(wk.b, wk.hk, c, static_cast<int>(divide((wk.u0 + wk.tiles) * run->runs - 1, run->total)));
      float o[C], M[kPerLane];
#pragma unroll
      for (int r = 0; r < C; ++r) o[r] = 0.0f;
#pragma unroll
      for (int y = 0; y < kPerLane; ++y) M[y] = -INFINITY;
      for (int kt = wk.k0; ok && kt < wk.k1; ++kt, ++x) {
        const uint32_t buf = x & 1;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[buf], (x >> 1) & 1, ctl, kSitePvDone)))) break;
        tc_fence_after();
        // the factors of the columns that this lane looks after
        const float vs = tile_v[x & 3];
        bool move = false;
#pragma unroll
        for (int y = 0; y < kPerLane; ++y) {
          const int r = (lane & (kLanes - 1)) + y * 32;
          const float m = tile_m[(x & 3) * C + r];
          float a = 1.0f;
          if (m > M[y] + kMoveBy) {
            a = ex2(M[y] - m);  // (0 at first)
            M[y] = m;
            move = true;
          }
          fac[r] = m == -INFINITY ? 0.0f : ex2(m - M[y]) * vs;
          fac[C + r] = a;
        }
        __syncwarp();
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int r = 0; r < C; ++r) o[r] *= fac[C + r];
        }
        const uint32_t at = tmem + (2 + buf) * 2 * C + lane_base;
#pragma unroll
        for (int r = 0; r < C; r += 16) {
          uint32_t hi[16], lo[16];
          tmem_ld16(at + r, hi);
          tmem_ld16(at + C + r, lo);
          tmem_ld_wait16(hi);
          tmem_ld_wait16(lo);
#pragma unroll
          for (int y = 0; y < 16; y += 4) {
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
#pragma unroll
        for (int y = 0; y < kPerLane; ++y) {
          const int r = (lane & (kLanes - 1)) + y * 32, row = first_row + r;
          float l = 0.0f;
#pragma unroll
          for (int w = 0; w < 8; ++w) {
            const float m = sum_m[(w >> 2) * C + r];
            l += m == -INFINITY ? sum_l[w * C + r] : sum_l[w * C + r] * ex2(m - M[y]);
          }
          const int node = row < unit_rows ? row % p.Nt : 0;
          const bool padding = wk.tail && ((dead[node >> 5] >> (node & 31)) & 1u);
          const bool any = l != 0.0f && !padding;
          fac[r] = any ? 1.0f / l : 0.0f;
          fac[C + r] = any ? 1.0f : 0.0f;
          if (warp == kWarpAdd && lane < kLanes && row < unit_rows) {
            const float lse2 = any ? (M[y] == -INFINITY ? 0.0f : M[y]) - kLift + log2f(l) : -INFINITY;
            const int h = wk.hk * p.G + row / p.Nt;
            if (whole)
              p.lse[(static_cast<long long>(wk.b) * p.H + h) * p.Nt + node] = any ? lse2 * kLn2 : -INFINITY;
            else
              p.part_lse[slot + r] = padding ? INFINITY : lse2;
          }
        }
        __syncwarp();
        if (whole) {
          const int rows = unit_rows - first_row;
          int node = first_row % p.Nt;
          __nv_bfloat16 *head = p.o + wk.b * p.so.b + (wk.hk * p.G + first_row / p.Nt) * p.so.h + col;
#pragma unroll
          for (int r = 0; r < C; ++r) {
            if (r < rows) head[node * p.so.n] = __float2bfloat16(fac[C + r] != 0.0f ? o[r] * fac[r] : 0.0f);
            if (++node == p.Nt) {
              node = 0;
              head += p.so.h;
            }
          }
        } else {
          float *part = p.part_o + slot * kD + col;
#pragma unroll
          for (int r = 0; r < C; ++r)
            if (first_row + r < unit_rows) part[r * kD] = fac[C + r] != 0.0f ? o[r] * fac[r] : 0.0f;
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
    // ------------------------------------------------------------ softmax, a key per thread
    regs_increase<kRegsSoftmax>();
    const int wg = warp >> 2, key = threadIdx.x & 127;
    float *most = floats(L::kOffMost) + wg * 4 * C;        // [4 warps][C]
    float *base = floats(L::kOffBase) + warp * 2 * C;      // 8 - m, then l's factor
    float *lmove = floats(L::kOffMove) + warp * C;
    uint32_t x = 0, seg = 0, nmask = 0;  // tiles before the segment, segments, masked ones
    bool ok = true;
    while (wk.next()) {
      const int n = wk.k1 - wk.k0;
      const long long scale_row = (static_cast<long long>(wk.b) * p.Hkv + wk.hk) * p.blocks;
      const int from = wk.base();
      float l[C], lm[kPerLane];  // l relative to lm, of the columns that lanes look after
#pragma unroll
      for (int r = 0; r < C; ++r) l[r] = 0.0f;
#pragma unroll
      for (int y = 0; y < kPerLane; ++y) lm[y] = -INFINITY;
      bool have_mask = false;
      // this key's scale, and the value scale of 16-key slice lane % 8 (0: behind the end)
      auto k_scale = [&](int kt) {
        const int j = kt * kKeys + key;
        return j < wk.len ? p.k_scale[scale_row + (j >> p.block_log2)] : 0.0f;
      };
      auto v_scale = [&](int kt) {
        const int j = kt * kKeys + (lane & 7) * 16;
        return j < wk.len ? p.v_scale[scale_row + (j >> p.block_log2)] : 0.0f;
      };
      const int kt0 = wk.k0 + ((x & 1) ^ wg);
      float ks = 0.0f, v8 = 0.0f;
      if (kt0 < wk.k1) {
        ks = k_scale(kt0);
        v8 = v_scale(kt0);
      }
      // (written before the products of this segment were issued; four in turn, for at most two tiles' scores are ahead)
      const float *rf = row_f + (seg & 3) * C;
      for (int kt = kt0; kt < wk.k1; kt += 2) {  // (a warp that gave up still meets the others)
        const uint32_t y0 = x + (kt - wk.k0), ph = (y0 >> 1) & 1;  // (y0 & 1 is wg)
        const float kn = ks, vmax = warp_max_f32(v8), own = __shfl_sync(0xffffffffu, v8, (key >> 4) & 7);
        if (kt + 2 < wk.k1) {
          ks = k_scale(kt + 2);
          v8 = v_scale(kt + 2);
        }
        const bool masked = kt * kKeys + kKeys > from;
        if (ok && masked && !have_mask) {
          ok = __all_sync(0xffffffffu, mbar_wait(mask_full, nmask & 1, ctl, kSiteMaskFull));
          have_mask = true;
        }
        // log2 of this value's scale over the tile's greatest; vanishing ones count as 2^-100 of it
        const float ratio = fmaxf(own / vmax, 7.8886090522101181e-31f);
        const float lr = own > 0.0f && vmax > 0.0f ? log2f(ratio) : 0.0f, inv = own > 0.0f && vmax > 0.0f ? 1.0f / ratio : 1.0f;
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&s_full[wg], ph, ctl, kSiteSFull));
        if (!ok) {
          named_barrier(1 + wg, 128);
          continue;
        }
        tc_fence_after();
        float s[C];
        const uint32_t at = tmem + wg * 2 * C + lane_base;
#pragma unroll
        for (int r = 0; r < C; r += 16) {
          uint32_t hi[16], lo[16];
          tmem_ld16(at + r, hi);
          tmem_ld16(at + C + r, lo);
          tmem_ld_wait16(hi);
          tmem_ld_wait16(lo);
#pragma unroll
          for (int y = 0; y < 16; y += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(rf + r + y);
            const float g[4] = {fminf(f.x * kn, FLT_MAX), fminf(f.y * kn, FLT_MAX), fminf(f.z * kn, FLT_MAX),
                                fminf(f.w * kn, FLT_MAX)};
#pragma unroll
            for (int z = 0; z < 4; ++z)
              s[r + y + z] = fmaf(__uint_as_float(hi[y + z]) + __uint_as_float(lo[y + z]), g[z], lr);
          }
        }
        const int node = kt * kKeys + key - from;
        if (masked) {
          int i = first_row % p.Nt, row = first_row;
#pragma unroll
          for (int r = 0; r < C; ++r) {
            const bool live = row < unit_rows && !((dead[i >> 5] >> (i & 31)) & 1u);
            if (!sees(bits, i, live, node, p.Nt)) s[r] = -INFINITY;
            ++row;
            if (++i == p.Nt) i = 0;
          }
        }
        // the tile's maxima: over the warp's keys, then over the four warps
#pragma unroll
        for (int r = 0; r < C; r += 4) {
          const float4 v = make_float4(warp_max_f32(s[r]), warp_max_f32(s[r + 1]), warp_max_f32(s[r + 2]),
                                       warp_max_f32(s[r + 3]));
          if (lane == 0) *reinterpret_cast<float4 *>(most + (warp & 3) * C + r) = v;
        }
        named_barrier(1 + wg, 128);
        bool move = false;
#pragma unroll
        for (int y = 0; y < kPerLane; ++y) {
          const int r = (lane & (kLanes - 1)) + y * 32;
          const float m = fmaxf(fmaxf(most[r], most[C + r]), fmaxf(most[2 * C + r], most[3 * C + r]));
          float a = 1.0f;
          if (m > lm[y] + kMoveBy) {
            a = ex2(lm[y] - m);
            lm[y] = m;
            move = true;
          }
          base[r] = kLift - (m == -INFINITY ? 0.0f : m);
          base[C + r] = m == -INFINITY ? 0.0f : ex2(m - lm[y]);
          lmove[r] = a;
          if ((warp & 3) == 0) tile_m[(y0 & 3) * C + r] = m;
        }
        if ((warp & 3) == 0 && lane == 0) tile_v[y0 & 3] = vmax;
        __syncwarp();
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int r = 0; r < C; ++r) l[r] *= lmove[r];
        }
        // the weights' buffer is free once tile y0 - 2's product is done
        if (y0 >= 2 && !(ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[wg], ph ^ 1, ctl, kSitePvDone)))) continue;
        uint8_t *prow = sP + wg * L::kTile + key * 128;
#pragma unroll
        for (int r = 0; r < C; r += 16) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int y = 0; y < 16; y += 4) {
            const float4 b = *reinterpret_cast<const float4 *>(base + r + y);
            const float4 g = *reinterpret_cast<const float4 *>(base + C + r + y);
            const float w0 = ex2(s[r + y] + b.x), w1 = ex2(s[r + y + 1] + b.y), w2 = ex2(s[r + y + 2] + b.z),
                        w3 = ex2(s[r + y + 3] + b.w);
            l[r + y] = fmaf(w0, g.x * inv, l[r + y]);
            l[r + y + 1] = fmaf(w1, g.y * inv, l[r + y + 1]);
            l[r + y + 2] = fmaf(w2, g.z * inv, l[r + y + 2]);
            l[r + y + 3] = fmaf(w3, g.w * inv, l[r + y + 3]);
            parts_of(pack_f16x2(w0, w1), pack_f16x2(w2, w3), &hi[y / 4], &lo[y / 4]);
          }
          *reinterpret_cast<uint4 *>(prow + (((r / 16) ^ (key & 7)) * 16)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4 *>(prow + (((r / 16 + C / 16) ^ (key & 7)) * 16)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        if (masked) {
          // V rows that no query row sees become zeros (0 * NaN is NaN)
          const uint32_t e_v = 2 * y0 + 1;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&full[e_v % S], (e_v / S) & 1, ctl, kSiteVFull)))) continue;
          if (node >= p.Nt || (node >= 0 && ((dead[node >> 5] >> (node & 31)) & 1u))) {
            uint4 *v = reinterpret_cast<uint4 *>(ring + (e_v % S) * L::kTile + key * 128);
#pragma unroll
            for (int y = 0; y < 8; ++y) v[y] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(&p_ready[wg]);
      }
      x += n;
      if (ok && wk.masked() && !have_mask)
        ok = __all_sync(0xffffffffu, mbar_wait(mask_full, nmask & 1, ctl, kSiteMaskFull));
      // ---- l over the warp's keys
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(l_empty, (seg & 1) ^ 1, ctl, kSiteLseEmpty));
      if (ok) {
#pragma unroll
        for (int y = 0; y < kPerLane; ++y) {
          float v[kLanes];
#pragma unroll
          for (int r = 0; r < kLanes; ++r) v[r] = l[y * 32 + r];
          const float sum = lane_sums<kLanes>(v);
          if (lane < kLanes) {
            sum_l[warp * C + y * 32 + lane] = sum;
            if ((warp & 3) == 0) sum_m[wg * C + y * 32 + lane] = lm[y];
          }
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
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmem);
  }
}

template <int C>
cudaError_t launch_tc(const CUtensorMap &tk, const CUtensorMap &tv, const Tree8Params &p, cudaStream_t stream) {
  using L = LayoutTc<C>;
  auto kern = fa_tree_fp8_tc_kernel<C>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kRequest);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(p.ranges) * p.groups, kThreads, L::kRequest, stream>>>(tk, tv, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree8_tc(const CUtensorMap &tk, const CUtensorMap &tv, const Tree8Params &p, cudaStream_t stream) {
  switch (p.rows) {
    case 16: return launch_tc<16>(tk, tv, p, stream);
    case 32: return launch_tc<32>(tk, tv, p, stream);
    default: return launch_tc<64>(tk, tv, p, stream);
  }
}

}  // namespace fa
