// fa_tree_fp8.cu -- attention of the newest rows of each sequence, or of a tree
// of drafted tokens, over a cache held in 8 bits.
//
// A key is its e4m3 codes times the scale of its block of rows; the scores are
// scale * ks * (q . codes), and a value's scale goes into its weight, so the
// products run on the codes.  Both are converted to f16 on their way to the
// matrix instructions (exact: e4m3 is a subset of f16) and multiplied there by q
// and by the weights in f16, summed in fp32.
//
// Rounding.  A row of q is scaled by a power of two so that its greatest value
// lies in [2^13, 2^14): f16 then holds every value of at least 2^-27 of that
// exactly.  Weights are 2^(t - m + 6) <= 2^14 in f16: off by at most 2^-11 of
// each, or 2^-31 of the row's greatest.  Scores, maxima, sums, O and the partial
// results are fp32.
//
// Layout.  The key rows of a 128-key tile come by TMA (128- or 64-byte swizzle)
// through a ring.  Each of eight warps takes 16-key slices of a tile and 16 query
// rows (m16n8k16: rows are query rows, columns keys).  The column order inside a
// product is free as long as both sides agree, so that a thread's share of a K
// row (and of four V rows) is 16-byte pieces that it reads from shared memory
// without conflicts:
//   column 2 t of 8 keys is row t, column 2 t + 1 is row (t ^ 1) + 4;
//   the k-th columns of q and K are the bytes of piece t, then piece t + 4;
//   column g of V's j-th product is byte j of piece c(g).
// The results of S = Q K^T are then the fragments that P V takes.  With few rows
// all warps share the 16 rows and take slices in turn, each with its own maximum,
// sum and O, joined in shared memory at the unit's end.

#include <cfloat>
#include <cstdint>
#include <cuda_fp16.h>

#include "fa_cache8.h"
#include "fa_runs.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 8;                      // of the products
constexpr int kWarpProducer = 8, kWarpMask = 9;
constexpr int kThreads = 384;
// Register split: 384 threads launched with 168 each; the products' warps take
// 208 (at 168 they spill at d = 128), the control warps keep 88.
constexpr uint32_t kRegsControl = 88, kRegsProducts = 208;
static_assert(128 * kRegsControl + 256 * kRegsProducts <= kThreads * 168, "register split");
constexpr int kModelCtas = 152;                // GB300's SMs: the grid the runs are cut for
constexpr float kMoveBy = 8.0f;                // a maximum moves only when exceeded by more (log2 units)
constexpr float kLift = 6.0f;                  // weights are 2^(t - m + kLift)
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kSlice = 16;                     // keys of a step of a warp

template <int D>
struct Layout8 {
  static constexpr uint32_t kTile = kKeys * D;                    // a K or V tile
  static constexpr int kStages = D == 128 ? 4 : 8;
  // first the small things, then (1 KB aligned) the ring, then the warps' results
  static constexpr uint32_t kOffBits = 0;                         // node bit rows, see bit_row()
  static constexpr uint32_t kOffDead = kOffBits + 32 * (1 + 2 + 3 + 4) * 4;
  static constexpr uint32_t kOffJump = kOffDead + 16;             // int8[128]: pointer doubling
  static constexpr uint32_t kOffRange = kOffJump + 128;           // RunStart
  static constexpr uint32_t kOffScan = kOffRange + 48;            // warps' sums
  static constexpr uint32_t kOffStats = kOffScan + 12 * 8;        // m and l of [warp][16 rows]
  static constexpr uint32_t kOffBar = kOffStats + 2 * kWarps * 16 * 4;
  static constexpr int kNumBars = 2 * kStages + 2;                // full, empty, mask_full, mask_empty
  static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;    // abort flag
  static constexpr uint32_t kSmall = (kOffMisc + 16 + 15) / 16 * 16;
  static constexpr uint32_t kRing = kStages * 2 * kTile;
  static constexpr uint32_t kRequest = kSmall + 1008 + kRing + kWarps * 16 * D * 4;
  static_assert(kOffBar % 8 == 0 && kOffRange % 8 == 0 && kOffScan % 8 == 0, "alignment");
  static_assert(kRequest <= 232448, "shared memory budget");
};

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Four e4m3 codes as two f16 pairs, exact.
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

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Whether node i sees the key that is `node` rows from the tree's start.
__device__ __forceinline__ bool sees(const uint32_t *bits, int i, bool live, int node, int Nt) {
  if (!live || node >= Nt) return false;
  if (node < 0) return true;
  if ((node >> 5) > (i >> 5)) return false;
  return (bits[bit_row(i) + (node >> 5)] >> (node & 31)) & 1u;
}

// Where a thread's pieces lie in a slice's rows (byte offsets).
template <int D>
struct Offsets {
  uint32_t k0, k1;   // K: row of column g, its pieces (one at d = 64)
  uint32_t va, vb;   // V: rows of columns 2 t and 2 t + 1
  int d0, d1;        // first columns of O that accumulator values 0 and 1 (of a row) belong to
  __device__ Offsets(int g, int t) {
    const int row = (g & 1) ? ((g >> 1) ^ 1) + 4 : g >> 1;
    const int ra = t, rb = (t ^ 1) + 4;
    if (D == 128) {
      const int c = (g >> 1) | ((g & 1) << 2);
      k0 = row * 128 + ((t ^ row) & 7) * 16;
      k1 = row * 128 + (((t + 4) ^ row) & 7) * 16;
      va = ra * 128 + ((c ^ ra) & 7) * 16;
      vb = rb * 128 + ((c ^ rb) & 7) * 16;
      d0 = 16 * t;
      d1 = 16 * (t + 4);
    } else {
      const int p = g >> 1, c = ((p & 1) << 1) | (p >> 1);
      k0 = row * 64 + ((t ^ (row >> 1)) & 3) * 16;
      k1 = k0;
      va = ra * 64 + ((c ^ (ra >> 1)) & 3) * 16 + (g & 1) * 8;
      vb = rb * 64 + ((c ^ (rb >> 1)) & 3) * 16 + (g & 1) * 8;
      d0 = 16 * (((t & 1) << 1) | (t >> 1));
      d1 = d0 + 8;
    }
  }
};

template <int N>
__device__ __forceinline__ void load_piece(uint32_t (&w)[N], const uint8_t *p) {
  if constexpr (N == 4) {
    const uint4 x = *reinterpret_cast<const uint4 *>(p);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    w[0] = x.x, w[1] = x.y;
  }
}

// A warp's 16 query rows over its share of a segment's keys.
template <int D>
struct Rows {
  uint32_t q[D / 16][4];
  float f0, f1;       // scale * log2 e of rows g and g + 8, and the power of two taken out of them
  float o[D / 8][4];
  float m0, m1, l0, l1;
  float vs;           // the value scale that O's weights are relative to

  __device__ void start() {
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[j][x] = 0.0f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.0f;
    vs = 0.0f;
  }

  // Row r of the unit's rows, one of this thread's two (a[x], a[x + 2] of each fragment).
  __device__ float load_q(const Tree8Params &p, int b, int hk, int r, int t, int x) {
    uint2 w[D / 16];
    float most = 0.0f;
    const bool on = r < p.G * p.Nt;
    const __nv_bfloat16 *row = p.q + b * p.sq.b + (hk * p.G + r / p.Nt) * p.sq.h + (r % p.Nt) * p.sq.n;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      w[s] = on ? *reinterpret_cast<const uint2 *>(row + 16 * (t + 4 * (s >> 2)) + 4 * (s & 3)) : make_uint2(0u, 0u);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t v = y ? w[s].y : w[s].x;
        const float a = fabsf(__uint_as_float(v << 16)), z = fabsf(__uint_as_float(v & 0xffff0000u));
        if (a <= FLT_MAX) most = fmaxf(most, a);
        if (z <= FLT_MAX) most = fmaxf(most, z);
      }
    }
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
    int e = static_cast<int>(__float_as_uint(most) >> 23) - 127 - 13;  // (0 and the subnormals: the least)
    e = e < -100 ? -100 : e;
    const float by = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      float v[4] = {__uint_as_float(w[s].x << 16), __uint_as_float(w[s].x & 0xffff0000u), __uint_as_float(w[s].y << 16),
                    __uint_as_float(w[s].y & 0xffff0000u)};
#pragma unroll
      for (int y = 0; y < 4; ++y) v[y] = fabsf(v[y]) <= FLT_MAX ? v[y] * by : NAN;
      q[s][x] = pack_f16x2(v[0], v[1]);
      q[s][x + 2] = pack_f16x2(v[2], v[3]);
    }
    return __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * p.scale_log2;
  }

  __device__ void rescale(float a0, float a1) {
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      o[j][0] *= a0;
      o[j][1] *= a0;
      o[j][2] *= a1;
      o[j][3] *= a1;
    }
  }

  // 16 keys at kt, vt.  MASK: node0 is the first one's place in the tree.
  template <bool MASK>
  __device__ void slice(const uint8_t *kt, const uint8_t *vt, const Offsets<D> &at, float ks, float vscale,
                        const uint32_t *bits, const uint32_t *dead, int i0, int i1, int node0, int Nt, int t) {
    float s[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.0f;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint32_t w[4];
        load_piece(w, kt + u * 8 * D + (h ? at.k1 : at.k0));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint2 c = codes_to_f16(w[x]);
          mma_f16(s[u], q[h * 4 + x], c.x, c.y);
        }
      }
    }
    const float fa = fminf(fmaxf(f0 * ks, -FLT_MAX), FLT_MAX), fb = fminf(fmaxf(f1 * ks, -FLT_MAX), FLT_MAX);
    uint32_t see = 0xffu;  // bit 4 u + x
    if (MASK) {
      see = 0;
      const bool v0 = i0 >= 0 && !((dead[i0 >> 5] >> (i0 & 31)) & 1u);
      const bool v1 = i1 >= 0 && !((dead[i1 >> 5] >> (i1 & 31)) & 1u);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int node = node0 + 8 * u + (e ? (t ^ 1) + 4 : t);
          see |= static_cast<uint32_t>(sees(bits, i0, v0, node, Nt)) << (4 * u + e);
          see |= static_cast<uint32_t>(sees(bits, i1, v1, node, Nt)) << (4 * u + 2 + e);
        }
    }
    float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        s[u][x] *= x < 2 ? fa : fb;
        if (MASK && !((see >> (4 * u + x)) & 1u)) s[u][x] = -INFINITY;
      }
      x0 = fmaxf(x0, fmaxf(s[u][0], s[u][1]));
      x1 = fmaxf(x1, fmaxf(s[u][2], s[u][3]));
    }
    if (__any_sync(0xffffffffu, x0 > m0 + kMoveBy || x1 > m1 + kMoveBy || vscale > vs)) {
#pragma unroll
      for (int x = 1; x < 4; x <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, x));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, x));
      }
      float a0 = 1.0f, a1 = 1.0f;
      if (x0 > m0 + kMoveBy) {
        a0 = ex2(m0 - x0);
        m0 = x0;
      }
      if (x1 > m1 + kMoveBy) {
        a1 = ex2(m1 - x1);
        m1 = x1;
      }
      l0 *= a0;
      l1 *= a1;
      if (vscale > vs) {
        const float r = vs / vscale;
        vs = vscale;
        a0 *= r;
        a1 *= r;
      }
      rescale(a0, a1);
    }
    const float b0 = kLift - (m0 == -INFINITY ? 0.0f : m0), b1 = kLift - (m1 == -INFINITY ? 0.0f : m1);
    const float r = vscale == vs ? 1.0f : vscale / vs;
    uint32_t pw[4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        w[x] = ex2(s[u][x] + (x < 2 ? b0 : b1));  // (hidden: 0)
      }
      l0 += w[0] + w[1];
      l1 += w[2] + w[3];
      pw[2 * u] = pack_f16x2(w[0] * r, w[1] * r);
      pw[2 * u + 1] = pack_f16x2(w[2] * r, w[3] * r);
    }
    const uint32_t a[4] = {pw[0], pw[1], pw[2], pw[3]};
    constexpr int kWords = D / 32;  // words of a thread's share of a V row
    uint32_t va[2][kWords], vb[2][kWords];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      load_piece(va[u], vt + u * 8 * D + at.va);
      load_piece(vb[u], vt + u * 8 * D + at.vb);
      if (MASK) {  // rows that no query row sees become zeros (0 * NaN is NaN)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int node = node0 + 8 * u + (e ? (t ^ 1) + 4 : t);
          if (node >= Nt || (node >= 0 && ((dead[node >> 5] >> (node & 31)) & 1u)))
#pragma unroll
            for (int y = 0; y < kWords; ++y) (e ? vb[u][y] : va[u][y]) = 0u;
        }
      }
    }
#pragma unroll
    for (int y = 0; y < kWords; ++y) {
      // bytes of rows 2 t and 2 t + 1 side by side: the f16 pairs of columns 4 y .. 4 y + 3
      const uint2 lo0 = codes_to_f16(__byte_perm(va[0][y], vb[0][y], 0x5140));
      const uint2 hi0 = codes_to_f16(__byte_perm(va[0][y], vb[0][y], 0x7362));
      const uint2 lo1 = codes_to_f16(__byte_perm(va[1][y], vb[1][y], 0x5140));
      const uint2 hi1 = codes_to_f16(__byte_perm(va[1][y], vb[1][y], 0x7362));
      mma_f16(o[4 * y], a, lo0.x, lo1.x);
      mma_f16(o[4 * y + 1], a, lo0.y, lo1.y);
      mma_f16(o[4 * y + 2], a, hi0.x, hi1.x);
      mma_f16(o[4 * y + 3], a, hi0.y, hi1.y);
    }
  }
};

// RT row tiles of 16 rows share a CTA; the 8 / RT warps of one take a tile's
// slices in turn.
template <int D, int RT>
__global__ void __launch_bounds__(kThreads, 1)
    fa_tree_fp8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const Tree8Params p) {
  using L = Layout8<D>;
  constexpr int S = L::kStages, KG = kWarps / RT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *small = smem_raw;
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + L::kSmall + 1023) &
                                              ~uintptr_t(1023));
  float *part = reinterpret_cast<float *>(ring + L::kRing);  // [warp][16][D]
  uint32_t *bits = reinterpret_cast<uint32_t *>(small + L::kOffBits);
  uint32_t *dead = reinterpret_cast<uint32_t *>(small + L::kOffDead);
  RunStart *run = reinterpret_cast<RunStart *>(small + L::kOffRange);
  float *st_m = reinterpret_cast<float *>(small + L::kOffStats), *st_l = st_m + kWarps * 16;
  uint64_t *full = reinterpret_cast<uint64_t *>(small + L::kOffBar);
  uint64_t *empty = full + S;
  uint64_t *mask_full = empty + S, *mask_empty = mask_full + 1;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(small + L::kOffMisc);
  const WaitCtl ctl{abort_flag, p.status};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = blockIdx.x % p.groups, c = blockIdx.x / p.groups;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    mbar_init(mask_full, 1);
    mbar_init(mask_empty, kWarps);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpProducer && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  const bool has_run = find_run<kThreads>(p, c, run, reinterpret_cast<long long *>(small + L::kOffScan));
  if (p.cuts && !p.cuts_by_unit && group == 0 && threadIdx.x == 0) p.cuts[c] = make_int4(-1, 0, 0, 0);
  if (!has_run) return;
  Walk<Tree8Params> wk(p, *run);

  if (warp >= kWarpProducer) regs_decrease<kRegsControl>();
  if (warp == kWarpProducer) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t e = 0;
      bool ok = true;
      while (ok && wk.next()) {
        for (int j = wk.k0; j < wk.k1; ++j, ++e) {
          const uint32_t sl = e % S;
          if (!(ok = mbar_wait(&empty[sl], ((e / S) & 1) ^ 1, ctl, kSiteKvEmpty))) break;
          uint8_t *at = ring + sl * 2 * L::kTile;
#ifdef FA_TEST_SKIP_FIRST_V_LOAD
          // Test builds only: the run's first V tile is never loaded, so the
          // wait for it runs out and the bounded-wait path is taken.
          mbar_arrive_expect_tx(&full[sl], 2 * L::kTile);
          tma_load_4d(at, &tm_k, &full[sl], 0, j * kKeys, wk.hk, wk.b);
          if (e > 0) tma_load_4d(at + L::kTile, &tm_v, &full[sl], 0, j * kKeys, wk.hk, wk.b);
#else
          mbar_arrive_expect_tx(&full[sl], 2 * L::kTile);
          tma_load_4d(at, &tm_k, &full[sl], 0, j * kKeys, wk.hk, wk.b);
          tma_load_4d(at + L::kTile, &tm_v, &full[sl], 0, j * kKeys, wk.hk, wk.b);
#endif
        }
      }
      // every copy issued lands before this thread leaves (bounded waits)
      for (uint32_t i = e > S ? e - S : 0; i < e; ++i) mbar_drain(&full[i % S], (i / S) & 1);
    }
    return;
  }
  if (warp == kWarpMask) {
    // ------------------------------------------------------------ the tree's table
    uint32_t n = 0;
    while (wk.next()) {
      if (!wk.masked()) continue;
      if (!__all_sync(0xffffffffu, mbar_wait(mask_empty, (n & 1) ^ 1, ctl, kSiteMaskEmpty))) break;
      build_table(p, wk.b, wk.base(), bits, dead, reinterpret_cast<volatile int8_t *>(small + L::kOffJump));
      warp_arrive(mask_full);
      ++n;
    }
    return;
  }

  if (warp > kWarpMask) return;

  // -------------------------------------------------------------- products
  regs_increase<kRegsProducts>();
  const int rt = warp % RT, kg = warp / RT, g = lane >> 2, t = lane & 3;
  const Offsets<D> at(g, t);
  const int first_row = group * (16 * RT), tile_row = first_row + rt * 16;
  const int unit_rows = p.G * p.Nt;
  const bool works = tile_row < unit_rows;
  const int r0 = tile_row + g, r1 = r0 + 8;
  const int i0 = r0 < unit_rows ? r0 % p.Nt : -1, i1 = r1 < unit_rows ? r1 % p.Nt : -1;
  Rows<D> rows;
  uint32_t e = 0, nmask = 0;
  bool ok = true;
  while (wk.next()) {
    if (threadIdx.x == 0 && group == 0 && p.cuts && wk.k0 == 0 && (!wk.tail || p.cuts_by_unit))
      p.cuts[p.cuts_by_unit ? wk.b * p.Hkv + wk.hk : c] =
          wk.tail ? make_int4(-1, 0, 0, 0)
                  : make_int4(wk.b, wk.hk, c, static_cast<int>(divide((wk.u0 + wk.tiles) * run->runs - 1, run->total)));
    rows.start();
    const long long scale_row = (static_cast<long long>(wk.b) * p.Hkv + wk.hk) * p.blocks;
    // lanes 0..7 hold the key scales of a tile's slices, lanes 8..15 the value scales
    auto scales = [&](int kt) -> float {
      if (lane >= 16) return 0.0f;
      int blk = (kt * kKeys + (lane & 7) * kSlice) >> p.block_log2;
      blk = blk < p.blocks ? blk : p.blocks - 1;
      return (lane < 8 ? p.k_scale : p.v_scale)[scale_row + blk];
    };
    float next_scales = 0.0f;
    if (works && ok) {
      next_scales = scales(wk.k0);
      rows.f0 = rows.load_q(p, wk.b, wk.hk, r0, t, 0);
      rows.f1 = rows.load_q(p, wk.b, wk.hk, r1, t, 1);
    }
    const int base = wk.base();
    bool have_mask = false;
    for (int kt = wk.k0; ok && kt < wk.k1; ++kt, ++e) {
      const float sc = next_scales;
      if (works && kt + 1 < wk.k1) next_scales = scales(kt + 1);
      if (kt * kKeys + kKeys > base && !have_mask) {
        ok = __all_sync(0xffffffffu, mbar_wait(mask_full, nmask & 1, ctl, kSiteMaskFull));
        have_mask = true;
        if (!ok) break;
      }
      const uint32_t sl = e % S;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&full[sl], (e / S) & 1, ctl, kSiteKvFull)))) break;
      if (works) {
        const uint8_t *kp = ring + sl * 2 * L::kTile, *vp = kp + L::kTile;
#pragma unroll 1
        for (int x = kg; x < kKeys / kSlice; x += KG) {
          const int j0 = kt * kKeys + x * kSlice;
          if (j0 >= wk.len) break;
          const float ks = __shfl_sync(0xffffffffu, sc, x), vsc = __shfl_sync(0xffffffffu, sc, 8 + x);
          if (j0 + kSlice > base)
            rows.template slice<true>(kp + x * kSlice * D, vp + x * kSlice * D, at, ks, vsc, bits, dead, i0, i1,
                                      j0 - base, p.Nt, t);
          else
            rows.template slice<false>(kp + x * kSlice * D, vp + x * kSlice * D, at, ks, vsc, bits, dead, i0, i1, 0,
                                       p.Nt, t);
        }
      }
      warp_arrive(&empty[sl]);
    }
    if (ok && wk.masked() && !have_mask)
      ok = __all_sync(0xffffffffu, mbar_wait(mask_full, nmask & 1, ctl, kSiteMaskFull));
    // ---- the segment's result: the warps' joined
    if (works) {
#pragma unroll
      for (int x = 1; x < 4; x <<= 1) {
        rows.l0 += __shfl_xor_sync(0xffffffffu, rows.l0, x);
        rows.l1 += __shfl_xor_sync(0xffffffffu, rows.l1, x);
      }
      float *to = part + (warp * 16 + g) * D;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        to[at.d0 + j] = rows.o[j][0] * rows.vs;
        to[at.d1 + j] = rows.o[j][1] * rows.vs;
        to[8 * D + at.d0 + j] = rows.o[j][2] * rows.vs;
        to[8 * D + at.d1 + j] = rows.o[j][3] * rows.vs;
      }
      if (t == 0) {
        st_m[warp * 16 + g] = rows.m0;
        st_m[warp * 16 + g + 8] = rows.m1;
        st_l[warp * 16 + g] = rows.l0;
        st_l[warp * 16 + g + 8] = rows.l1;
      }
    }
    if (!__all_sync(0xffffffffu, ok)) *abort_flag = 1;
    named_barrier(1, kWarps * 32);
    const bool fine = *abort_flag == 0;
    const bool whole = wk.whole();
    const long long slot = (static_cast<long long>(blockIdx.x) * 2 + (wk.k0 == 0 ? 1 : 0)) * (16 * RT);
    constexpr int kQuads = D / 4;  // threads of a row
    for (int x = threadIdx.x; fine && x < 16 * RT * kQuads; x += kWarps * 32) {
      const int lr = x / kQuads, col = x % kQuads * 4, r = first_row + lr;
      if (r >= unit_rows) break;
      const int wr = (lr >> 4) * 16 + (lr & 15);  // its place in warp lr / 16 of the first key group
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < KG; ++k) M = fmaxf(M, st_m[k * RT * 16 + wr]);
      float l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        const int y = k * RT * 16 + wr;
        const float m = st_m[y], f = m == -INFINITY ? (st_l[y] == 0.0f ? 0.0f : 1.0f) : (m == M ? 1.0f : ex2(m - M));
        l += st_l[y] * f;
        const float4 v = *reinterpret_cast<const float4 *>(part + y * D + col);
        if (f != 0.0f) {
          o[0] += v.x * f;
          o[1] += v.y * f;
          o[2] += v.z * f;
          o[3] += v.w * f;
        }
      }
      const int node = r % p.Nt, h = wk.hk * p.G + r / p.Nt;
      const bool padding = wk.tail && ((dead[node >> 5] >> (node & 31)) & 1u);
      const bool any = l != 0.0f && !padding;
      const float inv = any ? 1.0f / l : 0.0f;
#pragma unroll
      for (int y = 0; y < 4; ++y) o[y] = any ? o[y] * inv : 0.0f;
      const float lse2 = any ? (M == -INFINITY ? 0.0f : M) - kLift + log2f(l) : -INFINITY;
      if (whole) {
        *reinterpret_cast<uint2 *>(p.o + wk.b * p.so.b + h * p.so.h + node * p.so.n + col) =
            make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
        if (col == 0) p.lse[(static_cast<long long>(wk.b) * p.H + h) * p.Nt + node] = any ? lse2 * kLn2 : -INFINITY;
      } else {
        *reinterpret_cast<float4 *>(p.part_o + (slot + lr) * D + col) = make_float4(o[0], o[1], o[2], o[3]);
        if (col == 0) p.part_lse[slot + lr] = padding ? INFINITY : lse2;
      }
    }
    named_barrier(2, kWarps * 32);
    if (wk.masked()) {
      warp_arrive(mask_empty);
      ++nmask;
    }
    if (!fine) ok = false;
  }
}

// Merge the partial results of units cut by a run's end:
//   O = sum 2^(lse_s - M) O_s / sum 2^(lse_s - M).
// WARPS warps take one row of one cut unit, dealing the runs out among themselves
// (a run's row is one coalesced read) and adding up in a fixed order: eight where a
// unit is cut into many runs, one where it is cut into two or three (B16 H16 Nt32:
// 4864 rows, 15 us with eight).
constexpr int kMergeWarps = 8;

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
    l = l * fa + fb;
#pragma unroll
    for (int y = 0; y < kCols; ++y) o[y] = o[y] * fa + v[y] * fb;
    m = mn;
  }
  const int node = r % p.Nt, h = hk * p.G + r / p.Nt;
  __nv_bfloat16 *dst = p.o + b * p.so.b + h * p.so.h + node * p.so.n;
  float *lse = p.lse + (static_cast<long long>(b) * p.H + h) * p.Nt + node;
  if constexpr (WARPS == 1) {
    const bool any = m != -INFINITY && m != INFINITY;  // +inf: padding
#pragma unroll
    for (int y = 0; y < kCols; ++y) dst[y * 32 + lane] = __float2bfloat16(any ? o[y] / l : 0.0f);
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
  dst[threadIdx.x] = __float2bfloat16(any ? out / sum : 0.0f);
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

template <int D, int RT>
cudaError_t launch_rows(const CUtensorMap &tk, const CUtensorMap &tv, const Tree8Params &p, cudaStream_t stream) {
  using L = Layout8<D>;
  auto kern = fa_tree_fp8_kernel<D, RT>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kRequest);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(p.ranges) * p.groups, kThreads, L::kRequest, stream>>>(tk, tv, p);
  return cudaGetLastError();
}

}  // namespace

// Short caches are not cut inside a unit: see plan_tree.
constexpr int kWholeTiles = 8;

Tree8Plan plan_tree8(int B, int H, int Hkv, int Nt, int Nk, int d) {
  Tree8Plan pl{};
  const int rows = H / Hkv * Nt;  // (below 2^31: H < 2^24, Nt <= 128)
  pl.rows = rows <= 16 ? 16 : (rows <= 32 ? 32 : (d == 64 && rows <= 64 ? 64 : 128));
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
  cudaError_t e;
  if (p.d == 128) {
    e = p.rows <= 32 ? launch_tree8_tc(tk, tv, p, stream) : launch_tree8_rows(tk, tv, p, stream);
  } else {
    switch (p.rows) {
      case 16: e = launch_rows<64, 1>(tk, tv, p, stream); break;
      case 32: e = launch_rows<64, 2>(tk, tv, p, stream); break;
      case 64: e = launch_rows<64, 4>(tk, tv, p, stream); break;
      default: e = launch_rows<64, 8>(tk, tv, p, stream); break;
    }
  }
  if (e != cudaSuccess || !merge) return e;
  return p.d == 128 ? launch_merge8<128>(p, stream) : launch_merge8<64>(p, stream);
}

}  // namespace fa
