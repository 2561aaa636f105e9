// fa_key_weights.cu -- accumulated attention weight of each cached key:
//   w_j = w_in_j + sum over the query rows i (and the heads of the group)
//         that see key j of exp(scale q_i . k_j - lse_i).
//
// Two kernels.  With up to 64 query rows for a cache head (a decode step, a
// short window) the keys' bytes bound the pass: S^T = K Q^T on tcgen05,
// M = 128 keys, N = 16 to 64 columns, thread = key, so that the sum over the
// query rows stays in one thread and every key row is read once.  With more
// rows the exponentials and the products do: S = Q K^T, M = 128 query rows,
// N = 256 keys, described below at its kernel.  Neither uses atomics; the
// order of every sum is fixed.

#include <cstdint>

#include "fa_cache.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kKeys = 128;          // keys of an M tile; two per CTA
constexpr int kThreads = 384;
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpTable = 10;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTables = 4;          // stages of the column table (up to 64 rows)
constexpr long long kWindowBytes = 48ll << 20;  // query rows worked on at a time, under half of L2

template <int D, int NT>
struct KwLayout {
  static constexpr int kSlabs = D / 64;
  static constexpr uint32_t kKTile = kKeys * D * 2;
  static constexpr uint32_t kKBlock = 2 * kKTile;
  static constexpr uint32_t kQTile = NT * D * 2;
  // K blocks in flight: what shared memory leaves beside the query tiles
  static constexpr int kKBufs = D == 128 ? (NT == 64 ? 2 : 3) : (NT == 64 ? 4 : 6);
  static constexpr int kQBufs = 4;
  static constexpr uint32_t kOffQ = kKBufs * kKBlock;
  static constexpr uint32_t kOffTab = kOffQ + kQBufs * kQTile;  // per stage: float[NT], int[NT], int min
  static constexpr uint32_t kTabBytes = NT * 8 + 16;
  static constexpr uint32_t kOffBar = kOffTab + kTables * kTabBytes;
  // k_full, k_empty, q_full, q_empty, s_full[2][2], s_free[2][2], tab_full, tab_empty, drain
  static constexpr int kNumBars = 2 * kKBufs + 2 * kQBufs + 8 + 2 * kTables + 1;
  static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
  static constexpr uint32_t kBytes = kOffMisc + 16;
  static constexpr uint32_t kRequest = kBytes + 1024;
  static constexpr uint32_t kTmemCols = 4 * NT < 32 ? 32 : 4 * NT;
  static_assert(kRequest <= 232448, "shared memory budget");
  static_assert(kOffQ % 1024 == 0 && kQTile % 1024 == 0 && kOffBar % 8 == 0 && kTabBytes % 16 == 0, "alignment");
};

// One unit: its keys, and its column tiles x in [x0, x1): head group
// x / per_group, tile first + x % per_group of that group's rows.
struct Unit {
  int b, hk, key0, len, split;
  int first, per_group, x0, x1;
};

__device__ __forceinline__ Unit unit_at(const KeyWeightParams &p, uint32_t u) {
  Unit n;
  // windows of `window` cache heads; within one, block by block over its heads
  const uint32_t blocks = (p.Nk + 2 * kKeys - 1) / (2 * kKeys), heads = p.B * p.Hkv;
  const uint32_t v = u / p.splits, per = p.window * blocks;
  n.split = static_cast<int>(u - v * p.splits);
  const uint32_t w0 = v / per * p.window, in = min(static_cast<uint32_t>(p.window), heads - w0);
  const uint32_t at = v % per;
  const int bh = static_cast<int>(w0 + at % in);
  n.key0 = static_cast<int>(at / in) * 2 * kKeys;
  n.b = bh / p.Hkv;
  n.hk = bh - n.b * p.Hkv;
  n.len = cache_rows(p.cache_len, n.b, p.Nk);
  n.first = 0;
  if (n.key0 >= n.len) {  // behind the sequence: nothing to add
    n.per_group = n.x0 = n.x1 = 0;
    return n;
  }
  // causal: rows below key0 - (len - Nq) see none of the block's keys
  if (p.causal && p.tiles_per_head > 1) {
    const int row = n.key0 - (n.len - p.Nq);
    if (row > 0) n.first = row / kKeys;  // row < Nq, since key0 < len
  }
  n.per_group = p.tiles_per_head - n.first;
  const long long tiles = static_cast<long long>(p.head_groups) * n.per_group;
  n.x0 = static_cast<int>(tiles * n.split / p.splits);
  n.x1 = static_cast<int>(tiles * (n.split + 1) / p.splits);
  return n;
}

// Units in the order a CTA takes them (heaviest first within a window when
// causal): turn r takes unit r * grid + c, with c
// backwards in odd turns so that heavy and light units even out.
__device__ __forceinline__ uint32_t unit_index(uint32_t r) {
  return r * gridDim.x + ((r & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// Sum of exp2(s c + nl) over CH columns of a key's row of S^T; MASK: only the
// columns that see the key (key <= last).  nl in shared memory or registers.
template <bool MASK, int CH>
__device__ __forceinline__ float2 sum_columns(const uint32_t (&s)[CH], float2 cc, const float4 *nl, const int4 *last,
                                              int key) {
  float2 a0 = make_float2(0.f, 0.f), a1 = a0;
#pragma unroll
  for (int c = 0; c < CH; c += 4) {
    const float4 l4 = nl[c / 4];
    const float2 y0 =
        ffma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), cc, make_float2(l4.x, l4.y));
    const float2 y1 =
        ffma2(make_float2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), cc, make_float2(l4.z, l4.w));
    float p0 = ex2(y0.x), p1 = ex2(y0.y), p2 = ex2(y1.x), p3 = ex2(y1.y);
    if (MASK) {
      const int4 k4 = last[c / 4];
      p0 = key <= k4.x ? p0 : 0.0f;
      p1 = key <= k4.y ? p1 : 0.0f;
      p2 = key <= k4.z ? p2 : 0.0f;
      p3 = key <= k4.w ? p3 : 0.0f;
    }
    a0 = fadd2(a0, make_float2(p0, p1));
    a1 = fadd2(a1, make_float2(p2, p3));
  }
  return fadd2(a0, a1);
}

// A unit's sum for one key: into the weights, or into the split's partial sums.
__device__ __forceinline__ void store_weight(const KeyWeightParams &p, const Unit &n, int key, float total) {
  if (key >= p.Nk) return;
  const long long at = (static_cast<long long>(n.b) * p.Hkv + n.hk) * p.Nk + key;
  const float add = key < n.len ? total : 0.0f;
  if (p.splits > 1)
    p.part[n.split * (static_cast<long long>(p.B) * p.Hkv * p.Nk) + at] = add;
  else
    p.w[at] = p.w_in ? (key < n.len ? p.w_in[at] + add : p.w_in[at]) : add;
}

// Up to 64 query rows.  The units are 256-key blocks: unit u is block u / heads
// of cache head u % heads, and a CTA takes every grid-th (a persistent grid,
// one CTA per SM; stepping costs no division).
struct Block {
  const KeyWeightParams &p;
  int heads, blocks, d_bh, d_kb;
  int bh, kb;                      // cache head and block
  int b, hk, key0, len;
  __device__ explicit Block(const KeyWeightParams &pp) : p(pp) {
    heads = p.B * p.Hkv;
    blocks = (p.Nk + 2 * kKeys - 1) / (2 * kKeys);
    const int g = gridDim.x, c = blockIdx.x;
    d_bh = g % heads;
    d_kb = g / heads;
    bh = c % heads;
    kb = c / heads;
    load();
  }
  __device__ void load() {
    b = bh / p.Hkv;
    hk = bh - b * p.Hkv;
    key0 = kb * 2 * kKeys;
    len = cache_rows(p.cache_len, b, p.Nk);
  }
  __device__ bool done() const { return kb >= blocks; }
  __device__ bool empty() const { return key0 >= len; }  // behind the sequence: nothing to add
  __device__ void next() {
    bh += d_bh;
    kb += d_kb;
    if (bh >= heads) {
      bh -= heads;
      ++kb;
    }
    if (kb < blocks) load();
  }
};

// CTA (384 threads): warps 0..3 and 4..7 a key tile each, warp 8 TMA producer
// (K blocks through a ring of two to six, and the group's query rows), warp 9
// MMA issuer and TMEM owner, warp 10 the column table: the logsumexp of each
// column in log2 units, negated, and the last key it sees.  TMEM: two S^T
// buffers per warpgroup.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    fa_key_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const KeyWeightParams p) {
  using L = KwLayout<D, NT>;
  constexpr int KB = L::kKBufs, QB = L::kQBufs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
  uint64_t *k_empty = k_full + KB;
  uint64_t *q_full = k_empty + KB;
  uint64_t *q_empty = q_full + QB;
  uint64_t *s_full = q_empty + QB;      // [warpgroup][buffer]
  uint64_t *s_free = s_full + 4;
  uint64_t *tab_full = s_free + 4;
  uint64_t *tab_empty = tab_full + kTables;
  uint64_t *drain = tab_empty + kTables;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kOffMisc + 4);
  const WaitCtl ctl{abort_flag, p.status};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < KB; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < QB; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);
    }
    for (int i = 0; i < kTables; ++i) {
      mbar_init(&tab_full[i], 1);
      mbar_init(&tab_empty[i], 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == kWarpProducer) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      const uint32_t q_bytes = L::kSlabs * 128 * p.G * p.Nq;
      uint32_t nk = 0;
      for (Block n(p); !n.done(); n.next()) {
        if (n.empty()) continue;
        const uint32_t kb = nk % KB, qb = nk % QB;
        if (!mbar_wait(&k_empty[kb], ((nk / KB) & 1) ^ 1, ctl, kSiteKEmpty)) break;
#ifdef FA_TEST_SKIP_FIRST_V_LOAD
        if (nk == 0) {  // test builds only: the first block is never loaded
          ++nk;
          continue;
        }
#endif
        mbar_arrive_expect_tx(&k_full[kb], L::kKBlock);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int x = 0; x < L::kSlabs; ++x)
            tma_load_4d(smem + kb * L::kKBlock + t * L::kKTile + x * kKeys * 128, &tm_k, &k_full[kb], x * 64,
                        n.key0 + t * kKeys, n.hk, n.b);
        if (mbar_wait(&q_empty[qb], ((nk / QB) & 1) ^ 1, ctl, kSiteQEmpty)) {
          mbar_arrive_expect_tx(&q_full[qb], q_bytes);
#pragma unroll
          for (int s = 0; s < L::kSlabs; ++s)
            tma_load_4d(smem + L::kOffQ + qb * L::kQTile + s * NT * 128, &tm_q, &q_full[qb], s * 64, 0, n.hk * p.G,
                        n.b);
        } else {
          mbar_drain(&k_full[kb], (nk / KB) & 1);
          break;
        }
        ++nk;
      }
      // every copy issued lands before this thread leaves (bounded waits)
      for (uint32_t i = nk > KB ? nk - KB : 0; i < nk; ++i) mbar_drain(&k_full[i % KB], (i / KB) & 1);
      for (uint32_t i = nk > QB ? nk - QB : 0; i < nk; ++i) mbar_drain(&q_full[i % QB], (i / QB) & 1);
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t kId = idesc_bf16(kKeys, NT, false, false);
      const uint32_t aK = smem_addr(smem), aQ = smem_addr(smem + L::kOffQ);
      uint32_t nk = 0;
      bool ok = true;
      for (Block n(p); ok && !n.done(); n.next()) {
        if (n.empty()) continue;
        const uint32_t kb = nk % KB, qb = nk % QB, buf = nk & 1;
        if (!(ok = mbar_wait(&k_full[kb], (nk / KB) & 1, ctl, kSiteKFull))) break;
        if (!(ok = mbar_wait(&q_full[qb], (nk / QB) & 1, ctl, kSiteQFull))) break;
        const uint64_t dq = sdesc_sw128(aQ + qb * L::kQTile, 16, 1024);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!(ok = mbar_wait(&s_free[2 * t + buf], ((nk >> 1) & 1) ^ 1, ctl, kSiteSFree))) break;
          tc_fence_after();
          const uint64_t dk = sdesc_sw128(aK + kb * L::kKBlock + t * L::kKTile, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(tmem + (2 * t + buf) * NT, desc_add(dk, kmajor_step(kk, kKeys)), desc_add(dq, kmajor_step(kk, NT)),
                   kId, kk > 0 ? 1u : 0u);
          tc_commit(&s_full[2 * t + buf]);
        }
        if (!ok) break;
        tc_commit(&q_empty[qb]);
        tc_commit(&k_empty[kb]);
        ++nk;
      }
      tc_commit(drain);
      mbar_drain(drain, 0);
    }
  } else if (warp == kWarpTable) {
    // ------------------------------------------------------------ column tables
    constexpr int CPL = (NT + 31) / 32;  // columns per lane
    int row_g[CPL], row_i[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int col = c * 32 + lane;
      row_g[c] = col < p.G * p.Nq ? col / p.Nq : -1;
      row_i[c] = col % p.Nq;
    }
    uint32_t nk = 0;
    for (Block n(p); !n.done(); n.next()) {
      if (n.empty()) continue;
      const uint32_t st = nk % kTables;
      float lse[CPL];
#pragma unroll
      for (int c = 0; c < CPL; ++c)
        lse[c] = row_g[c] >= 0
                     ? p.lse[(static_cast<long long>(n.b) * p.H + n.hk * p.G + row_g[c]) * p.Nq + row_i[c]]
                     : -INFINITY;
      if (!__all_sync(0xffffffffu, mbar_wait(&tab_empty[st], ((nk / kTables) & 1) ^ 1, ctl, kSiteLseEmpty))) break;
      uint8_t *tab = smem + L::kOffTab + st * L::kTabBytes;
      int least = 0x7fffffff;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const int col = c * 32 + lane;
        const bool on = lse[c] != -INFINITY;
        const int last = on ? (p.causal ? n.len - p.Nq + row_i[c] : 0x7fffffff) : -1;
        if (col < NT) {
          reinterpret_cast<float *>(tab)[col] = on ? -(lse[c] * kLog2e) : 0.0f;
          reinterpret_cast<int *>(tab)[NT + col] = last;
          least = min(least, last);
        }
      }
      least = __reduce_min_sync(0xffffffffu, least);
      if (lane == 0) reinterpret_cast<int *>(tab)[2 * NT] = least;
      warp_arrive(&tab_full[st]);
      ++nk;
    }
  } else if (warp < kWarpProducer) {
    // ------------------------------------------------------------ weights
    const int t = warp >> 2, tid = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float2 cc = make_float2(p.scale_log2, p.scale_log2);
    uint32_t nk = 0;
    for (Block n(p); !n.done(); n.next()) {
      const int key = n.key0 + t * kKeys + tid;
      const long long at = static_cast<long long>(n.bh) * p.Nk + key;
      const float before = p.w_in && key < p.Nk ? p.w_in[at] : 0.0f;
      float total = 0.0f;
      if (!n.empty()) {
        const uint32_t buf = nk & 1, st = nk % kTables;
        const bool ok = mbar_wait(&tab_full[st], (nk / kTables) & 1, ctl, kSiteLseFull) &&
                        mbar_wait(&s_full[2 * t + buf], (nk >> 1) & 1, ctl, kSiteSFull);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const uint8_t *tab = smem + L::kOffTab + st * L::kTabBytes;
        const float4 *nl = reinterpret_cast<const float4 *>(tab);
        const int4 *last = reinterpret_cast<const int4 *>(tab + NT * 4);
        // hidden columns: padded or empty rows, or rows that do not see the tile's last key
        const bool mask = n.key0 + t * kKeys + kKeys - 1 > reinterpret_cast<const int *>(tab)[2 * NT];
        constexpr int CH = NT < 32 ? 16 : 32;  // columns at a time
        float2 sum = make_float2(0.f, 0.f);
        uint32_t s[NT / CH][CH];
        const uint32_t ts = tmem + (2 * t + buf) * NT + lane_base;
#pragma unroll
        for (int q = 0; q < NT / CH; ++q) {
          if constexpr (CH == 32)
            tmem_ld32(ts + q * CH, s[q]);
          else
            tmem_ld16(ts + q * CH, s[q]);
        }
#pragma unroll
        for (int q = 0; q < NT / CH; ++q) {
          if constexpr (CH == 32)
            tmem_ld_wait(s[q]);
          else
            tmem_ld_wait16(s[q]);
        }
        tc_fence_before();
        warp_arrive(&s_free[2 * t + buf]);
        if (mask) {
#pragma unroll
          for (int q = 0; q < NT / CH; ++q)
            sum = fadd2(sum, sum_columns<true, CH>(s[q], cc, nl + q * (CH / 4), last + q * (CH / 4), key));
        } else {
#pragma unroll
          for (int q = 0; q < NT / CH; ++q)
            sum = fadd2(sum, sum_columns<false, CH>(s[q], cc, nl + q * (CH / 4), last + q * (CH / 4), key));
        }
        warp_arrive(&tab_empty[st]);
        total = sum.x + sum.y;
        ++nk;
      }
      if (key < p.Nk) p.w[at] = key < n.len ? before + total : before;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// ------------------------------------------------------------------
// More than 64 query rows: S = Q K^T, M = 128 query rows, N = 256 keys.  S is
// read back as matrix fragments: a thread then holds four query rows of 16 of
// the keys, so that its rows' logsumexps are four registers (S^T would need a
// table of columns that every thread reads from shared memory, 1024 cycles a
// tile, as much as the products) and its running sums 16 (a thread that holds
// one row of 64 keys needs 64, which leaves no registers for a long load of S
// and made the kernel a sixth slower: 260 us where it takes 225).  The sums over
// query rows stay in the threads over all tiles; lanes and warps are added up
// once at the unit's end, through the unit's own K buffer, which the producer
// gets back after that.
//
// CTA (576 threads): four weight warpgroups, each 64 of the 256 keys (four warps
// per scheduler to hide the waits between tiles; eight warps of 128 keys and 208
// registers took 255 us), producer, MMA issuer.  TMEM: two S buffers of 256
// columns.
//
// What bounds it: a tile of 128 x 256 takes 1024 cycles of the tensor core and
// 1024 of the exponentials, and 1790 in all: the exponential unit is busy 56 % of
// the time, the tensor core 52 %, the issue slots 58 % (B1 H32 N4096 d128).  The rest is the
// weight warps' own chain between tiles (wait, load, a row's logsumexp and mask):
// knocking out the exponentials saves 15 %, the products 8 %, the fetch of the
// logsumexps with the mask 18 %.  No better: that work moved to an idle warp and
// a table in shared memory (more instructions than it saves), into the shadow of
// the load, or the warpgroups on alternate tiles instead of all on one.
// Measured, B4 H32 N4096 d128 causal: 206 us in a short run of calls, 1335
// TFLOP/s (0.69 of burst), 218 to 224 in a long one, with the SM clock that the
// power limit leaves; d64 198 us, with half the products and as many exponentials.

template <int D>
struct KwRowsLayout {
  static constexpr int kSlabs = D / 64;
  static constexpr uint32_t kKBlock = 2 * kKeys * D * 2;  // per 64-column slab 256 rows
  static constexpr int kKBufs = 2;
  static constexpr uint32_t kQTile = 128 * D * 2;
  static constexpr int kQBufs = D == 128 ? 3 : 6;
  static constexpr uint32_t kOffQ = kKBufs * kKBlock;
  static constexpr uint32_t kOffBar = kOffQ + kQBufs * kQTile;
  // k_full, k_empty, q_full, q_empty, s_full[2], s_free[2], drain
  static constexpr int kNumBars = 2 * kKBufs + 2 * kQBufs + 4 + 1;
  static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
  static constexpr uint32_t kBytes = kOffMisc + 16;
  static constexpr uint32_t kRequest = kBytes + 1024;
  static_assert(kRequest <= 232448, "shared memory budget");
  static_assert(kKBlock >= 2 * 4 * 128 * 4, "the sums fit the K buffer");
};

constexpr int kRowsThreads = 576;   // 16 weight warps, producer, MMA issuer
constexpr int kRowsProducer = 16, kRowsMma = 17;
constexpr int kWgKeys = 64;         // keys of a weight warpgroup
// x = *p if `on`.
__device__ __forceinline__ void load_if(float &x, const float *p, bool on) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q ld.global.f32 %0, [%1];\n\t}"
               : "+f"(x)
               : "l"(p), "r"(static_cast<uint32_t>(on)));
}

// 16 rows x 64 keys of S as a fragment (see tmem_ld_frag64): the thread holds
// rows lane / 4 and lane / 4 + 8, and of every 8 keys the two at j0 and j0 + 1.
// acc[c] += the sum over its two rows of exp2(s cc + nl) for its keys 8 c + j0
// and 8 c + j0 + 1; MASK: only keys j <= lim.
template <bool MASK>
__device__ __forceinline__ void add_rows(float2 (&acc)[kWgKeys / 8], const uint32_t (&s)[32], float2 cc, float nl0,
                                         float nl1, int lim0, int lim1, int j0) {
#pragma unroll
  for (int c = 0; c < kWgKeys / 8; ++c) {
    const float2 y0 = ffma2(make_float2(__uint_as_float(s[4 * c]), __uint_as_float(s[4 * c + 1])), cc,
                            make_float2(nl0, nl0));
    const float2 y1 = ffma2(make_float2(__uint_as_float(s[4 * c + 2]), __uint_as_float(s[4 * c + 3])), cc,
                            make_float2(nl1, nl1));
    float2 w0 = make_float2(ex2(y0.x), ex2(y0.y)), w1 = make_float2(ex2(y1.x), ex2(y1.y));
    if (MASK) {
      if (8 * c + j0 > lim0) w0.x = 0.0f;
      if (8 * c + j0 + 1 > lim0) w0.y = 0.0f;
      if (8 * c + j0 > lim1) w1.x = 0.0f;
      if (8 * c + j0 + 1 > lim1) w1.y = 0.0f;
    }
    acc[c] = fadd2(acc[c], fadd2(w0, w1));
  }
}

template <int D>
__global__ void __launch_bounds__(kRowsThreads, 1)
    fa_key_weights_rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                               const KeyWeightParams p) {
  using L = KwRowsLayout<D>;
  constexpr int KB = L::kKBufs, QB = L::kQBufs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
  uint64_t *k_empty = k_full + KB;
  uint64_t *q_full = k_empty + KB;
  uint64_t *q_empty = q_full + QB;
  uint64_t *s_full = q_empty + QB;  // [2 buffers]
  uint64_t *s_free = s_full + 2;
  uint64_t *drain = s_free + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kOffMisc + 4);
  const WaitCtl ctl{abort_flag, p.status};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < KB; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1 + 16);  // the unit's products, and its sums read
    }
    for (int i = 0; i < QB; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 16);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kRowsMma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= kRowsProducer) {
    if (warp == kRowsProducer && lane == 0) {
      // ---------------------------------------------------------- producer
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      const uint32_t q_bytes = L::kSlabs * 128 * (p.Nq > kKeys ? kKeys : p.gpt * p.Nq);
      uint32_t nk = 0, nq = 0;
      bool ok = true;
      for (uint32_t r = 0; ok; ++r) {
        const uint32_t u = unit_index(r);
        if (r * gridDim.x >= p.units) break;
        if (u >= p.units) continue;
        const Unit n = unit_at(p, u);
        if (n.x0 == n.x1) continue;
        const uint32_t kb = nk % KB;
        if (!(ok = mbar_wait(&k_empty[kb], ((nk / KB) & 1) ^ 1, ctl, kSiteKEmpty))) break;
        mbar_arrive_expect_tx(&k_full[kb], L::kKBlock);
#pragma unroll
        for (int s = 0; s < L::kSlabs; ++s)
          tma_load_4d(smem + kb * L::kKBlock + s * 2 * kKeys * 128, &tm_k, &k_full[kb], s * 64, n.key0, n.hk, n.b);
        ++nk;
        for (int x = n.x0; x < n.x1; ++x) {
          const int group = x / n.per_group, tile = n.first + x - group * n.per_group;
          const uint32_t qb = nq % QB;
          if (!(ok = mbar_wait(&q_empty[qb], ((nq / QB) & 1) ^ 1, ctl, kSiteQEmpty))) break;
#ifdef FA_TEST_SKIP_FIRST_V_LOAD
          // Test builds only: the first query tile is never loaded (see build.py).
          if (nq == 0) {
            ++nq;
            continue;
          }
#endif
          mbar_arrive_expect_tx(&q_full[qb], q_bytes);
#pragma unroll
          for (int s = 0; s < L::kSlabs; ++s)
            tma_load_4d(smem + L::kOffQ + qb * L::kQTile + s * 128 * 128, &tm_q, &q_full[qb], s * 64, tile * kKeys,
                        n.hk * p.G + group * p.gpt, n.b);
          ++nq;
        }
      }
      // every copy issued lands before this thread leaves (bounded waits)
      for (uint32_t i = nk > KB ? nk - KB : 0; i < nk; ++i) mbar_drain(&k_full[i % KB], (i / KB) & 1);
      for (uint32_t i = nq > QB ? nq - QB : 0; i < nq; ++i) mbar_drain(&q_full[i % QB], (i / QB) & 1);
    } else if (warp == kRowsMma && lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t kId = idesc_bf16(128, 2 * kKeys, false, false);
      const uint32_t aK = smem_addr(smem), aQ = smem_addr(smem + L::kOffQ);
      uint32_t nk = 0, nq = 0;
      bool ok = true;
      for (uint32_t r = 0; ok; ++r) {
        const uint32_t u = unit_index(r);
        if (r * gridDim.x >= p.units) break;
        if (u >= p.units) continue;
        const Unit n = unit_at(p, u);
        if (n.x0 == n.x1) continue;
        const uint32_t kb = nk % KB;
        if (!(ok = mbar_wait(&k_full[kb], (nk / KB) & 1, ctl, kSiteKFull))) break;
        const uint64_t dk = sdesc_sw128(aK + kb * L::kKBlock, 16, 1024);
        for (int x = n.x0; x < n.x1; ++x) {
          const uint32_t qb = nq % QB, buf = nq & 1;
          if (!(ok = mbar_wait(&q_full[qb], (nq / QB) & 1, ctl, kSiteQFull))) break;
          if (!(ok = mbar_wait(&s_free[buf], ((nq >> 1) & 1) ^ 1, ctl, kSiteSFree))) break;
          tc_fence_after();
          const uint64_t dq = sdesc_sw128(aQ + qb * L::kQTile, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(tmem + buf * 2 * kKeys, desc_add(dq, kmajor_step(kk, 128)), desc_add(dk, kmajor_step(kk, 2 * kKeys)),
                   kId, kk > 0 ? 1u : 0u);
          tc_commit(&s_full[buf]);
          tc_commit(&q_empty[qb]);
          ++nq;
        }
        if (ok) tc_commit(&k_empty[kb]);
        ++nk;
      }
      tc_commit(drain);
      mbar_drain(drain, 0);
    }
  } else {
    // ------------------------------------------------------------ weights
    const int t = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float2 cc = make_float2(p.scale_log2, p.scale_log2);
    // this thread's query row: packed tiles hold gpt heads of Nq rows
    const bool packed = p.Nq <= kKeys;
    const int row_g = packed ? row / p.Nq : 0, row_i = packed ? row % p.Nq : row;
    const bool row_in = !packed || row_g < p.gpt;
    uint32_t nk = 0, cnt = 0;
    bool ok = true;
    // (after a timeout the units are walked without work: every warp still
    // meets the others at the units' ends)
    for (uint32_t r = 0;; ++r) {
      const uint32_t u = unit_index(r);
      if (r * gridDim.x >= p.units) break;
      if (u >= p.units) continue;
      const Unit n = unit_at(p, u);
      const int key0 = n.key0 + t * kWgKeys;
      if (n.x0 == n.x1) {
        if (ok && row < kWgKeys) store_weight(p, n, key0 + row, 0.0f);
        continue;
      }
      // the tile to fetch next: this thread's row i of a head, its logsumexp at
      // `at` (if i < Nq and heads > 0, the group's heads from the row's own on)
      int tile = n.first + n.x0 % n.per_group, i = tile * kKeys + row_i;
      int heads = p.G - n.x0 / n.per_group * p.gpt - row_g;
      const float *at =
          p.lse + (static_cast<long long>(n.b) * p.H + n.hk * p.G + p.G - heads) * static_cast<long long>(p.Nq) + i;
      const int to_next = p.gpt * p.Nq - n.per_group * kKeys;  // of `at`, from behind a head's tiles to the next head's
      const int see = p.causal ? n.len - p.Nq - key0 : 1 << 30;  // row i sees this warpgroup's keys 0..see + i
      // A predicated load into the register that the next turn reads: a copy of
      // the value would wait for it here.  (-inf: no such row)
      auto fetch = [&](float &lse, int &lim) {
        lim = see + i;
        lse = -INFINITY;
        load_if(lse, at, row_in && heads > 0 && i < p.Nq);
        at += kKeys;
        i += kKeys;
        if (++tile == p.tiles_per_head) {
          tile = n.first;
          i = tile * kKeys + row_i;
          at += to_next;
          heads -= p.gpt;
        }
      };
      float2 acc[kWgKeys / 8];
#pragma unroll
      for (int c = 0; c < kWgKeys / 8; ++c) acc[c] = make_float2(0.f, 0.f);
      int lim;
      float lse;
      fetch(lse, lim);
      for (int x = n.x0; ok && x < n.x1; ++x, ++cnt) {
        const bool on = lse != -INFINITY;
        const float row_nl = on ? -(lse * kLog2e) : 0.0f;
        const int row_lim = on ? lim : -1;  // keys 0..row_lim are seen
        const uint32_t buf = cnt & 1;
        if (x + 1 < n.x1) fetch(lse, lim);
        const bool any = __any_sync(0xffffffffu, row_lim >= 0), all = __all_sync(0xffffffffu, row_lim >= kWgKeys - 1);
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&s_full[buf], (cnt >> 1) & 1, ctl, kSiteSFull)))) break;
        tc_fence_after();
        const uint32_t ts = tmem + buf * 2 * kKeys + t * kWgKeys + lane_base;
        if (any) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t s[32];
            tmem_ld_frag64(ts + half * (16u << 16), s);
            const int from = (lane >> 2) + 16 * half;
            const float nl0 = __shfl_sync(0xffffffffu, row_nl, from), nl1 = __shfl_sync(0xffffffffu, row_nl, from + 8);
            tmem_ld_wait(s);
            if (half == 1) {
              tc_fence_before();
              warp_arrive(&s_free[buf]);
            }
            if (all)
              add_rows<false>(acc, s, cc, nl0, nl1, 0, 0, 0);
            else
              add_rows<true>(acc, s, cc, nl0, nl1, __shfl_sync(0xffffffffu, row_lim, from),
                             __shfl_sync(0xffffffffu, row_lim, from + 8), (lane & 3) * 2);
          }
        } else {
          tc_fence_before();
          warp_arrive(&s_free[buf]);
        }
      }
      // ---- the unit's sums: over the lanes with the same keys (each step halves
      // the keys a lane keeps; lane l ends with keys 8 (l / 4) + 2 (l % 4) and the
      // next), then over the warps
#pragma unroll
      for (int o = 16, w = kWgKeys / 16; o > 2; o >>= 1, w >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int c = 0; c < w; ++c) {
          const float2 send = up ? acc[c] : acc[c + w], keep = up ? acc[c + w] : acc[c];
          acc[c] = make_float2(keep.x + __shfl_xor_sync(0xffffffffu, send.x, o),
                               keep.y + __shfl_xor_sync(0xffffffffu, send.y, o));
        }
      }
      float *red = reinterpret_cast<float *>(smem + (nk % KB) * L::kKBlock) + t * 4 * kWgKeys;
      if (ok) *reinterpret_cast<float2 *>(red + (warp & 3) * kWgKeys + lane * 2) = acc[0];
      named_barrier(1 + t, 128);
      if (ok) {
        if (row < kWgKeys) {
          const float sum =
              (red[row] + red[kWgKeys + row]) + (red[2 * kWgKeys + row] + red[3 * kWgKeys + row]);
          store_weight(p, n, key0 + row, sum);
        }
        fence_proxy_async_smem();
        warp_arrive(&k_empty[nk % KB]);
      }
      ++nk;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kRowsMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// w = w_in + the splits' sums, in order.
__global__ void __launch_bounds__(256) fa_key_weights_sum_kernel(const KeyWeightParams p) {
  const long long n = static_cast<long long>(p.B) * p.Hkv * p.Nk;
  const long long i = blockIdx.x * 256ll + threadIdx.x;
  if (i >= n) return;
  float s = 0.0f;
  for (int x = 0; x < p.splits; ++x) s += p.part[x * n + i];
  const int b = static_cast<int>(i / (static_cast<long long>(p.Hkv) * p.Nk)), j = static_cast<int>(i % p.Nk);
  const float before = p.w_in ? p.w_in[i] : 0.0f;
  p.w[i] = j < cache_rows(p.cache_len, b, p.Nk) ? before + s : before;
}

cudaError_t launch_sum(const KeyWeightParams &p, cudaStream_t stream) {
  const long long n = static_cast<long long>(p.B) * p.Hkv * p.Nk;
  fa_key_weights_sum_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D, int NT>
cudaError_t launch_kw(const CUtensorMap &tq, const CUtensorMap &tk, const KeyWeightParams &p, int sms,
                      cudaStream_t stream) {
  using L = KwLayout<D, NT>;
  auto kern = fa_key_weights_kernel<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kRequest);
  if (e != cudaSuccess) return e;
  const unsigned grid = p.units < static_cast<unsigned>(sms) ? p.units : static_cast<unsigned>(sms);
  kern<<<grid, kThreads, L::kRequest, stream>>>(tq, tk, p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_rows(const CUtensorMap &tq, const CUtensorMap &tk, const KeyWeightParams &p, int sms,
                        cudaStream_t stream) {
  using L = KwRowsLayout<D>;
  auto kern = fa_key_weights_rows_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kRequest);
  if (e != cudaSuccess) return e;
  const unsigned grid = p.units < static_cast<unsigned>(sms) ? p.units : static_cast<unsigned>(sms);
  kern<<<grid, kRowsThreads, L::kRequest, stream>>>(tq, tk, p);
  e = cudaGetLastError();
  return e == cudaSuccess && p.splits > 1 ? launch_sum(p, stream) : e;
}

template <int D>
cudaError_t launch_kw_d(int cols, const CUtensorMap &tq, const CUtensorMap &tk, const KeyWeightParams &p, int sms,
                        cudaStream_t stream) {
  switch (cols) {
    case 16: return launch_kw<D, 16>(tq, tk, p, sms, stream);
    case 32: return launch_kw<D, 32>(tq, tk, p, sms, stream);
    case 64: return launch_kw<D, 64>(tq, tk, p, sms, stream);
    default: return launch_rows<D>(tq, tk, p, sms, stream);
  }
}

}  // namespace

KeyWeightPlan plan_key_weights(int B, int H, int Hkv, int Nq, int Nk, int d) {
  KeyWeightPlan pl{};
  const int G = H / Hkv;
  if (Nq > 128) {
    pl.box_rows = 128;
    pl.gpt = 1;
    pl.tiles_per_head = (Nq + 127) / 128;
    pl.head_groups = G;
    pl.cols = 128;
  } else {
    pl.box_rows = Nq;
    pl.gpt = 128 / Nq < G ? 128 / Nq : G;
    pl.tiles_per_head = 1;
    pl.head_groups = (G + pl.gpt - 1) / pl.gpt;
    const int c = pl.gpt * Nq;
    pl.cols = c <= 16 ? 16 : (c <= 32 ? 32 : (c <= 64 ? 64 : 128));
  }
  // Few key blocks and many column tiles: the tiles are dealt out so that
  // about four units come to each of the 152 SMs.
  const long long units = static_cast<long long>(B) * Hkv * ((Nk + 255) / 256);
  const long long tiles = static_cast<long long>(pl.head_groups) * pl.tiles_per_head;
  long long s = (4 * 152 + units - 1) / units;
  if (s > tiles) s = tiles;
  pl.splits = units >= 2 * 152 || s < 1 ? 1 : static_cast<int>(s);
  // Every unit of a cache head reads the group's query rows: only as many
  // heads are worked on at a time as leave those rows in L2.  (B4 H32 N4096,
  // causal: 230 us over all 128 heads, whose rows take 134 MB, 225 in windows of
  // 48 heads, 222 head by head; but all 32 heads of a quarter of that, 33 MB, 57
  // us together and 66 head by head, since the heavy units then go first over
  // all of them.)
  const long long row_bytes = 2ll * G * Nq * d;
  const long long fit = kWindowBytes / row_bytes;
  const long long heads = static_cast<long long>(B) * Hkv;
  pl.window = static_cast<int>(fit < 1 ? 1 : (fit > heads ? heads : fit));
  return pl;
}

cudaError_t launch_key_weights(int d, int cols, const CUtensorMap &tq, const CUtensorMap &tk,
                               const KeyWeightParams &p, int sms, cudaStream_t stream) {
  return d == 64 ? launch_kw_d<64>(cols, tq, tk, p, sms, stream) : launch_kw_d<128>(cols, tq, tk, p, sms, stream);
}

}  // namespace fa
