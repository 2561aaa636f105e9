// fa_key_weights.cu -- accumulated attention weight of each cached key:
//   w_j = w_in_j + sum over the query rows i (and the heads of the group)
//         that see key j of exp(scale q_i . k_j - lse_i).
//
// The sum runs over the columns of S^T = K Q^T, so the product is formed that
// way round on tcgen05: M = 128 keys, N = query rows, and thread = key.  The
// row sum stays in one thread's registers: no shuffles, no atomics, a fixed
// order.  A CTA takes 256 keys (two M = 128 tiles, a softmax warpgroup each)
// and streams the group's query rows past them in tiles of up to 128 columns,
// so a query tile read from L2 serves 256 keys.
//
// What bounds it.  With many query rows the exponentials: 256 x 128 of them
// per column tile are 1024 cycles of the SM's 32 a cycle, against 512 on the
// tensor core.  With few (a decode step) the keys' bytes: the K blocks run
// through a ring of 64 KB buffers, several in flight.
//
// CTA (384 threads): warps 0..3 and 4..7 the two key tiles, warp 8 TMA
// producer, warp 9 MMA issuer and TMEM owner, warps 10 and 11 the column
// table (the logsumexp of each column in log2 units, negated, and the last
// key it sees) in turn.  TMEM: two S^T buffers per warpgroup.  Persistent:
// CTAs walk the units (256-key blocks), heaviest first when causal.

#include <cstdint>

#include "fa_cache.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kKeys = 128;          // keys of an M tile; two per CTA
constexpr int kThreads = 384;
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpTable = 10;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTables = 4;          // stages of the column table

template <int D, int NT>
struct KwLayout {
  static constexpr int kSlabs = D / 64;
  static constexpr uint32_t kKTile = kKeys * D * 2;
  static constexpr uint32_t kKBlock = 2 * kKTile;
  static constexpr uint32_t kQTile = NT * D * 2;
  // K blocks in flight: what shared memory leaves beside the query tiles
  static constexpr int kKBufs = D == 128 ? (NT >= 64 ? 2 : 3) : (NT >= 64 ? 4 : 6);
  static constexpr int kQBufs = NT == 128 ? 2 : 4;
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

__device__ __forceinline__ Unit unit_at(const KeyWeightParams &p, long long u) {
  Unit n;
  const int bh_all = p.B * p.Hkv;
  n.split = static_cast<int>(u % p.splits);
  const long long v = u / p.splits;
  const int bh = static_cast<int>(v % bh_all);
  n.key0 = static_cast<int>(v / bh_all) * 2 * kKeys;
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

// Units in the order a CTA takes them: turn r takes unit r * grid + c, with c
// backwards in odd turns so that heavy and light units even out.
__device__ __forceinline__ long long unit_index(int r) {
  const long long g = gridDim.x;
  return r * g + ((r & 1) ? g - 1 - blockIdx.x : blockIdx.x);
}

// One column tile on its way into a table stage (CPL columns a lane).
template <int CPL>
struct TableTile {
  float lse[CPL];
  int last[CPL];
  uint32_t at;
  bool on;
};

// Sum of exp2(s c + nl) over CH columns of a key's row of S^T; MASK: only the
// columns that see the key (key <= last).
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
      const uint32_t q_bytes = L::kSlabs * 128 * (p.tiles_per_head > 1 || p.Nq > kKeys ? kKeys : p.gpt * p.Nq);
      uint32_t nk = 0, nq = 0;
      bool ok = true;
      for (int r = 0; ok; ++r) {
        const long long u = unit_index(r);
        if (r * static_cast<long long>(gridDim.x) >= p.units) break;
        if (u >= p.units) continue;
        const Unit n = unit_at(p, u);
        if (n.x0 == n.x1) continue;
        const uint32_t kb = nk % KB;
        if (!(ok = mbar_wait(&k_empty[kb], ((nk / KB) & 1) ^ 1, ctl, kSiteKEmpty))) break;
        mbar_arrive_expect_tx(&k_full[kb], L::kKBlock);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int x = 0; x < L::kSlabs; ++x)
            tma_load_4d(smem + kb * L::kKBlock + t * L::kKTile + x * kKeys * 128, &tm_k, &k_full[kb], x * 64,
                        n.key0 + t * kKeys, n.hk, n.b);
        ++nk;
        for (int x = n.x0; x < n.x1; ++x) {
          const int group = x / n.per_group, tile = n.first + x - group * n.per_group;
          const uint32_t qb = nq % QB;
          if (!(ok = mbar_wait(&q_empty[qb], ((nq / QB) & 1) ^ 1, ctl, kSiteQEmpty))) break;
          mbar_arrive_expect_tx(&q_full[qb], q_bytes);
#pragma unroll
          for (int s = 0; s < L::kSlabs; ++s)
            tma_load_4d(smem + L::kOffQ + qb * L::kQTile + s * NT * 128, &tm_q, &q_full[qb], s * 64, tile * kKeys,
                        n.hk * p.G + group * p.gpt, n.b);
          ++nq;
        }
      }
      // every copy issued lands before this thread leaves (bounded waits)
      for (uint32_t i = nk > KB ? nk - KB : 0; i < nk; ++i) mbar_drain(&k_full[i % KB], (i / KB) & 1);
      for (uint32_t i = nq > QB ? nq - QB : 0; i < nq; ++i) mbar_drain(&q_full[i % QB], (i / QB) & 1);
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t kId = idesc_bf16(kKeys, NT, false, false);
      const uint32_t aK = smem_addr(smem), aQ = smem_addr(smem + L::kOffQ);
      uint32_t nk = 0, nq = 0;
      bool ok = true;
      for (int r = 0; ok; ++r) {
        const long long u = unit_index(r);
        if (r * static_cast<long long>(gridDim.x) >= p.units) break;
        if (u >= p.units) continue;
        const Unit n = unit_at(p, u);
        if (n.x0 == n.x1) continue;
        const uint32_t kb = nk % KB;
        if (!(ok = mbar_wait(&k_full[kb], (nk / KB) & 1, ctl, kSiteKFull))) break;
        tc_fence_after();
        for (int x = n.x0; ok && x < n.x1; ++x) {
          const uint32_t qb = nq % QB, buf = nq & 1;
          if (!(ok = mbar_wait(&q_full[qb], (nq / QB) & 1, ctl, kSiteQFull))) break;
          tc_fence_after();
          const uint64_t dq = sdesc_sw128(aQ + qb * L::kQTile, 16, 1024);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!(ok = mbar_wait(&s_free[2 * t + buf], ((nq >> 1) & 1) ^ 1, ctl, kSiteSFull))) break;
            tc_fence_after();
            const uint64_t dk = sdesc_sw128(aK + kb * L::kKBlock + t * L::kKTile, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss(tmem + (2 * t + buf) * NT, desc_add(dk, kmajor_step(kk, kKeys)),
                     desc_add(dq, kmajor_step(kk, NT)), kId, kk > 0 ? 1u : 0u);
            tc_commit(&s_full[2 * t + buf]);
          }
          if (!ok) break;
          tc_commit(&q_empty[qb]);
          ++nq;
        }
        if (ok) tc_commit(&k_empty[kb]);
        ++nk;
      }
      tc_commit(drain);
      mbar_drain(drain, 0);
    }
  } else if (warp >= kWarpTable) {
    // ------------------------------------------------------------ column tables
    // The two warps take the tiles in turn; the logsumexps of a warp's next
    // tile are in flight while it writes the current one.
    const int me = warp - kWarpTable;
    constexpr int CPL = (NT + 31) / 32;  // columns per lane
    uint32_t cnt = 0;
    using Tile = TableTile<CPL>;
    auto fetch = [&](const Unit &n, int x, uint32_t at) {
      Tile t;
      t.at = at;
      t.on = true;
      const int group = x / n.per_group, tile = n.first + x - group * n.per_group;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const int col = c * 32 + lane;
        int g, i;
        if (p.Nq > kKeys) {
          g = group;
          i = tile * kKeys + col;
        } else {
          g = group * p.gpt + col / p.Nq;
          i = col % p.Nq;
          if (col >= p.gpt * p.Nq) g = p.G;
        }
        const bool valid = col < NT && g < p.G && i < p.Nq;
        t.lse[c] = valid ? p.lse[(static_cast<long long>(n.b) * p.H + n.hk * p.G + g) * p.Nq + i] : -INFINITY;
        t.last[c] = p.causal ? n.len - p.Nq + i : 0x7fffffff;
      }
      return t;
    };
    bool ok = true;
    auto put = [&](const Tile &t) -> bool {
      const uint32_t st = t.at % kTables;
      if (!__all_sync(0xffffffffu, mbar_wait(&tab_empty[st], ((t.at / kTables) & 1) ^ 1, ctl, kSiteLseEmpty)))
        return false;
      uint8_t *tab = smem + L::kOffTab + st * L::kTabBytes;
      int least = 0x7fffffff;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const int col = c * 32 + lane;
        const bool on = t.lse[c] != -INFINITY;
        const int last = on ? t.last[c] : -1;
        if (col < NT) {
          reinterpret_cast<float *>(tab)[col] = on ? -(t.lse[c] * kLog2e) : 0.0f;
          reinterpret_cast<int *>(tab)[NT + col] = last;
          least = min(least, last);
        }
      }
      least = __reduce_min_sync(0xffffffffu, least);
      if (lane == 0) reinterpret_cast<int *>(tab)[2 * NT] = least;
      warp_arrive(&tab_full[st]);
      return true;
    };
    Tile held;
    held.on = false;
    for (int r = 0; ok; ++r) {
      const long long u = unit_index(r);
      if (r * static_cast<long long>(gridDim.x) >= p.units) break;
      if (u >= p.units) continue;
      const Unit n = unit_at(p, u);
      for (int x = n.x0; ok && x < n.x1; ++x, ++cnt) {
        if (static_cast<int>(cnt & 1) != me) continue;
        const Tile next = fetch(n, x, cnt);
        if (held.on) ok = put(held);
        held = next;
      }
    }
    if (ok && held.on) put(held);
  } else {
    // ------------------------------------------------------------ weights
    const int t = warp >> 2, tid = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float2 cc = make_float2(p.scale_log2, p.scale_log2);
    uint32_t cnt = 0;
    bool ok = true;
    for (int r = 0; ok; ++r) {
      const long long u = unit_index(r);
      if (r * static_cast<long long>(gridDim.x) >= p.units) break;
      if (u >= p.units) continue;
      const Unit n = unit_at(p, u);
      const int key = n.key0 + t * kKeys + tid;
      const int key_last = n.key0 + t * kKeys + kKeys - 1;
      float total = 0.0f;
      for (int x = n.x0; x < n.x1; ++x, ++cnt) {
        const uint32_t buf = cnt & 1, st = cnt % kTables;
        ok = mbar_wait(&tab_full[st], (cnt / kTables) & 1, ctl, kSiteLseFull) &&
             mbar_wait(&s_full[2 * t + buf], (cnt >> 1) & 1, ctl, kSiteSFull);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint8_t *tab = smem + L::kOffTab + st * L::kTabBytes;
        const float4 *nl = reinterpret_cast<const float4 *>(tab);
        const int4 *last = reinterpret_cast<const int4 *>(tab + NT * 4);
        // hidden columns: padded or empty rows, or rows that do not see the tile's last key
        const bool mask = key_last > reinterpret_cast<const int *>(tab)[2 * NT];
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
        total += sum.x + sum.y;
      }
      if (ok && key < p.Nk) {
        const long long at = (static_cast<long long>(n.b) * p.Hkv + n.hk) * p.Nk + key;
        const float add = key < n.len ? total : 0.0f;
        if (p.splits > 1)
          p.part[n.split * (static_cast<long long>(p.B) * p.Hkv * p.Nk) + at] = add;
        else
          p.w[at] = p.w_in ? (key < n.len ? p.w_in[at] + add : p.w_in[at]) : add;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
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

template <int D, int NT>
cudaError_t launch_kw(const CUtensorMap &tq, const CUtensorMap &tk, const KeyWeightParams &p, int sms,
                      cudaStream_t stream) {
  using L = KwLayout<D, NT>;
  auto kern = fa_key_weights_kernel<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kRequest);
  if (e != cudaSuccess) return e;
  const unsigned grid = p.units < sms ? static_cast<unsigned>(p.units) : static_cast<unsigned>(sms);
  kern<<<grid, kThreads, L::kRequest, stream>>>(tq, tk, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  const long long n = static_cast<long long>(p.B) * p.Hkv * p.Nk;
  fa_key_weights_sum_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_kw_d(int cols, const CUtensorMap &tq, const CUtensorMap &tk, const KeyWeightParams &p, int sms,
                        cudaStream_t stream) {
  switch (cols) {
    case 16: return launch_kw<D, 16>(tq, tk, p, sms, stream);
    case 32: return launch_kw<D, 32>(tq, tk, p, sms, stream);
    case 64: return launch_kw<D, 64>(tq, tk, p, sms, stream);
    default: return launch_kw<D, 128>(tq, tk, p, sms, stream);
  }
}

}  // namespace

KeyWeightPlan plan_key_weights(int B, int H, int Hkv, int Nq, int Nk) {
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
  return pl;
}

cudaError_t launch_key_weights(int d, int cols, const CUtensorMap &tq, const CUtensorMap &tk,
                               const KeyWeightParams &p, int sms, cudaStream_t stream) {
  return d == 64 ? launch_kw_d<64>(cols, tq, tk, p, sms, stream) : launch_kw_d<128>(cols, tq, tk, p, sms, stream);
}

}  // namespace fa
