// fa_append_fp8.cu -- rotary positions and the append to a cache held in 8 bits.
//
// A block of rows of a head has one scale, the least power of two by which its
// rows fit e4m3 (448): k turned by its positions in fp32 (fa_angles.cuh), or v,
// divided by it and rounded to codes once.  Where new rows go on in a block that
// holds rows already, the scale is the greater of the two; if it grew, the old
// rows' codes are rounded to it again (a shift of exponents, exact but for codes
// that fall below e4m3's normal range).
//
// What bounds it.  HBM: a token's q is read and written in bf16, its k and v are
// read in bf16 and written in 8 bits.  A CTA takes the tokens of one block of
// rows and walks heads: the tokens' angles are computed once, into shared memory,
// and a head's rows stay in registers between the search for their greatest value
// and the rounding, so nothing is read twice; the next three heads' rows are on their
// way meanwhile, copied asynchronously to places in shared memory that each thread
// has for itself (one head ahead in registers: B4 H32 Hkv8 N4001 d128 104 us).  Two pieces of 8 values are a thread's share of a head, so that a CTA has
// 256 to 1024 threads by the tokens in a block; with few tokens several heads share
// the CTA and the heads are cut across CTAs.

#include <cfloat>
#include <cstdint>

#include "fa_angles.cuh"
#include "fa_cache8.h"
#include "ptx.cuh"

namespace fa {
namespace {

__device__ __forceinline__ long long floor_shift(long long x, int s) { return x >> s; }  // (arithmetic: floors)

constexpr int kAhead = 3;  // heads on their way

__device__ __forceinline__ void copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}

// A value as e4m3 stores it: infinities become NaN (the conversion would
// saturate them).
__device__ __forceinline__ float storable(float x) { return fabsf(x) <= FLT_MAX ? x : NAN; }

// grid: x = blocks of rows (per_b of a sequence), y = head groups.  A head takes
// slots * d / 16 threads, all of the CTA's or a part.
template <bool INTERLEAVED, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) fa_append_fp8_kernel(const Append8Params p) {
  extern __shared__ float4 shared[];  // rows on their way [kAhead][2][threads], then cos and sin [slots][rot / 2]
  __shared__ uint32_t most[3][kThreads / 4];  // greatest values of the heads at work, used in turn
  const int per_row = p.d >> 4, half = p.rot >> 1, tid = threadIdx.x;
  const int lanes = per_row * p.slots;
  const int heads_at_once = kThreads / lanes;
  const int b = blockIdx.x / p.per_b, j = blockIdx.x - b * p.per_b;
  const int block = 1 << p.block_log2;
  const long long len = p.cache_len[b], start = len - p.N;
  // the block of rows [lo, lo + block) and the tokens n0 .. n0 + count - 1 in it
  const long long lo = (floor_shift(start, p.block_log2) + j) << p.block_log2;
  const long long from = lo > start ? lo : start, to = lo + block < len ? lo + block : len;
  if (from >= to) return;
  const int n0 = static_cast<int>(from - start), count = static_cast<int>(to - from);
  // of those, the ones with a row of the cache
  const bool any_row = from < p.Nk && to > 0;
  const bool has_old = start > lo && start > 0 && any_row;
  const int blk = any_row ? static_cast<int>(lo >> p.block_log2) : 0;

  float *cos_t = reinterpret_cast<float *>(shared + kAhead * 2 * kThreads), *sin_t = cos_t + p.slots * half;
  const int hl = tid / lanes, in_head = tid - hl * lanes;
  const int c = in_head & (per_row - 1), slot = in_head / per_row;
  const Pieces x = pieces_of<INTERLEAVED>(p.d, p.rot, c);
  const int heads = p.H + 2 * p.Hkv, step = heads_at_once * gridDim.y;
  const bool row_on = slot < count && from + slot >= 0 && from + slot < p.Nk;  // has a row of the cache
  // the rows of the head that this thread takes from h0 on
  auto ask = [&](int h0, int place) {
    const int hh = h0 + hl;
    const bool is_q = hh < p.H, is_k = !is_q && hh < p.H + p.Hkv;
    if (hh < heads && slot < count && (is_q || row_on)) {
      const int h = is_q ? hh : (is_k ? hh - p.H : hh - p.H - p.Hkv);
      const __nv_bfloat16 *row = is_q   ? p.q + b * p.sq.b + h * p.sq.h + (n0 + slot) * p.sq.n
                                 : is_k ? p.k + b * p.sk.b + h * p.sk.h + (n0 + slot) * p.sk.n
                                        : p.v + b * p.sv.b + h * p.sv.h + (n0 + slot) * p.sv.n;
      float4 *to = shared + place * 2 * kThreads + tid;
      copy16(to, row + x.c0);
      copy16(to + kThreads, row + x.c1);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ask(blockIdx.y * heads_at_once + i * step, i);

  for (int i = tid; i < 3 * (kThreads / 4); i += kThreads) most[i / (kThreads / 4)][i % (kThreads / 4)] = 0u;
  for (int e = tid; e < count * half; e += kThreads) {
    const int s = e / half, i = e - s * half;
    const long long pos = p.positions ? p.positions[b * p.pos_b + n0 + s] : from + s;
    float cs_e, sn_e;
    angle_of(pos, p.inv_freq[i], &cs_e, &sn_e);
    cos_t[e] = cs_e * p.factor;
    sin_t[e] = sn_e * p.factor;
  }
  __syncthreads();
  int turn = 0, place = 0;
  for (int h0 = blockIdx.y * heads_at_once; h0 < heads; h0 += step, place = place == kAhead - 1 ? 0 : place + 1) {
    const int hh = h0 + hl;
    const bool is_q = hh < p.H, is_k = !is_q && hh < p.H + p.Hkv;
    const bool head_on = hh < heads && (is_q || any_row);
    const bool on = head_on && slot < count && (is_q || row_on);
    const int h = is_q ? hh : (is_k ? hh - p.H : hh - p.H - p.Hkv);
    float *scale = (is_k ? p.ks : p.vs) + (static_cast<long long>(b) * p.Hkv + h) * p.blocks + blk;
    // the block's scale, if rows before these use it
    const float old = head_on && !is_q && has_old ? *scale : 0.0f;
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    const uint4 *mine = reinterpret_cast<const uint4 *>(shared + place * 2 * kThreads + tid);
    const uint4 w0 = mine[0], w1 = mine[kThreads];  // (what this thread asked for itself)
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    ask(h0 + kAhead * step, place);
    float y[16];
    float top = 0.0f;
    if (on) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 v = unpack2(w[i]);
        y[2 * i] = v.x;
        y[2 * i + 1] = v.y;
      }
      if (is_q || is_k) {
        // (whole quadruples: single values would meet in the same banks)
        float cs[8], sn[8];
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const int at = slot * half + ((i ? x.t1 : x.t0) ? (i ? x.p1 : x.p0) : 0);  // (pieces past rot have no angles)
          const float4 u = *reinterpret_cast<const float4 *>(cos_t + at), v = *reinterpret_cast<const float4 *>(sin_t + at);
          cs[i] = u.x, cs[i + 1] = u.y, cs[i + 2] = u.z, cs[i + 3] = u.w;
          sn[i] = v.x, sn[i + 1] = v.y, sn[i + 2] = v.z, sn[i + 3] = v.w;
        }
        if (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (!(i < 4 ? x.t0 : x.t1)) continue;
            const float a = y[2 * i], z = y[2 * i + 1];
            y[2 * i] = a * cs[i] - z * sn[i];
            y[2 * i + 1] = z * cs[i] + a * sn[i];
          }
        } else if (x.t0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a = y[i], z = y[8 + i];
            y[i] = a * cs[i] - z * sn[i];
            y[8 + i] = z * cs[i] + a * sn[i];
          }
        }
      }
      if (is_q) {
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = pack2(y[2 * i], y[2 * i + 1]);
        __nv_bfloat16 *dst = p.qo + b * p.sqo.b + h * p.sqo.h + (n0 + slot) * p.sqo.n;
        __stcs(reinterpret_cast<uint4 *>(dst + x.c0), make_uint4(o[0], o[1], o[2], o[3]));
        __stcs(reinterpret_cast<uint4 *>(dst + x.c1), make_uint4(o[4], o[5], o[6], o[7]));
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          y[i] = storable(y[i]);
          top = fmaxf(top, fabsf(y[i]));  // (fmaxf passes over NaN)
        }
      }
    }
    if (h0 + heads_at_once <= p.H) continue;  // (only q: the same for the whole CTA)
    // the heads' greatest values (that of this turn's slot was last read two barriers ago)
    const int now_turn = turn, next_turn = turn == 2 ? 0 : turn + 1;
    turn = next_turn;
    if (tid < heads_at_once) most[next_turn][tid] = 0u;
    // the lanes of a head within the warp first
    for (int o = 1; o < lanes && o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top > 0.0f && (lanes < 32 ? in_head == 0 : (tid & 31) == 0)) atomicMax(&most[now_turn][hl], __float_as_uint(top));
    __syncthreads();
    if (!head_on || is_q) continue;
    const float now = fmaxf(old, least_scale(__uint_as_float(most[now_turn][hl]))), inv = 1.0f / now;
    uint8_t *dst = is_k ? p.kc + b * p.skc.b + h * p.skc.h : p.vc + b * p.svc.b + h * p.svc.h;
    const long long dn = is_k ? p.skc.n : p.svc.n;
    if (has_old && now > old) {  // the rows before the new ones, 16 bytes a thread
      const int rows = static_cast<int>(start - lo) * per_row;
      const float r = old / now;
      for (int e = in_head; e < rows; e += lanes) {
        uint4 *at = reinterpret_cast<uint4 *>(dst + (lo + e / per_row) * dn + (e & (per_row - 1)) * 16);
        uint4 v = *at;
        v.x = rescale_codes(v.x, r);
        v.y = rescale_codes(v.y, r);
        v.z = rescale_codes(v.z, r);
        v.w = rescale_codes(v.w, r);
        *at = v;
      }
    }
    if (on) {
      uint8_t *row = dst + (from + slot) * dn;
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = pack_e4m3x4(y[4 * i] * inv, y[4 * i + 1] * inv, y[4 * i + 2] * inv, y[4 * i + 3] * inv);
      *reinterpret_cast<uint2 *>(row + x.c0) = make_uint2(o[0], o[1]);
      *reinterpret_cast<uint2 *>(row + x.c1) = make_uint2(o[2], o[3]);
    }
    if (in_head == 0) *scale = now;
  }
}

template <bool INTERLEAVED, int kThreads>
cudaError_t launch_append8_t(const Append8Params &p, cudaStream_t stream) {
  auto kern = fa_append_fp8_kernel<INTERLEAVED, kThreads>;
  const size_t smem = kAhead * 2 * kThreads * 16 + sizeof(float) * p.slots * p.rot;  // up to 96 + 64 KB
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kAhead * 2 * kThreads * 16 + 65536);
  if (e != cudaSuccess) return e;
  kern<<<dim3(static_cast<unsigned>(p.B) * p.per_b, p.head_groups), kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

// A head's lanes, 4 (one token, d = 64) to 1024, all in one CTA.
int threads_of(const Append8Params &p) {
  const int lanes = p.slots * (p.d / 16);
  return lanes > 512 ? 1024 : (lanes > 256 ? 512 : 256);
}

template <bool INTERLEAVED>
cudaError_t launch_append8_i(const Append8Params &p, cudaStream_t stream) {
  switch (threads_of(p)) {
    case 1024: return launch_append8_t<INTERLEAVED, 1024>(p, stream);
    case 512: return launch_append8_t<INTERLEAVED, 512>(p, stream);
    default: return launch_append8_t<INTERLEAVED, 256>(p, stream);
  }
}

}  // namespace

cudaError_t launch_append8(bool interleaved, const Append8Params &in, cudaStream_t stream) {
  Append8Params p = in;
  const int block = 1 << p.block_log2;
  p.per_b = (p.N - 1 + block - 1) / block + 1;
  p.slots = 1;
  while (p.slots < p.N && p.slots < block) p.slots *= 2;
  const int heads = p.H + 2 * p.Hkv, at_once = threads_of(p) / (p.slots * (p.d / 16));
  const long long blocks = static_cast<long long>(p.B) * p.per_b;
  long long groups = (heads + at_once - 1) / at_once;
  const long long want = (4 * 152 + blocks - 1) / blocks;  // four CTAs an SM where there are heads for them
  if (groups > want) groups = want;
  p.head_groups = groups > 65535 ? 65535 : static_cast<int>(groups);
  return interleaved ? launch_append8_i<true>(p, stream) : launch_append8_i<false>(p, stream);
}

}  // namespace fa
