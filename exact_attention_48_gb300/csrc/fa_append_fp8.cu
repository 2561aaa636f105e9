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
// read in bf16 and written in 8 bits.  A CTA takes the tokens of one block of rows
// and walks heads of q, of k or of v: a thread has two pieces of 8 values of each
// head and their angles in registers, a head's values stay there between the search
// for their greatest and the rounding, and the next three heads' are on their way,
// copied asynchronously to places in shared memory that each thread has for itself.
// 256 to 1024 threads by the tokens in a block; with few tokens several heads share
// the CTA.  B4 H32 Hkv8 N4001 d128 (360 MB, 53 us at the copy rate): one head ahead in
// registers 104 us, three in shared memory 92 (issue slots: 380 instructions a piece,
// many of them addresses); one of the three tensors a CTA, addresses stepped from
// head to head and infinities looked for by the greatest value alone 76, 0.70 of that rate (64
// registers, so that 1024 threads fit an SM; 44 to 52 bytes of spills stored, 32 to 36 loaded).  A CTA
// works out its tokens' angles itself (some 50 instructions each): with as few CTAs as
// fill the SMs B16 H16 Hkv1 N1500 d64 takes 23 us, with four times as many 29.

#include <cfloat>
#include <cstdint>

#include "fa_angles.cuh"
#include "fa_cache8.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kAhead = 3;  // heads on their way

__device__ __forceinline__ void copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}

// grid: x = blocks of rows (per_b of a sequence), y = groups of q heads, then of k
// heads, then of v heads.  A head takes slots * d / 16 threads, all of the CTA's or a
// part.
template <bool INTERLEAVED, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) fa_append_fp8_kernel(const Append8Params p) {
  extern __shared__ float4 shared[];  // rows on their way [kAhead][2][threads]
  __shared__ uint64_t turns[64];              // the pairs' fractions of a turn
  __shared__ uint32_t most[3][kThreads / 4];  // greatest values of the heads at work, used in turn
  const int per_row = p.d >> 4, tid = threadIdx.x;
  const int lanes = per_row * p.slots;
  const int b = blockIdx.x / p.per_b, j = blockIdx.x - b * p.per_b;
  const int block = 1 << p.block_log2;
  const long long len = p.cache_len[b], start = len - p.N;
  // the block of rows [lo, lo + block) and the tokens n0 .. n0 + count - 1 in it
  const long long lo = ((start >> p.block_log2) + j) << p.block_log2;  // (arithmetic: floors)
  const long long from = lo > start ? lo : start, to = lo + block < len ? lo + block : len;
  if (from >= to) return;
  const int n0 = static_cast<int>(from - start), count = static_cast<int>(to - from);
  // this CTA's tensor and its heads
  const bool is_q = static_cast<int>(blockIdx.y) < p.q_groups, is_v = static_cast<int>(blockIdx.y) >= p.q_groups + p.kv_groups;
  const int group = blockIdx.y - (is_q ? 0 : (is_v ? p.q_groups + p.kv_groups : p.q_groups));
  const int groups = is_q ? p.q_groups : p.kv_groups, heads = is_q ? p.H : p.Hkv;
  // of the tokens, k's and v's with a row of the cache
  if (!is_q && !(from < p.Nk && to > 0)) return;
  const bool has_old = !is_q && start > lo && start > 0;

  const int hl = tid / lanes, in_head = tid - hl * lanes;
  const int c = in_head & (per_row - 1), slot = in_head / per_row;
  const Pieces x = pieces_of<INTERLEAVED>(p.d, p.rot, c);
  const int step = kThreads / lanes * groups;
  const bool on = slot < count && (is_q || (from + slot >= 0 && from + slot < p.Nk));
  const int first = group * (kThreads / lanes) + hl;  // this thread's first head
  const Strides &ss = is_q ? p.sq : (is_v ? p.sv : p.sk);
  const __nv_bfloat16 *src = (is_q ? p.q : (is_v ? p.v : p.k)) + b * ss.b + first * ss.h + (n0 + slot) * ss.n + x.c0;
  const long long src_step = step * ss.h;
  const int c1 = x.c1 - x.c0;
  int asked = first;
  auto ask = [&](int place) {
    if (on && asked < heads) {
      float4 *to = shared + place * 2 * kThreads + tid;
      copy16(to, src);
      copy16(to + kThreads, src + c1);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    asked += step;
    src += src_step;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ask(i);

  if (!is_v && tid < p.rot / 2) turns[tid] = turn_fraction(p.inv_freq[tid]);
  for (int i = tid; i < 3 * (kThreads / 4); i += kThreads) most[i / (kThreads / 4)][i % (kThreads / 4)] = 0u;
  __syncthreads();
  // the angles of this thread's pairs (threads of other heads and of other CTAs compute the same ones: cheaper than
  // to share them where a thread keeps them for all of its heads)
  float cs[8], sn[8];
  if (!is_v && on) {
    const long long pos = p.positions ? p.positions[b * p.pos_b + n0 + slot] : from + slot;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = 1.0f;
      sn[i] = 0.0f;
      if (!(i < 4 ? x.t0 : x.t1)) continue;
      angle_of(pos, turns[i < 4 ? x.p0 + i : x.p1 + i - 4], &cs[i], &sn[i]);
      cs[i] *= p.factor;
      sn[i] *= p.factor;
    }
  }

  const long long row = from + slot;
  uint8_t *head8 = is_v ? p.vc + b * p.svc.b + first * p.svc.h : p.kc + b * p.skc.b + first * p.skc.h;
  const long long step8 = step * (is_v ? p.svc.h : p.skc.h), dn = is_v ? p.svc.n : p.skc.n;
  __nv_bfloat16 *out = p.qo + b * p.sqo.b + first * p.sqo.h + (n0 + slot) * p.sqo.n + x.c0;
  const long long out_step = step * p.sqo.h;
  float *scale = (is_v ? p.vs : p.ks) + (static_cast<long long>(b) * p.Hkv + first) * p.blocks +
                 (is_q ? 0 : static_cast<int>(lo >> p.block_log2));
  int turn = 0, place = 0;
  const int rounds = (heads - group * (kThreads / lanes) + step - 1) / step;  // (the same for the whole CTA)
  for (int i = 0, h = first; i < rounds; ++i, h += step, place = place == kAhead - 1 ? 0 : place + 1) {
    // the block's scale, if rows before these use it
    const float old = has_old && h < heads ? *scale : 0.0f;
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    const uint4 *mine = reinterpret_cast<const uint4 *>(shared + place * 2 * kThreads + tid);
    const uint4 w0 = mine[0], w1 = mine[kThreads];  // (what this thread asked for itself)
    ask(place);
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    float y[16];
    float top = 0.0f;
    if (on && h < heads) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 v = unpack2(w[e]);
        y[2 * e] = v.x;
        y[2 * e + 1] = v.y;
      }
      if (!is_v) {
        if (INTERLEAVED) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (!(e < 4 ? x.t0 : x.t1)) continue;
            const float a = y[2 * e], z = y[2 * e + 1];
            y[2 * e] = a * cs[e] - z * sn[e];
            y[2 * e + 1] = z * cs[e] + a * sn[e];
          }
        } else if (x.t0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a = y[e], z = y[8 + e];
            y[e] = a * cs[e] - z * sn[e];
            y[8 + e] = z * cs[e] + a * sn[e];
          }
        }
      }
      if (is_q) {
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = pack2(y[2 * e], y[2 * e + 1]);
        __stcs(reinterpret_cast<uint4 *>(out), make_uint4(o[0], o[1], o[2], o[3]));
        __stcs(reinterpret_cast<uint4 *>(out + c1), make_uint4(o[4], o[5], o[6], o[7]));
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(y[e]));  // (fmaxf passes over NaN)
        if (top == INFINITY) {  // infinities become NaN (the conversion would saturate them) and do not count
          top = 0.0f;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            y[e] = fabsf(y[e]) <= FLT_MAX ? y[e] : NAN;
            top = fmaxf(top, fabsf(y[e]));
          }
        }
      }
    }
    out += out_step;
    if (is_q) continue;
    // the heads' greatest values (that of this turn's slot was last read two barriers ago)
    const int now_turn = turn, next_turn = turn == 2 ? 0 : turn + 1;
    turn = next_turn;
    if (tid < kThreads / lanes) most[next_turn][tid] = 0u;
    // the lanes of a head within the warp first
    for (int o = 1; o < lanes && o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top > 0.0f && (lanes < 32 ? in_head == 0 : (tid & 31) == 0)) atomicMax(&most[now_turn][hl], __float_as_uint(top));
    __syncthreads();
    if (h < heads) {
      const float now = fmaxf(old, least_scale(__uint_as_float(most[now_turn][hl]))), inv = 1.0f / now;
      if (has_old && now > old) {  // the rows before the new ones, 16 bytes a thread
        const int rows = static_cast<int>(start - lo) * per_row;
        const float r = old / now;
        for (int e = in_head; e < rows; e += lanes) {
          uint4 *at = reinterpret_cast<uint4 *>(head8 + (lo + e / per_row) * dn + (e & (per_row - 1)) * 16);
          uint4 v = *at;
          v.x = rescale_codes(v.x, r);
          v.y = rescale_codes(v.y, r);
          v.z = rescale_codes(v.z, r);
          v.w = rescale_codes(v.w, r);
          *at = v;
        }
      }
      if (on) {
        uint8_t *dst = head8 + row * dn + x.c0;
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = pack_e4m3x4(y[4 * e] * inv, y[4 * e + 1] * inv, y[4 * e + 2] * inv, y[4 * e + 3] * inv);
        *reinterpret_cast<uint2 *>(dst) = make_uint2(o[0], o[1]);
        *reinterpret_cast<uint2 *>(dst + c1) = make_uint2(o[2], o[3]);
      }
      if (in_head == 0) *scale = now;
    }
    head8 += step8;
    scale += static_cast<long long>(step) * p.blocks;
  }
}

template <bool INTERLEAVED, int kThreads>
cudaError_t launch_append8_t(const Append8Params &p, cudaStream_t stream) {
  auto kern = fa_append_fp8_kernel<INTERLEAVED, kThreads>;
  constexpr int kBytes = kAhead * 2 * kThreads * 16;  // up to 96 KB
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  kern<<<dim3(static_cast<unsigned>(p.B) * p.per_b, p.q_groups + 2 * p.kv_groups), kThreads, kBytes, stream>>>(p);
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
  // Groups of heads, in proportion to the heads: a CTA an SM in all (each one works out its tokens' angles)
  const int at_once = threads_of(p) / (p.slots * (p.d / 16));
  const long long blocks = static_cast<long long>(p.B) * p.per_b, want = (152 + blocks - 1) / blocks;
  auto groups = [&](int heads) {
    const long long most = (heads + at_once - 1) / at_once, share = (want * heads + p.H + 2 * p.Hkv - 1) / (p.H + 2 * p.Hkv);
    const long long g = share < most ? share : most;
    return static_cast<int>(g < 1 ? 1 : (g > 20000 ? 20000 : g));
  };
  p.q_groups = groups(p.H);
  p.kv_groups = groups(p.Hkv);
  return interleaved ? launch_append8_i<true>(p, stream) : launch_append8_i<false>(p, stream);
}

}  // namespace fa
