// fa_cache_api.cu -- the C ABI of the operators around the key/value cache:
// argument validation, tensor maps, workspaces and launches.  The operations
// are defined in include/fa.h.

#include <cmath>
#include <cstdint>

#include "fa_cache.h"
#include "fa_host.h"

namespace fa {
namespace {

constexpr int kMaxRows = 1 << 30;       // rows of a cache, tokens of a call
constexpr int kMaxHeads = (1 << 24) - 1;  // B * H, and B * Hkv

// A memory range of an argument.
struct Range {
  uintptr_t lo, hi;
};
Range range_of(const void *p, long long bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, p ? lo + static_cast<uintptr_t>(bytes) : lo};
}
Range range_of(const void *p, int B, int H, int N, int d, const Strides &s) {
  Range r;
  span(p, B, H, N, d, s, &r.lo, &r.hi);
  return r;
}
bool meet(const Range &a, const Range &b) { return spans_overlap(a.lo, a.hi, b.lo, b.hi); }

// A stride of an int32 argument: up to a terabyte's elements, as other strides
// (products with it stay within 64 bits).
bool row_stride(int64_t s) { return s >= 0 && s < (1LL << 39); }

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A bf16 [B, H, N, d] argument with its strides.
struct View {
  const void *p;
  int H, N;
  Strides s;
};

bool make_view(const void *p, const int64_t *strides, int B, int H, int N, int d, View *v) {
  if (!p || !aligned16(p)) return false;
  v->p = p;
  v->H = H;
  v->N = N;
  return normalise(strides, B, H, N, d, &v->s);
}
bool overlap(const View &a, const View &b, int B, int d) {
  return may_overlap(a.p, a.s, a.H, a.N, b.p, b.s, b.H, b.N, B, d);
}
bool same_place(const View &a, const View &b) {
  return a.p == b.p && a.s.b == b.s.b && a.s.h == b.s.h && a.s.n == b.s.n;
}
Range range_of(const View &v, int B, int d) { return range_of(v.p, B, v.H, v.N, d, v.s); }
const __nv_bfloat16 *in(const View &v) { return static_cast<const __nv_bfloat16 *>(v.p); }
__nv_bfloat16 *out(const View &v) { return const_cast<__nv_bfloat16 *>(in(v)); }

// A call's workspace: the caller's, or taken on the stream for the call.
struct Scratch {
  void *ptr;
  size_t bytes, need;
  bool owned = false;
  Scratch(void *workspace, size_t workspace_bytes, size_t need_bytes)
      : ptr(need_bytes ? workspace : nullptr), bytes(workspace_bytes), need(need_bytes) {}
  // The caller's: large enough, aligned, apart from the call's other memory.
  fa_status_t check(const Range *used, int n) const {
    if (!ptr) return FA_OK;
    if (bytes < need) return FA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ptr) & 255u) return FA_ERR_INVALID_ARGUMENT;
    const Range r = range_of(ptr, static_cast<long long>(need));
    for (int i = 0; i < n; ++i)
      if (meet(r, used[i])) return FA_ERR_INVALID_ARGUMENT;
    return FA_OK;
  }
  bool take(cudaStream_t stream) {
    if (!need || ptr) return true;
    owned = cudaMallocAsync(&ptr, need, stream) == cudaSuccess;
    return owned;
  }
  bool give_back(cudaStream_t stream) { return !owned || cudaFreeAsync(ptr, stream) == cudaSuccess; }
};

fa_status_t check_d(int d) {
  if (d == 64 || d == 128) return FA_OK;
  return d < 1 ? FA_ERR_INVALID_ARGUMENT : FA_ERR_UNSUPPORTED;
}

// ------------------------------------------------------------------ rotary positions

fa_status_t check_rope(int B, int H, int Hkv, int N, int d, int rot, int interleaved, float factor) {
  if (B < 1 || H < 1 || Hkv < 0 || N < 1) return FA_ERR_INVALID_ARGUMENT;
  if (interleaved != 0 && interleaved != 1) return FA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(factor)) return FA_ERR_INVALID_ARGUMENT;
  const fa_status_t st = check_d(d);
  if (st != FA_OK) return st;
  if (rot < 1 || rot > d) return FA_ERR_INVALID_ARGUMENT;
  if (rot % 16) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * N > kMaxRows) return FA_ERR_INVALID_ARGUMENT;
  if (static_cast<long long>(B) * H > kMaxHeads || static_cast<long long>(B) * Hkv > kMaxHeads)
    return FA_ERR_INVALID_ARGUMENT;
  return FA_OK;
}

// Tokens of a CTA and CTAs along the head axis: up to 4 (d = 128) or 8 tokens
// (B4 H32 N4096 d128 and B8 H16 Hkv4 N2047 d64 82 and 16.6 us, twice as many 86 and
// 18.2; with CTAs of 256 threads 8 and 16 tokens 83 and 17.3), fewer while that
// leaves SMs without two CTAs, then the heads cut.
void plan_rope(RopeParams *p) {
  const long long all = static_cast<long long>(p->B) * p->N;
  int tokens = p->d == 128 ? 4 : 8;
  while (tokens > 1 && all / tokens < 2 * 152) tokens /= 2;
  const int at_once = 128 / (p->d / 16 * tokens);
  const long long blocks = (all + tokens - 1) / tokens;
  long long groups = (p->heads + at_once - 1) / at_once;
  const long long want = (4 * 152 + blocks - 1) / blocks;
  if (groups > want) groups = want;
  p->tokens = tokens;
  p->head_groups = groups > 65535 ? 65535 : static_cast<int>(groups);
}

fa_status_t rope_impl(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides, void *q_out,
                      const int64_t *q_out_strides, void *k_out, const int64_t *k_out_strides, const int *positions,
                      int64_t positions_stride, const float *inv_freq, int B, int H, int Hkv, int N, int d, int rot,
                      int interleaved, float factor, float sign, cudaStream_t stream) {
  const fa_status_t st = check_rope(B, H, Hkv, N, d, rot, interleaved, factor);
  if (st != FA_OK) return st;
  if (!inv_freq || !aligned4(inv_freq) || !aligned4(positions) || !row_stride(positions_stride)) return FA_ERR_INVALID_ARGUMENT;
  const bool has_k = Hkv > 0;
  View vq, vk{}, vqo, vko{};
  if (!make_view(q, q_strides, B, H, N, d, &vq) || !make_view(q_out, q_out_strides, B, H, N, d, &vqo))
    return FA_ERR_INVALID_ARGUMENT;
  if (has_k ? !make_view(k, k_strides, B, Hkv, N, d, &vk) || !make_view(k_out, k_out_strides, B, Hkv, N, d, &vko)
            : k || k_out)
    return FA_ERR_INVALID_ARGUMENT;
  if (!injective(B, H, N, d, vqo.s) || (has_k && !injective(B, Hkv, N, d, vko.s))) return FA_ERR_INVALID_ARGUMENT;
  // each output is its own input's place or shares nothing with any argument
  if (!same_place(vq, vqo) && overlap(vq, vqo, B, d)) return FA_ERR_INVALID_ARGUMENT;
  if (has_k) {
    if (!same_place(vk, vko) && overlap(vk, vko, B, d)) return FA_ERR_INVALID_ARGUMENT;
    if (overlap(vk, vqo, B, d) || overlap(vq, vko, B, d) || overlap(vqo, vko, B, d)) return FA_ERR_INVALID_ARGUMENT;
  }
  const Range pos = range_of(positions, (static_cast<long long>(B - 1) * positions_stride + N) * 4);
  const Range fr = range_of(inv_freq, rot / 2 * 4);
  const Range qo = range_of(vqo, B, d);
  if (meet(pos, qo) || meet(fr, qo)) return FA_ERR_INVALID_ARGUMENT;
  if (has_k) {
    const Range ko = range_of(vko, B, d);
    if (meet(pos, ko) || meet(fr, ko)) return FA_ERR_INVALID_ARGUMENT;
  }
  RopeParams p{};
  p.q = in(vq);
  p.qo = out(vqo);
  p.sq = vq.s;
  p.sqo = vqo.s;
  if (has_k) {
    p.k = in(vk);
    p.ko = out(vko);
    p.sk = vk.s;
    p.sko = vko.s;
  }
  p.positions = positions;
  p.pos_b = positions_stride;
  p.inv_freq = inv_freq;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.N = N;
  p.d = d;
  p.rot = rot;
  p.factor = factor;
  p.sign = sign;
  p.heads = H + Hkv;
  plan_rope(&p);
  return launch_rope(interleaved != 0, p, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// ------------------------------------------------------------------ caches

fa_status_t check_cache(int B, int H, int Hkv, int Nk, int d) {
  if (B < 1 || H < 1 || Hkv < 1 || Nk < 1) return FA_ERR_INVALID_ARGUMENT;
  const fa_status_t st = check_d(d);
  if (st != FA_OK) return st;
  if (H % Hkv) return FA_ERR_INVALID_ARGUMENT;
  if (static_cast<long long>(B) * H > kMaxHeads || Nk > kMaxRows) return FA_ERR_INVALID_ARGUMENT;
  return FA_OK;
}

constexpr int kTreeMaxNodes = 128;

fa_status_t check_tree(int B, int H, int Hkv, int Nt, int Nk, int d, float scale) {
  const fa_status_t st = check_cache(B, H, Hkv, Nk, d);
  if (st != FA_OK) return st;
  if (Nt < 1 || Nt > kTreeMaxNodes) return FA_ERR_INVALID_ARGUMENT;
  return std::isfinite(scale) ? FA_OK : FA_ERR_INVALID_ARGUMENT;
}

fa_status_t check_key_weights(int B, int H, int Hkv, int Nq, int Nk, int d, int causal, float scale) {
  const fa_status_t st = check_cache(B, H, Hkv, Nk, d);
  if (st != FA_OK) return st;
  if (Nq < 1 || Nq > kMaxRows || (causal != 0 && causal != 1)) return FA_ERR_INVALID_ARGUMENT;
  // 256-key blocks are counted in 31 bits (weights of 2 TiB)
  if (static_cast<long long>(B) * Hkv * ((Nk + 255) / 256) >= (1LL << 31)) return FA_ERR_INVALID_ARGUMENT;
  return std::isfinite(scale) ? FA_OK : FA_ERR_INVALID_ARGUMENT;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status_t fa_rope_frequencies(float *inv_freq, float *factor_out, int rot, double base, int scaling, double factor,
                                int original_len, double fast_turns, double slow_turns) {
  if (!inv_freq || !factor_out || rot < 2 || rot % 2 || !(base > 1.0) || !std::isfinite(base))
    return FA_ERR_INVALID_ARGUMENT;
  if (scaling < FA_ROPE_PLAIN || scaling > FA_ROPE_BY_PARTS) return FA_ERR_INVALID_ARGUMENT;
  if (scaling != FA_ROPE_PLAIN && !(factor >= 1.0 && std::isfinite(factor))) return FA_ERR_INVALID_ARGUMENT;
  if (scaling == FA_ROPE_BASE && rot == 2) return FA_ERR_INVALID_ARGUMENT;  // the exponent rot / (rot - 2)
  if (scaling == FA_ROPE_BY_PARTS &&
      (original_len < 1 || !(slow_turns > 0.0) || !(fast_turns > slow_turns) || !std::isfinite(fast_turns)))
    return FA_ERR_INVALID_ARGUMENT;
  const double two_pi = 6.283185307179586476925;
  if (scaling == FA_ROPE_BASE) base *= std::pow(factor, static_cast<double>(rot) / (rot - 2));
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == FA_ROPE_LINEAR) {
      f /= factor;
    } else if (scaling == FA_ROPE_BY_PARTS) {
      double keep = (original_len * f / two_pi - slow_turns) / (fast_turns - slow_turns);
      keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
      f = f * keep + f / factor * (1.0 - keep);
    }
    inv_freq[i] = static_cast<float>(f);
  }
  *factor_out = scaling == FA_ROPE_BY_PARTS ? static_cast<float>(1.0 + 0.1 * std::log(factor)) : 1.0f;
  return FA_OK;
}

fa_status_t fa_rope(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides, void *q_out,
                    const int64_t *q_out_strides, void *k_out, const int64_t *k_out_strides, const int *positions,
                    int64_t positions_stride, const float *inv_freq, int B, int H, int Hkv, int N, int d, int rot,
                    int interleaved, float factor, cudaStream_t stream) {
  return rope_impl(q, q_strides, k, k_strides, q_out, q_out_strides, k_out, k_out_strides, positions,
                   positions_stride, inv_freq, B, H, Hkv, N, d, rot, interleaved, factor, 1.0f, stream);
}

fa_status_t fa_rope_bwd(const void *dq_out, const int64_t *dq_out_strides, const void *dk_out,
                        const int64_t *dk_out_strides, void *dq, const int64_t *dq_strides, void *dk,
                        const int64_t *dk_strides, const int *positions, int64_t positions_stride,
                        const float *inv_freq, int B, int H, int Hkv, int N, int d, int rot, int interleaved,
                        float factor, cudaStream_t stream) {
  return rope_impl(dq_out, dq_out_strides, dk_out, dk_out_strides, dq, dq_strides, dk, dk_strides, positions,
                   positions_stride, inv_freq, B, H, Hkv, N, d, rot, interleaved, factor, -1.0f, stream);
}

fa_status_t fa_rope_append(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                           const void *v, const int64_t *v_strides, void *q_out, const int64_t *q_out_strides,
                           void *k_cache, const int64_t *k_cache_strides, void *v_cache,
                           const int64_t *v_cache_strides, const int *cache_seqlens, const int *positions,
                           int64_t positions_stride, const float *inv_freq, int B, int H, int Hkv, int N, int Nk,
                           int d, int rot, int interleaved, float factor, cudaStream_t stream) {
  const fa_status_t st = check_rope(B, H, Hkv, N, d, rot, interleaved, factor);
  if (st != FA_OK) return st;
  if (Hkv < 1 || Nk < 1 || Nk > kMaxRows) return FA_ERR_INVALID_ARGUMENT;
  if (!inv_freq || !cache_seqlens || !aligned4(inv_freq) || !aligned4(cache_seqlens) || !aligned4(positions) ||
      !row_stride(positions_stride))
    return FA_ERR_INVALID_ARGUMENT;
  View vq, vk, vv, vqo, vkc, vvc;
  if (!make_view(q, q_strides, B, H, N, d, &vq) || !make_view(k, k_strides, B, Hkv, N, d, &vk) ||
      !make_view(v, v_strides, B, Hkv, N, d, &vv) || !make_view(q_out, q_out_strides, B, H, N, d, &vqo) ||
      !make_view(k_cache, k_cache_strides, B, Hkv, Nk, d, &vkc) ||
      !make_view(v_cache, v_cache_strides, B, Hkv, Nk, d, &vvc))
    return FA_ERR_INVALID_ARGUMENT;
  if (!injective(B, H, N, d, vqo.s) || !injective(B, Hkv, Nk, d, vkc.s) || !injective(B, Hkv, Nk, d, vvc.s))
    return FA_ERR_INVALID_ARGUMENT;
  const View *ins[3] = {&vq, &vk, &vv}, *outs[3] = {&vqo, &vkc, &vvc};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 3; ++i) {
      if (o == 0 && i == 0 && same_place(vq, vqo)) continue;
      if (overlap(*ins[i], *outs[o], B, d)) return FA_ERR_INVALID_ARGUMENT;
    }
    for (int x = o + 1; x < 3; ++x)
      if (overlap(*outs[o], *outs[x], B, d)) return FA_ERR_INVALID_ARGUMENT;
    const Range r = range_of(*outs[o], B, d);
    if (meet(r, range_of(cache_seqlens, 4ll * B)) || meet(r, range_of(inv_freq, rot / 2 * 4)) ||
        meet(r, range_of(positions, (static_cast<long long>(B - 1) * positions_stride + N) * 4)))
      return FA_ERR_INVALID_ARGUMENT;
  }
  RopeParams p{};
  p.q = in(vq);
  p.k = in(vk);
  p.v = in(vv);
  p.qo = out(vqo);
  p.ko = out(vkc);
  p.vo = out(vvc);
  p.sq = vq.s;
  p.sk = vk.s;
  p.sv = vv.s;
  p.sqo = vqo.s;
  p.sko = vkc.s;
  p.svo = vvc.s;
  p.positions = positions;
  p.pos_b = positions_stride;
  p.inv_freq = inv_freq;
  p.cache_len = cache_seqlens;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.N = N;
  p.Nk = Nk;
  p.d = d;
  p.rot = rot;
  p.factor = factor;
  p.sign = 1.0f;
  p.heads = H + 2 * Hkv;
  plan_rope(&p);
  return launch_rope(interleaved != 0, p, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_tree_workspace_bytes(int B, int H, int Hkv, int Nt, int Nk, int d) {
  if (check_tree(B, H, Hkv, Nt, Nk, d, 1.0f) != FA_OK) return 0;
  const TreePlan pl = plan_tree(B, H, Hkv, Nt, Nk);
  return pl.merge ? round256(pl.part_rows * d * 4) + round256(pl.part_rows * 4) + round256(pl.ranges * sizeof(int4)) : 0;
}

fa_status_t fa_fwd_tree(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                        const void *v, const int64_t *v_strides, void *o, const int64_t *o_strides, float *lse,
                        const int *parents, int64_t parents_stride, const int *cache_seqlens, int B, int H, int Hkv,
                        int Nt, int Nk, int d, float scale, void *workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
  const fa_status_t st = check_tree(B, H, Hkv, Nt, Nk, d, scale);
  if (st != FA_OK) return st;
  if (!lse || !aligned16(lse) || !parents || !aligned4(parents) || !row_stride(parents_stride) || !aligned4(cache_seqlens))
    return FA_ERR_INVALID_ARGUMENT;
  View vq, vk, vv, vo;
  if (!make_view(q, q_strides, B, H, Nt, d, &vq) || !make_view(k, k_strides, B, Hkv, Nk, d, &vk) ||
      !make_view(v, v_strides, B, Hkv, Nk, d, &vv) || !make_view(o, o_strides, B, H, Nt, d, &vo))
    return FA_ERR_INVALID_ARGUMENT;
  if (!injective(B, H, Nt, d, vo.s)) return FA_ERR_INVALID_ARGUMENT;
  const Range rl = range_of(lse, 4ll * B * H * Nt), ro = range_of(vo, B, d);
  const Range par = range_of(parents, 4 * (static_cast<long long>(B - 1) * parents_stride + Nt));
  const Range len = range_of(cache_seqlens, 4ll * B);
  if (overlap(vq, vo, B, d) || overlap(vk, vo, B, d) || overlap(vv, vo, B, d)) return FA_ERR_INVALID_ARGUMENT;
  if (meet(rl, ro) || meet(par, ro) || meet(len, ro) || meet(par, rl) || meet(len, rl) ||
      meet(range_of(vq, B, d), rl) || meet(range_of(vk, B, d), rl) || meet(range_of(vv, B, d), rl))
    return FA_ERR_INVALID_ARGUMENT;
  const TreePlan pl = plan_tree(B, H, Hkv, Nt, Nk);
  const size_t need = fa_tree_workspace_bytes(B, H, Hkv, Nt, Nk, d);
  Scratch ws(workspace, workspace_bytes, need);
  const Range used[7] = {range_of(vq, B, d), range_of(vk, B, d), range_of(vv, B, d), ro, rl, par, len};
  const fa_status_t wst = ws.check(used, 7);
  if (wst != FA_OK) return wst;
  CUtensorMap tq, tk, tv;
  if (!encode_map(&tq, q, B, H, Nt, d, vq.s, Nt, pl.gpt) || !encode_map(&tk, k, B, Hkv, Nk, d, vk.s) ||
      !encode_map(&tv, v, B, Hkv, Nk, d, vv.s))
    return FA_ERR_CUDA;
  TreeParams p{};
  p.status = status_ptr();
  if (!p.status || !ws.take(stream)) return FA_ERR_CUDA;
  p.o = out(vo);
  p.lse = lse;
  p.so = vo.s;
  p.parents = parents;
  p.par_b = parents_stride;
  p.cache_len = cache_seqlens;
  p.part_o = static_cast<float *>(ws.ptr);
  if (need) {
    uint8_t *at = static_cast<uint8_t *>(ws.ptr) + round256(pl.part_rows * d * 4);
    p.part_lse = reinterpret_cast<float *>(at);
    p.cuts = reinterpret_cast<int4 *>(at + round256(pl.part_rows * 4));
  }
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.G = H / Hkv;
  p.Nt = Nt;
  p.Nk = Nk;
  p.d = d;
  p.gpt = pl.gpt;
  p.row_tiles = pl.row_tiles;
  p.groups = pl.groups;
  p.ranges = pl.ranges;
  p.split = pl.split;
  p.whole = pl.whole;
  p.cuts_by_unit = static_cast<long long>(B) * Hkv <= pl.ranges ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.neg = scale < 0.0f ? 1 : 0;
  const bool launched = launch_tree(tq, tk, tv, p, pl.merge, stream) == cudaSuccess;
  return ws.give_back(stream) && launched ? FA_OK : FA_ERR_CUDA;
}

size_t fa_key_weights_workspace_bytes(int B, int H, int Hkv, int Nq, int Nk, int d) {
  if (check_key_weights(B, H, Hkv, Nq, Nk, d, 0, 1.0f) != FA_OK) return 0;
  const KeyWeightPlan pl = plan_key_weights(B, H, Hkv, Nq, Nk, d);
  return pl.splits > 1 ? round256(static_cast<size_t>(pl.splits) * B * Hkv * Nk * 4) : 0;
}

fa_status_t fa_key_weights(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                           const float *lse, const float *weights_in, float *weights, const int *cache_seqlens, int B,
                           int H, int Hkv, int Nq, int Nk, int d, int causal, float scale, void *workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  const fa_status_t st = check_key_weights(B, H, Hkv, Nq, Nk, d, causal, scale);
  if (st != FA_OK) return st;
  if (!lse || !weights || !aligned16(lse) || !aligned16(weights) || !aligned16(weights_in) || !aligned4(cache_seqlens))
    return FA_ERR_INVALID_ARGUMENT;
  View vq, vk;
  if (!make_view(q, q_strides, B, H, Nq, d, &vq) || !make_view(k, k_strides, B, Hkv, Nk, d, &vk))
    return FA_ERR_INVALID_ARGUMENT;
  const long long wbytes = 4ll * B * Hkv * Nk;
  const Range rw = range_of(weights, wbytes);
  if (meet(rw, range_of(vq, B, d)) || meet(rw, range_of(vk, B, d)) || meet(rw, range_of(lse, 4ll * B * H * Nq)) ||
      meet(rw, range_of(cache_seqlens, 4ll * B)) || (weights_in != weights && meet(rw, range_of(weights_in, wbytes))))
    return FA_ERR_INVALID_ARGUMENT;
  const KeyWeightPlan pl = plan_key_weights(B, H, Hkv, Nq, Nk, d);
  Scratch ws(workspace, workspace_bytes, fa_key_weights_workspace_bytes(B, H, Hkv, Nq, Nk, d));
  const Range used[6] = {range_of(vq, B, d), range_of(vk, B, d), range_of(lse, 4ll * B * H * Nq), rw,
                         range_of(weights_in, wbytes), range_of(cache_seqlens, 4ll * B)};
  const fa_status_t wst = ws.check(used, 6);
  if (wst != FA_OK) return wst;
  const int sms = sm_count();
  CUtensorMap tq, tk;
  if (sms <= 0 || !encode_map(&tq, q, B, H, Nq, d, vq.s, pl.box_rows, pl.gpt) ||
      !encode_map(&tk, k, B, Hkv, Nk, d, vk.s, pl.cols == 128 ? 256 : 128))
    return FA_ERR_CUDA;
  KeyWeightParams p{};
  p.status = status_ptr();
  if (!p.status || !ws.take(stream)) return FA_ERR_CUDA;
  p.lse = lse;
  p.w_in = weights_in;
  p.w = weights;
  p.part = static_cast<float *>(ws.ptr);
  p.cache_len = cache_seqlens;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.G = H / Hkv;
  p.Nq = Nq;
  p.Nk = Nk;
  p.causal = causal;
  p.gpt = pl.gpt;
  p.tiles_per_head = pl.tiles_per_head;
  p.head_groups = pl.head_groups;
  p.splits = pl.splits;
  p.window = pl.window;
  p.units = static_cast<uint32_t>(static_cast<long long>(B) * Hkv * ((Nk + 255) / 256) * pl.splits);
  p.scale_log2 = scale * 1.4426950408889634f;
  const bool launched = launch_key_weights(d, pl.cols, tq, tk, p, sms, stream) == cudaSuccess;
  return ws.give_back(stream) && launched ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_cache_select(const float *weights, const int *cache_seqlens, int *kept, int *new_seqlens, int B,
                            int Hkv, int Nk, int keep, int first, int recent, cudaStream_t stream) {
  if (B < 1 || Hkv < 1 || Nk < 1 || Nk > kMaxRows || static_cast<long long>(B) * Hkv > kMaxHeads)
    return FA_ERR_INVALID_ARGUMENT;
  if (keep < 1 || keep > Nk || first < 0 || recent < 0 || static_cast<long long>(first) + recent > keep)
    return FA_ERR_INVALID_ARGUMENT;
  if (!weights || !kept || !new_seqlens || !aligned16(weights) || !aligned4(kept) || !aligned4(new_seqlens) ||
      !aligned4(cache_seqlens))
    return FA_ERR_INVALID_ARGUMENT;
  const Range rw = range_of(weights, 4ll * B * Hkv * Nk), rk = range_of(kept, 4ll * B * Hkv * keep);
  const Range rn = range_of(new_seqlens, 4ll * B), rl = range_of(cache_seqlens, 4ll * B);
  if (meet(rw, rk) || meet(rw, rn) || meet(rk, rn) || meet(rl, rk) || meet(rl, rn)) return FA_ERR_INVALID_ARGUMENT;
  SelectParams p{};
  p.w = weights;
  p.cache_len = cache_seqlens;
  p.kept = kept;
  p.new_len = new_seqlens;
  p.B = B;
  p.Hkv = Hkv;
  p.Nk = Nk;
  p.keep = keep;
  p.first = first;
  p.recent = recent;
  return launch_cache_select(p, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_cache_compact(const void *k, const int64_t *k_strides, const void *v, const int64_t *v_strides,
                             const float *weights, void *k_out, const int64_t *k_out_strides, void *v_out,
                             const int64_t *v_out_strides, float *weights_out, const int *kept,
                             int64_t kept_b_stride, int64_t kept_h_stride, const int *base, int B, int Hkv, int Nk,
                             int Nk_out, int M, int d, cudaStream_t stream) {
  fa_status_t st = check_cache(B, Hkv, Hkv, Nk, d);
  if (st != FA_OK) return st;
  if (Nk_out < 1 || Nk_out > kMaxRows || M < 1 || M > kMaxRows) return FA_ERR_INVALID_ARGUMENT;
  if (static_cast<long long>(B) * Hkv * ((M + 63) / 64) >= (1LL << 31)) return FA_ERR_INVALID_ARGUMENT;  // the grid
  if (!kept || !aligned4(kept) || !row_stride(kept_b_stride) || !row_stride(kept_h_stride) || !aligned4(base))
    return FA_ERR_INVALID_ARGUMENT;
  if ((weights == nullptr) != (weights_out == nullptr) || !aligned4(weights) || !aligned4(weights_out))
    return FA_ERR_INVALID_ARGUMENT;
  View vk, vv, vko, vvo;
  if (!make_view(k, k_strides, B, Hkv, Nk, d, &vk) || !make_view(v, v_strides, B, Hkv, Nk, d, &vv) ||
      !make_view(k_out, k_out_strides, B, Hkv, Nk_out, d, &vko) ||
      !make_view(v_out, v_out_strides, B, Hkv, Nk_out, d, &vvo))
    return FA_ERR_INVALID_ARGUMENT;
  if (!injective(B, Hkv, Nk_out, d, vko.s) || !injective(B, Hkv, Nk_out, d, vvo.s)) return FA_ERR_INVALID_ARGUMENT;
  // all outputs in their inputs' place, or none
  const bool in_place = Nk == Nk_out && same_place(vk, vko) && same_place(vv, vvo) && weights == weights_out;
  const Range rw = range_of(weights, 4ll * B * Hkv * Nk), rwo = range_of(weights_out, 4ll * B * Hkv * Nk_out);
  const Range rk = range_of(kept, 4 * (static_cast<long long>(B - 1) * kept_b_stride +
                                       static_cast<long long>(Hkv - 1) * kept_h_stride + M));
  const Range rb = range_of(base, 4ll * B);
  const View *ins[2] = {&vk, &vv}, *outs[2] = {&vko, &vvo};
  for (int o = 0; o < 2; ++o) {
    for (int i = 0; i < 2; ++i) {
      if (in_place && i == o) continue;
      if (overlap(*ins[i], *outs[o], B, d)) return FA_ERR_INVALID_ARGUMENT;
    }
    const Range r = range_of(*outs[o], B, d);
    if (meet(r, rk) || meet(r, rb) || meet(r, rwo) || meet(r, rw) || meet(rwo, range_of(*ins[o], B, d)))
      return FA_ERR_INVALID_ARGUMENT;
  }
  if (overlap(vko, vvo, B, d) || meet(rwo, rk) || meet(rwo, rb) || (!in_place && meet(rw, rwo)))
    return FA_ERR_INVALID_ARGUMENT;
  CompactParams p{};
  p.k = in(vk);
  p.v = in(vv);
  p.w = weights;
  p.ko = out(vko);
  p.vo = out(vvo);
  p.wo = weights_out;
  p.sk = vk.s;
  p.sv = vv.s;
  p.sko = vko.s;
  p.svo = vvo.s;
  p.kept = kept;
  p.kept_b = kept_b_stride;
  p.kept_h = kept_h_stride;
  p.base = base;
  p.B = B;
  p.Hkv = Hkv;
  p.Nk = Nk;
  p.Nout = Nk_out;
  p.M = M;
  p.d = d;
  p.in_place = in_place ? 1 : 0;
  return launch_cache_compact(p, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
