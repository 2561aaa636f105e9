// fa_cache8_api.cu -- the C ABI of the operators on a cache held in 8 bits and
// of the verification of drafted tokens: argument validation, tensor maps,
// workspaces and launches.  The operations are defined in include/fa.h.

#include <cmath>
#include <cstdint>

#include "fa_cache8.h"
#include "fa_views.h"

namespace fa {
namespace {

// A [B, Hkv, Nk, d] tensor of codes, a byte each: as a bf16 tensor of d / 2
// columns, so that the checks of views serve both.  The base and the strides in
// use are multiples of 16 bytes.
bool make_view8(const void *p, const int64_t *strides, int B, int H, int N, int d, View *v) {
  if (!strides) return false;
  int64_t half[3];
  for (int i = 0; i < 3; ++i) half[i] = strides[i] % 2 ? 1 : strides[i] / 2;  // (1: refused where it is used)
  return make_view(p, half, B, H, N, d / 2, v);
}
Strides bytes(const View &v) { return Strides{v.s.b * 2, v.s.h * 2, v.s.n * 2}; }

fa_status_t check_block(int block) {
  if (block < 1) return FA_ERR_INVALID_ARGUMENT;
  return block == 16 || block == 32 || block == 64 || block == 128 ? FA_OK : FA_ERR_UNSUPPORTED;
}
int log2_of(int block) { return block == 16 ? 4 : (block == 32 ? 5 : (block == 64 ? 6 : 7)); }
int blocks_of(int rows, int block) { return (rows + block - 1) / block; }
Range scales_of(const float *scale, int B, int Hkv, int rows, int block) {
  return range_of(scale, 4ll * B * Hkv * blocks_of(rows, block));
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_tree_fp8_workspace_bytes(int B, int H, int Hkv, int Nt, int Nk, int d) {
  if (check_tree(B, H, Hkv, Nt, Nk, d, 1.0f) != FA_OK) return 0;
  const Tree8Plan pl = plan_tree8(B, H, Hkv, Nt, Nk, d);
  return pl.merge ? round256(pl.part_rows * d * 4) + round256(pl.part_rows * 4) + round256(pl.ranges * sizeof(int4)) : 0;
}

fa_status_t fa_fwd_tree_fp8(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                            const void *v, const int64_t *v_strides, const float *k_scale, const float *v_scale,
                            void *o, const int64_t *o_strides, float *lse, const int *parents, int64_t parents_stride,
                            const int *cache_seqlens, int B, int H, int Hkv, int Nt, int Nk, int d, int block,
                            float scale, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  fa_status_t st = check_tree(B, H, Hkv, Nt, Nk, d, scale);
  if (st != FA_OK) return st;
  st = check_block(block);
  if (st != FA_OK) return st;
  if (!lse || !aligned16(lse) || !aligned4(parents) || !row_stride(parents_stride) || !aligned4(cache_seqlens) ||
      !k_scale || !v_scale || !aligned4(k_scale) || !aligned4(v_scale))
    return FA_ERR_INVALID_ARGUMENT;
  View vq, vk, vv, vo;
  if (!make_view(q, q_strides, B, H, Nt, d, &vq) || !make_view8(k, k_strides, B, Hkv, Nk, d, &vk) ||
      !make_view8(v, v_strides, B, Hkv, Nk, d, &vv) || !make_view(o, o_strides, B, H, Nt, d, &vo))
    return FA_ERR_INVALID_ARGUMENT;
  if (!injective(B, H, Nt, d, vo.s)) return FA_ERR_INVALID_ARGUMENT;
  const Range ro = range_of(vo, B, d), rl = range_of(lse, 4ll * B * H * Nt);
  const Range used[9] = {ro,
                         rl,
                         range_of(vq, B, d),
                         range_of(vk, B, d / 2),
                         range_of(vv, B, d / 2),
                         scales_of(k_scale, B, Hkv, Nk, block),
                         scales_of(v_scale, B, Hkv, Nk, block),
                         range_of(parents, parents ? 4 * (static_cast<long long>(B - 1) * parents_stride + Nt) : 0),
                         range_of(cache_seqlens, 4ll * B)};
  if (overlap(vq, vo, B, d) || meet(ro, rl) || meet(used[2], rl)) return FA_ERR_INVALID_ARGUMENT;
  for (int i = 3; i < 9; ++i)
    if (meet(used[i], ro) || meet(used[i], rl)) return FA_ERR_INVALID_ARGUMENT;
  const Tree8Plan pl = plan_tree8(B, H, Hkv, Nt, Nk, d);
  const size_t need = fa_tree_fp8_workspace_bytes(B, H, Hkv, Nt, Nk, d);
  Scratch ws(workspace, workspace_bytes, need);
  st = ws.check(used, 9);
  if (st != FA_OK) return st;
  CUtensorMap tk, tv;
  if (!encode_map_rows8(&tk, k, B, Hkv, Nk, d, bytes(vk), 128) || !encode_map_rows8(&tv, v, B, Hkv, Nk, d, bytes(vv), 128))
    return FA_ERR_CUDA;
  Tree8Params p{};
  p.status = status_ptr();
  if (!p.status || !ws.take(stream)) return FA_ERR_CUDA;
  p.q = in(vq);
  p.o = out(vo);
  p.lse = lse;
  p.sq = vq.s;
  p.so = vo.s;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
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
  p.block_log2 = log2_of(block);
  p.blocks = blocks_of(Nk, block);
  p.rows = pl.rows;
  p.groups = pl.groups;
  p.ranges = pl.ranges;
  p.whole = pl.whole;
  p.cuts_by_unit = static_cast<long long>(B) * Hkv <= pl.ranges ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  const bool launched = launch_tree8(tk, tv, p, pl.merge, stream) == cudaSuccess;
  return ws.give_back(stream) && launched ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_rope_append_fp8(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                               const void *v, const int64_t *v_strides, void *q_out, const int64_t *q_out_strides,
                               void *k_cache, const int64_t *k_cache_strides, void *v_cache,
                               const int64_t *v_cache_strides, float *k_scale, float *v_scale,
                               const int *cache_seqlens, const int *positions, int64_t positions_stride,
                               const float *inv_freq, int B, int H, int Hkv, int N, int Nk, int d, int rot,
                               int interleaved, float factor, int block, cudaStream_t stream) {
  fa_status_t st = check_rope(B, H, Hkv, N, d, rot, interleaved, factor);
  if (st != FA_OK) return st;
  st = check_block(block);
  if (st != FA_OK) return st;
  if (Hkv < 1 || Nk < 1 || Nk > kMaxRows) return FA_ERR_INVALID_ARGUMENT;
  if (!inv_freq || !cache_seqlens || !aligned4(inv_freq) || !aligned4(cache_seqlens) || !aligned4(positions) ||
      !row_stride(positions_stride) || !k_scale || !v_scale || !aligned4(k_scale) || !aligned4(v_scale))
    return FA_ERR_INVALID_ARGUMENT;
  View vq, vk, vv, vqo, vkc, vvc;
  if (!make_view(q, q_strides, B, H, N, d, &vq) || !make_view(k, k_strides, B, Hkv, N, d, &vk) ||
      !make_view(v, v_strides, B, Hkv, N, d, &vv) || !make_view(q_out, q_out_strides, B, H, N, d, &vqo) ||
      !make_view8(k_cache, k_cache_strides, B, Hkv, Nk, d, &vkc) ||
      !make_view8(v_cache, v_cache_strides, B, Hkv, Nk, d, &vvc))
    return FA_ERR_INVALID_ARGUMENT;
  if (!injective(B, H, N, d, vqo.s) || !injective(B, Hkv, Nk, d / 2, vkc.s) || !injective(B, Hkv, Nk, d / 2, vvc.s))
    return FA_ERR_INVALID_ARGUMENT;
  // no output shares an element with an input (but q_out with q) or another output
  if (!same_place(vq, vqo) && overlap(vq, vqo, B, d)) return FA_ERR_INVALID_ARGUMENT;
  if (overlap(vk, vqo, B, d) || overlap(vv, vqo, B, d) || overlap(vkc, vvc, B, d / 2)) return FA_ERR_INVALID_ARGUMENT;
  const Range ins[6] = {range_of(vq, B, d),
                        range_of(vk, B, d),
                        range_of(vv, B, d),
                        range_of(cache_seqlens, 4ll * B),
                        range_of(inv_freq, rot / 2 * 4),
                        range_of(positions, positions ? (static_cast<long long>(B - 1) * positions_stride + N) * 4 : 0)};
  const Range outs[5] = {range_of(vqo, B, d), range_of(vkc, B, d / 2), range_of(vvc, B, d / 2),
                         scales_of(k_scale, B, Hkv, Nk, block), scales_of(v_scale, B, Hkv, Nk, block)};
  for (int o = 0; o < 5; ++o) {
    for (int i = o == 0 ? 3 : 0; i < 6; ++i)
      if (meet(outs[o], ins[i])) return FA_ERR_INVALID_ARGUMENT;
    for (int x = o + 1; x < 5; ++x)
      if (!(o == 1 && x == 2) && meet(outs[o], outs[x])) return FA_ERR_INVALID_ARGUMENT;
  }
  Append8Params p{};
  p.q = in(vq);
  p.k = in(vk);
  p.v = in(vv);
  p.qo = out(vqo);
  p.kc = static_cast<uint8_t *>(k_cache);
  p.vc = static_cast<uint8_t *>(v_cache);
  p.ks = k_scale;
  p.vs = v_scale;
  p.sq = vq.s;
  p.sk = vk.s;
  p.sv = vv.s;
  p.sqo = vqo.s;
  p.skc = bytes(vkc);
  p.svc = bytes(vvc);
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
  p.block_log2 = log2_of(block);
  p.blocks = blocks_of(Nk, block);
  return launch_append8(interleaved != 0, p, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_cache_compact_fp8(const void *k, const int64_t *k_strides, const void *v, const int64_t *v_strides,
                                 const float *k_scale, const float *v_scale, void *k_out,
                                 const int64_t *k_out_strides, void *v_out, const int64_t *v_out_strides,
                                 float *k_scale_out, float *v_scale_out, const int *kept, int64_t kept_b_stride,
                                 int64_t kept_h_stride, const int *base, int B, int Hkv, int Nk, int Nk_out, int M,
                                 int d, int block, cudaStream_t stream) {
  fa_status_t st = check_cache(B, Hkv, Hkv, Nk, d);
  if (st != FA_OK) return st;
  st = check_block(block);
  if (st != FA_OK) return st;
  if (Nk_out < 1 || Nk_out > kMaxRows || M < 1 || M > kMaxRows) return FA_ERR_INVALID_ARGUMENT;
  if (static_cast<long long>(B) * Hkv * ((M + 127) / 128 + 1) >= (1LL << 30)) return FA_ERR_INVALID_ARGUMENT;  // the grid
  if (!kept || !aligned4(kept) || !row_stride(kept_b_stride) || !row_stride(kept_h_stride) || !aligned4(base))
    return FA_ERR_INVALID_ARGUMENT;
  if (!k_scale || !v_scale || !k_scale_out || !v_scale_out || !aligned4(k_scale) || !aligned4(v_scale) ||
      !aligned4(k_scale_out) || !aligned4(v_scale_out))
    return FA_ERR_INVALID_ARGUMENT;
  View vk, vv, vko, vvo;
  if (!make_view8(k, k_strides, B, Hkv, Nk, d, &vk) || !make_view8(v, v_strides, B, Hkv, Nk, d, &vv) ||
      !make_view8(k_out, k_out_strides, B, Hkv, Nk_out, d, &vko) ||
      !make_view8(v_out, v_out_strides, B, Hkv, Nk_out, d, &vvo))
    return FA_ERR_INVALID_ARGUMENT;
  if (!injective(B, Hkv, Nk_out, d / 2, vko.s) || !injective(B, Hkv, Nk_out, d / 2, vvo.s))
    return FA_ERR_INVALID_ARGUMENT;
  // all outputs in their inputs' place, or none
  const bool in_place = Nk == Nk_out && same_place(vk, vko) && same_place(vv, vvo) && k_scale == k_scale_out &&
                        v_scale == v_scale_out;
  if (overlap(vko, vvo, B, d / 2)) return FA_ERR_INVALID_ARGUMENT;
  if (in_place ? overlap(vk, vvo, B, d / 2) || overlap(vv, vko, B, d / 2)
               : overlap(vk, vko, B, d / 2) || overlap(vk, vvo, B, d / 2) || overlap(vv, vko, B, d / 2) ||
                     overlap(vv, vvo, B, d / 2))
    return FA_ERR_INVALID_ARGUMENT;
  const Range codes[4] = {range_of(vko, B, d / 2), range_of(vvo, B, d / 2), range_of(vk, B, d / 2),
                          range_of(vv, B, d / 2)};
  const Range lists[2] = {range_of(kept, 4 * (static_cast<long long>(B - 1) * kept_b_stride +
                                              static_cast<long long>(Hkv - 1) * kept_h_stride + M)),
                          range_of(base, 4ll * B)};
  const Range so[2] = {scales_of(k_scale_out, B, Hkv, Nk_out, block), scales_of(v_scale_out, B, Hkv, Nk_out, block)};
  const Range si[2] = {scales_of(k_scale, B, Hkv, Nk, block), scales_of(v_scale, B, Hkv, Nk, block)};
  if (meet(so[0], so[1])) return FA_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < 2; ++i) {
    for (int x = 0; x < 2; ++x) {
      if (meet(codes[i], lists[x]) || meet(so[i], lists[x]) || meet(codes[i], so[x]) || meet(codes[i], si[x]) ||
          meet(codes[2 + i], so[x]))
        return FA_ERR_INVALID_ARGUMENT;
      if (!(in_place && i == x) && meet(si[i], so[x])) return FA_ERR_INVALID_ARGUMENT;
    }
  }
  Compact8Params p{};
  p.k = static_cast<const uint8_t *>(k);
  p.v = static_cast<const uint8_t *>(v);
  p.ko = static_cast<uint8_t *>(k_out);
  p.vo = static_cast<uint8_t *>(v_out);
  p.ks = k_scale;
  p.vs = v_scale;
  p.kso = k_scale_out;
  p.vso = v_scale_out;
  p.sk = bytes(vk);
  p.sv = bytes(vv);
  p.sko = bytes(vko);
  p.svo = bytes(vvo);
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
  p.block_log2 = log2_of(block);
  p.blocks = blocks_of(Nk, block);
  p.blocks_out = blocks_of(Nk_out, block);
  p.in_place = in_place ? 1 : 0;
  return launch_compact8(p, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_tree_verify(const int *parents, int64_t parents_stride, const int *tokens, int64_t tokens_stride,
                           const float *target, int64_t target_b_stride, int64_t target_n_stride, const float *draft,
                           int64_t draft_b_stride, int64_t draft_n_stride, const float *uniforms,
                           int64_t uniforms_stride, int *accepted, int *counts, int *next_token, int B, int Nt, int V,
                           cudaStream_t stream) {
  if (B < 1 || B > kMaxHeads || Nt < 1 || Nt > kTreeMaxNodes || V < 1 || V > kMaxRows) return FA_ERR_INVALID_ARGUMENT;
  if (!parents || !tokens || !target || !uniforms || !accepted || !counts || !next_token || !aligned4(parents) ||
      !aligned4(tokens) || !aligned4(target) || !aligned4(draft) || !aligned4(uniforms) || !aligned4(accepted) ||
      !aligned4(counts) || !aligned4(next_token))
    return FA_ERR_INVALID_ARGUMENT;
  if (!row_stride(parents_stride) || !row_stride(tokens_stride) || !row_stride(uniforms_stride) ||
      !row_stride(target_b_stride) || !row_stride(target_n_stride) || !row_stride(draft_b_stride) ||
      !row_stride(draft_n_stride))
    return FA_ERR_INVALID_ARGUMENT;
  const long long rows = B - 1, nodes = Nt - 1;
  const Range ins[5] = {range_of(parents, 4 * (rows * parents_stride + Nt)),
                        range_of(tokens, 4 * (rows * tokens_stride + Nt)),
                        range_of(uniforms, 4 * (rows * uniforms_stride + Nt)),
                        range_of(target, 4 * (rows * target_b_stride + nodes * target_n_stride + V)),
                        range_of(draft, draft ? 4 * (rows * draft_b_stride + nodes * draft_n_stride + V) : 0)};
  const Range outs[3] = {range_of(accepted, 4ll * B * Nt), range_of(counts, 4ll * B), range_of(next_token, 4ll * B)};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 5; ++i)
      if (meet(outs[o], ins[i])) return FA_ERR_INVALID_ARGUMENT;
    for (int x = o + 1; x < 3; ++x)
      if (meet(outs[o], outs[x])) return FA_ERR_INVALID_ARGUMENT;
  }
  VerifyParams p{};
  p.parents = parents;
  p.tokens = tokens;
  p.par_b = parents_stride;
  p.tok_b = tokens_stride;
  p.target = target;
  p.draft = draft;
  p.tb = target_b_stride;
  p.tn = target_n_stride;
  p.db = draft_b_stride;
  p.dn = draft_n_stride;
  p.uniforms = uniforms;
  p.uni_b = uniforms_stride;
  p.accepted = accepted;
  p.counts = counts;
  p.next = next_token;
  p.B = B;
  p.Nt = Nt;
  p.V = V;
  return launch_verify(p, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
