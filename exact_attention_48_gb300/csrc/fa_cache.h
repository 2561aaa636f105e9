// fa_cache.h -- parameter blocks and launchers of the operators around the
// key/value cache (rotary positions, drafted-tree attention, key weights,
// eviction).  Not part of the ABI.
#pragma once

#include "fa_internal.h"

namespace fa {

// Rotary positions.  The row (b, n) of every head of up to three tensors:
// heads [0, H) are q, [H, H + Hkv) are k, [H + Hkv, H + 2 Hkv) are v (append
// form only, copied).  In the append form k and v rows go to cache row
// cache_len[b] - N + n and are skipped where that row lies outside [0, Nk).
struct RopeParams {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *qo, *ko, *vo;
  Strides sq, sk, sv, sqo, sko, svo;
  const int *positions;       // [B] rows of N with stride pos_b, or null
  long long pos_b;
  const float *inv_freq;      // [rot / 2] radians per position
  const int *cache_len;       // append form: [B]; else null
  int B, H, Hkv, N, Nk, d, rot;
  float factor;
  float sign;                 // +1 forward, -1 backward (the transposed rotation)
  int heads;                  // H + Hkv (+ Hkv)
  int tokens;                 // tokens of a CTA, a power of two up to 8
  int head_groups;            // CTAs along the head axis
};
cudaError_t launch_rope(bool interleaved, const RopeParams &p, cudaStream_t stream);

// Attention of a tree of Nt drafted tokens per sequence over a cache.  The G
// query heads of a cache head are cut into row tiles of `gpt` whole heads
// (gpt * Nt <= 128 rows); a CTA works on one row tile (`split`: its two
// softmax warpgroups take alternate key tiles) or on two.  The 128-key tiles
// of all (b, hk) units, one after the other, are cut into `ranges` equal
// runs; CTA x takes run x / groups for row tiles 2 * (x % groups) and + 1.
// A unit that ends up in several runs leaves a partial result for each.
struct TreeParams {
  __nv_bfloat16 *o;
  float *lse;                 // [B, H, Nt] contiguous
  Strides so;
  const int *parents;         // [B] rows of Nt with stride par_b
  long long par_b;
  const int *cache_len;       // [B] or null
  int *status;
  float *part_o;              // [2 * ctas][d][slot_rows], normalised
  float *part_lse;            // [2 * ctas][slot_rows], log2 units; +inf marks padding
  int4 *cuts;                 // units cut by a run's end: (b, hk, first run, last run), b = -1: none.  An entry
  int cuts_by_unit;           // per unit, or, where those are more, per run that a cut unit starts in
  int B, H, Hkv, G, Nt, Nk, d;
  int gpt, row_tiles, groups, ranges, split;
  int whole;                  // runs end at units' ends: no partial results
  float scale_log2;
  int neg;
};

// How a call is cut up: a function of the shape alone.
struct TreePlan {
  int gpt, row_tiles, groups, ranges, split, whole;
  bool merge;                 // some unit may end up in several runs
  size_t part_rows;           // rows of partial results
};
TreePlan plan_tree(int B, int H, int Hkv, int Nt, int Nk);

// tq: q with boxes of Nt rows x gpt heads.
cudaError_t launch_tree(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const TreeParams &p,
                        bool merge, cudaStream_t stream);

// Accumulated attention weight per key.  A unit is a block of 256 keys of one
// cache head.  Up to 64 query rows of the head's group are one column tile;
// more come in tiles of up to 128: whole heads packed together (`gpt` heads of
// Nq rows) or, for Nq > 128, 128 rows of one head.  With splits > 1 each unit's
// tiles are dealt to that many units whose partial sums a second kernel adds.
struct KeyWeightParams {
  const float *lse;           // [B, H, Nq] contiguous
  const float *w_in;          // [B, Hkv, Nk] or null
  float *w;
  float *part;                // [splits][B, Hkv, Nk] (splits > 1)
  const int *cache_len;       // [B] or null
  int *status;
  int B, H, Hkv, G, Nq, Nk, causal;
  int gpt, tiles_per_head, head_groups;  // tiles of a head group; groups of gpt heads
  int splits;
  int window;                 // cache heads worked on at a time
  uint32_t units;             // B * Hkv * ceil(Nk / 256) * splits, below 2^31
  float scale_log2;
};

struct KeyWeightPlan {
  int cols;                   // columns of a tile: 16, 32, 64 or 128
  int box_rows, gpt, tiles_per_head, head_groups, splits, window;
};
KeyWeightPlan plan_key_weights(int B, int H, int Hkv, int Nq, int Nk, int d);

// tq: q with boxes of box_rows rows x gpt heads; tk: k with boxes of 128 rows,
// 256 when cols is 128.
cudaError_t launch_key_weights(int d, int cols, const CUtensorMap &tq, const CUtensorMap &tk,
                               const KeyWeightParams &p, int sms, cudaStream_t stream);

// Rows to keep of each cache: ascending row numbers, -1 behind them.
struct SelectParams {
  const float *w;             // [B, Hkv, Nk]
  const int *cache_len;       // [B] or null
  int *kept;                  // [B, Hkv, keep]
  int *new_len;               // [B]
  int B, Hkv, Nk, keep, first, recent;
};
cudaError_t launch_cache_select(const SelectParams &p, cudaStream_t stream);

// Rows moved inside (or out of) a cache.
struct CompactParams {
  const __nv_bfloat16 *k, *v;
  const float *w;             // [B, Hkv, Nk] or null
  __nv_bfloat16 *ko, *vo;
  float *wo;                  // [B, Hkv, Nout] or null
  Strides sk, sv, sko, svo;
  const int *kept;            // row lists of M entries, strides kept_b and kept_h
  long long kept_b, kept_h;
  const int *base;            // [B] or null
  int B, Hkv, Nk, Nout, M, d;
  int in_place;
};
cudaError_t launch_cache_compact(const CompactParams &p, cudaStream_t stream);

// Valid rows of the cache of batch entry b, clamped into [0, Nk].
__device__ inline int cache_rows(const int *cache_len, int b, int Nk) {
  if (!cache_len) return Nk;
  const int n = cache_len[b];
  return n < 0 ? 0 : (n > Nk ? Nk : n);
}

}  // namespace fa
