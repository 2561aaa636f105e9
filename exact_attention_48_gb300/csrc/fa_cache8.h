// fa_cache8.h -- parameter blocks and launchers of the operators on a cache held
// in 8 bits (e4m3 codes, and for each block of rows of a head one power of two
// by which they are scaled), and of the verification of drafted tokens.  Not
// part of the ABI.
#pragma once

#include "fa_internal.h"

namespace fa {

// Attention of the newest rows of each sequence, or of a drafted tree, over an
// 8-bit cache.  The G * Nt query rows of a unit (b, hk), head after head, are
// cut into groups of `rows` rows, one CTA each; the 128-key tiles of all
// units are cut into `ranges` equal runs (fa_runs.cuh).  CTA x takes run
// x / groups for row group x % groups.
struct Tree8Params {
  const __nv_bfloat16 *q;
  __nv_bfloat16 *o;
  float *lse;                 // [B, H, Nt] contiguous
  Strides sq, so;
  const float *k_scale, *v_scale;  // [B, Hkv, blocks]
  const int *parents;         // [B] rows of Nt with stride par_b, or null: a chain
  long long par_b;
  const int *cache_len;       // [B] or null
  int *status;
  float *part_o;              // [2 * ctas][rows][d], normalised
  float *part_lse;            // [2 * ctas][rows], log2 units; +inf marks padding
  int4 *cuts;                 // as in TreeParams
  int cuts_by_unit;
  int B, H, Hkv, G, Nt, Nk, d;
  int block_log2, blocks;     // rows of a scale, scales of a head
  int rows, groups, ranges;
  int whole;                  // runs end at units' ends: no partial results
  float scale_log2;
};

struct Tree8Plan {
  int rows, groups, ranges, whole;
  bool merge;
  size_t part_rows;
};
Tree8Plan plan_tree8(int B, int H, int Hkv, int Nt, int Nk, int d);

// tk, tv: maps of encode_map_rows8 with boxes of 128 rows.
cudaError_t launch_tree8(const CUtensorMap &tk, const CUtensorMap &tv, const Tree8Params &p, bool merge,
                         cudaStream_t stream);
// Its main kernels: groups of 8, 16 or 32 rows, and of 128.
cudaError_t launch_tree8_tc(const CUtensorMap &tk, const CUtensorMap &tv, const Tree8Params &p, cudaStream_t stream);
cudaError_t launch_tree8_rows(const CUtensorMap &tk, const CUtensorMap &tv, const Tree8Params &p, cudaStream_t stream);

// Rotary positions and the append to an 8-bit cache: as RopeParams' append form,
// with codes and scales instead of bf16 rows.
struct Append8Params {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *qo;
  uint8_t *kc, *vc;
  float *ks, *vs;             // [B, Hkv, blocks]
  Strides sq, sk, sv, sqo;    // elements
  Strides skc, svc;           // bytes
  const int *positions;
  long long pos_b;
  const float *inv_freq;
  const int *cache_len;
  int B, H, Hkv, N, Nk, d, rot;
  float factor;
  int block_log2, blocks;
  int per_b;                  // blocks of rows that the N tokens of a sequence may touch
  int slots;                  // tokens of a CTA: min(N, rows of a block) rounded up to a power of two
  int q_groups, kv_groups;    // CTAs along the heads of q, of k and of v
};
cudaError_t launch_append8(bool interleaved, const Append8Params &p, cudaStream_t stream);

// Rows moved inside (or out of) an 8-bit cache.
struct Compact8Params {
  const uint8_t *k, *v;
  uint8_t *ko, *vo;
  const float *ks, *vs;       // [B, Hkv, blocks]
  float *kso, *vso;           // [B, Hkv, blocks_out]
  Strides sk, sv, sko, svo;   // bytes
  const int *kept;
  long long kept_b, kept_h;
  const int *base;            // [B] or null
  int B, Hkv, Nk, Nout, M, d;
  int block_log2, blocks, blocks_out;
  int in_place;
};
cudaError_t launch_compact8(const Compact8Params &p, cudaStream_t stream);

// Drafted tokens verified.
struct VerifyParams {
  const int *parents, *tokens;     // [B] rows of Nt
  long long par_b, tok_b;
  const float *target, *draft;     // [B, Nt, V], V contiguous; draft may be null
  long long tb, tn, db, dn;        // their strides, elements
  const float *uniforms;           // [B] rows of Nt
  long long uni_b;
  int *accepted, *counts, *next;   // [B, Nt], [B], [B]
  int B, Nt, V;
  int ranks;                       // CTAs of a sequence
};
cudaError_t launch_verify(VerifyParams p, cudaStream_t stream);

// ---- device helpers

#ifdef __CUDACC__
// The least power of two, 2^-100 or more, by which values of up to `a` (finite)
// fit e4m3's 448 = 1.75 * 2^8.
__device__ __forceinline__ float least_scale(float a) {
  const uint32_t bits = __float_as_uint(a);
  int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < 27 ? 27 : e;  // 127 - 100
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

// Four codes times r, rounded again (NaN stays NaN).
__device__ __forceinline__ uint32_t rescale_codes(uint32_t w, float r) {
  uint32_t out;
  asm("{\n\t.reg .b16 lo, hi, a, b, c, d;\n\t.reg .b32 x, y;\n\t.reg .f32 fa, fb, fc, fd;\n\t"
      "mov.b32 {lo, hi}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 x, lo;\n\tcvt.rn.f16x2.e4m3x2 y, hi;\n\t"
      "mov.b32 {a, b}, x;\n\tmov.b32 {c, d}, y;\n\t"
      "cvt.f32.f16 fa, a;\n\tcvt.f32.f16 fb, b;\n\tcvt.f32.f16 fc, c;\n\tcvt.f32.f16 fd, d;\n\t"
      "mul.rn.f32 fa, fa, %2;\n\tmul.rn.f32 fb, fb, %2;\n\tmul.rn.f32 fc, fc, %2;\n\tmul.rn.f32 fd, fd, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, fb, fa;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, fd, fc;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(out)
      : "r"(w), "f"(r));
  return out;
}
#endif

}  // namespace fa
