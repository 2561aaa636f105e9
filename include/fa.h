/*
 * fa.h -- C ABI of libfa.so, exact scaled-dot-product attention on one GB300.
 *
 * The method.  Attention O = softmax(Q K^T * scale) V is computed block by
 * block in on-chip memory (lexicon page "FlashAttention" (urworte.de),
 * section "Methodische Grundlagen": "Blockweise Verarbeitung"), with the
 * score, normalisation and weighting steps fused into one pass
 * ("Verschmelzung der Schritte") and the row normalisation kept as a running
 * statistic that corrects earlier partial results when a larger score shows
 * up ("Fortlaufende Normierung").  The backward pass recomputes the scores
 * instead of storing them ("Neuberechnung statt Speicherung").  The result
 * equals the conventional computation up to rounding ("Exaktheit").  The
 * N x N score matrix never reaches device memory, so memory grows linearly
 * in N (page "FlashAttention-2 (DE)" (systems-analysis.info), section
 * "Hintergrund").
 *
 * Conventions shared by every call below.
 *  - Tensors q, k, v, o, dO, dq, dk, dv are bf16, contiguous [B, H, N, d]
 *    (d fastest), except in the *_strided calls, which take any layout
 *    whose d elements are contiguous.  lse is fp32, contiguous [B, H, N].
 *    All pointers are
 *    device pointers owned by the caller, 16-byte aligned, non-null, and
 *    the library keeps none of them after the call returns.  The library
 *    owns only a device status word per device, and for fa_bwd and its
 *    strided and packed forms one side stream and two events per host
 *    thread and device.
 *  - B, H, N >= 1; d is 64 or 128 (FA_ERR_UNSUPPORTED otherwise);
 *    B*H*ceil(N/128) < 2^31 (one backward CTA per head and block of 128
 *    rows must fit a launch grid) and B*H*N*d < 2^39 elements per tensor
 *    (1 TiB of bf16: TMA byte strides stay below 2^40), which admits every
 *    tensor a GPU's memory can hold; element offsets are 64-bit
 *    throughout.
 *  - causal is 0 or 1.  With causal = 1, key j is visible to query i iff
 *    j <= i (square mask, aligned at the top-left).  Fully masked tiles are
 *    skipped.
 *  - scale is any finite float (the usual value is 1/sqrt(d)).
 *  - lse[i] = ln sum_{j visible} exp(scale * q_i . k_j): the natural-log
 *    logsumexp of the SCALED scores.
 *  - Outputs must not overlap inputs.
 *  - Every call is asynchronous on `stream` (0 = the legacy default
 *    stream) and validates all arguments on the host before any CUDA call;
 *    an invalid call launches nothing and returns an error code.
 *  - A kernel whose internal pipeline wait runs past its time limit stops,
 *    records FA_ERR_DEVICE_TIMEOUT in a per-device status word and returns;
 *    fa_device_status() reads and clears it.  Kernels never trap.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#if defined(__GNUC__)
#define FA_API __attribute__((visibility("default")))
#else
#define FA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARGUMENT = 1, /* null/misaligned pointer, bad size, non-finite scale, bad flag */
    FA_ERR_UNSUPPORTED = 2,      /* head dimension other than 64 or 128 */
    FA_ERR_WORKSPACE = 3,        /* caller workspace smaller than fa_bwd_workspace_bytes() */
    FA_ERR_CUDA = 4,             /* a CUDA runtime/driver call or launch failed */
    FA_ERR_DEVICE_TIMEOUT = 5    /* a kernel gave up on a pipeline wait (see fa_device_status) */
} fa_status_t;

/*
 * Forward pass: o = softmax(q k^T * scale) v and lse (see conventions).
 * Page "FlashAttention" (urworte.de), "Methodische Grundlagen": tiling,
 * fused steps and running normalisation; page "FlashAttention-2 (DE)",
 * "Technische Architektur", section 2: the work of one head is spread over
 * the SMs by query block.
 *   q, k, v : inputs  [B, H, N, d] bf16
 *   o       : output  [B, H, N, d] bf16
 *   lse     : output  [B, H, N] fp32
 * Bitwise reproducible from run to run for the same inputs.
 */
FA_API fa_status_t fa_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
                   int B, int H, int N, int d, int causal, float scale,
                   cudaStream_t stream);

/*
 * Bytes of device workspace fa_bwd needs for these sizes: D = rowsum(dO * O)
 * and the logsumexp in log2 units, each fp32 [B, H, Np] with N padded up to
 * Np, the next multiple of 128, each rounded up to 256 bytes.  Linear in N.
 * Returns 0 for sizes fa_bwd would reject.
 */
FA_API size_t fa_bwd_workspace_bytes(int B, int H, int N, int d);

/*
 * Backward pass: gradients of a loss L through o = attention(q, k, v), given
 * dO = dL/do and the lse saved by fa_fwd.  The scores and probabilities are
 * recomputed from q, k and lse; nothing of size N x N is stored (page
 * "FlashAttention" (urworte.de), "Methodische Grundlagen", paragraph
 * "Neuberechnung statt Speicherung").
 *   q, k, v, o, dO : inputs  [B, H, N, d] bf16 (o as written by fa_fwd)
 *   lse            : input   [B, H, N] fp32 (as written by fa_fwd)
 *   dq, dk, dv     : outputs [B, H, N, d] bf16
 *   workspace      : device scratch of at least fa_bwd_workspace_bytes()
 *                    bytes, 256-byte aligned, or NULL to let the library
 *                    take it with cudaMallocAsync/cudaFreeAsync on `stream`.
 * No atomics are used: dq, dk and dv are bitwise reproducible run to run.
 * The dK/dV kernel runs on `stream` and the dQ kernel next to it on a side
 * stream of the library's (one per host thread and device, created on the
 * first call with two events, kept until the process exits); `stream`
 * waits for both before any work enqueued after the call, so the ordering
 * a caller sees is that of a single stream.
 */
FA_API fa_status_t fa_bwd(const void *q, const void *k, const void *v, const void *o,
                   const void *dO, const float *lse, void *dq, void *dk, void *dv,
                   int B, int H, int N, int d, int causal, float scale,
                   void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Strided layouts.  The same two passes on tensors in any layout whose d
 * elements are contiguous: element (b, h, n, c) of a tensor lies at
 *     base + b * strides[0] + h * strides[1] + n * strides[2] + c
 * (strides in elements, int64, one array of three per tensor).  This covers
 * [B, N, H, d] ("BNHD", the layout of many frameworks' projections), the
 * q, k, v slices of one packed [B, N, 3, H, d] projection, and any padded
 * row pitch; the page "FlashAttention-2 (DE)" (systems-analysis.info),
 * section "Anwendung und Integration in das Oekosystem", names the
 * frameworks this is for.  Rules: every stride of a dimension of extent > 1
 * is a positive multiple of 8 elements (16 bytes) below 2^39 (the stride of
 * an extent-1 dimension is ignored); inputs may share memory with each
 * other (a packed projection); each output's elements are all distinct and
 * no output overlaps an input, another output or the workspace (checked on
 * the address ranges spanned).  lse stays contiguous [B, H, N].  Everything
 * else is as in fa_fwd / fa_bwd; with contiguous strides the results are
 * bitwise those of fa_fwd / fa_bwd.
 */
FA_API fa_status_t fa_fwd_strided(const void *q, const int64_t *q_strides, const void *k,
                                  const int64_t *k_strides, const void *v, const int64_t *v_strides,
                                  void *o, const int64_t *o_strides, float *lse, int B, int H, int N,
                                  int d, int causal, float scale, cudaStream_t stream);

FA_API fa_status_t fa_bwd_strided(const void *q, const int64_t *q_strides, const void *k,
                                  const int64_t *k_strides, const void *v, const int64_t *v_strides,
                                  const void *o, const int64_t *o_strides, const void *dO,
                                  const int64_t *dO_strides, const float *lse, void *dq,
                                  const int64_t *dq_strides, void *dk, const int64_t *dk_strides,
                                  void *dv, const int64_t *dv_strides, int B, int H, int N, int d,
                                  int causal, float scale, void *workspace, size_t workspace_bytes,
                                  cudaStream_t stream);

/*
 * Packed variable-length sequences ("varlen").  B sequences of different
 * lengths stored back to back along one row axis of T rows: sequence b is
 * rows [cu_seqlens[b], cu_seqlens[b+1]) of every tensor, and attends only
 * to itself (causal = 1: key j visible to query i iff j <= i, positions
 * counted from the sequence's first row).
 *   q, k, v, o, dO, dq, dk, dv : [T, H, d] bf16 with element strides
 *                    strides[0] between rows and strides[1] between heads
 *                    (d contiguous; same rules as the strided calls)
 *   lse          : [H, T] fp32, contiguous
 *   cu_seqlens   : device array of B + 1 int32 row offsets, 4-byte aligned:
 *                  0 = cu[0] <= cu[1] <= ... <= cu[B] = T, every length
 *                  cu[b+1] - cu[b] at most max_seqlen.  The kernels read it
 *                  on the device, so the host cannot check it; they clamp
 *                  every offset into [0, T] and every length to max_seqlen,
 *                  so a malformed array gives wrong results for the
 *                  sequences it describes, never an access outside the
 *                  tensors.  Zero-length sequences are allowed.
 *   max_seqlen   : the longest sequence (sizes the launch and the workspace)
 * The backward workspace is fa_bwd_workspace_bytes(B, H, max_seqlen, d).
 * The pages describe attention per sequence; packing several sequences into
 * one call is this library's reading of the framework integration that the
 * page "FlashAttention-2 (DE)", section "Anwendung und Integration in das
 * Oekosystem", names.
 */
FA_API fa_status_t fa_fwd_varlen(const void *q, const int64_t *q_strides, const void *k,
                                 const int64_t *k_strides, const void *v, const int64_t *v_strides,
                                 void *o, const int64_t *o_strides, float *lse,
                                 const int *cu_seqlens, int B, int H, int T, int max_seqlen, int d,
                                 int causal, float scale, cudaStream_t stream);

FA_API fa_status_t fa_bwd_varlen(const void *q, const int64_t *q_strides, const void *k,
                                 const int64_t *k_strides, const void *v, const int64_t *v_strides,
                                 const void *o, const int64_t *o_strides, const void *dO,
                                 const int64_t *dO_strides, const float *lse, void *dq,
                                 const int64_t *dq_strides, void *dk, const int64_t *dk_strides,
                                 void *dv, const int64_t *dv_strides, const int *cu_seqlens, int B,
                                 int H, int T, int max_seqlen, int d, int causal, float scale,
                                 void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * FP8 forward: the forward pass with Q, K, V given as e4m3 codes (OCP FP8
 * E4M3: 1 sign, 4 exponent bits with bias 7, 3 mantissa bits, no
 * infinities, 0x7F/0xFF NaN) and one fp32 scale per tensor: element value =
 * decoded code * q_scale (k_scale, v_scale).  Both products run on the
 * tensor core's 8-bit path.  The page "FlashAttention-2 (DE)", section
 * "Vergleich mit nachfolgenden Versionen" / "FlashAttention-3", names
 * low-precision FP8 as a FlashAttention-3 addition without a formula; what
 * this call computes, per row i (log2 units, x_ij = scale * log2(e) *
 * q_i . k_j on the decoded, scaled values, masked keys excluded):
 *   M_i = ceil(max_j x_ij);  w_ij = e4m3 rounding (nearest, ties to even)
 *   of 2^(x_ij - M_i + 8), at most 256;
 *   o_i = sum_j w_ij v_j / sum_j w_ij  (bf16);
 *   lse_i = ln 2 * (M_i - 8 + log2 sum_j 2^(x_ij - M_i + 8))  (fp32, exact
 *   logsumexp of the scaled scores, as in fa_fwd).
 * The weights are what an FP8 tensor-core product of P and V can apply; the
 * integer M_i makes them independent of how the keys are tiled (outside
 * e4m3's subnormal range, 2^(x - M + 8) < 2^-6, where the rounding grid of
 * a tiled pass may be finer).
 *   q8, k8, v8 : [B, H, N, d] e4m3 codes (1 byte each), contiguous
 *   o          : [B, H, N, d] bf16, lse : [B, H, N] fp32, contiguous
 *   d must be 128 (FA_ERR_UNSUPPORTED otherwise); the tensor scales must
 *   be finite; other conventions as above.
 */
FA_API fa_status_t fa_fwd_fp8(const void *q8, const void *k8, const void *v8, float q_scale,
                              float k_scale, float v_scale, void *o, float *lse, int B, int H, int N,
                              int d, int causal, float scale, cudaStream_t stream);

/*
 * Decode forward: Nq new query rows per (batch entry, head) against a cache
 * of keys and values, as in token-by-token generation.  The computation is
 * the forward pass above (o and lse, same definition and scale), with
 * rectangular shapes: per (b, h) the query rows are q[b, h, 0..Nq) and the
 * keys/values are the first len_b rows of the cache, len_b = cache_seqlens[b]
 * (all Nk rows when cache_seqlens is NULL).  The query rows are the LAST Nq
 * positions of the sequence: with causal = 1, query i sees key j iff
 * j <= len_b - Nq + i (mask aligned at the bottom-right; for Nq = 1 it is no
 * restriction); with causal = 0 it sees every key j < len_b.  A query row
 * that sees no key (len_b = 0, or causal with len_b - Nq + i < 0) gets
 * o = 0 and lse = -inf.
 *   q    : [B, H, Nq, d] bf16, element strides q_strides[3] (b, h, row)
 *   k, v : [B, H, Nk, d] bf16, element strides k_strides / v_strides (a
 *          cache stored [B, Nk, H, d] is strides {Nk*H*d, d, H*d})
 *   o    : [B, H, Nq, d] bf16, strides o_strides; must not overlap anything
 *   lse  : [B, H, Nq] fp32, contiguous
 *   cache_seqlens : NULL, or a device array of B int32 (4-byte aligned);
 *          the kernel clamps each value into [0, Nk], so a bad value gives a
 *          wrong result for its batch entry, never an access outside k, v
 *   1 <= Nq <= 8, Nk >= 1 (Nk <= 2^30), d 64 or 128, B*H < 2^24; strides
 *   follow the rules of the *_strided calls.
 *   workspace : device scratch of fa_decode_workspace_bytes(B, H, Nq, Nk, d)
 *          bytes (256-byte aligned; that size may be 0), or NULL to let the
 *          call take it with cudaMallocAsync/cudaFreeAsync on `stream`.
 * Work is split over the keys: each 128-key tile chunk of a head gives a
 * partial result normalised over its own keys and its logsumexp, and the
 * partials are merged with the same running-maximum correction the tiled
 * pass uses between key blocks; the chunk size depends on the shape only,
 * so the result is bitwise reproducible for the same inputs.  The
 * glossary page "FlashAttention" (blog.brdg.mn) places the method in model
 * serving next to the block-wise management of the key/value cache
 * (sections "Der Engpass ist der Weg zum Speicher, nicht das Rechnen" and
 * "Wo es verwechselt wird"); decoding against that cache is this call.
 * The cache's block management itself is not part of the library.
 */
FA_API size_t fa_decode_workspace_bytes(int B, int H, int Nq, int Nk, int d);

FA_API fa_status_t fa_fwd_decode(const void *q, const int64_t *q_strides, const void *k,
                                 const int64_t *k_strides, const void *v, const int64_t *v_strides,
                                 void *o, const int64_t *o_strides, float *lse,
                                 const int *cache_seqlens, int B, int H, int Nq, int Nk, int d,
                                 int causal, float scale, void *workspace, size_t workspace_bytes,
                                 cudaStream_t stream);

/*
 * Operators around the key/value cache: rotary positions, attention for a
 * tree of drafted tokens, the accumulated attention weight of each cached
 * key, and eviction by it.  The glossary page "FlashAttention"
 * (blog.brdg.mn) places the method in model serving next to the management
 * of that cache; the pages describe none of these calls, their definitions
 * are this library's.
 *
 * Conventions they share, beside those at the top of this file: tensors are
 * bf16 with element strides as in the *_strided calls; a cache is
 * [B, Hkv, Nk, d] with cache_seqlens as in fa_fwd_decode (int32 [B], 4-byte
 * aligned, NULL for all Nk rows; it counts the new rows; clamped into
 * [0, Nk]); queries may have H = G * Hkv heads, G of them sharing a cache
 * head (query head h uses cache head h / G).  B * H and B * Hkv are below
 * 2^24; Nk, the query rows and the tokens of a call (B * N) are at most
 * 2^30.  Values behind a sequence's last row are read as memory but never
 * used, whatever they are (infinities and NaN included), and rows that no
 * argument names are left as they were.  Every call may be captured into a
 * graph.
 */

/*
 * Rotary positions.  In the first `rot` columns of every row, pair i turns
 * by the angle a = position * inv_freq[i] and is scaled by `factor`:
 *     y1 = factor * (x1 cos a - x2 sin a),  y2 = factor * (x2 cos a + x1 sin a)
 * with pairs (i, i + rot/2), or (2i, 2i + 1) if interleaved = 1; the columns
 * past rot are copied.  Computed in fp32 and rounded once; the angle is taken
 * modulo a turn in 64-bit fixed point before it is rounded to fp32, within
 * 2^-25 of a turn for any 32-bit position and frequencies of up to 128 radians
 * per position.
 *   q, k           : inputs  [B, H, N, d] and [B, Hkv, N, d]; k and k_out are
 *                    NULL and Hkv = 0 when there is only q
 *   q_out, k_out   : outputs of the same shapes; each is its own input
 *                    (same pointer and strides: in place) or shares no
 *                    element with any argument
 *   positions      : int32, row (b, n) at positions[b * positions_stride + n]
 *                    (stride 0: shared by the batch), any value; NULL: n
 *   inv_freq       : fp32 [rot / 2], radians per position, finite
 *   rot            : a multiple of 16 up to d (FA_ERR_UNSUPPORTED otherwise)
 * fa_rope_bwd is the gradient: given dL/dq_out and dL/dk_out (same
 * positions, frequencies and factor) it writes dL/dq and dL/dk, the same
 * rotation by -a; the copied columns' gradients are copied.
 */
FA_API fa_status_t fa_rope(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                           void *q_out, const int64_t *q_out_strides, void *k_out, const int64_t *k_out_strides,
                           const int *positions, int64_t positions_stride, const float *inv_freq, int B, int H,
                           int Hkv, int N, int d, int rot, int interleaved, float factor, cudaStream_t stream);

FA_API fa_status_t fa_rope_bwd(const void *dq_out, const int64_t *dq_out_strides, const void *dk_out,
                               const int64_t *dk_out_strides, void *dq, const int64_t *dq_strides, void *dk,
                               const int64_t *dk_strides, const int *positions, int64_t positions_stride,
                               const float *inv_freq, int B, int H, int Hkv, int N, int d, int rot, int interleaved,
                               float factor, cudaStream_t stream);

/*
 * Rotary positions and the cache's new rows in one launch: q is rotated into
 * q_out (which may be q), k is rotated into k_cache and v copied into
 * v_cache.  The N tokens are the LAST N rows of the sequence, as in
 * fa_fwd_decode: token n of batch entry b goes to cache row
 * cache_seqlens[b] - N + n.  A row outside [0, Nk) is not written (here
 * cache_seqlens is not clamped).  positions NULL: the cache row; a drafted
 * tree or a cache that rows were evicted from passes its own.
 *   q [B, H, N, d]; k, v [B, Hkv, N, d]; k_cache, v_cache [B, Hkv, Nk, d];
 *   cache_seqlens is required.  No output shares an element with an input
 *   (but q_out with q) or with another output.
 */
FA_API fa_status_t fa_rope_append(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                                  const void *v, const int64_t *v_strides, void *q_out, const int64_t *q_out_strides,
                                  void *k_cache, const int64_t *k_cache_strides, void *v_cache,
                                  const int64_t *v_cache_strides, const int *cache_seqlens, const int *positions,
                                  int64_t positions_stride, const float *inv_freq, int B, int H, int Hkv, int N,
                                  int Nk, int d, int rot, int interleaved, float factor, cudaStream_t stream);

/* How fa_rope_frequencies scales for contexts longer than the training length. */
enum {
    FA_ROPE_PLAIN = 0,    /* inv_freq[i] = base^(-2i / rot) */
    FA_ROPE_LINEAR = 1,   /* positions divided: inv_freq[i] / factor */
    FA_ROPE_BASE = 2,     /* base enlarged: base * factor^(rot / (rot - 2)) */
    FA_ROPE_BY_PARTS = 3  /* see below */
};

/*
 * Host function: fills inv_freq (host memory, rot / 2 values) and
 * *factor_out (the `factor` of the calls above).  FA_ROPE_BY_PARTS keeps the
 * frequencies that make fast_turns turns or more over original_len
 * positions, divides those that make slow_turns or fewer by `factor`, blends
 * linearly in the turns between, and sets *factor_out = 1 + 0.1 ln factor;
 * the other schemes set 1.  factor >= 1 (unused by FA_ROPE_PLAIN),
 * base > 1, rot even (above 2 for FA_ROPE_BASE); original_len >= 1 and
 * fast_turns > slow_turns > 0 are used by FA_ROPE_BY_PARTS only.
 */
FA_API fa_status_t fa_rope_frequencies(float *inv_freq, float *factor_out, int rot, double base, int scaling,
                                       double factor, int original_len, double fast_turns, double slow_turns);

/*
 * Attention of a tree of Nt drafted tokens per sequence over its cache.  The
 * tree's nodes are the LAST Nt rows of the sequence (node i is cache row
 * len_b - Nt + i, its key and value already stored); parents[b, i] is the
 * node that node i follows, parents[b, i] < i, or -1 for the last row before
 * the tree.  Query row i sees every row before the tree, its own row and
 * its ancestors' rows:
 *     o = softmax(scale * q k^T) v and lse over the rows it sees.
 * A node whose parent is not in [-1, i), or whose cache row would be
 * negative (len_b < Nt), is padding, and so is every node below it: its
 * result is o = 0, lse = -inf, and no row sees it, whatever its cache row
 * holds.  (A value row that some node sees must be finite: one that is not
 * may reach the results of the nodes that do not see it.)
 * A score of -inf weighs nothing (a row with no other gets o = 0,
 * lse = -inf); a NaN, or a score of +inf, makes its own row NaN.
 *   q, o   : [B, H, Nt, d]; k, v : [B, Hkv, Nk, d]; lse : fp32 [B, H, Nt]
 *   parents: int32, node (b, i) at parents[b * parents_stride + i] (stride
 *            0: one tree for the whole batch)
 *   1 <= Nt <= 128; Nt = 1 with parent -1 is a decode step with grouped
 *   heads, a chain (parent i - 1) is the causal decode of several rows.
 *   workspace: fa_tree_workspace_bytes() bytes (may be 0), 256-byte
 *   aligned, or NULL to take it with cudaMallocAsync on `stream`.
 * Work is split over the keys; the split depends on the shape and on
 * cache_seqlens only, so results are bitwise reproducible.
 */
FA_API size_t fa_tree_workspace_bytes(int B, int H, int Hkv, int Nt, int Nk, int d);

FA_API fa_status_t fa_fwd_tree(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                               const void *v, const int64_t *v_strides, void *o, const int64_t *o_strides,
                               float *lse, const int *parents, int64_t parents_stride, const int *cache_seqlens,
                               int B, int H, int Hkv, int Nt, int Nk, int d, float scale, void *workspace,
                               size_t workspace_bytes, cudaStream_t stream);

/*
 * Accumulated attention weight of each cached key: for every row j < len_b
 *     weights[b, hk, j] = weights_in[b, hk, j]
 *         + sum over the G heads h of hk and the query rows i that see j of
 *           exp(scale * q[b, h, i] . k[b, hk, j] - lse[b, h, i]),
 * the column sums of an attention matrix, given its logsumexp.  The Nq query
 * rows are the LAST Nq positions: with causal = 1 row i sees j <= len_b - Nq
 * + i, with 0 every j < len_b.  These have to be the rows that lse was taken
 * over: fa_fwd's and fa_fwd_decode's with the same causal; of fa_fwd_tree's,
 * one node's (causal = 0) or a chain's (causal = 1).  The nodes of a tree with
 * branches see neither all rows nor the rows up to their own; call this for
 * the accepted branch, once fa_cache_compact has made it the sequence's next
 * rows, with its nodes' queries and lse and causal = 1 (shorter branches
 * padded in front, lse = -inf).  A query row whose lse is -inf adds nothing,
 * whatever q holds.
 * Rows j >= len_b get weights_in's value.
 *   q : [B, H, Nq, d]; k : [B, Hkv, Nk, d]; lse : fp32 [B, H, Nq]
 *   weights_in : fp32 [B, Hkv, Nk] or NULL (zeros); may be weights itself
 *   weights    : fp32 [B, Hkv, Nk], all of it written
 *   workspace  : fa_key_weights_workspace_bytes() bytes (may be 0), 256-byte
 *   aligned, or NULL to take it with cudaMallocAsync on `stream`.
 * Sums are fp32, in an order that the shape and cache_seqlens fix (no
 * atomics).
 */
FA_API size_t fa_key_weights_workspace_bytes(int B, int H, int Hkv, int Nq, int Nk, int d);

FA_API fa_status_t fa_key_weights(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                                  const float *lse, const float *weights_in, float *weights,
                                  const int *cache_seqlens, int B, int H, int Hkv, int Nq, int Nk, int d, int causal,
                                  float scale, void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Which rows of each cache head to keep.  A sequence of len_b <= keep rows
 * keeps them all.  A longer one keeps its `first` first rows, its `recent`
 * last rows and, of the rows between, the keep - first - recent with the
 * greatest weight (of equal weights the lower row; 0 and -0 are equal; a
 * NaN ranks below every number).
 *   weights    : fp32 [B, Hkv, Nk]
 *   kept       : int32 [B, Hkv, keep]: the kept rows, ascending; -1 behind
 *                them where the sequence is shorter than keep
 *   new_seqlens: int32 [B]: min(len_b, keep); not cache_seqlens itself
 *   0 <= first, recent; first + recent <= keep; 1 <= keep <= Nk
 */
FA_API fa_status_t fa_cache_select(const float *weights, const int *cache_seqlens, int *kept, int *new_seqlens,
                                   int B, int Hkv, int Nk, int keep, int first, int recent, cudaStream_t stream);

/*
 * Moves cache rows together: for every head and every i in [0, M) with
 * kept[i] >= 0, row base_b + i of k_out, v_out (and weights_out) becomes row
 * base_b + kept[i] of k, v (and weights).  A row of either side outside its
 * tensor is skipped.  Rows are moved bit by bit.
 *   k, v         : [B, Hkv, Nk, d]; weights : fp32 [B, Hkv, Nk] or NULL
 *   k_out, v_out : [B, Hkv, Nk_out, d]; weights_out : fp32 [B, Hkv, Nk_out],
 *                  NULL exactly if weights is
 *   kept         : int32, list of (b, h) at kept[b * kept_b_stride + h *
 *                  kept_h_stride] (strides 0: shared), M entries each;
 *                  B * Hkv * ceil(M / 64) < 2^31
 *   base         : int32 [B] or NULL (zeros)
 * Either every output is its input (same pointers and strides, Nk_out = Nk:
 * in place), and then the non-negative entries of a list must ascend
 * strictly and none may be below its place, kept[i] >= i (otherwise rows
 * hold wrong values; no other memory is touched), or no output shares an
 * element with an argument, and then the lists may be in any order and
 * name a row more than once.
 * With fa_cache_select's lists this evicts; with base_b the row before which
 * a drafted tree starts and kept the nodes of the accepted branch, it makes
 * that branch the sequence's next rows.
 * In place, rows behind the last place filled keep what they held, the weights
 * among them: set those to 0 before new rows are appended there and weighed.
 */
FA_API fa_status_t fa_cache_compact(const void *k, const int64_t *k_strides, const void *v,
                                    const int64_t *v_strides, const float *weights, void *k_out,
                                    const int64_t *k_out_strides, void *v_out, const int64_t *v_out_strides,
                                    float *weights_out, const int *kept, int64_t kept_b_stride,
                                    int64_t kept_h_stride, const int *base, int B, int Hkv, int Nk, int Nk_out,
                                    int M, int d, cudaStream_t stream);

/*
 * A cache held in 8 bits.  k and v are e4m3 codes (OCP E4M3, a byte each; NaN
 * but no infinities) [B, Hkv, Nk, d] with element strides that are multiples of
 * 16, and each block of `block` rows of a head has one scale: element (b, h, n, c)
 * stands for code * scale[b, h, n / block], scales fp32, contiguous
 * [B, Hkv, ceil(Nk / block)], powers of two from 2^-100 to 2^120.  block is 16,
 * 32, 64 or 128 (FA_ERR_UNSUPPORTED otherwise); k and v have scales of their own.
 * (e4m3 is a floating type: a scale between two powers of two would gain
 * nothing, and a block is given another one by a shift of its exponents.)  The
 * conventions of the operators around the cache above hold for these calls too.
 * A scale none of whose rows is in use may hold anything; to fa_fwd_tree_fp8 the
 * rows of padding nodes are not.
 */

/*
 * fa_rope_append to a cache held in 8 bits: q is rotated into q_out (which may be
 * q) in bf16; k, rotated in fp32, and v become cache rows, rounded once.  For each
 * block of rows that gets new ones,
 *     need  = the least power of two >= 2^-100 by which the greatest finite
 *             magnitude among its new rows is at most 448,
 *     scale = need, or the greater of need and the present scale if the block
 *             holds rows before the new ones (rows below cache_seqlens[b] - N),
 *     code  = e4m3(x / scale), to the nearest, ties to even; NaN and the
 *             infinities become NaN,
 * and where the scale grew the old rows' codes become e4m3(code * old / new):
 * exact but for codes that fall below e4m3's normal range.  Rows behind the
 * new ones keep their codes.  Other arguments as in fa_rope_append.
 */
FA_API fa_status_t fa_rope_append_fp8(const void *q, const int64_t *q_strides, const void *k,
                                      const int64_t *k_strides, const void *v, const int64_t *v_strides, void *q_out,
                                      const int64_t *q_out_strides, void *k_cache, const int64_t *k_cache_strides,
                                      void *v_cache, const int64_t *v_cache_strides, float *k_scale, float *v_scale,
                                      const int *cache_seqlens, const int *positions, int64_t positions_stride,
                                      const float *inv_freq, int B, int H, int Hkv, int N, int Nk, int d, int rot,
                                      int interleaved, float factor, int block, cudaStream_t stream);

/*
 * fa_fwd_tree over a cache held in 8 bits: q, o bf16, lse fp32, the tree, padding,
 * scores that are not finite and the workspace as there.  parents may be NULL: the
 * last Nt rows are a chain, each of which sees the rows up to its own (Nt = 1: one
 * new token; several: the causal decode).  The products run on the codes, q to
 * 2^-17.8 of a row's greatest magnitude, or of 2^-91 where that is less (exactly,
 * where its values are within 2^9 of that); scores, sums and o are fp32.  A weight is off by at most 2^-9 of itself,
 * or, times its value's scale, 2^-18 of the greatest such product among the 128 rows
 * that it is worked on with; there a value's scale below 2^-100 of the greatest one
 * counts as 2^-100 of it.  o is divided by the sum of the weights as they were before
 * that rounding (fa_fwd_tree's by the sum of the rounded ones).  A row of q that is not finite gives NaN.
 */
FA_API size_t fa_tree_fp8_workspace_bytes(int B, int H, int Hkv, int Nt, int Nk, int d);

FA_API fa_status_t fa_fwd_tree_fp8(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                                   const void *v, const int64_t *v_strides, const float *k_scale,
                                   const float *v_scale, void *o, const int64_t *o_strides, float *lse,
                                   const int *parents, int64_t parents_stride, const int *cache_seqlens, int B, int H,
                                   int Hkv, int Nt, int Nk, int d, int block, float scale, void *workspace,
                                   size_t workspace_bytes, cudaStream_t stream);

/*
 * fa_cache_compact of a cache held in 8 bits: for every head and every i in
 * [0, M) with kept[i] >= 0, row base_b + i of k_out, v_out becomes row base_b +
 * kept[i] of k, v.  A block of the output that rows move to gets the greatest
 * scale of the blocks they come from; rows of it before base_b are kept as well,
 * and its present scale counts with them (so out of place they, and that scale,
 * have to be there).  A row whose own scale was smaller has its codes rounded
 * to the new one, the others move bit by bit.  Rows of a written block that
 * are neither lose their values; blocks that no row moves to stay as they are.
 *   k_scale, v_scale         : [B, Hkv, ceil(Nk / block)]
 *   k_scale_out, v_scale_out : [B, Hkv, ceil(Nk_out / block)]
 *   B * Hkv * (ceil(M / 128) + 1) < 2^30
 * Either every output is its input (same pointers and strides, Nk_out = Nk: in
 * place; the lists must then ascend as for fa_cache_compact), or no output shares
 * an element with an argument.
 */
FA_API fa_status_t fa_cache_compact_fp8(const void *k, const int64_t *k_strides, const void *v,
                                        const int64_t *v_strides, const float *k_scale, const float *v_scale,
                                        void *k_out, const int64_t *k_out_strides, void *v_out,
                                        const int64_t *v_out_strides, float *k_scale_out, float *v_scale_out,
                                        const int *kept, int64_t kept_b_stride, int64_t kept_h_stride,
                                        const int *base, int B, int Hkv, int Nk, int Nk_out, int M, int d, int block,
                                        cudaStream_t stream);

/*
 * Verification of drafted tokens against the target's probabilities, from given
 * random numbers.  The tree is fa_fwd_tree's, and node 0 is its root (the last
 * token that is decided; parent -1).  target[b, n] is the target's distribution
 * at node n and draft[b, n] the one that n's children were drawn from, each one by
 * itself.  From the root on, a node's children are tried in ascending order: with
 *     R = target[b, n], S = 1
 * before the first, child i with token x = tokens[b, i] is accepted, and the walk
 * goes on from it, if
 *     uniforms[b, i] * draft[b, n, x] * S < R[x];
 * otherwise R becomes max(R - S * draft[b, n], 0) and S the sum of R.  Where no
 * child is left, the next token is the least y with
 *     R[0] + .. + R[y] > uniforms[b, 0] * (R[0] + .. + R[V - 1]).
 * Should R be zero there (rounding, or a token that its draft's row gives no
 * probability, can make it so), target[b, n] takes its place; -1 if that is zero
 * too.  The accepted tokens and the next one are then distributed as the
 * target's.  draft NULL: each child was chosen for certain (its token's draft
 * probability is 1 and the others' 0), as by a draft of likeliest tokens.
 *   parents, tokens, uniforms: node (b, i) at [b * stride + i]; a node whose
 *               parent is not in [0, i) or whose token is not in [0, V) is never
 *               tried; with parents[b, 0] != -1 the sequence is padding
 *   uniforms  : fp32, in [0, 1)
 *   target, draft : fp32, finite and not negative, row (b, n) at
 *               b * b_stride + n * n_stride, V contiguous values (4-byte aligned)
 *   accepted  : int32 [B, Nt]: the accepted nodes from the root on, -1 behind
 *               them: fa_cache_compact's list (base_b = len_b - Nt)
 *   counts    : int32 [B], how many; 0 for padding
 *   next_token: int32 [B]; -1 for padding
 *   1 <= Nt <= 128; V <= 2^30
 * Sums are taken to about 44 bits, so that a number decides as in the formulas.
 */
FA_API fa_status_t fa_tree_verify(const int *parents, int64_t parents_stride, const int *tokens,
                                  int64_t tokens_stride, const float *target, int64_t target_b_stride,
                                  int64_t target_n_stride, const float *draft, int64_t draft_b_stride,
                                  int64_t draft_n_stride, const float *uniforms, int64_t uniforms_stride,
                                  int *accepted, int *counts, int *next_token, int B, int Nt, int V,
                                  cudaStream_t stream);

/*
 * Size in bytes of the fixed device array that fa_bwd_noalloc uses as its
 * scratch (8 MiB).  Every GPU that loads the library holds this array until
 * the process exits.  It covers B * H * Np <= 1,048,576 padded rows, where
 * Np is N rounded up to a multiple of 128 (for example B*H = 32 heads of
 * N = 32768).
 */
#define FA_NOALLOC_SCRATCH_BYTES (8u << 20)

/*
 * Backward pass for callers that must not allocate device memory: the same
 * computation, arguments, layouts and results as fa_bwd, but with no
 * workspace argument and no allocation of any kind (no cudaMalloc,
 * cudaMallocAsync or cudaFree, and no side stream: its kernels run one
 * after the other on `stream`).  Its scratch lives in a fixed array of the
 * library (FA_NOALLOC_SCRATCH_BYTES); calls that would need more return
 * FA_ERR_WORKSPACE without launching anything.
 *
 * Who needs it: callers whose device memory is owned by someone else (a
 * framework's memory manager that must see every allocation) or planned up
 * front (a process that must not allocate once it runs), which can neither
 * pass fa_bwd a workspace nor let it take one.
 *
 * Set-up and sharing: every call looks up the array's device address in
 * the current context (cudaGetSymbolAddress, a host-side query; the first
 * lookup in a process may load the library's device code).  All calls share
 * the one array and it keeps the last
 * call's contents; nothing in it needs to start at zero.
 * Calls whose work overlaps on the GPU (other streams or host threads on
 * the same device) race on it, so the caller must order them.
 *
 * The pages describe no counterpart of this entry point.
 */
FA_API fa_status_t fa_bwd_noalloc(const void *q, const void *k, const void *v, const void *o,
                                  const void *dO, const float *lse, void *dq, void *dk, void *dv,
                                  int B, int H, int N, int d, int causal, float scale,
                                  cudaStream_t stream);

/*
 * Synchronises `stream`, then returns the status word the kernels of the
 * current device recorded (FA_OK or FA_ERR_DEVICE_TIMEOUT) and resets it to
 * FA_OK.  Returns FA_ERR_CUDA if the synchronisation itself fails.
 */
FA_API fa_status_t fa_device_status(cudaStream_t stream);

/*
 * Diagnostic: the wait site (a small positive integer naming the pipeline
 * barrier) of the first timeout recorded on the current device since the
 * status word was last cleared, 0 if none, -1 if it cannot be read.  Call it
 * before fa_device_status(), which clears the record.
 */
FA_API int fa_debug_last_wait_site(void);

/*
 * Diagnostic timing hook: the next fa_bwd call made by this host thread
 * records, on its stream, `start` right before the launch of its dK/dV
 * kernel, `mid` between that kernel and its dQ kernel, and `stop` right
 * after the dQ kernel, so both kernels can be timed with
 * cudaEventElapsedTime (that call runs the two kernels one after the
 * other on its stream, not side by side).  The events are created and owned by the caller;
 * the hook is used once and then cleared.  Returns FA_ERR_INVALID_ARGUMENT
 * if any event is NULL.
 */
FA_API fa_status_t fa_debug_time_next_bwd(cudaEvent_t start, cudaEvent_t mid, cudaEvent_t stop);

/* A static, NUL-terminated description of a status code. */
FA_API const char *fa_status_string(fa_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
