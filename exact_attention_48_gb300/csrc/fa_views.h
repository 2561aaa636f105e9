// fa_views.h -- argument checks that the entry points around the key/value cache
// share: views with their strides, memory ranges, workspaces, sizes.  Host side.
// Not part of the ABI.
#pragma once

#include <cmath>
#include <cstdint>

#include "fa_host.h"

namespace fa {

constexpr int kMaxRows = 1 << 30;       // rows of a cache, tokens of a call
constexpr int kMaxHeads = (1 << 24) - 1;  // B * H, and B * Hkv

// A memory range of an argument.
struct Range {
  uintptr_t lo, hi;
};
inline Range range_of(const void *p, long long bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, p ? lo + static_cast<uintptr_t>(bytes) : lo};
}
inline Range range_of(const void *p, int B, int H, int N, int d, const Strides &s) {
  Range r;
  span(p, B, H, N, d, s, &r.lo, &r.hi);
  return r;
}
inline bool meet(const Range &a, const Range &b) { return spans_overlap(a.lo, a.hi, b.lo, b.hi); }

// A stride of an int32 argument: up to a terabyte's elements, as other strides
// (products with it stay within 64 bits).
inline bool row_stride(int64_t s) { return s >= 0 && s < (1LL << 39); }

inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A bf16 [B, H, N, d] argument with its strides.
struct View {
  const void *p;
  int H, N;
  Strides s;
};

inline bool make_view(const void *p, const int64_t *strides, int B, int H, int N, int d, View *v) {
  if (!p || !aligned16(p)) return false;
  v->p = p;
  v->H = H;
  v->N = N;
  return normalise(strides, B, H, N, d, &v->s);
}
inline bool overlap(const View &a, const View &b, int B, int d) {
  return may_overlap(a.p, a.s, a.H, a.N, b.p, b.s, b.H, b.N, B, d);
}
inline bool same_place(const View &a, const View &b) {
  return a.p == b.p && a.s.b == b.s.b && a.s.h == b.s.h && a.s.n == b.s.n;
}
inline Range range_of(const View &v, int B, int d) { return range_of(v.p, B, v.H, v.N, d, v.s); }
inline const __nv_bfloat16 *in(const View &v) { return static_cast<const __nv_bfloat16 *>(v.p); }
inline __nv_bfloat16 *out(const View &v) { return const_cast<__nv_bfloat16 *>(in(v)); }

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

inline fa_status_t check_d(int d) {
  if (d == 64 || d == 128) return FA_OK;
  return d < 1 ? FA_ERR_INVALID_ARGUMENT : FA_ERR_UNSUPPORTED;
}

inline fa_status_t check_rope(int B, int H, int Hkv, int N, int d, int rot, int interleaved, float factor) {
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

inline fa_status_t check_cache(int B, int H, int Hkv, int Nk, int d) {
  if (B < 1 || H < 1 || Hkv < 1 || Nk < 1) return FA_ERR_INVALID_ARGUMENT;
  const fa_status_t st = check_d(d);
  if (st != FA_OK) return st;
  if (H % Hkv) return FA_ERR_INVALID_ARGUMENT;
  if (static_cast<long long>(B) * H > kMaxHeads || Nk > kMaxRows) return FA_ERR_INVALID_ARGUMENT;
  return FA_OK;
}

constexpr int kTreeMaxNodes = 128;

inline fa_status_t check_tree(int B, int H, int Hkv, int Nt, int Nk, int d, float scale) {
  const fa_status_t st = check_cache(B, H, Hkv, Nk, d);
  if (st != FA_OK) return st;
  if (Nt < 1 || Nt > kTreeMaxNodes) return FA_ERR_INVALID_ARGUMENT;
  return std::isfinite(scale) ? FA_OK : FA_ERR_INVALID_ARGUMENT;
}

}  // namespace fa
