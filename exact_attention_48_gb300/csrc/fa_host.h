// fa_host.h -- host-side helpers of the entry points (argument checks, tensor
// maps, the device status word).  Defined in fa_api.cu.  Not part of the ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include "fa_internal.h"

namespace fa {

// A [B, H, N, d] bf16 tensor with element strides s (d contiguous) viewed
// as 4-D (d, N, H, B); one box is 64 columns (128 bytes, the swizzle span) x
// box_rows rows x box_heads heads, stored head after head without a gap.
// Rows past N and heads past H read as 0.
bool encode_map(CUtensorMap *map, const void *base, int B, int H, int N, int d, const Strides &s,
                unsigned box_rows = 128, unsigned box_heads = 1);

// A caller's strides made usable: the stride of an extent-1 dimension is
// never used, so it is replaced by a harmless valid value; then every
// stride must be positive and a multiple of 8 elements (16 bytes: TMA and
// the 16-byte row accesses).  False if the layout is not supported.
bool normalise(const int64_t *in, int B, int H, int N, int d, Strides *out);

// Address span [lo, hi) of the elements of a strided tensor.
void span(const void *base, int B, int H, int N, int d, const Strides &s, uintptr_t *lo, uintptr_t *hi);

// No two elements of the tensor share an address (each stride covers the
// extent of the smaller ones): required of the outputs.
bool injective(int B, int H, int N, int d, const Strides &s);

bool spans_overlap(uintptr_t alo, uintptr_t ahi, uintptr_t blo, uintptr_t bhi);

// Whether two tensors of B batch entries (Ha, Hb heads; Na, Nb rows) may
// share an element.  Exact when both have the same nested strides;
// otherwise whether their address spans overlap.
bool may_overlap(const void *a, Strides sa, int Ha, int Na, const void *b, Strides sb, int Hb, int Nb, int B, int d);

// Device address of the current device's status block, null on error.
int *status_ptr();

bool aligned16(const void *p);

// SMs of the current device (cached per host thread and device), 0 if unknown.
int sm_count();

inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace fa
