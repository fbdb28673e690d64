// gdn_packed.hpp - device-side places of packed sequences and their chunks.
// Included by kernel sources only.
#pragma once

#include <hip/hip_runtime.h>

#include "gdn_chunk.hpp"

namespace gdn {
namespace {

struct Span {
    int first, len;
};
// Tokens of sequence b.  Offsets outside [0, tokens] count as the nearer end, and
// one below the one before it as equal to it, so no access leaves the tensors.
__device__ __forceinline__ Span span_of(const Packed &s, int b) {
    if (!s.offsets) {
        const int t = s.tokens / s.B;
        return Span{b * t, t};
    }
    const int first = max(0, min(s.offsets[b], s.tokens)), end = max(0, min(s.offsets[b + 1], s.tokens));
    return Span{first, max(0, end - first)};
}

// The state of sequence b, -1 if it has none.
__device__ __forceinline__ int slot_of(const Packed &s, int b) {
    if (!s.slots) return b;
    const int x = s.slots[b];
    return x >= 0 && x < s.n_slots ? x : -1;
}

__device__ __forceinline__ int place_of(int first, int b) { return first / kChunk + b; }

// The sequence whose chunks' places begin last at or before `place`.
__device__ __forceinline__ int sequence_at(const Packed &s, int place) {
    int lo = 0, hi = s.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (place_of(span_of(s, mid).first, mid) <= place)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

}  // namespace
}  // namespace gdn
