// What the balance loss's kernels and the gate's backward share: which
// sequence a token counts for.
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace xmoe {

// Sequence of token t (seq_offsets[s] <= t < seq_offsets[s + 1]); S where t is
// behind the last sequence, -1 in front of the first.  The LT consecutive lanes
// that ask for one t search together: each tests the last sequence of one LT-th
// of the range, so the range shrinks LT-fold per load (log_LT(S) steps).  All
// lanes of the wavefront take part.
template <int LT>
__device__ __forceinline__ int find_sequence(const int32_t *off, int S, int64_t t) {
    const int lane = threadIdx.x & 63, r = lane % LT;
    int base = 0, len = S, stride;
    do {
        stride = (len + LT - 1) / LT;
        const int end = min(base + len, S), start = base + r * stride;
        const bool past = start < end && off[min(start + stride, end)] <= t;
        const unsigned long long all = __ballot(past);
        const unsigned long long mine = LT == 64 ? all : (all >> (lane - r)) & ((1ull << (LT & 63)) - 1ull);
        base += __popcll(mine) * stride;
        len = stride;  // the part whose last sequence is not past t
    } while (stride > 1);
    return t < off[0] ? -1 : min(base, S);
}

}  // namespace xmoe
