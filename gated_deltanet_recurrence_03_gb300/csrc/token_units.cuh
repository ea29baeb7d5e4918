// Units of work along the tokens: sequences, or segments of them.
#pragma once

#include "gdn_internal.cuh"

namespace gdn {

// The tokens of a slot, and whether it is the first and the last one its sequence's scan visits; false for a slot
// without a sequence's segment (an empty sequence has one segment of no tokens).
struct Unit {
    int seq;
    long long t0, t1;
    bool first, last;
};
// Segment j of sequence i is slot floor(start_i / seg) + i + j (no prefix sum needed), so that all are below
// floor(tokens / seg) + nseq; seg = 0: a slot is a sequence.
__device__ __forceinline__ long long unit_base(const int32_t* cu, int T, int seg, int i) {
    long long s0, s1;
    seq_range(cu, i, T, s0, s1);
    return s0 / seg + i;
}
__device__ __forceinline__ bool unit_at(const int32_t* cu, int T, int nseq, int seg, int slot, bool rev, Unit& u) {
    if (!seg) {
        u.seq = slot;
        seq_range(cu, slot, T, u.t0, u.t1);
        u.first = u.last = true;
        return true;
    }
    int lo = 0, hi = nseq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (unit_base(cu, T, seg, mid) <= slot) lo = mid;
        else hi = mid - 1;
    }
    long long s0, s1;
    seq_range(cu, lo, T, s0, s1);
    const long long j = slot - (s0 / seg + lo), n = max(1LL, (s1 - s0 + seg - 1) / seg);
    if (j < 0 || j >= n) return false;
    u.seq = lo;
    u.t0 = s0 + j * seg;
    u.t1 = min(s1, u.t0 + seg);
    u.first = j == (rev ? n - 1 : 0);
    u.last = j == (rev ? 0 : n - 1);
    return true;
}

}  // namespace gdn
