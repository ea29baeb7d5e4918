// Units of work of the decayed scan's kernels: sequences, or segments of them.
#pragma once

#include "gdn_internal.cuh"

namespace gdn {

// Segments: segment j of sequence i is slot floor(start_i / seg) + i + j (no prefix sum needed); `states` holds
// [scan][slot][Hv][dk][dv] floats, first a segment's own contribution to the state, then the state at its first
// visited end.  seg = 0: one CTA walks a whole sequence, and a slot is a sequence.
struct SegArgs {
    DecayArgs a;
    int seg, slots;
    float* states;
};

// The tokens of a slot, and whether it is the first and the last one its sequence's scan visits; false for a slot
// without a sequence's segment (an empty sequence has one segment of no tokens).
struct Unit {
    int seq;
    long long t0, t1;
    bool first, last;
};
__device__ __forceinline__ bool unit_of(const SegArgs& ta, int slot, bool rev, Unit& u) {
    const DecayArgs& a = ta.a;
    if (!ta.seg) {
        u.seq = slot;
        seq_range(a.cu, slot, a.T, u.t0, u.t1);
        u.first = u.last = true;
        return true;
    }
    auto base = [&](int i) {
        long long s0, s1;
        seq_range(a.cu, i, a.T, s0, s1);
        return s0 / ta.seg + i;
    };
    int lo = 0, hi = a.nseq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (base(mid) <= slot) lo = mid;
        else hi = mid - 1;
    }
    long long s0, s1;
    seq_range(a.cu, lo, a.T, s0, s1);
    const long long j = slot - base(lo), n = max(1LL, (s1 - s0 + ta.seg - 1) / ta.seg);
    if (j < 0 || j >= n) return false;
    u.seq = lo;
    u.t0 = s0 + j * ta.seg;
    u.t1 = min(s1, u.t0 + ta.seg);
    u.first = j == (rev ? n - 1 : 0);
    u.last = j == (rev ? 0 : n - 1);
    return true;
}
__device__ __forceinline__ float* unit_state(const SegArgs& ta, int scan, int slot, int h) {
    return ta.states + (((size_t)scan * ta.slots + slot) * ta.a.Hv + h) * ta.a.dk * ta.a.dv;
}

// The decay's exponent that the kernels use: -100 below that (-inf among them); a NaN stays one and a value above 0 a
// growth, as the formula has them.
__host__ __device__ __forceinline__ float decay_exponent(float log_decay) {
    return log_decay < kMinLogDecay ? kMinLogDecay : log_decay;
}

// a + b as its rounded value and the rest, whichever is larger.
__host__ __device__ __forceinline__ float two_sum(float a, float b, float& rest) {
    const float t = a + b, z = t - a;
    rest = (a - (t - z)) + (b - z);
    return t;
}

// exp(g n) as hi + lo: one rounding of a chunk's decay would compound over the head's memory.  For x = g n in [-12, 12]
// the relative error is below 2^(s - 43) + 2^-44 exp(-x), s the halvings that bring |x| to 2^-10: 2^-43 up to there,
// 2^-30 at x = -8.  From the series on y = x / 2^s, then s squarings of 1 + e in two floats, (1 + e)^2 - 1 = 2 e + e^2.
// (In fp64 the same takes ten times as long on this chip.)  Below exp(-12) a chunk forgets nearly all and one float
// does; infinities, NaN and overflowing growths end there too, as expf has them.
__host__ __device__ __forceinline__ void decay_power(float g, float n, float& hi, float& lo) {
    float xh = g * n, xl = fmaf(g, n, -xh);
    if (!(fabsf(xh) <= 12.f)) {
        hi = expf(xh);
        if (hi > 0.f && hi <= 3e38f) hi = fmaf(hi, xl, hi);
        lo = 0.f;
        return;
    }
    int s = 0;
    while (fabsf(xh) > 0.0009765625f) {   // exact halvings, at most 14
        xh *= 0.5f;
        xl *= 0.5f;
        ++s;
    }
    const float p = xh * xh * fmaf(xh, fmaf(xh, 0.041666668f, 0.16666667f), 0.5f);
    float eh = xh + p, el = (p - (eh - xh)) + xl, rest;
    for (; s > 0; --s) {
        const float sq = eh * eh, low = fmaf(eh, eh, -sq) + fmaf(2.f * eh, el, 2.f * el);
        eh = two_sum(2.f * eh, sq, rest);
        el = rest + low;
    }
    hi = two_sum(1.f, eh, rest);
    lo = rest + el;
    const float t = hi + lo;
    lo -= t - hi;
    hi = t;
}

// The scan's main kernel (state_only = false), or the pass before it that forms every segment's own contribution to
// the state, on the tensor cores (bf16) and on the CUDA cores (fp32).
cudaError_t launch_decay_tc(const SegArgs& s, bool state_only);
cudaError_t launch_decay_f32(const SegArgs& s, bool state_only);
constexpr int kDecayColumns = 64;   // value columns of a CTA of either

}  // namespace gdn
