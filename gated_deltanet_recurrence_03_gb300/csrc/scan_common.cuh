// What the selective scan's kernels share: vectors of four token values, tiles of channels, the step's width dt.
#pragma once

#include "f32x2.cuh"
#include "gdn_internal.cuh"

namespace gdn {

constexpr int kScanThreads = 128;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The tokens of a slot, and whether it is its sequence's first and last one; false for a slot without a sequence's segment (an
// empty sequence has one segment of no tokens).
struct ScanUnit {
    int seq;
    long long t0, t1;
    bool first, last;
};
// Segment j of sequence i is slot floor(start_i / seg) + i + j (no prefix sum needed), so that all are below
// floor(tokens / seg) + nseq; seg = 0: a slot is a sequence.
__device__ __forceinline__ long long scan_unit_base(const int32_t* cu, int T, int seg, int i) {
    long long s0, s1;
    seq_range(cu, i, T, s0, s1);
    return s0 / seg + i;
}
__device__ __forceinline__ bool scan_unit_at(const int32_t* cu, int T, int nseq, int seg, int slot, ScanUnit& u) {
    if (!seg) {
        u.seq = slot;
        seq_range(cu, slot, T, u.t0, u.t1);
        u.first = u.last = true;
        return true;
    }
    int lo = 0, hi = nseq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (scan_unit_base(cu, T, seg, mid) <= slot) lo = mid;
        else hi = mid - 1;
    }
    long long s0, s1;
    seq_range(cu, lo, T, s0, s1);
    const long long j = slot - (s0 / seg + lo), n = max(1LL, (s1 - s0 + seg - 1) / seg);
    if (j < 0 || j >= n) return false;
    u.seq = lo;
    u.t0 = s0 + j * seg;
    u.t1 = min(s1, u.t0 + seg);
    u.first = j == 0;
    u.last = j == n - 1;
    return true;
}

// The row of a segment's first chunk among the chunks of kScanChunk tokens of all sequences; its others follow.  Segments
// are whole chunks but for a sequence's last, so that chunk c of sequence i is row floor(start_i / kScanChunk) + i + c, and
// all are below floor(tokens / kScanChunk) + nseq.
static_assert(kScanMinSegment % kScanChunk == 0, "segments are whole chunks");
__device__ __forceinline__ size_t scan_chunk_row(const ScanUnit& u) { return (size_t)(u.t0 / kScanChunk + u.seq); }

// Four adjacent values of a token's row as loaded, and as fp32.
template <typename T>
struct Raw4;
template <>
struct Raw4<float> {
    float4 r;
    __device__ __forceinline__ float4 f() const { return r; }
    __device__ __forceinline__ static Raw4 zero() { return {make_float4(0.f, 0.f, 0.f, 0.f)}; }
};
template <>
struct Raw4<__nv_bfloat16> {
    uint2 r;
    __device__ __forceinline__ float4 f() const {
        return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                           __uint_as_float(r.y & 0xffff0000u));
    }
    __device__ __forceinline__ static Raw4 zero() { return {make_uint2(0u, 0u)}; }
};
template <typename T>
__device__ __forceinline__ Raw4<T> load4(const T* p) {
    return *reinterpret_cast<const Raw4<T>*>(p);
}
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 ex2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A token's decay 2^(A dt).  ex2.approx is 0.5 to 2e-8 low on average for exponents between -1/2 and 0, which compounds over
// a channel's memory (77 tokens: 1.6e-6 of the state, of which 0.6e-6 is rounding); this much more in the exponent leaves
// an average within 0.9e-8 there, and 2^0 is 1 with it too.
constexpr float kDecayShift = 2e-8f;
__device__ __forceinline__ float decay(float A2, float dt) { return ex2(fmaf(A2, dt, kDecayShift)); }
__device__ __forceinline__ float2 decay(float2 A2, float dt) { return ex2(fma2(A2, all2(dt), all2(kDecayShift))); }
// A = -exp(A_log) in powers of two, finite: a token past a sequence's end has dt = 0 and must leave the state as it is.
__device__ __forceinline__ float rate2(float A_log) {
    const float A = -kLog2e * expf(A_log);
    return A < -3e38f ? -3e38f : A;
}
// The larger one, or NaN (fmaxf drops it).
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// dt = softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|) with the exponent's rounding put back, log1p(e) as e times a
// polynomial (a least-maximum fit of log1p(e) / e on [0, 1], 1.8e-8 off with its fp32 coefficients; with its roundings 1.6e-7).
__device__ __forceinline__ float2 softplus2(float2 x) {
    const float2 n = make_float2(fmaxf(-fabsf(x.x), -150.f), fmaxf(-fabsf(x.y), -150.f));   // finite: exp(-150) is 0
    const float2 t = mul2(n, all2(kLog2e));
    const float2 rest = fma2(n, all2(kLog2e), make_float2(-t.x, -t.y));
    float2 e = ex2(t);
    e = fma2(e, mul2(rest, all2(kLn2)), e);
    float2 p = all2(-0.0032440212f);
    p = fma2(p, e, all2(0.019851444f));
    p = fma2(p, e, all2(-0.056959499f));
    p = fma2(p, e, all2(0.10603651f));
    p = fma2(p, e, all2(-0.1530559f));
    p = fma2(p, e, all2(0.19675939f));
    p = fma2(p, e, all2(-0.24954134f));
    p = fma2(p, e, all2(0.33329964f));
    p = fma2(p, e, all2(-0.49999902f));
    p = fma2(p, e, all2(1.f));
    return fma2(p, e, make_float2(max_nan(x.x, 0.f), max_nan(x.y, 0.f)));
}
__device__ __forceinline__ float4 softplus4(float4 x) {
    const float2 a = softplus2(make_float2(x.x, x.y)), b = softplus2(make_float2(x.z, x.w));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float logistic_f(float x) { return rcp(1.f + ex2(-kLog2e * x)); }
__device__ __forceinline__ float2 logistic2(float2 x) {
    const float2 e = add2(ex2(mul2(x, all2(-kLog2e))), all2(1.f));
    return make_float2(rcp(e.x), rcp(e.y));
}
// y silu(z)
__device__ __forceinline__ float4 gated4(float4 y, float4 z) {
    const float2 za = make_float2(z.x, z.y), zb = make_float2(z.z, z.w);
    const float2 a = mul2(make_float2(y.x, y.y), mul2(za, logistic2(za)));
    const float2 b = mul2(make_float2(y.z, y.w), mul2(zb, logistic2(zb)));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) {
    const float2 x = add2(make_float2(a.x, a.y), make_float2(b.x, b.y)), y = add2(make_float2(a.z, a.w), make_float2(b.z, b.w));
    return make_float4(x.x, x.y, y.x, y.y);
}

// A tile of adjacent channels of one group: `width` tiles a group, the last one with fewer channels.
struct ChannelTile {
    int g, d0, n;   // group, first channel, channels
};
__device__ __forceinline__ ChannelTile channel_tile(int D, int G, int per_tile, int tile) {
    const int P = D / G, per_group = (P + per_tile - 1) / per_tile;
    ChannelTile c;
    c.g = tile / per_group;
    const int at = (tile - c.g * per_group) * per_tile;
    c.d0 = c.g * P + at;
    c.n = min(per_tile, P - at);
    return c;
}

// A lane holds two channels of four states each; the L lanes of a channel pair are P = 32 / L lanes apart: adjacent lanes then
// read the same B and C, 2.1 cycles of shared memory a 16-byte read instead of 3.9 with L adjacent lanes on L addresses.
template <int N>
struct ScanShape {
    static constexpr int L = N / 4, P = 32 / L, CH = 2 * P * (kScanThreads / 32);   // CH: channels of a tile
};
struct ScanLane {
    int n0, pair;   // first state, channel pair in the warp
    int ch[2];      // channels in the tile; every other of a pair's lanes holds them in the other order, so that one exchange
                    // leaves each with its first channel's sum
};
template <int N>
__device__ __forceinline__ ScanLane scan_lane(int tid) {
    constexpr int P = ScanShape<N>::P;
    ScanLane l;
    l.pair = tid % P;
    l.n0 = tid % 32 / P * 4;
    l.ch[0] = tid / 32 * 2 * P + 2 * l.pair + (tid / P & 1);
    l.ch[1] = l.ch[0] ^ 1;
    return l;
}
__device__ __forceinline__ void load_states(float2 (&x)[2], const float* p) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    x[0] = make_float2(f.x, f.y);
    x[1] = make_float2(f.z, f.w);
}
__device__ __forceinline__ void store_states(float* p, const float2 (&x)[2]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
}
// A lane's rates, zeros past the tile.
template <int N>
__device__ __forceinline__ void load_rates(float2 (&A2)[2][2], const float* A_log, const ChannelTile& tile, const ScanLane& l) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const bool own = l.ch[s] < tile.n;
        if (own) load_states(A2[s], A_log + (size_t)(tile.d0 + l.ch[s]) * N + l.n0);
#pragma unroll
        for (int i = 0; i < 2; ++i) A2[s][i] = own ? make_float2(rate2(A2[s][i].x), rate2(A2[s][i].y)) : all2(0.f);
    }
}
// Four adjacent columns of a [D] tensor from the tile's column c on; zeros past the tile or without one.
__device__ __forceinline__ float4 columns(const float* p, const ChannelTile& tile, int c) {
    return p && c < tile.n ? *reinterpret_cast<const float4*>(p + tile.d0 + c) : make_float4(0.f, 0.f, 0.f, 0.f);
}
// dt and dt u of four channels; dt = 0 past the end, where nothing changes.
__device__ __forceinline__ void form_dt(float2* to, float4 u, float4 delta, float4 bias, bool ok) {
    float4 d = softplus4(add4(delta, bias));
    if (!ok) d = make_float4(0.f, 0.f, 0.f, 0.f);
    float4* p = reinterpret_cast<float4*>(to);
    p[0] = make_float4(d.x, d.x * u.x, d.y, d.y * u.y);
    p[1] = make_float4(d.z, d.z * u.z, d.w, d.w * u.w);
}

// W values of a lane, summed over the W lanes that differ in lane / BIT % W: lane gets the sum of value lane / BIT % W.
template <int W, int BIT = 1>
__device__ __forceinline__ float transpose_sum(float (&v)[W], int lane) {
#pragma unroll
    for (int w = W, s = BIT; w > 1; w /= 2, s *= 2) {
        const bool up = lane & s;
#pragma unroll
        for (int i = 0; i < w / 2; ++i) {
            const float keep = up ? v[2 * i + 1] : v[2 * i], send = up ? v[2 * i] : v[2 * i + 1];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, s);
        }
    }
    return v[0];
}

}  // namespace gdn
