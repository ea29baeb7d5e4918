// What the selective scan's kernels share: vectors of four token values, tiles of channels, the step's width dt.
#pragma once

#include "f32x2.cuh"
#include "token_units.cuh"

namespace gdn {

constexpr int kScanThreads = 128;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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
// polynomial (a least-maximum fit of log1p(e) / e on [0, 1], 5e-9 off; with its roundings 1.6e-7).
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
    const float2 a = mul2(make_float2(y.x, y.y), mul2(za, logistic2(za))), b = mul2(make_float2(y.z, y.w), mul2(zb, logistic2(zb)));
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
