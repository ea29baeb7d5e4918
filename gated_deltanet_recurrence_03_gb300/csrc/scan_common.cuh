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
// A = -exp(A_log) in powers of two, finite: a token past a sequence's end has dt = 0 and must leave the state as it is.
__device__ __forceinline__ float rate2(float A_log) {
    const float A = -kLog2e * expf(A_log);
    return A < -3e38f ? -3e38f : A;
}
// dt = softplus(x), as the raw gates have it.
__device__ __forceinline__ float softplus_f(float x) { return fmaxf(x, 0.f) + log1pf(__expf(-fabsf(x))); }
__device__ __forceinline__ float logistic_f(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

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
