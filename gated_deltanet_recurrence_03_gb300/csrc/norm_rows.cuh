// What the norms over rows share: vectors of eight values, groups of threads that hold a row, their sums.
#pragma once

#include <algorithm>
#include <atomic>

#include "bulk_ring.cuh"
#include "f32x2.cuh"
#include "gdn_internal.cuh"

namespace gdn {

constexpr int kVec = 8;   // values of one vector of a thread

// Eight values as four pairs; the arithmetic is two fp32 operations an instruction.
struct V8 {
    float2 v[4];
};
// Eight values of either type at p (shared or global memory) as fp32, and back.
__device__ __forceinline__ V8 load8(const float* p) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    return {{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
}
__device__ __forceinline__ V8 load8(const __nv_bfloat16* p) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    V8 x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    return x;
}
__device__ __forceinline__ void store8(float* p, const V8& x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const V8& x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x.v[i].x, x.v[i].y);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A block holds `groups` row groups of `tpr` threads (a multiple of 32), each with a row of its own.
struct Group {
    int tpr, id, tid;   // threads of a row; this thread's group and place in it
};
__device__ __forceinline__ void group_sync(const Group& g) {
    if (g.tpr == 32) __syncwarp();
    else if (g.tpr == (int)blockDim.x) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(g.tpr) : "memory");
}
// Sums of N values over a row group's threads, in a fixed order; every thread gets them.  `buf` holds 32 N floats
// of the group, zero past its warps, and may be written again after the group's next synchronisation.
template <int N>
__device__ __forceinline__ void group_sum(float (&x)[N], float* buf, const Group& g) {
    const int lane = g.tid & 31, warp = g.tid >> 5, nw = g.tpr >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
    if (nw == 1) {
        __syncwarp();
        return;
    }
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) buf[i * 32 + warp] = x[i];
    group_sync(g);
#pragma unroll
    for (int i = 0; i < N; ++i) {   // every thread adds the warps' sums: no second round of shuffles
        float4 t = *reinterpret_cast<const float4*>(buf + i * 32);
        for (int w = 4; w < nw; w += 4) {
            const float4 u = *reinterpret_cast<const float4*>(buf + i * 32 + w);
            t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
        }
        x[i] = (t.x + t.y) + (t.z + t.w);
    }
}

// Shared memory of a block: the groups' reduction buffers (128 floats each), mbarriers, two constants a column, and the
// groups' rings.
struct RowSmem {
    float *red, *m, *wq;
    uint64_t* bars;
    int* abort;
    uint8_t* rings;
};
__device__ __forceinline__ RowSmem carve(uint8_t* p, int groups, int D) {
    RowSmem s;
    s.red = reinterpret_cast<float*>(p);
    s.bars = reinterpret_cast<uint64_t*>(s.red + groups * 128);
    s.abort = reinterpret_cast<int*>(s.bars + groups * kRingWords);
    s.m = reinterpret_cast<float*>(s.abort + 4);
    s.wq = s.m + D;
    s.rings = reinterpret_cast<uint8_t*>(s.wq + D);
    return s;
}
inline size_t smem_bytes(int groups, int D, int row_bytes, int stages) {
    return (size_t)groups * 128 * 4 + groups * kRingWords * 8 + 16 + (size_t)2 * D * 4 + (size_t)groups * stages * row_bytes;
}

constexpr size_t kSmemMax = 227 * 1024;

// The shared-memory limit of a kernel belongs to a device: raised once on each.
template <auto KERNEL>
cudaError_t allow_smem(size_t bytes = kSmemMax) {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> done[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
    return e;
}

// Vectors a thread holds, threads a row, row groups and ring stages a block, blocks.  With two vectors a thread a row's
// exchanges take half the threads and each has twice the work between them (block norm): 255 -> 209 us (backward, 16384 x 4096),
// 234 -> 187 us (32768 x 2048), 129 -> 81 us (65536 x 264); four are no better (201, 194 us; forward 119 -> 130 us).
// One vector where a row fits one warp, and where no SM has more than one row, whose latency then counts (4.2 against
// 5.5 us forward, 37 x 2048).
// A block fills an SM: up to 1024 threads and kSmemMax bytes, with as many groups as leave each at least two
// stages; past one warp a row the groups are limited by the named barriers.
struct RowShape {
    int v, tpr, groups, stages, blocks;
    size_t smem;
};
inline RowShape row_shape(int D, long long rows, int row_bytes, int threads2 = 512) {   // threads2: with two vectors a thread
    const int nv = D / kVec;
    RowShape s;
    s.v = nv <= 32 || (nv <= 512 && rows <= 152) ? 1 : 2;
    s.tpr = ((nv + s.v - 1) / s.v + 31) / 32 * 32;
    s.groups = std::max(1, (s.v == 1 ? 1024 : threads2) / s.tpr);
    if (s.tpr > 32) s.groups = std::min(s.groups, 8);
    s.groups = (int)std::min<long long>(s.groups, std::max(1LL, (rows + 151) / 152));   // few rows: every SM has some
    while (s.groups > 1 && smem_bytes(s.groups, D, row_bytes, 2) > kSmemMax) --s.groups;
    s.stages = kRingMaxStages;
    while (s.stages > 1 && smem_bytes(s.groups, D, row_bytes, s.stages) > kSmemMax) --s.stages;
    s.blocks = (int)std::min<long long>(152, (rows + s.groups - 1) / s.groups);
    s.smem = smem_bytes(s.groups, D, row_bytes, s.stages);
    return s;
}

}  // namespace gdn
