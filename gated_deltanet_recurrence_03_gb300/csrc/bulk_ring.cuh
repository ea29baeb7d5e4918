// The rows that a group of threads will need, in shared memory ahead of their use.
#pragma once

#include <cuda_bf16.h>

#include "tc_ptx.cuh"

namespace gdn {

// A group's mbarriers in shared memory, one a stage, and behind them the count of rows asked for (in memory: a register of
// every thread would be held for the one that issues).
constexpr int kRingMaxStages = 4;
constexpr int kRingWords = kRingMaxStages + 2;   // of 8 bytes each, a multiple of 16 in all
__device__ __forceinline__ void ring_init(uint64_t* bars) {   // by one thread, before the block's next barrier
    for (int i = 0; i < kRingMaxStages; ++i) tc::mbar_init(tc::smem_u32(bars + i), 1);
    *reinterpret_cast<int*>(bars + kRingMaxStages) = 0;
}

// `stages` rows of N tensors of D values, row k's pieces copied by one thread of the group with bulk copies that complete
// on the stage's mbarrier.  A wait that runs out sets *abort and the status word: the rows are then wrong, the issuing
// thread asks for no more, and its drain() keeps the block's shared memory until the copies in flight have landed.
template <typename T, int N>
struct BulkRing {
    const void* src[N];
    uint8_t* base;
    uint64_t* bars;   // kRingWords of them
    int D, stages;
    volatile int* abort;
    unsigned* status;
    unsigned status_flag;
    unsigned long long limit_ns;
    __device__ __forceinline__ uint32_t bar(int k) const { return tc::smem_u32(bars) + 8 * (k % stages); }
    __device__ __forceinline__ int& issued() const { return *reinterpret_cast<int*>(bars + kRingMaxStages); }
    __device__ __forceinline__ void issue(int k, long long row) {
        const uint32_t bytes = (uint32_t)D * sizeof(T), b = bar(k);
        uint32_t to = tc::smem_u32(base) + (k % stages) * N * bytes;
        tc::mbar_arrive_expect_tx(b, N * bytes);
#pragma unroll
        for (int t = 0; t < N; ++t) tc::bulk_g2s(to + t * bytes, static_cast<const T*>(src[t]) + (size_t)row * D, bytes, b);
        issued() = k + 1;
    }
    // Whether the issuing thread may go on; read here, it is there when the thread comes to issue (read there, a call of
    // 16384 rows of 4096 bf16 values takes 120.9 us instead of 119.4).
    __device__ __forceinline__ bool wait(int k) const {
        tc::mbar_wait_bounded(bar(k), (uint32_t)(k / stages) & 1, abort, status, status_flag, limit_ns);
        return !*abort;
    }
    __device__ __forceinline__ const T* at(int k, int t) const {
        return reinterpret_cast<const T*>(base) + (size_t)((k % stages) * N + t) * D;
    }
    // By the issuing thread after its last row: nothing to do but after a wait that ran out (its own, or another
    // group's, which ends this group's waits too).
    __device__ __forceinline__ void drain() const {
        if (!*abort) return;
        const int n = issued();
        for (int k = n > stages ? n - stages : 0; k < n; ++k)
            tc::mbar_wait_drain(bar(k), (uint32_t)(k / stages) & 1, limit_ns);
    }
};

}  // namespace gdn
