// Test-only: what the kernels' shared pieces do when a bounded wait runs out (a copy that a test drops, an arrival that
// never comes): they end, within their limits, and say so.
#include <cuda_bf16.h>
#include <stdint.h>

#include "bulk_ring.cuh"

namespace {

constexpr int kD = 64, kThreads = 64;

// A group of 64 threads copies `rows` rows of 64 floats from src to dst through a ring, as the block norm walks its rows.
// The copy of row `drop` is never made.  result = {rows asked for, 1 if the abort flag is set}.
__global__ void __launch_bounds__(kThreads, 1)
ring_kernel(const float* src, float* dst, int rows, int stages, int drop, unsigned long long limit_ns, unsigned* status,
            int* result) {
    __shared__ __align__(128) float buf[gdn::kRingMaxStages * kD];
    __shared__ __align__(16) uint64_t bars[gdn::kRingWords];
    __shared__ int abort_flag;
    const int tid = threadIdx.x;
    if (tid == 0) {
        abort_flag = 0;
        gdn::ring_init(bars);
        gdn::tc::mbar_fence_init();
    }
    __syncthreads();
    gdn::BulkRing<float, 1> ring;
    ring.src[0] = src;
    ring.base = reinterpret_cast<uint8_t*>(buf);
    ring.bars = bars;
    ring.D = kD;
    ring.stages = stages;
    ring.abort = &abort_flag;
    ring.status = status;
    ring.status_flag = 1u;
    ring.limit_ns = limit_ns;
    auto ask = [&](int k) {
        if (k == drop) {
            gdn::tc::mbar_arrive_expect_tx(ring.bar(k), kD * 4);
            ring.issued() = k + 1;
        } else {
            ring.issue(k, k);
        }
    };
    if (tid == 0)
        for (int k = 0; k < stages && k < rows; ++k) ask(k);
    for (int k = 0; k < rows; ++k) {
        const bool go = ring.wait(k);
        if (stages > 1) __syncthreads();
        if (tid == 0 && go && k > 0 && stages > 1 && k + stages - 1 < rows) ask(k + stages - 1);
        dst[k * kD + tid] = ring.at(k, 0)[tid];
        if (stages == 1 && k + 1 < rows) {
            __syncthreads();
            if (tid == 0 && go) ask(k + 1);
        }
    }
    if (tid == 0) {
        ring.drain();
        result[0] = ring.issued();
        result[1] = abort_flag;
    }
}

// Two warps that hand rows to each other through a named barrier, as the decayed scan's output warps do: each waits for
// an arrival of its own in every round, and the pair decides at the barrier.  Warp 1's arrival of round `drop` never
// comes.  result = {rounds that warp 0 finished, rounds that warp 1 finished}.
__global__ void __launch_bounds__(64, 1)
pair_kernel(int rounds, int drop, unsigned long long limit_ns, unsigned* status, int* result) {
    __shared__ __align__(8) uint64_t bars[2];
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < 2; ++i) gdn::tc::mbar_init(gdn::tc::smem_u32(bars + i), 1);
        gdn::tc::mbar_fence_init();
    }
    __syncthreads();
    int done = 0;
    for (int it = 0; it < rounds; ++it) {
        const uint32_t bar = gdn::tc::smem_u32(bars + warp);
        if (lane == 0 && (warp == 0 || it != drop)) gdn::tc::mbar_arrive(bar);
        bool ok = __all_sync(~0u, gdn::tc::mbar_wait_bounded(bar, it & 1, &abort_flag, status, 1u, limit_ns));
        ok = gdn::tc::named_barrier_all(1, 64, ok);
        if (!ok) break;
        ++done;
    }
    if (lane == 0) result[warp] = done;
}

}  // namespace

extern "C" int giveup_pair(int rounds, int drop, unsigned long long limit_ns, unsigned* status, int* result) {
    pair_kernel<<<1, 64>>>(rounds, drop, limit_ns, status, result);
    return cudaGetLastError() == cudaSuccess ? 0 : 3;
}

extern "C" int giveup_ring(const float* src, float* dst, int rows, int stages, int drop, unsigned long long limit_ns,
                           unsigned* status, int* result) {
    if (stages < 1 || stages > gdn::kRingMaxStages || rows < 1) return 1;
    ring_kernel<<<1, kThreads>>>(src, dst, rows, stages, drop, limit_ns, status, result);
    return cudaGetLastError() == cudaSuccess ? 0 : 3;
}
