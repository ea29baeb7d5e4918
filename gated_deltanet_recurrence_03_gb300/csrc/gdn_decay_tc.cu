// The decayed scan (gdn_internal.cuh, DecayScan) on the tcgen05 tensor cores: bf16, head dims 32, 64 and 128.
//
// Inside a chunk of C = 128 tokens, n of them valid, with w_d = a^d and S the state at the chunk's first
// visited end (its start; its end in a reverse scan), in token order r, j = 0 .. n - 1:
//   forward   out_r = so (w_{r+1} q_r S + su sum_{j<=r} w_{r-j} (q_r.k_j) v_j),  S <- w_n S + su sum_j w_{n-1-j} k_j v_j^T
//   reverse   out_r = so (w_{n-1-r} q_r S + su sum_{j>=r} w_{j-r} (q_r.k_j) v_j), S <- w_n S + su sum_j w_{j+1} k_j v_j^T
//
// One CTA walks one sequence (or one segment of it) of one value head for 64 of its value columns, so that a
// 128-wide head keeps two SMs busy; the two read the same q and k tiles, the second time from L2.  Per chunk
// four products (M = 128 each):
//   QK [128 x 128] = Q K^T;   PV [128 x 64] = P V, P = the decayed, masked QK as the bf16 A operand in TMEM;
//   QS [128 x 64] = Q S_bf16;   KV [dk x 64] = K^T V~, V~ = V scaled by su w, in three bf16 parts side by side.
// The state is kept in registers in fp32 (64 columns of one row a thread), so the products of a chunk wait for
// the state only in QS: KV goes to a fresh accumulator, and S <- w_n S + KV is one FMA per element (with w_n in
// two floats: one rounding of it would compound over the head's memory).  V~'s three parts hold its fp32 value
// exactly, K is exact, so the states that leave the kernel have fp32 accuracy; P and the state's copy in QS are
// rounded to bf16, each 2^-9 of terms whose sum is rounded to bf16 anyway.
//
// Bound by the chunk's chain of hand-overs and by shared memory, not by the tensor pipe: a chunk moves about 400 KB
// through shared memory (tiles in, V's parts written and read, P's and the state's operands, outputs), 3100 cycles at
// 128 bytes a cycle, and takes about 4000; the tensor pipe is 40 % active, HBM at 32 % of its peak.  Measured (bf16,
// 2 x 8192 tokens, 32 value heads and 16 query/key heads of 128): forward 144 us with the final state (2.9 TB/s of the
// bytes that it must move), 135 us without; backward 519 us, of it 423 us in this kernel's three scans, 398 us where
// no heads are shared.  What brought it there from 318 us: the first tiles' prefetch to L2 (176 -> 154 us); the parts
// of V side by side in one product of N = 192; QS ahead of P in the issue order; the outputs through shared memory in
// whole rows (stored from the registers in 16-byte pieces: 20 % slower); two parts instead of three where no state
// leaves (backward 603 -> 540 us); one streaming sum over shared heads for both gradients (537 -> 515 us); 64 / 72 / 128 registers for
// issue / work / state (56 / 72 / 136: 572 us).
// 64 columns a CTA: a whole 128-wide head would not fit (state, V's parts and two stages of tiles) and would leave
// half of the SMs idle here.
//
// Warps: 0-7 form P; 8-15 scale and split V and write the outputs; 16-19 keep the state; 20 issues the MMAs, 21
// the copies; 22 and 23 see to values of V that are not finite.  Hand-overs are mbarriers; every wait on one is bounded.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <climits>
#include <mutex>

#include "decay_unit.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace {

using namespace tc;
using bf16 = __nv_bfloat16;

constexpr int kC = 128;       // tokens of a chunk
constexpr int kHalf = kDecayColumns;
constexpr int kMaxParts = 3;  // bf16 parts of the scaled V

// Shared memory (bytes from the 1024-aligned base).  Panels: 128 rows x 64 bf16, 128-byte swizzle.
constexpr uint32_t kPanel = 16384;
constexpr uint32_t S_Q = 0;                          // 2 stages x 2 panels
constexpr uint32_t S_K = S_Q + 2 * 2 * kPanel;       // 2 stages x 2 panels
constexpr uint32_t S_V = S_K + 2 * 2 * kPanel;       // 2 stages x 1 panel
constexpr uint32_t S_VP = S_V + 2 * kPanel;          // the three parts of the scaled V
constexpr uint32_t S_SB = S_VP + kMaxParts * kPanel; // the state in bf16 (128 dk rows); between its uses, the outputs
constexpr uint32_t S_SLOW = S_V + kPanel;            // one chunk only: the state copy's second part
constexpr uint32_t S_OUT = S_VP + 2 * kPanel;        // with two parts: the outputs on their way
constexpr uint32_t S_BAR = S_SB + kPanel;
constexpr uint32_t kBarBytes = 256;
constexpr uint32_t S_PW = S_BAR + kBarBytes;         // w_0 .. w_128
constexpr uint32_t S_ODD = S_PW + 132 * 4;           // 64 columns of V: the first token with a value that is not finite
constexpr uint32_t kSmem = S_ODD + 64 * 4 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");

enum Bar : uint32_t {
    B_FULLQK = 0,   // 2: q and k tiles of a stage have landed
    B_FULLV = 2,    // 2: the v tile
    B_QK = 4,       // QK is complete
    B_QKFREE = 5,   // QK has been read
    B_P = 6,        // P is in TMEM
    B_VP = 7,       // 2: the parts of V's rows 0-63, 64-127 are in shared memory
    B_KVHALF = 9,   // the products of rows 0-63 are complete
    B_KV = 10,      // KV is complete
    B_KVFREE = 11,  // KV has been read
    B_S = 12,       // the state's bf16 copy is in shared memory
    B_O = 13,       // QS and PV are complete
    B_OFREE = 14,   // QS and PV have been read
    B_FREE = 15,    // 2: every product of the chunk in a stage is complete
    B_SBFREE = 17,  // the outputs have left the place of the state's copy
    B_GAMMA = 18,   // w_n in two floats
    B_DRAIN = 19,
    B_COUNT = 20
};

// TMEM columns (all 512): KV holds the products with V's (up to three) parts side by side.
constexpr uint32_t T_QK = 0, T_P = 128, T_QS = 192, T_PV = 256, T_KV = 320;
constexpr uint32_t kTmemCols = 512;

// 24 warps, six groups of four.  Registers a thread: 80 at launch; P's and V's groups give up 8 and the issuing
// warps' 16, and the state's takes them (64 hold its part of the state): 4 x 72 + 128 + 64 = 6 x 80.
constexpr int kThreads = 24 * 32;
constexpr int kRegsWork = 72, kRegsIssue = 64, kRegsState = 128;
constexpr int kBarOutputs = 5;   // named barriers: 1-4 the pairs of output warps
constexpr int kWarpV = 8, kWarpState = 16, kWarpMma = 20, kWarpCopy = 21;
constexpr float kFactored = 5.f;  // log decays of a larger size (or NaN) are not factored over 16 columns

struct Maps {
    CUtensorMap q, k, v;
};
struct TcArgs : SegArgs {
    Maps maps[kMaxScans];
};


__device__ __forceinline__ void named_barrier_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t&>(d)) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t&>(d)) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(reinterpret_cast<uint64_t&>(d)) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}
__device__ __forceinline__ float2 as_float2(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }
__device__ __forceinline__ uint32_t pack_bf16(float2 x) { return tc::pack_bf16(x.x, x.y); }
// x as a sum of bf16 values: each is x, or what is left of it, cut to eight significant bits (the differences are
// exact in fp32), the last of two rounded.  Three hold x exactly, two to 2^-17.  A pair's two values are packed.
template <int PARTS>
__device__ __forceinline__ void split_bf16(float2 x, uint32_t (&part)[PARTS]) {
    constexpr uint32_t kCut = 0xffff0000u, kSign = 0x80000000u;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        const uint32_t a = __float_as_uint(x.x), b = __float_as_uint(x.y);
        if (PARTS == 2 && p == 1) {
            part[p] = pack_bf16(x);
        } else {
            part[p] = __byte_perm(a, b, 0x7632);
            if (p + 1 < PARTS) x = add2(x, as_float2((a & kCut) ^ kSign, (b & kCut) ^ kSign));
        }
    }
}
// mbar_wait_bounded in fewer instructions, and with each test suspended for up to a millisecond: the roles' loops
// share the schedulers and one instruction cache, and a polling warp takes both from the others.
__device__ __forceinline__ bool try_wait_long(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int* abort, unsigned* status) {
    if (try_wait_long(bar, parity)) return true;
    const unsigned long long t0 = globaltimer();
    while (!*abort) {
        if (try_wait_long(bar, parity)) return true;
        if (globaltimer() - t0 > kWaitLimitNs) {
            *abort = 1;
            atomicOr(status, kStatusTimeout);
        }
    }
    return false;
}

// The same by a whole warp: one answer for all lanes, which must not part where one of them gives up.  (A vote
// after a wait of each lane's own makes the compiler spill: 160 us instead of 140 for 2 x 8192 tokens.)
__device__ __forceinline__ bool warp_wait_or_abort(uint32_t bar, uint32_t parity, volatile int* abort, unsigned* status) {
    if (__all_sync(~0u, try_wait_long(bar, parity))) return true;
    const unsigned long long t0 = globaltimer();
    while (true) {
        if (__any_sync(~0u, *abort)) return false;
        if (__all_sync(~0u, try_wait_long(bar, parity))) return true;
        if (globaltimer() - t0 > kWaitLimitNs) {
            *abort = 1;
            atomicOr(status, kStatusTimeout);
        }
    }
}

__device__ __forceinline__ int slot_of(const DecayArgs& a) { return blockIdx.x / (a.dv > kHalf ? 2 : 1) / a.Hv; }

// One scan's CTA.  REV: a reverse scan; F32: the outputs are float; PARTS: bf16 parts of the scaled V (three where
// the last state is wanted, which then has fp32 accuracy; two where it only serves the outputs, whose own rounding
// is 2^-9); STATE: only a segment's contribution to the state, from zeros, no outputs; FINE: one chunk or none, with P
// and the state's copy in two bf16 parts each: an output of few tokens is a sum of few roundings, up to 1.7 times the
// output type's own where one score rules it, and a lone chunk has the time (the same 15 us a call).  (Template
// arguments, not branches, for the instruction cache's sake.)
template <bool REV, bool F32, int PARTS, bool STATE, bool FINE>
__device__ __forceinline__ void decay_tc_body(const TcArgs& ta, const Unit& unit) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    auto bar = [&](uint32_t b) { return sb + S_BAR + 8 * b; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + S_BAR + 8 * B_COUNT);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + S_BAR + 8 * B_COUNT + 4);
    float* gamma = reinterpret_cast<float*>(sm + S_BAR + 8 * B_COUNT + 8);   // w_128, w_n of the last chunk: hi, lo each
    float* pw = reinterpret_cast<float*>(sm + S_PW);
    int* odd = reinterpret_cast<int*>(sm + S_ODD);

    const DecayArgs& a = ta.a;
    const DecayScan& s = a.scan[blockIdx.y];
    const Maps& maps = ta.maps[blockIdx.y];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int dk = a.dk, dv = a.dv;
    const int zs = dv > kHalf ? 2 : 1, z = blockIdx.x % zs;   // 64-column parts of the values: this CTA's
    const int h = blockIdx.x / zs % a.Hv;
    const int slot = slot_of(a);
    const int width = min(kHalf, dv - kHalf * z);             // 32 where dv = 32: the tile's other columns are zeros
    const int steps = dk / 16, panels = dk > 64 ? 2 : 1;      // of q and k rows (32-wide ones lie in 64-wide panels)
    constexpr bool rev = REV;
    const long long t0 = unit.t0, t1 = unit.t1;
    const int nch = (int)((t1 - t0 + kC - 1) / kC);
    const int tail = (int)(t1 - t0) - (nch - 1) * kC;   // valid tokens of the last chunk
    const float g = decay_exponent(a.log_decay[h]);

    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tc_fence_before();
    }
    if (tid == 0) {
        *abort_flag = 0;
        for (uint32_t b = 0; b < B_COUNT; ++b) {
            const uint32_t count = b == B_QKFREE || b == B_P || b == B_OFREE || b == B_SBFREE ? 8
                                   : b == B_KVFREE || b == B_S || b == B_VP || b == B_VP + 1 ? 4 : 1;
            mbar_init(bar(b), count);
        }
        mbar_fence_init();
    }
    if (tid < 64) odd[tid] = INT_MAX;
    if (tid <= kC) pw[tid] = tid ? expf(g * (float)tid) : 1.f;
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);   // this warp's quarter of the lanes

    unsigned* status = a.status;
    auto wait_one = [&](uint32_t b, uint32_t parity) {
        return wait_or_abort(bar(b), parity & 1, abort_flag, status);
    };
    auto wait = [&](uint32_t b, uint32_t parity) { return warp_wait_or_abort(bar(b), parity & 1, abort_flag, status); };
    auto arrive = [&](uint32_t b) {   // once for the warp, after all its lanes
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(b));
    };
    auto chunk_of = [&](int it) { return rev ? nch - 1 - it : it; };
    auto valid_of = [&](int it) { return chunk_of(it) == nch - 1 ? tail : kC; };

    if (warp > kWarpCopy) {
        regs_dec<kRegsIssue>();   // there to make the group of four whole, and for columns of V that are not finite
        // (in the output warps the same code takes 2 to 5 % of the gradients' time, wherever it stands)
        if (!STATE) {
            named_barrier_sync(kBarOutputs, 320);   // every output is written
            const int c = tid & 63, from = odd[c];
            if (from != INT_MAX && c < width) {
                const int it = from / kC, n = valid_of(it);
#pragma unroll 1
                for (int v = from % kC; v < n; ++v) {
                    const size_t e = (size_t)(t0 + (long long)chunk_of(it) * kC + (rev ? n - 1 - v : v)) * s.out_stride +
                                     (size_t)h * dv + kHalf * z + c;
                    if (F32) static_cast<uint32_t*>(s.out)[e] = 0x7fffffffu;   // NaN
                    else static_cast<uint16_t*>(s.out)[e] = 0x7fffu;
                }
            }
        }
    } else if (warp == kWarpCopy) {
        regs_dec<kRegsIssue>();
        // ------------------------------------------------------------ copies
        if (lane == 0 && nch > 0) {
            const int hq = h / s.q_div, hk = h / s.k_div, hv = h / s.v_div;
            auto load = [&](int it) {
                const int st = it & 1, t = (int)t0 + chunk_of(it) * kC;
                const uint32_t bv = bar(B_FULLV + st), bqk = bar(B_FULLQK + st);
                mbar_arrive_expect_tx(bv, kPanel);
                tma_load_3d(sb + S_V + st * kPanel, &maps.v, 64 * z, hv, t, bv);
                mbar_arrive_expect_tx(bqk, (STATE ? 1 : 2) * panels * kPanel);
#pragma unroll 1
                for (int p = 0; p < panels; ++p) {
                    if (!STATE) tma_load_3d(sb + S_Q + (2 * st + p) * kPanel, &maps.q, 64 * p, hq, t, bqk);
                    tma_load_3d(sb + S_K + (2 * st + p) * kPanel, &maps.k, 64 * p, hk, t, bqk);
                }
            };
            auto prefetch = [&](int it) {   // into L2: the loads wait for a stage to be free and then cannot wait for DRAM
                if (it >= nch) return;
                const int t = (int)t0 + chunk_of(it) * kC;
                tma_prefetch_3d(&maps.v, 64 * z, hv, t);
#pragma unroll 1
                for (int p = z; p < panels; p += zs) {   // with two CTAs for a head each takes half of q and k
                    if (!STATE) tma_prefetch_3d(&maps.q, 64 * p, hq, t);
                    tma_prefetch_3d(&maps.k, 64 * p, hk, t);
                }
            };
            int loaded = 0;
            for (; loaded < 2 && loaded < nch; ++loaded) load(loaded);
            prefetch(2);
            prefetch(3);
#pragma unroll 1
            for (int x = 0; x < 2; ++x) decay_power(g, (float)(x ? tail : kC), gamma[2 * x], gamma[2 * x + 1]);   // of a full, of the last chunk
            mbar_arrive(bar(B_GAMMA));
            for (; loaded < nch; ++loaded) {   // into the stage of the chunk two back
                if (!wait_one(B_FREE + (loaded & 1), (loaded >> 1) - 1)) break;
                load(loaded);
                prefetch(loaded + 2);
            }
            // whichever wait gives up, now or later: no copy may still be landing when the shared memory is released
            for (int it = max(0, loaded - 2); it < loaded; ++it) {
                mbar_wait_drain(bar(B_FULLQK + (it & 1)), (it >> 1) & 1, kWaitLimitNs);
                mbar_wait_drain(bar(B_FULLV + (it & 1)), (it >> 1) & 1, kWaitLimitNs);
            }
        }
        __syncwarp();
    } else if (warp == kWarpMma) {
        regs_dec<kRegsIssue>();
        // ------------------------------------------------------------ products
        // The whole warp runs the loop and one elected lane issues: always the same one, so that a commit
        // covers every product before it.
        const uint64_t dQ = smem_desc(sb + S_Q, 16, 1024), dK = smem_desc(sb + S_K, 16, 1024),
                       dKt = smem_desc(sb + S_K, kPanel, 1024), dV = smem_desc(sb + S_V, 1024, 1024),
                       dVP = smem_desc(sb + S_VP, kPanel, 1024), dSB = smem_desc(sb + S_SB, 1024, 1024);
        bool ok = true;
        for (int it = nch > 0 ? -1 : 0; it < nch; ++it) {
            const int st = it & 1;
            if (it >= 0) {
                // K^T V~: V's parts are there (and, in a last chunk, the rows past its end are zero)
                ok = wait(B_VP, it) && (it < 1 || wait(B_KVFREE, it - 1));
                if (!ok) break;
                tc_fence_after();
                // (rows past dk of the product come from whatever lies behind k's panel: nothing reads them)
                const uint64_t kt = dKt + ((st * 2 * kPanel) >> 4);
                // half the rows at a time, so that the first half's parts are replaced while the second runs
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_bf16(tmem + T_KV, kt + ((ks * 2048) >> 4), dVP + ((ks * 2048) >> 4),
                                 idesc_bf16(128, 64 * PARTS, 1, 1), ks > 0);
                    mma_commit(bar(B_KVHALF));
                }
                __syncwarp();
                ok = wait(B_VP + 1, it);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 4; ks < 8; ++ks)
                        mma_bf16(tmem + T_KV, kt + ((ks * 2048) >> 4), dVP + ((ks * 2048) >> 4),
                                 idesc_bf16(128, 64 * PARTS, 1, 1), 1);
                    mma_commit(bar(B_KV));
                    if (STATE) mma_commit(bar(B_FREE + st));
                }
                __syncwarp();
            }
            if (STATE) {   // the next chunk's k (with scores to form, its arrival is waited for below)
                if (it + 1 < nch) ok = wait(B_FULLQK + ((it + 1) & 1), (it + 1) >> 1);
                if (!ok) break;
                continue;
            }
            // the next chunk's scores: P is formed from them while this chunk's outputs and the next KV and QS run
            if (it + 1 < nch) {
                ok = wait(B_FULLQK + ((it + 1) & 1), (it + 1) >> 1) && (it < 0 || wait(B_QKFREE, it));
                if (!ok) break;
                tc_fence_after();
                const uint32_t o = (((it + 1) & 1) * 2 * kPanel) >> 4;
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        if (ks >= steps) break;
                        const uint32_t x = o + (((ks >> 2) * kPanel + (ks & 3) * 32) >> 4);
                        mma_bf16(tmem + T_QK, dQ + x, dK + x, idesc_bf16(128, 128, 0, 0), ks > 0);
                    }
                    mma_commit(bar(B_QK));
                }
                __syncwarp();
            }
            if (it >= 0) {
                const uint64_t q = dQ + ((st * 2 * kPanel) >> 4);
                ok = wait(B_S, it) && (it < 1 || wait(B_OFREE, it - 1));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        if (ks >= steps) break;
                        mma_bf16(tmem + T_QS, q + (((ks >> 2) * kPanel + (ks & 3) * 32) >> 4), dSB + ((ks * 2048) >> 4),
                                 idesc_bf16(128, 64, 0, 1), ks > 0);
                    }
                    if (FINE) {
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            if (ks >= steps) break;
                            mma_bf16(tmem + T_QS, q + (((ks >> 2) * kPanel + (ks & 3) * 32) >> 4),
                                     dSB + ((int)(S_SLOW - S_SB) / 16 + (ks * 2048) / 16), idesc_bf16(128, 64, 0, 1), 1);
                        }
                    }
                }
                __syncwarp();
                ok = wait(B_P, it);
                if (!ok) break;
                tc_fence_after();
                const uint64_t v = dV + ((st * kPanel) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_bf16_ta(tmem + T_PV, tmem + T_P + 8 * ks, v + ((ks * 2048) >> 4), idesc_bf16(128, 64, 0, 1),
                                    ks > 0);
                    if (FINE) {
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_bf16_ta(tmem + T_PV, tmem + T_QK + 64 * (ks >> 2) + 8 * (ks & 3), v + ((ks * 2048) >> 4),
                                        idesc_bf16(128, 64, 0, 1), 1);
                    }
                    mma_commit(bar(B_O));
                    mma_commit(bar(B_FREE + st));
                }
                __syncwarp();
            }
        }
        if (nch > 0 && ok) wait(B_FREE + ((nch - 1) & 1), (nch - 1) >> 1);   // the last arrival of a commit
        if (*abort_flag) {   // every product issued is complete before TMEM and shared memory are released
            if (elect_one()) mma_commit(bar(B_DRAIN));
            __syncwarp();
            mbar_wait_drain(bar(B_DRAIN), 0, kWaitLimitNs);
        }
        __syncwarp();
    } else if (warp < kWarpV) {
        regs_dec<kRegsWork>();
        // ------------------------------------------------------------ P: rows 32 (warp % 4) .., half warp / 4 of the columns
        const int half = warp >> 2, r0 = 32 * (warp & 3), r = r0 + lane;
        const float f = s.so * s.su, g2 = g * 1.44269504f;
        float2 wj[8];   // 1 / w_0 .. 1 / w_15 (backwards in a reverse scan)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            wj[e] = make_float2(exp2f(-g2 * (float)(rev ? 15 - 2 * e : 2 * e)), exp2f(-g2 * (float)(rev ? 14 - 2 * e : 2 * e + 1)));
        for (int it = 0; !STATE && it < nch; ++it) {
            const int n = valid_of(it);
            if (!wait(B_QK, it)) break;
            tc_fence_after();
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {   // 16 columns at a time
                const int j0 = 64 * half + 16 * b;
                uint32_t x[16], p[8], low[8];
                tmem_ld16(tl + T_QK + j0, x);
                tmem_wait_ld();
                if (b == 3) {
                    tc_fence_before();
                    arrive(B_QKFREE);
                }
                // how many of the 16 columns row r sees: the first ones (forward) or the last ones (reverse), of
                // those before the sequence's end
                const int seen = rev ? j0 + 16 - r : r - j0 + 1;
                const int last = rev ? n - j0 : 16;
                if (rev ? r0 > j0 + 15 : r0 + 31 < j0) {   // none, for the whole warp
#pragma unroll
                    for (int e = 0; e < 8; ++e) p[e] = low[e] = 0u;
                } else {
                    const auto put = [&](int e, float2 y) {
                        if (FINE) {
                            uint32_t part[2];
                            split_bf16<2>(y, part);
                            p[e] = part[0];
                            low[e] = part[1];
                        } else {
                            p[e] = pack_bf16(y);
                        }
                    };
                    if (fabsf(g) <= kFactored) {   // w_|r - j| = w_(seen - 1) / w_(distance of j from the block's far end)
                        const float fr = f * exp2f(g2 * (float)max(seen - 1, 0));
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            put(e, mul2(mul2(make_float2(fr, fr), wj[e]), as_float2(x[2 * e], x[2 * e + 1])));
                    } else {              // strong decays, element by element
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int d0 = rev ? j0 + 2 * e - r : r - j0 - 2 * e, d1 = rev ? d0 + 1 : d0 - 1;
                            put(e, make_float2(f * pw[max(d0, 0)] * __uint_as_float(x[2 * e]),
                                               f * pw[max(d1, 0)] * __uint_as_float(x[2 * e + 1])));
                        }
                    }
                    // masked columns become zeros whatever they hold: on the diagonal, and past the end in reverse
                    if (rev ? r0 + 31 > j0 || n < kC : r0 < j0 + 15) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const bool lo = rev ? 16 - 2 * e <= seen && 2 * e < last : 2 * e < seen;
                            const bool hi = rev ? 15 - 2 * e <= seen && 2 * e + 1 < last : 2 * e + 1 < seen;
                            const uint32_t keep = (lo ? 0xffffu : 0u) | (hi ? 0xffff0000u : 0u);
                            p[e] &= keep;
                            if (FINE) low[e] &= keep;
                        }
                    }
                }
                if (b == 0) {   // the previous chunk's PV has read P
                    if (it > 0) wait(B_O, it - 1);
                    tc_fence_after();
                }
                tmem_st8(tl + T_P + j0 / 2, p);
                if (FINE) tmem_st8(tl + T_QK + 64 * half + 8 * b, low);   // scores that this warp has read
            }
            tmem_wait_st();
            tc_fence_before();
            arrive(B_P);
        }
    } else if (warp < kWarpState) {
        regs_dec<kRegsWork>();
        // ------------------------------------------------------------ V's parts and the outputs: half a row a thread
        const int r = 32 * (warp & 3) + lane, half = (warp >> 1) & 1, c0 = 4 * ((warp - kWarpV) >> 2);
        auto split = [&](int it) {
            const int st = it & 1, n = valid_of(it);
            if (!wait(B_FULLV + st, it >> 1)) return false;
            if (n < kC) {   // the rows past the sequence's end are zero wherever they are summed over
                if (!wait(B_FULLQK + st, it >> 1)) return false;
                if (r >= n) {
#pragma unroll 1
                    for (int c = 0; c < 12; ++c) {   // in v's panel and k's two
                        const uint32_t panel = c < 4 ? S_V + st * kPanel : S_K + (2 * st + (c >> 2) - 1) * kPanel;
                        *reinterpret_cast<uint4*>(sm + panel + swz(r, c0 + (c & 3))) = make_uint4(0, 0, 0, 0);
                    }
                }
            }
            const float w = r < n ? s.su * pw[rev ? r + 1 : n - 1 - r] : 0.f;
            uint4 v[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = *reinterpret_cast<const uint4*>(sm + S_V + st * kPanel + swz(r, c0 + c));
            // the products of the previous chunk that read these rows' parts are complete
            if (it > 0 && !wait(half ? B_KV : B_KVHALF, it - 1)) return false;
            float2 zero = make_float2(0.f, 0.f);   // NaN after a value that is not finite
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t y[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
                uint32_t o[4][PARTS];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 x = as_float2(y[e] << 16, y[e] & 0xffff0000u);
                    split_bf16<PARTS>(mul2(make_float2(w, w), x), o[e]);
                    if (!STATE) zero = fma2(x, make_float2(0.f, 0.f), zero);
                }
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
                    *reinterpret_cast<uint4*>(sm + S_VP + p * kPanel + swz(r, c0 + c)) = make_uint4(o[0][p], o[1][p], o[2][p], o[3][p]);
            }
            if (!STATE && !(zero.x + zero.y == 0.f)) {
                // It would make NaN of a masked zero of P.  So it leaves V's panel, and a warp apart makes its column's outputs
                // of the chunk NaN from its token on; later chunks see it through the state.
#pragma unroll 1
                for (int c = 8 * c0; c < 8 * c0 + 32; ++c) {
                    uint16_t* x = reinterpret_cast<uint16_t*>(sm + S_V + st * kPanel + swz(r, c >> 3)) + (c & 7);
                    if ((*x & 0x7f80) != 0x7f80) continue;
                    *x = 0;
                    atomicMin(odd + c, it * kC + (rev ? n - 1 - r : r));
                }
            }
            fence_proxy_async_smem();
            arrive(B_VP + half);
            return true;
        };
        // A chunk's outputs (rows of 128 bytes at a time) pass through the third part's place or, with three parts,
        // that of the state's copy, which QS has read: warps w and w + 4 hold the two halves of the same 32 rows,
        // and each writes 16 whole rows.
        constexpr uint32_t kOut = PARTS == 2 ? S_OUT : S_SB;
        constexpr int esize = F32 ? 4 : 2;
        const int pair = 1 + (warp & 3), own = 32 * (warp & 3) + 4 * c0 + (lane >> 3), chunk = lane & 7;
        uint8_t* const out = static_cast<uint8_t*>(s.out) + ((size_t)h * dv + kHalf * z) * esize +
                             (F32 ? (chunk >> 2) * 128 + (chunk & 3) * 16 : chunk * 16);
        const size_t pitch = (size_t)s.out_stride * esize;
        // A wait that gives up leaves its warp going on with whatever is there, until the pair decides at a barrier: a warp
        // that stopped alone would leave its partner waiting there for ever.
        auto write_outputs = [&](int it) {
            const int n = valid_of(it);
            wait(B_O, it);
            tc_fence_after();
            const float w = s.so * pw[rev ? max(n - 1 - r, 0) : r + 1];
            uint8_t* const first = out + (size_t)(t0 + (long long)chunk_of(it) * kC) * pitch;
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                uint32_t qs[16], pv[16];
                tmem_ld16(tl + T_QS + 8 * c0 + 16 * b, qs);
                tmem_ld16(tl + T_PV + 8 * c0 + 16 * b, pv);
                tmem_wait_ld();
                if (b) {
                    tc_fence_before();
                    arrive(B_OFREE);
                }
                float2 o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[e] = fma2(make_float2(w, w), as_float2(qs[2 * e], qs[2 * e + 1]), as_float2(pv[2 * e], pv[2 * e + 1]));
                // (the rows staged before have been read)
                if (PARTS == 2 && !b) {
                    if (!named_barrier_all(pair, 64, !*abort_flag)) return false;
                } else if (F32) {
                    named_barrier_sync(pair, 64);
                }
                if (F32) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        *reinterpret_cast<float4*>(sm + kOut + swz(r, c0 + c)) =
                            make_float4(o[2 * c].x, o[2 * c].y, o[2 * c + 1].x, o[2 * c + 1].y);
                } else {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        *reinterpret_cast<uint4*>(sm + kOut + swz(r, c0 + 2 * b + c)) =
                            make_uint4(pack_bf16(o[4 * c]), pack_bf16(o[4 * c + 1]), pack_bf16(o[4 * c + 2]), pack_bf16(o[4 * c + 3]));
                }
                if (F32 || b) {
                    if (PARTS == 3) {
                        if (!named_barrier_all(pair, 64, !*abort_flag)) return false;
                    } else {
                        named_barrier_sync(pair, 64);
                    }
#pragma unroll
                    for (int x = 0; x < 16; x += 4)
                        if (own + x < n && (F32 ? 32 * (chunk >> 2) + 16 * b + 4 * (chunk & 3) : 8 * chunk) < width)
                            *reinterpret_cast<uint4*>(first + (size_t)(own + x) * pitch + (F32 ? 64 * b : 0)) =
                                *reinterpret_cast<const uint4*>(sm + kOut + swz(own + x, chunk));
                }
            }
            if (PARTS == 3) arrive(B_SBFREE);
            return true;
        };
        for (int it = -1; it < nch; ++it) {
            if (it + 1 < nch && !split(it + 1) && STATE) break;
            if (!STATE && it >= 0 && !write_outputs(it)) break;
        }
        if (!STATE) named_barrier_sync(kBarOutputs, 320);
    } else {
        // ------------------------------------------------------------ the state: row R of dk, 64 columns a thread
        regs_inc<kRegsState>();
        const int R = tid - 32 * kWarpState;
        const size_t base = ((size_t)unit.seq * a.Hv + h) * dk * dv;
        const float* const init = STATE ? nullptr : ta.seg ? unit_state(ta, blockIdx.y, slot, h) : s.init ? s.init + base : nullptr;
        float* const final = STATE ? unit_state(ta, blockIdx.y, slot, h) : s.final && unit.last ? s.final + base : nullptr;
        // (rows past dk and columns past dv hold what the products leave there and go nowhere)
        float2 S[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) S[e] = make_float2(0.f, 0.f);
        if (init && R < dk) {
            if (s.init_t && !ta.seg) {
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    if (2 * e >= width) break;
                    const float* x = init + (size_t)(kHalf * z + 2 * e) * dk + R;
                    S[e] = make_float2(x[0], x[dk]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    if (2 * e >= width) break;
                    const float4 x = *reinterpret_cast<const float4*>(init + (size_t)R * dv + kHalf * z + 2 * e);
                    S[e] = make_float2(x.x, x.y);
                    S[e + 1] = make_float2(x.z, x.w);
                }
            }
        }
        auto write_sb = [&] {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                if (FINE) {
                    uint32_t y[4][2];
#pragma unroll
                    for (int e = 0; e < 4; ++e) split_bf16<2>(S[4 * c + e], y[e]);
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        *reinterpret_cast<uint4*>(sm + (p ? S_SLOW : S_SB) + swz(R, c)) = make_uint4(y[0][p], y[1][p], y[2][p], y[3][p]);
                } else {
                    *reinterpret_cast<uint4*>(sm + S_SB + swz(R, c)) =
                        make_uint4(pack_bf16(S[4 * c]), pack_bf16(S[4 * c + 1]), pack_bf16(S[4 * c + 2]), pack_bf16(S[4 * c + 3]));
                }
            }
            fence_proxy_async_smem();
            arrive(B_S);
        };
        bool ok = true;
        if (nch > 0) {
            if (!STATE) write_sb();
            ok = wait(B_GAMMA, 0);
        }
        for (int it = 0; ok && it < nch; ++it) {
            const int x = valid_of(it) == kC ? 0 : 2;
            const float2 ghi = make_float2(gamma[x], gamma[x]), glo = make_float2(gamma[x + 1], gamma[x + 1]);
            if (it + 1 == nch && !final) break;   // nobody needs the last state
            if (!(ok = wait(B_KV, it))) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t d[PARTS][16];
#pragma unroll
                for (int p = 0; p < PARTS; ++p) tmem_ld16(tl + T_KV + 64 * p + 16 * b, d[p]);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float2 y = as_float2(d[1][2 * e], d[1][2 * e + 1]);
                    if (PARTS == 3) y = add2(as_float2(d[PARTS - 1][2 * e], d[PARTS - 1][2 * e + 1]), y);
                    y = add2(y, as_float2(d[0][2 * e], d[0][2 * e + 1]));
                    S[8 * b + e] = fma2(ghi, S[8 * b + e], fma2(glo, S[8 * b + e], y));
                }
            }
            tc_fence_before();
            arrive(B_KVFREE);
            if (!STATE && it + 1 < nch) {
                // QS has read the copy of the state, and the outputs (with three parts) have passed through its place
                if (!(ok = wait(PARTS == 3 ? B_SBFREE : B_O, it))) break;
                write_sb();
            }
        }
        if (final && ok && R < dk) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                if (2 * e >= width) break;
                *reinterpret_cast<float4*>(final + (size_t)R * dv + kHalf * z + 2 * e) =
                    make_float4(S[e].x, S[e].y, S[e + 1].x, S[e + 1].y);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// SHORT: units of one chunk, which take the finer form, may be among the call's.  A kernel of its own for calls
// without them: the registers that the compiler gives to twelve forms in one cost the backward pass of two sequences
// of 8192 tokens 566 us instead of 540.
template <bool SHORT, bool REV, bool F32, int PARTS>
__device__ __forceinline__ void decay_tc_scan(const TcArgs& ta, Unit unit) {
    if (!SHORT && !unit_of(ta, slot_of(ta.a), REV, unit)) return;
    if (SHORT && unit.t1 - unit.t0 <= kC) decay_tc_body<REV, F32, PARTS, false, true>(ta, unit);
    else decay_tc_body<REV, F32, PARTS, false, false>(ta, unit);
}

template <bool SHORT>
__global__ void __launch_bounds__(kThreads, 1)
decay_tc_kernel(const __grid_constant__ TcArgs ta) {
    const DecayScan& s = ta.a.scan[blockIdx.y];
    Unit unit;
    if (SHORT && !unit_of(ta, slot_of(ta.a), s.reverse, unit)) return;
    if (s.out_f32) {   // a part of a sum over shared heads: no state is asked of such a scan
        if (s.reverse) decay_tc_scan<SHORT, true, true, 2>(ta, unit);
        else decay_tc_scan<SHORT, false, true, 2>(ta, unit);
    } else if (s.final) {
        if (s.reverse) decay_tc_scan<SHORT, true, false, 3>(ta, unit);
        else decay_tc_scan<SHORT, false, false, 3>(ta, unit);
    } else {
        if (s.reverse) decay_tc_scan<SHORT, true, false, 2>(ta, unit);
        else decay_tc_scan<SHORT, false, false, 2>(ta, unit);
    }
}

// Segments, first: what each adds to the state (the last one visited adds to none).
template <bool REV>
__device__ __forceinline__ void decay_tc_state(const TcArgs& ta) {
    Unit unit;
    if (unit_of(ta, slot_of(ta.a), REV, unit) && !unit.last) decay_tc_body<REV, false, 3, true, false>(ta, unit);
}
__global__ void __launch_bounds__(kThreads, 1)
decay_tc_state_kernel(const __grid_constant__ TcArgs ta) {
    if (ta.a.scan[blockIdx.y].reverse) decay_tc_state<true>(ta);
    else decay_tc_state<false>(ta);
}

// ------------------------------------------------------------------ host side
// [tokens, heads, d] bf16 tensor, token rows `stride` elements apart; box of 128 tokens x 1 head x 64 values (of a
// head of 32 the other 32 are filled with zeros), 128-byte swizzle.
cudaError_t make_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, const void* base, long long tokens,
                     int heads, int d, long long stride) {
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, kC};
    const cuuint32_t elem[3] = {1, 1, 1};
    const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, elem,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t set_attributes() {
    constexpr int kMaxDevices = 64;
    static std::mutex mu;
    static bool done[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(decay_tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(decay_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(decay_tc_state_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e == cudaSuccess) done[dev] = true;
    return e;
}

}  // namespace

cudaError_t launch_decay_tc(const SegArgs& seg, bool state_only) {
    const DecayArgs& a = seg.a;
    const auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
    if (!encode) return cudaErrorNotSupported;
    cudaError_t e = set_attributes();
    if (e != cudaSuccess) return e;
    TcArgs t;
    static_cast<SegArgs&>(t) = seg;
    for (int i = 0; i < a.num_scans; ++i) {
        const DecayScan& s = a.scan[i];
        Maps& m = t.maps[i];
        if ((e = make_map(encode, &m.q, s.q, a.tokens, a.Hv / s.q_div, a.dk, s.q_stride)) != cudaSuccess) return e;
        if ((e = make_map(encode, &m.k, s.k, a.tokens, a.Hv / s.k_div, a.dk, s.k_stride)) != cudaSuccess) return e;
        if ((e = make_map(encode, &m.v, s.v, a.tokens, a.Hv / s.v_div, a.dv, s.v_stride)) != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)((long long)t.slots * a.Hv * (a.dv > kHalf ? 2 : 1)), (unsigned)a.num_scans);
    if (state_only) decay_tc_state_kernel<<<grid, kThreads, kSmem, a.stream>>>(t);
    else if (a.cu || a.T <= kC) decay_tc_kernel<true><<<grid, kThreads, kSmem, a.stream>>>(t);
    else decay_tc_kernel<false><<<grid, kThreads, kSmem, a.stream>>>(t);
    return cudaGetLastError();
}

}  // namespace gdn
