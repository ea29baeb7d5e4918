// Gradients of the selective scan.  With p = dy silu(z), lam = dL/dh walked backwards,
//     lam_t = C_t p_t + a_{t+1} lam_{t+1},   dC = sum_d p h,   dB = sum_d lam dt u,   q = sum_n lam B,
//     w = lam a h_{t-1},   r = sum_n A w,   dA = sum_t dt w,   du = dt q + skip p,   d(dt) = u q + r,
//     d(delta) = d(dt) sigmoid(delta + bias),   dz = dy (sum_n C h + skip u) silu'(z)
// (w from a lam, which is the next lam).
//
// Every segment of tokens is a block's work on its own.  A first kernel walks it forwards from zero and leaves the state
// every K tokens, and what the segment adds to the state behind it and to the adjoint before it; launch_scan_join makes
// those the state before each segment and the adjoint behind it.  Then a block takes its segment's chunks of K tokens from
// the last to the first: each is walked forwards with its states in registers, then backwards.  Sums over a group's channels
// (dB, dC) leave as one partial sum a tile, sums over tokens (dA_log, dskip, dbias) as one a segment; the last kernel adds
// them in order.
//
// 2 x 8192 tokens of 4096 channels of 16 states, bf16: 1605 us (first walk 428, join 29, chunks 1113, sums 26).  Bound by
// instructions and shared memory together: a warp's token of two channels and four states a lane is about 220 instructions,
// 12 of them exchanges; issue slots 64 %, shared-memory pipe 61 %, fp32 pipe 45 %, at 166 registers (three blocks an SM;
// two 5 % slower, four spill and are 3 % slower).  HBM would take 139 us for each tensor once, some 380 us for the 2.6 GB
// that this method moves (u, delta, z and dy twice, the states before the chunks and the partial sums of B and C written and
// read), three exponentials a state and token 345 us.
// From 2857 us: raw rows by asynchronous copies, no bank conflicts, h kept rather than a h 1877; no state walked twice for
// the chunks' starts 1687; four blocks an SM in the first walk 1656; a chunk's sum of dt asked for ahead 1636; one launch of
// sums 1632; lam and dA under a condition in a sequence's last chunk, which leaves no register to spill, 1597 - 1605.  Not
// kept: eight states a lane with 6-token chunks (602 against 519 us for 2 x 2048 tokens: spills), a's held from one walk for
// the other (spills), segments in the chunks' kernel from states kept in shared memory (520 us), the chunks' rows found anew
// from the segment at every chunk (1634 us: spills).
#include <algorithm>

#include "norm_rows.cuh"
#include "scan_common.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace {

constexpr int kChunk = kScanChunk;   // tokens whose states a thread holds

// A thread's vectors of four channels: column c4, rows k0, k0 + kStep, ...
template <int N>
struct Own {
    static constexpr int kCols = ScanShape<N>::CH / 4, kStep = kScanThreads / kCols;
    int c4, k0;
    __device__ __forceinline__ explicit Own(int tid) : c4(tid % kCols * 4), k0(tid / kCols) {}
};

// ---------------------------------------------------------------- the segments' ends
// Each segment's contribution to the state behind it, from zero, and to the adjoint before it, sum_t (a_first .. a_t) C_t
// p_t; its sum of dt; and the state and the sum before each chunk but the first.
template <int N, typename T>
__global__ void __launch_bounds__(kScanThreads, 4) scan_ends_kernel(const __grid_constant__ ScanArgs a) {
    using S = ScanShape<N>;
    using O = Own<N>;
    constexpr int CH = S::CH, K = 16, VEC = (K * CH / 4 + kScanThreads - 1) / kScanThreads,
                  BC = (2 * K * N / 4 + kScanThreads - 1) / kScanThreads;
    static_assert(K % kChunk == 0, "tiles are whole chunks");
    __shared__ __align__(16) float2 s_dt[K][CH];
    __shared__ __align__(16) float s_p[K][CH];
    __shared__ __align__(16) float s_bc[2][K][N];
    const int tiles = a.G * ((a.D / a.G + CH - 1) / CH), slot = blockIdx.x / tiles;
    const ChannelTile tile = channel_tile(a.D, a.G, CH, blockIdx.x % tiles);
    ScanUnit u;
    if (!scan_unit_at(a.cu, a.T, a.nseq, a.seg, slot, u)) return;
    const int tid = threadIdx.x, len = (int)(u.t1 - u.t0);
    const ScanLane l = scan_lane<N>(tid);
    const O own(tid);
    const size_t DN = (size_t)a.D * N;
    float2 A2[2][2], h[2][2], lam[2][2], E[2][2];
    float sum_dt[2] = {0.f, 0.f};
    load_rates<N>(A2, a.A_log, tile, l);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            h[s][i] = lam[s][i] = all2(0.f);
            E[s][i] = all2(1.f);
        }
    const float4 bias = columns(a.dt_bias, tile, own.c4);
    const bool some = own.c4 < tile.n;
    // the thread's first vector of the next tile
    auto first = [&](const void* p, long long stride) {
        return static_cast<const T*>(p) + (u.t0 + own.k0) * stride + tile.d0 + own.c4;
    };
    const T *pu = first(a.u, a.u_stride), *pd = first(a.delta, a.delta_stride), *pg = first(a.gy, a.D),
            *pz = a.z ? first(a.z, a.z_stride) : nullptr;
    Raw4<T> ru[VEC], rd[VEC], rz[VEC], rg[VEC], rbc[BC];
    auto load = [&](int t) {   // the tiles in order
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const int k = own.k0 + v * O::kStep;
            const bool ok = some && t + k < len && k < K;
            const long long row = v * O::kStep;
            ru[v] = ok ? load4(pu + row * a.u_stride) : Raw4<T>::zero();
            rd[v] = ok ? load4(pd + row * a.delta_stride) : Raw4<T>::zero();
            rg[v] = ok ? load4(pg + row * a.D) : Raw4<T>::zero();
            if (pz) rz[v] = ok ? load4(pz + row * a.z_stride) : Raw4<T>::zero();
        }
        pu += K * a.u_stride;
        pd += K * a.delta_stride;
        pg += (long long)K * a.D;
        if (pz) pz += K * a.z_stride;
#pragma unroll
        for (int v = 0; v < BC; ++v) {
            const int i = tid + v * kScanThreads, which = i / (K * N / 4), k = i / (N / 4) % K, n = i % (N / 4) * 4;
            const T* p = static_cast<const T*>(which == 0 ? a.B : a.C) + (size_t)tile.g * N + n;
            const long long stride = which == 0 ? a.b_stride : a.c_stride;
            rbc[v] = which < 2 && t + k < len ? load4(p + (u.t0 + t + k) * stride) : Raw4<T>::zero();
        }
    };
    if (len > 0) load(0);
    for (int t = 0; t < len; t += K) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const int k = own.k0 + v * O::kStep;
            if (k >= K) break;
            form_dt(&s_dt[k][own.c4], ru[v].f(), rd[v].f(), bias, some && t + k < len);
            *reinterpret_cast<float4*>(&s_p[k][own.c4]) = pz ? gated4(rg[v].f(), rz[v].f()) : rg[v].f();
        }
#pragma unroll
        for (int v = 0; v < BC; ++v) {
            const int i = tid + v * kScanThreads, which = i / (K * N / 4), k = i / (N / 4) % K, n = i % (N / 4) * 4;
            if (which < 2) *reinterpret_cast<float4*>(&s_bc[which][k][n]) = rbc[v].f();
        }
        __syncthreads();
        if (t + K < len) load(t + K);
#pragma unroll 1
        for (int k0 = 0; k0 < K; k0 += kChunk) {
            if (t + k0 > 0 && t + k0 < len)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (l.ch[s] >= tile.n) continue;
                    const size_t row = scan_chunk_row(u) + (t + k0) / kChunk, d = tile.d0 + l.ch[s];
                    store_states(a.chunks + row * DN + d * N + l.n0, h[s]);
                    if (l.n0 == 0) a.chunk_dt[row * a.D + d] = sum_dt[s];
                }
#pragma unroll
            for (int k = k0; k < k0 + kChunk; ++k) {
                float2 B[2], C[2];
                load_states(B, &s_bc[0][k][l.n0]);
                load_states(C, &s_bc[1][k][l.n0]);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const float2 dd = s_dt[k][l.ch[s]];
                    const float p = s_p[k][l.ch[s]];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 e = decay(A2[s][i], dd.x);
                        h[s][i] = fma2(e, h[s][i], mul2(B[i], all2(dd.y)));
                        E[s][i] = mul2(E[s][i], e);
                        lam[s][i] = fma2(E[s][i], mul2(C[i], all2(p)), lam[s][i]);
                    }
                    sum_dt[s] += dd.x;
                }
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (l.ch[s] >= tile.n) continue;
        const size_t d = tile.d0 + l.ch[s];
        store_states(a.states + (size_t)slot * DN + d * N + l.n0, h[s]);
        store_states(a.adjoints + (size_t)slot * DN + d * N + l.n0, lam[s]);
        if (l.n0 == 0) a.sum_dt[(size_t)slot * a.D + d] = sum_dt[s];
    }
}

// ---------------------------------------------------------------- the gradients
// Four values; zeros where there is none.
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, bool ok, float) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, bool ok, __nv_bfloat16) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(ok ? 8 : 0) : "memory");
}
__device__ __forceinline__ void copies_done() {
    asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
}

// A stage holds a chunk as it is in memory: K tokens of u, delta, z, dy, B and C, and the state before it.  A thread reads
// back only what it copied itself.
template <int N, typename T>
struct Stages {
    using S = ScanShape<N>;
    float4 first[2][kScanThreads];   // the state before the segment
    float4 state[2][2][kScanThreads];
    T rows[2][4 * kChunk][S::CH];
    T bc_rows[2][2 * kChunk][N];
};

template <int N, typename T>
__global__ void __launch_bounds__(kScanThreads, 3) scan_bwd_kernel(const __grid_constant__ ScanArgs a) {
    using S = ScanShape<N>;
    using O = Own<N>;
    constexpr int L = S::L, P = S::P, CH = S::CH, K = kChunk, kRow = CH + 8;
    constexpr int TT = L < 4 ? 1 : 2;   // tokens whose sums over the lanes are finished together
    constexpr int VEC = (K * CH / 4 + kScanThreads - 1) / kScanThreads, BC = (2 * K * N / 4 + kScanThreads - 1) / kScanThreads;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Stages<N, T>& sm = *reinterpret_cast<Stages<N, T>*>(smem_raw);
    // arrays of their own, so that what is stored to one does not hold back the next token's loads from another
    __shared__ __align__(16) float2 s_dt[K][CH];                              // dt, dt u
    __shared__ __align__(16) float s_p[K][CH];
    __shared__ __align__(16) float s_bc[2][K][N];
    __shared__ __align__(16) float s_sums[3][K][kRow];                     // y, q, r
    __shared__ __align__(16) float s_red[kScanThreads / 32][K][2 * N];        // dB, dC of each warp
    const int tiles = a.G * ((a.D / a.G + CH - 1) / CH), slot = blockIdx.x / tiles, tile_id = blockIdx.x % tiles;
    const ChannelTile tile = channel_tile(a.D, a.G, CH, tile_id);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const ScanLane l = scan_lane<N>(tid);
    const O own(tid);
    const bool some = own.c4 < tile.n;
    const size_t DN = (size_t)a.D * N;
    ScanUnit u;
    if (!scan_unit_at(a.cu, a.T, a.nseq, a.seg, slot, u)) u.t0 = u.t1 = u.seq = 0, u.first = false;
    const int len = (int)(u.t1 - u.t0), chunks = (len + K - 1) / K;
    const size_t chunk_row = scan_chunk_row(u);
    float* const part_A = a.part_A + (size_t)slot * DN;
    float* const part_s = a.part_s + (size_t)slot * 2 * a.D + tile.d0;
    auto channel = [&](int s) { return (size_t)(tile.d0 + l.ch[s]); };
    auto take = [&](const float* p, int s, float2 (&x)[2]) {   // zeros where there is none
        x[0] = x[1] = all2(0.f);
        if (p && l.ch[s] < tile.n) load_states(x, p + channel(s) * N + l.n0);
    };
    auto put = [&](float* p, int s, const float2 (&x)[2]) {
        if (l.ch[s] < tile.n) store_states(p + channel(s) * N + l.n0, x);
    };

    float2 A2[2][2], lam[2][2], gA[2][2];
    load_rates<N>(A2, a.A_log, tile, l);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        gA[s][0] = gA[s][1] = all2(0.f);
        float2 x[2];
        take(len ? a.states + (size_t)slot * DN : nullptr, s, x);
        store_states(&sm.first[s][tid].x, x);
        take(len ? a.adjoints + (size_t)slot * DN : nullptr, s, lam[s]);
    }
    const float4 bias = columns(a.dt_bias, tile, own.c4), skip = columns(a.skip, tile, own.c4);
    float4 g_skip = make_float4(0.f, 0.f, 0.f, 0.f), g_bias = g_skip;

    // asks for the chunk at token t of the segment
    auto ask_rows = [&](int st, int x, const void* p, long long stride, int t) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const int k = own.k0 + v * O::kStep;
            if (k >= K) break;
            const bool ok = some && t + k < len;
            const T* from = static_cast<const T*>(p) + (ok ? (u.t0 + t + k) * stride + tile.d0 + own.c4 : 0);
            copy_async(tc::smem_u32(&sm.rows[st][x * K + k][own.c4]), from, ok, T{});
        }
    };
    auto ask = [&](int st, int t) {
        ask_rows(st, 0, a.u, a.u_stride, t);
        ask_rows(st, 1, a.delta, a.delta_stride, t);
        if (a.z) ask_rows(st, 2, a.z, a.z_stride, t);
        ask_rows(st, 3, a.gy, a.D, t);
#pragma unroll
        for (int v = 0; v < BC; ++v) {
            const int i = tid + v * kScanThreads, k = i / (N / 4), n = i % (N / 4) * 4;
            if (k >= 2 * K) break;
            const bool c = k >= K, ok = t + k % K < len;
            const T* from = static_cast<const T*>(c ? a.C : a.B) +
                            (ok ? (u.t0 + t + k % K) * (c ? a.c_stride : a.b_stride) + (size_t)tile.g * N + n : 0);
            copy_async(tc::smem_u32(&sm.bc_rows[st][k][n]), from, ok, T{});
        }
        const float* state = a.chunks + (chunk_row + t / K) * DN;
#pragma unroll
        for (int s = 0; s < 2; ++s) {   // nothing before the first chunk
            const bool ok = t > 0 && l.ch[s] < tile.n;
            copy_async(tc::smem_u32(&sm.state[st][s][tid]), ok ? state + channel(s) * N + l.n0 : a.A_log, ok, 0.f);
        }
    };

    float cum[2] = {0.f, 0.f};   // dt up to the chunk
    auto ask_cum = [&](int c) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
            cum[s] = c > 0 && l.ch[s] < tile.n ? a.chunk_dt[(chunk_row + c) * a.D + channel(s)] : 0.f;
    };
    if (chunks > 0) ask(0, (chunks - 1) * K), ask_cum(chunks - 1);
    for (int c = chunks - 1; c >= 0; --c) {
        const int t = c * K, tokens = min(K, len - t), st = (chunks - 1 - c) & 1;
        copies_done();
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const int k = own.k0 + v * O::kStep;
            if (k >= K) break;
            const float4 g = load4(&sm.rows[st][3 * K + k][own.c4]).f();
            form_dt(&s_dt[k][own.c4], load4(&sm.rows[st][k][own.c4]).f(), load4(&sm.rows[st][K + k][own.c4]).f(), bias,
                    some && k < tokens);
            *reinterpret_cast<float4*>(&s_p[k][own.c4]) = a.z ? gated4(g, load4(&sm.rows[st][2 * K + k][own.c4]).f()) : g;
        }
#pragma unroll
        for (int v = 0; v < BC; ++v) {
            const int i = tid + v * kScanThreads, k = i / (N / 4), n = i % (N / 4) * 4;
            if (k >= 2 * K) break;
            *reinterpret_cast<float4*>(&s_bc[0][k][n]) = load4(&sm.bc_rows[st][k][n]).f();
        }
        float2 hs[K][2][2], before[2][2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float2 f[2], x[2];
            load_states(f, &sm.first[s][tid].x);
            load_states(x, &sm.state[st][s][tid].x);
#pragma unroll
            for (int i = 0; i < 2; ++i) before[s][i] = fma2(decay(A2[s][i], cum[s]), f[i], x[i]);
        }
        __syncthreads();
        if (c > 0) ask(st ^ 1, t - K), ask_cum(c - 1);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float2 B[2];
            load_states(B, &s_bc[0][k][l.n0]);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const float2 dd = s_dt[k][l.ch[s]];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    hs[k][s][i] = fma2(decay(A2[s][i], dd.x), k ? hs[k ? k - 1 : 0][s][i] : before[s][i],
                                       mul2(B[i], all2(dd.y)));
            }
        }
        // the decays are formed again: held from here, they would take as many registers as the states
        asm volatile("" ::: "memory");
        float sum[3][TT];   // y, q, r of the lane's first channel
#pragma unroll
        for (int k = K - 1; k >= 0; --k) {
            float2 B[2], C[2], gB[2], gC[2];
            load_states(B, &s_bc[0][k][l.n0]);
            load_states(C, &s_bc[1][k][l.n0]);
            float part[3][2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const float2 dd = s_dt[k][l.ch[s]];
                const float p = s_p[k][l.ch[s]];
                float2 y, q, r;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 hh = hs[k][s][i], prev = k ? hs[k ? k - 1 : 0][s][i] : before[s][i];
                    lam[s][i] = fma2(C[i], all2(p), lam[s][i]);
                    gC[i] = s == 0 ? mul2(hh, all2(p)) : fma2(hh, all2(p), gC[i]);
                    gB[i] = s == 0 ? mul2(lam[s][i], all2(dd.y)) : fma2(lam[s][i], all2(dd.y), gB[i]);
                    y = i == 0 ? mul2(hh, C[i]) : fma2(hh, C[i], y);
                    q = i == 0 ? mul2(lam[s][i], B[i]) : fma2(lam[s][i], B[i], q);
                    const float2 down = mul2(lam[s][i], decay(A2[s][i], dd.x)), w = mul2(down, prev);
                    r = i == 0 ? mul2(w, A2[s][i]) : fma2(w, A2[s][i], r);
                    // behind the end too, dt = 0 leaves both as they are, but for 0 times an infinite state and a rate that
                    // is no number
                    if (k < tokens) {
                        lam[s][i] = down;
                        gA[s][i] = fma2(w, all2(dd.x), gA[s][i]);
                    }
                }
                part[0][s] = y.x + y.y;
                part[1][s] = q.x + q.y;
                part[2][s] = r.x + r.y;
            }
            // the next lane of the pair holds the channels in the other order: each gets its first one's sums
#pragma unroll
            for (int x = 0; x < 3; ++x) sum[x][k % TT] = part[x][0] + __shfl_xor_sync(0xffffffffu, part[x][1], P);
            if (k % TT == 0)
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    float s = transpose_sum<TT, 2 * P>(sum[x], lane);
#pragma unroll
                    for (int o = 2 * P * TT; o < 32; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
                    s_sums[x][k + lane / (2 * P) % TT][l.ch[0]] = s;
                }
            // sums over the pairs of the warp, values 2 j (dB) and 2 j + 1 (dC) of four states
            constexpr int R = 8 / (P < 8 ? P : 8);
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 b = gB[j / 2], g = gC[j / 2];
                v[2 * j] = j & 1 ? b.y : b.x;
                v[2 * j + 1] = j & 1 ? g.y : g.x;
            }
#pragma unroll
            for (int w = 8, x = 1; x < P && w > 1; w /= 2, x *= 2) {
                const bool up = lane & x;
#pragma unroll
                for (int i = 0; i < w / 2; ++i) {
                    const float mine = up ? v[2 * i + 1] : v[2 * i], theirs = up ? v[2 * i] : v[2 * i + 1];
                    v[i] = mine + __shfl_xor_sync(0xffffffffu, theirs, x);
                }
            }
#pragma unroll
            for (int x = 8; x < P; x *= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], x);
            if (P <= 8 || l.pair < 8)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int i = r * (8 / R) + l.pair % (8 / R);
                    s_red[warp][k][(i & 1) * N + l.n0 + i / 2] = v[r];
                }
        }
        __syncthreads();
        if (some)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const int k = own.k0 + v * O::kStep;
                if (k >= tokens) break;
                const long long row = u.t0 + t + k;
                const size_t d = tile.d0 + own.c4;
                auto raw = [&](int x) { return load4(&sm.rows[st][x * K + k][own.c4]).f(); };
                auto f4 = [&](const float* p) { return *reinterpret_cast<const float4*>(p); };
                const float4 x4 = raw(0), d4 = add4(raw(1), bias), g4 = raw(3), p4 = f4(&s_p[k][own.c4]);
                const float4 y4 = f4(&s_sums[0][k][own.c4]), q4 = f4(&s_sums[1][k][own.c4]), r4 = f4(&s_sums[2][k][own.c4]);
                const float4 ta = f4(&s_dt[k][own.c4].x), tb = f4(&s_dt[k][own.c4 + 2].x);
                float2 gu[2], gd[2], gs[2], gz[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    auto pick = [&](float4 f) { return e == 0 ? make_float2(f.x, f.y) : make_float2(f.z, f.w); };
                    const float2 x = pick(x4), p = pick(p4), q = pick(q4), sk = pick(skip);
                    const float2 dt = e == 0 ? make_float2(ta.x, ta.z) : make_float2(tb.x, tb.z);
                    gu[e] = fma2(dt, q, mul2(sk, p));
                    gd[e] = mul2(fma2(x, q, mul2(pick(r4), all2(kLn2))), logistic2(pick(d4)));
                    gs[e] = mul2(p, x);
                    if (a.z) {   // silu'(z) = s (1 + z (1 - s))
                        const float2 z = pick(raw(2)), sg = logistic2(z), full = fma2(sk, x, pick(y4));
                        gz[e] = mul2(mul2(pick(g4), full), mul2(sg, fma2(z, fma2(sg, all2(-1.f), all2(1.f)), all2(1.f))));
                    }
                }
                auto join = [](const float2 (&x)[2]) { return make_float4(x[0].x, x[0].y, x[1].x, x[1].y); };
                store4(static_cast<T*>(a.gu) + row * a.D + d, join(gu));
                store4(static_cast<T*>(a.gdelta) + row * a.D + d, join(gd));
                if (a.z) store4(static_cast<T*>(a.gz) + row * a.gz_stride + d, join(gz));
                g_skip = add4(g_skip, join(gs));
                g_bias = add4(g_bias, join(gd));
            }
        for (int i = tid; i < tokens * N / 2; i += kScanThreads) {
            const int k = i / (N / 2), n = i % (N / 2) * 4;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kScanThreads / 32; ++w) s = add4(s, *reinterpret_cast<const float4*>(&s_red[w][k][n]));
            *reinterpret_cast<float4*>(a.part_bc + ((size_t)tile_id * a.tokens + u.t0 + t + k) * 2 * N + n) = s;
        }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        put(part_A, s, gA[s]);
        if (!a.gh0 || !u.first) continue;
        // an empty sequence's initial state is its final one
        if (len == 0) take(a.gh ? a.gh + (size_t)u.seq * DN : nullptr, s, lam[s]);
        put(a.gh0 + (size_t)u.seq * DN, s, lam[s]);
    }
    // the threads with the same channels, in order
    float4* const fold = &sm.state[0][0][0];
    __syncthreads();
    fold[2 * tid] = g_skip;
    fold[2 * tid + 1] = g_bias;
    __syncthreads();
    for (int i = tid; i < 2 * O::kCols; i += kScanThreads) {
        const int c = i >> 1;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x = c; x < kScanThreads; x += O::kCols) s = add4(s, fold[2 * x + (i & 1)]);
        if (c * 4 < tile.n) *reinterpret_cast<float4*>(part_s + (i & 1) * a.D + c * 4) = s;
    }
}

// The partial sums, added in order.  Blocks below bc_blocks: dB and dC of a token over the tiles of each group, a vector of
// four a thread.  The others: dA_log = A sum dA, dskip and dbias over the segments, vectors of four columns of the slots'
// rows of D N + 2 D sums, eight threads a vector.
constexpr int kSumCols = 32, kSumRows = 8;
template <typename T>
__device__ __forceinline__ void bc_sums(const ScanArgs& a, int tiles_per_group) {
    const int per = a.G * a.N / 2;   // vectors of a token
    const long long i = (long long)blockIdx.x * (kSumCols * kSumRows) + threadIdx.x, t = i / per;
    if (t >= a.tokens) return;
    if (a.cu) {   // a token of no sequence has no partial sums
        long long s0, s1, e0, e1;
        seq_range(a.cu, 0, a.T, s0, s1);
        seq_range(a.cu, a.nseq - 1, a.T, e0, e1);
        if (t < s0 || t >= e1) return;
    }
    const int j = (int)(i % per), g = j / (a.N / 2), n = j % (a.N / 2) * 4;
    const float* p = a.part_bc + ((size_t)g * tiles_per_group * a.tokens + t) * 2 * a.N + n;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int x = 0; x < tiles_per_group; ++x) s = add4(s, *reinterpret_cast<const float4*>(p + (size_t)x * a.tokens * 2 * a.N));
    const bool is_c = n >= a.N;
    T* to = static_cast<T*>(is_c ? a.gC : a.gB) + t * (is_c ? a.gc_stride : a.gb_stride);
    store4(to + (size_t)g * a.N + (is_c ? n - a.N : n), s);
}
template <typename T>
__global__ void __launch_bounds__(kSumCols * kSumRows) scan_sums_kernel(const __grid_constant__ ScanArgs a, int tiles_per_group,
                                                                       unsigned bc_blocks) {
    if (blockIdx.x < bc_blocks) {
        bc_sums<T>(a, tiles_per_group);
        return;
    }
    __shared__ float4 red[kSumRows][kSumCols];
    const int x = threadIdx.x % kSumCols, y = threadIdx.x / kSumCols;
    const size_t DN = (size_t)a.D * a.N, c = ((size_t)(blockIdx.x - bc_blocks) * kSumCols + x) * 4;
    const bool rate = c < DN, any = c < DN + 2 * a.D;
    const float* p = rate ? a.part_A + c : a.part_s + (c - DN);
    const size_t row = rate ? DN : 2 * (size_t)a.D;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (any)
#pragma unroll 4
        for (int r = y; r < a.slots; r += kSumRows) s = add4(s, *reinterpret_cast<const float4*>(p + r * row));
    red[y][x] = s;
    __syncthreads();
    if (y != 0 || !any) return;
#pragma unroll
    for (int r = 1; r < kSumRows; ++r) s = add4(s, red[r][x]);
    if (rate) {
        if (!a.gA) return;
        const float4 l = *reinterpret_cast<const float4*>(a.A_log + c);
        auto rate = [](float A_log) {   // finite, as in the walk: no state is left there, and the sum it takes is 0
            const float A = -expf(A_log);
            return A < -3e38f ? -3e38f : A;
        };
        *reinterpret_cast<float4*>(a.gA + c) = make_float4(rate(l.x) * s.x, rate(l.y) * s.y, rate(l.z) * s.z, rate(l.w) * s.w);
    } else {
        float* to = c < DN + a.D ? a.gskip : a.gbias;
        if (to) *reinterpret_cast<float4*>(to + (c < DN + a.D ? c - DN : c - DN - a.D)) = s;
    }
}

template <int N, typename T>
cudaError_t bwd_typed(const ScanArgs& a) {
    using S = ScanShape<N>;
    cudaError_t e = allow_smem<scan_bwd_kernel<N, T>>(sizeof(Stages<N, T>));
    if (e != cudaSuccess) return e;
    const int per_group = (a.D / a.G + S::CH - 1) / S::CH;
    const unsigned blocks = (unsigned)((long long)a.slots * a.G * per_group);
    scan_ends_kernel<N, T><<<blocks, kScanThreads, 0, a.stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess || (e = launch_scan_join(a, true)) != cudaSuccess) return e;
    scan_bwd_kernel<N, T><<<blocks, kScanThreads, sizeof(Stages<N, T>), a.stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    constexpr int kThreads = kSumCols * kSumRows;
    const long long bc = ((long long)a.tokens * a.G * N / 2 + kThreads - 1) / kThreads;
    const long long cols = ((long long)a.D * N + 2 * a.D) / 4;
    const unsigned blocks_of_sums = (unsigned)(bc + (cols + kSumCols - 1) / kSumCols);
    scan_sums_kernel<T><<<blocks_of_sums, kThreads, 0, a.stream>>>(a, per_group, (unsigned)bc);
    return cudaGetLastError();
}
template <typename T>
cudaError_t bwd_n(const ScanArgs& a) {
    switch (a.N) {
        case 8: return bwd_typed<8, T>(a);
        case 16: return bwd_typed<16, T>(a);
        case 32: return bwd_typed<32, T>(a);
        case 64: return bwd_typed<64, T>(a);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

ScanBwdLayout scan_bwd_layout(long long tokens, int D, int G, int N, int nseq) {
    ScanBwdLayout l{};
    const int ch = 2 * kScanThreads / (N / 4);
    const long long tiles = (long long)G * ((D / G + ch - 1) / ch);
    // some 4000 blocks, nine for each place on an SM
    const long long seg = (tokens * tiles / 4000 + kScanMinSegment - 1) / kScanMinSegment * kScanMinSegment;
    l.seg = (int)std::min(512LL, std::max((long long)kScanMinSegment, seg));
    l.slots = tokens / l.seg + nseq;
    size_t at = 0;
    auto place = [&](size_t floats) {
        const size_t p = at;
        at += (floats * 4 + 255) / 256 * 256;
        return p;
    };
    const size_t DN = (size_t)D * N, slots = (size_t)l.slots;
    place(slots * DN);   // the states
    l.adjoints = place(slots * DN);
    l.sum_dt = place(slots * D);
    const size_t rows = (size_t)(tokens / kChunk + nseq);
    l.chunks = place(rows * DN);
    l.chunk_dt = place(rows * D);
    l.part_A = place(slots * DN);
    l.part_s = place(slots * 2 * D);
    l.part_bc = place((size_t)tiles * tokens * 2 * N);
    l.total = at;
    return l;
}

cudaError_t launch_scan_bwd(const ScanArgs& a) {
    return a.dtype == GDN_BF16 ? bwd_n<__nv_bfloat16>(a) : bwd_n<float>(a);
}

}  // namespace gdn
