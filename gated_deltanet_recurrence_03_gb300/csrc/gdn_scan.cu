// The selective state space scan: per sequence, channel d of group g(d) and state n, with dt = softplus(delta + bias)
// and A = -exp(A_log),
//     h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t,      y_t = (sum_n C_t h_t + skip u_t) silu(z_t).
//
// Per tile of K tokens a block forms dt and dt u of its channels and B, C in fp32 in shared memory, walks the tile with the
// states in registers, and applies skip and gate to the sums.  A state and token costs one exponential, 2 fp32 pairs of
// operations and its share of the tile's reads; those, not HBM, bound the prompt: 2 x 8192 tokens of 4096 channels of 16
// states, bf16, 357 us, where HBM would take 79 and the exponentials alone (32 a clock and SM, measured) 115 us.  What is
// left: 512 warps of two channels a lane are all there are, one for each scheduler of 128 SMs, and a warp of its own runs
// at 45 % of what its pipes take (74 cycles a token against 33 instructions); the helpers' instructions come on top.  From
// 798 us: dt by a packed polynomial and helpers apart from the walk 516, two channels a lane 409, registers for 16 tokens
// 373, for 32 tokens 357.  One channel a lane, twice the warps: 391 us, shared-memory reads.
#include <algorithm>

#include "norm_rows.cuh"
#include "scan_common.cuh"

namespace gdn {
namespace {

// Per-thread shares of a tile of K tokens by CH channels among M threads: 4-channel vectors, and 4-state vectors of B and C.
template <int N, int K, int M>
struct Share {
    static constexpr int kVecs = (K * ScanShape<N>::CH / 4 + M - 1) / M, kBC = (2 * K * N / 4 + M - 1) / M;
};
struct Rows {
    const void* p;
    long long stride;
};

// Vectors of the tile's tensors as loaded, from the thread's first one on; zeros past the end and where there is none.
template <typename T>
struct Walk {
    const T* p;       // the thread's first vector of the tile, or nullptr
    int step;         // elements between its vectors (a row stride is at most 2^24)
};
template <int CH, int M, typename T>
__device__ __forceinline__ Walk<T> walk_of(Rows src, int d0, long long t0, int channels, int tid) {
    const int k = tid / (CH / 4), c = tid % (CH / 4) * 4;
    const T* p = static_cast<const T*>(src.p);
    return {p && c < channels ? p + (t0 + k) * src.stride + d0 + c : nullptr, (int)src.stride * (M / (CH / 4))};
}
template <int CH, int M, typename T, int V>
__device__ __forceinline__ void load_rows(Raw4<T> (&x)[V], const Walk<T>& w, int tokens, int tid) {
#pragma unroll
    for (int v = 0; v < V; ++v)
        x[v] = w.p && tid / (CH / 4) + v * (M / (CH / 4)) < tokens ? load4(w.p + (size_t)v * w.step) : Raw4<T>::zero();
}
// B, then C (C.p may be nullptr), of group g.
template <int K, int N, int M, typename T, int V>
__device__ __forceinline__ void load_bc(Raw4<T> (&x)[V], Rows B, Rows C, int g, long long t0, int tokens, int tid) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = tid + v * M, which = i / (K * N / 4), k = i / (N / 4) % K, n = i % (N / 4) * 4;
        const Rows r = which == 0 ? B : C;
        x[v] = which < 2 && k < tokens && r.p ? load4(static_cast<const T*>(r.p) + (t0 + k) * r.stride + (size_t)g * N + n)
                                              : Raw4<T>::zero();
    }
}
template <int K, int CH, int M, typename T, int V>
__device__ __forceinline__ void form_tile_dt(float2 (&to)[K][CH], const Raw4<T> (&u)[V], const Raw4<T> (&delta)[V], float4 bias,
                                             int tokens, int channels, int tid) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = tid + v * M, k = i / (CH / 4), c = i % (CH / 4) * 4;
        if (k >= K) break;
        form_dt(&to[k][c], u[v].f(), delta[v].f(), bias, k < tokens && c < channels);
    }
}
template <int K, int N, int M, typename T, int V>
__device__ __forceinline__ void form_bc(float (&to)[2][K][N], const Raw4<T> (&x)[V], int tid) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = tid + v * M, which = i / (K * N / 4), k = i / (N / 4) % K, n = i % (N / 4) * 4;
        if (which < 2) *reinterpret_cast<float4*>(&to[which][k][n]) = x[v].f();
    }
}
// Each segment's own contribution to the state, from zero, and its sum of dt.  Issue slots 64 %, special functions 55 %, the
// fp32 pipe 58 % of their rates: 159 us for 46,547 packed tokens of 1024 channels (199 us in half as many segments).
template <int N, typename T>
__global__ void __launch_bounds__(kScanThreads) scan_state_kernel(const __grid_constant__ ScanArgs a) {
    constexpr int CH = ScanShape<N>::CH, K = 16, M = kScanThreads;
    using S = Share<N, K, M>;
    __shared__ __align__(16) float2 s_dt[K][CH];
    __shared__ __align__(16) float s_bc[2][K][N];
    const int tiles = a.G * ((a.D / a.G + CH - 1) / CH), slot = blockIdx.x / tiles;
    const ChannelTile tile = channel_tile(a.D, a.G, CH, blockIdx.x % tiles);
    ScanUnit u;
    if (!scan_unit_at(a.cu, a.T, a.nseq, a.seg, slot, u)) return;
    if (u.last) return;   // nothing reads it
    const int tid = threadIdx.x, c4 = tid % (CH / 4) * 4;
    const ScanLane l = scan_lane<N>(tid);
    const size_t DN = (size_t)a.D * N;
    float2 A2[2][2], h[2][2];
    float sum_dt[2] = {0.f, 0.f};
    load_rates<N>(A2, a.A_log, tile, l);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) h[s][i] = all2(0.f);
    const float4 bias = columns(a.dt_bias, tile, c4);
    const Rows B{a.B, a.b_stride}, C{nullptr, 0};
    Raw4<T> ru[S::kVecs], rd[S::kVecs], rbc[S::kBC];
    auto load = [&](long long t0) {
        const int tokens = (int)min((long long)K, u.t1 - t0);
        auto get = [&](auto& x, const void* p, long long stride) {
            load_rows<CH, M>(x, walk_of<CH, M, T>(Rows{p, stride}, tile.d0, t0, tile.n, tid), tokens, tid);
        };
        get(ru, a.u, a.u_stride);
        get(rd, a.delta, a.delta_stride);
        load_bc<K, N, M>(rbc, B, C, tile.g, t0, tokens, tid);
    };
    load(u.t0);
    for (long long t0 = u.t0; t0 < u.t1; t0 += K) {
        const int tokens = (int)min((long long)K, u.t1 - t0);
        form_tile_dt<K, CH, M>(s_dt, ru, rd, bias, tokens, tile.n, tid);
        form_bc<K, N, M>(s_bc, rbc, tid);
        __syncthreads();
        if (t0 + K < u.t1) load(t0 + K);
#pragma unroll 4
        for (int k = 0; k < K; ++k) {
            float2 B2[2];
            load_states(B2, &s_bc[0][k][l.n0]);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const float2 dd = s_dt[k][l.ch[s]];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 e = decay(A2[s][i], dd.x);
                    h[s][i] = fma2(e, h[s][i], mul2(B2[i], all2(dd.y)));
                }
                sum_dt[s] += dd.x;
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (l.ch[s] >= tile.n) continue;
        const size_t d = tile.d0 + l.ch[s];
        store_states(a.states + (size_t)slot * DN + d * N + l.n0, h[s]);
        if (l.n0 == 0) a.sum_dt[(size_t)slot * a.D + d] = sum_dt[s];
    }
}

// The outputs.  Four warps walk the states; others form the next tile's dt, dt u, B and C in shared memory and finish the
// last one's outputs meanwhile (one barrier a tile), so that the walk waits for neither.  Where whole sequences are walked
// (SEG false) few blocks are there and the walk itself is what takes the time: registers for a whole tile's instructions in
// any order, eight warps of helpers (four: 102 against 98 us for 2 x 2048 tokens).  Segments fill the GPU: two blocks an SM
// with bf16 (fp32 vectors would not fit the registers), four warps of helpers (46,547 packed tokens, all three launches: 394
// us; one block of twelve warps an SM 428; three blocks 429, registers spilled).
__host__ __device__ constexpr int helpers(bool seg) { return seg ? 128 : 256; }
template <int N>
struct MainShape {
    static constexpr int K = N == 8 ? 16 : 32, CH = ScanShape<N>::CH;
    static constexpr int kRow = CH + (N == 8 ? 0 : 256 / N);   // floats of a row of sums: no bank conflicts
    static constexpr size_t kSums = sizeof(float) * 2 * K * kRow;
};
template <int N, typename T, bool SEG>
__global__ void __launch_bounds__(kScanThreads + helpers(SEG), SEG && sizeof(T) == 2 ? 2 : 1)
scan_main_kernel(const __grid_constant__ ScanArgs a) {
    constexpr int L = ScanShape<N>::L, CH = ScanShape<N>::CH, P = ScanShape<N>::P;
    constexpr int K = MainShape<N>::K, M = helpers(SEG), kRow = MainShape<N>::kRow;
    using S = Share<N, K, M>;
    // arrays of their own, so that what is stored to the sums does not hold back the next tokens' loads
    __shared__ __align__(16) float2 s_dt[2][K][CH];
    __shared__ __align__(16) float s_bc[2][2][K][N];
    extern __shared__ __align__(16) uint8_t smem[];
    float(*const s_y)[K][kRow] = reinterpret_cast<float(*)[K][kRow]>(smem);
    const int tiles = a.G * ((a.D / a.G + CH - 1) / CH), slot = blockIdx.x / tiles;
    const ChannelTile tile = channel_tile(a.D, a.G, CH, blockIdx.x % tiles);
    ScanUnit u;
    if (!scan_unit_at(a.cu, a.T, a.nseq, a.seg, slot, u)) return;
    const int n = (int)((u.t1 - u.t0 + K - 1) / K);
    const size_t DN = (size_t)a.D * N;
    if (threadIdx.x >= kScanThreads) {
        const int tid = threadIdx.x - kScanThreads, c4 = tid % (CH / 4) * 4;
        const float4 bias = columns(a.dt_bias, tile, c4), skip = columns(a.skip, tile, c4);
        const Rows B{a.B, a.b_stride}, C{a.C, a.c_stride};
        Raw4<T> ru[S::kVecs], rd[S::kVecs], rz[S::kVecs], rbc[S::kBC];   // the next tile's
        Raw4<T> cu[S::kVecs], cz[S::kVecs], pu[S::kVecs], pz[S::kVecs];  // of the tile that is walked, of the last one
        auto tokens_of = [&](int i) { return (int)min((long long)K, u.t1 - u.t0 - (long long)i * K); };
        Walk<T> wu = walk_of<CH, M, T>(Rows{a.u, a.u_stride}, tile.d0, u.t0, tile.n, tid);
        Walk<T> wd = walk_of<CH, M, T>(Rows{a.delta, a.delta_stride}, tile.d0, u.t0, tile.n, tid);
        Walk<T> wz = walk_of<CH, M, T>(Rows{a.z, a.z_stride}, tile.d0, u.t0, tile.n, tid);
        T* out = static_cast<T*>(a.y) + (u.t0 + tid / (CH / 4)) * a.D + tile.d0 + c4;
        auto load = [&](int i) {   // the tiles in order
            const int tokens = tokens_of(i);
            load_rows<CH, M>(ru, wu, tokens, tid);
            load_rows<CH, M>(rd, wd, tokens, tid);
            load_rows<CH, M>(rz, wz, tokens, tid);
            load_bc<K, N, M>(rbc, B, C, tile.g, u.t0 + (long long)i * K, tokens, tid);
            auto next = [](Walk<T>& w, long long stride) { if (w.p) w.p += K * stride; };
            next(wu, a.u_stride);
            next(wd, a.delta_stride);
            next(wz, a.z_stride);
        };
        auto form = [&](int i) {
            form_tile_dt<K, CH, M>(s_dt[i & 1], ru, rd, bias, tokens_of(i), tile.n, tid);
            form_bc<K, N, M>(s_bc[i & 1], rbc, tid);
        };
        auto finish = [&](int i, const Raw4<T> (&fu)[S::kVecs], const Raw4<T> (&fz)[S::kVecs]) {
            const int tokens = c4 < tile.n ? tokens_of(i) : 0;
#pragma unroll
            for (int v = 0; v < S::kVecs; ++v) {
                const int k = tid / (CH / 4) + v * (M / (CH / 4));
                if (k >= tokens) break;
                float4 y = *reinterpret_cast<const float4*>(&s_y[i & 1][k][c4]);
                const float4 x = fu[v].f();
                const float2 ya = fma2(make_float2(skip.x, skip.y), make_float2(x.x, x.y), make_float2(y.x, y.y));
                const float2 yb = fma2(make_float2(skip.z, skip.w), make_float2(x.z, x.w), make_float2(y.z, y.w));
                y = make_float4(ya.x, ya.y, yb.x, yb.y);
                if (a.z) y = gated4(y, fz[v].f());
                store4(out + (size_t)v * (M / (CH / 4)) * a.D, y);
            }
            out += (size_t)K * a.D;
        };
        auto keep = [&]() {
#pragma unroll
            for (int v = 0; v < S::kVecs; ++v) {
                pu[v] = cu[v];
                pz[v] = cz[v];
                cu[v] = ru[v];
                cz[v] = rz[v];
            }
        };
        if (n > 0) {
            load(0);
            form(0);
            keep();
            if (n > 1) load(1);
        }
        __syncthreads();
        for (int i = 0; i < n; ++i) {
            if (i + 1 < n) form(i + 1);
            keep();   // pu, pz: tile i
            if (i + 2 < n) load(i + 2);
            __syncthreads();
            finish(i, pu, pz);
        }
        return;
    }
    const ScanLane l = scan_lane<N>(threadIdx.x);
    float2 A2[2][2], h[2][2];
    load_rates<N>(A2, a.A_log, tile, l);
    const float* from = SEG ? a.states + (size_t)slot * DN : a.h0 ? a.h0 + (size_t)u.seq * DN : nullptr;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        h[s][0] = h[s][1] = all2(0.f);
        if (from && l.ch[s] < tile.n) load_states(h[s], from + (size_t)(tile.d0 + l.ch[s]) * N + l.n0);
    }
    __syncthreads();
    constexpr int TT = L / 2;              // tokens whose sums over the lanes are finished together
    constexpr int U = SEG ? 8 : K;                   // tokens between which instructions can be moved: no store before a load
    for (int i = 0; i < n; ++i) {
        const float2(*dt)[CH] = s_dt[i & 1];
        const float(*bc)[K][N] = s_bc[i & 1];
#pragma unroll 1
        for (int k0 = 0; k0 < K; k0 += U) {
            float out[U / TT];
#pragma unroll
            for (int j = 0; j < U; j += TT) {
                float sum[TT];
#pragma unroll
                for (int e = 0; e < TT; ++e) {
                    const int k = k0 + j + e;
                    float2 B2[2], C2[2];
                    load_states(B2, &bc[0][k][l.n0]);
                    load_states(C2, &bc[1][k][l.n0]);
                    float part[2];
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const float2 dd = dt[k][l.ch[s]];
                        float2 y;
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            h[s][x] = fma2(decay(A2[s][x], dd.x), h[s][x], mul2(B2[x], all2(dd.y)));
                            y = x == 0 ? mul2(h[s][x], C2[x]) : fma2(h[s][x], C2[x], y);
                        }
                        part[s] = y.x + y.y;
                    }
                    // the next lane of the pair holds the channels in the other order: each gets its first one's sum
                    sum[e] = part[0] + __shfl_xor_sync(0xffffffffu, part[1], P);
                }
                out[j / TT] = transpose_sum<TT, 2 * P>(sum, threadIdx.x);
            }
#pragma unroll
            for (int j = 0; j < U; j += TT) s_y[i & 1][k0 + j + threadIdx.x / (2 * P) % TT][l.ch[0]] = out[j / TT];
        }
        __syncthreads();
    }
    if (a.h_final && u.last)
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (l.ch[s] < tile.n) store_states(a.h_final + (size_t)u.seq * DN + (size_t)(tile.d0 + l.ch[s]) * N + l.n0, h[s]);
}

// The segments' contributions, in place: states to the state before each segment, adjoints (blockIdx.y 1) to the
// adjoint a_{t+1} lam_{t+1} behind it.
__global__ void __launch_bounds__(kScanThreads) scan_join_kernel(const __grid_constant__ ScanArgs a) {
    const size_t DN = (size_t)a.D * a.N;
    const int blocks = (int)((DN / 4 + kScanThreads - 1) / kScanThreads), seq = blockIdx.x / blocks;
    const size_t at = ((size_t)(blockIdx.x % blocks) * kScanThreads + threadIdx.x) * 4;
    if (at >= DN) return;
    const int d = (int)(at / a.N);
    long long s0, s1;
    seq_range(a.cu, seq, a.T, s0, s1);
    const long long base = s0 / a.seg + seq, n = max(1LL, (s1 - s0 + a.seg - 1) / a.seg);
    const float4 l = *reinterpret_cast<const float4*>(a.A_log + at);
    const float A[4] = {rate2(l.x), rate2(l.y), rate2(l.z), rate2(l.w)};
    const bool adj = blockIdx.y == 1;
    const float* init = adj ? a.gh : a.h0;
    float4 h = init ? *reinterpret_cast<const float4*>(init + seq * DN + at) : make_float4(0.f, 0.f, 0.f, 0.f);
    float* s = (adj ? a.adjoints : a.states) + at;
    constexpr int W = 8;   // segments whose contributions are loaded ahead
    for (long long j0 = 0; j0 < n; j0 += W) {
        float4 x[W];
        float dt[W];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const size_t slot = base + (adj ? n - 1 - j0 - w : j0 + w);
            if (j0 + w < n - 1) {   // the last one's is not needed
                x[w] = *reinterpret_cast<const float4*>(s + slot * DN);
                dt[w] = a.sum_dt[slot * a.D + d];
            }
        }
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (j0 + w >= n) break;
            const size_t slot = base + (adj ? n - 1 - j0 - w : j0 + w);
            *reinterpret_cast<float4*>(s + slot * DN) = h;
            if (j0 + w < n - 1)
                h = make_float4(fmaf(decay(A[0], dt[w]), h.x, x[w].x), fmaf(decay(A[1], dt[w]), h.y, x[w].y),
                                fmaf(decay(A[2], dt[w]), h.z, x[w].z), fmaf(decay(A[3], dt[w]), h.w, x[w].w));
        }
    }
}

// One token for each of the rows, in place on the states: eight states a lane, so that the functions of dt and of the gate,
// which the L lanes of a channel all form, weigh little.  A block has a tile of channels and every `splits`-th row; what a
// row needs is asked for while the one before it is worked on.  256 rows of 4096 channels of 16 states, bf16: 26.9 us a
// call, 5.3 TB/s, 0.78 of the copy bandwidth (four states a lane 34.8 us, held by its instructions; without rows ahead
// 36 - 43 us; two or more rows ahead spill: 41 us and more).
template <typename T>
struct StepRow {
    float4 h[2];
    Raw4<T> b[2], c[2];
    T u, delta, z;
    float* at;   // the lane's states, or nullptr
};
constexpr int kStepStates = 8, kStepBlocks = 6;   // states a lane, blocks an SM
template <int N, typename T>
__global__ void __launch_bounds__(kScanThreads, kStepBlocks)
scan_step_kernel(const __grid_constant__ ScanStepArgs a, int splits) {
    constexpr int L = N / kStepStates, CH = kScanThreads / L;
    const int tiles = (a.D + CH - 1) / CH, split = blockIdx.x / tiles;
    const int d = blockIdx.x % tiles * CH + threadIdx.x / L, n0 = threadIdx.x % L * kStepStates;
    const bool own = d < a.D;   // D is a multiple of 8, a warp's channels may not be
    auto slot_of = [&](int row) {   // -1: no such row, or one without a request
        const int slot = row < a.rows ? a.slots ? a.slots[row] : row : -1;
        return slot < a.num_slots ? slot : -1;
    };
    const size_t g = own ? d / (a.D / a.G) : 0;
    auto load = [&](int row, int slot) {
        StepRow<T> x;
        x.at = own && slot >= 0 ? a.h + ((size_t)slot * a.D + d) * N + n0 : nullptr;
        if (x.at) {
            const T* b = static_cast<const T*>(a.B) + row * a.b_stride + g * N + n0;
            const T* c = static_cast<const T*>(a.C) + row * a.c_stride + g * N + n0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x.h[i] = __ldcs(reinterpret_cast<const float4*>(x.at) + i);
                x.b[i] = load4(b + 4 * i);
                x.c[i] = load4(c + 4 * i);
            }
            x.u = static_cast<const T*>(a.u)[row * a.u_stride + d];
            x.delta = static_cast<const T*>(a.delta)[row * a.delta_stride + d];
            if (a.z) x.z = static_cast<const T*>(a.z)[row * a.z_stride + d];
        }
        return x;
    };
    StepRow<T> next = load(split, slot_of(split));
    int slot = slot_of(split + splits);
    float2 A[4];
    const float bias = own && a.dt_bias ? a.dt_bias[d] : 0.f, skip = own && a.skip ? a.skip[d] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        A[i] = all2(0.f);
        if (own) {
            const float2 l = *reinterpret_cast<const float2*>(a.A_log + (size_t)d * N + n0 + 2 * i);
            A[i] = make_float2(rate2(l.x), rate2(l.y));
        }
    }
    for (int row = split; row < a.rows; row += splits) {
        const StepRow<T> x = next;
        next = load(row + splits, slot);
        slot = slot_of(row + 2 * splits);
        float s = 0.f;
        if (x.at) {
            const float u = to_f32(x.u), dt = softplus2(all2(to_f32(x.delta) + bias)).x, w = dt * u;
            float2 y = all2(0.f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 b = x.b[i].f(), c = x.c[i].f();
                const float2 p = fma2(decay(A[2 * i], dt), make_float2(x.h[i].x, x.h[i].y),
                                      mul2(make_float2(b.x, b.y), all2(w)));
                const float2 q = fma2(decay(A[2 * i + 1], dt), make_float2(x.h[i].z, x.h[i].w),
                                      mul2(make_float2(b.z, b.w), all2(w)));
                __stcs(reinterpret_cast<float4*>(x.at) + i, make_float4(p.x, p.y, q.x, q.y));
                y = fma2(p, make_float2(c.x, c.y), fma2(q, make_float2(c.z, c.w), y));
            }
            s = y.x + y.y;
            if (n0 == 0) s = fmaf(skip, u, s);
        }
#pragma unroll
        for (int o = L / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (!own || n0) continue;
        if (a.z && x.at) {
            const float z = to_f32(x.z);
            s *= z * logistic_f(z);
        }
        static_cast<T*>(a.y)[(size_t)row * a.D + d] = from_f32<T>(s);
    }
}

template <int N>
unsigned blocks_of(const ScanArgs& a) {
    return (unsigned)((long long)a.slots * a.G * ((a.D / a.G + ScanShape<N>::CH - 1) / ScanShape<N>::CH));
}
template <int N, typename T, bool SEG>
cudaError_t main_typed(const ScanArgs& a) {
    constexpr size_t smem = MainShape<N>::kSums;
    const cudaError_t e = allow_smem<scan_main_kernel<N, T, SEG>>(smem);
    if (e != cudaSuccess) return e;
    scan_main_kernel<N, T, SEG><<<blocks_of<N>(a), kScanThreads + helpers(SEG), smem, a.stream>>>(a);
    return cudaGetLastError();
}

template <int N, typename T>
cudaError_t fwd_typed(const ScanArgs& a) {
    if (!a.seg) return main_typed<N, T, false>(a);
    scan_state_kernel<N, T><<<blocks_of<N>(a), kScanThreads, 0, a.stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_scan_join(a, false);
    return e == cudaSuccess ? main_typed<N, T, true>(a) : e;
}
// Rows are split over the blocks that fit the 152 SMs, each with a few of them where there are more.
template <int N, typename T>
cudaError_t step_typed(const ScanStepArgs& a) {
    constexpr int CH = kScanThreads / (N / kStepStates);
    const long long tiles = (a.D + CH - 1) / CH;
    const int splits = (int)std::min<long long>(a.rows, std::max(1LL, kStepBlocks * 152 / tiles));
    scan_step_kernel<N, T><<<(unsigned)(tiles * splits), kScanThreads, 0, a.stream>>>(a, splits);
    return cudaGetLastError();
}

#define GDN_SCAN_N(FN, a)                                        \
    switch ((a).N) {                                             \
        case 8: return FN<8, T>(a);                              \
        case 16: return FN<16, T>(a);                            \
        case 32: return FN<32, T>(a);                            \
        case 64: return FN<64, T>(a);                            \
    }                                                            \
    return cudaErrorInvalidValue;
template <typename T>
cudaError_t fwd_n(const ScanArgs& a) { GDN_SCAN_N(fwd_typed, a) }
template <typename T>
cudaError_t step_n(const ScanStepArgs& a) { GDN_SCAN_N(step_typed, a) }
#undef GDN_SCAN_N

}  // namespace

// Whole walks, a block a sequence and channel tile, or segments, whose states are formed first: 60 % more work, on all SMs.
// A wave of whole walks (152 blocks of four walking warps, one an SM) takes the time of its tokens however few its blocks,
// segments that of all tokens x warps and some 18 us more.  The two meet where a wave costs as much as segments of `wave`
// warps, the 18 us being 150,000 tokens x warps of them.  Measured, whole / segments in us a call, by warps (batch x channels
// x states / 256), 16 states a channel, bf16:
//   8192 tokens: 256 359 / 277, 320 359 / 347, 352 359 / 359, 384 358 / 387, 448 358 / 473, 512 359 / 527, 608 358 / 569,
//     in two waves 640 709 / 631, 704 709 / 689, 768 709 / 773, in three 1280 1061 / 1197;
//   32768: 320 1411 / 1234, 384 1411 / 1519;  2048: 128 96 / 55, 224 96 / 76, 288 96 / 94, 384 95 / 121;
//   1024: 128 51 / 39, 224 51 / 55;
// fp32, whose segments' vectors leave registers for one block an SM in place of two:
//   8192 tokens: 256 375 / 335, 288 373 / 373, 384 373 / 467, 512 373 / 629, 640 740 / 758;
//   2048: 224 99 / 90, 288 99 / 113;
// 8 states a channel, shorter tiles, 8192 tokens:
//   bf16 320 509 / 461, 368 512 / 509, 448 511 / 632;  fp32 288 544 / 510, 320 546 / 568.
// Near the border the choice costs 5 % at most.  Packed sequences are taken as one long one, the worst case of their lengths,
// which are on the device: several share a wave.  A segment has at least 256 tokens, and there are about 8 x 608 warps of
// work in all (4 x: 452, 12 x: 430, 16 x: 457 against 428 us for 46,547 packed tokens of 1024 channels).
static int scan_fwd_segment(long long tokens, int D, int G, int N, int nseq, bool packed, int dtype) {
    const long long T = packed ? tokens : tokens / nseq;
    const int ch = 2 * kScanThreads / (N / 4);
    const long long blocks = (long long)G * ((D / G + ch - 1) / ch) * (packed ? 1 : nseq);
    const long long waves = packed ? 1 : (blocks + 151) / 152, wave = (dtype == GDN_BF16 ? 360 : 310) + (N == 8 ? 30 : 0);
    if (waves * T * wave <= 4 * blocks * T + 150000) return 0;
    const long long want = 8 * 608;   // warps
    const long long per = tokens * std::max(1LL, (long long)D * N / 256) / want;
    const long long seg = std::max(256LL, (per + 63) / 64 * 64);
    return T <= seg ? 0 : (int)std::min<long long>(seg, 1 << 20);
}
ScanFwdLayout scan_fwd_layout(long long tokens, int D, int G, int N, int nseq, bool packed, int dtype) {
    ScanFwdLayout l{};
    l.seg = scan_fwd_segment(tokens, D, G, N, nseq, packed, dtype);
    l.slots = l.seg ? tokens / l.seg + nseq : nseq;
    if (l.seg) {
        l.sum_dt = ((size_t)l.slots * D * N * 4 + 255) / 256 * 256;
        l.total = l.sum_dt + (size_t)l.slots * D * 4;
    }
    return l;
}

cudaError_t launch_scan_join(const ScanArgs& a, bool adjoints) {
    const long long blocks = ((long long)a.D * a.N / 4 + kScanThreads - 1) / kScanThreads * a.nseq;
    scan_join_kernel<<<dim3((unsigned)blocks, adjoints ? 2 : 1), kScanThreads, 0, a.stream>>>(a);
    return cudaGetLastError();
}
cudaError_t launch_scan_fwd(const ScanArgs& a) {
    return a.dtype == GDN_BF16 ? fwd_n<__nv_bfloat16>(a) : fwd_n<float>(a);
}
cudaError_t launch_scan_step(const ScanStepArgs& a) {
    return a.dtype == GDN_BF16 ? step_n<__nv_bfloat16>(a) : step_n<float>(a);
}

}  // namespace gdn
