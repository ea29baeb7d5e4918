// Gradients of the selective scan.  With p = dy silu(z), lam = dL/dh walked backwards,
//     lam_t = C_t p_t + a_{t+1} lam_{t+1},   dC = sum_d p h,   dB = sum_d lam dt u,   q = sum_n lam B,
//     w = lam a h_{t-1},   r = sum_n A w,   dA = sum_t dt w,   du = dt q + skip p,   d(dt) = u q + r,
//     d(delta) = d(dt) sigmoid(delta + bias),   dz = dy (sum_n C h + skip u) silu'(z)
// (a h_{t-1} is kept rather than h_{t-1}, so that w needs no division and h = a h_{t-1} + dt u B).
//
// Every segment of kSegment tokens is a block's work on its own, with the state before it and the adjoint behind it
// formed first (launch_scan_states).  A block walks its segment forwards, keeping the state every K tokens in shared
// memory, then the chunks of K tokens backwards: each is walked forwards again with a and a h_{t-1} in registers, then
// backwards.  Sums over a group's channels (dB, dC) leave as one partial sum a tile, sums over tokens (dA_log, dskip,
// dbias) as one a segment; the last kernels add them in order.
#include <algorithm>

#include "norm_rows.cuh"
#include "scan_common.cuh"

namespace gdn {
namespace {

constexpr int kChunk = 8;   // tokens whose a and a h_{t-1} a thread holds

// A lane has two channels of four states each: L lanes a channel pair.
template <int N>
struct Shape {
    static constexpr int L = N / 4, CH = 2 * kScanThreads / L, K = kChunk;
    static constexpr int kRow = CH + 8;
    static constexpr int kVecs = (K * CH / 4 + kScanThreads - 1) / kScanThreads;
    static constexpr int kBC = (2 * K * N / 4 + kScanThreads - 1) / kScanThreads;
    static constexpr int kSlots = 32 / L;   // channel pairs of a warp
};

template <int N>
struct Smem {
    float4 tok[kChunk][Shape<N>::CH];             // dt, dt u, p
    float bc[2][4][kChunk][N];                    // B, C, the states of each four in the order of a lane: entry r is r ^ perm
    float sums[3][kChunk][Shape<N>::kRow];        // y, q, r
    float red[kScanThreads / 32][kChunk][2 * N];  // dB, dC of each warp
    float4 state[kScanSegment / kChunk][2][kScanThreads];
};

template <int N, typename T>
struct Tile {
    Raw4<T> u[Shape<N>::kVecs], d[Shape<N>::kVecs], z[Shape<N>::kVecs], gy[Shape<N>::kVecs];
    Raw4<T> bc[Shape<N>::kBC];
};

// FULL: all of a chunk; else what the states need.
template <int N, typename T, bool FULL>
__device__ __forceinline__ void load_tile(Tile<N, T>& t, const ScanArgs& a, const ChannelTile& tile, long long t0, int tokens) {
    using S = Shape<N>;
    const int tid = threadIdx.x;
#pragma unroll
    for (int v = 0; v < S::kVecs; ++v) {
        const int i = tid + v * kScanThreads, k = i / (S::CH / 4), c = i % (S::CH / 4) * 4;
        const bool ok = k < tokens && c < tile.n;
        const size_t row = t0 + k, d = tile.d0 + c;
        auto get = [&](const void* p, long long stride) {
            return ok && p ? load4(static_cast<const T*>(p) + row * stride + d) : Raw4<T>::zero();
        };
        t.u[v] = get(a.u, a.u_stride);
        t.d[v] = get(a.delta, a.delta_stride);
        if (FULL) {
            t.z[v] = get(a.z, a.z_stride);
            t.gy[v] = get(a.gy, a.D);
        }
    }
#pragma unroll
    for (int v = 0; v < S::kBC; ++v) {
        const int i = tid + v * kScanThreads, which = i / (S::K * N / 4), k = i / (N / 4) % S::K, n = i % (N / 4) * 4;
        const bool ok = which < (FULL ? 2 : 1) && k < tokens;
        const T* p = static_cast<const T*>(which == 0 ? a.B : a.C) + (size_t)tile.g * N + n;
        t.bc[v] = ok ? load4(p + (t0 + k) * (which == 0 ? a.b_stride : a.c_stride)) : Raw4<T>::zero();
    }
}

// A tile's values in fp32 in shared memory.
template <int N, typename T, bool FULL>
__device__ __forceinline__ void form_tile(const Tile<N, T>& t, Smem<N>& sm, const ScanArgs& a, int channels, int tokens,
                                          float4 bias) {
    using S = Shape<N>;
    const int tid = threadIdx.x;
#pragma unroll
    for (int v = 0; v < S::kVecs; ++v) {
        const int i = tid + v * kScanThreads, k = i / (S::CH / 4), c = i % (S::CH / 4) * 4;
        if (k >= S::K) break;
        const float4 x = t.u[v].f(), d = t.d[v].f();
        const bool ok = k < tokens && c < channels;
        const float4 sp = softplus4(add4(d, bias));
        float dt[4] = {sp.x, sp.y, sp.z, sp.w}, p[4] = {0.f, 0.f, 0.f, 0.f};
        const float uu[4] = {x.x, x.y, x.z, x.w};
        if (FULL) {
            float4 g = t.gy[v].f();
            if (a.z) g = gated4(g, t.z[v].f());
            p[0] = g.x; p[1] = g.y; p[2] = g.z; p[3] = g.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dt[e] = ok ? dt[e] : 0.f;   // dt = 0: a token past the end changes nothing
            sm.tok[k][c + e] = make_float4(dt[e], dt[e] * uu[e], p[e], 0.f);
        }
    }
#pragma unroll
    for (int v = 0; v < S::kBC; ++v) {
        const int i = tid + v * kScanThreads, which = i / (S::K * N / 4), k = i / (N / 4) % S::K, n = i % (N / 4) * 4;
        if (which >= 2) continue;
        const float4 b = t.bc[v].f();
        *reinterpret_cast<float4*>(&sm.bc[which][0][k][n]) = b;
        *reinterpret_cast<float4*>(&sm.bc[which][1][k][n]) = make_float4(b.y, b.x, b.w, b.z);
        *reinterpret_cast<float4*>(&sm.bc[which][2][k][n]) = make_float4(b.z, b.w, b.x, b.y);
        *reinterpret_cast<float4*>(&sm.bc[which][3][k][n]) = make_float4(b.w, b.z, b.y, b.x);
    }
}

// Entry r of a lane's four states is state r ^ perm.
__device__ __forceinline__ float4 permuted(float4 x, int perm) {
    if (perm & 1) x = make_float4(x.y, x.x, x.w, x.z);
    if (perm & 2) x = make_float4(x.z, x.w, x.x, x.y);
    return x;
}

// Four values a lane, entry r belonging to state r ^ perm: their sums over the warp's channel pairs, so that a lane ends
// with entry 0 (and, with two channel pairs a warp, 1).  The lanes that are exchanged with hold the other entries first,
// so no value has to be selected.
template <int N>
__device__ __forceinline__ void channel_sum(float (&v)[4]) {
    constexpr int L = N / 4, kSlots = 32 / L;
    v[0] += __shfl_xor_sync(0xffffffffu, v[2], L);
    v[1] += __shfl_xor_sync(0xffffffffu, v[3], L);
    if (kSlots >= 4) v[0] += __shfl_xor_sync(0xffffffffu, v[1], 2 * L);
#pragma unroll
    for (int o = 4 * L; o < 32; o *= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
}

template <int N, typename T>
__global__ void __launch_bounds__(kScanThreads, 2) scan_bwd_kernel(const __grid_constant__ ScanArgs a) {
    using S = Shape<N>;
    constexpr int L = S::L, CH = S::CH, K = S::K, TT = L / 2;   // TT: tokens whose sums over states are finished together
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem<N>& sm = *reinterpret_cast<Smem<N>*>(smem_raw);
    const int tiles = a.G * ((a.D / a.G + CH - 1) / CH), slot = blockIdx.x / tiles, tile_id = blockIdx.x % tiles;
    const ChannelTile tile = channel_tile(a.D, a.G, CH, tile_id);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n4 = lane % L * 4, pair = lane / L, swap = lane & 1;
    const int perm = ((pair & 1) ? 2 : 0) | ((S::kSlots >= 4 && (pair & 2)) ? 1 : 0);
    const int c4 = tid % (CH / 4) * 4;
    // the lane's channels: the lanes of a pair hold them in the other order, as the states' entries
    int ch[2];
    ch[0] = warp * 2 * S::kSlots + pair * 2 + swap;
    ch[1] = ch[0] ^ 1;
    const size_t DN = (size_t)a.D * N;
    size_t at[2];
    bool own[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        own[s] = ch[s] < tile.n;
        at[s] = (size_t)(tile.d0 + ch[s]) * N + n4;
    }
    float* const part_A = a.part_A + (size_t)slot * DN;
    float* const part_s = a.part_s + (size_t)slot * 2 * a.D + tile.d0;
    Unit u;
    if (!unit_at(a.cu, a.T, a.nseq, a.seg, slot, false, u)) u.t0 = u.t1 = 0, u.first = false;
    const long long len = u.t1 - u.t0;
    const int chunks = (int)((len + K - 1) / K);

    float2 A2[2][2], h[2][2], lam[2][2], gA[2][2];
    auto take = [&](const float* p, int s, float2 (&x)[2]) {
        const float4 f = p && own[s] ? permuted(*reinterpret_cast<const float4*>(p + at[s]), perm) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[0] = make_float2(f.x, f.y);
        x[1] = make_float2(f.z, f.w);
    };
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        take(a.A_log, s, A2[s]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            A2[s][i] = own[s] ? make_float2(rate2(A2[s][i].x), rate2(A2[s][i].y)) : all2(0.f);
            gA[s][i] = all2(0.f);
        }
        const bool some = len > 0;   // not an empty slot, whose sequence is none
        take(!some ? nullptr : a.seg ? a.states + (size_t)slot * DN : a.h0 ? a.h0 + (size_t)u.seq * DN : nullptr, s, h[s]);
        take(!some ? nullptr : a.seg ? a.adjoints + (size_t)slot * DN : a.gh ? a.gh + (size_t)u.seq * DN : nullptr, s, lam[s]);
    }
    float4 bias = make_float4(0.f, 0.f, 0.f, 0.f), skip = bias, g_skip = bias, g_bias = bias;
    if (c4 < tile.n) {
        if (a.dt_bias) bias = *reinterpret_cast<const float4*>(a.dt_bias + tile.d0 + c4);
        if (a.skip) skip = *reinterpret_cast<const float4*>(a.skip + tile.d0 + c4);
    }
    auto put = [&](float* p, int s, const float2 (&x)[2]) {
        if (own[s]) *reinterpret_cast<float4*>(p + at[s]) = permuted(make_float4(x[0].x, x[0].y, x[1].x, x[1].y), perm);
    };

    // forwards: the state before each chunk
    Tile<N, T> raw;
    auto tokens_of = [&](int c) { return (int)min((long long)K, len - (long long)c * K); };
    if (chunks > 1) load_tile<N, T, false>(raw, a, tile, u.t0, K);
    for (int c = 0; c < chunks; ++c) {
#pragma unroll
        for (int s = 0; s < 2; ++s) sm.state[c][s][tid] = make_float4(h[s][0].x, h[s][0].y, h[s][1].x, h[s][1].y);
        if (c + 1 == chunks) break;
        __syncthreads();
        form_tile<N, T, false>(raw, sm, a, tile.n, K, bias);
        __syncthreads();
        if (c + 2 < chunks) load_tile<N, T, false>(raw, a, tile, u.t0 + (c + 1) * K, K);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float4 b = *reinterpret_cast<const float4*>(&sm.bc[0][perm][k][n4]);
            const float2 B[2] = {make_float2(b.x, b.y), make_float2(b.z, b.w)};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const float2 dd = *reinterpret_cast<const float2*>(&sm.tok[k][ch[s]]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    h[s][i] = fma2(decay(A2[s][i], dd.x), h[s][i], mul2(B[i], all2(dd.y)));
                }
            }
        }
    }

    if (chunks > 0) load_tile<N, T, true>(raw, a, tile, u.t0 + (long long)(chunks - 1) * K, tokens_of(chunks - 1));
    for (int c = chunks - 1; c >= 0; --c) {
        const long long t0 = u.t0 + (long long)c * K;
        const int tokens = tokens_of(c);
        __syncthreads();
        form_tile<N, T, true>(raw, sm, a, tile.n, tokens, bias);
        const Tile<N, T> cur = raw;
        __syncthreads();
        if (c > 0) load_tile<N, T, true>(raw, a, tile, t0 - K, K);
        float2 aa[K][2][2], P[K][2][2];   // a and a h_{t-1}
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const float4 f = sm.state[c][s][tid];
            h[s][0] = make_float2(f.x, f.y);
            h[s][1] = make_float2(f.z, f.w);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float4 b = *reinterpret_cast<const float4*>(&sm.bc[0][perm][k][n4]);
            const float2 B[2] = {make_float2(b.x, b.y), make_float2(b.z, b.w)};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const float2 dd = *reinterpret_cast<const float2*>(&sm.tok[k][ch[s]]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    aa[k][s][i] = decay(A2[s][i], dd.x);
                    P[k][s][i] = mul2(aa[k][s][i], h[s][i]);
                    h[s][i] = fma2(B[i], all2(dd.y), P[k][s][i]);
                }
            }
        }
#pragma unroll
        for (int kk = K - TT; kk >= 0; kk -= TT) {
            float sum[3][TT];   // y, q, r of the lane's first channel
#pragma unroll
            for (int e = TT - 1; e >= 0; --e) {
                const int k = kk + e;
                const float4 b = *reinterpret_cast<const float4*>(&sm.bc[0][perm][k][n4]);
                const float4 cc = *reinterpret_cast<const float4*>(&sm.bc[1][perm][k][n4]);
                const float2 B[2] = {make_float2(b.x, b.y), make_float2(b.z, b.w)};
                const float2 C[2] = {make_float2(cc.x, cc.y), make_float2(cc.z, cc.w)};
                float2 gB[2], gC[2];
                float part[3][2];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const float4 dd = sm.tok[k][ch[s]];   // dt, dt u, p
                    float2 y, q, r;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        lam[s][i] = fma2(C[i], all2(dd.z), lam[s][i]);
                        const float2 hh = fma2(B[i], all2(dd.y), P[k][s][i]), w = mul2(lam[s][i], P[k][s][i]);
                        gC[i] = s == 0 ? mul2(hh, all2(dd.z)) : fma2(hh, all2(dd.z), gC[i]);
                        gB[i] = s == 0 ? mul2(lam[s][i], all2(dd.y)) : fma2(lam[s][i], all2(dd.y), gB[i]);
                        y = i == 0 ? mul2(hh, C[i]) : fma2(hh, C[i], y);
                        q = i == 0 ? mul2(lam[s][i], B[i]) : fma2(lam[s][i], B[i], q);
                        r = i == 0 ? mul2(w, A2[s][i]) : fma2(w, A2[s][i], r);
                        gA[s][i] = fma2(w, all2(dd.x), gA[s][i]);
                        lam[s][i] = mul2(lam[s][i], aa[k][s][i]);
                    }
                    part[0][s] = y.x + y.y;
                    part[1][s] = q.x + q.y;
                    part[2][s] = r.x + r.y;
                }
#pragma unroll
                for (int x = 0; x < 3; ++x) sum[x][e] = part[x][0] + __shfl_xor_sync(0xffffffffu, part[x][1], 1);
                float vB[4] = {gB[0].x, gB[0].y, gB[1].x, gB[1].y}, vC[4] = {gC[0].x, gC[0].y, gC[1].x, gC[1].y};
                channel_sum<N>(vB);
                channel_sum<N>(vC);
                float* to = &sm.red[warp][k][n4 + perm];
                if (S::kSlots >= 4) {
                    if (pair == (perm & 1 ? 2 : 0) + (perm & 2 ? 1 : 0)) {   // one of the lanes that have the sums
                        to[0] = vB[0];
                        to[N] = vC[0];
                    }
                } else {
                    to[0] = vB[0];
                    to[N] = vC[0];
                    sm.red[warp][k][n4 + (perm ^ 1)] = vB[1];
                    sm.red[warp][k][n4 + (perm ^ 1) + N] = vC[1];
                }
            }
#pragma unroll
            for (int x = 0; x < 3; ++x) sm.sums[x][kk + (lane >> 1) % TT][ch[0]] = transpose_sum<TT, 2>(sum[x], lane);
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < S::kVecs; ++v) {
            const int i = tid + v * kScanThreads, k = i / (CH / 4);
            if (k >= tokens || c4 >= tile.n) continue;
            const size_t row = t0 + k, d = tile.d0 + c4;
            const float4 x4 = cur.u[v].f(), d4 = cur.d[v].f(), g4 = cur.gy[v].f(), z4 = cur.z[v].f();
            const float uu[4] = {x4.x, x4.y, x4.z, x4.w}, raw_d[4] = {d4.x + bias.x, d4.y + bias.y, d4.z + bias.z, d4.w + bias.w};
            const float gg[4] = {g4.x, g4.y, g4.z, g4.w}, zz[4] = {z4.x, z4.y, z4.z, z4.w};
            const float sk[4] = {skip.x, skip.y, skip.z, skip.w};
            float gu[4], gd[4], gz[4], gs[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 tk = sm.tok[k][c4 + e];
                const float y = sm.sums[0][k][c4 + e], q = sm.sums[1][k][c4 + e], r = sm.sums[2][k][c4 + e] * kLn2;
                gu[e] = fmaf(tk.x, q, sk[e] * tk.z);
                gd[e] = fmaf(uu[e], q, r) * logistic_f(raw_d[e]);
                gs[e] = tk.z * uu[e];
                const float sg = logistic_f(zz[e]);
                gz[e] = gg[e] * fmaf(sk[e], uu[e], y) * sg * fmaf(zz[e], 1.f - sg, 1.f);
            }
            store4(static_cast<T*>(a.gu) + row * a.D + d, make_float4(gu[0], gu[1], gu[2], gu[3]));
            store4(static_cast<T*>(a.gdelta) + row * a.D + d, make_float4(gd[0], gd[1], gd[2], gd[3]));
            if (a.z) store4(static_cast<T*>(a.gz) + row * a.gz_stride + d, make_float4(gz[0], gz[1], gz[2], gz[3]));
            g_skip.x += gs[0]; g_skip.y += gs[1]; g_skip.z += gs[2]; g_skip.w += gs[3];
            g_bias.x += gd[0]; g_bias.y += gd[1]; g_bias.z += gd[2]; g_bias.w += gd[3];
        }
        for (int i = tid; i < tokens * 2 * N; i += kScanThreads) {
            const int k = i / (2 * N), n = i % (2 * N);
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kScanThreads / 32; ++w) s += sm.red[w][k][n];
            a.part_bc[((size_t)tile_id * a.tokens + t0 + k) * 2 * N + n] = s;
        }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        put(part_A, s, gA[s]);
        if (a.gh0 && u.first && len > 0) put(a.gh0 + (size_t)u.seq * DN, s, lam[s]);
    }
    // an empty sequence's initial state is its final one
    if (a.gh0 && u.first && len == 0)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float2 x[2];
            take(a.gh ? a.gh + (size_t)u.seq * DN : nullptr, s, x);
            put(a.gh0 + (size_t)u.seq * DN, s, x);
        }
    // the threads with the same channels, in order
    __syncthreads();
    float4* const fold = reinterpret_cast<float4*>(smem_raw);
    fold[2 * tid] = g_skip;
    fold[2 * tid + 1] = g_bias;
    __syncthreads();
    for (int i = tid; i < 2 * (CH / 4); i += kScanThreads) {
        const int c = i >> 1;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x = c; x < kScanThreads; x += CH / 4) {
            const float4 y = fold[2 * x + (i & 1)];
            s.x += y.x; s.y += y.y; s.z += y.z; s.w += y.w;
        }
        if (c * 4 < tile.n) *reinterpret_cast<float4*>(part_s + (i & 1) * a.D + c * 4) = s;
    }
}

// dB and dC of a token, over the tiles of each group.
template <typename T>
__global__ void __launch_bounds__(256) scan_bc_sums_kernel(const __grid_constant__ ScanArgs a, int tiles_per_group) {
    const int per = a.G * a.N / 2;   // vectors of four: dB and dC of the groups
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, t = i / per;
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
    for (int x = 0; x < tiles_per_group; ++x) {
        const float4 y = *reinterpret_cast<const float4*>(p + (size_t)x * a.tokens * 2 * a.N);
        s.x += y.x; s.y += y.y; s.z += y.z; s.w += y.w;
    }
    const bool is_c = n >= a.N;
    T* to = static_cast<T*>(is_c ? a.gC : a.gB) + t * (is_c ? a.gc_stride : a.gb_stride);
    store4(to + (size_t)g * a.N + (is_c ? n - a.N : n), s);
}

// dA_log = sum over the segments of A dA, dskip, dbias: 32 columns a block of the slots' rows of D N + 2 D sums.
__global__ void __launch_bounds__(1024) scan_weight_sums_kernel(const __grid_constant__ ScanArgs a) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const size_t DN = (size_t)a.D * a.N, c = (size_t)blockIdx.x * 32 + lane;
    const bool rate = c < DN, any = c < DN + 2 * a.D;
    const float* p = rate ? a.part_A + c : a.part_s + (c - DN);
    const size_t row = rate ? DN : 2 * (size_t)a.D;
    float s = 0.f;
    if (any)
        for (int r = grp; r < a.slots; r += 32) s += p[r * row];
    red[grp][lane] = s;
    __syncthreads();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (grp < o) red[grp][lane] += red[grp + o][lane];
        __syncthreads();
    }
    if (grp != 0 || !any) return;
    s = red[0][lane];
    if (rate) {
        if (a.gA) a.gA[c] = -expf(a.A_log[c]) * s;
    } else if (c < DN + a.D) {
        if (a.gskip) a.gskip[c - DN] = s;
    } else if (a.gbias) {
        a.gbias[c - DN - a.D] = s;
    }
}

template <int N, typename T>
cudaError_t bwd_typed(const ScanArgs& a) {
    using S = Shape<N>;
    cudaError_t e = allow_smem<scan_bwd_kernel<N, T>>();
    if (e != cudaSuccess) return e;
    const int per_group = (a.D / a.G + S::CH - 1) / S::CH;
    scan_bwd_kernel<N, T><<<(unsigned)((long long)a.slots * a.G * per_group), kScanThreads, sizeof(Smem<N>), a.stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const long long vecs = (long long)a.tokens * a.G * N / 2;
    scan_bc_sums_kernel<T><<<(unsigned)((vecs + 255) / 256), 256, 0, a.stream>>>(a, per_group);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const size_t cols = (size_t)a.D * N + 2 * a.D;
    scan_weight_sums_kernel<<<(unsigned)((cols + 31) / 32), 1024, 0, a.stream>>>(a);
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

ScanBwdLayout scan_bwd_layout(long long tokens, int D, int G, int N, int nseq, bool packed) {
    ScanBwdLayout l{};
    // one segment a sequence: nothing to join
    l.seg = !packed && tokens / nseq <= kScanSegment ? 0 : kScanSegment;
    l.slots = l.seg ? tokens / kScanSegment + nseq : nseq;
    const size_t states = ((size_t)l.slots * D * N * 4 + 255) / 256 * 256, rows = ((size_t)l.slots * D * 4 + 255) / 256 * 256;
    const int ch = 2 * kScanThreads / (N / 4), tiles = G * ((D / G + ch - 1) / ch);
    l.adjoints = l.seg ? states : 0;   // the states come first
    l.sum_dt = 2 * l.adjoints;
    l.part_A = l.sum_dt + (l.seg ? rows : 0);
    l.part_s = l.part_A + states;
    l.part_bc = l.part_s + 2 * rows;
    l.total = l.part_bc + (size_t)tiles * tokens * 2 * N * 4;
    return l;
}

cudaError_t launch_scan_bwd(const ScanArgs& a) {
    if (a.seg) {
        const cudaError_t e = launch_scan_states(a);
        if (e != cudaSuccess) return e;
    }
    return a.dtype == GDN_BF16 ? bwd_n<__nv_bfloat16>(a) : bwd_n<float>(a);
}

}  // namespace gdn
