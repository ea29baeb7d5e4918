// The selective state space scan: per sequence, channel d of group g(d) and state n, with dt = softplus(delta + bias)
// and A = -exp(A_log),
//     h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t,      y_t = (sum_n C_t h_t + skip u_t) silu(z_t).
//
// A warp holds 32 / L channels, L = N / 4 lanes a channel with four states each.  Per tile of K tokens a block forms dt
// and dt u of its channels and B, C in fp32 in shared memory, walks the tile, and applies skip and gate to the sums.
#include <algorithm>

#include "scan_common.cuh"

namespace gdn {
namespace {

template <int N>
struct Shape {
    static constexpr int L = N / 4, CH = kScanThreads / L, K = N <= 16 ? 16 : 32;
    static constexpr int kRow = CH + (32 / L > 4 ? 32 / L : 4);   // floats of a row of sums: no bank conflicts
    static constexpr int kVecs = (K * CH / 4 + kScanThreads - 1) / kScanThreads;   // 4-channel vectors a thread
    static constexpr int kBC = (2 * K * N / 4 + kScanThreads - 1) / kScanThreads;  // 4-state vectors of B and C a thread
};

// The raw values of a thread's share of a tile.
template <int N, typename T, int IN>
struct Tile {
    Raw4<T> x[IN][Shape<N>::kVecs];
    Raw4<T> bc[Shape<N>::kBC];
};

template <int N, typename T, int IN>
__device__ __forceinline__ void load_tile(Tile<N, T, IN>& t, const T* const (&src)[IN], const long long (&stride)[IN],
                                          const T* B, long long b_stride, const T* C, long long c_stride, long long t0,
                                          int tokens, int channels) {
    using S = Shape<N>;
    const int tid = threadIdx.x;
#pragma unroll
    for (int v = 0; v < S::kVecs; ++v) {
        const int i = tid + v * kScanThreads, k = i / (S::CH / 4), c = i % (S::CH / 4) * 4;
        const bool ok = k < tokens && c < channels;
#pragma unroll
        for (int x = 0; x < IN; ++x)
            t.x[x][v] = ok && src[x] ? load4(src[x] + (t0 + k) * stride[x] + c) : Raw4<T>::zero();
    }
#pragma unroll
    for (int v = 0; v < S::kBC; ++v) {
        const int i = tid + v * kScanThreads, which = i / (S::K * N / 4), k = i / (N / 4) % S::K, n = i % (N / 4) * 4;
        const T* p = which == 0 ? B : C;
        t.bc[v] = which < 2 && k < tokens && p ? load4(p + (t0 + k) * (which == 0 ? b_stride : c_stride) + n) : Raw4<T>::zero();
    }
}

// The outputs, or (STATE) each segment's own contribution to the state, from zero, and its sum of dt.  ADJ: also the
// contribution of its outputs to the adjoint of the state before it, sum_t (a_first .. a_t) C_t p_t, p = dy silu(z).
template <int N, typename T, bool STATE, bool ADJ>
__global__ void __launch_bounds__(kScanThreads) scan_kernel(const __grid_constant__ ScanArgs a) {
    using S = Shape<N>;
    constexpr int L = S::L, CH = S::CH, K = S::K;
    constexpr int IN = STATE && !ADJ ? 2 : ADJ ? 4 : 3;
    __shared__ __align__(16) float2 s_dt[K][CH];
    __shared__ __align__(16) float s_p[ADJ ? K : 1][CH];
    __shared__ __align__(16) float s_bc[2][K][N];
    __shared__ __align__(16) float s_y[STATE ? 1 : K][S::kRow];
    const int tiles = a.G * ((a.D / a.G + CH - 1) / CH), slot = blockIdx.x / tiles;
    const ChannelTile tile = channel_tile(a.D, a.G, CH, blockIdx.x % tiles);
    Unit u;
    if (!unit_at(a.cu, a.T, a.nseq, a.seg, slot, false, u)) return;
    if (STATE && (ADJ ? u.first && u.last : u.last)) return;   // nothing reads it
    const int tid = threadIdx.x, lane = tid & 31, cl = tid / L, n4 = tid % L * 4;
    const int c4 = tid % (CH / 4) * 4;   // the thread's channels in the elementwise work
    const bool own = cl < tile.n;
    const size_t at = (size_t)(tile.d0 + cl) * N + n4, DN = (size_t)a.D * N;

    float2 A2[2], h[2], lam[2], E[2];
    h[0] = h[1] = lam[0] = lam[1] = all2(0.f);
    E[0] = E[1] = all2(1.f);
    A2[0] = A2[1] = all2(0.f);
    float sum_dt = 0.f;
    if (own) {
        const float4 l = *reinterpret_cast<const float4*>(a.A_log + at);
        A2[0] = make_float2(rate2(l.x), rate2(l.y));
        A2[1] = make_float2(rate2(l.z), rate2(l.w));
        if (!STATE) {
            const float* from = a.seg ? a.states + (size_t)slot * DN : a.h0 ? a.h0 + (size_t)u.seq * DN : nullptr;
            if (from) {
                const float4 f = *reinterpret_cast<const float4*>(from + at);
                h[0] = make_float2(f.x, f.y);
                h[1] = make_float2(f.z, f.w);
            }
        }
    }
    float4 bias = make_float4(0.f, 0.f, 0.f, 0.f), skip = bias;
    if (c4 < tile.n) {
        if (a.dt_bias) bias = *reinterpret_cast<const float4*>(a.dt_bias + tile.d0 + c4);
        if (!STATE && a.skip) skip = *reinterpret_cast<const float4*>(a.skip + tile.d0 + c4);
    }
    auto head = [&](const void* p) { return p ? static_cast<const T*>(p) + tile.d0 : nullptr; };
    const T* src[IN];
    long long stride[IN];
    src[0] = head(a.u); stride[0] = a.u_stride;
    src[1] = head(a.delta); stride[1] = a.delta_stride;
    if constexpr (IN > 2) { src[2] = head(a.z); stride[2] = a.z_stride; }
    if constexpr (IN > 3) { src[3] = head(a.gy); stride[3] = a.D; }
    const T* B = static_cast<const T*>(a.B) + (size_t)tile.g * N;
    const T* C = STATE && !ADJ ? nullptr : static_cast<const T*>(a.C) + (size_t)tile.g * N;

    Tile<N, T, IN> raw;
    load_tile<N, T, IN>(raw, src, stride, B, a.b_stride, C, a.c_stride, u.t0, (int)min((long long)K, u.t1 - u.t0), tile.n);
    for (long long t0 = u.t0; t0 < u.t1; t0 += K) {
        const int tokens = (int)min((long long)K, u.t1 - t0);
        Raw4<T> cu[S::kVecs], cz[S::kVecs];
#pragma unroll
        for (int v = 0; v < S::kVecs; ++v) {
            const int i = tid + v * kScanThreads, k = i / (CH / 4);
            if (k >= K) break;
            float4 x = raw.x[0][v].f(), d = raw.x[1][v].f();
            const bool ok = k < tokens && c4 < tile.n;   // a token past the end leaves the state as it is: dt = 0
            d.x = ok ? softplus_f(d.x + bias.x) : 0.f;
            d.y = ok ? softplus_f(d.y + bias.y) : 0.f;
            d.z = ok ? softplus_f(d.z + bias.z) : 0.f;
            d.w = ok ? softplus_f(d.w + bias.w) : 0.f;
            float4* to = reinterpret_cast<float4*>(&s_dt[k][c4]);
            to[0] = make_float4(d.x, d.x * x.x, d.y, d.y * x.y);
            to[1] = make_float4(d.z, d.z * x.z, d.w, d.w * x.w);
            cu[v] = raw.x[0][v];
            if constexpr (!STATE) cz[v] = raw.x[2][v];
            if constexpr (ADJ) {
                float4 p = raw.x[3][v].f();
                if (a.z) {
                    const float4 z = raw.x[2][v].f();
                    p.x *= z.x * logistic_f(z.x);
                    p.y *= z.y * logistic_f(z.y);
                    p.z *= z.z * logistic_f(z.z);
                    p.w *= z.w * logistic_f(z.w);
                }
                *reinterpret_cast<float4*>(&s_p[k][c4]) = p;
            }
        }
#pragma unroll
        for (int v = 0; v < S::kBC; ++v) {
            const int i = tid + v * kScanThreads, which = i / (K * N / 4), k = i / (N / 4) % K, n = i % (N / 4) * 4;
            if (which < 2) *reinterpret_cast<float4*>(&s_bc[which][k][n]) = raw.bc[v].f();
        }
        __syncthreads();
        if (t0 + K < u.t1)
            load_tile<N, T, IN>(raw, src, stride, B, a.b_stride, C, a.c_stride, t0 + K, (int)min((long long)K, u.t1 - t0 - K),
                                tile.n);
#pragma unroll 1
        for (int k0 = 0; k0 < K; k0 += L) {
            float part[L];
#pragma unroll
            for (int e = 0; e < L; ++e) {
                const int k = k0 + e;
                const float2 dd = s_dt[k][cl];
                const float4 b = *reinterpret_cast<const float4*>(&s_bc[0][k][n4]);
                float2 ar[2], w[2] = {make_float2(b.x, b.y), make_float2(b.z, b.w)};
                float2 c[2];
                if constexpr (!STATE || ADJ) {
                    const float4 x = *reinterpret_cast<const float4*>(&s_bc[1][k][n4]);
                    c[0] = make_float2(x.x, x.y);
                    c[1] = make_float2(x.z, x.w);
                }
                float2 y = all2(0.f);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ar[i] = mul2(A2[i], all2(dd.x));
                    ar[i] = make_float2(ex2(ar[i].x), ex2(ar[i].y));
                    h[i] = fma2(ar[i], h[i], mul2(w[i], all2(dd.y)));
                    if constexpr (!STATE) y = i == 0 ? mul2(h[i], c[i]) : fma2(h[i], c[i], y);
                    if constexpr (ADJ) {
                        E[i] = mul2(E[i], ar[i]);
                        lam[i] = fma2(E[i], mul2(c[i], all2(s_p[k][cl])), lam[i]);
                    }
                }
                if constexpr (STATE) sum_dt += dd.x;
                part[e] = y.x + y.y;
            }
            if constexpr (!STATE) s_y[k0 + lane % L][cl] = transpose_sum<L>(part, lane);
        }
        __syncthreads();
        if constexpr (!STATE) {
#pragma unroll
            for (int v = 0; v < S::kVecs; ++v) {
                const int i = tid + v * kScanThreads, k = i / (CH / 4);
                if (k >= tokens || c4 >= tile.n) continue;
                float4 y = *reinterpret_cast<const float4*>(&s_y[k][c4]);
                const float4 x = cu[v].f();
                y = make_float4(fmaf(skip.x, x.x, y.x), fmaf(skip.y, x.y, y.y), fmaf(skip.z, x.z, y.z), fmaf(skip.w, x.w, y.w));
                if (a.z) {
                    const float4 z = cz[v].f();
                    y.x *= z.x * logistic_f(z.x);
                    y.y *= z.y * logistic_f(z.y);
                    y.z *= z.z * logistic_f(z.z);
                    y.w *= z.w * logistic_f(z.w);
                }
                store4(static_cast<T*>(a.y) + (t0 + k) * a.D + tile.d0 + c4, y);
            }
        }
    }
    if (!own) return;
    const float4 hf = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
    if constexpr (STATE) {
        *reinterpret_cast<float4*>(a.states + (size_t)slot * DN + at) = hf;
        if constexpr (ADJ)
            *reinterpret_cast<float4*>(a.adjoints + (size_t)slot * DN + at) = make_float4(lam[0].x, lam[0].y, lam[1].x, lam[1].y);
        if (n4 == 0) a.sum_dt[(size_t)slot * a.D + tile.d0 + cl] = sum_dt;
    } else if (a.h_final && u.last) {
        *reinterpret_cast<float4*>(a.h_final + (size_t)u.seq * DN + at) = hf;
    }
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
                h = make_float4(fmaf(ex2(A[0] * dt[w]), h.x, x[w].x), fmaf(ex2(A[1] * dt[w]), h.y, x[w].y),
                                fmaf(ex2(A[2] * dt[w]), h.z, x[w].z), fmaf(ex2(A[3] * dt[w]), h.w, x[w].w));
        }
    }
}

// One token for each of N rows, in place on the states: L lanes a channel, four states each.
template <int N, typename T>
__global__ void __launch_bounds__(kScanThreads) scan_step_kernel(const __grid_constant__ ScanStepArgs a) {
    constexpr int L = N / 4, CH = kScanThreads / L;
    const int tiles = (a.D + CH - 1) / CH, row = blockIdx.x / tiles, d = blockIdx.x % tiles * CH + threadIdx.x / L;
    const int n4 = threadIdx.x % L * 4;
    const bool own = d < a.D;   // D is a multiple of 8, a warp's channels may not be
    const int slot = a.slots ? a.slots[row] : row;
    T* const y = static_cast<T*>(a.y) + (size_t)row * a.D + d;
    if (slot < 0 || slot >= a.num_slots) {   // a row without a request
        if (own && n4 == 0) *y = from_f32<T>(0.f);
        return;
    }
    float s = 0.f, u = 0.f;
    if (own) {
        float4* const hp = reinterpret_cast<float4*>(a.h + ((size_t)slot * a.D + d) * N + n4);
        const float4 h = *hp, l = *reinterpret_cast<const float4*>(a.A_log + (size_t)d * N + n4);
        const int g = d / (a.D / a.G);
        const float4 b = load4(static_cast<const T*>(a.B) + (size_t)row * a.b_stride + (size_t)g * N + n4).f();
        const float4 c = load4(static_cast<const T*>(a.C) + (size_t)row * a.c_stride + (size_t)g * N + n4).f();
        u = to_f32(static_cast<const T*>(a.u)[(size_t)row * a.u_stride + d]);
        const float raw = to_f32(static_cast<const T*>(a.delta)[(size_t)row * a.delta_stride + d]);
        const float dt = softplus_f(raw + (a.dt_bias ? a.dt_bias[d] : 0.f)), w = dt * u;
        const float4 x = make_float4(
            fmaf(ex2(dt * rate2(l.x)), h.x, w * b.x), fmaf(ex2(dt * rate2(l.y)), h.y, w * b.y),
            fmaf(ex2(dt * rate2(l.z)), h.z, w * b.z), fmaf(ex2(dt * rate2(l.w)), h.w, w * b.w));
        *hp = x;
        s = fmaf(x.x, c.x, x.y * c.y) + fmaf(x.z, c.z, x.w * c.w);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (!own || n4) return;
    if (a.skip) s = fmaf(a.skip[d], u, s);
    if (a.z) {
        const float z = to_f32(static_cast<const T*>(a.z)[(size_t)row * a.z_stride + d]);
        s *= z * logistic_f(z);
    }
    *y = from_f32<T>(s);
}

template <int N>
int tiles_of(const ScanArgs& a) {
    return a.G * ((a.D / a.G + Shape<N>::CH - 1) / Shape<N>::CH);
}

template <int N, typename T>
cudaError_t fwd_typed(const ScanArgs& a) {
    const unsigned blocks = (unsigned)((long long)a.slots * tiles_of<N>(a));
    if (a.seg) {
        scan_kernel<N, T, true, false><<<blocks, kScanThreads, 0, a.stream>>>(a);
        const cudaError_t e = launch_scan_join(a, false);
        if (e != cudaSuccess) return e;
    }
    scan_kernel<N, T, false, false><<<blocks, kScanThreads, 0, a.stream>>>(a);
    return cudaGetLastError();
}
template <int N, typename T>
cudaError_t adj_typed(const ScanArgs& a) {
    scan_kernel<N, T, true, true><<<(unsigned)((long long)a.slots * tiles_of<N>(a)), kScanThreads, 0, a.stream>>>(a);
    return cudaGetLastError();
}
template <int N, typename T>
cudaError_t step_typed(const ScanStepArgs& a) {
    constexpr int CH = kScanThreads / (N / 4);
    scan_step_kernel<N, T><<<(unsigned)((long long)a.rows * ((a.D + CH - 1) / CH)), kScanThreads, 0, a.stream>>>(a);
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
cudaError_t adj_n(const ScanArgs& a) { GDN_SCAN_N(adj_typed, a) }
template <typename T>
cudaError_t step_n(const ScanStepArgs& a) { GDN_SCAN_N(step_typed, a) }
#undef GDN_SCAN_N

}  // namespace

// A sequence is walked by one block a channel tile where the tiles of all sequences fill the GPU, else in segments,
// whose states are formed first.
int scan_fwd_segment(long long tokens, int D, int N, int nseq, bool packed) {
    const long long warps = (long long)D * N / 128 * (packed ? 1 : nseq);   // at work at once, in the worst case
    if (warps >= 608) return 0;
    const long long want = 4 * 608;   // warps
    const long long per = tokens * std::max(1LL, (long long)D * N / 128) / want;
    const long long seg = std::max(256LL, (per + 63) / 64 * 64);
    return tokens / (packed ? 1 : nseq) <= seg ? 0 : (int)std::min<long long>(seg, 1 << 20);
}
ScanFwdLayout scan_fwd_layout(long long tokens, int D, int N, int nseq, bool packed) {
    ScanFwdLayout l{};
    l.seg = scan_fwd_segment(tokens, D, N, nseq, packed);
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
cudaError_t launch_scan_states(const ScanArgs& a) {
    const cudaError_t e = a.dtype == GDN_BF16 ? adj_n<__nv_bfloat16>(a) : adj_n<float>(a);
    return e == cudaSuccess ? launch_scan_join(a, true) : e;
}
cudaError_t launch_scan_step(const ScanStepArgs& a) {
    return a.dtype == GDN_BF16 ? step_n<__nv_bfloat16>(a) : step_n<float>(a);
}

}  // namespace gdn
