// Layer norm over rows of D values with the residual add in front of it: r = x + b, with m = mean(r),
// v = mean((r - m)^2) and rh = (r - m) / sqrt(v + eps),
//     n = rh w + bias,
// and its gradients for dr, dn (inv = 1 / sqrt(v + eps)):
//     h = dn w,  dx = db = dr + inv (h - mean(h) - rh mean(h rh)),  dw = sum dn rh,  dbias = sum dn (over the rows).
// n is formed from r before its rounding, and the gradients from r formed again from x and b.
//
// No sum of squares around zero is taken, so that a row far from zero loses no more than its mean's rounding: the mean is off
// by some 2^-24 |m| for each addition that a value passes (8 to 14), n and rh by that over the row's deviation.  Forward,
// every warp takes the mean m_w of its n_w values first and sums around that, and the warps' sums, exchanged once, join by
// m = sum n_w m_w / D, sum (r - m)^2 = sum [M_w + n_w (m_w - m)^2] (exact but for the roundings of the m_w, of which the sum of
// squares keeps only products with the m_w - m).  Backward the row's mean is exchanged before the other three sums.
// Rows pass through the ring of the block norm (norm_rows.cuh) and are held in registers between the sums.
//
// 16,384 rows of 4096 bf16 values with the residual: forward 94.6 us, 0.84 of the measured copy bandwidth (two exchanges a
// row 101.3, and two row groups an SM 104.5 us); gradients 132.7 us, 0.74 of it, HBM 58 %, issue slots 45 % of their rates:
// each row's two exchanges with only two row groups of 128 registers a thread on an SM.  One exchange of four sums: 144 us
// (more instructions); three groups, registers spilled: the same as two.
#include "norm_rows.cuh"

namespace gdn {
namespace {

// Threads of a block with two vectors a thread: with more row groups at work on an SM the exchanges of one hide behind the
// others (16384 x 4096 forward: 512 threads 98.9, 768 94.6, 1024 102.8 us, where registers spill; gradients 512).
constexpr int kFwdThreads = 768, kBwdThreads = 512;

__device__ __forceinline__ void set_up(const RowSmem& s, const float* w, const float* bias, int D, int groups) {
    for (int i = threadIdx.x; i < groups * 128; i += blockDim.x) s.red[i] = 0.f;
    if ((int)threadIdx.x < groups) ring_init(s.bars + threadIdx.x * kRingWords);
    if (threadIdx.x == 0) *s.abort = 0;
    tc::mbar_fence_init();
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
        s.m[c] = w[c];
        s.wq[c] = bias ? bias[c] : 0.f;
    }
    __syncthreads();
}

constexpr int kWarps = 16;   // of a row group at most
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
// What the warps of a row group hold: `count` [kWarps] (n_w, zero past the group's warps), shared by the block.
__device__ __forceinline__ float set_up_counts(float* count, const Group& g, int nv, int V) {
    int n = 0;
    for (int i = 0; i < V; ++i) n += min(max(nv - i * g.tpr - (g.tid & ~31), 0), 32) * kVec;
    if (g.id == 0 && (g.tid & 31) == 0) count[g.tid >> 5] = (float)n;
    if (g.id == 0 && g.tid < kWarps && g.tid >= g.tpr >> 5) count[g.tid] = 0.f;
    __syncthreads();
    return (float)n;
}

// The group's ring: x, [b], then the backward's dn, [dr].
template <typename T, int N>
__device__ __forceinline__ void set_up_ring(BulkRing<T, N>& ring, const RowSmem& sm, const LayerNormArgs& a, const Group& g,
                                            int stages) {
    ring.base = sm.rings + (size_t)g.id * stages * N * a.D * sizeof(T);
    ring.bars = sm.bars + g.id * kRingWords;
    ring.D = a.D;
    ring.stages = stages;
    ring.abort = sm.abort;
    ring.status = a.status;
    ring.status_flag = kStatusTimeout;
    ring.limit_ns = kWaitLimitNs;
}

template <int V, typename T, bool ADD>
__global__ void __launch_bounds__(V == 1 ? 1024 : kFwdThreads, 1)
layer_norm_fwd_kernel(const __grid_constant__ LayerNormArgs a, int tpr, int stages) {
    constexpr int N = ADD ? 2 : 1;
    extern __shared__ __align__(128) uint8_t smem[];
    const Group g{tpr, (int)threadIdx.x / tpr, (int)threadIdx.x % tpr};
    const int nv = a.D / kVec, groups = blockDim.x / tpr;
    const RowSmem sm = carve(smem, groups, a.D);
    set_up(sm, a.w, a.bias, a.D, groups);
    float* const red = sm.red + g.id * 128;
    const float invD = 1.f / (float)a.D;
    float* const count = sm.red + 64;   // of group 0: the exchanges take 64 floats of a group's 128
    const float n_w = set_up_counts(count, g, nv, V), inv_w = n_w > 0.f ? 1.f / n_w : 0.f;
    const int nw = tpr >> 5;
    BulkRing<T, N> ring;
    ring.src[0] = a.x;
    if constexpr (ADD) ring.src[1] = a.b;
    set_up_ring(ring, sm, a, g, stages);
    const long long step = (long long)gridDim.x * groups, first = (long long)blockIdx.x * groups + g.id;
    if (g.tid == 0)
        for (int k = 0; k < stages && first + k * step < a.rows; ++k) ring.issue(k, first + k * step);
    int k = 0;
    for (long long row = first; row < a.rows; row += step, ++k) {
        const bool go = ring.wait(k);
        const size_t base = (size_t)row * a.D;
        V8 r[V];
        float2 q = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = g.tid + i * tpr;
            if (c < nv) {
                r[i] = load8(ring.at(k, 0) + c * kVec);
                if constexpr (ADD) {
                    const V8 b = load8(ring.at(k, 1) + c * kVec);
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[i].v[e] = add2(r[i].v[e], b.v[e]);
                    store8(static_cast<T*>(a.r) + base + c * kVec, r[i]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) q = add2(q, r[i].v[e]);
            }
        }
        float mean = warp_sum(q.x + q.y) * inv_w;
        q = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (g.tid + i * tpr < nv)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 d = add2(r[i].v[e], all2(-mean));
                    q = fma2(d, d, q);
                }
        float m2 = warp_sum(q.x + q.y);
        if (nw > 1) {
            float* const buf = red + (k & 1) * 2 * kWarps;   // m_w, M_w; the other one may still be read
            if ((g.tid & 31) == 0) {
                buf[g.tid >> 5] = mean;
                buf[kWarps + (g.tid >> 5)] = m2;
            }
            group_sync(g);
            mean = m2 = 0.f;
            for (int w = 0; w < nw; w += 4) {
                const float4 n = *reinterpret_cast<const float4*>(count + w), m = *reinterpret_cast<const float4*>(buf + w);
                mean += fmaf(n.x, m.x, n.y * m.y) + fmaf(n.z, m.z, n.w * m.w);
            }
            mean *= invD;
            for (int w = 0; w < nw; w += 4) {
                const float4 n = *reinterpret_cast<const float4*>(count + w), m = *reinterpret_cast<const float4*>(buf + w);
                const float4 q4 = *reinterpret_cast<const float4*>(buf + kWarps + w);
                const float dx = m.x - mean, dy = m.y - mean, dz = m.z - mean, dw = m.w - mean;
                m2 += (fmaf(n.x * dx, dx, q4.x) + fmaf(n.y * dy, dy, q4.y)) +
                      (fmaf(n.z * dz, dz, q4.z) + fmaf(n.w * dw, dw, q4.w));
            }
        } else {
            __syncwarp();
        }
        // past this every thread of the group has read this row: its stage is free
        if (g.tid == 0 && go && row + stages * step < a.rows) ring.issue(k + stages, row + stages * step);
        const float inv = rsqrtf(fmaf(m2, invD, a.eps));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = g.tid + i * tpr;
            if (c < nv) {
                const V8 w = load8(sm.m + c * kVec);
                V8 y = load8(sm.wq + c * kVec);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y.v[e] = fma2(mul2(add2(r[i].v[e], all2(-mean)), all2(inv)), w.v[e], y.v[e]);
                store8(static_cast<T*>(a.n) + base + c * kVec, y);
            }
        }
    }
    if (g.tid == 0) ring.drain();
}

// The sums over the rows stay in registers; a block's groups are added in order in shared memory, part [gridDim.x][2 D]
// gets the blocks' sums (dw, then dbias), and layer_norm_sums_kernel adds those in order.
template <int V, typename T, bool ADD, bool RES>
__global__ void __launch_bounds__(V == 1 ? 1024 : kBwdThreads, 1)
layer_norm_bwd_kernel(const __grid_constant__ LayerNormArgs a, float* __restrict__ part, int tpr, int stages) {
    constexpr int N = 2 + ADD + RES, DN = 1 + ADD;
    extern __shared__ __align__(128) uint8_t smem[];
    const Group g{tpr, (int)threadIdx.x / tpr, (int)threadIdx.x % tpr};
    const int nv = a.D / kVec, groups = blockDim.x / tpr;
    const RowSmem sm = carve(smem, groups, a.D);
    set_up(sm, a.w, nullptr, a.D, groups);
    float* const red = sm.red + g.id * 128;
    const float invD = 1.f / (float)a.D;
    BulkRing<T, N> ring;
    ring.src[0] = a.x;
    if constexpr (ADD) ring.src[1] = a.b;
    ring.src[DN] = a.gn;
    if constexpr (RES) ring.src[DN + 1] = a.gr;
    set_up_ring(ring, sm, a, g, stages);
    const long long step = (long long)gridDim.x * groups, first = (long long)blockIdx.x * groups + g.id;
    if (g.tid == 0)
        for (int k = 0; k < stages && first + k * step < a.rows; ++k) ring.issue(k, first + k * step);
    V8 gw[V], gb[V], w[V];   // the thread's columns are the same in every row
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (g.tid + i * tpr < nv) w[i] = load8(sm.m + (g.tid + i * tpr) * kVec);
#pragma unroll
        for (int e = 0; e < 4; ++e) gw[i].v[e] = gb[i].v[e] = make_float2(0.f, 0.f);
    }
    int k = 0;
    for (long long row = first; row < a.rows; row += step, ++k) {
        const bool go = ring.wait(k);
        V8 r[V], dn[V];
        float2 q = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = g.tid + i * tpr;
            if (c < nv) {
                r[i] = load8(ring.at(k, 0) + c * kVec);
                if constexpr (ADD) {
                    const V8 b = load8(ring.at(k, 1) + c * kVec);
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[i].v[e] = add2(r[i].v[e], b.v[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) q = add2(q, r[i].v[e]);
            }
        }
        float s1[1] = {q.x + q.y};
        group_sum(s1, red + 96, g);
        // past this every thread of the group has finished the previous row: its stage is free
        if (g.tid == 0 && go && k > 0 && stages > 1 && row + (stages - 1) * step < a.rows)
            ring.issue(k + stages - 1, row + (stages - 1) * step);
        const float2 m = all2(-s1[0] * invD);
        float2 qh = make_float2(0.f, 0.f), qr = qh;   // sums of h and h (r - m)
        q = qh;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = g.tid + i * tpr;
            if (c < nv) {
                dn[i] = load8(ring.at(k, DN) + c * kVec);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    r[i].v[e] = add2(r[i].v[e], m);
                    q = fma2(r[i].v[e], r[i].v[e], q);
                    const float2 h = mul2(dn[i].v[e], w[i].v[e]);
                    qh = add2(qh, h);
                    qr = fma2(h, r[i].v[e], qr);
                }
            }
        }
        float s[3] = {q.x + q.y, qh.x + qh.y, qr.x + qr.y};
        group_sum(s, red, g);
        const float inv = rsqrtf(fmaf(s[0], invD, a.eps));
        const float2 mh = all2(-s[1] * invD), mr = all2(-s[2] * inv * invD);   // -mean(h), -mean(h rh)
        const size_t base = (size_t)row * a.D;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = g.tid + i * tpr;
            if (c < nv) {
                V8 dx;
                if constexpr (RES) dx = load8(ring.at(k, DN + 1) + c * kVec);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 rh = mul2(r[i].v[e], all2(inv));
                    gw[i].v[e] = fma2(dn[i].v[e], rh, gw[i].v[e]);
                    gb[i].v[e] = add2(dn[i].v[e], gb[i].v[e]);
                    const float2 t = fma2(rh, mr, fma2(dn[i].v[e], w[i].v[e], mh));
                    dx.v[e] = RES ? fma2(all2(inv), t, dx.v[e]) : mul2(all2(inv), t);
                }
                store8(static_cast<T*>(a.gx) + base + c * kVec, dx);
            }
        }
        if (stages == 1 && row + step < a.rows) {
            group_sync(g);
            if (g.tid == 0 && go) ring.issue(k + 1, row + step);
        }
    }
    if (g.tid == 0) ring.drain();
    if (!part) return;
    float* p = part + (size_t)blockIdx.x * 2 * a.D;
    float* const sums = sm.m;   // [2 D]: the constants are done with
    for (int x = 0; x < groups; ++x) {   // the groups one after another
        __syncthreads();
        if (g.id != x) continue;
        float* to = x + 1 == groups ? p : sums;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (g.tid + i * tpr) * kVec;
            if (c >= a.D) continue;
            V8* acc[2] = {&gw[i], &gb[i]};
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                if (x > 0) {
                    const V8 o = load8(sums + y * a.D + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[y]->v[e] = add2(o.v[e], acc[y]->v[e]);
                }
                store8(to + y * a.D + c, *acc[y]);
            }
        }
    }
}

// Column c of the 2 D summed over the blocks' rows of `part`, in order: 32 columns a block, 32 row groups added by a
// shared-memory tree.
__global__ void __launch_bounds__(1024) layer_norm_sums_kernel(const float* __restrict__ part, int rows, int D,
                                                               float* __restrict__ gw, float* __restrict__ gbias) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < 2 * D)
        for (int r = grp; r < rows; r += 32) s += part[(size_t)r * 2 * D + c];
    red[grp][lane] = s;
    __syncthreads();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (grp < o) red[grp][lane] += red[grp + o][lane];
        __syncthreads();
    }
    if (grp != 0 || c >= 2 * D) return;
    float* to = c < D ? gw : gbias;
    if (to) to[c < D ? c : c - D] = red[0][lane];
}

int value_bytes(const LayerNormArgs& a) { return a.dtype == GDN_BF16 ? 2 : 4; }

template <int V, typename T, bool ADD>
cudaError_t fwd_one(const LayerNormArgs& a, const RowShape& s) {
    const cudaError_t e = allow_smem<layer_norm_fwd_kernel<V, T, ADD>>();
    if (e != cudaSuccess) return e;
    layer_norm_fwd_kernel<V, T, ADD><<<s.blocks, s.tpr * s.groups, s.smem, a.stream>>>(a, s.tpr, s.stages);
    return cudaGetLastError();
}
template <int V, typename T, bool ADD, bool RES>
cudaError_t bwd_one(const LayerNormArgs& a, const RowShape& s, float* part) {
    const cudaError_t e = allow_smem<layer_norm_bwd_kernel<V, T, ADD, RES>>();
    if (e != cudaSuccess) return e;
    layer_norm_bwd_kernel<V, T, ADD, RES><<<s.blocks, s.tpr * s.groups, s.smem, a.stream>>>(a, part, s.tpr, s.stages);
    return cudaGetLastError();
}
template <int V, typename T>
cudaError_t fwd_v(const LayerNormArgs& a, const RowShape& s) {
    return a.b ? fwd_one<V, T, true>(a, s) : fwd_one<V, T, false>(a, s);
}
template <int V, typename T>
cudaError_t bwd_v(const LayerNormArgs& a, const RowShape& s, float* part) {
    if (a.b) return a.gr ? bwd_one<V, T, true, true>(a, s, part) : bwd_one<V, T, true, false>(a, s, part);
    return a.gr ? bwd_one<V, T, false, true>(a, s, part) : bwd_one<V, T, false, false>(a, s, part);
}
template <typename T>
cudaError_t fwd_typed(const LayerNormArgs& a) {
    const RowShape s = row_shape(a.D, a.rows, (a.b ? 2 : 1) * a.D * value_bytes(a), kFwdThreads);
    return s.v == 1 ? fwd_v<1, T>(a, s) : fwd_v<2, T>(a, s);
}
template <typename T>
cudaError_t bwd_typed(const LayerNormArgs& a, const RowShape& s, float* part) {
    return s.v == 1 ? bwd_v<1, T>(a, s, part) : bwd_v<2, T>(a, s, part);
}

}  // namespace

cudaError_t launch_layer_norm_fwd(const LayerNormArgs& a) {
    return a.dtype == GDN_BF16 ? fwd_typed<__nv_bfloat16>(a) : fwd_typed<float>(a);
}

// At most one block for each SM, whatever the type and the tensors: the scratch is a function of rows and D.
size_t layer_norm_bwd_workspace_bytes(long long rows, int D) {
    return (size_t)std::max(1LL, std::min(152LL, rows)) * 2 * D * 4;
}

cudaError_t launch_layer_norm_bwd(const LayerNormArgs& a) {
    const RowShape s = row_shape(a.D, a.rows, (2 + (a.b != nullptr) + (a.gr != nullptr)) * a.D * value_bytes(a), kBwdThreads);
    float* part = a.gw || a.gbias ? static_cast<float*>(a.workspace) : nullptr;
    if (s.blocks) {
        const cudaError_t e = a.dtype == GDN_BF16 ? bwd_typed<__nv_bfloat16>(a, s, part) : bwd_typed<float>(a, s, part);
        if (e != cudaSuccess) return e;
    }
    if (!part) return cudaSuccess;
    layer_norm_sums_kernel<<<(unsigned)((2 * a.D + 31) / 32), 1024, 0, a.stream>>>(part, s.blocks, a.D, a.gw, a.gbias);
    return cudaGetLastError();
}

}  // namespace gdn
