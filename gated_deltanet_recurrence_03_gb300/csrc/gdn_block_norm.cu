// The surroundings of a layer's block in one pass over the rows: the norm after the block, its gate and
// residual scale, the residual add, and the norm before the next block.  Per row of D values
//     y = b / sqrt(mean(b^2) + eps) w_post,   r = x + c sigmoid(u) y,   n = r / sqrt(mean(r^2) + eps) w_pre
// (c = 1 and sigmoid(u) = 1 where they are not given; u is one logit a value or one a row), and its
// gradients for dr, dn (ib, ir the two inverse norms, bh = b ib, rh = r ir, s = sigmoid(u)):
//     h = dn w_pre,  dx = dr + ir (h - rh mean(h rh)),  dy = dx c s,  e = dy w_post,
//     db = ib (e - bh mean(e bh)),  du = dx c y s (1 - s),
//     dw_post = sum dy bh,  dw_pre = sum dn rh,  dc = sum dx s y   (sums over the rows).
// n is formed from r before r is rounded to its storage type, and the gradients from r formed again from
// x, b, u in fp32, so neither carries r's rounding.
//
// A row is read from HBM once: it passes through a ring in shared memory (bulk copies, up to four rows ahead of a group
// of threads) and is held in registers between the two norms; one block an SM of up to 1024 threads walks the rows.
// The forward pass is bound by HBM and its instructions alike, the backward pass by its instructions and shared-memory
// reads.  Measured, 16,384 rows of 4096 bf16 values with a gate: forward 119 us, 0.84 of the measured copy bandwidth
// (161 us with loads straight to registers; 130 us with the next row's in registers, whose moves wait for the loads;
// 197 us with both sums of a row in one exchange; 126 us with one vector a thread); backward 207 us, 0.77 of it (from
// 627: sums of the weights' gradients in registers 444, one pass over the row 374, packed arithmetic 333, one sum for
// the two weights 318, the ring 254, two vectors a thread 207).
#include <algorithm>

#include "norm_rows.cuh"

namespace gdn {
namespace {

// Logits below -87 act as -87 (1e-38): past 2^126 the fast division is not defined.  A NaN stays one.
__device__ __forceinline__ float sigmoid_f(float u) { return __fdividef(1.f, 1.f + __expf(u < -87.f ? 87.f : -u)); }
__device__ __forceinline__ V8 gate8(const V8& u) {
    V8 s;
#pragma unroll
    for (int i = 0; i < 4; ++i) s.v[i] = make_float2(sigmoid_f(u.v[i].x), sigmoid_f(u.v[i].y));
    return s;
}

__device__ __forceinline__ void set_up(const RowSmem& s, const BlockNormArgs& a, int groups) {
    for (int i = threadIdx.x; i < groups * 128; i += blockDim.x) s.red[i] = 0.f;
    if ((int)threadIdx.x < groups) ring_init(s.bars + threadIdx.x * kRingWords);
    if (threadIdx.x == 0) *s.abort = 0;
    tc::mbar_fence_init();
    for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
        s.m[c] = a.res_scale ? a.post_w[c] * a.res_scale[c] : a.post_w[c];
        s.wq[c] = a.pre_w[c];
    }
    __syncthreads();
}

template <int V, typename T, bool GATE>
__global__ void __launch_bounds__(V == 1 ? 1024 : 512, 1)
block_norm_fwd_kernel(const __grid_constant__ BlockNormArgs a, int tpr, int stages) {
    constexpr int N = GATE ? 3 : 2;
    extern __shared__ __align__(128) uint8_t smem[];
    const Group g{tpr, (int)threadIdx.x / tpr, (int)threadIdx.x % tpr};
    const int nv = a.D / kVec, groups = blockDim.x / tpr;
    const RowSmem sm = carve(smem, groups, a.D);
    set_up(sm, a, groups);
    float* const red = sm.red + g.id * 128;
    const float invD = 1.f / (float)a.D;
    const bool one = !GATE && a.gate;
    BulkRing<T, N> ring;
    ring.src[0] = a.b;
    ring.src[1] = a.x;
    if constexpr (GATE) ring.src[2] = a.gate;
    ring.base = sm.rings + (size_t)g.id * stages * N * a.D * sizeof(T);
    ring.bars = sm.bars + g.id * kRingWords;
    ring.D = a.D;
    ring.stages = stages;
    ring.abort = sm.abort;
    ring.status = a.status;
    ring.status_flag = kStatusTimeout;
    ring.limit_ns = kWaitLimitNs;
    const long long step = (long long)gridDim.x * groups, first = (long long)blockIdx.x * groups + g.id;
    if (g.tid == 0)
        for (int k = 0; k < stages && first + k * step < a.rows; ++k) ring.issue(k, first + k * step);
    int k = 0;
    for (long long row = first; row < a.rows; row += step, ++k) {
        const float logit = one ? to_f32(static_cast<const T*>(a.gate)[row]) : 0.f;
        const bool go = ring.wait(k);
        const T *pb = ring.at(k, 0), *px = ring.at(k, 1), *pu = GATE ? ring.at(k, N - 1) : nullptr;
        float2 q = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = g.tid + i * tpr;
            if (c < nv) {
                const V8 b = load8(pb + c * kVec);
#pragma unroll
                for (int e = 0; e < 4; ++e) q = fma2(b.v[e], b.v[e], q);
            }
        }
        float sum[1] = {q.x + q.y};
        group_sum(sum, red, g);
        // past this every thread of the group has finished the previous row: its stage is free
        if (g.tid == 0 && go && k > 0 && stages > 1 && row + (stages - 1) * step < a.rows)
            ring.issue(k + stages - 1, row + (stages - 1) * step);
        const float ib = rsqrtf(fmaf(sum[0], invD, a.eps)) * (one ? sigmoid_f(logit) : 1.f);
        V8 r[V];
        const size_t base = (size_t)row * a.D;
        q = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = g.tid + i * tpr;
            if (c < nv) {
                const V8 b = load8(pb + c * kVec), x = load8(px + c * kVec);
                V8 w = load8(sm.m + c * kVec);
                if constexpr (GATE) {
                    const V8 s = gate8(load8(pu + c * kVec));
#pragma unroll
                    for (int e = 0; e < 4; ++e) w.v[e] = mul2(w.v[e], s.v[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    r[i].v[e] = fma2(mul2(b.v[e], all2(ib)), w.v[e], x.v[e]);
                    q = fma2(r[i].v[e], r[i].v[e], q);
                }
                store8(static_cast<T*>(a.r) + base + c * kVec, r[i]);
            }
        }
        sum[0] = q.x + q.y;
        group_sum(sum, red + 64, g);
        const float ir = rsqrtf(fmaf(sum[0], invD, a.eps));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = g.tid + i * tpr;
            if (c < nv) {
                V8 y = load8(sm.wq + c * kVec);
#pragma unroll
                for (int e = 0; e < 4; ++e) y.v[e] = mul2(mul2(r[i].v[e], all2(ir)), y.v[e]);
                store8(static_cast<T*>(a.n) + base + c * kVec, y);
            }
        }
        if (stages == 1 && row + step < a.rows) {
            group_sync(g);
            if (g.tid == 0 && go) ring.issue(k + 1, row + step);
        }
    }
    if (g.tid == 0) ring.drain();
}

// Backward.  With m = w_post c everything but the weights' sums needs only m and w_pre: e = dx s m (= dy w_post),
// du = e bh (1 - s), and the sums of dw_post and dc are c A and w_post A with one A = sum dx s bh.  The sums over
// the rows stay in registers; a block's groups are added in order in shared memory, part [gridDim.x][2 D] gets the
// blocks' sums (A, then dw_pre), and block_norm_sums_kernel adds those in order.
template <int V, typename T, bool GATE>
__global__ void __launch_bounds__(V == 1 ? 1024 : 512, 1)
block_norm_bwd_kernel(const __grid_constant__ BlockNormArgs a, float* __restrict__ part, int tpr, int stages) {
    constexpr int N = GATE ? 5 : 4;
    extern __shared__ __align__(128) uint8_t smem[];
    const Group g{tpr, (int)threadIdx.x / tpr, (int)threadIdx.x % tpr};
    const int nv = a.D / kVec, groups = blockDim.x / tpr;
    const RowSmem sm = carve(smem, groups, a.D);
    set_up(sm, a, groups);
    float* const red = sm.red + g.id * 128;
    const float invD = 1.f / (float)a.D;
    const bool one = !GATE && a.gate;
    BulkRing<T, N> ring;
    ring.src[0] = a.b;
    ring.src[1] = a.x;
    ring.src[2] = a.gn;
    ring.src[3] = a.gr;
    if constexpr (GATE) ring.src[4] = a.gate;
    ring.base = sm.rings + (size_t)g.id * stages * N * a.D * sizeof(T);
    ring.bars = sm.bars + g.id * kRingWords;
    ring.D = a.D;
    ring.stages = stages;
    ring.abort = sm.abort;
    ring.status = a.status;
    ring.status_flag = kStatusTimeout;
    ring.limit_ns = kWaitLimitNs;
    const long long step = (long long)gridDim.x * groups, first = (long long)blockIdx.x * groups + g.id;
    if (g.tid == 0)
        for (int k = 0; k < stages && first + k * step < a.rows; ++k) ring.issue(k, first + k * step);
    V8 gA[V], gq[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) gA[i].v[e] = gq[i].v[e] = make_float2(0.f, 0.f);
    int k = 0;
    for (long long row = first; row < a.rows; row += step, ++k) {
        const float logit = one ? to_f32(static_cast<const T*>(a.gate)[row]) : 0.f;
        const bool go = ring.wait(k);
        const T *pb = ring.at(k, 0), *px = ring.at(k, 1), *pn = ring.at(k, 2), *pr = ring.at(k, 3),
                *pu = GATE ? ring.at(k, N - 1) : nullptr;
        float2 q = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = g.tid + i * tpr;
            if (c < nv) {
                const V8 b = load8(pb + c * kVec);
#pragma unroll
                for (int e = 0; e < 4; ++e) q = fma2(b.v[e], b.v[e], q);
            }
        }
        float s1[1] = {q.x + q.y};
        group_sum(s1, red, g);
        // past this every thread of the group has finished the previous row: its stage is free
        if (g.tid == 0 && go && k > 0 && stages > 1 && row + (stages - 1) * step < a.rows)
            ring.issue(k + stages - 1, row + (stages - 1) * step);
        const float ib = rsqrtf(fmaf(s1[0], invD, a.eps));
        const float gate1 = one ? sigmoid_f(logit) : 1.f;
        const size_t base = (size_t)row * a.D;
        V8 r[V], s[V];
        float2 qh = make_float2(0.f, 0.f);
        q = qh;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = g.tid + i * tpr;
            if (c < nv) {
                if constexpr (GATE) s[i] = gate8(load8(pu + c * kVec));
                const V8 b = load8(pb + c * kVec), x = load8(px + c * kVec), m = load8(sm.m + c * kVec);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 y = mul2(mul2(b.v[e], all2(ib)), m.v[e]);
                    r[i].v[e] = fma2(y, GATE ? s[i].v[e] : all2(gate1), x.v[e]);
                    q = fma2(r[i].v[e], r[i].v[e], q);
                }
                const V8 dn = load8(pn + c * kVec), wq = load8(sm.wq + c * kVec);
#pragma unroll
                for (int e = 0; e < 4; ++e) qh = fma2(mul2(dn.v[e], wq.v[e]), r[i].v[e], qh);
            }
        }
        float s2[2] = {q.x + q.y, qh.x + qh.y};
        group_sum(s2, red + 64, g);
        const float ir = rsqrtf(fmaf(s2[0], invD, a.eps));
        const float mh = s2[1] * ir * invD;   // mean(h rh)
        float2 qe = make_float2(0.f, 0.f);    // sum e bh
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = g.tid + i * tpr;
            if (c < nv) {
                const V8 dn = load8(pn + c * kVec), wq = load8(sm.wq + c * kVec);
                V8 dx = load8(pr + c * kVec);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 rh = mul2(r[i].v[e], all2(ir));
                    gq[i].v[e] = fma2(dn.v[e], rh, gq[i].v[e]);
                    dx.v[e] = fma2(all2(ir), fma2(rh, all2(-mh), mul2(dn.v[e], wq.v[e])), dx.v[e]);
                }
                store8(static_cast<T*>(a.gx) + base + c * kVec, dx);
                const V8 b = load8(pb + c * kVec), m = load8(sm.m + c * kVec);
                V8 du;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 bh = mul2(b.v[e], all2(ib)), sdx = mul2(dx.v[e], GATE ? s[i].v[e] : all2(gate1));
                    gA[i].v[e] = fma2(sdx, bh, gA[i].v[e]);
                    r[i].v[e] = mul2(sdx, m.v[e]);   // e
                    const float2 eb = mul2(r[i].v[e], bh);
                    qe = add2(qe, eb);
                    if (GATE) du.v[e] = fma2(eb, make_float2(-s[i].v[e].x, -s[i].v[e].y), eb);
                }
                if (GATE) store8(static_cast<T*>(a.ggate) + base + c * kVec, du);
            }
        }
        float s3[1] = {qe.x + qe.y};
        group_sum(s3, red + 32, g);   // not the next row's first buffer
        const float me = -s3[0] * invD;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = g.tid + i * tpr;
            if (c < nv) {
                V8 b = load8(pb + c * kVec);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    b.v[e] = mul2(all2(ib), fma2(mul2(b.v[e], all2(ib)), all2(me), r[i].v[e]));
                store8(static_cast<T*>(a.gb) + base + c * kVec, b);
            }
        }
        if (one && g.tid == 0) static_cast<T*>(a.ggate)[row] = from_f32<T>(s3[0] * (1.f - gate1));
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
            V8* acc[2] = {&gA[i], &gq[i]};
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

// Column c of the 2 D summed over the blocks' rows of `part`, in order: 32 columns a block, 32 row groups added by
// a shared-memory tree; then the weights' gradients c A, sum dn rh, w_post A (each [D], or nullptr).
__global__ void __launch_bounds__(1024) block_norm_sums_kernel(const float* __restrict__ part, int rows,
                                                               const __grid_constant__ BlockNormArgs a) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < 2 * a.D)
        for (int r = grp; r < rows; r += 32) s += part[(size_t)r * 2 * a.D + c];
    red[grp][lane] = s;
    __syncthreads();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (grp < o) red[grp][lane] += red[grp + o][lane];
        __syncthreads();
    }
    if (grp != 0 || c >= 2 * a.D) return;
    s = red[0][lane];
    if (c >= a.D) {
        if (a.g_pre) a.g_pre[c - a.D] = s;
    } else {
        if (a.g_post) a.g_post[c] = a.res_scale ? s * a.res_scale[c] : s;
        if (a.g_scale) a.g_scale[c] = s * a.post_w[c];
    }
}

RowShape fwd_shape(const BlockNormArgs& a) {
    const bool full = a.gate && a.gate_cols > 1;
    return row_shape(a.D, a.rows, (full ? 3 : 2) * a.D * (a.dtype == GDN_BF16 ? 2 : 4));
}
// The backward's blocks do not depend on the type or the gate, so that the scratch is a function of rows and D: the
// row bytes only change how many groups share a block, and blocks is at most one for each SM.
RowShape bwd_shape(const BlockNormArgs& a) {
    const bool full = a.gate && a.gate_cols > 1;
    return row_shape(a.D, a.rows, (full ? 5 : 4) * a.D * (a.dtype == GDN_BF16 ? 2 : 4));
}

template <int V, typename T, bool GATE>
cudaError_t fwd_one(const BlockNormArgs& a, const RowShape& s) {
    const cudaError_t e = allow_smem<block_norm_fwd_kernel<V, T, GATE>>();
    if (e != cudaSuccess) return e;
    block_norm_fwd_kernel<V, T, GATE><<<s.blocks, s.tpr * s.groups, s.smem, a.stream>>>(a, s.tpr, s.stages);
    return cudaGetLastError();
}
template <int V, typename T, bool GATE>
cudaError_t bwd_one(const BlockNormArgs& a, const RowShape& s, float* part) {
    const cudaError_t e = allow_smem<block_norm_bwd_kernel<V, T, GATE>>();
    if (e != cudaSuccess) return e;
    block_norm_bwd_kernel<V, T, GATE><<<s.blocks, s.tpr * s.groups, s.smem, a.stream>>>(a, part, s.tpr, s.stages);
    return cudaGetLastError();
}
template <typename T>
cudaError_t fwd_typed(const BlockNormArgs& a) {
    const RowShape s = fwd_shape(a);
    const bool full = a.gate && a.gate_cols > 1;
    if (s.v == 1) return full ? fwd_one<1, T, true>(a, s) : fwd_one<1, T, false>(a, s);
    return full ? fwd_one<2, T, true>(a, s) : fwd_one<2, T, false>(a, s);
}
template <typename T>
cudaError_t bwd_typed(const BlockNormArgs& a, const RowShape& s, float* part) {
    const bool full = a.gate && a.gate_cols > 1;
    if (s.v == 1) return full ? bwd_one<1, T, true>(a, s, part) : bwd_one<1, T, false>(a, s, part);
    return full ? bwd_one<2, T, true>(a, s, part) : bwd_one<2, T, false>(a, s, part);
}

}  // namespace

cudaError_t launch_block_norm_fwd(const BlockNormArgs& a) {
    return a.dtype == GDN_BF16 ? fwd_typed<__nv_bfloat16>(a) : fwd_typed<float>(a);
}

size_t block_norm_bwd_workspace_bytes(long long rows, int D) {
    return (size_t)std::max(1LL, std::min(152LL, rows)) * 2 * D * 4;
}

cudaError_t launch_block_norm_bwd(const BlockNormArgs& a) {
    const RowShape s = bwd_shape(a);
    float* part = (a.g_post || a.g_pre || a.g_scale) ? static_cast<float*>(a.workspace) : nullptr;
    if (s.blocks) {
        const cudaError_t e = a.dtype == GDN_BF16 ? bwd_typed<__nv_bfloat16>(a, s, part) : bwd_typed<float>(a, s, part);
        if (e != cudaSuccess) return e;
    }
    if (!part) return cudaSuccess;
    block_norm_sums_kernel<<<(unsigned)((2 * a.D + 31) / 32), 1024, 0, a.stream>>>(part, s.blocks, a);
    return cudaGetLastError();
}

}  // namespace gdn
