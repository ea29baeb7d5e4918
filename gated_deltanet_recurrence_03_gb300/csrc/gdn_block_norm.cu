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
#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kVec = 8;   // values of one vector of a thread

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Sums of N values over the block's threads, in a fixed order; every thread gets them.  `buf` holds 32 N
// floats and is free again after the next call's barrier (callers alternate two buffers).
template <int N>
__device__ __forceinline__ void block_sum(float (&x)[N], float* buf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
    if (nw == 1) return;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) buf[i * 32 + warp] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = lane < nw ? buf[i * 32 + lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
    }
}

__device__ __forceinline__ float sigmoid_f(float u) { return 1.f / (1.f + __expf(-u)); }

template <int V, typename T>
__global__ void __launch_bounds__(V == 1 ? 512 : 1024)
block_norm_fwd_kernel(const __grid_constant__ BlockNormArgs a) {
    __shared__ float buf[2][32];
    const int nv = a.D / kVec, tid = threadIdx.x, NT = blockDim.x;
    const size_t row = blockIdx.x, base = row * a.D;
    const T* x = static_cast<const T*>(a.x) + base;
    const T* b = static_cast<const T*>(a.b) + base;
    float fb[V][8], fr[V][8];
    float sum[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * NT;
#pragma unroll
        for (int e = 0; e < 8; ++e) fb[i][e] = fr[i][e] = 0.f;
        if (c < nv) {
            load8(b + c * kVec, fb[i]);
            load8(x + c * kVec, fr[i]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] = fmaf(fb[i][e], fb[i][e], sum[0]);
    }
    block_sum(sum, buf[0]);
    const float ib = rsqrtf(sum[0] / (float)a.D + a.eps);
    const float gate1 = a.gate && a.gate_cols == 1 ? sigmoid_f(to_f32(static_cast<const T*>(a.gate)[row])) : 1.f;
    sum[0] = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * NT;
        if (c < nv) {
            float w[8], t[8];
            load8(a.post_w + c * kVec, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = fb[i][e] * ib * w[e] * gate1;
            if (a.res_scale) {
                load8(a.res_scale + c * kVec, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] *= w[e];
            }
            if (a.gate && a.gate_cols > 1) {
                load8(static_cast<const T*>(a.gate) + base + c * kVec, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] *= sigmoid_f(w[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                fr[i][e] += t[e];
                sum[0] = fmaf(fr[i][e], fr[i][e], sum[0]);
            }
        }
    }
    block_sum(sum, buf[1]);
    const float ir = rsqrtf(sum[0] / (float)a.D + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * NT;
        if (c < nv) {
            float w[8];
            load8(a.pre_w + c * kVec, w);
            store8(static_cast<T*>(a.r) + base + c * kVec, fr[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] *= fr[i][e] * ir;
            store8(static_cast<T*>(a.n) + base + c * kVec, w);
        }
    }
}

// Backward: a block takes rows blockIdx.x, + gridDim.x, ... and keeps its columns' three weight sums in
// registers over them; part [gridDim.x][3 D] gets them, and column_sum_kernel adds the blocks in order.
template <int V, typename T>
__global__ void __launch_bounds__(V == 1 ? 512 : 1024)
block_norm_bwd_kernel(const __grid_constant__ BlockNormArgs a, float* __restrict__ part) {
    __shared__ float buf[3][64];
    const int nv = a.D / kVec, tid = threadIdx.x, NT = blockDim.x;
    float gp[V][8], gq[V][8], gc[V][8];   // sums of dw_post, dw_pre, dc
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) gp[i][e] = gq[i][e] = gc[i][e] = 0.f;
    const float invD = 1.f / (float)a.D;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const size_t base = (size_t)row * a.D;
        float fb[V][8], fr[V][8], s1[1] = {0.f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = tid + i * NT;
#pragma unroll
            for (int e = 0; e < 8; ++e) fb[i][e] = fr[i][e] = 0.f;
            if (c < nv) {
                load8(static_cast<const T*>(a.b) + base + c * kVec, fb[i]);
                load8(static_cast<const T*>(a.x) + base + c * kVec, fr[i]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) s1[0] = fmaf(fb[i][e], fb[i][e], s1[0]);
        }
        block_sum(s1, buf[0]);
        const float ib = rsqrtf(s1[0] * invD + a.eps);
        const float gate1 = a.gate && a.gate_cols == 1 ? sigmoid_f(to_f32(static_cast<const T*>(a.gate)[row])) : 1.f;
        float s2[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = tid + i * NT;
            if (c < nv) {
                float w[8], t[8], dn[8];
                load8(a.post_w + c * kVec, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = fb[i][e] * ib * w[e] * gate1;
                if (a.res_scale) {
                    load8(a.res_scale + c * kVec, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) t[e] *= w[e];
                }
                if (a.gate && a.gate_cols > 1) {
                    load8(static_cast<const T*>(a.gate) + base + c * kVec, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) t[e] *= sigmoid_f(w[e]);
                }
                load8(static_cast<const T*>(a.gn) + base + c * kVec, dn);
                load8(a.pre_w + c * kVec, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    fr[i][e] += t[e];
                    s2[0] = fmaf(fr[i][e], fr[i][e], s2[0]);
                    s2[1] = fmaf(dn[e] * w[e], fr[i][e], s2[1]);
                }
            }
        }
        block_sum(s2, buf[1]);
        const float ir = rsqrtf(s2[0] * invD + a.eps);
        const float mh = s2[1] * ir * invD;   // mean(h rh)
        float s3[2] = {0.f, 0.f};             // sum e bh, sum du / (s (1 - s)) of a one-logit gate
        float fe[V][8];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = tid + i * NT;
            if (c < nv) {
                float wq[8], dn[8], dx[8], wp[8], cs[8], s[8];
                load8(a.pre_w + c * kVec, wq);
                load8(static_cast<const T*>(a.gn) + base + c * kVec, dn);
                load8(static_cast<const T*>(a.gr) + base + c * kVec, dx);
                load8(a.post_w + c * kVec, wp);
#pragma unroll
                for (int e = 0; e < 8; ++e) cs[e] = 1.f;
                if (a.res_scale) load8(a.res_scale + c * kVec, cs);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] = gate1;
                if (a.gate && a.gate_cols > 1) {
                    load8(static_cast<const T*>(a.gate) + base + c * kVec, s);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[e] = sigmoid_f(s[e]);
                }
                float du[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float rh = fr[i][e] * ir, bh = fb[i][e] * ib, y = bh * wp[e];
                    gq[i][e] = fmaf(dn[e], rh, gq[i][e]);
                    dx[e] += ir * (dn[e] * wq[e] - rh * mh);
                    gc[i][e] = fmaf(dx[e] * s[e], y, gc[i][e]);
                    const float dy = dx[e] * cs[e] * s[e];
                    gp[i][e] = fmaf(dy, bh, gp[i][e]);
                    fe[i][e] = dy * wp[e];
                    s3[0] = fmaf(fe[i][e], bh, s3[0]);
                    const float d = dx[e] * cs[e] * y;
                    s3[1] += d;
                    du[e] = d * s[e] * (1.f - s[e]);
                    fb[i][e] = bh;
                }
                store8(static_cast<T*>(a.gx) + base + c * kVec, dx);
                if (a.gate && a.gate_cols > 1) store8(static_cast<T*>(a.ggate) + base + c * kVec, du);
            }
        }
        block_sum(s3, buf[2]);
        const float me = s3[0] * invD;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = tid + i * NT;
            if (c < nv) {
#pragma unroll
                for (int e = 0; e < 8; ++e) fe[i][e] = ib * (fe[i][e] - fb[i][e] * me);
                store8(static_cast<T*>(a.gb) + base + c * kVec, fe[i]);
            }
        }
        if (tid == 0 && a.gate && a.gate_cols == 1)
            static_cast<T*>(a.ggate)[row] = from_f32<T>(s3[1] * gate1 * (1.f - gate1));
    }
    if (part) {
        float* p = part + (size_t)blockIdx.x * 3 * a.D;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = tid + i * NT;
            if (c < nv) {
                store8(p + c * kVec, gp[i]);
                store8(p + a.D + c * kVec, gq[i]);
                store8(p + 2 * a.D + c * kVec, gc[i]);
            }
        }
    }
}

constexpr int kBwdBlocks = 608;   // 152 SMs x 4

long long bwd_blocks(long long rows) { return rows < kBwdBlocks ? rows : kBwdBlocks; }

// Vectors a thread holds and the block's threads: one vector a thread up to 512 threads, then more.
void shape_of(int D, int& v, int& threads) {
    const int nv = D / kVec;
    v = nv <= 512 ? 1 : (nv <= 1024 ? 2 : 4);
    threads = ((nv + v - 1) / v + 31) / 32 * 32;
}

}  // namespace

cudaError_t launch_block_norm_fwd(const BlockNormArgs& a) {
    int v, nt;
    shape_of(a.D, v, nt);
    const unsigned grid = (unsigned)a.rows;
#define GDN_BN_FWD(V_)                                                                          \
    if (v == V_) {                                                                              \
        if (a.dtype == GDN_BF16) block_norm_fwd_kernel<V_, __nv_bfloat16><<<grid, nt, 0, a.stream>>>(a); \
        else block_norm_fwd_kernel<V_, float><<<grid, nt, 0, a.stream>>>(a);                    \
    }
    GDN_BN_FWD(1) GDN_BN_FWD(2) GDN_BN_FWD(4)
#undef GDN_BN_FWD
    return cudaGetLastError();
}

size_t block_norm_bwd_workspace_bytes(long long rows, int D) { return (size_t)bwd_blocks(rows) * 3 * D * 4 + (size_t)3 * D * 4; }

cudaError_t launch_block_norm_bwd(const BlockNormArgs& a) {
    int v, nt;
    shape_of(a.D, v, nt);
    const unsigned grid = (unsigned)bwd_blocks(a.rows);
    float* part = (a.g_post || a.g_pre || a.g_scale) ? static_cast<float*>(a.workspace) : nullptr;
    if (grid) {
#define GDN_BN_BWD(V_)                                                                          \
    if (v == V_) {                                                                              \
        if (a.dtype == GDN_BF16) block_norm_bwd_kernel<V_, __nv_bfloat16><<<grid, nt, 0, a.stream>>>(a, part); \
        else block_norm_bwd_kernel<V_, float><<<grid, nt, 0, a.stream>>>(a, part);              \
    }
        GDN_BN_BWD(1) GDN_BN_BWD(2) GDN_BN_BWD(4)
#undef GDN_BN_BWD
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !part) return e;
    float* sums = part + (size_t)grid * 3 * a.D;
    column_sum_kernel<<<(unsigned)((3 * a.D + 31) / 32), kColSumThreads, 0, a.stream>>>(part, grid, 3 * a.D, sums);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    float* dst[3] = {a.g_post, a.g_pre, a.g_scale};
    for (int i = 0; i < 3; ++i)
        if (dst[i]) {
            e = cudaMemcpyAsync(dst[i], sums + (size_t)i * a.D, (size_t)a.D * 4, cudaMemcpyDeviceToDevice, a.stream);
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

}  // namespace gdn
