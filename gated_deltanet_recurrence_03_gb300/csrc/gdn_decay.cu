// Linear attention with a decay for each value head: the scan behind gdn_decay_attn_fwd and, three times,
// behind gdn_decay_attn_bwd (gdn_internal.cuh, DecayScan).  The token-by-token form on CUDA cores: one CTA
// owns one (sequence, value head) state, dk / 32 adjacent lanes own one of its columns (32 rows each, in
// registers), and the tokens' q, k and v are staged through shared memory a few at a time.
#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kTB = 16;   // tokens staged per round

template <int DK, int DV, typename T>
__global__ void __launch_bounds__(DV * (DK / 32))
decay_serial_kernel(const __grid_constant__ DecayArgs a) {
    constexpr int SPLIT = DK / 32, NT = DV * SPLIT;
    __shared__ __align__(16) float sk[kTB][DK];
    __shared__ __align__(16) float sq[kTB][DK];
    __shared__ float sv[kTB][DV];
    const DecayScan& s = a.scan[blockIdx.y];
    const int h = blockIdx.x % a.Hv, i = blockIdx.x / a.Hv, tid = threadIdx.x;
    const int j = tid / SPLIT, part = tid % SPLIT;   // column of S, rows part * 32 .. + 31
    long long t0, t1;
    seq_range(a.cu, i, a.T, t0, t1);
    // the decay in two floats: a rounding error in it would compound over the head's whole memory
    const double ad = exp((double)fmaxf(a.log_decay[h], kMinLogDecay));
    const float al = (float)ad, al_lo = (float)(ad - (double)al);
    const size_t sbase = ((size_t)i * a.Hv + h) * DK * DV;
    float st[32];
#pragma unroll
    for (int r = 0; r < 32; ++r) {
        const int row = part * 32 + r;
        st[r] = s.init ? s.init[sbase + (s.init_t ? (size_t)j * DK + row : (size_t)row * DV + j)] : 0.f;
    }
    const T* q = static_cast<const T*>(s.q) + (size_t)(h / s.q_div) * DK;
    const T* k = static_cast<const T*>(s.k) + (size_t)(h / s.k_div) * DK;
    const T* v = static_cast<const T*>(s.v) + (size_t)(h / s.v_div) * DV;
    for (long long done = 0; done < t1 - t0; done += kTB) {
        const int nt = (int)min((long long)kTB, t1 - t0 - done);
        const long long tb = s.reverse ? t1 - done - nt : t0 + done;
        __syncthreads();   // the previous round has read the staging buffers
        for (int e = tid; e < nt * DK; e += NT) {
            const int tt = e / DK, c = e % DK;
            sk[tt][c] = s.su * to_f32(k[(size_t)(tb + tt) * s.k_stride + c]);
            sq[tt][c] = s.so * to_f32(q[(size_t)(tb + tt) * s.q_stride + c]);
        }
        for (int e = tid; e < nt * DV; e += NT) sv[e / DV][e % DV] = to_f32(v[(size_t)(tb + e / DV) * s.v_stride + e % DV]);
        __syncthreads();
        for (int x = 0; x < nt; ++x) {
            const int tt = s.reverse ? nt - 1 - x : x;
            const float vj = sv[tt][j];
            float o = 0.f;
#pragma unroll
            for (int r = 0; r < 32; ++r) {
                if (!s.reverse) st[r] = fmaf(al, st[r], al_lo * st[r]);
                st[r] = fmaf(sk[tt][part * 32 + r], vj, st[r]);
                o = fmaf(sq[tt][part * 32 + r], st[r], o);
                if (s.reverse) st[r] = fmaf(al, st[r], al_lo * st[r]);
            }
#pragma unroll
            for (int m = 1; m < SPLIT; m <<= 1) o += __shfl_xor_sync(0xffffffffu, o, m);
            if (part == 0) {
                const size_t at = (size_t)(tb + tt) * s.out_stride + (size_t)h * DV + j;
                if (s.out_f32) static_cast<float*>(s.out)[at] = o;
                else static_cast<T*>(s.out)[at] = from_f32<T>(o);
            }
        }
    }
    if (s.final) {
#pragma unroll
        for (int r = 0; r < 32; ++r) s.final[sbase + (size_t)(part * 32 + r) * DV + j] = st[r];
    }
}

template <typename T>
__global__ void head_sum_kernel(const float* __restrict__ part, T* __restrict__ out, long long out_stride,
                                long long total, int Hqk, int G, int d) {
    const long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x;   // 4 values each
    if (e >= total) return;
    const int v = d / 4;
    const int c = (int)(e % v);
    const long long th = e / v;   // token * Hqk + head
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < G; ++i) {
        const float4 x = reinterpret_cast<const float4*>(part)[(th * G + i) * v + c];
        acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
    }
    T* o = out + (th / Hqk) * out_stride + (th % Hqk) * d + 4 * c;
    o[0] = from_f32<T>(acc.x); o[1] = from_f32<T>(acc.y); o[2] = from_f32<T>(acc.z); o[3] = from_f32<T>(acc.w);
}

template <typename T>
cudaError_t launch_serial(const DecayArgs& a) {
    const dim3 grid((unsigned)((long long)a.nseq * a.Hv), (unsigned)a.num_scans);
#define GDN_DECAY_CASE(DK_, DV_)                                                                  \
    if (a.dk == DK_ && a.dv == DV_) {                                                             \
        decay_serial_kernel<DK_, DV_, T><<<grid, DV_ * (DK_ / 32), 0, a.stream>>>(a);             \
        return cudaGetLastError();                                                                \
    }
    GDN_DECAY_CASE(32, 32) GDN_DECAY_CASE(32, 64) GDN_DECAY_CASE(32, 128)
    GDN_DECAY_CASE(64, 32) GDN_DECAY_CASE(64, 64) GDN_DECAY_CASE(64, 128)
    GDN_DECAY_CASE(128, 32) GDN_DECAY_CASE(128, 64) GDN_DECAY_CASE(128, 128)
#undef GDN_DECAY_CASE
    return cudaErrorInvalidValue;
}

}  // namespace

size_t decay_scan_workspace_bytes(int dtype, int dk, int dv, int Hv, int nseq, long long tokens, bool packed, int num_scans) {
    return dtype == GDN_BF16 ? decay_scan_tc_workspace_bytes(dk, dv, Hv, nseq, tokens, packed, num_scans) : 0;
}

cudaError_t launch_decay_scan(const DecayArgs& a) {
    return a.dtype == GDN_BF16 ? launch_decay_scan_tc(a) : launch_serial<float>(a);
}

cudaError_t launch_head_sum(const float* part, void* out, long long out_stride, long long tokens, int Hqk, int G, int d,
                            int dtype, cudaStream_t stream) {
    const long long total = tokens * Hqk * (d / 4);
    const unsigned blocks = (unsigned)((total + 255) / 256);
    if (dtype == GDN_BF16)
        head_sum_kernel<<<blocks, 256, 0, stream>>>(part, static_cast<__nv_bfloat16*>(out), out_stride, total, Hqk, G, d);
    else
        head_sum_kernel<<<blocks, 256, 0, stream>>>(part, static_cast<float*>(out), out_stride, total, Hqk, G, d);
    return cudaGetLastError();
}

}  // namespace gdn
