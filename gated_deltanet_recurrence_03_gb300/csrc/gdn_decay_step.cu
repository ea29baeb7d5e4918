// One token for each of N sequences through linear attention with a decay for each value head, in place on
// the states: S <- a S + k v^T, out = scale S^T q, with a = exp(max(log_decay[h], -100)), NaN for NaN.  Expanded as
// out = scale (a S_old^T q + (k . q) v), so that the state is read once and written once and the sum over its
// rows does not wait for the update.
//
// One CTA owns CW adjacent columns of one (row n, value head) state: thread (row group, column lane) holds
// its rows' four columns in registers, loads and stores are 128-bit and cover whole CW * 4 byte row pieces,
// and the row sums go through shared memory once.
//
// Bound by HBM: 256 sequences of 32 heads of 128 x 128 (2 x 512 MiB of states) take 153.6 us = 7.0 TB/s, 1.05 of the
// measured copy bandwidth.  What counts is that a CTA's loads are all in flight before its first store: with each row
// stored as soon as it is loaded the compiler keeps few loads ahead, and it takes 176 us.  Streaming accesses make no
// difference in this form.
#include "decay_unit.cuh"

namespace gdn {
namespace {

// Rows of a state that a thread holds.
__host__ __device__ constexpr int rows_of(int DK, int CW) { return DK / (256 / (CW / 4)); }

// Two CTAs an SM where a thread holds 16 rows, so that all of them have registers; without the bound the compiler takes
// fewer and loads in turns (160 against 153.6 us, 256 x 32 states of 128 x 128).  With fewer rows a thread the compiler's
// own choice (0), of fewer registers and more CTAs, is better than a bound of 1 (58 against 67 us, 1024 x 32 states of
// 32 x 32).
template <int DK, int DV, int CW, typename T>
__global__ void __launch_bounds__(256, rows_of(DK, CW) >= 16 ? 2 : 0)
decay_step_kernel(const __grid_constant__ DecayStepArgs a) {
    constexpr int LX = CW / 4, RG = 256 / LX, RPT = rows_of(DK, CW), SL = DV / CW;
    static_assert(RPT >= 1 && DK % RG == 0 && DV % CW == 0, "tile");
    __shared__ __align__(16) float red[RG][CW + 4];
    __shared__ float skq;
    const int sl = blockIdx.x % SL;
    const int nh = blockIdx.x / SL, n = nh / a.Hv, h = nh % a.Hv, hk = h / (a.Hv / a.Hqk);
    const int tid = threadIdx.x, lx = tid % LX, rg = tid / LX;
    const int slot = a.slots ? a.slots[n] : n;
    T* out = static_cast<T*>(a.out) + (size_t)nh * DV + sl * CW;
    if (slot < 0 || slot >= a.num_slots) {   // a row without a request
        for (int j = tid; j < CW; j += 256) out[j] = from_f32<T>(0.f);
        return;
    }
    float* S = a.S + ((size_t)slot * a.Hv + h) * DK * DV + sl * CW + 4 * lx;
    float4 st[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) st[r] = __ldcs(reinterpret_cast<const float4*>(S + (size_t)(rg * RPT + r) * DV));
    const T* q = static_cast<const T*>(a.q) + (size_t)n * a.q_stride + (size_t)hk * DK;
    const T* k = static_cast<const T*>(a.k) + (size_t)n * a.k_stride + (size_t)hk * DK;
    const T* v = static_cast<const T*>(a.v) + (size_t)n * a.v_stride + (size_t)h * DV + sl * CW;
    const float al = expf(decay_exponent(a.log_decay[h]));
    float vj[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) vj[e] = to_f32(v[4 * lx + e]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const float qr = to_f32(q[rg * RPT + r]);
        acc.x = fmaf(st[r].x, qr, acc.x); acc.y = fmaf(st[r].y, qr, acc.y);
        acc.z = fmaf(st[r].z, qr, acc.z); acc.w = fmaf(st[r].w, qr, acc.w);
    }
    reinterpret_cast<float4*>(&red[rg][0])[lx] = acc;
    if (tid < 32) {
        float kq = 0.f;
        for (int i = tid; i < DK; i += 32) kq = fmaf(to_f32(k[i]), to_f32(q[i]), kq);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, o);
        if (tid == 0) skq = kq;
    }
    __syncthreads();
    // the stores after the barrier: none can come between the loads
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const float kr = to_f32(k[rg * RPT + r]);
        __stcs(reinterpret_cast<float4*>(S + (size_t)(rg * RPT + r) * DV),
               make_float4(fmaf(kr, vj[0], al * st[r].x), fmaf(kr, vj[1], al * st[r].y), fmaf(kr, vj[2], al * st[r].z),
                           fmaf(kr, vj[3], al * st[r].w)));
    }
    if (tid < CW) {
        float s = 0.f;
#pragma unroll 8
        for (int x = 0; x < RG; ++x) s += red[x][tid];
        out[tid] = from_f32<T>(a.scale * fmaf(al, s, skq * to_f32(v[tid])));
    }
}

// A CTA takes a whole state (row pieces of up to 512 bytes) where there are at least four states for each of the 152
// SMs; below that 32-column pieces, so that one sequence's 32 heads of 128 columns still reach 128 SMs.  Measured on
// 256 x 32 states of 128 x 128, with rows stored as they were loaded: 178 us whole, 184 us in pieces.
constexpr long long kWideRows = 4 * 152;

template <int DK, int DV, typename T>
cudaError_t launch_typed(const DecayStepArgs& a) {
    if ((long long)a.N * a.Hv >= kWideRows)
        decay_step_kernel<DK, DV, DV, T><<<(unsigned)((long long)a.N * a.Hv), 256, 0, a.stream>>>(a);
    else
        decay_step_kernel<DK, DV, 32, T><<<(unsigned)((long long)a.N * a.Hv * (DV / 32)), 256, 0, a.stream>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_dims(const DecayStepArgs& a) {
#define GDN_STEP_CASE(DK_, DV_) \
    if (a.dk == DK_ && a.dv == DV_) return launch_typed<DK_, DV_, T>(a);
    GDN_STEP_CASE(32, 32) GDN_STEP_CASE(32, 64) GDN_STEP_CASE(32, 128)
    GDN_STEP_CASE(64, 32) GDN_STEP_CASE(64, 64) GDN_STEP_CASE(64, 128)
    GDN_STEP_CASE(128, 32) GDN_STEP_CASE(128, 64) GDN_STEP_CASE(128, 128)
#undef GDN_STEP_CASE
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_decay_step(const DecayStepArgs& a) {
    return a.dtype == GDN_BF16 ? launch_dims<__nv_bfloat16>(a) : launch_dims<float>(a);
}

}  // namespace gdn
