// One token for each of N sequences through linear attention with a decay for each value head, in place on
// the states: S <- a S + k v^T, out = scale S^T q, with a = exp(max(log_decay[h], -100)).  Expanded as
// out = scale (a S_old^T q + (k . q) v), so that the state is read once and written once and the sum over its
// rows does not wait for the update.
//
// One CTA owns CW adjacent columns of one (row n, value head) state: thread (row group, column lane) holds
// its rows' four columns in registers, loads and stores are 128-bit and cover whole CW * 4 byte row pieces,
// and the row sums go through shared memory once.
//
// Bound by HBM: 256 sequences of 32 heads of 128 x 128 (2 x 512 MiB of states) take 178.5 us = 6.05 TB/s, 0.90 of the
// measured copy bandwidth.  Loads and stores stream past the caches (184 us without); limited to two or three CTAs an
// SM it takes 275 or 197 us.
#include "gdn_internal.cuh"

namespace gdn {
namespace {

template <int DK, int DV, int CW, typename T>
__global__ void __launch_bounds__(256)
decay_step_kernel(const __grid_constant__ DecayStepArgs a) {
    constexpr int LX = CW / 4, RG = 256 / LX, RPT = DK / RG, SL = DV / CW;
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
    const float al = expf(fmaxf(a.log_decay[h], kMinLogDecay));
    float vj[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) vj[e] = to_f32(v[4 * lx + e]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const float qr = to_f32(q[rg * RPT + r]), kr = to_f32(k[rg * RPT + r]);
        acc.x = fmaf(st[r].x, qr, acc.x); acc.y = fmaf(st[r].y, qr, acc.y);
        acc.z = fmaf(st[r].z, qr, acc.z); acc.w = fmaf(st[r].w, qr, acc.w);
        __stcs(reinterpret_cast<float4*>(S + (size_t)(rg * RPT + r) * DV),
               make_float4(fmaf(kr, vj[0], al * st[r].x), fmaf(kr, vj[1], al * st[r].y), fmaf(kr, vj[2], al * st[r].z),
                           fmaf(kr, vj[3], al * st[r].w)));
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
    if (tid < CW) {
        float s = 0.f;
#pragma unroll 8
        for (int x = 0; x < RG; ++x) s += red[x][tid];
        out[tid] = from_f32<T>(a.scale * fmaf(al, s, skq * to_f32(v[tid])));
    }
}

// A CTA takes a whole state (row pieces of up to 512 bytes, all of a thread's loads in flight) where there are at
// least four states for each of the 152 SMs; below that 32-column pieces, so that one sequence's 32 heads of 128
// columns still reach 128 SMs.  Measured on 256 x 32 states of 128 x 128: 178 us whole (6.05 TB/s, 0.90 of the copy
// rate), 184 us in pieces; capped at two CTAs a SM 275 us.
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
