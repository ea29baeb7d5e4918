// Linear attention with a decay for each value head: the scan behind gdn_decay_attn_fwd and, three times, behind
// gdn_decay_attn_bwd (gdn_internal.cuh, DecayScan): how long sequences are cut, and the passes over them.
#include <algorithm>

#include "decay_unit.cuh"

namespace gdn {
namespace {

// Between the two passes over segments: the state at each one's first visited end, S <- a^length S + the segment's own part, walked in
// the scan's order; one float4 of one (sequence, head)'s state a thread, the parts of eight segments loaded at once.
constexpr int kJoinThreads = 256, kJoinAhead = 8;
__global__ void __launch_bounds__(kJoinThreads) decay_join_kernel(const __grid_constant__ SegArgs ta) {
    const DecayArgs& a = ta.a;
    const DecayScan& s = a.scan[blockIdx.y];
    const int dk = a.dk, dv = a.dv, blocks = dk * dv / 4 / kJoinThreads;   // of one state (at least 32 x 32)
    const int part = blockIdx.x % blocks, h = (blockIdx.x / blocks) % a.Hv, i = blockIdx.x / blocks / a.Hv;
    long long s0, s1;
    seq_range(a.cu, i, a.T, s0, s1);
    const int n = (int)max(1LL, (s1 - s0 + ta.seg - 1) / ta.seg), slot0 = (int)(s0 / ta.seg) + i;
    __shared__ float w[4];   // the decay over a whole and over the last segment, in two floats each
    if (threadIdx.x < 2) {
        const long long len = threadIdx.x ? s1 - s0 - (long long)(n - 1) * ta.seg : ta.seg;
        decay_power(decay_exponent(a.log_decay[h]), (float)len, w[2 * threadIdx.x], w[2 * threadIdx.x + 1]);
    }
    __syncthreads();
    const int e = (part * kJoinThreads + threadIdx.x) * 4, row = e / dv, col = e % dv;
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (s.init) {
        const float* x = s.init + ((size_t)i * a.Hv + h) * dk * dv;
        S = s.init_t ? make_float4(x[col * dk + row], x[(col + 1) * dk + row], x[(col + 2) * dk + row], x[(col + 3) * dk + row])
                     : *reinterpret_cast<const float4*>(x + e);
    }
    for (int j0 = 0; j0 < n; j0 += kJoinAhead) {
        float4 add[kJoinAhead];
#pragma unroll
        for (int x = 0; x < kJoinAhead; ++x) {
            const int j = j0 + x, at = slot0 + (s.reverse ? n - 1 - j : j);
            if (j + 1 < n) add[x] = *reinterpret_cast<const float4*>(unit_state(ta, blockIdx.y, at, h) + e);
        }
#pragma unroll
        for (int x = 0; x < kJoinAhead; ++x) {
            const int j = j0 + x, at = s.reverse ? n - 1 - j : j;
            if (j >= n) break;
            *reinterpret_cast<float4*>(unit_state(ta, blockIdx.y, slot0 + at, h) + e) = S;
            const float hi = w[at == n - 1 ? 2 : 0], lo = w[at == n - 1 ? 3 : 1];
            if (j + 1 < n)
                S = make_float4(fmaf(hi, S.x, fmaf(lo, S.x, add[x].x)), fmaf(hi, S.y, fmaf(lo, S.y, add[x].y)),
                                fmaf(hi, S.z, fmaf(lo, S.z, add[x].z)), fmaf(hi, S.w, fmaf(lo, S.w, add[x].w)));
        }
    }
}

// A sum over shared heads reads G fp32 parts and writes one row, and is bound by HBM: a thread takes eight values of
// one token and query/key head (two 16-byte loads of each part, read once and so streamed; one 16- or two 16-byte
// stores), and both gradients' sums share a launch.
constexpr int kSumThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kSumThreads) head_sum_kernel(const __grid_constant__ HeadSums a) {
    const int which = blockIdx.x & 1, hk = (blockIdx.x >> 1) % a.Hqk, lanes = a.d / 8;
    const long long t = (long long)((blockIdx.x >> 1) / a.Hqk) * (kSumThreads / lanes) + threadIdx.x / lanes;
    if (t >= a.tokens) return;
    const int c = threadIdx.x % lanes * 8;
    const float* part = a.part[which] + ((size_t)t * a.Hqk + hk) * a.G * a.d + c;
    float x[8] = {};
#pragma unroll 2
    for (int i = 0; i < a.G; ++i) {
        const float4 lo = __ldcs(reinterpret_cast<const float4*>(part + (size_t)i * a.d));
        const float4 hi = __ldcs(reinterpret_cast<const float4*>(part + (size_t)i * a.d) + 1);
        x[0] += lo.x; x[1] += lo.y; x[2] += lo.z; x[3] += lo.w;
        x[4] += hi.x; x[5] += hi.y; x[6] += hi.z; x[7] += hi.w;
    }
    __align__(16) T y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = from_f32<T>(x[e]);
    T* out = static_cast<T*>(a.out[which]) + (size_t)t * a.out_stride[which] + (size_t)hk * a.d + c;
#pragma unroll
    for (int e = 0; e < (int)sizeof(T) / 2; ++e) reinterpret_cast<uint4*>(out)[e] = reinterpret_cast<const uint4*>(y)[e];
}

// Tokens of a segment, 0 for whole sequences.  One CTA walks one slot, so a call of few sequences and heads leaves most
// of the card idle and is bound by its longest sequence; in n segments a sequence takes 1 / n of its chunks' time
// plus that of the pass that forms the segments' parts of the state (a third of the main pass).  So sequences are cut
// where at least two segments of each find one of the card's `places` of their own; the lengths of packed sequences
// are not known here, and their total is cut instead (a sequence shorter than that is one segment).  Segments
// shorter than four chunks of their kernel would be mostly start-up.  Measured: 46,546 packed tokens (one sequence
// of 40,961) of 6 heads of 128, bf16: 709 us whole, 182 us in 3712-token segments (each sequence's last segment is a part
// of one, so these are 17 units x 12 CTAs, a second wave on 152 SMs that is a third full); 1212 tokens of 13 heads: 55 us
// with 1024 tokens as the least, 46 us with 512.
int segment_tokens(long long tokens, int nseq, bool packed, int ctas, int places, int min_segment) {
    long long seg;
    if (packed) {
        if (ctas * 2 > places) return 0;
        seg = (tokens * ctas + places - 1) / places;
    } else {
        const long long n = places / ((long long)nseq * ctas);
        if (n < 2) return 0;
        seg = (tokens / nseq + n - 1) / n;
    }
    seg = std::max<long long>((seg + 127) / 128 * 128, min_segment);
    return seg < (packed ? tokens : tokens / nseq) ? (int)seg : 0;
}
long long segment_slots(long long tokens, int nseq, int seg) { return seg ? tokens / seg + nseq : nseq; }


// Segment tokens and slots of a call, and the bytes of its segments' states.
SegArgs plan_of(int dtype, int dv, int Hv, int nseq, long long tokens, bool packed, int num_scans) {
    SegArgs p{};
    const int ctas = (dv > kDecayColumns ? dv / kDecayColumns : 1) * Hv * num_scans;   // of one slot
    // the tensor-core kernel fills an SM and takes 128 tokens a chunk, the fp32 one shares an SM with another
    p.seg = dtype == GDN_BF16 ? segment_tokens(tokens, nseq, packed, ctas, 152, 512)
                              : segment_tokens(tokens, nseq, packed, ctas, 304, 128);
    p.slots = (int)segment_slots(tokens, nseq, p.seg);
    return p;
}

}  // namespace

size_t decay_scan_workspace_bytes(int dtype, int dk, int dv, int Hv, int nseq, long long tokens, bool packed, int num_scans) {
    const SegArgs p = plan_of(dtype, dv, Hv, nseq, tokens, packed, num_scans);
    return p.seg ? (size_t)p.slots * Hv * num_scans * dk * dv * sizeof(float) : 0;
}

cudaError_t launch_decay_scan(const DecayArgs& a) {
    SegArgs p = plan_of(a.dtype, a.dv, a.Hv, a.nseq, a.tokens, a.cu != nullptr, a.num_scans);
    p.a = a;
    p.states = static_cast<float*>(a.workspace);
    const auto pass = a.dtype == GDN_BF16 ? launch_decay_tc : launch_decay_f32;
    if (p.seg) {
        cudaError_t e = pass(p, true);
        if (e != cudaSuccess) return e;
        const dim3 grid((unsigned)((long long)a.nseq * a.Hv * (a.dk * a.dv / 4 / kJoinThreads)), (unsigned)a.num_scans);
        decay_join_kernel<<<grid, kJoinThreads, 0, a.stream>>>(p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return pass(p, false);
}

cudaError_t launch_head_sums(const HeadSums& a, int dtype, cudaStream_t stream) {
    const int per = kSumThreads / (a.d / 8);
    const unsigned blocks = 2u * (unsigned)((a.tokens + per - 1) / per * a.Hqk);
    if (dtype == GDN_BF16) head_sum_kernel<__nv_bfloat16><<<blocks, kSumThreads, 0, stream>>>(a);
    else head_sum_kernel<float><<<blocks, kSumThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
