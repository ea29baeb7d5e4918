// The decayed scan (gdn_internal.cuh, DecayScan) for fp32 inputs, on the CUDA cores.  The tensor cores would need
// every operand in three bf16 parts and six products of them, and mma.sync in tf32 three products, which at about six
// SM cycles for each of 1024 FMAs is 18 cycles where packed fp32 FMAs (128 a cycle) take 8 at their rate.  What this
// kernel reaches is a fifth of that rate (below): split products might be ahead of it, and are not built.
//
// The chunked form with C = 32 tokens (the quadratic part of a token's work grows with C and is below the two
// dk x dv products of the state at these head dims).  With w_d = a^d, n valid tokens, S the state at the first
// visited end of the chunk (see gdn_decay_tc.cu for the reverse scan's formulas):
//     P_rj = so su w_{r-j} (q_r . k_j),   out = so diag(w_{r+1}) Q S + P V,   S <- w_n S + K^T (su diag(w_{n-1-j}) V)
// One CTA of 256 threads walks one unit of one value head for up to 64 value columns.  The state stays in
// registers (rows x 4 columns a thread) and is copied to shared memory once a chunk for Q S; products are register
// tiles of packed FMAs over float4 reads; the next chunk's rows are loaded while this one is computed.
//
// Bound by shared memory: each float4 that a product reads feeds 8 or 16 FMAs, and the L1 pipe is 81 % busy in the
// main pass, the FMA pipe 21 %.  Measured, packed backward of 1344 tokens (the longest sequence 700), 8 heads of 64:
// 4.6 ms as matrix products and a token loop in plain tensor operations, 287 us token by token in one CTA a head,
// 121 us in chunks, 98 us in segments of 128 tokens, 66 us with those spread over two CTAs an SM, 63.5 us with
// P V over the columns that a row sees (16 + 38.5 us in the state and the main pass).  2 x 2048 tokens of 32 heads of 128:
// 541 us.
#include "decay_unit.cuh"

namespace gdn {
namespace {

constexpr int kC = 32, kNT = 256;
constexpr long long kFewCtas = 76;   // half of the 152 SMs

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)), "l"(*reinterpret_cast<uint64_t*>(&c)));
    return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 all2(float x) { return make_float2(x, x); }

template <int DK, int DV>   // DV: the CTA's value columns
struct Tile {
    static constexpr int LK = DK + 4, LV = DV + 4, LP = kC + 4;   // row pitches: float4 rows on different banks
    static constexpr int CG = DV / 4, RG = kNT / CG;              // 4-column groups, row groups
    static constexpr int SR = DK / RG, OR = kC / RG < 1 ? 1 : kC / RG;   // rows a thread of the state, of the outputs
    static constexpr int OT = kC < RG ? kC : RG;                  // row groups with outputs
    static constexpr int Q_ = 0, K_ = Q_ + kC * LK, V_ = K_ + kC * LK, W_ = V_ + kC * LV, P_ = W_ + kC * LV,
                         S_ = P_ + kC * LP, T_ = S_ + DK * LV, FLOATS = T_ + 40;
    static constexpr size_t BYTES = (size_t)FLOATS * 4;
};

// N rows' floats of one token (row pitch of the matrix irrelevant): x[0 .. N - 1].
template <int N>
__device__ __forceinline__ void load_vec(const float* p, float (&x)[N]) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + i);
            x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
        }
    } else if constexpr (N == 2) {
        const float2 v = *reinterpret_cast<const float2*>(p);
        x[0] = v.x; x[1] = v.y;
    } else {
        x[0] = p[0];
    }
}

template <int DK, int DV, bool STATE>
__global__ void __launch_bounds__(kNT, DK == 128 ? 1 : 2)
decay_f32_kernel(const __grid_constant__ SegArgs ta) {
    using L = Tile<DK, DV>;
    extern __shared__ __align__(16) float sm[];
    float *const Q = sm + L::Q_, *const K = sm + L::K_, *const V = sm + L::V_, *const W = sm + L::W_, *const P = sm + L::P_,
                *const Ss = sm + L::S_, *const pw = sm + L::T_;
    const DecayArgs& a = ta.a;
    const DecayScan& s = a.scan[blockIdx.y];
    const int zs = a.dv / DV, z = blockIdx.x % zs, h = blockIdx.x / zs % a.Hv, slot = blockIdx.x / zs / a.Hv;
    const bool rev = s.reverse;
    Unit unit;
    if (!unit_of(ta, slot, rev, unit)) return;
    if (STATE && unit.last) return;
    const int tid = threadIdx.x, cg = tid % L::CG, rg = tid / L::CG;
    const int len = (int)(unit.t1 - unit.t0), nch = (len + kC - 1) / kC, tail = len - (nch - 1) * kC;
    const float g = decay_exponent(a.log_decay[h]);
    if (tid <= kC) pw[tid] = tid ? expf(g * (float)tid) : 1.f;
    if (tid < 2) decay_power(g, (float)(tid ? tail : kC), pw[34 + 2 * tid], pw[35 + 2 * tid]);   // of a full, of the last chunk
    const size_t base = ((size_t)unit.seq * a.Hv + h) * DK * a.dv;
    const float* const init = STATE ? nullptr : ta.seg ? unit_state(ta, blockIdx.y, slot, h) : s.init ? s.init + base : nullptr;
    float* const final = STATE ? unit_state(ta, blockIdx.y, slot, h) : s.final && unit.last ? s.final + base : nullptr;
    float2 S[L::SR][2];
    const int row0 = rg * L::SR, col0 = DV * z + 4 * cg;
#pragma unroll
    for (int r = 0; r < L::SR; ++r) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (init && s.init_t && !ta.seg)
            x = make_float4(init[(size_t)col0 * DK + row0 + r], init[(size_t)(col0 + 1) * DK + row0 + r],
                            init[(size_t)(col0 + 2) * DK + row0 + r], init[(size_t)(col0 + 3) * DK + row0 + r]);
        else if (init)
            x = *reinterpret_cast<const float4*>(init + (size_t)(row0 + r) * a.dv + col0);
        S[r][0] = make_float2(x.x, x.y);
        S[r][1] = make_float2(x.z, x.w);
    }
    const float* const gq = static_cast<const float*>(s.q) + (size_t)(h / s.q_div) * DK;
    const float* const gk = static_cast<const float*>(s.k) + (size_t)(h / s.k_div) * DK;
    const float* const gv = static_cast<const float*>(s.v) + (size_t)(h / s.v_div) * a.dv + DV * z;
    // the chunk's rows in registers: q and k rows of DK / 4 float4, v rows of DV / 4; rows past the end are zeros
    constexpr int NK = kC * DK / 4 / kNT, NV = kC * DV / 4 / kNT;
    float4 fq[NK], fk[NK], fv[NV];
    auto chunk_at = [&](int it) { return unit.t0 + (long long)(rev ? nch - 1 - it : it) * kC; };
    auto valid_of = [&](int it) { return (rev ? nch - 1 - it : it) == nch - 1 ? tail : kC; };
    auto load = [&](int it) {
        const long long t = chunk_at(it);
        const int n = valid_of(it);
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int e = tid + i * kNT, r = e / (DK / 4), c = e % (DK / 4) * 4;
            fk[i] = r < n ? *reinterpret_cast<const float4*>(gk + (size_t)(t + r) * s.k_stride + c) : zero;
            if (!STATE) fq[i] = r < n ? *reinterpret_cast<const float4*>(gq + (size_t)(t + r) * s.q_stride + c) : zero;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = tid + i * kNT, r = e / (DV / 4), c = e % (DV / 4) * 4;
            fv[i] = r < n ? *reinterpret_cast<const float4*>(gv + (size_t)(t + r) * s.v_stride + c) : zero;
        }
    };
    if (nch > 0) load(0);
    __syncthreads();   // the tables
    for (int it = 0; it < nch; ++it) {
        const int n = valid_of(it);
        const long long t = chunk_at(it);
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int e = tid + i * kNT, r = e / (DK / 4), c = e % (DK / 4) * 4;
            *reinterpret_cast<float4*>(K + r * L::LK + c) = fk[i];
            if (!STATE) *reinterpret_cast<float4*>(Q + r * L::LK + c) = fq[i];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = tid + i * kNT, r = e / (DV / 4), c = e % (DV / 4) * 4;
            const float w = r < n ? s.su * pw[rev ? r + 1 : n - 1 - r] : 0.f;
            if (!STATE) *reinterpret_cast<float4*>(V + r * L::LV + c) = fv[i];
            *reinterpret_cast<float4*>(W + r * L::LV + c) = make_float4(w * fv[i].x, w * fv[i].y, w * fv[i].z, w * fv[i].w);
        }
        if (!STATE) {
#pragma unroll
            for (int r = 0; r < L::SR; ++r)
                *reinterpret_cast<float4*>(Ss + (row0 + r) * L::LV + 4 * cg) =
                    make_float4(S[r][0].x, S[r][0].y, S[r][1].x, S[r][1].y);
        }
        __syncthreads();
        if (it + 1 < nch) load(it + 1);
        float2 O[L::OR][2];
        if (!STATE) {
            {   // P, two rows by two columns a thread
                const int r0 = tid / 16 * 2, j0 = tid % 16;   // columns j0 and j0 + 16: k rows on different banks
                float2 acc[2][2] = {{all2(0.f), all2(0.f)}, {all2(0.f), all2(0.f)}};
                if (rev ? j0 + 16 >= r0 : j0 <= r0 + 1) {
#pragma unroll 4
                    for (int c = 0; c < DK; c += 4) {
                        float4 x[2], y[2];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            x[u] = *reinterpret_cast<const float4*>(Q + (r0 + u) * L::LK + c);
                            y[u] = *reinterpret_cast<const float4*>(K + (j0 + 16 * u) * L::LK + c);
                        }
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int v = 0; v < 2; ++v) {
                                acc[u][v] = fma2(make_float2(x[u].x, x[u].y), make_float2(y[v].x, y[v].y), acc[u][v]);
                                acc[u][v] = fma2(make_float2(x[u].z, x[u].w), make_float2(y[v].z, y[v].w), acc[u][v]);
                            }
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const int d = rev ? j0 + 16 * v - r0 - u : r0 + u - j0 - 16 * v;
                        P[(r0 + u) * L::LP + j0 + 16 * v] =
                            d >= 0 && j0 + 16 * v < n ? s.so * s.su * pw[max(d, 0)] * (acc[u][v].x + acc[u][v].y) : 0.f;
                    }
                }
            }
            if (rg < L::OT) {   // Q S, then its row factors
#pragma unroll
                for (int r = 0; r < L::OR; ++r) O[r][0] = O[r][1] = all2(0.f);
#pragma unroll 2
                for (int c = 0; c < DK; c += 4) {
                    float x[L::OR][4];
#pragma unroll
                    for (int r = 0; r < L::OR; ++r) load_vec(Q + (rg * L::OR + r) * L::LK + c, x[r]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float4 y = *reinterpret_cast<const float4*>(Ss + (c + u) * L::LV + 4 * cg);
#pragma unroll
                        for (int r = 0; r < L::OR; ++r) {
                            O[r][0] = fma2(all2(x[r][u]), make_float2(y.x, y.y), O[r][0]);
                            O[r][1] = fma2(all2(x[r][u]), make_float2(y.z, y.w), O[r][1]);
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < L::OR; ++r) {
                    const int row = rg * L::OR + r;
                    const float w = s.so * pw[rev ? max(n - 1 - row, 0) : row + 1];
                    O[r][0].x *= w; O[r][0].y *= w; O[r][1].x *= w; O[r][1].y *= w;
                }
            }
            __syncthreads();
            if (rg < L::OT) {
                // P V over the columns that the rows see: a value of V that is not finite would make NaN of a masked
                // zero.  A warp's rows lie in one block of four columns, whose masked values act as zeros.
                static_assert(L::OR * (32 / L::CG) <= 4, "rows of a warp");
                const int diag = rg * L::OR / 4 * 4;
                const auto add = [&](int j, bool masked) {
                    float x[L::OR][4];
#pragma unroll
                    for (int r = 0; r < L::OR; ++r) load_vec(P + (rg * L::OR + r) * L::LP + j, x[r]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float4 y = *reinterpret_cast<const float4*>(V + (j + u) * L::LV + 4 * cg);
#pragma unroll
                        for (int r = 0; r < L::OR; ++r) {
                            const int row = rg * L::OR + r;
                            if (masked && (rev ? j + u < row : j + u > row)) continue;
                            O[r][0] = fma2(all2(x[r][u]), make_float2(y.x, y.y), O[r][0]);
                            O[r][1] = fma2(all2(x[r][u]), make_float2(y.z, y.w), O[r][1]);
                        }
                    }
                };
#pragma unroll 2
                for (int j = rev ? diag + 4 : 0; j < (rev ? kC : diag); j += 4) add(j, false);
                add(diag, true);
#pragma unroll
                for (int r = 0; r < L::OR; ++r) {
                    const int row = rg * L::OR + r;
                    if (row < n)
                        *reinterpret_cast<float4*>(static_cast<float*>(s.out) + (size_t)(t + row) * s.out_stride +
                                                   (size_t)h * a.dv + col0) =
                            make_float4(O[r][0].x, O[r][0].y, O[r][1].x, O[r][1].y);
                }
            }
        }
        if (it + 1 < nch || final) {   // the state
            const float2 hi = all2(pw[n == kC ? 34 : 36]), lo = all2(pw[n == kC ? 35 : 37]);
            float2 acc[L::SR][2];
#pragma unroll
            for (int r = 0; r < L::SR; ++r) acc[r][0] = acc[r][1] = all2(0.f);
#pragma unroll 4
            for (int j = 0; j < kC; ++j) {
                float x[L::SR];
                load_vec(K + j * L::LK + row0, x);
                const float4 y = *reinterpret_cast<const float4*>(W + j * L::LV + 4 * cg);
#pragma unroll
                for (int r = 0; r < L::SR; ++r) {
                    acc[r][0] = fma2(all2(x[r]), make_float2(y.x, y.y), acc[r][0]);
                    acc[r][1] = fma2(all2(x[r]), make_float2(y.z, y.w), acc[r][1]);
                }
            }
#pragma unroll
            for (int r = 0; r < L::SR; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) S[r][e] = fma2(hi, S[r][e], fma2(lo, S[r][e], acc[r][e]));
        }
        __syncthreads();
    }
    if (final) {
#pragma unroll
        for (int r = 0; r < L::SR; ++r)
            *reinterpret_cast<float4*>(final + (size_t)(row0 + r) * a.dv + col0) =
                make_float4(S[r][0].x, S[r][0].y, S[r][1].x, S[r][1].y);
    }
}

template <int DK, int DV>
cudaError_t launch_typed(const SegArgs& s, bool state_only) {
    const auto kernel = state_only ? decay_f32_kernel<DK, DV, true> : decay_f32_kernel<DK, DV, false>;
    constexpr size_t smem = Tile<DK, DV>::BYTES;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)((long long)s.slots * s.a.Hv * (s.a.dv / DV)), (unsigned)s.a.num_scans);
    kernel<<<grid, kNT, smem, s.a.stream>>>(s);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_f32(const SegArgs& s, bool state_only) {
    // 32 columns a CTA where 64 would leave half of the SMs without one: the scores are then formed twice, but by
    // SMs that would idle.  (Taken up to twice as many CTAs as SMs it measured 102.2 us against 101.3 us on the packed
    // backward of 1344 tokens, 8 heads of 64, in coarser segments: no gain there.)
    const int dk = s.a.dk;
    const long long ctas = (long long)s.slots * s.a.Hv * s.a.num_scans * ((s.a.dv + 63) / 64);
    const int dv = s.a.dv < kDecayColumns || ctas < kFewCtas ? 32 : kDecayColumns;
#define GDN_DECAY_CASE(DK_, DV_) \
    if (dk == DK_ && dv == DV_) return launch_typed<DK_, DV_>(s, state_only);
    GDN_DECAY_CASE(32, 32) GDN_DECAY_CASE(64, 32) GDN_DECAY_CASE(128, 32)
    GDN_DECAY_CASE(32, 64) GDN_DECAY_CASE(64, 64) GDN_DECAY_CASE(128, 64)
#undef GDN_DECAY_CASE
    return cudaErrorInvalidValue;
}

}  // namespace gdn
