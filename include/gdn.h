/*
 * gdn.h -- C ABI of the GB300 (sm_103a) Gated DeltaNet recurrence library (libgdn.so).
 *
 * The operation (per sequence, per value head h, state S: dk x dv, fp32):
 *
 *     S_t = a_t S_{t-1} + beta_t k_t (v_t - a_t S_{t-1}^T k_t)^T,   a_t = exp(g_t)
 *     o_t = scale * S_t^T q_t
 *
 * as stated in "Transformer by Hand, ch. 7 -- Gated DeltaNet: the token-by-token
 * recurrence", section "The formula", and computed step by step (decay, look up
 * with k, write the difference times beta, read with q) by the delta_rule
 * listing of section "qwen/deltanet.py" of the same chapter.  Value head h uses
 * query/key head floor(h / (Hv / Hqk)), the repeat_interleave of the
 * GatedDeltaNet shell in the same listing.  The chunk-parallel prefill computes
 * the same result up to rounding ("mathematically equivalent to the token loop",
 * learn-llm page "linear attention", remark on flash-linear-attention).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every tensor pointer is CALLER-OWNED DEVICE memory, contiguous, row-major.
 *   q, k, v, out and the states are 16-byte aligned; g and beta are aligned to
 *   their element size.  The library never allocates, frees or retains device
 *   memory; scratch space is passed in as opts->workspace.
 * - Calls are asynchronous on opts->stream: a return of GDN_OK means the work was
 *   validated and enqueued.  Device-side failures (a bounded wait that ran out)
 *   are read with gdn_check_device_status().
 * - Argument errors are detected on the host before anything is enqueued; nothing
 *   is written in that case.
 * - The values of g (finite, <= 0) and beta (in [0, 1]) are the caller's
 *   contract; they are not checked.  Kernels never read or write outside the
 *   buffers described by the sizes, whatever the values (cu_seqlens entries are
 *   clamped to [0, T]).
 * - Thread safety: calls on different streams may run concurrently; a workspace
 *   must not be shared by calls that overlap on the device.
 * - The layout of gdn_opts_t belongs to GDN_VERSION_MAJOR.GDN_VERSION_MINOR: the library reads (and
 *   gdn_opts_init writes) the whole struct, so a program calls only a library of the minor version
 *   that it was compiled for, which gdn_version() / 100 == GDN_VERSION / 100 tells.
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* 0.4: gdn_opts_t has conv_bias and grad_conv_bias. */
#define GDN_VERSION_MAJOR 0
#define GDN_VERSION_MINOR 4
#define GDN_VERSION_PATCH 0
#define GDN_VERSION (GDN_VERSION_MAJOR * 10000 + GDN_VERSION_MINOR * 100 + GDN_VERSION_PATCH)

typedef enum gdn_status {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARG = 1, /* null pointer, bad size, misalignment, Hv % Hqk != 0 ... */
    GDN_ERR_UNSUPPORTED = 2, /* head dims or chunk outside the supported set, wrong GPU */
    GDN_ERR_CUDA = 3,        /* a CUDA runtime call or launch failed (see gdn_last_error) */
    GDN_ERR_TIMEOUT = 4,     /* a bounded device-side wait ran out (gdn_check_device_status) */
    GDN_ERR_WORKSPACE = 5    /* workspace missing or smaller than the size query asked for */
} gdn_status_t;

typedef enum gdn_dtype {
    GDN_F32 = 0,  /* q, k, v, g, beta and out are float */
    GDN_BF16 = 1  /* q, k, v, g, beta and out are bfloat16; the state is always float */
} gdn_dtype_t;

/* opts->flags */
#define GDN_NORMALIZE_QK 0x1u /* divide q and k by sqrt(sum x^2 + 1e-6) inside the kernel
                                 (the l2norm step of delta_rule); off: inputs are used as given */
#define GDN_RAW_GATES 0x2u    /* the g and beta arguments hold the raw per-token projections a and b of
                                 the GatedDeltaNet shell ("qwen/deltanet.py", forward): the kernels form
                                 beta = sigmoid(b) and g = -exp(A_log[h]) * softplus(a + dt_bias[h]) in
                                 fp32; opts->A_log and opts->dt_bias ([Hv] float) are then required */
#define GDN_OUTPUT_GATE 0x4u  /* out = RMSNorm(o) * norm_weight * silu(z) per (token, value head), the
                                 gated normalisation of the shell (GatedRMSNorm(out, z)): o is divided by
                                 sqrt(mean over dv of o^2 + norm_eps); opts->z ([..., Hv, dv] like out,
                                 dtype) and opts->norm_weight ([dv] float) are then required */

typedef struct gdn_opts {
    int dtype;                  /* gdn_dtype_t of q, k, v, g, beta, out.  Default GDN_BF16. */
    int chunk;                  /* prefill chunk length: 16, 32 or 64 (0 -> 64; others rejected).
                                   Every chunk length gives the token loop's result up to rounding
                                   (the chunked form is the loop regrouped), and both chunked kernel
                                   families are built on 64-token tensor-core tiles: they serve all
                                   three values with 64-token chunks, so results do not depend on it. */
    float scale;                /* multiplies every output o_t.  Default 1.0f. */
    unsigned flags;             /* GDN_NORMALIZE_QK | GDN_RAW_GATES | GDN_OUTPUT_GATE, default 0 */
    const int32_t* cu_seqlens;  /* prefill only: DEVICE pointer to num_seqs+1 int32 token offsets
                                   (0 = cu[0] <= cu[1] <= ... <= cu[num_seqs] = T) of packed
                                   sequences; requires B == 1.  NULL: B sequences of T tokens. */
    int num_seqs;               /* number of packed sequences when cu_seqlens != NULL */
    void* workspace;            /* DEVICE scratch of >= gdn_chunk_fwd_workspace_size() bytes,
                                   256-byte aligned; may be NULL when that size is 0 */
    size_t workspace_bytes;
    void* stream;               /* cudaStream_t to enqueue on; NULL = legacy default stream */
    void** events;              /* optional cudaEvent_t[num_events]: events[0] is recorded before
                                   the first kernel of the call and events[i] after kernel i
                                   (kernel-level timing); NULL = none */
    int num_events;
    const float* A_log;         /* [Hv] per-head log forgetting speed (GDN_RAW_GATES), DEVICE */
    const float* dt_bias;       /* [Hv] per-head bias added to a (GDN_RAW_GATES), DEVICE */
    const void* z;              /* output gate input, same shape and dtype as out (GDN_OUTPUT_GATE), DEVICE */
    const float* norm_weight;   /* [dv] (GDN_OUTPUT_GATE), DEVICE */
    float norm_eps;             /* GDN_OUTPUT_GATE epsilon; default 1e-6 */
    float* grad_A_log;          /* gdn_recurrent_bwd with GDN_RAW_GATES: [Hv] dL/dA_log out, DEVICE; NULL = not computed */
    float* grad_dt_bias;        /* gdn_recurrent_bwd with GDN_RAW_GATES: [Hv] dL/ddt_bias out, DEVICE; NULL = not computed */
    const float* conv_bias;     /* gdn_causal_conv1d_*: [C] added before the SiLU, DEVICE; NULL = none */
    float* grad_conv_bias;      /* gdn_causal_conv1d_bwd: [C] dL/dconv_bias out, DEVICE; NULL = not computed */
} gdn_opts_t;

/* Fill *opts with the defaults listed above. */
void gdn_opts_init(gdn_opts_t* opts);

/*
 * gdn_chunk_fwd -- chunked prefill over whole sequences.
 *
 *   q, k     [B, T, Hqk, dk]  dtype          query / key (unit length unless GDN_NORMALIZE_QK)
 *   v        [B, T, Hv, dv]   dtype
 *   g        [B, T, Hv]       dtype          log decay, a_t = exp(g_t)
 *   beta     [B, T, Hv]       dtype          write strength
 *   S0       [nseq, Hv, dk, dv] float or NULL (zero state); nseq = B, or num_seqs when packed
 *   out      [B, T, Hv, dv]   dtype          written for every token (rounded to nearest even)
 *   S_final  [nseq, Hv, dk, dv] float or NULL (not written); may equal S0 (in-place update)
 *
 * Supported: dk, dv in {32, 64, 128}; Hv a multiple of Hqk; B, T >= 0.  T = 0 copies S0 to
 * S_final (zeros when S0 is NULL).  Three kernel families, chosen in this order (opts->chunk does
 * not take part in the choice: the two chunked families block in 64-token chunks for every value):
 *   - bf16 inputs with dk = dv = 128: the tcgen05 tensor-core path; it needs the workspace
 *     (GDN_ERR_WORKSPACE if missing or too small).  Its two kernels run back to back, the second
 *     launched with programmatic stream serialisation so that its set-up overlaps the first one's
 *     last CTAs; an event in opts->events[1] (recorded between them) makes it a plain launch;
 *   - other inputs, when the workspace is at least gdn_chunk_fwd_workspace_size() bytes (256-byte
 *     aligned): the same chunk algebra on split-tf32 tensor-core MMAs in fp32 accuracy,
 *     GDN_NORMALIZE_QK and GDN_RAW_GATES included;
 *   - otherwise the token-serial CUDA-core kernel, which needs no workspace.
 * out must not overlap any input.
 *
 * Errors: GDN_ERR_INVALID_ARG for null required pointers, negative sizes, Hv % Hqk != 0,
 * pointers not 16-byte aligned, cu_seqlens with B != 1 or num_seqs < 1; GDN_ERR_UNSUPPORTED for
 * head dims or a chunk outside the sets above or a device that is not sm_103; GDN_ERR_WORKSPACE
 * when the tensor-core path is selected and the workspace is missing or too small;
 * GDN_ERR_CUDA when a launch fails.
 */
gdn_status_t gdn_chunk_fwd(const void* q, const void* k, const void* v, const void* g,
                           const void* beta, const float* S0, void* out, float* S_final, int B,
                           int T, int Hqk, int Hv, int dk, int dv, const gdn_opts_t* opts);

/* Bytes of device workspace gdn_chunk_fwd needs for these sizes and options (0 if none). */
size_t gdn_chunk_fwd_workspace_size(int B, int T, int Hqk, int Hv, int dk, int dv,
                                    const gdn_opts_t* opts);

/*
 * gdn_recurrent_step -- one decode step: one new token for each of N sequences.
 *
 *   q, k   [N, Hqk, dk] dtype;  v [N, Hv, dv] dtype;  g, beta [N, Hv] dtype
 *   S      [N, Hv, dk, dv] float, read and UPDATED IN PLACE (the state carried between calls,
 *          as delta_rule takes S in and returns the final S)
 *   out    [N, Hv, dv] dtype
 *
 * One pass over the state: each (sequence, head) table is read once and written once.
 * Supported: dk, dv in {32, 64, 128}; Hv a multiple of Hqk; N >= 0 (N = 0 is a no-op).
 * opts->chunk, cu_seqlens and workspace are ignored.  Errors as for gdn_chunk_fwd.
 */
gdn_status_t gdn_recurrent_step(const void* q, const void* k, const void* v, const void* g,
                                const void* beta, float* S, void* out, int N, int Hqk, int Hv,
                                int dk, int dv, const gdn_opts_t* opts);

/*
 * gdn_chunk_fwd_noalloc -- gdn_chunk_fwd for callers that cannot allocate device memory.
 * (No counterpart in the pages: it is a service of this library.)
 *
 * Same arguments, layouts and results as gdn_chunk_fwd; opts->workspace and workspace_bytes are
 * ignored.  The scratch the tensor-core path needs comes from a 64 MiB array built into the
 * library, which every GPU that loads the library holds until the process exits.  Meant for
 * callers that must not call cudaMalloc/cudaFree at this point (a host framework that owns all
 * device memory, a fixed memory budget, code that must not synchronise the device).  The call
 * allocates nothing.
 *
 * Limit: on the tensor-core path, problems whose gdn_chunk_fwd_workspace_size() exceeds 64 MiB
 * are rejected with GDN_ERR_WORKSPACE before anything is launched (for 32 value heads of dim 128
 * that is about 40 chunks of 64 tokens, ~2.5k tokens, per call); other shapes that large run the
 * token-serial kernel.  The 64 MiB are committed on a device when the library's module that
 * holds the array is loaded there: with CUDA's default lazy module loading that is the first call
 * of this entry point on that device (which also looks up the array's device address), with
 * CUDA_MODULE_LOADING=EAGER it is context creation.  A caller that owns nearly all device memory
 * should therefore make its first call early, before the rest of the memory goes to its pool, and
 * before any stream capture; if loading fails the call returns GDN_ERR_CUDA with CUDA's reason in
 * gdn_last_error().  On a device that is not sm_103 it returns GDN_ERR_UNSUPPORTED, as
 * gdn_chunk_fwd does.  All calls on a device share the array, which keeps the previous call's
 * contents (no part of it needs to start at zero); calls that overlap on the GPU race on it, so
 * order them.
 */
gdn_status_t gdn_chunk_fwd_noalloc(const void* q, const void* k, const void* v, const void* g,
                                   const void* beta, const float* S0, void* out, float* S_final,
                                   int B, int T, int Hqk, int Hv, int dk, int dv,
                                   const gdn_opts_t* opts);

/*
 * gdn_causal_conv1d_fwd -- the short causal convolution that feeds q, k and v: depthwise (each
 * channel on its own), window K, then SiLU, as in the GatedDeltaNet shell of "Transformer by Hand,
 * ch. 7" (conv1d with groups = channels and padding K - 1, cut to the first T outputs, SiLU):
 *     y[t, c] = silu( sum_{i<K} w[c, i] * x[t - (K - 1) + i, c] )
 * Inputs before a sequence's first token come from cache_in (zeros when NULL).
 *
 *   x          [B, T, C] dtype, token rows x_stride elements apart (0 = C; a channel slice of a wider
 *              packed projection can be passed directly), 16-byte aligned
 *   w          [C, K] float; w[c, K-1] weighs the current token
 *   cache_in   [nseq, K-1, C] dtype or NULL: the K-1 inputs preceding each sequence, oldest first
 *   y          [B, T, C] dtype; must not overlap x or either cache
 *   cache_out  [nseq, K-1, C] dtype or NULL: the last K-1 inputs of each sequence (what a decode step
 *              needs next; for sequences shorter than K-1 the older entries come from cache_in)
 * nseq = B, or num_seqs with opts->cu_seqlens (B == 1, packed sequences, state reset at each start).
 * opts->conv_bias ([C] float, 4-byte aligned) is added before the SiLU where it is not NULL, as the conv in front of a
 * selective scan has it: in every call of the convolution here and below.
 * Supported: C a multiple of 8, 1 <= K <= 4.  opts->dtype, cu_seqlens, num_seqs, stream are used.
 */
gdn_status_t gdn_causal_conv1d_fwd(const void* x, long long x_stride, const float* w, const void* cache_in,
                                   void* y, void* cache_out, int B, int T, int C, int K,
                                   const gdn_opts_t* opts);

/*
 * gdn_causal_conv1d_step -- one decode token per sequence through the same convolution, with the
 * 3-token (K-1) cache the learn-llm page describes ("at inference the most recent 3 tokens' inputs
 * are cached"):  x [N, C] (rows x_stride apart), cache [N, K-1, C] read and updated in place (shifted
 * by one token), y [N, C].
 */
gdn_status_t gdn_causal_conv1d_step(const void* x, long long x_stride, const float* w, void* cache, void* y,
                                    int N, int C, int K, const gdn_opts_t* opts);

/*
 * gdn_causal_conv1d_fwd_qkv / gdn_causal_conv1d_step_qkv -- the same convolutions over the packed
 * projection of the GatedDeltaNet shell (its q, k and v channels side by side in one row: q in
 * [0, Cq), k in [Cq, Cq + Ck), v in [Cq + Ck, C), C = Cq + Ck + Cv), in one launch, writing the three
 * channel ranges to three dense tensors -- the layouts gdn_chunk_fwd and gdn_recurrent_step take:
 *
 *   x          [B, T, C] (fwd) or [N, C] (step) dtype, rows x_stride elements apart (0 = C)
 *   w          [C, K] float, the channels in the same q | k | v order
 *   y_q, y_k, y_v  [B, T, Cq], [B, T, Ck], [B, T, Cv] (fwd) or [N, Cq], [N, Ck], [N, Cv] (step) dtype
 *   caches     as for the single-output calls, over all C channels
 * Cq, Ck, Cv positive multiples of 8; the results are bit-identical to the single-output call
 * followed by a split of y.  Errors and options as for the single-output calls.
 */
gdn_status_t gdn_causal_conv1d_fwd_qkv(const void* x, long long x_stride, const float* w, const void* cache_in,
                                       void* y_q, void* y_k, void* y_v, void* cache_out, int B, int T, int Cq,
                                       int Ck, int Cv, int K, const gdn_opts_t* opts);
gdn_status_t gdn_causal_conv1d_step_qkv(const void* x, long long x_stride, const float* w, void* cache, void* y_q,
                                        void* y_k, void* y_v, int N, int Cq, int Ck, int Cv, int K,
                                        const gdn_opts_t* opts);

/*
 * gdn_causal_conv1d_bwd -- gradients through gdn_causal_conv1d_fwd, given grad_y = dL/dy and, for a
 * decode that continues from the outgoing cache, grad_cache_out = dL/dcache_out.  With xp a sequence's
 * inputs padded on the left by its K-1 cached inputs, u_t = sum_i w[c, i] xp[t + i] and
 * du_t = grad_y[t] silu'(u_t):
 *     grad_x (and grad_cache_in for the cached rows) = sum_i w[c, i] du_{p - i} at input position p,
 *     plus grad_cache_out for the inputs the outgoing cache holds;
 *     grad_w[c, i] = sum over all tokens of du_t xp[t + i].
 *   x, x_stride, w, cache_in, B, T, C, K, cu_seqlens / num_seqs, dtype: as gdn_causal_conv1d_fwd
 *   grad_y           [B, T, C] dtype, dense (the gradients of the q, k and v slices side by side for
 *                    the packed projection), 16-byte aligned
 *   grad_cache_out   [nseq, K-1, C] dtype or NULL (no loss on the outgoing cache)
 *   grad_x           [B, T, C] float, dense, 16-byte aligned (overwritten)
 *   grad_w           [C, K] float or NULL (not computed); summed over 64-token slots in a fixed order
 *                    through opts->workspace (256-byte aligned, gdn_causal_conv1d_bwd_workspace_size
 *                    bytes; GDN_ERR_WORKSPACE if missing)
 *   grad_cache_in    [nseq, K-1, C] float or NULL (not written), 16-byte aligned
 * opts->grad_conv_bias, where not NULL, receives [C] floats, the sum of du_t over all tokens, in the same fixed order (the
 * workspace is then needed for it too, and gdn_causal_conv1d_bwd_workspace_size counts it); it needs opts->conv_bias.
 * Deterministic.  Asynchronous on opts->stream; events[0] / [1] around the kernels.
 */
size_t gdn_causal_conv1d_bwd_workspace_size(int B, int T, int C, int K, const gdn_opts_t* opts);
gdn_status_t gdn_causal_conv1d_bwd(const void* x, long long x_stride, const float* w, const void* cache_in,
                                   const void* grad_y, const void* grad_cache_out, float* grad_x, float* grad_w,
                                   float* grad_cache_in, int B, int T, int C, int K, const gdn_opts_t* opts);

/*
 * gdn_recurrent_bwd -- the backward pass: gradients of a loss L(out, S_final) of gdn_chunk_fwd with
 * respect to q, k, v, g, beta and S0, given grad_out = dL/dout and grad_S_final = dL/dS_final.  It is
 * the adjoint of the token loop of "Transformer by Hand, ch. 7" (section "The formula"), which the
 * learn-llm "linear attention" page trains through autograd:
 *     lam = dL/dS_t;  lam += scale q_t do_t^T;  dq_t = scale S_t do_t;  dk_t = lam u_t + S_{t-1} dp;
 *     dv_t = beta_t du;  dbeta_t = du.(v_t - a_t p_t);  dg_t = a_t (<lam, S_{t-1}> - beta_t du.p_t);
 *     lam <- a_t lam + k_t dp^T;  dS0 = lam at the start,
 * with p_t = S_{t-1}^T k_t, u_t = beta_t (v_t - a_t p_t), du = lam^T k_t, dp = -a_t beta_t du.
 *
 *   q, k, v, g, beta, S0, B, T, Hqk, Hv, dk, dv, cu_seqlens/num_seqs, scale, dtype: as gdn_chunk_fwd
 *   grad_out       [B, T, Hv, dv] in the inputs' dtype
 *   grad_S_final   [nseq, Hv, dk, dv] float, or NULL (no loss on the final state)
 *   grad_q, grad_k [B, T, Hqk, dk] float (a query/key head sums over the value heads that read it)
 *   grad_v         [B, T, Hv, dv] float;  grad_g, grad_beta [B, T, Hv] float
 *   grad_S0        [nseq, Hv, dk, dv] float, or NULL (not written)
 * Gradients are always fp32.  Pointers need only element alignment.
 * opts->flags may hold GDN_NORMALIZE_QK and GDN_RAW_GATES (GDN_OUTPUT_GATE: GDN_ERR_UNSUPPORTED): the
 * gradients are then those of the forward with the same flags, with respect to its raw inputs -- the
 * unnormalised q, k (dx = r dx_n - r^3 (x . dx_n) x, r = (x . x + 1e-6)^-1/2) and the raw projections
 * a, b passed as g, beta (da = dg (-exp(A_log)) sigmoid(a + dt_bias), db = dbeta beta (1 - beta)) --
 * and, when opts->grad_A_log / grad_dt_bias are not NULL, [Hv] fp32 sums over all tokens of dg g and
 * of da (overwritten, deterministic order).  With either flag the inputs' front-end outputs are formed
 * in fp32: for bf16 inputs with dk = dv = 128 (16-byte aligned q, k, grad_out) inside the kernels,
 * which read the raw inputs and form the per-row l2 scalars and the gates in fp32; otherwise as fp32
 * copies in the workspace (gdn_recurrent_bwd_workspace_size grows accordingly), on which the whole
 * backward runs in fp32 (the split-tf32 kernels).  It is computed through the chunked form
 * of the loop (64-token chunks): the workspace (256-byte aligned, gdn_recurrent_bwd_workspace_size
 * bytes) holds per (chunk, value head) the chunk's UT inverse, decay-masked Q K^T, W, U, decay
 * prefix sums, the state at the chunk start and its adjoint, and dU, all fp32; GDN_ERR_WORKSPACE if
 * missing or too small.  For bf16 inputs with dk = dv = 128 and 16-byte aligned q, k and grad_out the
 * two chunk chains run on the tcgen05 tensor cores (fp32 accuracy through three-part bf16 operand
 * splits).  Asynchronous on opts->stream; events[0] before the four kernels and events[i] after
 * kernel i (1: WY factors, 2: forward chain, 3: adjoint chain, 4: chunk-local gradients).
 */
size_t gdn_recurrent_bwd_workspace_size(int B, int T, int Hqk, int Hv, int dk, int dv, const gdn_opts_t* opts);
gdn_status_t gdn_recurrent_bwd(const void* q, const void* k, const void* v, const void* g, const void* beta,
                               const float* S0, const void* grad_out, const float* grad_S_final, float* grad_q,
                               float* grad_k, float* grad_v, float* grad_g, float* grad_beta, float* grad_S0,
                               int B, int T, int Hqk, int Hv, int dk, int dv, const gdn_opts_t* opts);

/*
 * gdn_output_gate_fwd -- the output gate of the GatedDeltaNet shell on its own ("Transformer by Hand,
 * ch. 7", listing "qwen/deltanet.py": out = GatedRMSNorm(o, z); its parts table: normalised per head,
 * then times silu(z)), per row of dv values (one token and value head):
 *     y_j = o_j / sqrt(mean_j(o_j^2) + eps) * norm_weight_j * silu(z_j)
 * the same pass gdn_chunk_fwd applies with GDN_OUTPUT_GATE, for callers that keep the recurrence's
 * output o (a training step needs it for the backward below).
 *   o, z, y        [rows, dv] dtype (opts->dtype), 16-byte aligned; y may equal o (in place)
 *   norm_weight    [dv] float;  eps = opts->norm_eps
 * Supported dv: 32, 64, 128.  Asynchronous on opts->stream; events[0] / [1] around the kernel.
 */
gdn_status_t gdn_output_gate_fwd(const void* o, const void* z, const float* norm_weight, void* y, long long rows,
                                 int dv, const gdn_opts_t* opts);

/*
 * gdn_output_gate_bwd -- gradients through gdn_output_gate_fwd given grad_y = dL/dy: with
 * inv = (mean(o^2) + eps)^-1/2, o_hat = o inv and gy = grad_y norm_weight silu(z), per row
 *     grad_o = inv (gy - o_hat mean(gy o_hat)),   grad_z = grad_y o_hat norm_weight silu'(z),
 * and grad_norm_weight = sum over all rows of grad_y o_hat silu(z).
 *   o, z, grad_y            [rows, dv] dtype, 16-byte aligned
 *   grad_o, grad_z          [rows, dv] float (overwritten), 16-byte aligned
 *   grad_norm_weight        [dv] float (overwritten), or NULL (not computed); its sum over rows is
 *                           taken in a fixed order through opts->workspace (256-byte aligned,
 *                           gdn_output_gate_bwd_workspace_size bytes; GDN_ERR_WORKSPACE if missing)
 * Deterministic.  Asynchronous on opts->stream; events[0] / [1] around the kernels.
 */
size_t gdn_output_gate_bwd_workspace_size(long long rows, int dv, const gdn_opts_t* opts);
gdn_status_t gdn_output_gate_bwd(const void* o, const void* z, const float* norm_weight, const void* grad_y,
                                 float* grad_o, float* grad_z, float* grad_norm_weight, long long rows, int dv,
                                 const gdn_opts_t* opts);

/*
 * gdn_decay_attn_fwd -- linear attention with a decay for each value head: the rung of the update-rule
 * table (learn-llm page "linear attention") below the delta rule, plain writes into a decaying state,
 * with the decay a constant of the head (a_h = exp(log_decay[h])):
 *     S_t = a_h S_{t-1} + k_t v_t^T,     o_t = scale * S_t^T q_t
 * over whole sequences.  Value head h reads query/key head floor(h / (Hv / Hqk)).
 *   q, k        [B, T, Hqk, dk] dtype, token rows q_stride / k_stride elements apart (0 = dense: Hqk dk)
 *   v           [B, T, Hv, dv] dtype, rows v_stride apart (0 = Hv dv).  Slices of one packed q | k | v
 *               projection can be passed directly; strides are multiples of 16 bytes
 *   log_decay   [Hv] float, <= 0 for a decay (values below -100, -inf among them, act as -100: exp(-100) leaves
 *               nothing; above 0 the state grows by the same formula, and a NaN makes its head's results NaN)
 *   S0          [nseq, Hv, dk, dv] float or NULL (zero states); nseq = B, or num_seqs when packed
 *   out         [B, T, Hv, dv] dtype, dense; must not overlap any input
 *   S_final     [nseq, Hv, dk, dv] float or NULL (not written); may equal S0 (in-place update)
 * Supported: dk, dv in {32, 64, 128}; Hv a multiple of Hqk; B, T >= 0, sequences of no tokens included
 * (their S_final is S0, or zeros), nseq Hv < 2^27, B T < 2^31.  States, sums and decays are fp32.  With
 * bf16 inputs the outputs of sequences of more than 128 tokens hold, beside their own rounding, that of
 * the decayed scores and of the state's copy that q reads to bf16 (0.0023 to 0.0024 of the whole in all,
 * against 0.0017 for the outputs' own); shorter sequences do not, and S_final never does.  A value (a NaN, say) in one
 * sequence's tokens never reaches another sequence's results, nor results of its own that the formula does not
 * give it to (earlier tokens' outputs).  opts->workspace: 256-byte aligned, of
 * gdn_decay_attn_fwd_workspace_size bytes (GDN_ERR_WORKSPACE if that is not 0 and it is missing or too
 * small).  opts->flags must be 0; dtype, scale, cu_seqlens, num_seqs, stream and events[0] / [1] (around
 * the kernels) are used.  Errors otherwise as for gdn_chunk_fwd.
 */
size_t gdn_decay_attn_fwd_workspace_size(int B, int T, int Hqk, int Hv, int dk, int dv, const gdn_opts_t* opts);
gdn_status_t gdn_decay_attn_fwd(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                                long long v_stride, const float* log_decay, const float* S0, void* out, float* S_final,
                                int B, int T, int Hqk, int Hv, int dk, int dv, const gdn_opts_t* opts);

/*
 * gdn_decay_attn_step -- one token for each of N rows through the same recurrence, the states updated in
 * place: q, k [N, Hqk, dk], v [N, Hv, dv] dtype (row strides as above), out [N, Hv, dv] dtype, dense.
 *   S       [num_slots, Hv, dk, dv] float: a pool of states
 *   slots   [N] int32 DEVICE or NULL: row n uses state slots[n] (NULL: state n, num_slots >= N).  A row
 *           whose slot is outside 0 .. num_slots - 1 (-1, say) is idle: its out row is zeros, no state is
 *           touched.  Two rows must not name the same state.
 * Each state is read once and written once.  opts->flags must be 0; cu_seqlens and workspace are ignored.
 */
gdn_status_t gdn_decay_attn_step(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                                 long long v_stride, const float* log_decay, float* S, const int32_t* slots,
                                 int num_slots, void* out, int N, int Hqk, int Hv, int dk, int dv,
                                 const gdn_opts_t* opts);

/*
 * gdn_decay_attn_bwd -- gradients of a loss on (out, S_final) of gdn_decay_attn_fwd with respect to q, k,
 * v and S0 (the decays are constants of the heads and have none).  With lam = dL/dS, walked backwards
 * from grad_S_final:
 *     lam += scale q_t do_t^T;  dq_t = scale S_t do_t;  dk_t = lam v_t;  dv_t = lam^T k_t;  lam <- a lam;
 *     dS0 = lam at the start
 *   q, k, v and their strides, log_decay, S0, B, T, Hqk, Hv, dk, dv: as gdn_decay_attn_fwd
 *   grad_out       [B, T, Hv, dv] dtype, dense
 *   grad_S_final   [nseq, Hv, dk, dv] float or NULL (no loss on the final states)
 *   grad_q, grad_k [B, T, Hqk, dk] dtype, grad_v [B, T, Hv, dv] dtype: the inputs' type, as the backward
 *                  of the convolution that feeds q, k, v takes them; rows gq_stride / gk_stride / gv_stride
 *                  elements apart (0 = dense), so the three can be slices of one packed tensor.  Sums over
 *                  the value heads that share a query/key head are fp32, rounded once
 *   grad_S0        [nseq, Hv, dk, dv] float or NULL (not written)
 * No output may overlap an input or another output (the three scans run side by side).
 * Deterministic.  opts->workspace: 256-byte aligned, gdn_decay_attn_bwd_workspace_size bytes.
 */
size_t gdn_decay_attn_bwd_workspace_size(int B, int T, int Hqk, int Hv, int dk, int dv, const gdn_opts_t* opts);
gdn_status_t gdn_decay_attn_bwd(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                                long long v_stride, const float* log_decay, const float* S0, const void* grad_out,
                                const float* grad_S_final, void* grad_q, long long gq_stride, void* grad_k,
                                long long gk_stride, void* grad_v, long long gv_stride, float* grad_S0, int B, int T,
                                int Hqk, int Hv, int dk, int dv, const gdn_opts_t* opts);

/*
 * gdn_block_norm_fwd -- what surrounds a layer's block, in one pass over the rows: the norm after the
 * block, its gate and residual scale, the residual add, and the norm before the next block.  Per row of D
 * values, with b the block's output and x the residual stream:
 *     y = b / sqrt(mean(b^2) + eps) * post_weight
 *     r = x + res_scale * sigmoid(gate) * y            (the new residual stream)
 *     n = r / sqrt(mean(r^2) + eps) * pre_weight       (the next block's input; r before its rounding)
 *   x, b, r, n               [rows, D] dtype, 16-byte aligned; r may equal x and n may equal b (in place)
 *   gate                     logits [rows, D] (gate_cols = D) or [rows] (gate_cols = 1) dtype, or NULL (no gate)
 *   res_scale                [D] float or NULL (1)
 *   post_weight, pre_weight  [D] float
 * Supported: D a multiple of 8 up to 8192, rows >= 0.  eps = opts->norm_eps; opts->flags must be 0.
 */
gdn_status_t gdn_block_norm_fwd(const void* x, const void* b, const void* gate, int gate_cols, const float* res_scale,
                                const float* post_weight, const float* pre_weight, void* r, void* n, long long rows,
                                int D, const gdn_opts_t* opts);

/*
 * gdn_block_norm_bwd -- gradients through gdn_block_norm_fwd given grad_r = dL/dr and grad_n = dL/dn, from
 * the forward's inputs (r is formed again, so nothing of the forward has to be kept).
 *   grad_x, grad_b           [rows, D] dtype, 16-byte aligned
 *   grad_gate                like gate, dtype (required with a gate)
 *   grad_post, grad_pre, grad_res_scale   [D] float, each may be NULL (not computed): sums over the rows in
 *                            a fixed order through opts->workspace (256-byte aligned,
 *                            gdn_block_norm_bwd_workspace_size bytes; needed if one of them is wanted)
 * Deterministic.  Errors and options as for gdn_block_norm_fwd.
 */
size_t gdn_block_norm_bwd_workspace_size(long long rows, int D, const gdn_opts_t* opts);
gdn_status_t gdn_block_norm_bwd(const void* x, const void* b, const void* gate, int gate_cols, const float* res_scale,
                                const float* post_weight, const float* pre_weight, const void* grad_r,
                                const void* grad_n, void* grad_x, void* grad_b, void* grad_gate, float* grad_post,
                                float* grad_pre, float* grad_res_scale, long long rows, int D, const gdn_opts_t* opts);

/*
 * gdn_selective_scan_fwd -- the selective state space scan: a recurrence with a diagonal state for each channel whose
 * decay and write strength come from the token (the gated-linear rung of the update-rule table, learn-llm page "linear
 * attention", with a state of N values a channel).  Per sequence, channel d of group g(d) = floor(d / (D / G)) and state n:
 *     dt_t = softplus(delta_t + dt_bias),   A = -exp(A_log),   h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t
 *     y_t  = (sum_n C_t h_t + skip u_t) silu(z_t)
 *   u, delta, z  [B, T, D] dtype, token rows u_stride / delta_stride / z_stride elements apart (0 = dense: D); z may be
 *                NULL (no gate).  u is what gdn_causal_conv1d_fwd writes
 *   Bm, Cm       [B, T, G, N] dtype, rows b_stride / c_stride apart (0 = G N).  Slices of one packed projection can be
 *                passed directly; strides are multiples of 16 bytes and at most 2^24 elements
 *   A_log        [D, N] float;  skip, dt_bias [D] float, each may be NULL (0)
 *   h0           [nseq, D, N] float or NULL (zero states); nseq = B, or num_seqs when packed
 *   y            [B, T, D] dtype, dense; must not overlap any input
 *   h_final      [nseq, D, N] float or NULL (not written); may equal h0 (in-place update)
 * Supported: N in {8, 16, 32, 64}; D a multiple of 8 G; B, T >= 0, sequences of no tokens included (their h_final is h0,
 * or zeros), B T < 2^31.  dt, decays, states and sums are fp32.  Token rows of no sequence (behind the last one's end)
 * are not written.  A value that is not finite reaches only the results that the formula gives it to (its channel's
 * later tokens, or, from B and C, its group's).  opts->workspace: 256-byte aligned, of
 * gdn_selective_scan_fwd_workspace_size bytes (GDN_ERR_WORKSPACE if that is not 0 and it is missing or too small).
 * opts->flags must be 0; dtype, cu_seqlens, num_seqs, stream and events[0] / [1] (around the kernels) are used; scale is
 * not.  All pointers are 16-byte aligned.  Errors otherwise as for gdn_chunk_fwd.
 */
size_t gdn_selective_scan_fwd_workspace_size(int B, int T, int D, int G, int N, const gdn_opts_t* opts);
gdn_status_t gdn_selective_scan_fwd(const void* u, long long u_stride, const void* delta, long long delta_stride,
                                    const float* A_log, const void* Bm, long long b_stride, const void* Cm,
                                    long long c_stride, const float* skip, const float* dt_bias, const void* z,
                                    long long z_stride, const float* h0, void* y, float* h_final, int B, int T, int D,
                                    int G, int N, const gdn_opts_t* opts);

/*
 * gdn_selective_scan_step -- one token for each of `rows` rows through the same recurrence, the states updated in place:
 * u, delta, z [rows, D], Bm, Cm [rows, G, N] dtype (row strides as above), y [rows, D] dtype, dense.
 *   h       [num_slots, D, N] float: a pool of states
 *   slots   [rows] int32 DEVICE or NULL: row n uses state slots[n] (NULL: state n, num_slots >= rows).  A row whose slot
 *           is outside 0 .. num_slots - 1 (-1, say) is idle: its y row is zeros, no state is touched.  Two rows must not
 *           name the same state.
 * y overlaps no input.  Each state is read once and written once.  opts->flags must be 0; cu_seqlens and workspace are ignored.
 */
gdn_status_t gdn_selective_scan_step(const void* u, long long u_stride, const void* delta, long long delta_stride,
                                     const float* A_log, const void* Bm, long long b_stride, const void* Cm,
                                     long long c_stride, const float* skip, const float* dt_bias, const void* z,
                                     long long z_stride, float* h, const int32_t* slots, int num_slots, void* y,
                                     int rows, int D, int G, int N, const gdn_opts_t* opts);

/*
 * gdn_selective_scan_bwd -- gradients of a loss on (y, h_final) of gdn_selective_scan_fwd, from its inputs, grad_y =
 * dL/dy and grad_h_final = dL/dh_final.  With p = grad_y silu(z) and lam = dL/dh walked backwards from grad_h_final,
 *     lam_t = C_t p_t + a_{t+1} lam_{t+1};   dC = sum_d p h;   dB = sum_d lam dt u;   q = sum_n lam B;
 *     w = lam a h_{t-1};   du = dt q + skip p;   ddelta = (u q + sum_n A w) sigmoid(delta + dt_bias);
 *     dA_log = A sum_t dt w;   dskip = sum_t p u;   ddt_bias = sum_t ddelta;   dz = grad_y (sum_n C h + skip u) silu'(z);
 *     dh0 = a_1 lam_1
 *   inputs, strides, B, T, D, G, N   as gdn_selective_scan_fwd
 *   grad_y         [B, T, D] dtype, dense;  grad_h_final [nseq, D, N] float or NULL (no loss on the final states)
 *   grad_u, grad_delta   [B, T, D] dtype, dense
 *   grad_B, grad_C       [B, T, G, N] dtype, rows gb_stride / gc_stride elements apart (0 = dense), and grad_z (required
 *                  with z) [B, T, D] dtype, rows gz_stride apart: they can be slices of packed gradients
 *   grad_A_log [D, N], grad_skip [D], grad_dt_bias [D], grad_h0 [nseq, D, N] float, each may be NULL (not computed)
 * Sums are fp32 and rounded once.  No output may overlap an input or another output.  Deterministic.
 * opts->workspace: 256-byte aligned, gdn_selective_scan_bwd_workspace_size bytes: in floats about D N for every 8 tokens
 * and every sequence (states that are kept), 3 (N + 1) D for every segment of 32 to 512 tokens and every sequence, and 2 N
 * for every token and tile of 1024 / N channels of a group (sums for grad_B and grad_C).  2 x 8192 tokens of 4096 channels
 * of 16 states: 0.75 GB, where a bf16 tensor of the tokens has 0.13; the same tokens as 256 sequences 1.04 GB.
 */
size_t gdn_selective_scan_bwd_workspace_size(int B, int T, int D, int G, int N, const gdn_opts_t* opts);
gdn_status_t gdn_selective_scan_bwd(const void* u, long long u_stride, const void* delta, long long delta_stride,
                                    const float* A_log, const void* Bm, long long b_stride, const void* Cm,
                                    long long c_stride, const float* skip, const float* dt_bias, const void* z,
                                    long long z_stride, const float* h0, const void* grad_y, const float* grad_h_final,
                                    void* grad_u, void* grad_delta, float* grad_A_log, void* grad_B, long long gb_stride,
                                    void* grad_C, long long gc_stride, float* grad_skip, float* grad_dt_bias,
                                    void* grad_z, long long gz_stride, float* grad_h0, int B, int T, int D, int G, int N,
                                    const gdn_opts_t* opts);

/*
 * gdn_layer_norm_fwd -- layer norm with the residual add in front of it, in one pass over the rows: per row of D values
 *     r = x + b,   n = (r - mean(r)) / sqrt(mean((r - mean(r))^2) + eps) * weight + bias
 * (n from r before its rounding).
 *   x, n      [rows, D] dtype, 16-byte aligned; n may equal x or b (in place)
 *   b, r      [rows, D] dtype, both or neither (NULL: r = x); r may equal x or b, but not n
 *   weight    [D] float;  bias [D] float or NULL (0)
 * Supported: D a multiple of 8 up to 8192, rows >= 0.  eps = opts->norm_eps; opts->flags must be 0.
 */
gdn_status_t gdn_layer_norm_fwd(const void* x, const void* b, const float* weight, const float* bias, void* n, void* r,
                                long long rows, int D, const gdn_opts_t* opts);

/*
 * gdn_layer_norm_bwd -- gradients through gdn_layer_norm_fwd given grad_n = dL/dn and, for a residual stream that goes
 * on, grad_r = dL/dr, from the forward's inputs (r is formed again, so nothing of the forward has to be kept).
 *   grad_r                     [rows, D] dtype or NULL (no loss on r)
 *   grad_x                     [rows, D] dtype, 16-byte aligned: the gradient of x, and of b
 *   grad_weight, grad_bias     [D] float, each may be NULL (not computed): sums over the rows in a fixed order through
 *                              opts->workspace (256-byte aligned, gdn_layer_norm_bwd_workspace_size bytes; needed if one
 *                              of them is wanted)
 * grad_x overlaps no input.  Deterministic.  Errors and options as for gdn_layer_norm_fwd.
 */
size_t gdn_layer_norm_bwd_workspace_size(long long rows, int D, const gdn_opts_t* opts);
gdn_status_t gdn_layer_norm_bwd(const void* x, const void* b, const float* weight, const void* grad_n, const void* grad_r,
                                void* grad_x, float* grad_weight, float* grad_bias, long long rows, int D,
                                const gdn_opts_t* opts);

/* Synchronise `stream` (cudaStream_t, NULL = legacy), then read and clear the device status word
 * that kernels set when a bounded wait runs out.  GDN_OK if clear, GDN_ERR_TIMEOUT if set,
 * GDN_ERR_CUDA if the synchronisation itself failed. */
gdn_status_t gdn_check_device_status(void* stream);

/* Static description of a status code. */
const char* gdn_status_string(gdn_status_t status);

/* Message of the last failure on the calling thread ("" if none). */
const char* gdn_last_error(void);

/* GDN_VERSION of the header that the library was built with: major * 10000 + minor * 100 + patch. */
int gdn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
