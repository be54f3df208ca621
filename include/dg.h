/*
 * dg.h -- C ABI of the MI355X (gfx950) block-scaled FP8 GEMM library.
 *
 * Computes D = A . B^T in bf16 from e4m3 operands with fine-grained fp32
 * scales, and its two MoE grouped forms.  The operation is the one defined by
 * Lesson 13 "DeepSeek DeepGEMM core architecture and Hopper FP8 operator
 * breakdown" (hpc.payai.win), Fig. 13-1 and its closed-form equation:
 *
 *   D[i,j] = sum_g alpha[i,g] * beta[j/128, g] * sum_{k<128} A[i,128g+k] * B[j,128g+k]
 *
 * where each 128-wide K block's partial product is scaled by alpha*beta and
 * added into an fp32 accumulator inside the main loop, and the epilogue only
 * converts to bf16 (round to nearest even).  Layout is NT: A is [M,K] and B is
 * [N,K], both K-contiguous (DeepGEMM architecture deep dive, blog.123qwe.co.kr,
 * section 3, "D = A @ B.T").
 *
 * Conventions shared by every entry point
 *   - e4m3 means OCP FP8 E4M3FN (bias 7, max 448, 0x7F/0xFF NaN), passed as
 *     uint8_t bytes; bf16 is passed as uint16_t bit patterns.
 *   - Every array pointer is a DEVICE pointer owned by the caller; the library
 *     never allocates, frees or synchronises on these calls.  Pointers must be
 *     16-byte aligned (DG_ERR_ALIGN otherwise) except the scale, index and
 *     workspace arrays, which need 4-byte alignment.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *     Every call only enqueues work on that stream and returns; the calls
 *     allocate nothing and never read device data on the host, so they may be
 *     captured into a hipGraph.  Kernel faults surface through the usual HIP
 *     stream error reporting.
 *   - Shapes are int64_t.  K must be a positive multiple of 128, N a positive
 *     multiple of 16, row counts >= 0 (0 rows = nothing to do, DG_OK).
 *   - Return value: DG_OK or one of the DG_ERR_* codes below; on error nothing
 *     is enqueued and dg_get_last_error() returns a message (thread-local).
 *   - Scale layouts: activation scales alpha are MN-major, [K/128][rows] fp32
 *     (per expert for the masked form); weight scales beta are
 *     [ceil(N/128)][K/128] fp32 per expert.  alpha = amax/448 over each 1x128
 *     row group; beta = amax/448 over each 128x128 block (Lesson 13,
 *     Fig. 13-1).
 *   - D rows that the operation does not define (padding rows of the
 *     contiguous form, rows past masked_m of the masked form) are never
 *     written.
 *   - Results are deterministic: the same inputs give bit-identical outputs.
 *   - Sizes: the kernels address one launch's activations, scales and
 *     outputs, and one expert's weights, with 32-bit byte offsets from 64-bit
 *     bases.  A call with more rows than that allows runs as several row
 *     chunks enqueued back to back on `stream` (each planned on its own; the
 *     results are those of one launch per chunk).  Rejected with DG_ERR_SHAPE:
 *     one expert's weights of 4 GiB or more ((N + 256) * K bytes, bf16: twice
 *     that), activation scales of 4 GiB or more, more than 1024 groups, and
 *     the K-grouped form past 32-bit offsets (see there).
 */
#ifndef DG_H
#define DG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  DG_OK = 0,
  DG_ERR_INVALID_ARG = 1, /* null pointer, bad enum value */
  DG_ERR_SHAPE = 2,       /* K % 128 (K % 64 for bf16), N % 16, negative sizes, G out of [1, 1024],
                             weights of 4 GiB or more per expert */
  DG_ERR_ALIGN = 3,       /* pointer alignment */
  DG_ERR_WORKSPACE = 4,   /* workspace pointer given with a size that is not a multiple of 4 */
  DG_ERR_DEVICE = 5,      /* no HIP device, or the current device is not gfx950 */
  DG_ERR_LAUNCH = 6       /* the kernel launch itself failed */
};

/* Operation ids for dg_get_workspace_size. */
enum {
  DG_OP_GEMM_NT = 0,
  DG_OP_CONTIGUOUS = 1,
  DG_OP_MASKED = 2,
  DG_OP_BF16_GEMM_NT = 3,
  DG_OP_GEMM_NT_UE8M0 = 4,
  DG_OP_K_GROUPED = 5, /* dg_k_grouped_fp8_gemm_nt_contiguous (plan description only) */
  DG_OP_MXFP4_GEMM_NT = 6,
  DG_OP_MOE_GATE = 7,  /* workspace only: rows = T, N = E */
  DG_OP_MOE_LAYOUT = 8, /* workspace only: rows = T, K = k */
  DG_OP_MOE_EXPERTS = 9,    /* workspace only: rows = T k, N = H, K = I */
  DG_OP_RMS_NORM_BWD = 10,  /* workspace only: rows = M, K */
  DG_OP_EPILOGUE_BWD = 11   /* workspace only: rows = M, N */
};

/* Activations of dg_fp8_gemm_nt_epilogue: z, max(z, 0), z / (1 + e^-z), z Phi(z)
 * (the normal distribution's), and z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2. */
enum { DG_ACT_NONE = 0, DG_ACT_RELU = 1, DG_ACT_SILU = 2, DG_ACT_GELU = 3, DG_ACT_GELU_TANH = 4 };

/* Scales of a quantised output: one fp32 or one UE8M0 code (packed) per 1x128. */
enum { DG_SCALE_F32 = 0, DG_SCALE_UE8M0 = 1 };

/* Element types of the operators that take more than one. */
enum { DG_F32 = 0, DG_BF16 = 1 };

/*
 * Dense GEMM.  Lesson 13, Fig. 13-1; DeepGEMM's "normal" GEMM (the Feb-2025
 * release article on dakule.com, usage section).
 *   A   [M,K]  e4m3, row-major          sfa [K/128][M] fp32
 *   B   [N,K]  e4m3, row-major          sfb [ceil(N/128)][K/128] fp32
 *   D   [M,N]  bf16, row-major (written)
 * workspace: optional scratch for splitting K across workgroups when the
 *   output has too few tiles to fill the GPU (small M).  Pass NULL/0 to run
 *   without it (possibly slower; the split changes only the fp32 summation
 *   order, so results agree within rounding, and each configuration is
 *   deterministic).  Required size for the full split is
 *   dg_get_workspace_size(DG_OP_GEMM_NT, M, N, K, 1); a smaller buffer limits
 *   the split.  The workspace MUST be zero-filled before its first use (e.g.
 *   hipMemset once after allocation): whenever the plan splits K (the
 *   skinny kernel, at up to 2048 rows, or a partial last round of 256 x 128
 *   tiles) its first 4 KiB hold per-tile completion counters and the fp32
 *   partials follow; every call leaves the counters at zero again, so a workspace stays reusable across calls and
 *   shapes without clearing.  Calls that share one workspace must be ordered
 *   on one stream.
 */
int dg_fp8_gemm_nt(const uint8_t* A, const float* sfa, const uint8_t* B, const float* sfb,
                   uint16_t* D, int64_t M, int64_t N, int64_t K, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * Allocation-free dense GEMM, for callers that cannot allocate (code under
 * graph capture, tight serving loops, harnesses that forbid allocation):
 * dg_fp8_gemm_nt with no workspace argument.  Same operands, result and plan
 * as dg_fp8_gemm_nt given a workspace of dg_get_workspace_size(DG_OP_GEMM_NT,
 * M, N, K, 1) bytes (so the outputs are bit-identical); the K-split partials
 * and counters live in a static device array of 40 MiB that every GPU the
 * library runs on holds until the process ends.  Shapes whose split-K scratch
 * would exceed 40 MiB return DG_ERR_WORKSPACE (none does under the default
 * plans on 256 CUs).  Nothing is allocated; the first call on a device
 * resolves the array's address and clears its counter area with a small
 * kernel on `stream`.  Calls that overlap on one GPU (other streams, other
 * threads, concurrent graph replays) share the array and race: order them.
 */
int dg_fp8_gemm_nt_noalloc(const uint8_t* A, const float* sfa, const uint8_t* B, const float* sfb,
                           uint16_t* D, int64_t M, int64_t N, int64_t K, void* stream);

/*
 * M-grouped contiguous GEMM (MoE training forward / prefill).  Lesson 13,
 * Fig. 13-3 (contiguous layout); deep-dive blog section 3 (grouped API table,
 * per-expert segments aligned to the M block).
 *   A         [M_total,K] e4m3, rows of all experts concatenated
 *   sfa       [K/128][M_total] fp32
 *   B         [G,N,K] e4m3 (one weight per expert, same N and K for all)
 *   sfb       [G][ceil(N/128)][K/128] fp32
 *   m_indices [M_total] int32, device: expert of each row; a value outside
 *             [0,G) marks a padding row, whose D row is not written
 *   D         [M_total,N] bf16
 * Each aligned block of dg_get_m_alignment_for_contiguous_layout() rows must
 * hold rows of at most one expert (segments padded to that alignment); rows
 * of a block whose index differs from the block's expert are not written.
 * G must be in [1, 1024]; each expert's weights are addressed from the
 * expert's own base.  workspace: unused, pass NULL/0.
 */
int dg_m_grouped_fp8_gemm_nt_contiguous(const uint8_t* A, const float* sfa, const uint8_t* B,
                                        const float* sfb, uint16_t* D, const int32_t* m_indices,
                                        int64_t M_total, int64_t N, int64_t K, int64_t G,
                                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * M-grouped masked GEMM (MoE decode under graph capture).  Lesson 13,
 * Fig. 13-3 (masked layout) and the answer to Q3: fixed-capacity buffers per
 * expert and a device array of valid row counts read by the kernel, so the
 * launch never depends on host knowledge of the counts.
 *   A        [G,max_m,K] e4m3             sfa [G][K/128][max_m] fp32
 *   B        [G,N,K] e4m3                 sfb [G][ceil(N/128)][K/128] fp32
 *   masked_m [G] int32, device: expert g's rows [0, clamp(masked_m[g],0,max_m))
 *            are computed; all other rows of D are not written
 *   D        [G,max_m,N] bf16
 * G must be in [1, 1024]; each expert's A, alpha, weights and D are
 * addressed from the expert's own base, so one expert's rows must fit 32-bit
 * offsets ((max_m + 256) * K and max_m * N * 2 bytes below 4 GiB).
 * expected_m: host hint of the typical masked_m (0 = unknown); it is not
 *   used (the launch shape and the results never depend on it).
 * workspace: unused, pass NULL/0.
 */
int dg_m_grouped_fp8_gemm_nt_masked(const uint8_t* A, const float* sfa, const uint8_t* B,
                                    const float* sfb, uint16_t* D, const int32_t* masked_m,
                                    int64_t G, int64_t max_m, int64_t N, int64_t K,
                                    int64_t expected_m, void* workspace, size_t workspace_bytes,
                                    void* stream);

/*
 * Accumulating dense GEMM, D = C + A . B^T in fp32.  Deep-dive blog, section 3:
 * every GEMM of the library has the form D = C + A @ B (NT: A @ B^T).
 *   A, sfa, B, sfb as for dg_fp8_gemm_nt
 *   C [M,N] fp32, row-major, or NULL (read as zeros); may equal D (in place)
 *   D [M,N] fp32, row-major (written)
 * D = fl32(C + acc): the fp32 accumulator of the promoted GEMM plus C, rounded
 * once.  workspace as for dg_fp8_gemm_nt (same size query, DG_OP_GEMM_NT,
 * which covers both forms).
 */
int dg_fp8_gemm_nt_acc(const uint8_t* A, const float* sfa, const uint8_t* B, const float* sfb,
                       const float* C, float* D, int64_t M, int64_t N, int64_t K, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * Dense GEMM with bias, activation and residual: z = A . B^T + bias,
 * D = act(z) + residual, all in fp32 and rounded once to bf16 (the activations
 * are within 1e-4 of their values before that, where these are above 2^-118; an
 * infinite z gives NaN where the formula has inf * 0: silu and gelu_tanh of
 * -inf, and the slopes of silu and gelu).
 *   A, sfa, B, sfb, workspace as for dg_fp8_gemm_nt (same size query)
 *   bias     [N] fp32 or NULL      act  one of DG_ACT_*
 *   residual [M,N] bf16 or NULL; may equal D (in place)
 *   pre      [M,N] bf16 or NULL (written): z, what dg_epilogue_bwd reads
 * bias, residual and pre are 16-byte aligned; apart from residual = D no two
 * arrays overlap.
 */
int dg_fp8_gemm_nt_epilogue(const uint8_t* A, const float* sfa, const uint8_t* B, const float* sfb, const float* bias,
                            int act, const uint16_t* residual, uint16_t* pre, uint16_t* D, int64_t M, int64_t N,
                            int64_t K, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradient of that epilogue: dz = dy act'(pre) (the residual's gradient is dy,
 * the operands' are products of dz).
 *   dy [M,N] bf16        pre [M,N] bf16, unused (may be NULL) for DG_ACT_NONE
 *   dz [M,N] bf16 or NULL (written); may equal dy or pre
 *   q  [M,N] e4m3 and sf [N/128][M] fp32, both or neither (written): the 1x128
 *      quantisation of dz before its rounding (rules of dg_quant_1x128), the
 *      left operand of the product that gives A's gradient; N a multiple of 128
 *   dbias [N] fp32 or NULL (written): the sum of dz over the rows (zeros for M = 0)
 * N is a multiple of 16.  workspace: required with dbias,
 * dg_get_workspace_size(DG_OP_EPILOGUE_BWD, M, N, 0, 1) bytes; it need not be
 * zero, and its first 4 KiB are left as they are.  Deterministic.
 */
int dg_epilogue_bwd(const uint16_t* dy, const uint16_t* pre, int act, uint16_t* dz, uint8_t* q, float* sf, float* dbias,
                    int64_t M, int64_t N, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Root-mean-square norm of rows, with the residual's addition before it and the
 * next product's quantisation after it:
 *   h = x + residual, rounded to `dtype` (x itself without a residual)
 *   r = 1 / sqrt(mean(h^2) + eps),  v = (h r) weight
 *   x, residual [M,K] of `dtype` (DG_F32 or DG_BF16), residual may be NULL
 *   weight [K] of `weight_dtype`
 *   h    [M,K] of `dtype` (written), may be NULL without a residual; may equal x or residual
 *   y    [M,K] of `dtype` or NULL (written): v rounded; may equal x or residual, not h
 *   q    [M,K] e4m3 or NULL (written) with sf: the 1x128 quantisation of v in
 *        fp32, scales and rules of dg_quant_1x128 (DG_SCALE_F32: sf [K/128][M]
 *        fp32) or dg_quant_1x128_ue8m0 (DG_SCALE_UE8M0: sf [ceil(K/512)][M] int32)
 *   rstd [M] fp32 or NULL (written): r
 * At least one of y and q is given.  K is a multiple of 8 (with q: of 128) up to
 * 16384, M below 2^23, eps positive; sums are fp32, so a row whose sum of squares
 * passes 3.4e38 has r = 0.  A row with a NaN gives NaN in y, one with an infinity
 * zeros, and NaN at the infinity; codes of such rows are unspecified.
 * Deterministic.
 *
 * dg_rms_norm_bwd: with n = h r,
 *   dx [M,K] of `dtype` (written) = dh + r (weight dy - n mean(weight dy n))
 *   dw [K] fp32 (written) = sum over the rows of dy n (zeros for M = 0)
 * dy [M,K] and dh [M,K] (the gradient that reaches h by other ways, or NULL) of
 * `dtype`; h and rstd are dg_rms_norm's (x without a residual).  dx is the
 * gradient of x and of the residual; it may equal dy, h or dh.  workspace:
 * required, dg_get_workspace_size(DG_OP_RMS_NORM_BWD, M, 0, K, 1) bytes; it need
 * not be zero, and its first 4 KiB are left as they are.  Deterministic.
 */
int dg_rms_norm(const void* x, const void* residual, const void* weight, int dtype, int weight_dtype, void* h, void* y,
                uint8_t* q, void* sf, int scale_kind, float* rstd, int64_t M, int64_t K, float eps, void* stream);
int dg_rms_norm_bwd(const void* dy, const void* h, const void* weight, const float* rstd, int dtype, int weight_dtype,
                    const void* dh, void* dx, float* dw, int64_t M, int64_t K, void* workspace, size_t workspace_bytes,
                    void* stream);

/*
 * K-grouped contiguous GEMM (MoE weight gradient), D[g] = C[g] + A_g . B_g^T
 * in fp32.  Deep-dive blog, section 3: the K-grouped contiguous family groups
 * along K with M and N fixed and serves the backward pass of MoE weights;
 * every GEMM there has the form D = C + A @ B, and contiguous segments are
 * aligned to the block size (M and K).  Group g owns the K range that starts
 * after the first g segments: A_g = A[:, seg g], B_g = B[:, seg g].
 *   A   [M,K] e4m3, row-major (K = the sum of the segments, e.g. tokens)
 *   sfa [K/128][M] fp32: one scale per row per 128 K (1x128, Lesson 13 Fig. 13-1)
 *   B   [N,K] e4m3, row-major
 *   sfb [K/128][N] fp32: also per row per 128 K (both operands are activations)
 *   ks  [G] int32, device: K length of each group, a multiple of 128 (zero
 *       allowed).  Read by the kernel: group g covers K blocks
 *       [sum_{h<g} floor(ks[h]/128), + floor(ks[g]/128)), negative lengths
 *       count as 0 and blocks past K/128 are dropped; K positions after the
 *       last segment belong to no group.
 *   C   [G,M,N] fp32 or NULL (zeros); may equal D (in place)
 *   D   [G,M,N] fp32 (written, every group; a group without K blocks gets C[g])
 * D[g] = fl32(C[g] + acc_g), acc_g the fp32 accumulator of the promoted
 * products over the group's blocks.  G must be in [1, 1024]; problems whose
 * A, B or per-group D byte offsets exceed 32 bits are rejected with
 * DG_ERR_SHAPE.  workspace: unused, pass NULL/0.
 */
int dg_k_grouped_fp8_gemm_nt_contiguous(const uint8_t* A, const float* sfa, const uint8_t* B,
                                        const float* sfb, const float* C, float* D,
                                        const int32_t* ks, int64_t G, int64_t M, int64_t N,
                                        int64_t K, void* workspace, size_t workspace_bytes,
                                        void* stream);

/*
 * BF16 dense GEMM, D = A . B^T, no scales.  BF16 is among the library's
 * precisions (deep-dive blog, section 1 overview table); the Ascend 950
 * article (benchmarks section) measures this GEMM at M=4096, N=7168, K=16384.
 *   A [M,K] bf16, row-major      B [N,K] bf16, row-major
 *   D [M,N] bf16, row-major (written); fp32 accumulation, round-to-nearest-even
 * K must be a multiple of 64, N of 16.  workspace: as for dg_fp8_gemm_nt
 * (optional, lets a partial last round of tiles split along K; size from
 * dg_get_workspace_size(DG_OP_BF16_GEMM_NT, M, N, K, 1); zero-filled before
 * first use, left reusable).
 */
int dg_bf16_gemm_nt(const uint16_t* A, const uint16_t* B, uint16_t* D, int64_t M, int64_t N, int64_t K,
                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * 1x128 activation quantiser.  Lesson 13, Fig. 13-1 (one scale per token per
 * 128 K elements, scale = amax/448).
 *   x   [G,M,K] fp32 (G=1 for a plain [M,K] matrix)
 *   q   [G,M,K] e4m3 (written)
 *   sfa [G][K/128][M] fp32 (written)
 * alpha = fl32(amax / 448) by IEEE division; q = e4m3_RNE(fl32(x / alpha)),
 * ties to even, sign of zero kept, saturating at +-448; a group with amax = 0
 * (or amax/448 underflowing to 0) gets alpha = 1.  Non-finite inputs give
 * unspecified codes.  Bit-exact and deterministic.  Limits: G <= 65535,
 * M <= 2^31 - 16 and ceil(M / 16) * (K / 128) < 2^31 (else DG_ERR_SHAPE); x and q 16-byte
 * aligned, sfa 4-byte aligned (else DG_ERR_ALIGN).
 */
int dg_quant_1x128(const float* x, uint8_t* q, float* sfa, int64_t G, int64_t M, int64_t K,
                   void* stream);

/*
 * 128x128 weight quantiser.  Lesson 13, Fig. 13-1 (one scale per 128x128
 * block of the weight, stored fp32).
 *   x   [G,N,K] fp32       q [G,N,K] e4m3 (written)
 *   sfb [G][ceil(N/128)][K/128] fp32 (written)
 * Same rounding rules as dg_quant_1x128; when N is not a multiple of 128 the
 * last block's amax covers only its existing rows.
 */
int dg_quant_128x128(const float* x, uint8_t* q, float* sfb, int64_t G, int64_t N, int64_t K,
                     void* stream);

/*
 * UE8M0 (power-of-two) scale variant.  Lesson 13 (the notes after Fig. 13-1):
 * newer library versions accept UE8M0 scales besides fp32; deep-dive blog,
 * section 3: on the newer architecture four UE8M0 scales are packed into one
 * 32-bit integer.  Same granularity and per-128-K promotion as the fp32 form.
 * A code c means 2^(c - 127); codes of four consecutive K blocks share one
 * int32, block 4w + j in byte j (bits 8j..8j+7), unused bytes zero.
 *   sfa [ceil(K/512)][M] int32 (MN-major, as the fp32 layout)
 *   sfb [ceil(N/128)][ceil(K/512)] int32
 * The quantisers choose c so that 2^(c-127) is the smallest power of two not
 * below amax/448 (clamped to codes [0, 254]; an all-zero group gets 127) and
 * write q = e4m3_RNE(x * 2^(127-c)), an exact power-of-two scaling.
 * dg_fp8_gemm_nt_ue8m0: D [M,N] bf16 = A . B^T with those scales; the matrix
 * cores apply the scales and add each K block's product to the fp32
 * accumulator, rounded once.  workspace as for dg_fp8_gemm_nt (size from
 * dg_get_workspace_size(DG_OP_GEMM_NT_UE8M0, M, N, K, 1)).
 */
int dg_quant_1x128_ue8m0(const float* x, uint8_t* q, int32_t* sfa, int64_t G, int64_t M, int64_t K,
                         void* stream);
int dg_quant_128x128_ue8m0(const float* x, uint8_t* q, int32_t* sfb, int64_t G, int64_t N, int64_t K,
                           void* stream);
int dg_fp8_gemm_nt_ue8m0(const uint8_t* A, const int32_t* sfa, const uint8_t* B, const int32_t* sfb,
                         uint16_t* D, int64_t M, int64_t N, int64_t K, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * M-grouped contiguous and masked GEMMs with UE8M0 scales (the grouped forms
 * of dg_fp8_gemm_nt_ue8m0; deep-dive blog, section 3: the grouped GEMMs take
 * the scale formats of the plain ones).  Operands, index arrays, outputs and
 * rules as for dg_m_grouped_fp8_gemm_nt_contiguous / _masked, with packed
 * int32 scales (four K blocks per word, block 4w + j in byte j):
 *   contiguous: sfa [ceil(K/512)][M_total], sfb [G][ceil(N/128)][ceil(K/512)]
 *   masked:     sfa [G][ceil(K/512)][max_m], sfb [G][ceil(N/128)][ceil(K/512)]
 * (dg_quant_1x128_ue8m0 with G groups writes the masked activation layout,
 * dg_quant_128x128_ue8m0 with G experts the weight layout).
 */
int dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0(const uint8_t* A, const int32_t* sfa, const uint8_t* B,
                                              const int32_t* sfb, uint16_t* D, const int32_t* m_indices,
                                              int64_t M_total, int64_t N, int64_t K, int64_t G,
                                              void* workspace, size_t workspace_bytes, void* stream);
int dg_m_grouped_fp8_gemm_nt_masked_ue8m0(const uint8_t* A, const int32_t* sfa, const uint8_t* B,
                                          const int32_t* sfb, uint16_t* D, const int32_t* masked_m,
                                          int64_t G, int64_t max_m, int64_t N, int64_t K, int64_t expected_m,
                                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * Microscaled 4-bit floating point: e2m1 elements (magnitudes 0, 0.5, 1, 1.5,
 * 2, 3, 4, 6; sign in bit 3), two to a byte along K (the even element in the
 * lower nibble), with one power-of-two scale per 32 elements of a row, code c
 * meaning 2^(c - 127) and 255 meaning NaN.  The codes of the four blocks of 128
 * elements share one int32 (block 4 w + j in byte j), words MN-major:
 * [K/128][rows].  K is a positive multiple of 128.
 *
 * dg_quant_mxfp4: rows of x (dtype DG_F32 or DG_BF16) to codes and scales.
 *   x  [G,R,K] (row_token null), or [T,K] gathered by token: row r of group g
 *      takes row row_token[g][r] of x; rows whose entry is outside [0, T) are
 *      not written
 *   q  [G,R,K/2] (written)      sf [G][K/128][R] int32 (written)
 * c is the least code with 6 * 2^(c - 127) >= amax of the block, clamped to
 * [0, 253]; a block of zeros gets 127; a block that holds a NaN or an infinity
 * gets 255 and zero elements.  Elements are x * 2^(127 - c), an exact scaling,
 * rounded to nearest, ties to the even mantissa, the sign of zero kept.
 * Bit-exact and deterministic.  T is ignored when row_token is null.
 * Limits: G <= 65535, R and K < 2^31, ceil(R / 4) * ceil(K / 512) < 2^24; x, q 16-byte
 * aligned, sf and row_token 4-byte aligned.
 *
 * dg_dequant_mxfp4: the values back, y [G,R,K] of `dtype` (exact in both, past
 * their range infinite; a block of code 255 gives NaN).
 */
int dg_quant_mxfp4(const void* x, int dtype, uint8_t* q, int32_t* sf, const int32_t* row_token, int64_t G,
                   int64_t T, int64_t R, int64_t K, void* stream);
int dg_dequant_mxfp4(const uint8_t* q, const int32_t* sf, void* y, int dtype, int64_t G, int64_t R, int64_t K,
                     void* stream);

/*
 * Products of microscaled 4-bit operands, D = A . B^T in bf16: dense,
 * M-grouped contiguous and M-grouped masked, with the operands, index arrays,
 * undefined rows and rules of the FP8 forms of the same names, except
 *   A [rows,K/2], B [(G,)N,K/2] packed e2m1
 *   sfa [K/128][rows] int32, sfb [(G)][K/128][N] int32 (masked sfa
 *   [G][K/128][max_m]): both operands scaled per row and 32 elements
 * The matrix cores apply the scales; sums are fp32, rounded once to bf16.
 * A row or column with a NaN code (255) gives NaN.  K is a positive multiple
 * of 128 up to 2^24, N of 16, and (K / 128 + 8) words of 4 bytes for each row of
 * one operand (masked: of one expert) take less than 4 GiB; codes and outputs
 * are addressed in 64 bits.  Plans of about 2^23 tiles (of 64 x 64 or 128 x 256)
 * and more are refused.  Sums that fit 24 bits are exact.  Deterministic.
 * workspace (dense only): as for dg_fp8_gemm_nt: optional, zero-filled before
 * its first use and left reusable, full size
 * dg_get_workspace_size(DG_OP_MXFP4_GEMM_NT, M, N, K, 1).
 */
int dg_mxfp4_gemm_nt(const uint8_t* A, const int32_t* sfa, const uint8_t* B, const int32_t* sfb, uint16_t* D,
                     int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes, void* stream);
int dg_m_grouped_mxfp4_gemm_nt_contiguous(const uint8_t* A, const int32_t* sfa, const uint8_t* B,
                                          const int32_t* sfb, uint16_t* D, const int32_t* m_indices,
                                          int64_t M_total, int64_t N, int64_t K, int64_t G, void* workspace,
                                          size_t workspace_bytes, void* stream);
int dg_m_grouped_mxfp4_gemm_nt_masked(const uint8_t* A, const int32_t* sfa, const uint8_t* B, const int32_t* sfb,
                                      uint16_t* D, const int32_t* masked_m, int64_t G, int64_t max_m, int64_t N,
                                      int64_t K, int64_t expected_m, void* workspace, size_t workspace_bytes,
                                      void* stream);

/*
 * Router: the k experts of each token, their weights, the experts' loads and
 * the balance loss.
 *   logits   [T,E] of `dtype` (DG_F32 or DG_BF16), E in [1, 1024], k in [1, min(E, 16)]
 *   valid    [T] bytes or NULL: tokens with 0 (padding) take no part
 *   topk_idx [T,k] int32 (written): experts of the k largest logits, largest
 *            first, of equal ones the lower expert first; -inf and NaN are
 *            never chosen; -1 where nothing is left to choose
 *   topk_w   [T,k] fp32 (written): with p = softmax(logits of the row),
 *            w_scale * p_j / (sum of the chosen p) if renorm, else w_scale * p_j;
 *            0 where topk_idx is -1 (NaN in a row whose probabilities are NaN)
 *   counts   [E+1] int32 (written): choices c_e of each expert, then the number n
 *            of tokens with a choice
 *   prob_sum [E] fp32 (written): P_e = sum of p_te over the tokens
 *   loss     [1] fp32 (written): loss_coef * E / (C n) * sum_e c_e P_e, C = sum_e c_e
 *            (0 when nothing is routed)
 * A masked token, or one whose logits are all -inf, has no expert and enters
 * no sum.  A row with a NaN or +inf has NaN probabilities: its weights, prob_sum
 * and the loss are NaN, its experts are still distinct and in range.
 * workspace: required, dg_get_workspace_size(DG_OP_MOE_GATE, T, E, k, 1) bytes
 * (which also serve fewer tokens of as many experts), zero-filled before its first use and left reusable, by the other operators
 * too: the first 4 KiB of any operator's workspace are counters, zero between
 * calls.  Calls that share one must be ordered on one stream.  Deterministic.
 *
 * dg_moe_gate_bwd: dlogits [T,E] (of `dtype`, written) = gradient of
 * sum(dw * topk_w) + dloss * loss, the counts being constants.  topk_idx,
 * topk_w, counts are dg_moe_gate's; dw [T,k] fp32 or NULL (zeros); dloss [1]
 * fp32 on the device or NULL (zero).  Rows without an expert get zeros.
 */
int dg_moe_gate(const void* logits, int dtype, const uint8_t* valid, int32_t* topk_idx, float* topk_w,
                int32_t* counts, float* prob_sum, float* loss, int64_t T, int64_t E, int64_t k, int renorm,
                float w_scale, float loss_coef, void* workspace, size_t workspace_bytes, void* stream);
int dg_moe_gate_bwd(const void* logits, int dtype, const int32_t* topk_idx, const float* topk_w,
                    const int32_t* counts, const float* dw, const float* dloss, void* dlogits, int64_t T,
                    int64_t E, int64_t k, int renorm, float w_scale, float loss_coef, void* stream);

/*
 * Row order of the grouped products from the chosen experts.  topk_idx [T,k]
 * holds experts; expert first_expert + g is group g of [0, G) here, other
 * entries (another GPU's experts, -1) are skipped.  A group's choices take its
 * rows in (token, choice) order.
 *   contiguous: group g's rows start at a multiple of 128, groups in order.
 *     counts    [G] int32 (written): all of the group's choices, also those
 *               that got no row
 *     m_indices [M_total] int32 (written): group of each row, -1 on padding
 *     row_token [M_total] int32 (written): token of each row, -1 on padding
 *     row_of    [T,k] int32 (written): row of each choice, -1 if it has none
 *     M_total = T k + 127 G rounded up to 128 always suffices; choices past
 *     M_total get no row.
 *   masked: group g's rows are [g max_m, g max_m + masked_m[g]); choices past
 *     max_m get no row.
 *     masked_m [G] int32 (written): the rows taken, at most max_m;
 *     row_token [G,max_m], row_of [T,k] as above.
 * k in [1, 16], G in [1, 1024], T k + 128 G < 2^31.  workspace: required,
 * dg_get_workspace_size(DG_OP_MOE_LAYOUT, T, 0, k, G) bytes, which also serve
 * fewer tokens, choices and groups; it need not be zero, and its first 4 KiB are left as they are, so it may be one that other
 * operators use, in calls ordered on one stream.  Deterministic.
 */
int dg_moe_layout_contiguous(const int32_t* topk_idx, int32_t* counts, int32_t* m_indices, int32_t* row_token,
                             int32_t* row_of, int64_t T, int64_t k, int64_t first_expert, int64_t G,
                             int64_t M_total, void* workspace, size_t workspace_bytes, void* stream);
int dg_moe_layout_masked(const int32_t* topk_idx, int32_t* masked_m, int32_t* row_token, int32_t* row_of,
                         int64_t T, int64_t k, int64_t first_expert, int64_t G, int64_t max_m, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * Expert rows back to tokens: y[t] = sum_j w[t,j] rows[row_of[t,j]] over the
 * choices with a row in [0, R), summed in fp32 in the order of the choices.
 *   rows [R,N] bf16   row_of [T,k] int32   w [T,k] fp32   y [T,N] of `dtype` (written)
 * dg_moe_combine_bwd: drows [R,N] bf16: drows[row_of[t,j]] = w[t,j] dy[t] (rows
 * of no choice are not written; a row belongs to one choice at most), and
 * dw [T,k] fp32 (written): the dot product of rows[row_of[t,j]] and dy[t], 0
 * without a row.  dy [T,N] of `dtype`.  N is a multiple of 16.  Deterministic.
 */
int dg_moe_combine(const uint16_t* rows, const int32_t* row_of, const float* w, void* y, int dtype, int64_t T,
                   int64_t k, int64_t N, int64_t R, void* stream);
int dg_moe_combine_bwd(const void* dy, int dtype, const uint16_t* rows, const int32_t* row_of, const float* w,
                       uint16_t* drows, float* dw, int64_t T, int64_t k, int64_t N, int64_t R, void* stream);

/*
 * The experts of a mixture-of-experts layer for a few tokens, in two kernels:
 *   y[t] = sum_j topk_w[t,j] W2_e (silu(W1g_e x[t]) * (W1u_e x[t])),  e = topk_idx[t,j] - first_expert in [0, G)
 * (other choices, -1 among them, add nothing; a token without one gets zeros).
 *   x [T,H] bf16            topk_idx [T,k] int32, topk_w [T,k] fp32 (as from dg_moe_gate)
 *   y [T,H] bf16 (written); may equal x
 *   w1 [G,2 I,H]: rows [0, I) the gate projection, [I, 2 I) the up projection;  w2 [G,H,I]
 *   fp8:   e4m3, s1 [G][2 I / 128][H/128] and s2 [G][H / 128][I/128] fp32 (dg_quant_128x128)
 *   mxfp4: packed e2m1 ([G,2 I,H/2] and [G,H,I/2] bytes), s1 [G][H/128][2 I] and s2 [G][I/128][H] int32 (dg_quant_mxfp4)
 * Activations stay bf16: the weights are widened exactly, products are summed in
 * fp32, the inner activations are rounded to bf16 once and y once; a token's
 * experts are added in the order of their numbers (an e2m1 element past bf16's range, scale
 * codes 253 and above, is infinite).  A choice named twice counts twice.  A NaN or infinity
 * of a token, a weight or an expert stays with the tokens that chose it.
 * T in [0, 64], k in [1, 16], G in [1, 1024], H and I multiples of 128 up to
 * 32768.  workspace: required, dg_get_workspace_size(DG_OP_MOE_EXPERTS, T k, H,
 * I, 1) bytes, which also serve fewer tokens and choices; as for
 * dg_fp8_gemm_nt it is zero-filled before its first use and left reusable, by
 * the other operators too, in calls ordered on one stream.  Deterministic.
 */
int dg_moe_experts_fp8(const uint16_t* x, const int32_t* topk_idx, const float* topk_w, const uint8_t* w1, const float* s1,
                       const uint8_t* w2, const float* s2, uint16_t* y, int64_t T, int64_t k, int64_t first_expert, int64_t G,
                       int64_t H, int64_t I, void* workspace, size_t workspace_bytes, void* stream);
int dg_moe_experts_mxfp4(const uint16_t* x, const int32_t* topk_idx, const float* topk_w, const uint8_t* w1, const int32_t* s1,
                         const uint8_t* w2, const int32_t* s2, uint16_t* y, int64_t T, int64_t k, int64_t first_expert, int64_t G,
                         int64_t H, int64_t I, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes that let `op` use its full K split for this shape with the
 * current CU cap (0 = none used); a call split into row chunks reuses it for
 * every chunk. */
size_t dg_get_workspace_size(int op, int64_t rows, int64_t N, int64_t K, int64_t G);

/* Text description of the launch plan the library would use for `op` at this
 * shape on the current device with a full workspace, e.g. "kernel=wide
 * tile=256x256 grid=256 tiles=448 whole=448 tail=0x1" (DG_OP_GEMM_NT,
 * DG_OP_GEMM_NT_UE8M0, DG_OP_BF16_GEMM_NT, DG_OP_CONTIGUOUS with rows = M_total
 * and G the expert count, DG_OP_K_GROUPED with rows = M, G the group count
 * and K the total K, and DG_OP_MASKED with rows = max_m and G the expert
 * count, whose task count depends on masked_m and is given as its maximum;
 * "" for invalid shapes); for a call split into row chunks it describes the
 * first chunk and ends in "chunks=n".  "weights=nt" marks plans whose weight
 * loads carry the non-temporal cache policy (each weight line read by one
 * workgroup: dense calls with M <= 64, masked calls with max_m <= 128).
 * The pointer stays valid until the next call on the same thread.
 * Debugging aids, read from the environment on every call:
 *   DG_FORCE_CONFIG   comma-separated; "kernel=wide" / "kernel=persistent"
 *                     force the 256x256 or the 256x128 (128x256 grouped) tile
 *                     kernel wherever the planner chooses between them, and
 *                     "chunk_rows=<n>" splits calls into row chunks of at
 *                     most n rows (rounded down to a multiple of 256, at
 *                     least 256), and "skinny=<bm>x<wn>x<s>x<p>" makes calls
 *                     with at most 2048 rows use bm-row tiles (64 or 128) of
 *                     4 wn columns (wn 16 or 32), a K split of s (bounded by
 *                     the K blocks and the workspace) and ring depth p (one
 *                     of the compiled depths; other values are ignored,
 *                     and the epilogue form keeps the tile's default);
 *                     "mxfp4=<bm>x<bn>[x<s>]" makes the microscaled 4-bit
 *                     products use tiles of that shape (64x64, 128x256 or
 *                     256x256) where their form has it, 64x64 tiles with a
 *                     K split of s; results stay within the same bounds
 *   DG_PRINT_CONFIGS  print every launch's plan on stderr
 *   DG_CHECK_LAYOUT   the contiguous forms copy m_indices to the host
 *                     (synchronising the stream; skipped while the stream is
 *                     being captured) and reject, with DG_ERR_INVALID_ARG, a
 *                     layout whose aligned 128-row block holds rows of two
 *                     experts */
const char* dg_describe_plan(int op, int64_t rows, int64_t N, int64_t K, int64_t G);

/* Row alignment of expert segments in the contiguous layout (deep-dive blog,
 * section 3: contiguous segments aligned to the M block).  Always 128. */
int dg_get_m_alignment_for_contiguous_layout(void);

/* Cap on the number of compute units the kernels plan for (analog of the
 * "set max SM count" utility in the Feb-2025 release article).  n <= 0 resets
 * to the device's count.  Process-wide; returns DG_OK. */
int dg_set_num_cus(int n);
/* Current cap (the device's CU count when no cap is set; 0 if no device). */
int dg_get_num_cus(void);

/* Message of the last error on this thread ("" if none). */
const char* dg_get_last_error(void);
/* Library version string. */
const char* dg_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DG_H */
