/*
 * swiglu_gemm.h -- C ABI of the MI355X (gfx950) GEMM / fused SwiGLU-GEMM library
 * (libswiglu_gemm.so).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All matrix pointers are DEVICE pointers owned by the caller; the library keeps
 *   no pointer after the enqueued work has finished.  Matrices are row-major with
 *   a leading dimension (the distance, in elements, between the starts of two
 *   consecutive stored rows).
 * - `stream` is a hipStream_t passed as void* (NULL = the default stream).  Every
 *   call is asynchronous: it enqueues kernels on `stream` and returns without
 *   synchronising.
 * - Return value: 0 on success; -i when argument i (1-based) is invalid, checked
 *   before any HIP call; a positive hipError_t when a HIP call failed.  Nothing is
 *   printed and nothing aborts.
 * - Output buffers must not overlap input buffers.
 * - dtype codes: SG_F32 = 0, SG_F16 = 1, SG_BF16 = 2, SG_F8E4M3 = 3 (OCP e4m3fn:
 *   bias 7, largest magnitude 448, no infinities).  Every product is accumulated
 *   in fp32 and rounded to the output type (nearest-even) once, at the end.
 * - Split-K workspace (fp32 partial sums) is owned by the library: one buffer per
 *   device, grown on first need (to a power of two, at least 1 MiB), released by
 *   sg_release().  A call fetches it once and passes that address to each of its
 *   kernels.  Growth never synchronises the device: the smaller buffer, which work
 *   enqueued earlier may still read, is kept until sg_release().  Calls that need
 *   the workspace and run concurrently on different streams of one device are
 *   serialised by the caller (the library does not order streams).
 * - Problems with 1..32 rows of A ('N') may run on the decode kernels: a persistent
 *   stream-K pass over the weight and, when a column tile is shared by several
 *   work-groups, a second fix-up launch that adds their partial sums (a fixed
 *   order: results are run-to-run identical).  Its partial sums live in the same
 *   kind of library-owned workspace, with the same rule for concurrent streams.
 */
#ifndef SWIGLU_GEMM_H
#define SWIGLU_GEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SG_F32 = 0,
    SG_F16 = 1,
    SG_BF16 = 2,
    SG_F8E4M3 = 3
} sg_dtype;

/*
 * sg_gemm: C = alpha * op(A) * op(B) + beta * C_old.
 *
 * The BLAS update of "GEMM o Coração Matemático" §1 (op is the identity or the
 * transpose; alpha and beta scalars), row-major as in its §2.
 *
 *  1 transA  'N'/'n': op(A) = A, A stored M x K (lda >= max(1,K));
 *            'T'/'t': op(A) = A^T, A stored K x M (lda >= max(1,M)).
 *  2 transB  'N'/'n': op(B) = B, B stored K x N (ldb >= max(1,N));
 *            'T'/'t': op(B) = B^T, B stored N x K (ldb >= max(1,K)).
 *  3 M, 4 N, 5 K   sizes of op(A) (M x K), op(B) (K x N) and C (M x N); >= 0.
 *  6 alpha   fp32 scalar.
 *  7 A, 8 lda, 9 B, 10 ldb   operands (see above).
 *  11 beta   fp32 scalar.  beta == 0: C is write-only (C_old is never read, so
 *            NaN/Inf there cannot propagate).
 *  12 C, 13 ldc   M x N output, ldc >= max(1,N).  Elements outside the logical
 *            M x N block (the ld padding) are never written.
 *  14 dtype  SG_F32: A, B, C fp32.  SG_F16 / SG_BF16: A, B, C in that type.
 *            SG_F8E4M3: A, B e4m3 codes, C bf16; per-tensor scales are folded
 *            into alpha by the caller (alpha = s_A * s_B * alpha').
 *  15 stream hipStream_t (void*).
 * Quick returns: M == 0 or N == 0 does nothing; K == 0 or alpha == 0 computes
 * C = beta * C_old without reading A or B.
 * Alignment: any element-aligned pointers and leading dimensions are accepted.
 * For fp16, bf16 and e4m3 the direct-to-LDS kernels run when A and B are 16-byte
 * aligned and lda, ldb times the element size are multiples of 16 (any M, N, K);
 * other fp16 / bf16 problems run on a register-staged kernel, other e4m3 problems
 * on a kernel with one thread per output.
 * Invalid: trans flag (-1/-2), negative size (-3/-4/-5), NULL A/B when they are
 * read (-7/-9), ld too small (-8/-10/-13), NULL C (-12), unknown dtype (-14).
 */
int sg_gemm(char transA, char transB, int64_t M, int64_t N, int64_t K,
            float alpha, const void* A, int64_t lda, const void* B, int64_t ldb,
            float beta, void* C, int64_t ldc, int dtype, void* stream);

/* Activations of the GEMM epilogue (sg_epilogue.activation). */
typedef enum {
    SG_ACT_NONE = 0,
    SG_ACT_RELU = 1,      /* max(x, 0) */
    SG_ACT_GELU = 2,      /* x * Phi(x) = x/2 * (1 + erf(x / sqrt 2)) */
    SG_ACT_GELU_TANH = 3, /* x/2 * (1 + tanh(sqrt(2/pi) * (x + 0.044715 x^3))) */
    SG_ACT_SILU = 4       /* x / (1 + e^-x) */
} sg_activation;

/* Extra steps of the GEMM epilogue, applied before the single store. */
typedef struct {
    const void* bias;   /* NULL, or N values (device memory), one per column of C */
    int bias_dtype;     /* SG_F32, SG_F16 or SG_BF16 (ignored when bias is NULL) */
    int activation;     /* sg_activation, applied after the bias */
    int out_dtype;      /* -1: C has sg_gemm's output type; SG_F8E4M3: C holds e4m3 codes */
    float out_scale;    /* SG_F8E4M3 output: per-tensor scale s_C > 0 (finite; its fp32
                           reciprocal must be finite too) */
} sg_epilogue;

/*
 * sg_gemm_noalloc: sg_gemm for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid hipMalloc).
 *
 * Arguments, semantics, kernels and results are those of sg_gemm (bit-identical
 * output for the same problem, with one exception below).  The split-K partial
 * sums, the decode path's partial sums and the 16-byte-row copies of e4m3 operands
 * whose rows are not 16-byte multiples, which sg_gemm keeps in library-allocated
 * workspace, live here in a fixed device array of SG_NOALLOC_SCRATCH_BYTES built
 * into the library: every GPU the library runs on holds one copy until the process
 * ends.  No call allocates or frees device memory (its device address is looked up
 * once per device, on the first call there).
 * - A problem whose chosen kernels need more scratch than that returns
 *   SG_STATUS_SCRATCH_LIMIT before enqueuing anything (C is untouched).
 * - The exception: e4m3 operands whose copies would not fit run the one-thread-
 *   per-output kernel instead of the tile kernels (same tolerance, different
 *   summation order, so not the same bits as sg_gemm).
 * - Every call on one GPU shares that GPU's array, which keeps the last call's
 *   contents; nothing in it needs to start at zero (each partial sum is written
 *   before it is read).  Calls that overlap in time on one GPU (different streams,
 *   or host threads enqueuing concurrently) race on it: order them.
 */
#define SG_NOALLOC_SCRATCH_BYTES (32u << 20)
#define SG_STATUS_SCRATCH_LIMIT (-100)
int sg_gemm_noalloc(char transA, char transB, int64_t M, int64_t N, int64_t K, float alpha,
                    const void* A, int64_t lda, const void* B, int64_t ldb, float beta, void* C,
                    int64_t ldc, int dtype, void* stream);

/*
 * sg_gemm_ex: sg_gemm with the steps a fused GEMM epilogue folds in before the
 * accumulator is stored ("GEMM o Coração Matemático" §1, closing paragraph, and
 * §13.3, closing paragraph: bias and activations in the epilogue; "为什么 GEMM 是
 * CUDA 的必修课", list of optimisations, epilogue fusion of bias, activation,
 * scale and quantisation):
 *     v = alpha * op(A) * op(B) + beta * C_old
 *     y = act(v + bias[n])
 *     C[m, n] = y rounded once to the output type, or, with out_dtype SG_F8E4M3,
 *               the OCP e4m3fn code of y * r, r = 1/out_scale rounded to fp32
 *               (round to nearest, ties to even, saturating at +-448, NaN to 0x7F;
 *               the per-tensor scale of §12.4; exact division for power-of-two
 *               scales).
 * Attention scores QK^T / sqrt(d_h) are the plain call with transB = 'T' and
 * alpha = 1/sqrt(d_h) (§1); the fused Q, K, V projection is one call on the
 * concatenated weight [W_Q W_K W_V] (N = 3d, §13.1).
 *
 * Arguments 1-14 and 16 as sg_gemm (15 there is the stream):
 *  15 epi    NULL or the steps above; NULL, or no bias, SG_ACT_NONE and
 *            out_dtype -1, is exactly sg_gemm.
 *  16 stream hipStream_t (void*).
 * With an e4m3 output C is M x N bytes (ldc in elements = bytes) and beta must
 * be 0.  Quick returns as sg_gemm: K == 0 or alpha == 0 gives
 * C = out(act(beta * C_old + bias)).
 * Invalid: as sg_gemm; beta != 0 with an e4m3 output (-11); an unknown
 * activation, bias dtype or out_dtype, or out_scale not finite and > 0 (-15).
 */
int sg_gemm_ex(char transA, char transB, int64_t M, int64_t N, int64_t K, float alpha,
               const void* A, int64_t lda, const void* B, int64_t ldb, float beta, void* C,
               int64_t ldc, int dtype, const sg_epilogue* epi, void* stream);

/*
 * sg_gemm_strided_batched: for b in [0, batch): C_b = alpha * op(A_b) * op(B_b)
 * + beta * C_b, with X_b = X + b * strideX elements -- the same BLAS update as
 * sg_gemm ("GEMM o Coração Matemático" §1, §2) over a batch of equally shaped
 * problems in one launch: the batched products of the same page's §13.2, where
 * attention's score and context steps are one GEMM per (sequence, head).
 *
 * Arguments 1-8 and 10, 11, 13-15, 18, 19 as sg_gemm (transA, transB, M, N, K,
 * alpha, A, lda, B, ldb, beta, C, ldc, dtype, stream); 9 strideA, 12 strideB,
 * 16 strideC: element distance between consecutive problems (>= 0; 0 repeats
 * the operand for every problem; strideC must keep the outputs disjoint:
 * >= (M-1)*ldc + N when batch > 1); 17 batch: number of problems, 0..65535.
 * Split-K is not used inside a batch.  Quick returns as sg_gemm, per problem;
 * batch == 0 does nothing.
 * Invalid: as sg_gemm at the shifted positions (-1..-5, -7, -8, -10, -11, -14,
 * -15, -18), negative stride (-9/-12), overlapping outputs (-16), batch (-17).
 */
int sg_gemm_strided_batched(char transA, char transB, int64_t M, int64_t N, int64_t K,
                            float alpha, const void* A, int64_t lda, int64_t strideA,
                            const void* B, int64_t ldb, int64_t strideB, float beta, void* C,
                            int64_t ldc, int64_t strideC, int64_t batch, int dtype,
                            void* stream);

/*
 * sg_swiglu_gemm: Y = SiLU(s * A * W1) ⊙ (s * A * W2), s = scale_a * scale_w.
 *
 * The gated MLP of "Resumo Técnico: Sobreposição de Ativação em Nível de Tile para
 * Inferência Eficiente de LLM" (Definição do Problema), computed as ONE GEMM over
 * [M, 2N, K] on the column-interleaved W_fused of its Metodologia / Kernel-2 (even
 * columns gate = W1, odd columns up = W2); the epilogue pairs columns (2n, 2n+1)
 * in registers, so the gate and up intermediates never reach memory.
 * SiLU(x) = x / (1 + e^-x).  The scales are the per-tensor dequantisation factors
 * (value = s * code, zero point 0) of "GEMM o Coração Matemático" §12.4, applied
 * to the fp32 sums before SiLU.
 *
 *  1 A       M x K, contiguous (ld = K).
 *  2 Wfused  K x 2N, contiguous (ld = 2N).
 *  3 Y       M x N, contiguous (ld = N).
 *  4 M, 5 N, 6 K   >= 0.
 *  7 dtype   SG_BF16: A, W bf16, Y bf16.  SG_F16: A, W fp16, Y fp16.
 *            SG_F8E4M3: A, W e4m3 codes, Y bf16.
 *  8 scale_a, 9 scale_w   fp32 per-tensor scales; finite and > 0; must be 1.0
 *            unless dtype is SG_F8E4M3.
 *  10 stream hipStream_t (void*).
 * Quick returns: M == 0 or N == 0 does nothing; K == 0 writes Y = 0.
 * Invalid: NULL pointer (-1/-2/-3), negative size (-4/-5/-6), unsupported dtype
 * (-7), bad scale (-8/-9).
 */
int sg_swiglu_gemm(const void* A, const void* Wfused, void* Y,
                   int64_t M, int64_t N, int64_t K, int dtype,
                   float scale_a, float scale_w, void* stream);

/*
 * sg_swiglu_gemm_w12: the same Y = SiLU(s * A * W1) ⊙ (s * A * W2) from separate,
 * non-interleaved W1 and W2 -- the weight layout of Kernel-1 in "Resumo Técnico:
 * Sobreposição de Ativação em Nível de Tile para Inferência Eficiente de LLM"
 * (Metodologia).  One work-group tile loads BN/2 columns of W1 and the same BN/2
 * columns of W2 side by side, so gate and up of every output still meet in
 * registers and never reach memory.  Results equal sg_swiglu_gemm on the
 * interleaved W_fused to the same tolerance (and, for the same tile configuration,
 * bit for bit).
 *
 *  1 A       M x K, contiguous (ld = K).
 *  2 W1, 3 W2   K x N each, contiguous (ld = N).
 *  4 Y       M x N, contiguous (ld = N).
 *  5 M, 6 N, 7 K   >= 0.
 *  8 dtype   as sg_swiglu_gemm.   9 scale_a, 10 scale_w   as sg_swiglu_gemm.
 *  11 stream hipStream_t (void*).
 * Shapes the direct kernel cannot take (rows of A, W1 or W2 that are not 16-byte
 * multiples, unaligned pointers) are run by interleaving W1, W2 into a
 * library-owned buffer (grown on demand, freed by sg_release) and calling
 * sg_swiglu_gemm; calls on several streams of one device must not overlap then.
 * Quick returns: M == 0 or N == 0 does nothing; K == 0 writes Y = 0.
 * Invalid: NULL pointer (-1/-2/-3/-4), negative size (-5/-6/-7), unsupported dtype
 * (-8), bad scale (-9/-10).
 */
int sg_swiglu_gemm_w12(const void* A, const void* W1, const void* W2, void* Y,
                       int64_t M, int64_t N, int64_t K, int dtype,
                       float scale_a, float scale_w, void* stream);

/*
 * sg_interleave_gate_up: Wfused[k, 2n] = W1[k, n], Wfused[k, 2n+1] = W2[k, n]
 * (the W_fused layout of the same page's Kernel-2).  Bit-exact copy.
 *  1 W1, 2 W2   K x N contiguous; 3 Wfused  K x 2N contiguous;
 *  4 K, 5 N >= 0; 6 dtype any sg_dtype (element size 4, 2, 2 or 1 bytes);
 *  7 stream.
 * Invalid: NULL pointer (-1/-2/-3), negative size (-4/-5), unknown dtype (-6).
 */
int sg_interleave_gate_up(const void* W1, const void* W2, void* Wfused,
                          int64_t K, int64_t N, int dtype, void* stream);

/*
 * sg_silu_mul: Y = SiLU(G) ⊙ U, elementwise over M x N contiguous matrices (the
 * separate activation step of the unfused MLP that the same page's Definição do
 * Problema describes: two GEMMs write Gate and Up to memory, then this reads them).
 *  1 G, 2 U, 3 Y   M x N contiguous, dtype SG_BF16 or SG_F16 (all three);
 *  4 M, 5 N >= 0; 6 dtype; 7 stream.
 * Invalid: NULL pointer (-1/-2/-3), negative size (-4/-5), unsupported dtype (-6).
 */
int sg_silu_mul(const void* G, const void* U, void* Y, int64_t M, int64_t N,
                int dtype, void* stream);

/*
 * Products grouped by expert (mixture-of-experts MLPs)
 * ----------------------------------------------------
 * The M rows of A are sorted by expert: expert e owns rows offsets[e] .. offsets[e+1]-1,
 * R_e for short.  `offsets` is DEVICE memory, experts + 1 ascending int32 row numbers in
 * [0, M] (experts 1..65536); an expert may own no row.  Rows before offsets[0] and from
 * offsets[experts] on belong to no expert: they are neither read nor written, nor are gaps
 * between the experts' matrices.  What lies between the end of one row and the next, and
 * the rest of the 16-byte piece that holds a row's last element, may be loaded; it never
 * counts.  The host never reads the offsets, so a call can be captured into a HIP graph
 * and replayed with other offsets.  The kernels clamp each offset to [0, M]; a table that
 * does not ascend gives unspecified rows of the output (nothing outside it is written).
 * These calls allocate nothing and use no workspace: calls on different streams may
 * overlap.  Results are run-to-run identical.
 * Alignment: any element-aligned pointers and leading dimensions are accepted; 16-byte
 * aligned operands with rows and strides of 16-byte multiples run on the direct-to-LDS
 * tile kernels, others on a 64 x 64 tile kernel that loads element by element.
 * A problem of more than about 2^22 output tiles, or a 4-bit one whose 256 rows of codes
 * exceed 2^31 bytes, returns hipErrorInvalidConfiguration.  Matrices more than 2^44
 * elements apart are an invalid stride; the stride of a single matrix does not count.
 */

/*
 * sg_grouped_gemm: C[r] = alpha * scale[e] * A[r] * op(B_e) + beta * C_old[r] for r in R_e,
 * B_e = B + e * strideB elements.
 *  1 transB  'N': B_e stored K x N; 'T': B_e stored N x K (the input gradient of a
 *            product with B_e stored K' x N' is the 'T' call with N = K', K = N').
 *  2 experts, 3 offsets   see above.
 *  4 M, 5 N, 6 K   >= 0; M: rows of A and C in all.
 *  7 alpha   fp32 scalar.   8 scale   NULL, or `experts` fp32 factors (device memory).
 *  9 A, 10 lda   M x K.   11 B, 12 ldb, 13 strideB (>= 0; 0: one weight for all).
 *  14 beta   fp32 scalar; 0: C is write-only.   15 C, 16 ldc   M x N.
 *  17 dtype  SG_F16, SG_BF16 (A, B, C), or SG_F8E4M3 (A, B; C bf16).
 *  18 stream.
 * Quick returns: M == 0 or N == 0 does nothing; K == 0 or alpha == 0 computes
 * C = beta * C_old in the experts' rows.
 * Invalid: -i for argument i as in sg_gemm (NULL operands that are read, leading
 * dimensions too small, negative sizes or strides, unsupported dtype).
 */
int sg_grouped_gemm(char transB, int64_t experts, const int32_t* offsets, int64_t M, int64_t N,
                    int64_t K, float alpha, const float* scale, const void* A, int64_t lda,
                    const void* B, int64_t ldb, int64_t strideB, float beta, void* C,
                    int64_t ldc, int dtype, void* stream);

/*
 * sg_grouped_gemm_wgrad: C_e = alpha * A[R_e]^T * D[R_e] + beta * C_e (K x N), the weight
 * gradient of the product above with D the gradient of its output.  An expert without
 * rows gets beta * C_e (zeros for beta == 0).
 *  1 experts, 2 offsets   see above.   3 M, 4 N, 5 K   >= 0.   6 alpha   fp32 scalar.
 *  7 A, 8 lda   M x K.   9 D, 10 ldd   M x N.   11 beta   fp32 scalar; 0: C write-only.
 *  12 C, 13 ldc, 14 strideC   C_e = C + e * strideC elements; strideC >= (K-1)*ldc + N.
 *  15 dtype  of A and D: SG_F16 or SG_BF16.   16 c_dtype   dtype or SG_F32.
 *  17 stream.
 * Quick returns: N == 0 or K == 0 does nothing; M == 0 or alpha == 0 computes
 * C_e = beta * C_e (alpha does not count where there are no products).
 */
int sg_grouped_gemm_wgrad(int64_t experts, const int32_t* offsets, int64_t M, int64_t N,
                          int64_t K, float alpha, const void* A, int64_t lda, const void* D,
                          int64_t ldd, float beta, void* C, int64_t ldc, int64_t strideC,
                          int dtype, int c_dtype, void* stream);

/*
 * sg_grouped_swiglu_gemm: Y[r] = SiLU(s_e * g) ⊙ (s_e * u), (g, u) = A[r] * (W1_e, W2_e),
 * s_e = alpha * scale[e], from the column-interleaved W_fused of sg_swiglu_gemm for each
 * expert.
 *  1 experts, 2 offsets   see above.
 *  3 A  M x K, 4 Wfused  experts x K x 2N, 5 Y  M x N; contiguous.
 *  6 M, 7 N, 8 K   >= 0.
 *  9 dtype   SG_F16, SG_BF16 (all three), or SG_F8E4M3 (A, W codes; Y bf16).
 *  10 alpha  fp32, finite and > 0; 1.0 unless dtype is SG_F8E4M3.
 *  11 scale  NULL, or `experts` fp32 factors (device memory; SG_F8E4M3 only).
 *  12 stream.
 * Quick returns: M == 0 or N == 0 does nothing; K == 0 writes Y = 0 in the experts' rows.
 */
int sg_grouped_swiglu_gemm(int64_t experts, const int32_t* offsets, const void* A,
                           const void* Wfused, void* Y, int64_t M, int64_t N, int64_t K,
                           int dtype, float alpha, const float* scale, void* stream);

/*
 * sg_grouped_swiglu_gemm_bwd: dH (M x 2N), the gradient of the gate and up products from
 * the gradient dY (M x N) of Y.  The products are computed again from A and Wfused, so the
 * forward need not keep them.  With sig = 1 / (1 + e^-g):
 *     dH[r, 2n]   = dY * u * sig * (1 + g * (1 - sig))      dH[r, 2n+1] = dY * g * sig
 * in fp32, rounded once.  dA is then sg_grouped_gemm('T', dH, Wfused) and the gradient of
 * Wfused sg_grouped_gemm_wgrad(A, dH).
 *  1 experts, 2 offsets, 3 A, 4 Wfused   as the forward.   5 dY  M x N, 6 dH  M x 2N;
 *  contiguous.   7 M, 8 N, 9 K   >= 0.   10 dtype   SG_F16 or SG_BF16.   11 stream.
 */
int sg_grouped_swiglu_gemm_bwd(int64_t experts, const int32_t* offsets, const void* A,
                               const void* Wfused, const void* dY, void* dH, int64_t M,
                               int64_t N, int64_t K, int dtype, void* stream);

/*
 * Microscaled 4-bit floating point (OCP MX FP4)
 * ---------------------------------------------
 * A matrix of M rows and K columns is held as e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and
 * their negatives) in blocks of 32 along a row, each with one e8m0 scale 2^(s - 127)
 * (s == 255: every element of the block is NaN):
 *   codes   M rows of SG_MXFP4_ROW_BYTES(K) bytes; element 2i in the low half of byte i;
 *           the last block of a row is filled with zeros.
 *   scales  SG_MXFP4_SCALE_BYTES(M, K) bytes: tiles of 32 rows x 8 blocks, 256 bytes each,
 *           all tiles of 32 rows one after the other; the byte of row r, block b is at
 *           256*((r/32)*ceil(K/256) + b/8) + 128*((b/4)%2) + 4*(r%32) + b%4.
 *           Bytes of rows and blocks outside the matrix are not used.
 * A batch of matrices follows one another, each with its own codes and tiles of scales.
 * These calls allocate nothing and use no workspace.  A matrix of more than 2^22 tiles of
 * scales returns hipErrorInvalidConfiguration from the quantisation and its inverse.
 */
#define SG_MXFP4_ROW_BYTES(K) ((((int64_t)(K) + 31) / 32) * 16)
#define SG_MXFP4_SCALE_BYTES(M, K) \
    ((((int64_t)(M) + 31) / 32) * (((int64_t)(K) + 255) / 256) * 256)

/*
 * sg_mxfp4_quantize: codes and scales of X.  For each block, t = max |x|:
 * scale 2^(floor(log2 t) - 2), not below 2^-127 (t == 0: 2^-127); codes x / scale rounded
 * to the nearest e2m1 value, ties to the even code, saturating at +-6.  A block with an
 * infinity or a NaN gets scale 255 and zero codes.
 *  1 X, 2 ldx, 3 strideX   `batch` matrices M x K, strideX elements apart (>= 0).
 *  4 batch (0..65535), 5 M, 6 K   >= 0.   7 dtype   of X: SG_F32, SG_F16 or SG_BF16.
 *  8 codes, 9 scales   outputs, 4-byte aligned, or NULL.
 *  10 values   NULL, or the values the codes and scales stand for, batch x M x K
 *            contiguous, rounded to X's type (exact but for multiples of scales below
 *            2^-23 in fp16).
 *  11 stream.
 * Invalid: as above; codes, scales and values all NULL (-8).
 */
int sg_mxfp4_quantize(const void* X, int64_t ldx, int64_t strideX, int64_t batch, int64_t M,
                      int64_t K, int dtype, void* codes, void* scales, void* values,
                      void* stream);

/*
 * sg_mxfp4_dequantize: X = the values of codes and scales, rounded to X's type.
 *  1 codes (4-byte aligned), 2 scales, 3 batch, 4 M, 5 K, 6 X, 7 ldx, 8 strideX
 *  (>= (M-1)*ldx + K for more than one matrix), 9 dtype (SG_F32, SG_F16, SG_BF16), 10 stream.
 */
int sg_mxfp4_dequantize(const void* codes, const void* scales, int64_t batch, int64_t M,
                        int64_t K, void* X, int64_t ldx, int64_t strideX, int dtype,
                        void* stream);

/*
 * sg_mxfp4_tile_scales: scales stored as rows of bytes (`batch` matrices M x blocks, rows
 * ld, matrices `stride` bytes apart) to the tiles above; padding becomes 0.
 *  1 src, 2 ld, 3 stride, 4 batch, 5 M, 6 blocks, 7 dst (4-byte aligned), 8 stream.
 */
int sg_mxfp4_tile_scales(const void* src, int64_t ld, int64_t stride, int64_t batch, int64_t M,
                         int64_t blocks, void* dst, void* stream);

/*
 * sg_mxfp4_gemm: C = alpha * A * B^T, A (M x K) and B (N x K) held as above, fp32 sums; or,
 * with offsets, C[r] = alpha * A[r] * B_e^T for r in R_e, B a batch of `experts` matrices.
 *  1 experts, 2 offsets   as the grouped products; offsets NULL with experts 1: every row.
 *  3 M, 4 N, 5 K   >= 0.   6 alpha   fp32 scalar.
 *  7 A codes (16-byte aligned), 8 A scales (4), 9 B codes (16), 10 B scales (4).
 *  11 C, 12 ldc   M x N, written only.   13 dtype   of C: SG_F32, SG_F16 or SG_BF16.
 *  14 stream.
 * Quick returns: M == 0 or N == 0 does nothing; K == 0 or alpha == 0 writes zeros.
 */
int sg_mxfp4_gemm(int64_t experts, const int32_t* offsets, int64_t M, int64_t N, int64_t K,
                  float alpha, const void* A, const void* As, const void* B, const void* Bs,
                  void* C, int64_t ldc, int dtype, void* stream);

/*
 * sg_mxfp4_swiglu_gemm: Y = SiLU(A * W1^T) ⊙ (A * W2^T) from W of 2N rows, gate and up
 * interleaved (row 2n = W1's row n, row 2n+1 = W2's); offsets as sg_mxfp4_gemm.
 *  1 experts, 2 offsets, 3 M, 4 N, 5 K; 6 A codes, 7 A scales, 8 W codes, 9 W scales;
 *  10 Y  M x N contiguous; 11 dtype of Y: SG_F16 or SG_BF16; 12 stream.
 */
int sg_mxfp4_swiglu_gemm(int64_t experts, const int32_t* offsets, int64_t M, int64_t N,
                         int64_t K, const void* A, const void* As, const void* W,
                         const void* Ws, void* Y, int dtype, void* stream);

/*
 * Routing to experts
 * ------------------
 * What stands around the products grouped by expert: each token's experts and their weights
 * from the router's logits, the rows sorted by expert, and each token's rows to their places
 * and back.  A token's place (t, j), j < top_k, is its j-th expert; flat, place t * top_k + j.
 * These calls allocate nothing and use no workspace; results are run-to-run identical.
 * Any element-aligned pointers and leading dimensions are accepted.  No result may overlap an
 * input (sg_combine_rows: out may be the residual).  Calls that need 2^32 threads return
 * hipErrorInvalidConfiguration: more than 2^26 - 4 tokens of the router or its gradient, or places of
 * combining's gradient; rows (of spreading and combining) from 2^24 on of more than 1024 elements, shorter
 * ones in proportion.
 */
typedef enum { SG_ROUTE_SOFTMAX = 0, SG_ROUTE_SIGMOID = 1 } sg_route_scoring;
#define SG_ROUTE_MAX_EXPERTS 1024
#define SG_ROUTE_MAX_TOP_K 64

/*
 * sg_route_experts: for each row x of X, s = softmax(x) or s = 1 / (1 + e^-x), and
 *     ids = the top_k experts by c = s + bias, the largest first, of equal ones the lowest index
 *     weights = scale * s[id], with renormalize scale * s[id] / (sum of s over the chosen)
 * In groups (groups > 1) of experts / groups neighbours each, the experts come from the
 * top_groups groups whose group_top best c have the largest sum.  c is compared in 64 bits;
 * without bias the logits are, which order the experts as their scores do.  Weights are
 * computed in fp32 (renormalised ones from the chosen experts' log scores, so that they do
 * not underflow all together).
 * A logit of -infinity, or a bias of -infinity or NaN, keeps the expert from being chosen; where
 * fewer than top_k are left, the places behind get id -1 and weight 0.  NaN logits come behind every
 * number: their experts are chosen where the others run out, the lowest index first, and count in
 * their group only where it has no other.  The others' scores are those of the row without them;
 * logits of +infinity share softmax's whole.  The weights of the experts chosen in a row with a NaN
 * logit, or with softmax with +infinity, are NaN.
 *  1 X, 2 ldx   T x E logits.   3 T (0..2^30)   4 E (1..SG_ROUTE_MAX_EXPERTS)
 *  5 dtype   of X: SG_F32, SG_F16, SG_BF16.   6 top_k   1..min(E, SG_ROUTE_MAX_TOP_K).
 *  7 scoring   sg_route_scoring.   8 bias   NULL, or E fp32 values.
 *  9 groups   1..64, divides E.   10 top_groups   1..groups.   11 group_top   1 or 2.
 *  12 renormalize   0 or 1.   13 scale   fp32, finite.
 *  14 mask   NULL, or T bytes: where 0, the row is not read, its ids are -1, its weights 0.
 *  15 ids   T x top_k int32, contiguous.   16 weights   T x top_k fp32, contiguous.
 *  17 stream.
 */
int sg_route_experts(const void* X, int64_t ldx, int64_t T, int64_t E, int dtype, int64_t top_k,
                     int scoring, const float* bias, int64_t groups, int64_t top_groups,
                     int group_top, int renormalize, float scale, const uint8_t* mask,
                     int32_t* ids, float* weights, void* stream);

/*
 * sg_route_experts_bwd: dX from the gradient g of the weights, the choice held fixed.  With
 * p = weights / scale and G = scale * g:
 *     renormalised       dx[id] = p (G - sum G p), times (1 - s) for sigmoid; 0 elsewhere
 *     softmax            dx[e] = s_e * (G_e - sum G p), G_e = 0 where e is not chosen
 *     sigmoid            dx[id] = G s (1 - s); 0 elsewhere
 * in fp32, rounded once.  Ids outside 0..E-1 are empty places; a row of empty places gets
 * zeros and is not read.  Renormalised and sigmoid gradients read the chosen logits alone: a NaN
 * elsewhere in the row does not show in them.
 *  1 X, 2 ldx, 3 T, 4 E, 5 dtype, 6 top_k, 7 scoring   as the forward.   8 renormalize
 *  9 scale   10 ids, 11 dweights   T x top_k.   12 dX, 13 lddx   T x E of X's type.  14 stream.
 */
int sg_route_experts_bwd(const void* X, int64_t ldx, int64_t T, int64_t E, int dtype,
                         int64_t top_k, int scoring, int renormalize, float scale,
                         const int32_t* ids, const float* dweights, void* dX, int64_t lddx,
                         void* stream);

/*
 * sg_sort_experts: the places 0..n-1 sorted by their expert, stably:
 *     offsets[e]   places of experts below e (experts + 1 of them: the grouped products' table)
 *     order[r]     the place that is row r, -1 from offsets[experts] on
 *     place[i]     the row of place i (order[place[i]] == i), -1 where ids[i] is outside
 *                  0..experts-1
 * Every expert's work-groups read all ids, `parts` of them to count and all of them together once
 * more to write: 4 n * (experts + 1) * (parts + 1) bytes from the caches at most, where parts is 1
 * below 16384 ids and else as many, 1 to 8, as leave 256 work-groups in all.  65536 ids of 64 experts
 * are 68 MB and take 9.4 us, 131072 of 256 experts 21 us, 2^20 of 5000 experts 1.35 ms.
 *  1 ids, 2 n (0..2^30)   3 experts (1..65536)   4 offsets, 5 order, 6 place (order or place
 *  may be NULL)   7 stream.
 */
int sg_sort_experts(const int32_t* ids, int64_t n, int64_t experts, int32_t* offsets,
                    int32_t* order, int32_t* place, void* stream);

/*
 * sg_spread_rows: Y[place[t, j]] = X[t], or weights[t, j] * X[t] (fp32, rounded once).  Places
 * outside 0..M-1 are empty; rows of Y that no place names stay as they are.  Its gradient is
 * sg_combine_rows of Y's gradient.
 *  1 X, 2 ldx   T x D.   3 T, 4 D   >= 0.   5 dtype   SG_F32, SG_F16 or SG_BF16.
 *  6 place   T x top_k, no two places of one row (or either's values).   7 top_k (1..65536)
 *  8 weights   NULL, or T x top_k fp32.   9 M   rows of Y.   10 Y, 11 ldy.   12 stream.
 */
int sg_spread_rows(const void* X, int64_t ldx, int64_t T, int64_t D, int dtype,
                   const int32_t* place, int64_t top_k, const float* weights, int64_t M, void* Y,
                   int64_t ldy, void* stream);

/*
 * sg_combine_rows: out[t] = residual[t] + sum over j of weights[t, j] * Z[place[t, j]], summed
 * in fp32 in the order of j, rounded once.  Places outside 0..M-1 are left out (their weights
 * do not count); a token without a place gets its residual, or zeros.
 *  1 Z, 2 ldz   M x D.   3 M, 4 D, 5 T   >= 0.   6 dtype   of Z, residual and out.
 *  7 place, 8 top_k, 9 weights   as sg_spread_rows; weights NULL: 1.
 *  10 residual (NULL: none), 11 ldr   T x D.   12 out, 13 ldo   T x D.   14 stream.
 */
int sg_combine_rows(const void* Z, int64_t ldz, int64_t M, int64_t D, int64_t T, int dtype,
                    const int32_t* place, int64_t top_k, const float* weights,
                    const void* residual, int64_t ldr, void* out, int64_t ldo, void* stream);

/*
 * sg_combine_rows_bwd, from the gradient dOut (T x D) of out:
 *     dZ[place[t, j]] = weights[t, j] * dOut[t]       rows that no place names stay as they are
 *     dweights[t, j] = dot(dOut[t], Z[place[t, j]])   0 for an empty place
 *  1 dOut, 2 lddo, 3 Z, 4 ldz, 5 M, 6 D, 7 T, 8 dtype, 9 place, 10 top_k, 11 weights (not NULL).
 *  12 dZ, 13 lddz   M x D, or NULL.   14 dweights   T x top_k fp32, or NULL (Z is then not read).
 *  15 stream.
 */
int sg_combine_rows_bwd(const void* dOut, int64_t lddo, const void* Z, int64_t ldz, int64_t M,
                        int64_t D, int64_t T, int dtype, const int32_t* place, int64_t top_k,
                        const float* weights, void* dZ, int64_t lddz, float* dweights,
                        void* stream);

/*
 * 4-bit integer weights with group scales
 * ---------------------------------------
 * A weight of N rows and K columns (the B of C = A * B^T) is held as codes 0..15, and for each
 * `group` (32, 64 or 128) columns of a row a scale of the activations' type (SG_F16 or SG_BF16)
 * and, optionally, a zero point of 8 bits:
 *     W[n, k] = scale[n, k / group] * (code[n, k] - zero[n, k / group]),  zero = 8 where none is held
 *   codes   SG_INT4_CODE_BYTES(N, K) bytes: tiles of 16 rows x 128 columns, 1024 bytes each, all
 *           tiles of 16 rows one after the other.  Element (r, c) of a tile, with s = c / 32,
 *           q = c % 32 / 8, i = c % 8: nibble i / 2 + 4 * (i % 2), counted from the low half of the
 *           first byte, of the four bytes at 16 * (16 * q + r) + 4 * s.
 *   scales  SG_INT4_SCALES(N, K, group) values: tiles of 16 rows x 4 groups: row r, group g at
 *   zeros   64 * ((r / 16) * ceil(groups / 4) + g / 4) + 4 * (r % 16) + g % 4; as many bytes.
 *           What lies outside the matrix is not used; sg_int4_quantize and _pack write zeros.
 * A batch of weights follows one another.  These calls allocate nothing and use no workspace;
 * results are run-to-run identical.
 */
#define SG_INT4_CODE_BYTES(N, K) \
    ((((int64_t)(N) + 15) / 16) * (((int64_t)(K) + 127) / 128) * 1024)
#define SG_INT4_SCALES(N, K, group) \
    ((((int64_t)(N) + 15) / 16) * ((((int64_t)(K) + (group) - 1) / (group) + 3) / 4) * 64)

/*
 * sg_int4_quantize: the codes of W.  For each group, without zeros: scale = max |w| / 7, codes
 * w / scale + 8; with zeros: lo = min(0, w), hi = max(0, w), scale = (hi - lo) / 15, zero =
 * -lo / scale and codes w / scale + zero.  The scale is computed in fp32 and rounded to its type
 * first; zeros and codes follow from the rounded one: each quotient is rounded to the nearest integer,
 * ties to even, before the zero point (or 8) is added, and what comes out saturates at 0 and 15.
 * A group of zeros, or whose scale rounds to 0, gets scale 0, zero 8 and codes 8.  An infinity or a
 * NaN, or a scale past its type's range, makes the group's scale NaN (zero and codes 8).
 *  1 W, 2 ldw, 3 strideW   `batch` weights N x K, strideW elements apart.   4 batch (0..65535)
 *  5 N, 6 K   >= 0.   7 dtype   of W: SG_F32, SG_F16 or SG_BF16.   8 group.
 *  9 codes (16-byte aligned), 10 scales (8), 11 zeros (4; NULL: none).
 *  12 scale_dtype   SG_F16 or SG_BF16.   13 stream.
 */
int sg_int4_quantize(const void* W, int64_t ldw, int64_t strideW, int64_t batch, int64_t N,
                     int64_t K, int dtype, int64_t group, void* codes, void* scales, void* zeros,
                     int scale_dtype, void* stream);

/*
 * sg_int4_pack: the same from codes, scales and zeros held one after the other: src codes N x K
 * bytes (their low four bits count), scales and zeros N x ceil(K / group) (zeros: bytes, or
 * NULL), all contiguous, for `batch` weights.
 *  1 src, 2 src_scales, 3 src_zeros (NULL with 10 NULL), 4 batch, 5 N, 6 K, 7 group, 8 codes,
 *  9 scales, 10 zeros, 11 stream.   Alignment as above; src_scales 2 bytes.
 */
int sg_int4_pack(const void* src, const void* src_scales, const void* src_zeros, int64_t batch,
                 int64_t N, int64_t K, int64_t group, void* codes, void* scales, void* zeros,
                 void* stream);

/*
 * sg_int4_dequantize: W = the values, fp32, rounded once to W's type.
 *  1 codes, 2 scales, 3 zeros (NULL: 8), 4 scale_dtype, 5 batch, 6 N, 7 K, 8 group, 9 W, 10 ldw,
 *  11 strideW (>= (N-1)*ldw + K for more than one), 12 dtype of W, 13 stream.
 */
int sg_int4_dequantize(const void* codes, const void* scales, const void* zeros, int scale_dtype,
                       int64_t batch, int64_t N, int64_t K, int64_t group, void* W, int64_t ldw,
                       int64_t strideW, int dtype, void* stream);

/*
 * sg_int4_gemm: C = alpha * A * W^T; with offsets C[r] = alpha * A[row(r)] * W_e^T for r in R_e
 * (see the products grouped by expert), W a batch of `experts` weights.  row(r) = r, or with
 * `order` (the table of sg_sort_experts) order[r] / top_k, so that the tokens' rows need not be
 * spread first; rows of C whose order is outside 0 .. T * top_k - 1 are undefined.  Sums are
 * fp32: codes meet A unscaled, each group's sum then its scale, so the weights are not rounded.
 * bf16 products take the codes from 16 up and (16 + zero) out of the sums: an infinity in A, a
 * value of it above 2^120, or sums of (16 + max(15, zero)) * scale * |a| past fp32's range give NaN or
 * an infinity where they count.  Those sums are larger than the values', so an fp32 C of bf16 operands
 * is less exact than an ordinary fp32 sum: K = 4096, rms error over C's rms 2^-22 to 2^-21 for activations
 * without a mean, up to 2^-18 with a mean of four times their spread (fp16: 2^-23).  A bf16 C rounds
 * off more.
 * From some hundred rows on sg_int4_dequantize and a 16-bit product (sg_gemm with transB) are faster: bf16
 * by 4096 x 11008 from about 768 rows (groups of 64 with zero points: 512), 1024 rows 119 and 103 us, 4096
 * rows 433 and 304 us; by 4096 x 4096 from about 1536 rows.
 * Products of more than 2^22 work-groups (tiles of 64 x 128 at the largest: 2^35 values of C) return
 * hipErrorInvalidConfiguration.  C may not overlap an input.
 *  1 experts, 2 offsets   as sg_mxfp4_gemm.   3 order   NULL, or M int32.   4 top_k (1..65536;
 *  1 without order).   5 T   rows of A (T = M without order).   6 M   rows of C.   7 N, 8 K,
 *  9 group.
 *  10 alpha   fp32.   11 A, 12 lda   T x K.   13 codes (16-byte aligned), 14 scales (8),
 *  15 zeros (4, or NULL).   16 C, 17 ldc   M x N, written only.
 *  18 dtype   of A and the scales: SG_F16 or SG_BF16.   19 c_dtype   dtype or SG_F32.  20 stream.
 * Quick returns: M == 0 or N == 0 does nothing; K == 0 or alpha == 0 writes zeros.
 */
int sg_int4_gemm(int64_t experts, const int32_t* offsets, const int32_t* order, int64_t top_k,
                 int64_t T, int64_t M, int64_t N, int64_t K, int64_t group, float alpha,
                 const void* A, int64_t lda, const void* codes, const void* scales,
                 const void* zeros, void* C, int64_t ldc, int dtype, int c_dtype, void* stream);

/*
 * sg_int4_swiglu_gemm: Y = SiLU(A * W1^T) ⊙ (A * W2^T) from W of 2N rows, gate and up
 * interleaved (row 2n = W1's row n, row 2n+1 = W2's); the rest as sg_int4_gemm.
 *  1 experts, 2 offsets, 3 order, 4 top_k, 5 T, 6 M, 7 N, 8 K, 9 group, 10 A, 11 lda, 12 codes,
 *  13 scales, 14 zeros, 15 Y, 16 ldy   M x N.   17 dtype   of A, the scales and Y.   18 stream.
 */
int sg_int4_swiglu_gemm(int64_t experts, const int32_t* offsets, const int32_t* order,
                        int64_t top_k, int64_t T, int64_t M, int64_t N, int64_t K, int64_t group,
                        const void* A, int64_t lda, const void* codes, const void* scales,
                        const void* zeros, void* Y, int64_t ldy, int dtype, void* stream);

/* Text for a status code returned by any sg_* call (static storage). */
const char* sg_status_string(int status);

/* Identifies the build (static storage): "swiglu_gemm source <hash> gfx950", where
 * <hash> is 16 hex digits of the SHA-256 over the library's kernel and ABI sources
 * (swiglu_gemm_amd/build.py, source_hash).  The Python binding compares it with the
 * sources beside the library and refuses a library built from other sources. */
const char* sg_build_info(void);

/*
 * Describes the kernel configuration chosen by the most recent successful
 * sg_gemm / sg_swiglu_gemm call on the calling thread (tile, split count; for a
 * problem run as two launches over column ranges, "columns 0..n1" and the tail's
 * configuration; for the decode kernels their grid and units) as a NUL-terminated
 * string copied into buf (at most len bytes).  Returns the full length of the
 * description.  Meant for logs and tests; the format is not a stable interface.
 */
int sg_last_config(char* buf, int len);

/* Frees the library-owned workspace buffers (current and outgrown) on every device,
 * after synchronising each device that holds one. */
void sg_release(void);

#ifdef __cplusplus
}
#endif

#endif /* SWIGLU_GEMM_H */
