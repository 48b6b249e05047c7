/*
 * experts.h — operators of a mixture-of-experts layer, in libsgemm_gb300.so:
 * the sort of (token, choice) pairs by expert, the row copies that go with
 * it and their gradients, one product per expert over its group of rows with
 * the gradient of the experts' matrices, and matrix-vector products with
 * 4-bit weights for serving single tokens.
 *
 * Conventions are those of sgemm.h: sizes and strides are int64_t element
 * counts, pointers are device pointers owned by the caller, calls enqueue on
 * `stream` and return, status codes are sgemm_status values and on an error
 * nothing is enqueued. Nothing is kept between calls. Outputs must not
 * overlap inputs.
 *
 * Pairs and groups. T tokens choose top_k experts each. Pair p = t * top_k + j
 * is token t's j-th choice. Sorting the P = T * top_k pairs by expert, stably,
 * and those without an expert (an id below 0 or not below `experts`: dropped)
 * last, gives every pair a slot in 0 .. P-1. Group e holds the slots
 * offsets[e] .. offsets[e + 1] - 1; slots from offsets[experts] on belong to
 * dropped pairs. Arrays of slots and offsets are read with bounds checks: a
 * slot outside 0 .. P-1 counts as dropped, an offset is limited to 0 .. rows,
 * offsets[0] is taken as 0. Offsets that decrease give wrong rows but no
 * access outside the arrays.
 *
 * Numbers. Rows are fp32, bf16 or fp16. Sums are held in fp32 and rounded
 * once to the row type; the order of every sum is fixed by the sizes, so the
 * same call gives the same bits. No atomics touch results.
 *
 * Streams and graphs. Calls may be captured in a CUDA graph once a call of the
 * same kind has run on the device (the first sets kernels and the scratch pool
 * up). A kernel may become resident while the one before it in the stream ends;
 * it reads nothing before that one's end.
 */
#ifndef SGEMM_GB300_EXPERTS_H
#define SGEMM_GB300_EXPERTS_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of rows, weights and scales. */
enum sgemm_type {
    SGEMM_TYPE_F32 = 0,
    SGEMM_TYPE_BF16 = 1,
    SGEMM_TYPE_F16 = 2
};

/* Largest `experts` and `top_k` of the calls below. */
#define SGEMM_EXPERTS_MAX 4096
#define SGEMM_TOP_K_MAX 64
/* Most rows of one sgemm_w4_matvec call. */
#define SGEMM_W4_ROWS_MAX 65535

/*
 * Sorts the pairs by expert.
 *   ids        T x top_k ids, contiguous, int32 (id_bits = 32) or int64 (64).
 *   offsets    out, experts + 1 values.
 *   order      out, P values: the pair at each slot.
 *   slot       out, T x top_k values: the slot of each pair.
 *   workspace  workspace_bytes bytes, 16-byte aligned, at least
 *              sgemm_experts_sort_workspace(P, experts) (0 for few pairs:
 *              NULL is then accepted). Contents need not be set.
 * P must be below 2^31. T == 0: offsets is set to zeros.
 */
int sgemm_experts_sort(const void *ids, int id_bits, int64_t tokens, int64_t top_k, int64_t experts,
                       int32_t *offsets, int32_t *order, int32_t *slot, void *workspace, size_t workspace_bytes,
                       sgemm_stream_t stream);
size_t sgemm_experts_sort_workspace(int64_t pairs, int64_t experts);

/*
 * xs[slot[t][j]] = x[t] for every pair, zero rows for dropped pairs.
 *   x, ldx     T x width, row stride ldx >= width.
 *   slot, offsets, experts   as sgemm_experts_sort gives them.
 *   xs, ldxs   out, P x width.
 */
int sgemm_experts_gather(int type, int64_t tokens, int64_t top_k, int64_t experts, int64_t width, const void *x,
                         int64_t ldx, const int32_t *slot, const int32_t *offsets, void *xs, int64_t ldxs,
                         sgemm_stream_t stream);

/*
 * y[t] = sum over j of weights[t][j] * h[slot[t][j]], dropped pairs left out
 * (a token with none left gives a zero row).
 *   h, ldh     P x width rows in slot order.
 *   weights    T x top_k fp32, contiguous; NULL: every weight is 1, which is
 *              the gradient of sgemm_experts_gather (h its output's gradient,
 *              y its input's).
 *   y, ldy     out, T x width.
 */
int sgemm_experts_combine(int type, int64_t tokens, int64_t top_k, int64_t experts, int64_t width, const void *h,
                          int64_t ldh, const float *weights, const int32_t *slot, const int32_t *offsets, void *y,
                          int64_t ldy, sgemm_stream_t stream);

/*
 * Gradients of sgemm_experts_combine:
 *   dh[slot[t][j]] = weights[t][j] * dy[t]            (P x width; dropped: 0)
 *   dweights[t][j] = sum over i of dy[t][i] * h[slot[t][j]][i]   (fp32; dropped: 0)
 * `weights` as above but not NULL.
 */
int sgemm_experts_combine_grad(int type, int64_t tokens, int64_t top_k, int64_t experts, int64_t width,
                               const void *dy, int64_t lddy, const void *h, int64_t ldh, const float *weights,
                               const int32_t *slot, const int32_t *offsets, void *dh, int64_t lddh,
                               float *dweights, sgemm_stream_t stream);

/*
 * One product per group: C[s] = A[s] * op(B[e]) for the rows s of group e;
 * rows of C outside every group are set to zero.
 *   A, lda     rows x K.
 *   B, ldb     experts matrices strideB elements apart (strideB >= one
 *              matrix), each K x N (SGEMM_OP_N) or N x K (SGEMM_OP_T).
 *   C, ldc     out, rows x N.
 * rows must be below 2^31 - 1024. fp32 inputs follow sgemm_f32's accuracy
 * bound and its rules for infinities and NaN, and the variant that
 * sgemm_set_variant chose: SGEMM_AUTO and SGEMM_TF32X3 the three-term TF32
 * split (two 11-bit parts of each factor, the product of the low parts left
 * out), whose error on normal inputs is up to 0.7e-6 of the result's norm where
 * that of fp32 sums is 0.1e-6 (of a few dozen terms) to 0.6e-6 (of a thousand);
 * SGEMM_FFMA fp32 multiply-adds, one after the other, about eight times slower. bf16 and fp16 products are exact in fp32 and
 * summed in fp32, where the tensor core cuts a running sum at every 16 products:
 * about 2e-8 of it each time, 2e-5 for sums of 16384, far below the rounding of the
 * result. A row's result depends on that row and its expert's matrix only,
 * whatever the other sizes (16-bit operands whose rows are not 16-byte aligned
 * are summed in one of two orders, by the sizes). The gradient of A is the same
 * call on C's gradient with transB the other way round.
 */
int sgemm_experts_gemm(int type, int transB, int64_t rows, int64_t N, int64_t K, int64_t experts,
                       const int32_t *offsets, const void *A, int64_t lda, const void *B, int64_t ldb,
                       int64_t strideB, void *C, int64_t ldc, sgemm_stream_t stream);

/*
 * One product per group over its rows: C[e] = sum over s in group e of
 * A[s]^T * B[s] (an empty group gives zeros). rows must be below 2^31 - 1024.
 *   A, lda     rows x M.
 *   B, ldb     rows x N.
 *   C, ldc     out, experts matrices of M x N, strideC elements apart.
 * The gradient of sgemm_experts_gemm's B: with A its A and B its C's
 * gradient for SGEMM_OP_N, the two exchanged for SGEMM_OP_T.
 */
int sgemm_experts_gemm_wgrad(int type, int64_t rows, int64_t M, int64_t N, int64_t experts, const int32_t *offsets,
                             const void *A, int64_t lda, const void *B, int64_t ldb, void *C, int64_t ldc,
                             int64_t strideC, sgemm_stream_t stream);

/*
 * y[r][n] = sum over k of (q[e][n][k] - zero[e][n][k / group]) *
 *           scale[e][n][k / group] * x[r][k],   e = ids[r], or 0 without ids.
 *   x, ldx     rows x K.
 *   q          experts x N x K 4-bit values, contiguous, two to a byte, the
 *              even k in the low four bits. K is even.
 *   group      values of k that share a scale: 32, 64, 128 or 256; the last
 *              group of a row may be shorter.
 *   scales     experts x N x ceil(K / group) of scale_type, contiguous.
 *   zeros      experts x N x ceil(K / group) bytes of 0 .. 15 (the low four
 *              bits are used), contiguous; NULL: every zero point is 8.
 *   ids        rows int32; NULL: every row uses matrix 0 (experts must be
 *              1). A row whose id is below 0 or not below experts is zero.
 *   y, ldy     out, rows x N, of x's type.
 * Meant for few rows: the matrices are read once per eight rows that share
 * one. q - zero is exact, so an x whose q is the zero point adds nothing, however
 * large it is. The inner sums are scaled group by group; where one overflows
 * and x is finite the output is summed again in 64 bits (K a multiple of 32 and q
 * 16-byte aligned; otherwise every term is scaled first, and sums are fp32).
 */
int sgemm_w4_matvec(int type, int64_t rows, int64_t N, int64_t K, int64_t group, int64_t experts,
                    const int32_t *ids, const void *x, int64_t ldx, const uint8_t *q, const void *scales,
                    int scale_type, const uint8_t *zeros, void *y, int64_t ldy, sgemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_GB300_EXPERTS_H */
