/*
 * fp8.h — products of matrices in 8-bit floating point with a scale for each
 * block of 128, in libsgemm_gb300.so: the quantisation, the product of a
 * training step or a server, dense or one per expert of a mixture, and its
 * gradients.
 *
 * Conventions are those of sgemm.h and experts.h: sizes and strides are int64_t
 * element counts, pointers are device pointers owned by the caller, calls
 * enqueue on `stream` and return, status codes are sgemm_status values and on
 * an error nothing is enqueued. Nothing is kept between calls; the gradient of few
 * matrices over many rows takes sums of slices of them from the library's
 * stream-ordered pool, otherwise no memory is allocated. Outputs must not overlap
 * inputs.
 *
 * Values. E4M3 (4 exponent bits, 3 digits, largest value 448, no infinity) and
 * E5M2 (largest finite value 57344). An element stands for its 8-bit value
 * times the fp32 scale of its block. Blocks are 128 consecutive elements along
 * the direction that a product sums, by 1 or by 128 elements across it:
 *
 *   SGEMM_FP8_ROWS     1 x 128: rows of a matrix whose columns are summed over.
 *                      scales: ceil(cols / 128) x rows.
 *   SGEMM_FP8_COLUMNS  128 x 1: a matrix whose rows are summed over (gradients
 *                      of weights). scales: ceil(rows / 128) x cols.
 *   SGEMM_FP8_BLOCKS   128 x 128: weights, read either way round.
 *                      scales: ceil(rows / 128) x ceil(cols / 128).
 *
 * Scales are contiguous, the summed direction's blocks first for the first two.
 * The last block of a direction may be shorter.
 *
 * Groups. With experts and offsets (see experts.h) rows are sorted by expert.
 * SGEMM_FP8_COLUMNS then starts its blocks anew with every group and stores
 * every block as 128 rows, zeros after the group's last one: block i of the
 * groups in order is rows 128 i .. 128 i + 127. There is room for
 * sgemm_fp8_blocks(rows, experts) blocks; those not needed, and rows outside
 * every group, are zeros.
 */
#ifndef SGEMM_GB300_FP8_H
#define SGEMM_GB300_FP8_H

#include "experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 8-bit element types. */
enum sgemm_fp8_type {
    SGEMM_FP8_E4M3 = 0,
    SGEMM_FP8_E5M2 = 1
};

/* Shapes of the blocks that share a scale. */
enum sgemm_fp8_block {
    SGEMM_FP8_ROWS = 0,
    SGEMM_FP8_COLUMNS = 1,
    SGEMM_FP8_BLOCKS = 2
};

#define SGEMM_FP8_BLOCK_SIZE 128

/*
 * q = x * (1 / scale), the reciprocal and the product rounded to fp32, then to
 * the nearest 8-bit value, ties to even. scale = max |x| over the block / the
 * type's largest value, rounded to fp32 and at least 2^-126; with pow2 the
 * smallest power of two not below that.
 *   type            of x: sgemm_type.
 *   items           matrices, strideX and strideQ apart (strides are not read
 *                   for one); more than one only for SGEMM_FP8_BLOCKS.
 *   x, ldx          rows x cols.
 *   offsets         experts + 1 group bounds or NULL; only for
 *                   SGEMM_FP8_COLUMNS.
 *   q, ldq          out, rows x cols (128 * sgemm_fp8_blocks(rows, experts) x
 *                   cols with offsets). A product wants q 16-byte aligned and
 *                   ldq a multiple of 16.
 *   scales          out, contiguous, items times the sizes above.
 * Infinities and NaN become NaN and do not count for the block's scale.
 */
int sgemm_fp8_quantize(int type, int block, int to, int pow2, int64_t items, int64_t rows, int64_t cols,
                       const void *x, int64_t ldx, int64_t strideX, int64_t experts, const int32_t *offsets, void *q,
                       int64_t ldq, int64_t strideQ, float *scales, sgemm_stream_t stream);
/* floor((rows + 127 * min(rows, experts)) / 128): blocks that any groups of `rows` rows can need. */
int64_t sgemm_fp8_blocks(int64_t rows, int64_t experts);

/*
 * C[s] = A[s] op(B), or with offsets C[s] = A[s] op(B[e]) for the rows s of
 * group e and zero for rows outside every group.
 *   out_type   of C: sgemm_type.
 *   A, lda     rows x K of type_a; sA its SGEMM_FP8_ROWS scales.
 *   B, ldb     experts matrices strideB elements apart, each K x N
 *              (SGEMM_OP_N) or N x K (SGEMM_OP_T), of type_b; sB their
 *              SGEMM_FP8_BLOCKS scales.
 *   offsets    experts + 1 group bounds; NULL: one matrix, experts == 1.
 *   C, ldc     out, rows x N.
 * A and B are 16-byte aligned, lda, ldb and strideB multiples of 16; rows must
 * be below 2^31 - 1024. Every block of 128 products is summed on the tensor
 * cores in fp32 and scaled by the product of its two scales (which should
 * neither overflow nor fall below 2^-126), the blocks are added up in fp32 in an
 * order that is always the same, and the sum is rounded once to C's type. A row's
 * result depends on that row and its matrix, and on whether the call takes the
 * kernel for few rows (without offsets, SGEMM_OP_T, at most 16 rows, or 32 for a
 * small N), which adds the blocks up in another order. The gradient of A is the
 * same call on C's gradient, quantised in rows, with transB the other way round.
 */
int sgemm_fp8_gemm(int out_type, int transB, int type_a, int type_b, int64_t rows, int64_t N, int64_t K,
                   int64_t experts, const int32_t *offsets, const void *A, int64_t lda, const float *sA,
                   const void *B, int64_t ldb, int64_t strideB, const float *sB, void *C, int64_t ldc,
                   sgemm_stream_t stream);

/*
 * C = A^T B, or with offsets C[e] = A_e^T B_e over the rows of group e (zeros
 * for an empty group): the gradient of sgemm_fp8_gemm's B, with A its A and B
 * its C's gradient for SGEMM_OP_N, the two exchanged for SGEMM_OP_T.
 *   A, lda     rows x M of type_a; sA its SGEMM_FP8_COLUMNS scales. With
 *              offsets rows are counted as sgemm_fp8_quantize stores them:
 *              a multiple of 128.
 *   B, ldb     rows x N of type_b, sB, likewise.
 *   C, ldc     out, experts matrices of M x N, strideC elements apart.
 * Alignment, limits and sums as for sgemm_fp8_gemm, except that few matrices over
 * many rows are summed in slices of the rows, whose fp32 sums are then added in
 * order. The sizes (and the device's number of SMs) say into how many. Only when
 * the pool has no memory for them are the rows summed in one piece, which rounds
 * otherwise.
 */
int sgemm_fp8_gemm_wgrad(int out_type, int type_a, int type_b, int64_t rows, int64_t M, int64_t N, int64_t experts,
                         const int32_t *offsets, const void *A, int64_t lda, const float *sA, const void *B,
                         int64_t ldb, const float *sB, void *C, int64_t ldc, int64_t strideC, sgemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_GB300_FP8_H */
