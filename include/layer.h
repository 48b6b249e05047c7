/*
 * layer.h — a whole mixture-of-experts layer for a few tokens, in
 * libsgemm_gb300.so: what a server runs for a decoding step, in two kernels.
 *
 * Conventions are those of sgemm.h and experts.h: sizes and strides are int64_t
 * element counts, pointers are device pointers owned by the caller, calls
 * enqueue on `stream` and return, status codes are sgemm_status values and on
 * an error nothing is enqueued. Nothing is kept between calls, no memory is
 * allocated. Outputs must not overlap inputs. The order of every sum is fixed
 * by the sizes and the ids, so the same call gives the same bits.
 */
#ifndef SGEMM_GB300_LAYER_H
#define SGEMM_GB300_LAYER_H

#include "fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How the experts' matrices are held. */
enum sgemm_layer_weights {
    SGEMM_LAYER_SAME = 0, /* in the type of x */
    SGEMM_LAYER_E4M3 = 1, /* 8-bit, SGEMM_FP8_BLOCKS scales */
    SGEMM_LAYER_E5M2 = 2
};

/* Most (token, choice) pairs of a call. Beyond, sort the pairs and make a
 * product per expert (experts.h): the matrices are then no longer all the work. */
#define SGEMM_LAYER_PAIRS_MAX 512

/*
 * y[t] = sum over j of weights[t][j] * W2[e] h,   e = ids[t][j],
 *   h = act(W1[e] x[t])                            (gated == 0), or
 *   h[f] = act((W1[e] x[t])[f]) * (W1[e] x[t])[hidden + f]   (gated != 0).
 * A pair whose id is below 0 or not below `experts` is left out; a token with
 * none left gives a zero row.
 *   type        of x and y: sgemm_type.
 *   held        of W1 and W2: sgemm_layer_weights.
 *   activation  sgemm_activation.
 *   x, ldx      tokens x width.
 *   ids         tokens x top_k, contiguous, int32 (id_bits = 32) or int64 (64).
 *   weights     tokens x top_k fp32, contiguous.
 *   W1, ld1     experts matrices stride1 elements apart, each hidden (2 * hidden
 *               when gated: those of the activation first) x width.
 *   W2, ld2     experts matrices stride2 apart, each width x hidden.
 *   s1, s2      scales of 8-bit matrices, contiguous, ceil(rows / 128) x
 *               ceil(columns / 128) for each expert; otherwise not read.
 *   y, ldy      out, tokens x width.
 *   workspace   workspace_bytes bytes, 16-byte aligned, at least
 *               sgemm_experts_layer_workspace(tokens, top_k, hidden). Contents
 *               need not be set. Not to be shared by calls that may run at once.
 * tokens * top_k is SGEMM_LAYER_PAIRS_MAX at most. Sums are fp32; h is held in
 * fp32 (with x of 16 bits as two bf16 terms, 16 bits of it), y is rounded once.
 * Each expert's matrices are read once per 8 pairs that share it. 8-bit ones
 * start on 16-byte boundaries, with ld1, ld2, stride1 and stride2 multiples of 16;
 * otherwise every width, alignment and stride is served, fastest where rows are
 * 16-byte aligned. Infinities and NaN follow IEEE arithmetic, except that an
 * infinite element of a 16-bit W2, which meets both terms of h, may give NaN in
 * place of an infinity.
 */
int sgemm_experts_layer(int type, int held, int activation, int gated, int64_t tokens, int64_t top_k,
                        int64_t experts, int64_t width, int64_t hidden, const void *x, int64_t ldx, const void *ids,
                        int id_bits, const float *weights, const void *W1, int64_t ld1, int64_t stride1,
                        const float *s1, const void *W2, int64_t ld2, int64_t stride2, const float *s2, void *y,
                        int64_t ldy, void *workspace, size_t workspace_bytes, sgemm_stream_t stream);
size_t sgemm_experts_layer_workspace(int64_t tokens, int64_t top_k, int64_t hidden);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_GB300_LAYER_H */
