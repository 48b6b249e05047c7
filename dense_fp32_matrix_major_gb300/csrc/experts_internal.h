// Internal declarations of the mixture-of-experts operators (the public ABI
// is include/experts.h). Launchers run after argument checks; they return an
// sgemm_status code and add the kernels they enqueue to *launches.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "experts.h"
#include "sgemm_internal.h"

namespace sgemm {
namespace ex {

inline int64_t type_size(int type) { return type == SGEMM_TYPE_F32 ? 4 : 2; }

// Sort of P pairs (experts_route.cu). sort_blocks: blocks of the two-kernel
// form, 0 for the single-block form.
int sort_blocks(int64_t pairs, int64_t experts);
int sort_launch(const void *ids, int id_bits, int64_t pairs, int64_t experts, int32_t *offsets, int32_t *order,
                int32_t *slot, int32_t *workspace, const DeviceInfo &dev, cudaStream_t stream, int *launches);

// The pairs of T tokens and their rows.
struct Route {
    int64_t tokens, top_k, experts, width;
    const int32_t *slot;
    const int32_t *offsets;
};

int gather_launch(int type, const Route &r, const void *x, int64_t ldx, void *xs, int64_t ldxs, const DeviceInfo &dev,
                  cudaStream_t stream, int *launches);
int combine_launch(int type, const Route &r, const void *h, int64_t ldh, const float *weights, void *y, int64_t ldy,
                   const DeviceInfo &dev, cudaStream_t stream, int *launches);
int combine_grad_launch(int type, const Route &r, const void *dy, int64_t lddy, const void *h, int64_t ldh,
                        const float *weights, void *dh, int64_t lddh, float *dweights, const DeviceInfo &dev,
                        cudaStream_t stream, int *launches);

// One product per group (experts_gemm.cu). wgrad = false: C[s] = A[s] op(B[e]),
// A rows x K, C rows x N. wgrad = true: C[e] = A_e^T B_e, A rows x M, B rows x N.
struct GroupedProblem {
    bool wgrad;
    int type, transB;
    int64_t rows, M, N, K, experts;
    const int32_t *offsets;
    const void *A;
    int64_t lda;
    const void *B;
    int64_t ldb, strideB;
    void *C;
    int64_t ldc, strideC;
    int split = 1;  // wgrad: slices of a group's rows; C is then fp32, an item per slice, rows 16-byte aligned
};
int grouped_launch(const GroupedProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches);
// fp32 on SM pairs (experts_gemm_f32.cu).
bool grouped_f32_supports(const GroupedProblem &p);
void grouped_f32_tile(const GroupedProblem &p, int64_t *high, int64_t *wide);  // of C
int grouped_f32_launch(const GroupedProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches);
// bf16 and fp16 on SM pairs (experts_gemm_16.cu).
bool grouped16_supports(const GroupedProblem &p);
int grouped16_launch(const GroupedProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches);

// Matrix-vector products with 4-bit weights (w4_matvec.cu).
struct W4Problem {
    int type, scale_type;
    int64_t rows, N, K, group, experts;
    const int32_t *ids;
    const void *x;
    int64_t ldx;
    const uint8_t *q;
    const void *scales;
    const uint8_t *zeros;
    void *y;
    int64_t ldy;
};
int w4_launch(const W4Problem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches);

}  // namespace ex

// Records the launches of the last successful call (sgemm_last_launch_count)
// and the variant of the last fp32 product (sgemm_last_variant_used).
void note_launches(int launches);
void note_variant(int variant);
// The caller's choice (sgemm_set_variant).
int chosen_variant();

}  // namespace sgemm
