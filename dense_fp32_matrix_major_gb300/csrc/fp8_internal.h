// Internal declarations of the 8-bit floating point operators (the public ABI
// is include/fp8.h). Launchers run after argument checks; they return an
// sgemm_status code and add the kernels they enqueue to *launches.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "experts_internal.h"
#include "fp8.h"

namespace sgemm {
namespace f8 {

constexpr int BLOCK = SGEMM_FP8_BLOCK_SIZE;

inline int64_t blocks_of(int64_t n) { return (n + BLOCK - 1) / BLOCK; }

// Quantisation (fp8_quantize.cu).
struct QuantizeProblem {
    int type, block, to, pow2;
    int64_t items, rows, cols;
    const void *x;
    int64_t ldx, strideX;
    int64_t experts;
    const int32_t *offsets;
    uint8_t *q;
    int64_t ldq, strideQ;
    float *scales;
};
int quantize_launch(const QuantizeProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches);

// Products (fp8_gemm.cu). wgrad = false: C[s] = A[s] op(B[e]), A rows x K, C
// rows x N. wgrad = true: C[e] = A_e^T B_e, A rows x M, B rows x N.
struct GemmProblem {
    bool wgrad;
    int out_type, transB, type_a, type_b;
    int64_t rows, M, N, K, experts;
    const int32_t *offsets;
    const void *A;
    int64_t lda;
    const float *sA;
    const void *B;
    int64_t ldb, strideB;
    const float *sB;
    void *C;
    int64_t ldc, strideC;
    int split = 1;  // wgrad: slices of a group's rows; C is then fp32, an item per slice
};
int gemm_launch(const GemmProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches);

// The same for a few rows (fp8_few.cu): whether it takes the problem, and the launch.
bool gemm_few(const GemmProblem &p, const DeviceInfo &dev);
int gemm_few_launch(const GemmProblem &p, cudaStream_t stream, int *launches);

}  // namespace f8
}  // namespace sgemm
