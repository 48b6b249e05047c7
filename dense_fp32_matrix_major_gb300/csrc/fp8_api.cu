// C ABI of the 8-bit floating point operators: argument checks and dispatch.
// The declarations and the contract of every entry point are in fp8.h.
#include <cuda_runtime.h>
#include <stdint.h>

#include "api_checks.h"
#include "fp8_internal.h"

namespace sgemm {
namespace f8 {
namespace {

using namespace api;
using ex::type_size;

bool fp8_ok(int type) { return type == SGEMM_FP8_E4M3 || type == SGEMM_FP8_E5M2; }

bool experts_ok(int64_t experts, const int32_t *offsets) {
    return experts >= 1 && experts <= SGEMM_EXPERTS_MAX && (offsets || experts == 1);
}

// An operand that TMA reads: rows that start on 16-byte boundaries.
bool aligned(const Span &s) {
    return s.empty() || (s.begin() % 16 == 0 && s.ld % 16 == 0 && (s.items == 1 || s.stride % 16 == 0));
}

// Sizes within tensor map coordinates.
bool coordinate(int64_t n) { return n >= 0 && n < INT32_MAX / 2; }

// Zeros in C (an empty sum).
int clear(const Span &c, cudaStream_t stream) {
    for (int64_t i = 0; i < c.items; ++i) {
        void *p = static_cast<uint8_t *>(const_cast<void *>(c.p)) + i * c.stride * c.size;
        if (cudaMemset2DAsync(p, static_cast<size_t>(c.ld * c.size), 0, static_cast<size_t>(c.cols * c.size),
                              static_cast<size_t>(c.rows), stream) != cudaSuccess) {
            cudaGetLastError();
            return SGEMM_ERR_LAUNCH;
        }
    }
    return SGEMM_OK;
}

}  // namespace
}  // namespace f8
}  // namespace sgemm

using namespace sgemm;
using namespace sgemm::f8;
using namespace sgemm::api;
using sgemm::ex::type_size;

extern "C" {

int64_t sgemm_fp8_blocks(int64_t rows, int64_t experts) {
    if (rows < 0 || rows > kMostRows || experts < 1 || experts > SGEMM_EXPERTS_MAX) return 0;
    return (rows + (BLOCK - 1) * (rows < experts ? rows : experts)) / BLOCK;
}

int sgemm_fp8_quantize(int type, int block, int to, int pow2, int64_t items, int64_t rows, int64_t cols,
                       const void *x, int64_t ldx, int64_t strideX, int64_t experts, const int32_t *offsets, void *q,
                       int64_t ldq, int64_t strideQ, float *scales, sgemm_stream_t stream) {
    if (!type_ok(type) || block < SGEMM_FP8_ROWS || block > SGEMM_FP8_BLOCKS || !fp8_ok(to) || items < 0 ||
        rows < 0 || cols < 0 || rows > kMostRows || cols > kMostRows || (items != 1 && block != SGEMM_FP8_BLOCKS) ||
        (offsets && block != SGEMM_FP8_COLUMNS) || !experts_ok(experts, offsets))
        return SGEMM_ERR_INVALID_ARG;
    const int64_t stored = offsets ? BLOCK * sgemm_fp8_blocks(rows, experts) : rows;
    const int64_t high = block == SGEMM_FP8_ROWS ? rows : blocks_of(stored);
    const int64_t wide = block == SGEMM_FP8_COLUMNS ? cols : blocks_of(cols);
    const Span in{x, rows, cols, ldx, type_size(type), items, strideX}, out{q, stored, cols, ldq, 1, items, strideQ},
        off = flat(offsets, offsets ? experts + 1 : 0, 4);
    if (!in.ok() || !out.ok() || !off.ok()) return SGEMM_ERR_INVALID_ARG;
    if (high > 0 && wide > 0 && items > kLimit / high / wide) return SGEMM_ERR_INVALID_ARG;
    const Span sc = flat(scales, items * high * wide, 4);
    if (!sc.ok() || out.overlaps(in) || out.overlaps(off) || out.overlaps(sc) || sc.overlaps(in) || sc.overlaps(off))
        return SGEMM_ERR_INVALID_ARG;
    const QuantizeProblem p{type, block, to, pow2 != 0, items, rows, cols, x, ldx, strideX, experts, offsets,
                            static_cast<uint8_t *>(q), ldq, strideQ, scales};
    return enqueue([&](const DeviceInfo &dev, int *launches) {
        if (in.empty()) return static_cast<int>(SGEMM_OK);
        return quantize_launch(p, dev, reinterpret_cast<cudaStream_t>(stream), launches);
    });
}

int sgemm_fp8_gemm(int out_type, int transB, int type_a, int type_b, int64_t rows, int64_t N, int64_t K,
                   int64_t experts, const int32_t *offsets, const void *A, int64_t lda, const float *sA,
                   const void *B, int64_t ldb, int64_t strideB, const float *sB, void *C, int64_t ldc,
                   sgemm_stream_t stream) {
    if (!type_ok(out_type) || (transB != SGEMM_OP_N && transB != SGEMM_OP_T) || !fp8_ok(type_a) || !fp8_ok(type_b) ||
        rows < 0 || rows > kMostRows || !coordinate(N) || !coordinate(K) || !experts_ok(experts, offsets))
        return SGEMM_ERR_INVALID_ARG;
    const Span a{A, rows, K, lda, 1}, b{B, transB ? N : K, transB ? K : N, ldb, 1, experts, strideB},
        c{C, rows, N, ldc, type_size(out_type)}, off = flat(offsets, offsets ? experts + 1 : 0, 4),
        sa = flat(sA, blocks_of(K) * rows, 4), sb = flat(sB, experts * blocks_of(K) * blocks_of(N), 4);
    if (!a.ok() || !b.ok() || !c.ok() || !off.ok() || !sa.ok() || !sb.ok()) return SGEMM_ERR_INVALID_ARG;
    if (!aligned(a) || !aligned(b)) return SGEMM_ERR_INVALID_ARG;
    if (c.overlaps(a) || c.overlaps(b) || c.overlaps(off) || c.overlaps(sa) || c.overlaps(sb))
        return SGEMM_ERR_INVALID_ARG;
    GemmProblem p{};
    p.wgrad = false;
    p.out_type = out_type;
    p.transB = transB;
    p.type_a = type_a;
    p.type_b = type_b;
    p.rows = rows;
    p.M = rows;
    p.N = N;
    p.K = K;
    p.experts = experts;
    p.offsets = offsets;
    p.A = A;
    p.lda = lda;
    p.sA = sA;
    p.B = B;
    p.ldb = ldb;
    p.strideB = strideB;
    p.sB = sB;
    p.C = C;
    p.ldc = ldc;
    return enqueue([&](const DeviceInfo &dev, int *launches) {
        if (c.empty()) return static_cast<int>(SGEMM_OK);
        if (K == 0) return clear(c, reinterpret_cast<cudaStream_t>(stream));
        return gemm_launch(p, dev, reinterpret_cast<cudaStream_t>(stream), launches);
    });
}

int sgemm_fp8_gemm_wgrad(int out_type, int type_a, int type_b, int64_t rows, int64_t M, int64_t N, int64_t experts,
                         const int32_t *offsets, const void *A, int64_t lda, const float *sA, const void *B,
                         int64_t ldb, const float *sB, void *C, int64_t ldc, int64_t strideC, sgemm_stream_t stream) {
    if (!type_ok(out_type) || !fp8_ok(type_a) || !fp8_ok(type_b) || rows < 0 || rows > kMostRows || !coordinate(M) ||
        !coordinate(N) || !experts_ok(experts, offsets) || (offsets && rows % BLOCK != 0))
        return SGEMM_ERR_INVALID_ARG;
    const Span a{A, rows, M, lda, 1}, b{B, rows, N, ldb, 1}, c{C, M, N, ldc, type_size(out_type), experts, strideC},
        off = flat(offsets, offsets ? experts + 1 : 0, 4), sa = flat(sA, blocks_of(rows) * M, 4),
        sb = flat(sB, blocks_of(rows) * N, 4);
    if (!a.ok() || !b.ok() || !c.ok() || !off.ok() || !sa.ok() || !sb.ok()) return SGEMM_ERR_INVALID_ARG;
    if (!aligned(a) || !aligned(b)) return SGEMM_ERR_INVALID_ARG;
    if (c.overlaps(a) || c.overlaps(b) || c.overlaps(off) || c.overlaps(sa) || c.overlaps(sb))
        return SGEMM_ERR_INVALID_ARG;
    GemmProblem p{};
    p.wgrad = true;
    p.out_type = out_type;
    p.type_a = type_a;
    p.type_b = type_b;
    p.rows = rows;
    p.M = M;
    p.N = N;
    p.K = rows;
    p.experts = experts;
    p.offsets = offsets;
    p.A = A;
    p.lda = lda;
    p.sA = sA;
    p.B = B;
    p.ldb = ldb;
    p.sB = sB;
    p.C = C;
    p.ldc = ldc;
    p.strideC = strideC;
    return enqueue([&](const DeviceInfo &dev, int *launches) {
        if (c.empty()) return static_cast<int>(SGEMM_OK);
        if (rows == 0) return clear(c, reinterpret_cast<cudaStream_t>(stream));
        return gemm_launch(p, dev, reinterpret_cast<cudaStream_t>(stream), launches);
    });
}

}  // extern "C"
