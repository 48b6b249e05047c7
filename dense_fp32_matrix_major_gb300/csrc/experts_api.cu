// C ABI of the mixture-of-experts operators: argument checks and dispatch.
// The declarations and the contract of every entry point are in experts.h.
#include <cuda_runtime.h>
#include <stdint.h>

#include "api_checks.h"
#include "experts_internal.h"

namespace sgemm {
namespace ex {
namespace {

using namespace api;

// The pairs of a call: counts in range and P below 2^31.
bool pairs_ok(int64_t tokens, int64_t top_k, int64_t experts) {
    return tokens >= 0 && top_k >= 1 && top_k <= SGEMM_TOP_K_MAX && experts >= 1 && experts <= SGEMM_EXPERTS_MAX &&
           tokens <= INT32_MAX / top_k;
}

}  // namespace
}  // namespace ex
}  // namespace sgemm

using namespace sgemm;
using namespace sgemm::ex;
using namespace sgemm::api;

extern "C" {

size_t sgemm_experts_sort_workspace(int64_t pairs, int64_t experts) {
    if (pairs < 0 || pairs > INT32_MAX || experts < 1 || experts > SGEMM_EXPERTS_MAX) return 0;
    return static_cast<size_t>(sort_blocks(pairs, experts)) * static_cast<size_t>(experts + 1) * sizeof(int32_t);
}

int sgemm_experts_sort(const void *ids, int id_bits, int64_t tokens, int64_t top_k, int64_t experts,
                       int32_t *offsets, int32_t *order, int32_t *slot, void *workspace, size_t workspace_bytes,
                       sgemm_stream_t stream) {
    if (!pairs_ok(tokens, top_k, experts) || (id_bits != 32 && id_bits != 64)) return SGEMM_ERR_INVALID_ARG;
    const int64_t pairs = tokens * top_k;
    const size_t need = sgemm_experts_sort_workspace(pairs, experts);
    const Span in = flat(ids, pairs, id_bits / 8), off = flat(offsets, experts + 1, 4), ord = flat(order, pairs, 4),
               slo = flat(slot, pairs, 4), ws = flat(workspace, static_cast<int64_t>(need), 16);
    if (!in.ok() || !off.ok() || !ord.ok() || !slo.ok() || !ws.ok() || workspace_bytes < need)
        return SGEMM_ERR_INVALID_ARG;
    const Span wsb = flat(workspace, static_cast<int64_t>(need), 1);
    if (off.overlaps(in) || ord.overlaps(in) || slo.overlaps(in) || off.overlaps(ord) || off.overlaps(slo) ||
        ord.overlaps(slo) || wsb.overlaps(in) || wsb.overlaps(off) || wsb.overlaps(ord) || wsb.overlaps(slo))
        return SGEMM_ERR_INVALID_ARG;
    return enqueue([&](const DeviceInfo &dev, int *launches) {
        return sort_launch(ids, id_bits, pairs, experts, offsets, order, slot, static_cast<int32_t *>(workspace), dev,
                           reinterpret_cast<cudaStream_t>(stream), launches);
    });
}

int sgemm_experts_gather(int type, int64_t tokens, int64_t top_k, int64_t experts, int64_t width, const void *x,
                         int64_t ldx, const int32_t *slot, const int32_t *offsets, void *xs, int64_t ldxs,
                         sgemm_stream_t stream) {
    if (!type_ok(type) || !pairs_ok(tokens, top_k, experts) || width < 0) return SGEMM_ERR_INVALID_ARG;
    const int64_t size = type_size(type), pairs = tokens * top_k;
    const Span in{x, tokens, width, ldx, size}, out{xs, pairs, width, ldxs, size}, slo = flat(slot, pairs, 4),
        off = flat(offsets, experts + 1, 4);
    if (!in.ok() || !out.ok() || !slo.ok() || !off.ok()) return SGEMM_ERR_INVALID_ARG;
    if (out.overlaps(in) || out.overlaps(slo) || out.overlaps(off)) return SGEMM_ERR_INVALID_ARG;
    const Route r{tokens, top_k, experts, width, slot, offsets};
    return enqueue([&](const DeviceInfo &dev, int *launches) {
        if (out.empty()) return static_cast<int>(SGEMM_OK);
        return gather_launch(type, r, x, ldx, xs, ldxs, dev, reinterpret_cast<cudaStream_t>(stream), launches);
    });
}

int sgemm_experts_combine(int type, int64_t tokens, int64_t top_k, int64_t experts, int64_t width, const void *h,
                          int64_t ldh, const float *weights, const int32_t *slot, const int32_t *offsets, void *y,
                          int64_t ldy, sgemm_stream_t stream) {
    if (!type_ok(type) || !pairs_ok(tokens, top_k, experts) || width < 0) return SGEMM_ERR_INVALID_ARG;
    const int64_t size = type_size(type), pairs = tokens * top_k;
    const Span in{h, pairs, width, ldh, size}, out{y, tokens, width, ldy, size}, slo = flat(slot, pairs, 4),
        off = flat(offsets, experts + 1, 4), w = flat(weights, weights ? pairs : 0, 4);
    if (!in.ok() || !out.ok() || !slo.ok() || !off.ok() || !w.ok()) return SGEMM_ERR_INVALID_ARG;
    if (out.overlaps(in) || out.overlaps(slo) || out.overlaps(off) || out.overlaps(w)) return SGEMM_ERR_INVALID_ARG;
    const Route r{tokens, top_k, experts, width, slot, offsets};
    return enqueue([&](const DeviceInfo &dev, int *launches) {
        if (out.empty()) return static_cast<int>(SGEMM_OK);
        return combine_launch(type, r, h, ldh, weights, y, ldy, dev, reinterpret_cast<cudaStream_t>(stream), launches);
    });
}

int sgemm_experts_combine_grad(int type, int64_t tokens, int64_t top_k, int64_t experts, int64_t width,
                               const void *dy, int64_t lddy, const void *h, int64_t ldh, const float *weights,
                               const int32_t *slot, const int32_t *offsets, void *dh, int64_t lddh,
                               float *dweights, sgemm_stream_t stream) {
    if (!type_ok(type) || !pairs_ok(tokens, top_k, experts) || width < 0) return SGEMM_ERR_INVALID_ARG;
    const int64_t size = type_size(type), pairs = tokens * top_k;
    const Span g{dy, tokens, width, lddy, size}, in{h, pairs, width, ldh, size}, out{dh, pairs, width, lddh, size},
        slo = flat(slot, pairs, 4), off = flat(offsets, experts + 1, 4), w = flat(weights, pairs, 4),
        dw = flat(dweights, pairs, 4);
    if (!g.ok() || !in.ok() || !out.ok() || !slo.ok() || !off.ok() || !w.ok() || !dw.ok())
        return SGEMM_ERR_INVALID_ARG;
    if (out.overlaps(g) || out.overlaps(in) || out.overlaps(slo) || out.overlaps(off) || out.overlaps(w) ||
        dw.overlaps(g) || dw.overlaps(in) || dw.overlaps(slo) || dw.overlaps(off) || dw.overlaps(w) ||
        out.overlaps(dw))
        return SGEMM_ERR_INVALID_ARG;
    const Route r{tokens, top_k, experts, width, slot, offsets};
    return enqueue([&](const DeviceInfo &dev, int *launches) {
        if (dw.empty()) return static_cast<int>(SGEMM_OK);
        return combine_grad_launch(type, r, dy, lddy, h, ldh, weights, dh, lddh, dweights, dev,
                                   reinterpret_cast<cudaStream_t>(stream), launches);
    });
}

int sgemm_experts_gemm(int type, int transB, int64_t rows, int64_t N, int64_t K, int64_t experts,
                       const int32_t *offsets, const void *A, int64_t lda, const void *B, int64_t ldb,
                       int64_t strideB, void *C, int64_t ldc, sgemm_stream_t stream) {
    if (!type_ok(type) || (transB != SGEMM_OP_N && transB != SGEMM_OP_T) || rows < 0 || rows > kMostRows || N < 0 ||
        K < 0 || experts < 1 || experts > SGEMM_EXPERTS_MAX)
        return SGEMM_ERR_INVALID_ARG;
    const int64_t size = type_size(type);
    const Span a{A, rows, K, lda, size}, c{C, rows, N, ldc, size}, off = flat(offsets, experts + 1, 4),
        b{B, transB ? N : K, transB ? K : N, ldb, size, experts, strideB};
    if (!a.ok() || !b.ok() || !c.ok() || !off.ok()) return SGEMM_ERR_INVALID_ARG;
    if (c.overlaps(a) || c.overlaps(b) || c.overlaps(off)) return SGEMM_ERR_INVALID_ARG;
    GroupedProblem p{};
    p.wgrad = false;
    p.type = type;
    p.transB = transB;
    p.rows = rows;
    p.M = rows;
    p.N = N;
    p.K = K;
    p.experts = experts;
    p.offsets = offsets;
    p.A = A;
    p.lda = lda;
    p.B = B;
    p.ldb = ldb;
    p.strideB = strideB;
    p.C = C;
    p.ldc = ldc;
    return enqueue([&](const DeviceInfo &dev, int *launches) {
        if (c.empty()) return static_cast<int>(SGEMM_OK);
        return grouped_launch(p, dev, reinterpret_cast<cudaStream_t>(stream), launches);
    });
}

int sgemm_experts_gemm_wgrad(int type, int64_t rows, int64_t M, int64_t N, int64_t experts, const int32_t *offsets,
                             const void *A, int64_t lda, const void *B, int64_t ldb, void *C, int64_t ldc,
                             int64_t strideC, sgemm_stream_t stream) {
    if (!type_ok(type) || rows < 0 || rows > kMostRows || M < 0 || N < 0 || experts < 1 ||
        experts > SGEMM_EXPERTS_MAX)
        return SGEMM_ERR_INVALID_ARG;
    const int64_t size = type_size(type);
    const Span a{A, rows, M, lda, size}, b{B, rows, N, ldb, size}, off = flat(offsets, experts + 1, 4),
        c{C, M, N, ldc, size, experts, strideC};
    if (!a.ok() || !b.ok() || !c.ok() || !off.ok()) return SGEMM_ERR_INVALID_ARG;
    if (c.overlaps(a) || c.overlaps(b) || c.overlaps(off)) return SGEMM_ERR_INVALID_ARG;
    GroupedProblem p{};
    p.wgrad = true;
    p.type = type;
    p.rows = rows;
    p.M = M;
    p.N = N;
    p.K = rows;
    p.experts = experts;
    p.offsets = offsets;
    p.A = A;
    p.lda = lda;
    p.B = B;
    p.ldb = ldb;
    p.C = C;
    p.ldc = ldc;
    p.strideC = strideC;
    return enqueue([&](const DeviceInfo &dev, int *launches) {
        if (c.empty()) return static_cast<int>(SGEMM_OK);
        return grouped_launch(p, dev, reinterpret_cast<cudaStream_t>(stream), launches);
    });
}

int sgemm_w4_matvec(int type, int64_t rows, int64_t N, int64_t K, int64_t group, int64_t experts,
                    const int32_t *ids, const void *x, int64_t ldx, const uint8_t *q, const void *scales,
                    int scale_type, const uint8_t *zeros, void *y, int64_t ldy, sgemm_stream_t stream) {
    if (!type_ok(type) || !type_ok(scale_type) || rows < 0 || rows > SGEMM_W4_ROWS_MAX || N < 0 || K < 0 ||
        K % 2 != 0 || K > INT32_MAX || (group != 32 && group != 64 && group != 128 && group != 256) || experts < 1 ||
        experts > SGEMM_EXPERTS_MAX || (!ids && experts != 1))
        return SGEMM_ERR_INVALID_ARG;
    const int64_t size = type_size(type), groups = (K + group - 1) / group;
    if (N > kLimit / (K + 1) / experts) return SGEMM_ERR_INVALID_ARG;
    const Span in{x, rows, K, ldx, size}, out{y, rows, N, ldy, size}, w = flat(q, experts * N * (K / 2), 1),
        s = flat(scales, experts * N * groups, type_size(scale_type)),
        z = flat(zeros, zeros ? experts * N * groups : 0, 1), id = flat(ids, ids ? rows : 0, 4);
    if (!in.ok() || !out.ok() || !w.ok() || !s.ok() || !z.ok() || !id.ok()) return SGEMM_ERR_INVALID_ARG;
    if (out.overlaps(in) || out.overlaps(w) || out.overlaps(s) || out.overlaps(z) || out.overlaps(id))
        return SGEMM_ERR_INVALID_ARG;
    const W4Problem p{type, scale_type, rows, N, K, group, experts, ids, x, ldx, q, scales, zeros, y, ldy};
    return enqueue([&](const DeviceInfo &dev, int *launches) {
        if (out.empty()) return static_cast<int>(SGEMM_OK);
        return w4_launch(p, dev, reinterpret_cast<cudaStream_t>(stream), launches);
    });
}

}  // extern "C"
