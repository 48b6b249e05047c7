// C ABI of the mixture-of-experts layer for a few tokens: argument checks and
// dispatch. The contract of every entry point is in layer.h.
#include <cuda_runtime.h>
#include <stdint.h>

#include "api_checks.h"
#include "layer_internal.h"

namespace sgemm {
namespace fl {

int layer_launch(const LayerProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    const int64_t per_x = 16 / ex::type_size(p.type);
    LArgs a{};
    a.pairs = static_cast<int>(p.tokens * p.top_k);
    a.top_k = static_cast<int>(p.top_k);
    a.experts = static_cast<int>(p.experts);
    a.tokens = static_cast<int>(p.tokens);
    a.activation = p.activation;
    a.gated = p.gated;
    a.width = static_cast<int>(p.width);
    a.hidden = static_cast<int>(p.hidden);
    a.x = p.x;
    a.ldx = p.ldx;
    a.x_size = static_cast<int>(ex::type_size(p.type));
    a.x_type = p.type;
    a.x_vector = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && (p.tokens == 1 || p.ldx % per_x == 0);
    a.ids = p.ids;
    a.id_bits = p.id_bits;
    a.weights = p.weights;
    a.w1 = p.w1;
    a.ld1 = p.ld1;
    a.stride1 = p.experts > 1 ? p.stride1 : 0;
    a.s1 = p.s1;
    a.w2 = p.w2;
    a.ld2 = p.ld2;
    a.stride2 = p.experts > 1 ? p.stride2 : 0;
    a.s2 = p.s2;
    a.y = p.y;
    a.ldy = p.ldy;
    a.h = p.h;
    a.ldh = h_stride(p.hidden);
    if (p.type == SGEMM_TYPE_F32) return layer_launch_f32(p, a, dev, stream, launches);
    if (p.held == SGEMM_LAYER_SAME) return layer_launch_16(p, a, dev, stream, launches);
    return layer_launch_fp8(p, a, dev, stream, launches);
}

}  // namespace fl
}  // namespace sgemm

using namespace sgemm;
using namespace sgemm::api;
using namespace sgemm::fl;

extern "C" {

size_t sgemm_experts_layer_workspace(int64_t tokens, int64_t top_k, int64_t hidden) {
    if (tokens < 0 || top_k < 1 || top_k > SGEMM_TOP_K_MAX || tokens > MAX_PAIRS / top_k || hidden < 0 ||
        hidden > kMostHidden)
        return 0;
    return static_cast<size_t>(tokens * top_k * h_stride(hidden)) * sizeof(float);
}

int sgemm_experts_layer(int type, int held, int activation, int gated, int64_t tokens, int64_t top_k,
                        int64_t experts, int64_t width, int64_t hidden, const void *x, int64_t ldx, const void *ids,
                        int id_bits, const float *weights, const void *W1, int64_t ld1, int64_t stride1,
                        const float *s1, const void *W2, int64_t ld2, int64_t stride2, const float *s2, void *y,
                        int64_t ldy, void *workspace, size_t workspace_bytes, sgemm_stream_t stream) {
    if (!type_ok(type) || held < SGEMM_LAYER_SAME || held > SGEMM_LAYER_E5M2 || activation < SGEMM_ACT_NONE ||
        activation > SGEMM_ACT_SILU || tokens < 0 || top_k < 1 || top_k > SGEMM_TOP_K_MAX ||
        tokens > MAX_PAIRS / top_k || experts < 1 || experts > SGEMM_EXPERTS_MAX || width < 0 || width > kMostRows ||
        hidden < 0 || hidden > kMostHidden || (id_bits != 32 && id_bits != 64))
        return SGEMM_ERR_INVALID_ARG;
    const int64_t pairs = tokens * top_k, rows1 = gated ? 2 * hidden : hidden;
    const bool fp8 = held != SGEMM_LAYER_SAME;
    const int64_t size = ex::type_size(type), wsize = fp8 ? 1 : size;
    auto blocks = [](int64_t n) { return (n + SGEMM_FP8_BLOCK_SIZE - 1) / SGEMM_FP8_BLOCK_SIZE; };
    const size_t need = sgemm_experts_layer_workspace(tokens, top_k, hidden);
    const Span in{x, tokens, width, ldx, size}, id = flat(ids, pairs, id_bits / 8), w = flat(weights, pairs, 4),
        m1{W1, rows1, width, ld1, wsize, experts, stride1}, m2{W2, width, hidden, ld2, wsize, experts, stride2},
        c1 = flat(s1, fp8 ? experts * blocks(rows1) * blocks(width) : 0, 4),
        c2 = flat(s2, fp8 ? experts * blocks(width) * blocks(hidden) : 0, 4), out{y, tokens, width, ldy, size},
        ws = flat(workspace, static_cast<int64_t>(need / 16), 16);
    if (!in.ok() || !id.ok() || !w.ok() || !m1.ok() || !m2.ok() || !c1.ok() || !c2.ok() || !out.ok() || !ws.ok() ||
        workspace_bytes < need)
        return SGEMM_ERR_INVALID_ARG;
    // Rows of 8-bit matrices start on 16-byte boundaries, as sgemm_fp8_gemm wants them.
    for (const Span *s : {&m1, &m2})
        if (fp8 && !s->empty() && (s->begin() % 16 != 0 || s->ld % 16 != 0 || (experts > 1 && s->stride % 16 != 0)))
            return SGEMM_ERR_INVALID_ARG;
    for (const Span *s : {&in, &id, &w, &m1, &m2, &c1, &c2})
        if (out.overlaps(*s) || ws.overlaps(*s)) return SGEMM_ERR_INVALID_ARG;
    if (out.overlaps(ws)) return SGEMM_ERR_INVALID_ARG;
    const LayerProblem p{type, held,    activation, gated != 0, tokens, top_k, experts, width, hidden, x,
                         ldx,  ids,     id_bits,    weights,    W1,     ld1,   stride1, s1,    W2,     ld2,
                         stride2, s2,   y,          ldy,        static_cast<float *>(workspace)};
    return enqueue([&](const DeviceInfo &dev, int *launches) {
        if (out.empty()) return static_cast<int>(SGEMM_OK);
        return layer_launch(p, dev, reinterpret_cast<cudaStream_t>(stream), launches);
    });
}

}  // extern "C"
