// Internal declarations of the mixture-of-experts layer for a few tokens (the
// public ABI is include/layer.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "experts_internal.h"
#include "layer.h"

namespace sgemm {
namespace fl {

constexpr int MAX_PAIRS = SGEMM_LAYER_PAIRS_MAX;

// Floats between the workspace's rows (one per pair).
inline int64_t h_stride(int64_t hidden) { return (hidden + 3) / 4 * 4; }

struct LayerProblem {
    int type, held, activation, gated;
    int64_t tokens, top_k, experts, width, hidden;
    const void *x;
    int64_t ldx;
    const void *ids;
    int id_bits;
    const float *weights;
    const void *w1;
    int64_t ld1, stride1;
    const float *s1;
    const void *w2;
    int64_t ld2, stride2;
    const float *s2;
    void *y;
    int64_t ldy;
    float *h;
};
int layer_launch(const LayerProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches);

}  // namespace fl
}  // namespace sgemm
