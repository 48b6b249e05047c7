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

// Hidden features: the tiles of 512 entries fit 32 bits.
constexpr int64_t kMostHidden = INT64_C(1) << 24;

// Floats between the workspace's rows (one per pair); half of a row is 16-byte aligned.
inline int64_t h_stride(int64_t hidden) { return (hidden + 7) / 8 * 8; }

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
// The kernels' arguments.
struct LArgs {
    int pairs, top_k, experts, tokens;
    int activation, gated;
    int width, hidden;
    const void *x;
    int64_t ldx;
    int x_size, x_type;  // bytes of a value; sgemm_type, y's too
    int x_vector;        // rows of x are 16-byte aligned
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
    int64_t ldh;  // rows of h: fp32, or with x of 16 bits two bf16 terms, the first ones and then the second
};

int layer_launch(const LayerProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches);
// By the type of x and how the matrices are held.
int layer_launch_f32(const LayerProblem &p, const LArgs &a, const DeviceInfo &dev, cudaStream_t stream, int *launches);
int layer_launch_16(const LayerProblem &p, const LArgs &a, const DeviceInfo &dev, cudaStream_t stream, int *launches);
int layer_launch_fp8(const LayerProblem &p, const LArgs &a, const DeviceInfo &dev, cudaStream_t stream, int *launches);

}  // namespace fl
}  // namespace sgemm
