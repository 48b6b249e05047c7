// The layer for a few tokens with bf16 or fp16 x and 8-bit matrices.
#include "layer_few.cuh"

namespace sgemm {
namespace fl {

int layer_launch_fp8(const LayerProblem &p, const LArgs &a, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    const bool bf16 = p.type == SGEMM_TYPE_BF16;
    if (p.held == SGEMM_LAYER_E4M3)
        return bf16 ? launch_layer<E4M3, BF8, BF8_H, __nv_bfloat16>(p, a, dev, stream, launches)
                    : launch_layer<E4M3, HALF8, BF8_H, __half>(p, a, dev, stream, launches);
    return bf16 ? launch_layer<E5M2, BF8, BF8_H, __nv_bfloat16>(p, a, dev, stream, launches)
                : launch_layer<E5M2, HALF8, BF8_H, __half>(p, a, dev, stream, launches);
}

}  // namespace fl
}  // namespace sgemm
