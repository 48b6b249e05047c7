// The layer for a few tokens with bf16 or fp16 x and matrices.
#include "layer_few.cuh"

namespace sgemm {
namespace fl {

int layer_launch_16(const LayerProblem &p, const LArgs &a, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    if (p.type == SGEMM_TYPE_BF16)
        return launch_layer<BF16, NATIVE, PLANES, __nv_bfloat16>(p, a, dev, stream, launches);
    return launch_layer<F16, NATIVE, TF32_H, __half>(p, a, dev, stream, launches);
}

}  // namespace fl
}  // namespace sgemm
