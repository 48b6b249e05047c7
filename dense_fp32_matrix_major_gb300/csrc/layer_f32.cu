// The layer for a few tokens with fp32 x: multiply-adds on fp32 or 8-bit matrices.
#include "layer_few.cuh"

namespace sgemm {
namespace fl {

int layer_launch_f32(const LayerProblem &p, const LArgs &a, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    if (p.held == SGEMM_LAYER_E4M3) return launch_layer<E4M3, FMA, FMA, float>(p, a, dev, stream, launches);
    if (p.held == SGEMM_LAYER_E5M2) return launch_layer<E5M2, FMA, FMA, float>(p, a, dev, stream, launches);
    return launch_layer<F32, FMA, FMA, float>(p, a, dev, stream, launches);
}

}  // namespace fl
}  // namespace sgemm
