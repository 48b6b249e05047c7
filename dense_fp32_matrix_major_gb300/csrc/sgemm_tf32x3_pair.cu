// Launcher of the tensor-core SGEMM on SM pairs; the kernel and its design are
// in tf32x3_pair.cuh.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "sgemm.h"
#include "sgemm_internal.h"
#include "tf32x3_pair.cuh"

namespace sgemm {
namespace {

constexpr int kMaxDevices = 64;
std::once_flag g_pair_once[kMaxDevices][8];
cudaError_t g_pair_err[kMaxDevices][8];
int g_pair_clusters[kMaxDevices][8];

template <bool VEC_C, bool TA, bool TB>
int launch_pair(const Problem &p, const DeviceInfo &dev, int sk_mode, bool cpa, bool after_copy, cudaStream_t stream,
                int *launches) {
    auto kernel = tf32x3_pair_kernel<VEC_C, TA, TB>;
    constexpr int idx = (VEC_C ? 1 : 0) + (TA ? 2 : 0) + (TB ? 4 : 0);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(pr::THREADS);
    cfg.dynamicSmemBytes = pr::SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    std::call_once(g_pair_once[dev.device][idx], [&] {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, pr::SMEM_BYTES);
        int n = 0;
        if (e == cudaSuccess) {
            cudaLaunchConfig_t q = cfg;
            q.gridDim = dim3(2 * (dev.sm_count / 2));
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &q);
        }
        g_pair_err[dev.device][idx] = e;
        g_pair_clusters[dev.device][idx] = n;
    });
    const int clusters = g_pair_clusters[dev.device][idx];
    if (g_pair_err[dev.device][idx] != cudaSuccess || clusters < 1) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    int *flag = watchdog_flag_device_ptr();
    if (!flag) return SGEMM_ERR_LAUNCH;
    alignas(64) CUtensorMap mapA{}, mapB{}, mapC{};
    if (!cpa) {  // operands through TMA; otherwise the kernel's cp.async loaders read A and B
        const bool ok_a =
            TA ? encode_map(&mapA, p.A, p.K, p.M, p.lda, p.batch, p.strideA, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B)
               : encode_map(&mapA, p.A, p.M, p.K, p.lda, p.batch, p.strideA, BK, pr::HM, CU_TENSOR_MAP_SWIZZLE_128B);
        const bool ok_b =
            TB ? encode_map(&mapB, p.B, p.N, p.K, p.ldb, p.batch, p.strideB, BK, pr::HN, CU_TENSOR_MAP_SWIZZLE_128B)
               : encode_map(&mapB, p.B, p.K, p.N, p.ldb, p.batch, p.strideB, pr::HN, BK, CU_TENSOR_MAP_SWIZZLE_NONE);
        if (!ok_a || !ok_b) return SGEMM_ERR_LAUNCH;
    }
    // C through TMA when its rows allow 16-byte aligned boxes and C is not
    // read (beta = 0; split tiles are reduce-added either way).
    const bool c_tma = VEC_C && p.beta == 0.0f &&
                       encode_map(&mapC, p.C, p.M, p.N, p.ldc, p.batch, p.strideC, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B);
    if (!c_tma) mapC = mapA;  // not read by the kernel

    const int64_t tiles_m = (p.M + pr::PM - 1) / pr::PM, tiles_n = (p.N + pr::PN - 1) / pr::PN;
    const int64_t k_blocks = (p.K + BK - 1) / BK;
    if (tiles_m * tiles_n * p.batch > INT32_MAX / 2 || k_blocks > INT32_MAX / 2) return SGEMM_ERR_UNSUPPORTED;
    const int tiles = static_cast<int>(tiles_m * tiles_n * p.batch);
    // One pair per two SMs, as many pairs as fit at once. A stream-K share
    // below 4 k-blocks costs more in fix-up than it saves. Accumulation
    // chains are bounded by the folds inside the kernel, so units may span
    // any number of k-blocks.
    const Schedule sch = make_schedule(tiles, k_blocks, clusters, sk_mode, 4, 0.25);
    const int split = tiles - sch.dp_tiles;
    int rc = split_tiles_prepare(p, pr::PM, pr::PN, static_cast<int>(tiles_n), static_cast<int>(tiles_m * tiles_n),
                                 sch.dp_tiles, split, stream, launches);
    if (rc != SGEMM_OK) return rc;
    Args a{};
    a.M = p.M;
    a.N = p.N;
    a.K = p.K;
    a.A = p.A;
    a.lda = p.lda;
    a.B = p.B;
    a.ldb = p.ldb;
    a.cpa = cpa ? 1 : 0;
    a.ta = TA ? 1 : 0;
    a.tb = TB ? 1 : 0;
    a.C = p.C;
    a.ldc = p.ldc;
    a.tiles_n = static_cast<int>(tiles_n);
    a.k_blocks = static_cast<int>(k_blocks);
    a.dp_tiles = sch.dp_tiles;
    a.sk_ctas = sch.sk_ctas;
    a.sk_iters = sch.sk_iters;
    a.timeout_ns = wait_limit_ns(p.K);
    a.watchdog = flag;
    a.alpha = p.alpha;
    a.beta = p.beta;
    a.strideA = p.strideA;
    a.strideB = p.strideB;
    a.strideC = p.strideC;
    a.tiles_per_item = static_cast<int>(tiles_m * tiles_n);
    a.a_shared = p.strideA == 0;
    a.b_shared = p.strideB == 0;
    a.bias = p.bias;
    a.bias_kind = p.bias_kind;
    a.act = p.act;
    a.ep = p.has_epilogue();
    a.kb_cap = 0;
    a.sk_switch_kb = 0;  // a unit switch costs no MMA time: the accumulators alternate
    a.signal_dependents = (split > 0 && p.act != SGEMM_ACT_NONE) ? 1 : 0;
    a.c_tma = c_tma ? 1 : 0;
    cfg.gridDim = dim3(2 * sch.grid);
    // Behind our own beta pre-pass (which touches only C, and which started
    // after everything before it in the stream had finished) the main loop
    // may overlap it; the epilogue waits for it (griddepcontrol.wait).
    // Right behind the aligned copies of A and B the prologue overlaps them
    // and the loaders wait.
    a.wait_inputs = (after_copy && split == 0) ? 1 : 0;
    cfg.numAttrs = (split > 0 || a.wait_inputs) ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, mapA, mapB, mapC, a, ex::GroupTiles{}) != cudaSuccess) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    ++*launches;
    return split_tiles_finish(p, pr::PM, pr::PN, static_cast<int>(tiles_n), static_cast<int>(tiles_m * tiles_n),
                              sch.dp_tiles, split, stream, launches, a.signal_dependents != 0);
}

}  // namespace

int tf32x3_pair_launch(const Problem &p, const DeviceInfo &dev, int sk_mode, bool cpa, cudaStream_t stream,
                       int *launches, bool after_copy) {
    if (dev.device < 0 || dev.device >= kMaxDevices) return SGEMM_ERR_DEVICE;
    const bool vc = (p.ldc % 4 == 0) && (p.strideC % 4 == 0) && (reinterpret_cast<uintptr_t>(p.C) % 16 == 0);
    const int form = (vc ? 1 : 0) + (p.transA ? 2 : 0) + (p.transB ? 4 : 0);
    switch (form) {
        case 0: return launch_pair<false, false, false>(p, dev, sk_mode, cpa, after_copy, stream, launches);
        case 1: return launch_pair<true, false, false>(p, dev, sk_mode, cpa, after_copy, stream, launches);
        case 2: return launch_pair<false, true, false>(p, dev, sk_mode, cpa, after_copy, stream, launches);
        case 3: return launch_pair<true, true, false>(p, dev, sk_mode, cpa, after_copy, stream, launches);
        case 4: return launch_pair<false, false, true>(p, dev, sk_mode, cpa, after_copy, stream, launches);
        case 5: return launch_pair<true, false, true>(p, dev, sk_mode, cpa, after_copy, stream, launches);
        case 6: return launch_pair<false, true, true>(p, dev, sk_mode, cpa, after_copy, stream, launches);
        default: return launch_pair<true, true, true>(p, dev, sk_mode, cpa, after_copy, stream, launches);
    }
}

}  // namespace sgemm
