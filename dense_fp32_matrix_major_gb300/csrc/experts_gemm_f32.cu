// Products per expert in fp32: launcher of the tensor-core SGEMM kernel on SM
// pairs (tf32x3_pair.cuh) over row groups. Accuracy and the treatment of
// infinities and NaN are that kernel's. Bound by shared memory (operand tiles,
// their split, folds) where groups are long: 8192 rows, 8 experts, 1024 -> 2048
// 170 us (202 TFLOP/s, of 320 with three TF32 products for one; 154 us where groups
// are even, their gradient of the matrices 149 us); by reading and splitting B,
// which goes through registers value by value however few rows there are, where
// they are short: 64 rows, two for each of 32 experts, 2048 -> 2048 137 us (3.9 TB/s).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "experts_internal.h"
#include "tf32x3_pair.cuh"

namespace sgemm {
namespace ex {
namespace {

constexpr int kMaxDevices = 64;
std::once_flag g_once[kMaxDevices][9];
cudaError_t g_err[kMaxDevices][9];
int g_clusters[kMaxDevices][9];

// Folds of the accumulators. The tensor core cuts its running sum at every MMA
// (half a unit of the last place on average, towards zero), so the error grows
// with the MMAs that add to a large running sum. The single product folds every
// 8 k-blocks, 96 such MMAs: 2.0e-6 of the result's norm on normal inputs, where
// fp32 sums give 0.57e-6 at K = 1024. Here a fold every 5 k-blocks, the small
// products (lo hi, hi lo) of the first 4 before any large one, leaves 28: 0.7e-6.
// Folds move the tile through shared memory and held stages are not refilled:
// 8192 rows, 8 experts, 1024 -> 2048 took 179 us (now 170); 4 k-blocks with 3
// ahead 187 us (0.64e-6), 6 with 4 ahead 175 us (0.98e-6), 6 with 3 ahead 171 us
// (1.15e-6).
constexpr int GROUP_FOLD = 5, GROUP_LEAD = 4;

template <bool VEC_C, bool TA, bool TB, PairUnits UNITS>
int launch(const GroupedProblem &p, const Problem &q, bool cpa, const DeviceInfo &dev, cudaStream_t stream,
           int *launches) {
    auto kernel = tf32x3_pair_kernel<VEC_C, TA, TB, UNITS, GROUP_FOLD, GROUP_LEAD>;
    constexpr bool WG = sums_rows(UNITS), COLS = transposed(UNITS);
    constexpr int idx = COLS ? 6 + (WG ? 2 : TA ? 1 : 0) : (VEC_C ? 3 : 0) + (WG ? 2 : TB ? 1 : 0);
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
    std::call_once(g_once[dev.device][idx], [&] {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, pr::SMEM_BYTES);
        int n = 0;
        if (e == cudaSuccess) {
            cudaLaunchConfig_t c = cfg;
            c.gridDim = dim3(2 * (dev.sm_count / 2));
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &c);
        }
        g_err[dev.device][idx] = e;
        g_clusters[dev.device][idx] = n;
    });
    const int clusters = g_clusters[dev.device][idx];
    int *flag = watchdog_flag_device_ptr();
    if (g_err[dev.device][idx] != cudaSuccess || clusters < 1 || !flag) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B, plain = CU_TENSOR_MAP_SWIZZLE_NONE;
    alignas(64) CUtensorMap mapA{}, mapB{}, mapC{};
    if (!cpa) {
        const bool ok =
            WG && COLS ? encode_map(&mapA, q.B, p.rows, p.N, q.ldb, 1, 0, 32, 32, sw) &&
                             encode_map(&mapB, q.A, p.rows, p.M, q.lda, 1, 0, pr::HN, BK, plain)
            : COLS ? (TA ? encode_map(&mapA, q.B, p.K, p.N, q.ldb, p.experts, q.strideB, 32, 32, sw)
                       : encode_map(&mapA, q.B, p.N, p.K, q.ldb, p.experts, q.strideB, BK, pr::HM, sw)) &&
                       encode_map(&mapB, q.A, p.rows, p.K, q.lda, 1, 0, BK, pr::HN, sw)
            : WG ? encode_map(&mapA, q.A, p.rows, p.M, q.lda, 1, 0, 32, 32, sw) &&
                     encode_map(&mapB, q.B, p.rows, p.N, q.ldb, 1, 0, pr::HN, BK, plain)
               : encode_map(&mapA, q.A, p.rows, p.K, q.lda, 1, 0, BK, pr::HM, sw) &&
                     (TB ? encode_map(&mapB, q.B, p.N, p.K, q.ldb, p.experts, q.strideB, BK, pr::HN, sw)
                         : encode_map(&mapB, q.B, p.K, p.N, q.ldb, p.experts, q.strideB, pr::HN, BK, plain));
        if (!ok) return SGEMM_ERR_LAUNCH;
    }
    const int64_t c_rows = WG ? p.M : p.rows, c_items = WG ? p.experts * p.split : 1;
    const int64_t c_stride = c_items > 1 ? p.strideC : 0;
    const bool c_tma = !COLS && VEC_C && tma_operand_ok(q.C, p.ldc, c_stride, c_rows, c_items) &&
                       encode_map(&mapC, q.C, c_rows, p.N, p.ldc, c_items, c_stride, 32, 32, sw);
    if (!c_tma) mapC = mapA;  // not read by the kernel

    const int64_t wide = COLS ? pr::PM : pr::PN, high = COLS ? pr::PN : pr::PM;  // of a tile of C
    const int64_t tiles_n = (p.N + wide - 1) / wide, tiles_m = WG ? (p.M + high - 1) / high : 1;
    if (tiles_m * tiles_n > INT32_MAX / 2) return SGEMM_ERR_UNSUPPORTED;
    Args a{};
    a.M = COLS ? p.N : p.M;
    a.N = COLS ? p.M : p.N;
    a.K = p.K;
    a.A = COLS ? q.B : q.A;
    a.lda = COLS ? q.ldb : q.lda;
    a.strideA = COLS ? q.strideB : 0;
    a.B = COLS ? q.A : q.B;
    a.ldb = COLS ? q.lda : q.ldb;
    a.strideB = COLS ? 0 : q.strideB;
    a.C = q.C;
    a.ldc = p.ldc;
    a.strideC = c_stride;
    a.cpa = cpa ? 1 : 0;
    a.ta = TA ? 1 : 0;
    a.tb = TB ? 1 : 0;
    a.c_tma = c_tma ? 1 : 0;
    a.timeout_ns = static_cast<uint64_t>(watchdog_ms()) * 1000000ull;
    a.watchdog = flag;
    const GroupTiles gt{p.offsets,
                        static_cast<int>(p.rows),
                        static_cast<int>(p.experts),
                        WG ? p.M : 0,
                        p.K,
                        static_cast<int>(tiles_m),
                        static_cast<int>(tiles_n),
                        p.split};
    // Every group may end in a part of a tile, and so may the rest.
    const int64_t units =
        WG ? tiles_m * tiles_n * p.experts * p.split : ((p.rows + high - 1) / high + p.experts) * tiles_n;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (units < clusters ? units : clusters)));
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, mapA, mapB, mapC, a, gt) != cudaSuccess) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    ++*launches;
    return SGEMM_OK;
}

// Whether the rows of C are the MMA's narrow side (C^T: 256 columns of C a
// tile, rows by the 32) or its wide side (128 columns a tile, rows by the 256):
// what a call is charged, with groups that end half a step short on average.
// Narrow (C^T from registers) against wide (C through TMA): 168 and 179 us (8192
// rows, 8 experts, 2048 -> 1024), 113 and 275 us (64 rows, 32 experts, 2048 ->
// 2048; the matrices alone are 79 us of DRAM); for 8192 rows, 8 experts, 1024 ->
// 128, where half of a narrow tile would be columns of nothing, wide takes 40 us.
// wgrad: 158 and 183 us for groups of two rows, 179 and 175 us for groups of 1024
// (narrow 149 us since no sums are repaired among the folds).
bool rows_narrow(const GroupedProblem &p) {
    auto charged = [&](int64_t step) {
        return p.wgrad ? (p.M + step - 1) / step * step : p.rows + p.experts * step / 2;
    };
    const int64_t narrow = (p.N + pr::PM - 1) / pr::PM * pr::PM * charged(pr::COL_STEP);
    const int64_t wide = (p.N + pr::PN - 1) / pr::PN * pr::PN * charged(pr::PM);
    return narrow <= wide;
}

// Operands that tensor maps cannot describe are either copied into aligned rows
// first or loaded by the kernel with 4-byte copies, which take it 6 us a k-block.
// What the busiest pair's k-blocks would cost that way against the copies' time.
// Copied and loaded: 92 and 541 us (1745 rows, 64 experts, 2761 -> 35, B stored 35 x
// 2761; 257 us stored 2761 x 35, whose short rows a block copies one by one), 58 and
// 218 us (2000 rows, 8 experts, 1001 -> 1001); 905 and 232 us (5 rows, 64
// experts, 2047 -> 2047: the copy takes every expert's matrix).
bool copy_first(const GroupedProblem &p, size_t bytes, const DeviceInfo &dev) {
    int64_t high, wide;
    grouped_f32_tile(p, &high, &wide);
    const int64_t tiles_n = (p.N + wide - 1) / wide, workers = dev.sm_count / 2;
    const int64_t tiles_m = p.wgrad ? (p.M + high - 1) / high * p.experts * p.split
                                    : (p.rows + high - 1) / high + (p.rows < p.experts ? p.rows : p.experts) / 2;
    const int64_t depth = p.wgrad ? p.rows / (p.experts * p.split) + 1 : p.K;
    const double k_blocks = static_cast<double>((tiles_m * tiles_n + workers - 1) / workers) *
                            static_cast<double>((depth + BK - 1) / BK);
    return 2.0 * static_cast<double>(bytes) / 5e6 + 10.0 < 5.5 * k_blocks;
}

template <bool VEC_C>
int launch_form(const GroupedProblem &p, const Problem &q, bool cpa, const DeviceInfo &dev, cudaStream_t stream,
                int *launches) {
    if (rows_narrow(p)) {
        if (p.wgrad) return launch<true, true, false, GROUP_WGRAD_COLS>(p, q, cpa, dev, stream, launches);
        return p.transB == SGEMM_OP_T ? launch<true, false, true, GROUP_COLS>(p, q, cpa, dev, stream, launches)
                                      : launch<true, true, true, GROUP_COLS>(p, q, cpa, dev, stream, launches);
    }
    if (p.wgrad) return launch<VEC_C, true, false, GROUP_WGRAD>(p, q, cpa, dev, stream, launches);
    return p.transB == SGEMM_OP_T ? launch<VEC_C, false, true, GROUP_ROWS>(p, q, cpa, dev, stream, launches)
                                  : launch<VEC_C, false, false, GROUP_ROWS>(p, q, cpa, dev, stream, launches);
}

}  // namespace

// Sizes that fit tensor map coordinates, and a sum to make.
bool grouped_f32_supports(const GroupedProblem &p) {
    const int64_t lim = INT32_MAX / 2;
    return p.type == SGEMM_TYPE_F32 && p.rows > 0 && p.rows < lim && p.M < lim && p.N < lim && p.K < lim &&
           (p.wgrad || p.K > 0);
}

void grouped_f32_tile(const GroupedProblem &p, int64_t *high, int64_t *wide) {
    const bool narrow = rows_narrow(p);
    *high = narrow ? pr::PN : pr::PM;
    *wide = narrow ? pr::PM : pr::PN;
}

int grouped_f32_launch(const GroupedProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    if (dev.device < 0 || dev.device >= kMaxDevices) return SGEMM_ERR_DEVICE;
    // The operands as the library's single product describes them: A stored
    // rows x M and B rows x N, summed along the rows, or A rows x K and one B
    // per group.
    Problem q{};
    q.M = p.M;
    q.N = p.N;
    q.K = p.K;
    q.A = static_cast<const float *>(p.A);
    q.lda = p.lda;
    q.B = static_cast<const float *>(p.B);
    q.ldb = p.ldb;
    q.C = static_cast<float *>(p.C);
    q.ldc = p.ldc;
    q.transA = p.wgrad ? SGEMM_OP_T : SGEMM_OP_N;
    q.transB = p.wgrad ? SGEMM_OP_N : p.transB;
    q.batch = p.wgrad ? 1 : p.experts;
    q.strideB = q.batch > 1 ? p.strideB : 0;
    const int64_t b_rows = q.transB == SGEMM_OP_T ? q.N : q.K;
    bool cpa = !tma_operand_ok(q.A, q.lda, 0, p.rows, 1) || !tma_operand_ok(q.B, q.ldb, q.strideB, b_rows, q.batch);
    float *scratch = nullptr;
    const size_t bytes = cpa ? repack_bytes(q) : 0;
    if (cpa && copy_first(p, bytes, dev)) {
        scratch = scratch_alloc(dev, bytes, stream);
        if (scratch) {
            Problem copied;
            const int rc = repack_into(q, dev, scratch, bytes, stream, &copied, launches);
            if (rc != SGEMM_OK) {
                scratch_free(scratch, stream);
                return rc;
            }
            q = copied;
            cpa = false;
        }
    }
    const bool vec_c = p.ldc % 4 == 0 && reinterpret_cast<uintptr_t>(p.C) % 16 == 0 &&
                       (!p.wgrad || p.experts * p.split == 1 || p.strideC % 4 == 0);
    const int rc = vec_c ? launch_form<true>(p, q, cpa, dev, stream, launches)
                         : launch_form<false>(p, q, cpa, dev, stream, launches);
    scratch_free(scratch, stream);
    return rc;
}

}  // namespace ex
}  // namespace sgemm
