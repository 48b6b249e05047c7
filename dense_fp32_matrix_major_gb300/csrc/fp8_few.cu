// Products of a few rows in 8-bit floating point: C = A B^T, A of at most 32
// rows, B N x K, with the scales of fp8_gemm.cu:
//
//     C[s][n] = sum over blocks b of sA[b][s] sB[n / 128][b] P_b[s][n]
//
// Bound by reading B once, and in short calls by the latency of that. A tile of
// fp8_gemm.cu covers 256 columns, which leaves most of the SMs without one; here
// a CTA takes 16 columns and its eight warps every eighth block of K, so that
// there are eight warps for every 16 columns, each with the next blocks' loads on
// their way (three blocks with 8 rows; one with more, whose registers A takes:
// 16 rows of 4096 x 4096 6.7 us, with two 7.4). A warp's sums over its blocks, in
// order, are joined in the warps' order. 8 rows of 16384 x 8192: 26 us, 5.1 TB/s
// of B. With loads that may meet the rows' end, each under a branch of its own, 35.
//
// Matrix instructions m16n8k32: 16 columns of C by 8 rows. The 32 values of k may
// be taken in any order that A and B share, so a thread's fragments are 16
// consecutive bytes of a row, loaded from memory straight into registers: 64
// bytes a row and load, each byte of B read once; A comes from L2. (tcgen05 wants
// both staged in shared memory and 128 columns of C a tile.)
#include <cuda_runtime.h>
#include <stdint.h>

#include "experts_common.cuh"
#include "fp8_internal.h"

namespace sgemm {
namespace f8 {
namespace {

constexpr int WARPS = 8, COLS = 16;

struct FewArgs {
    int rows, blocks;
    int64_t N, K;
    const uint8_t *A;
    int64_t lda;
    const float *sA;
    const uint8_t *B;
    int64_t ldb;
    const float *sB;
    void *C;
    int64_t ldc;
    int out_type;
};

// 16 bytes of B, read once.
__device__ __forceinline__ uint4 load_once(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The first n of 16 bytes, zeros for the others.
__device__ __forceinline__ uint4 load_part(const uint8_t *p, int64_t n) {
    if (n >= 16) return __ldg(reinterpret_cast<const uint4 *>(p));
    uint64_t lo = 0, hi = 0;
#pragma unroll 1
    for (int i = static_cast<int>(n) - 1; i >= 0; --i) {
        hi = (hi << 8) | (lo >> 56);
        lo = (lo << 8) | p[i];
    }
    return make_uint4(static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                      static_cast<uint32_t>(hi >> 32));
}

// d += a b; a: 16 columns of C (B's rows), b: 8 rows (A's).
template <bool A5, bool B5>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
#define SGEMM_MMA(TB, TA)                                                                        \
    asm("mma.sync.aligned.m16n8k32.row.col.f32." TB "." TA ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, " \
        "{%0, %1, %2, %3};"                                                                      \
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                         \
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
    if (A5 && B5) SGEMM_MMA("e5m2", "e5m2");
    if (A5 && !B5) SGEMM_MMA("e4m3", "e5m2");
    if (!A5 && B5) SGEMM_MMA("e5m2", "e4m3");
    if (!A5 && !B5) SGEMM_MMA("e4m3", "e4m3");
#undef SGEMM_MMA
}

// One block of K: its bytes of B and A and their factors.
template <int TILES>
struct Slot {
    uint4 b[2][2], x[TILES][2];
    float fb, fx[TILES][2];
};

// TILES: of 8 rows.
template <int TILES, bool A5, bool B5>
__global__ void __launch_bounds__(WARPS * 32, 2) fp8_few_kernel(const __grid_constant__ FewArgs a) {
    constexpr int SLOTS = TILES == 1 ? 3 : 1;  // blocks of a warp on their way
    __shared__ float part[WARPS][8 * TILES][COLS + 1];
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    const int g = lane >> 2, t = lane & 3;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * COLS;
    // Rows and columns past the end: the last one's, not written.
    const uint8_t *b[2], *x[TILES];
#pragma unroll
    for (int h = 0; h < 2; ++h) b[h] = a.B + min(n0 + 8 * h + g, a.N - 1) * a.ldb + 16 * t;
#pragma unroll
    for (int i = 0; i < TILES; ++i) x[i] = a.A + min(8 * i + g, a.rows - 1) * a.lda + 16 * t;
    const float *sb = a.sB + n0 / BLOCK * a.blocks;
    float acc[TILES][4];
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    auto factors = [&](Slot<TILES> &s, int block) {
        s.fb = __ldg(sb + block);
#pragma unroll
        for (int i = 0; i < TILES; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                s.fx[i][j] = 8 * i + 2 * t + j < a.rows
                                 ? __ldg(a.sA + static_cast<int64_t>(block) * a.rows + 8 * i + 2 * t + j)
                                 : 0.0f;
    };
    auto add = [&](const Slot<TILES> &s) {
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint4 &lo = s.b[c][0], &hi = s.b[c][1], &y = s.x[i][c];
                mma<A5, B5>(p, lo.x, hi.x, lo.y, hi.y, y.x, y.y);
                mma<A5, B5>(p, lo.z, hi.z, lo.w, hi.w, y.z, y.w);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(p[j], s.fx[i][j & 1] * s.fb, acc[i][j]);
        }
    };
    const int full = static_cast<int>(a.K / BLOCK);  // blocks without an end in them
    auto fetch = [&](Slot<TILES> &s, int block) {
        if (block >= full) return;
        const int64_t k = static_cast<int64_t>(block) * BLOCK;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int h = 0; h < 2; ++h) s.b[c][h] = load_once(b[h] + k + 64 * c);
#pragma unroll
            for (int i = 0; i < TILES; ++i) s.x[i][c] = __ldg(reinterpret_cast<const uint4 *>(x[i] + k + 64 * c));
        }
        factors(s, block);
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    Slot<TILES> slots[SLOTS];
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) fetch(slots[u], warp + u * WARPS);
    for (int first = warp; first < full; first += SLOTS * WARPS) {
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
            const int block = first + u * WARPS;
            if (block >= full) break;
            add(slots[u]);
            fetch(slots[u], block + SLOTS * WARPS);
        }
    }
    if (full < a.blocks && full % WARPS == warp) {
        Slot<TILES> s;
        const int64_t k = static_cast<int64_t>(full) * BLOCK;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
            const int64_t n = a.K - k - 64 * c - 16 * t;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 v = load_part(b[h] + k + 64 * c, n);
                s.b[0][h] = c ? s.b[0][h] : v;
                s.b[1][h] = v;
            }
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                const uint4 v = load_part(x[i] + k + 64 * c, n);
                s.x[i][0] = c ? s.x[i][0] : v;
                s.x[i][1] = v;
            }
        }
        factors(s, full);
        add(s);
    }
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[warp][8 * i + 2 * t + (j & 1)][8 * (j >> 1) + g] = acc[i][j];
    __syncthreads();
    for (int at = static_cast<int>(threadIdx.x); at < a.rows * COLS; at += WARPS * 32) {
        const int s = at / COLS, c = at % COLS;
        if (n0 + c >= a.N) continue;
        float sum = part[0][s][c];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) sum += part[w][s][c];
        const int64_t to = s * a.ldc + n0 + c;
        if (a.out_type == SGEMM_TYPE_F32)
            static_cast<float *>(a.C)[to] = sum;
        else if (a.out_type == SGEMM_TYPE_BF16)
            static_cast<__nv_bfloat16 *>(a.C)[to] = __float2bfloat16_rn(sum);
        else
            static_cast<__half *>(a.C)[to] = __float2half_rn(sum);
    }
}

template <bool A5, bool B5>
cudaError_t launch_types(const cudaLaunchConfig_t &cfg, const FewArgs &a) {
    if (a.rows <= 8) return cudaLaunchKernelEx(&cfg, fp8_few_kernel<1, A5, B5>, a);
    if (a.rows <= 16) return cudaLaunchKernelEx(&cfg, fp8_few_kernel<2, A5, B5>, a);
    return cudaLaunchKernelEx(&cfg, fp8_few_kernel<4, A5, B5>, a);
}

}  // namespace

// One matrix N x K, and so few rows that its bytes are what counts. 17 to 32
// rows, whose bytes of A are twice B's here, only where fp8_gemm.cu's tiles
// would leave half of the SM pairs without one. 8 rows of 4096 x 4096: 5.4 us here, 21.6
// there; 16384 x 8192: 26 and 41. 16 rows: 6.7 and 21.7; 39.4 and 41.7. 32 rows of
// 4096 x 4096: 9.6 and 20.8; 8192 x 4096: 17.3 and 22.9; 12288 x 4096: 24.1 and 24.0;
// 16384 x 8192: 54 and 41.
bool gemm_few(const GemmProblem &p, const DeviceInfo &dev) {
    if (p.wgrad || p.offsets || p.transB != SGEMM_OP_T) return false;
    return p.rows <= 16 || (p.rows <= 32 && (p.N + 255) / 256 * 4 <= dev.sm_count);
}

int gemm_few_launch(const GemmProblem &p, cudaStream_t stream, int *launches) {
    FewArgs a{};
    a.rows = static_cast<int>(p.rows);
    a.blocks = static_cast<int>(blocks_of(p.K));
    a.N = p.N;
    a.K = p.K;
    a.A = static_cast<const uint8_t *>(p.A);
    a.lda = p.lda;
    a.sA = p.sA;
    a.B = static_cast<const uint8_t *>(p.B);
    a.ldb = p.ldb;
    a.sB = p.sB;
    a.C = p.C;
    a.ldc = p.ldc;
    a.out_type = p.out_type;
    const int64_t ctas = (p.N + COLS - 1) / COLS;
    if (ctas > INT32_MAX) return SGEMM_ERR_UNSUPPORTED;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(WARPS * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool a5 = p.type_a == SGEMM_FP8_E5M2, b5 = p.type_b == SGEMM_FP8_E5M2;
    const cudaError_t e = a5 ? (b5 ? launch_types<true, true>(cfg, a) : launch_types<true, false>(cfg, a))
                             : (b5 ? launch_types<false, true>(cfg, a) : launch_types<false, false>(cfg, a));
    if (e != cudaSuccess) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    ++*launches;
    return SGEMM_OK;
}

}  // namespace f8
}  // namespace sgemm
