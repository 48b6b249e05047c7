// One product per group of rows, any type, alignment and form, on the CUDA
// cores:
//
//     C[s] = A[s] op(B[e(s)])                     (rows)
//     C[e] = sum over s in group e of A[s]^T B[s]  (wgrad)
//
// The group bounds are read on the device, so no call waits for the host. A
// block makes one 64 x 64 tile of C with 16 x 16 threads, 4 x 4 sums each,
// in fp32 from 64 x 16 tiles in shared memory; every product in fp32.
//
// Also the choice between the kernels, and the split of long sums of wgrad.
#include <cuda_runtime.h>
#include <stdint.h>

#include "experts_common.cuh"
#include "experts_internal.h"

namespace sgemm {
namespace ex {
namespace {

constexpr int TILE = 64, DEPTH = 16, GEMM_THREADS = 256;

struct SimpleArgs {
    bool wgrad, trans;
    int rows, experts;
    int64_t M, N, K;
    const int32_t *offsets;
    const void *A;
    int64_t lda;
    const void *B;
    int64_t ldb, strideB;
    void *C;
    int64_t ldc, strideC;
    int tiles_n;
};

// rows: blockIdx.x = row tile * tiles_n + column tile. wgrad: the same over a
// matrix's tiles, blockIdx.y the group.
template <class T>
__global__ void __launch_bounds__(GEMM_THREADS) grouped_simple_kernel(const SimpleArgs a) {
    __shared__ float As[DEPTH][TILE + 1], Bs[DEPTH][TILE + 1];
    const int tid = static_cast<int>(threadIdx.x);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x % a.tiles_n) * TILE;
    const int mt = static_cast<int>(blockIdx.x / a.tiles_n);
    // op(A)[m][k] at A + m * am + k * ak, op(B)[k][n] at B + k * bk + n * bn.
    const T *A = static_cast<const T *>(a.A), *B = static_cast<const T *>(a.B);
    T *C = static_cast<T *>(a.C);
    int64_t m_count, k_count, am, ak, bk, bn;
    if (a.wgrad) {
        const int e = static_cast<int>(blockIdx.y);
        const int begin = group_start(a.offsets, e, a.rows);
        const int end = max(begin, group_start(a.offsets, e + 1, a.rows));
        k_count = end - begin;
        am = 1, ak = a.lda, bk = a.ldb, bn = 1;
        m_count = min(static_cast<int64_t>(TILE), a.M - static_cast<int64_t>(mt) * TILE);
        A += begin * a.lda + static_cast<int64_t>(mt) * TILE;
        B += begin * a.ldb;
        C += e * a.strideC + static_cast<int64_t>(mt) * TILE * a.ldc;
    } else {
        const RowTile rt = row_tile_of(a.offsets, a.experts, a.rows, TILE, mt);
        if (rt.group < 0) return;
        m_count = rt.end - rt.begin;
        k_count = rt.group < a.experts ? a.K : 0;
        am = a.lda, ak = 1, bk = a.trans ? 1 : a.ldb, bn = a.trans ? a.ldb : 1;
        A += rt.begin * a.lda;
        if (rt.group < a.experts) B += rt.group * a.strideB;
        C += rt.begin * a.ldc;
    }
    const int64_t n_count = min(static_cast<int64_t>(TILE), a.N - n0);
    B += n0 * bn;
    float sum[4][4] = {};
    const int ty = tid >> 4, tx = tid & 15;
    for (int64_t k0 = 0; k0 < k_count; k0 += DEPTH) {
        // Threads run along the operand's contiguous direction.
#pragma unroll
        for (int i = 0; i < TILE * DEPTH / GEMM_THREADS; ++i) {
            const int x = tid + i * GEMM_THREADS;
            const int m = ak == 1 ? x / DEPTH : x % TILE, ka = ak == 1 ? x % DEPTH : x / TILE;
            As[ka][m] = m < m_count && k0 + ka < k_count ? to_f32(A[m * am + (k0 + ka) * ak]) : 0.0f;
            const int n = bk == 1 ? x / DEPTH : x % TILE, kb = bk == 1 ? x % DEPTH : x / TILE;
            Bs[kb][n] = n < n_count && k0 + kb < k_count ? to_f32(B[n * bn + (k0 + kb) * bk]) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < DEPTH; ++k) {
            float x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = As[k][ty + 16 * i];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = Bs[k][tx + 16 * i];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[i][j] = fmaf(x[i], y[j], sum[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (ty + 16 * i < m_count && tx + 16 * j < n_count)
                C[(ty + 16 * i) * a.ldc + n0 + tx + 16 * j] = from_f32<T>(sum[i][j]);
}

int simple_launch(const GroupedProblem &p, cudaStream_t stream, int *launches) {
    SimpleArgs a{};
    a.wgrad = p.wgrad;
    a.trans = p.transB == SGEMM_OP_T;
    a.rows = static_cast<int>(p.rows);
    a.experts = static_cast<int>(p.experts);
    a.M = p.M;
    a.N = p.N;
    a.K = p.K;
    a.offsets = p.offsets;
    a.A = p.A;
    a.lda = p.lda;
    a.B = p.B;
    a.ldb = p.ldb;
    a.strideB = p.strideB;
    a.C = p.C;
    a.ldc = p.ldc;
    a.strideC = p.strideC;
    const int64_t tiles_n = (p.N + TILE - 1) / TILE;
    // Every group may end in a part of a tile.
    const int64_t tiles_m = p.wgrad ? (p.M + TILE - 1) / TILE : (p.rows + TILE - 1) / TILE + p.experts;
    if (tiles_n > INT32_MAX / tiles_m) return SGEMM_ERR_UNSUPPORTED;
    a.tiles_n = static_cast<int>(tiles_n);
    const dim3 grid(static_cast<unsigned>(tiles_m * tiles_n), p.wgrad ? static_cast<unsigned>(p.experts) : 1u);
    if (p.type == SGEMM_TYPE_F32)
        grouped_simple_kernel<float><<<grid, GEMM_THREADS, 0, stream>>>(a);
    else if (p.type == SGEMM_TYPE_BF16)
        grouped_simple_kernel<__nv_bfloat16><<<grid, GEMM_THREADS, 0, stream>>>(a);
    else
        grouped_simple_kernel<__half><<<grid, GEMM_THREADS, 0, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return SGEMM_ERR_LAUNCH;
    ++*launches;
    return SGEMM_OK;
}

// wgrad in slices: few matrices whose tiles leave most SM pairs idle are summed
// over slices of their groups' rows, each into fp32 sums of its own, which a
// second kernel adds in the order of the slices.
struct Join {
    const float *part;
    void *C;
    int64_t rows;  // experts * M
    int64_t M, N, ld, ldc, strideC;
    int split, vector;
};

constexpr int JOIN_THREADS = 256;
template <class T>
__global__ void __launch_bounds__(JOIN_THREADS) join_slices_kernel(const Join j) {
    const int64_t vecs = j.ld / 4, total = j.rows * vecs, item = j.M * j.ld;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * JOIN_THREADS + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * JOIN_THREADS) {
        const int64_t row = i / vecs, n = (i - row * vecs) * 4, e = row / j.M, m = row - e * j.M;
        const float *p = j.part + e * j.split * item + m * j.ld + n;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int k = 0; k < j.split; ++k, p += item) {
            const float4 v = __ldcs(reinterpret_cast<const float4 *>(p));
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        T *c = static_cast<T *>(j.C) + e * j.strideC + m * j.ldc + n;
        const Pack<T, 4> out{{from_f32<T>(s.x), from_f32<T>(s.y), from_f32<T>(s.z), from_f32<T>(s.w)}};
        if (j.vector && n + 4 <= j.N) {
            store_pack(c, out);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (n + k < j.N) c[k] = out.v[k];
        }
    }
}

// Slices that pay: a k-block takes a pair 0.55 us (fp32, 32 rows) or 0.22 us (16
// bits, 64 rows); the sums are written and read at 5 TB/s, the second launch
// and its wait take 6 us. Groups are taken as even. In slices and whole, one
// group of 30000 rows, cold: 64 x 64 fp32 37 and 552 us, bf16 33 and 119 us; 512 x 512
// fp32 91 and 593 us, bf16 35 and 138 us; 2000 rows, 64 x 64: fp32 24 and 49 us.
int slices_of(const GroupedProblem &p, const DeviceInfo &dev) {
    int64_t high = 256, wide = 256;
    const bool f32 = p.type == SGEMM_TYPE_F32;
    if (f32) grouped_f32_tile(p, &high, &wide);
    const int64_t tiles = (p.M + high - 1) / high * ((p.N + wide - 1) / wide) * p.experts, pairs = dev.sm_count / 2;
    if (2 * tiles > pairs) return 1;
    const double k_blocks = static_cast<double>(p.rows) / static_cast<double>(p.experts * (f32 ? 32 : 64));
    int64_t split = pairs / tiles;
    if (split > k_blocks / 4) split = static_cast<int64_t>(k_blocks / 4);
    if (split < 2) return 1;
    const double sums = 8.0 * static_cast<double>(split * p.experts * p.M * p.N) / 5e6;
    const double saved = k_blocks * (1.0 - 1.0 / static_cast<double>(split)) * (f32 ? 0.55 : 0.22);
    return saved > 6.0 + sums ? static_cast<int>(split) : 1;
}

int tensor_launch(const GroupedProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    return p.type == SGEMM_TYPE_F32 ? grouped_f32_launch(p, dev, stream, launches)
                                    : grouped16_launch(p, dev, stream, launches);
}

int sliced_launch(const GroupedProblem &p, int split, float *sums, const DeviceInfo &dev, cudaStream_t stream,
                  int *launches) {
    GroupedProblem q = p;
    q.split = split;
    q.C = sums;
    q.ldc = slice_ld(p.N);
    q.strideC = p.M * q.ldc;
    const int rc = tensor_launch(q, dev, stream, launches);
    if (rc != SGEMM_OK) return rc;
    return join_slices_launch(p.type, sums, split, p.experts, p.M, p.N, p.C, p.ldc, p.strideC, dev, stream, launches);
}

}  // namespace

int join_slices_launch(int type, const float *sums, int split, int64_t experts, int64_t M, int64_t N, void *C,
                       int64_t ldc, int64_t strideC, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    const int64_t size = type_size(type), ld = slice_ld(N);
    Join j{sums, C, experts * M, M, N, ld, ldc, experts > 1 ? strideC : 0, split, 0};
    j.vector = (reinterpret_cast<uintptr_t>(C) % (4 * size) | (ldc % 4) | (j.strideC % 4)) == 0;
    const int64_t blocks = (j.rows * (ld / 4) + JOIN_THREADS - 1) / JOIN_THREADS, most = 8LL * dev.sm_count;
    const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
    if (type == SGEMM_TYPE_F32)
        join_slices_kernel<float><<<grid, JOIN_THREADS, 0, stream>>>(j);
    else if (type == SGEMM_TYPE_BF16)
        join_slices_kernel<__nv_bfloat16><<<grid, JOIN_THREADS, 0, stream>>>(j);
    else
        join_slices_kernel<__half><<<grid, JOIN_THREADS, 0, stream>>>(j);
    if (cudaGetLastError() != cudaSuccess) return SGEMM_ERR_LAUNCH;
    ++*launches;
    return SGEMM_OK;
}

int grouped_launch(const GroupedProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    // fp32 on the tensor cores is the three-term TF32 split; a caller who wants
    // fp32 multiply-adds has chosen them for every product (8192 rows, 8 experts,
    // 1024 -> 2048: 1268 us in place of 165; error 0.57e-6 in place of 0.71e-6).
    const bool f32 = p.type == SGEMM_TYPE_F32, cores = f32 && chosen_variant() == SGEMM_FFMA;
    if (!cores && (grouped_f32_supports(p) || grouped16_supports(p))) {
        int rc = SGEMM_ERR_UNSUPPORTED;
        const int split = p.wgrad ? slices_of(p, dev) : 1;
        if (split > 1) {
            const int64_t bytes = split * p.experts * p.M * slice_ld(p.N) * 4;
            if (float *sums = scratch_alloc(dev, static_cast<size_t>(bytes), stream)) {
                rc = sliced_launch(p, split, sums, dev, stream, launches);
                scratch_free(sums, stream);
            }
        }
        if (rc == SGEMM_ERR_UNSUPPORTED) rc = tensor_launch(p, dev, stream, launches);
        if (rc == SGEMM_OK && f32) note_variant(SGEMM_TF32X3);
        if (rc != SGEMM_ERR_UNSUPPORTED) return rc;  // no memory for copies or slices: nothing was enqueued
    }
    const int rc = simple_launch(p, stream, launches);
    if (rc == SGEMM_OK && f32) note_variant(SGEMM_FFMA);
    return rc;
}

}  // namespace ex
}  // namespace sgemm
