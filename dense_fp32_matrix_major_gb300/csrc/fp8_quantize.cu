// Quantisation to 8-bit floating point with a scale for each block of 128:
//
//     scale = max(max |x| / largest, 2^-126)      (or the power of two above)
//     q     = x * (1 / scale), rounded to the nearest 8-bit value
//
// Bound by memory: x is read once, held in registers while the block's maximum
// is found, and q written once. The reciprocal and the product are rounded to
// fp32 before the rounding to 8 bits, one multiplication and half a conversion a
// value; a quotient rounded once would differ only within 2^-23 of a border
// between 8-bit values, for six more instructions a value.
//
// Work. 1 x 128 blocks: a warp takes 512 values of a row, 16 a lane, eight lanes
// a block. 128 x 1 and 128 x 128 blocks: 256 threads take 128 x 128 values, 64 a
// thread; maxima are joined through shared memory.
#include <cuda_runtime.h>
#include <stdint.h>

#include "experts_common.cuh"
#include "fp8_internal.h"

namespace sgemm {
namespace f8 {
namespace {

using ex::from_f32;
using ex::group_start;
using ex::load_pack;
using ex::Pack;
using ex::row_tile_of;
using ex::RowTile;
using ex::to_f32;

constexpr int THREADS = 256;
constexpr float SMALLEST_SCALE = 1.17549435e-38f;  // 2^-126

struct QArgs {
    int64_t rows, cols;
    const void *x;
    int64_t ldx, strideX;
    const int32_t *offsets;
    int experts;
    uint8_t *q;
    int64_t ldq, strideQ;
    float *scales;
    int pow2;
    int q_vector;  // rows of q start 16 bytes apart
};

template <bool E5M2>
struct Fp8;
template <>
struct Fp8<false> {
    static constexpr float LARGEST = 448.0f;
    // Two values, rounded to nearest even and limited to the largest; NaN stays NaN.
    static __device__ __forceinline__ uint32_t pair(float lo, float hi) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
        return r;
    }
};
template <>
struct Fp8<true> {
    static constexpr float LARGEST = 57344.0f;
    static __device__ __forceinline__ uint32_t pair(float lo, float hi) {
        uint16_t r;
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
        return r;
    }
};

// The scale of a block whose largest magnitude is `most`.
template <bool E5M2>
__device__ __forceinline__ float scale_of(float most, int pow2) {
    float s = fmaxf(most / Fp8<E5M2>::LARGEST, SMALLEST_SCALE);
    // The next power of two: digits that are not zero carry into the exponent.
    if (pow2) s = __uint_as_float((__float_as_uint(s) + 0x007FFFFFu) & 0x7F800000u);
    return s;
}

// Eight values as 8-bit ones; inverse(i): of value i. infinite: some may be
// infinite and become NaN (the conversion would limit them to the largest).
template <bool E5M2, class I>
__device__ __forceinline__ uint2 convert8(const float (&x)[8], I &&inverse, bool infinite) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * inverse(i);
    if (infinite) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(x[i]) == __int_as_float(0x7F800000)) y[i] = __int_as_float(0x7FFFFFFF);
    }
    using F = Fp8<E5M2>;
    return make_uint2(F::pair(y[0], y[1]) | (F::pair(y[2], y[3]) << 16), F::pair(y[4], y[5]) | (F::pair(y[6], y[7]) << 16));
}

// The larger magnitude of finite values; an infinity is seen to by the caller.
__device__ __forceinline__ float larger(float most, float x) { return fmaxf(most, fabsf(x)); }

// The same, infinities left out.
__device__ __forceinline__ float larger_finite(float most, float x) {
    const float v = fabsf(x);
    return v < __int_as_float(0x7F800000) ? fmaxf(most, v) : most;
}

template <class T, int N>
__device__ __forceinline__ void load_vector(const T *p, float (&v)[N]) {
    constexpr int PER = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < N; i += PER) {
        const Pack<T, PER> a = load_pack<T, PER>(p + i);
#pragma unroll
        for (int j = 0; j < PER; ++j) v[i + j] = to_f32(a.v[j]);
    }
}

// ------------------------------------------------------------- 1 x 128 blocks

constexpr int LANE_VALUES = 16, WARP_VALUES = 32 * LANE_VALUES;

template <class T, bool E5M2, bool VECTOR>
__global__ void __launch_bounds__(THREADS) quantize_rows_kernel(const __grid_constant__ QArgs a) {
    const int lane = static_cast<int>(threadIdx.x & 31);
    const int64_t chunks = (a.cols + WARP_VALUES - 1) / WARP_VALUES;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5);
    const int64_t row = item / chunks, c0 = (item - row * chunks) * WARP_VALUES + lane * LANE_VALUES;
    if (row >= a.rows) return;
    const T *x = static_cast<const T *>(a.x) + row * a.ldx + c0;
    float v[LANE_VALUES];
    if (VECTOR && c0 + LANE_VALUES <= a.cols) {
        load_vector<T, LANE_VALUES>(x, v);
    } else {
#pragma unroll
        for (int i = 0; i < LANE_VALUES; ++i) v[i] = c0 + i < a.cols ? to_f32(x[i]) : 0.0f;
    }
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < LANE_VALUES; ++i) most = larger(most, v[i]);
#pragma unroll
    for (int d = 1; d < 8; d *= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    const bool infinite = __any_sync(0xffffffffu, most == __int_as_float(0x7F800000));
    if (infinite) {
        most = 0.0f;
#pragma unroll
        for (int i = 0; i < LANE_VALUES; ++i) most = larger_finite(most, v[i]);
#pragma unroll
        for (int d = 1; d < 8; d *= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    }
    const float scale = scale_of<E5M2>(most, a.pow2), inverse = 1.0f / scale;
    if (c0 >= a.cols) return;
    if ((lane & 7) == 0) a.scales[c0 / BLOCK * a.rows + row] = scale;
    uint32_t out[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = v[8 * h + i];
        const uint2 q = convert8<E5M2>(w, [&](int) { return inverse; }, infinite);
        out[2 * h] = q.x;
        out[2 * h + 1] = q.y;
    }
    uint8_t *to = a.q + row * a.ldq + c0;
    if (a.q_vector && c0 + LANE_VALUES <= a.cols) {
        *reinterpret_cast<uint4 *>(to) = make_uint4(out[0], out[1], out[2], out[3]);
    } else {
#pragma unroll
        for (int i = 0; i < LANE_VALUES; ++i)
            if (c0 + i < a.cols) to[i] = static_cast<uint8_t>(out[i / 4] >> (8 * (i % 4)));
    }
}

// ----------------------------------------------- 128 x 1 and 128 x 128 blocks

// Columns of a thread: VECTOR: eight next to one another; otherwise sixteen
// apart, so that a warp's scalar loads are next to one another, and q goes
// through shared memory on its way out.
template <class T, bool E5M2, bool COLUMNS, bool VECTOR>
__global__ void __launch_bounds__(THREADS) quantize_tiles_kernel(const __grid_constant__ QArgs a) {
    __shared__ float most_of[COLUMNS ? 8 * BLOCK : 8];
    __shared__ float scale_s[COLUMNS ? BLOCK : 1], inverse_s[COLUMNS ? BLOCK : 1];
    __shared__ int infinite_s;
    __shared__ alignas(16) uint8_t tile[VECTOR ? 16 : BLOCK * (BLOCK + 16)];
    const int tid = static_cast<int>(threadIdx.x), part = tid & 15, r0 = tid >> 4, warp = tid >> 5, lane = tid & 31;
    const int64_t c0 = static_cast<int64_t>(blockIdx.y) * BLOCK;
    if (tid == 0) infinite_s = 0;
    // Rows of x, and the row of q they start at.
    int64_t begin = static_cast<int64_t>(blockIdx.x) * BLOCK;
    const int64_t at = begin;
    int rows = static_cast<int>(min(static_cast<int64_t>(BLOCK), a.rows - begin)), kept = rows;
    if (COLUMNS && a.offsets) {
        const RowTile t = row_tile_of(a.offsets, a.experts, static_cast<int>(a.rows), BLOCK, static_cast<int>(blockIdx.x));
        const bool used = t.group >= 0 && t.group < a.experts;
        begin = used ? t.begin : 0;
        rows = used ? t.end - t.begin : 0;
        kept = BLOCK;
    }
    const T *x = static_cast<const T *>(a.x) + blockIdx.z * a.strideX + begin * a.ldx + c0;
    const int64_t cols = a.cols - c0;
    auto col = [&](int j) { return VECTOR ? 8 * part + j : part + 16 * j; };
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        const T *p = x + r * a.ldx;
        if (VECTOR && r < rows && 8 * part + 8 <= cols) {
            load_vector<T, 8>(p + 8 * part, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = r < rows && col(j) < cols ? to_f32(p[col(j)]) : 0.0f;
        }
    }
    float most[COLUMNS ? 8 : 1], inverse[COLUMNS ? 8 : 1];
    // Joins the maxima of the block's threads, or of a column's.
    auto join = [&](auto &&larger_of) {
#pragma unroll
        for (int j = 0; j < (COLUMNS ? 8 : 1); ++j) most[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) most[COLUMNS ? j : 0] = larger_of(most[COLUMNS ? j : 0], v[i][j]);
        if (COLUMNS) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                most[j] = fmaxf(most[j], __shfl_xor_sync(0xffffffffu, most[j], 16));
                if (lane < 16) most_of[warp * BLOCK + col(j)] = most[j];
            }
        } else {
#pragma unroll
            for (int d = 1; d < 32; d *= 2) most[0] = fmaxf(most[0], __shfl_xor_sync(0xffffffffu, most[0], d));
            if (lane == 0) most_of[warp] = most[0];
        }
        __syncthreads();
        if (COLUMNS ? tid < BLOCK : tid == 0) {
            float m = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) m = fmaxf(m, most_of[COLUMNS ? w * BLOCK + tid : w]);
            if (m == __int_as_float(0x7F800000)) infinite_s = 1;
            const float s = scale_of<E5M2>(m, a.pow2);
            scale_s[COLUMNS ? tid : 0] = s;
            inverse_s[COLUMNS ? tid : 0] = 1.0f / s;
        }
        __syncthreads();
    };
    join(larger);
    const bool infinite = infinite_s != 0;
    if (infinite) {
        __syncthreads();
        join(larger_finite);
    }
#pragma unroll
    for (int j = 0; j < (COLUMNS ? 8 : 1); ++j) inverse[j] = inverse_s[COLUMNS ? col(j) : 0];
    if (COLUMNS) {
        if (tid < BLOCK && tid < cols) a.scales[blockIdx.x * a.cols + c0 + tid] = scale_s[tid];
    } else if (tid == 0) {
        a.scales[(static_cast<int64_t>(blockIdx.z) * gridDim.x + blockIdx.x) * gridDim.y + blockIdx.y] = scale_s[0];
    }
    uint8_t *q = a.q + blockIdx.z * a.strideQ + at * a.ldq + c0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        const uint2 o = convert8<E5M2>(v[i], [&](int j) { return inverse[COLUMNS ? j : 0]; }, infinite);
        if (VECTOR) {
            uint8_t *to = q + r * a.ldq + 8 * part;
            if (r >= kept) continue;
            if (a.q_vector && 8 * part + 8 <= cols) {
                *reinterpret_cast<uint2 *>(to) = o;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (8 * part + j < cols) to[j] = static_cast<uint8_t>((j < 4 ? o.x : o.y) >> (8 * (j & 3)));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                tile[r * (BLOCK + 16) + col(j)] = static_cast<uint8_t>((j < 4 ? o.x : o.y) >> (8 * (j & 3)));
        }
    }
    if (VECTOR) return;
    __syncthreads();
    // Sixteen bytes a thread, eight threads a row.
    for (int r = tid >> 3; r < kept; r += THREADS / 8) {
        const int c = 16 * (tid & 7);
        const uint8_t *from = tile + r * (BLOCK + 16) + c;
        uint8_t *to = q + r * a.ldq + c;
        if (a.q_vector && c + 16 <= cols) {
            *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from);
        } else {
            for (int j = 0; j < 16; ++j)
                if (c + j < cols) to[j] = from[j];
        }
    }
}

template <class T, bool E5M2>
int launch_type(const QuantizeProblem &p, const QArgs &a, bool vector, cudaStream_t stream) {
    if (p.block == SGEMM_FP8_ROWS) {
        const int64_t warps = p.rows * ((p.cols + WARP_VALUES - 1) / WARP_VALUES), per = THREADS / 32;
        const int64_t blocks = (warps + per - 1) / per;
        if (blocks > INT32_MAX) return SGEMM_ERR_UNSUPPORTED;
        auto kernel = vector ? quantize_rows_kernel<T, E5M2, true> : quantize_rows_kernel<T, E5M2, false>;
        kernel<<<static_cast<unsigned>(blocks), THREADS, 0, stream>>>(a);
    } else {
        const int64_t wide = blocks_of(p.cols),
                      high = p.offsets ? sgemm_fp8_blocks(p.rows, p.experts) : blocks_of(p.rows);
        if (high > INT32_MAX || wide > 65535 || p.items > 65535) return SGEMM_ERR_UNSUPPORTED;
        const dim3 grid(static_cast<unsigned>(high), static_cast<unsigned>(wide), static_cast<unsigned>(p.items));
        auto kernel = p.block == SGEMM_FP8_COLUMNS
                          ? (vector ? quantize_tiles_kernel<T, E5M2, true, true> : quantize_tiles_kernel<T, E5M2, true, false>)
                          : (vector ? quantize_tiles_kernel<T, E5M2, false, true>
                                    : quantize_tiles_kernel<T, E5M2, false, false>);
        kernel<<<grid, THREADS, 0, stream>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

template <class T>
int launch_any(const QuantizeProblem &p, const QArgs &a, bool vector, cudaStream_t stream) {
    return p.to == SGEMM_FP8_E5M2 ? launch_type<T, true>(p, a, vector, stream)
                                  : launch_type<T, false>(p, a, vector, stream);
}

}  // namespace

int quantize_launch(const QuantizeProblem &p, const DeviceInfo &, cudaStream_t stream, int *launches) {
    QArgs a{};
    a.rows = p.rows;
    a.cols = p.cols;
    a.x = p.x;
    a.ldx = p.ldx;
    a.strideX = p.items > 1 ? p.strideX : 0;
    a.offsets = p.offsets;
    a.experts = static_cast<int>(p.experts);
    a.q = p.q;
    a.ldq = p.ldq;
    a.strideQ = p.items > 1 ? p.strideQ : 0;
    a.scales = p.scales;
    a.pow2 = p.pow2;
    a.q_vector = reinterpret_cast<uintptr_t>(p.q) % 16 == 0 && p.ldq % 16 == 0 && a.strideQ % 16 == 0;
    const int64_t per = 16 / ex::type_size(p.type);
    const bool vector = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ldx % per == 0 && a.strideX % per == 0;
    int rc;
    if (p.type == SGEMM_TYPE_F32)
        rc = launch_any<float>(p, a, vector, stream);
    else if (p.type == SGEMM_TYPE_BF16)
        rc = launch_any<__nv_bfloat16>(p, a, vector, stream);
    else
        rc = launch_any<__half>(p, a, vector, stream);
    if (rc == SGEMM_OK)
        ++*launches;
    else
        cudaGetLastError();
    return rc;
}

}  // namespace f8
}  // namespace sgemm
