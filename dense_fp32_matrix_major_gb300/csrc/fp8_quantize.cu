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
// a block (16384 x 2048 bf16: 18.2 us, 5.5 TB/s). 128 x 1 and 128 x 128 blocks:
// 256 threads take tiles of 128 x 128 values, 64 a thread; maxima are joined
// through shared memory. Between its loads, the join and its stores such a block
// leaves memory idle, so where x can be copied to shared memory as it is
// (16-bit, 16-byte aligned) each SM's blocks take tiles one after the other with
// the next one's copies on their way: 19.8 us for 16384 x 2048 bf16 (5.1 TB/s; 37.9
// with a tile a block, held in registers), 26 us in 32 groups, of whose stored rows a
// fifth are padding. fp32 tiles would be 64 KB, one block of an SM: there a tile a
// block, three blocks an SM (16 x 2049 x 1537: 48 us, with two 54; 16 x 2048 x 1536
// 42).
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

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
    unsigned high, wide;  // blocks of rows and of columns of an item
    unsigned tiles;       // 128 x 128 tiles of all
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

// 16-bit values two at a time, half the instructions of fp32 maxima: without its
// sign, a value that is not NaN is larger when its bits are, and infinities and NaN
// have the largest bits. (In rows, where memory is the bound, it gains nothing.)
__device__ __forceinline__ uint32_t larger_bits(uint32_t most, uint32_t two) {
    return __vmaxu2(most, two & 0x7FFF7FFFu);
}
template <class T>
constexpr uint32_t INFINITE_BITS = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;

// The value of magnitude bits below INFINITE_BITS.
template <class T>
__device__ __forceinline__ float value_of_bits(uint32_t bits) {
    if (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(static_cast<uint16_t>(bits)));
    return __uint_as_float(bits << 16);
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

// How a thread gets its 8 x 8 values, rows 16 apart:
//   ASYNC   16-bit values in rows that are 16-byte aligned: eight columns next to one
//           another, copied to shared memory while the CTA is at the tile before;
//   VECTOR  32-bit values in such rows: the same columns, straight to registers;
//   SCALAR  columns 16 apart, so that a warp's loads are next to one another; q goes
//           through shared memory on its way out.
enum Load { ASYNC, VECTOR, SCALAR };

constexpr int TILE_STAGES = 2, TILE_CTAS = 3;  // ASYNC: tiles in shared memory, CTAs of an SM
constexpr int TILE_STAGE = 8 * THREADS * 16;

// 16 bytes of which the first `bytes` are read, the others zero.
__device__ __forceinline__ void copy_async(uint32_t to, const void *from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

// Tiles of 128 x 128 values, in the order items, row blocks, columns.
template <class T, bool E5M2, bool COLUMNS, Load LOAD>
__global__ void __launch_bounds__(THREADS, LOAD == ASYNC || !COLUMNS ? TILE_CTAS : 2)
    quantize_tiles_kernel(const __grid_constant__ QArgs a) {
    constexpr int MAXIMA = COLUMNS ? 8 : 1;
    __shared__ alignas(16) float most_of[COLUMNS ? 8 * BLOCK : 8];
    __shared__ float inverse_s[COLUMNS ? BLOCK : 1];
    __shared__ alignas(16) uint8_t tile[LOAD == SCALAR ? BLOCK * (BLOCK + 16) : 16];
    extern __shared__ __align__(16) uint8_t staged[];
    const int tid = static_cast<int>(threadIdx.x), part = tid & 15, r0 = tid >> 4, warp = tid >> 5, lane = tid & 31;
    const unsigned high = a.high, wide = a.wide;
    unsigned first = blockIdx.x, last = first + 1;
    if constexpr (LOAD == ASYNC) {
        const unsigned each = a.tiles / gridDim.x, more = a.tiles % gridDim.x;
        first = each * blockIdx.x + min(blockIdx.x, more);
        last = first + each + (blockIdx.x < more);
    }

    struct Place {
        int item, row_block, col_block;
        int64_t begin;   // first row of x
        int rows, kept;  // rows of x in the tile, rows of q
    };
    // The place of tile u, after that of the tile before it.
    auto place = [&](unsigned u, Place &p) {
        const int before = p.row_block;
        const unsigned row_blocks = u / wide;
        p.item = static_cast<int>(row_blocks / high);
        p.row_block = static_cast<int>(row_blocks % high);
        p.col_block = static_cast<int>(u % wide);
        if (COLUMNS && a.offsets) {
            if (p.row_block == before) return;
            const RowTile t =
                row_tile_of(a.offsets, a.experts, static_cast<int>(a.rows), BLOCK, p.row_block);
            const bool used = t.group >= 0 && t.group < a.experts;
            p.begin = used ? t.begin : 0;
            p.rows = used ? t.end - t.begin : 0;
            p.kept = BLOCK;
        } else {
            p.begin = static_cast<int64_t>(p.row_block) * BLOCK;
            p.rows = p.kept = static_cast<int>(min(static_cast<int64_t>(BLOCK), a.rows - p.begin));
        }
    };
    auto col = [&](int j) { return LOAD == SCALAR ? part + 16 * j : 8 * part + j; };
    const uint32_t slot = LOAD == ASYNC ? static_cast<uint32_t>(__cvta_generic_to_shared(staged)) + 16u * tid : 0u;
    auto fetch = [&](const Place &p, unsigned n) {
        const T *x = static_cast<const T *>(a.x) + p.item * a.strideX + p.begin * a.ldx + static_cast<int64_t>(p.col_block) * BLOCK;
        const int64_t left = a.cols - static_cast<int64_t>(p.col_block) * BLOCK - 8 * part;
        const int bytes = left <= 0 ? 0 : static_cast<int>(min(left, static_cast<int64_t>(8)) * sizeof(T));
        const uint32_t to = slot + n % TILE_STAGES * TILE_STAGE;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + 16 * i, some = r < p.rows ? bytes : 0;
            copy_async(to + 16u * THREADS * i, some ? x + r * a.ldx + 8 * part : static_cast<const T *>(a.x), some);
        }
    };
    Place here{-1, -1, -1, 0, 0, 0}, ahead = here;
    if (LOAD == ASYNC) {
        place(first, ahead);
        fetch(ahead, 0);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    for (unsigned u = first; u < last; ++u) {
        constexpr int PER = 16 / sizeof(T);
        Pack<T, PER> v[LOAD == ASYNC ? 1 : 8][8 / PER];
        const uint8_t *from = staged + (u - first) % TILE_STAGES * TILE_STAGE + 16 * tid;
        // Row i of the thread's values. ASYNC: from shared memory whenever they are
        // needed: in registers from the maximum to the conversion they were 64 fp32
        // values, spilled.
        auto row = [&](int i, float (&w)[8]) {
            if constexpr (LOAD == ASYNC) {
                const Pack<T, 8> x = *reinterpret_cast<const Pack<T, 8> *>(from + 16 * THREADS * i);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = to_f32(x.v[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = to_f32(v[i][j / PER].v[j % PER]);
            }
        };
        if constexpr (LOAD == ASYNC) {
            static_assert(TILE_STAGES == 2, "the tile after this one is on its way");
            here = ahead;
            if (u + 1 < last) {
                place(u + 1, ahead);
                fetch(ahead, u + 1 - first);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            place(u, here);
            const T *x = static_cast<const T *>(a.x) + here.item * a.strideX + here.begin * a.ldx +
                         static_cast<int64_t>(here.col_block) * BLOCK;
            const int64_t cols = a.cols - static_cast<int64_t>(here.col_block) * BLOCK;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = r0 + 16 * i;
                const T *p = x + r * a.ldx;
                if (LOAD == VECTOR && r < here.rows && 8 * part + 8 <= cols) {
#pragma unroll
                    for (int h = 0; h < 8 / PER; ++h) v[i][h] = load_pack<T, PER>(p + 8 * part + PER * h);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[i][j / PER].v[j % PER] = r < here.rows && col(j) < cols ? p[col(j)] : from_f32<T>(0.0f);
                }
            }
        }
        const int64_t c0 = static_cast<int64_t>(here.col_block) * BLOCK, cols = a.cols - c0;
        float most[MAXIMA], inverse[MAXIMA];
        // The scale of a block with the largest magnitude m.
        auto settle = [&](float m) {
            const float s = scale_of<E5M2>(m, a.pow2);
            inverse_s[COLUMNS ? tid : 0] = 1.0f / s;
            if (!COLUMNS)
                a.scales[u] = s;
            else if (tid < cols)
                a.scales[here.row_block * a.cols + c0 + tid] = s;
        };
        // Joins the maxima of the block's threads, or of a column's; whether one of
        // them is infinite (or, by bits, NaN).
        auto join_bits = [&] {
            uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 x = *reinterpret_cast<const uint4 *>(from + 16 * THREADS * i);
                m[0] = larger_bits(m[0], x.x), m[1] = larger_bits(m[1], x.y);
                m[2] = larger_bits(m[2], x.z), m[3] = larger_bits(m[3], x.w);
            }
            uint32_t *of = reinterpret_cast<uint32_t *>(most_of);
            if (COLUMNS) {
#pragma unroll
                for (int k = 0; k < 4; ++k) m[k] = __vmaxu2(m[k], __shfl_xor_sync(0xffffffffu, m[k], 16));
                if (lane < 16) *reinterpret_cast<uint4 *>(of + warp * (BLOCK / 2) + 4 * part) = make_uint4(m[0], m[1], m[2], m[3]);
            } else {
                uint32_t one = __vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3]));
                one = max(one & 0xFFFFu, one >> 16);
                one = __reduce_max_sync(0xffffffffu, one);
                if (lane == 0) of[warp] = one;
            }
            __syncthreads();
            bool infinite = false;
            if (COLUMNS ? tid < BLOCK : tid == 0) {
                uint32_t b = 0;
#pragma unroll
                for (int w = 0; w < 8; ++w)
                    b = max(b, COLUMNS ? static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(of)[w * BLOCK + tid]) : of[w]);
                infinite = b >= INFINITE_BITS<T>;
                settle(value_of_bits<T>(b));
            }
            return __syncthreads_or(infinite) != 0;
        };
        auto join = [&](auto &&larger_of) {
#pragma unroll
            for (int j = 0; j < MAXIMA; ++j) most[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float w[8];
                row(i, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) most[COLUMNS ? j : 0] = larger_of(most[COLUMNS ? j : 0], w[j]);
            }
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
            bool infinite = false;
            if (COLUMNS ? tid < BLOCK : tid == 0) {
                float m = 0.0f;
#pragma unroll
                for (int w = 0; w < 8; ++w) m = fmaxf(m, most_of[COLUMNS ? w * BLOCK + tid : w]);
                infinite = m == __int_as_float(0x7F800000);
                settle(m);
            }
            return __syncthreads_or(infinite) != 0;
        };
        bool infinite;
        if constexpr (LOAD == ASYNC)
            infinite = join_bits();
        else
            infinite = join(larger);
        if (infinite) join(larger_finite);
#pragma unroll
        for (int j = 0; j < MAXIMA; ++j) inverse[j] = inverse_s[COLUMNS ? col(j) : 0];
        uint8_t *q = a.q + here.item * a.strideQ + static_cast<int64_t>(here.row_block) * BLOCK * a.ldq + c0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + 16 * i;
            float w[8];
            row(i, w);
            const uint2 o = convert8<E5M2>(w, [&](int j) { return inverse[COLUMNS ? j : 0]; }, infinite);
            if (LOAD != SCALAR) {
                uint8_t *to = q + r * a.ldq + 8 * part;
                if (r >= here.kept) continue;
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
        if (LOAD != SCALAR) continue;
        __syncthreads();
        // Sixteen bytes a thread, eight threads a row.
        for (int r = tid >> 3; r < here.kept; r += THREADS / 8) {
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
        // The next tile's first write to `tile` comes after a barrier.
    }
}

template <class T, bool E5M2, bool COLUMNS>
int launch_tiles(QArgs a, bool vector, const DeviceInfo &dev, cudaStream_t stream) {
    if (!vector) {
        quantize_tiles_kernel<T, E5M2, COLUMNS, SCALAR><<<a.tiles, THREADS, 0, stream>>>(a);
    } else if constexpr (sizeof(T) == 4) {
        quantize_tiles_kernel<T, E5M2, COLUMNS, VECTOR><<<a.tiles, THREADS, 0, stream>>>(a);
    } else {
        auto kernel = quantize_tiles_kernel<T, E5M2, COLUMNS, ASYNC>;
        constexpr int bytes = TILE_STAGES * TILE_STAGE;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
        const unsigned ctas = static_cast<unsigned>(TILE_CTAS * dev.sm_count);
        kernel<<<a.tiles < ctas ? a.tiles : ctas, THREADS, bytes, stream>>>(a);
    }
    return SGEMM_OK;
}

template <class T, bool E5M2>
int launch_type(const QuantizeProblem &p, const QArgs &a, bool vector, const DeviceInfo &dev, cudaStream_t stream) {
    if (p.block == SGEMM_FP8_ROWS) {
        const int64_t warps = p.rows * ((p.cols + WARP_VALUES - 1) / WARP_VALUES), per = THREADS / 32;
        const int64_t blocks = (warps + per - 1) / per;
        if (blocks > INT32_MAX) return SGEMM_ERR_UNSUPPORTED;
        auto kernel = vector ? quantize_rows_kernel<T, E5M2, true> : quantize_rows_kernel<T, E5M2, false>;
        kernel<<<static_cast<unsigned>(blocks), THREADS, 0, stream>>>(a);
    } else {
        const int rc = p.block == SGEMM_FP8_COLUMNS ? launch_tiles<T, E5M2, true>(a, vector, dev, stream)
                                                    : launch_tiles<T, E5M2, false>(a, vector, dev, stream);
        if (rc != SGEMM_OK) return rc;
    }
    return cudaGetLastError() == cudaSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

template <class T>
int launch_any(const QuantizeProblem &p, const QArgs &a, bool vector, const DeviceInfo &dev, cudaStream_t stream) {
    return p.to == SGEMM_FP8_E5M2 ? launch_type<T, true>(p, a, vector, dev, stream)
                                  : launch_type<T, false>(p, a, vector, dev, stream);
}

}  // namespace

int quantize_launch(const QuantizeProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    QArgs a{};
    a.rows = p.rows;
    a.cols = p.cols;
    const int64_t high = p.offsets ? sgemm_fp8_blocks(p.rows, p.experts) : blocks_of(p.rows), wide = blocks_of(p.cols);
    if (p.block != SGEMM_FP8_ROWS && (high > INT32_MAX || wide > INT32_MAX || high * wide > INT32_MAX / p.items))
        return SGEMM_ERR_UNSUPPORTED;
    a.high = static_cast<unsigned>(high);
    a.wide = static_cast<unsigned>(wide);
    a.tiles = static_cast<unsigned>(high * wide * p.items);
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
        rc = launch_any<float>(p, a, vector, dev, stream);
    else if (p.type == SGEMM_TYPE_BF16)
        rc = launch_any<__nv_bfloat16>(p, a, vector, dev, stream);
    else
        rc = launch_any<__half>(p, a, vector, dev, stream);
    if (rc == SGEMM_OK)
        ++*launches;
    else
        cudaGetLastError();
    return rc;
}

}  // namespace f8
}  // namespace sgemm
