// Matrix-vector products with 4-bit weights and group scales:
//
//     y[r][n] = sum_g scale[n][g] * sum_{k in g} (q[n][k] - zero[n][g]) x[r][k]
//
// for up to eight rows r at a time that share a matrix. Bound by reading q:
// half a byte per weight, so the arithmetic has to keep out of the way.
//
// Arithmetic. q - zero is a whole number of magnitude at most 15, exact in
// bf16 and fp16, so the inner sums run on warp matrix instructions
// (16 rows of q x 16 k x 8 rows of x, fp32 sums) with the rows of x as the
// narrow side; eight is their width, which is why eight rows share a pass.
// (tcgen05 wants its operands in shared or tensor memory and 128 rows a
// tile; here the weights go from global memory to registers once and are
// used once.) The inner sum of a group is scaled in fp32. x in bf16 or fp16
// goes in as it is. x in fp32 is cut into three bf16 terms that add up to it
// (3 x 8 bits cover its 24), each multiplied exactly.
//
// A 4-bit value v becomes floating point by placing it in the low bits of
// the number 2^7 (bf16, whose last place there is 1) or 2^10 (fp16), and
// subtracting 2^7 + zero (2^10 + zero): both exact. One 32-bit word holds
// k = 0 .. 7; masking it shifted by 4 j gives the pair (j, j + 4), so x is
// laid out in shared memory in the order 0 4 1 5 2 6 3 7.
//
// Work. A block takes 16 * row_tiles rows of q; its 16 warps are row_tiles
// tiles times 16 / row_tiles interleaved shares of k, joined in shared
// memory. Four lanes load 64 contiguous bytes of a row, 128 values of k.
#include <cuda_runtime.h>
#include <stdint.h>

#include "experts_common.cuh"
#include "experts_internal.h"

namespace sgemm {
namespace ex {
namespace {

constexpr int W4_THREADS = 512;
constexpr int W4_WARPS = W4_THREADS / 32;
constexpr int W4_ROWS = 8;    // rows of x that share a pass
constexpr int STEP = 128;     // values of k per warp step
constexpr int AHEAD = 4;      // steps whose weights a warp loads at once
constexpr int X_BYTES = 96 * 1024;  // shared memory for x

struct W4Args {
    int rows, experts;
    int64_t N, K;
    int groups;       // per row of q
    int group_shift;  // log2 of the group
    int row_tiles;    // 16-row tiles per block: 1, 2, 4 or 8
    int chunk;        // values of k staged at once, a multiple of STEP
    int nb;           // rows of x that shared memory has room for
    const int32_t *ids;
    const void *x;
    int64_t ldx;
    const uint8_t *q;
    const void *scales;
    int scale_type;
    const uint8_t *zeros;
    void *y;
    int64_t ldy;
};

// How a row type enters the matrix instruction: terms of x, the bits of 2^7
// or 2^10, and the instruction itself.
template <class T>
struct Operand;

template <>
struct Operand<__nv_bfloat16> {
    static constexpr int TERMS = 1;
    static constexpr uint32_t ONE = 0x43004300u;  // 128, 128 in bf16
    static __device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t b) {
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&d);
    }
    static __device__ __forceinline__ void split(__nv_bfloat16 x, uint16_t (&t)[1]) { t[0] = __bfloat16_as_ushort(x); }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

template <>
struct Operand<__half> {
    static constexpr int TERMS = 1;
    static constexpr uint32_t ONE = 0x64006400u;  // 1024, 1024 in fp16
    static __device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t b) {
        const __half2 d = __hsub2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&d);
    }
    static __device__ __forceinline__ void split(__half x, uint16_t (&t)[1]) { t[0] = __half_as_ushort(x); }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

template <>
struct Operand<float> {
    static constexpr int TERMS = 3;
    static constexpr uint32_t ONE = Operand<__nv_bfloat16>::ONE;
    static __device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t b) {
        return Operand<__nv_bfloat16>::minus(a, b);
    }
    // The top 16 bits of x are a bf16 (truncated, so it cannot overflow); what
    // is left is exact in fp32 and is cut the same way. Infinities and NaN go
    // whole into the first term (a NaN kept a NaN).
    static __device__ __forceinline__ void split(float x, uint16_t (&t)[3]) {
        uint32_t bits = __float_as_uint(x);
        if ((bits & 0x7F800000u) == 0x7F800000u) {
            t[0] = static_cast<uint16_t>((bits >> 16) | ((bits & 0x007FFFFFu) ? 0x0040u : 0u));
            t[1] = t[2] = 0;
            return;
        }
        t[0] = static_cast<uint16_t>(bits >> 16);
        x -= __uint_as_float(bits & 0xFFFF0000u);
        bits = __float_as_uint(x);
        t[1] = static_cast<uint16_t>(bits >> 16);
        x -= __uint_as_float(bits & 0xFFFF0000u);
        t[2] = static_cast<uint16_t>(__float_as_uint(x) >> 16);
    }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        Operand<__nv_bfloat16>::mma(c, a, b0, b1);
    }
};

__device__ __forceinline__ float scale_at(const W4Args &a, int64_t i) {
    if (a.scale_type == SGEMM_TYPE_F32) return __ldg(static_cast<const float *>(a.scales) + i);
    const uint16_t h = __ldg(static_cast<const uint16_t *>(a.scales) + i);
    return a.scale_type == SGEMM_TYPE_BF16 ? __uint_as_float(static_cast<uint32_t>(h) << 16)
                                           : __half2float(__ushort_as_half(h));
}

// 16 bytes of a row of q from k on (32 values); zeros past the row's end.
template <bool ALIGNED>
__device__ __forceinline__ uint4 load_q(const uint8_t *row, int64_t k, int64_t K) {
    if (ALIGNED) return k < K ? __ldcs(reinterpret_cast<const uint4 *>(row + k / 2)) : make_uint4(0, 0, 0, 0);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int64_t kk = k + 8 * i + 2 * b;
            if (kk < K) w[i] |= static_cast<uint32_t>(__ldg(row + kk / 2)) << (8 * b);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Words of the four lanes of a quad transposed: lane t's word u becomes lane
// u's word t.
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4], int t) {
#pragma unroll
    for (int r = 1; r < 4; ++r) {
        // Exchange word t ^ r with the lane t ^ r.
        uint32_t send = w[0];
#pragma unroll
        for (int i = 1; i < 4; ++i) send = (t ^ r) == i ? w[i] : send;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, send, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (t ^ r) == i ? got : w[i];
    }
}

// WIDE: groups of 128 or more, so that one step of a row has one scale and a
// lane's 16 bytes are its own k. Otherwise the quad's words are transposed,
// so that each pair of matrix instructions covers 32 consecutive k.
template <class T, bool WIDE, bool ALIGNED>
__global__ void __launch_bounds__(W4_THREADS, 1) w4_kernel(const W4Args a) {
    using Op = Operand<T>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int members[W4_ROWS];
    __shared__ int member_count;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int64_t n_first = static_cast<int64_t>(blockIdx.x) * 16 * a.row_tiles;
    T *y = static_cast<T *>(a.y);

    // Rows of x that this block serves: eight consecutive ones, or, with ids,
    // this row and the next seven of the same expert where an eighth of them
    // starts here.
    int expert = 0, nb = 0;
    if (!a.ids) {
        const int r0 = static_cast<int>(blockIdx.y) * W4_ROWS;
        nb = min(W4_ROWS, a.rows - r0);
        if (threadIdx.x < W4_ROWS) members[threadIdx.x] = r0 + static_cast<int>(threadIdx.x);
    } else {
        const int r = static_cast<int>(blockIdx.y);
        expert = __ldg(a.ids + r);
        if (expert < 0 || expert >= a.experts) {
            for (int64_t n = n_first + threadIdx.x; n < min(a.N, n_first + 16 * a.row_tiles); n += W4_THREADS)
                y[r * a.ldy + n] = from_f32<T>(0.0f);
            return;
        }
        int before = 0;
        for (int r0 = 0; r0 < r; r0 += W4_THREADS) {
            const int i = r0 + static_cast<int>(threadIdx.x);
            before += __syncthreads_count(i < r && __ldg(a.ids + i) == expert);
        }
        if (before % W4_ROWS != 0) return;
        if (warp == 0) {
            int have = 0;
            for (int r0 = r; r0 < a.rows && have < W4_ROWS; r0 += 32) {
                const bool mine = r0 + lane < a.rows && __ldg(a.ids + r0 + lane) == expert;
                const unsigned all = __ballot_sync(0xffffffffu, mine);
                const int at = have + __popc(all & ((1u << lane) - 1u));
                if (mine && at < W4_ROWS) members[at] = r0 + lane;
                have += __popc(all);
            }
            if (lane == 0) member_count = min(have, W4_ROWS);
        }
        __syncthreads();
        nb = member_count;
    }
    __syncthreads();

    const int shares = W4_WARPS / a.row_tiles;
    const int tile = warp / shares, share = warp % shares;
    // Rows of q of this lane: n0 + g and n0 + g + 8; past the last row they
    // repeat it and are not written.
    const int64_t n0 = n_first + 16 * tile;
    const int64_t row_lo = static_cast<int64_t>(expert) * a.N + min(n0 + g, a.N - 1);
    const int64_t row_hi = static_cast<int64_t>(expert) * a.N + min(n0 + g + 8, a.N - 1);
    const uint8_t *q_lo = a.q + row_lo * (a.K / 2), *q_hi = a.q + row_hi * (a.K / 2);
    float sum[4] = {};

    for (int64_t c0 = 0; c0 < a.K; c0 += a.chunk) {
        const int64_t c1 = min(a.K, c0 + a.chunk);
        const int steps = static_cast<int>((c1 - c0 + STEP - 1) / STEP);
        // x of this chunk: term, step, unit u, row, lane t, 8 values. Unit u of
        // lane t covers k = 32 t + 8 u (WIDE) or 32 u + 8 t of the step.
        if (c0 > 0) __syncthreads();
        const int vecs = steps * 16 * nb;
        for (int i = threadIdx.x; i < vecs; i += W4_THREADS) {
            const int r = i / (steps * 16), o = i - r * (steps * 16);  // o: eighth of this row's chunk
            const int st = o >> 4, piece = o & 15;
            const int u = WIDE ? piece & 3 : piece >> 2, tt = WIDE ? piece >> 2 : piece & 3;
            const int64_t k = c0 + o * 8;
            const T *src = static_cast<const T *>(a.x) + members[r] * a.ldx + k;
            uint16_t v[Op::TERMS][8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint16_t terms[Op::TERMS];
                Op::split(k + j < a.K ? src[j] : from_f32<T>(0.0f), terms);
                const int at = (j & 3) * 2 + (j >> 2);
#pragma unroll
                for (int m = 0; m < Op::TERMS; ++m) v[m][at] = terms[m];
            }
#pragma unroll
            for (int m = 0; m < Op::TERMS; ++m) {
                const int64_t at = ((static_cast<int64_t>(m * steps + st) * 4 + u) * nb + r) * 4 + tt;
                uint4 w;
                w.x = v[m][0] | (static_cast<uint32_t>(v[m][1]) << 16);
                w.y = v[m][2] | (static_cast<uint32_t>(v[m][3]) << 16);
                w.z = v[m][4] | (static_cast<uint32_t>(v[m][5]) << 16);
                w.w = v[m][6] | (static_cast<uint32_t>(v[m][7]) << 16);
                reinterpret_cast<uint4 *>(smem)[at] = w;
            }
        }
        __syncthreads();
        for (int s0 = share; s0 < steps; s0 += shares * AHEAD) {
            uint4 lo[AHEAD], hi[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int64_t k = c0 + static_cast<int64_t>(s0 + i * shares) * STEP + t * 32;
                lo[i] = load_q<ALIGNED>(q_lo, k, c1);
                hi[i] = load_q<ALIGNED>(q_hi, k, c1);
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int st = s0 + i * shares;
                if (st >= steps) break;  // uniform over the warp
                uint32_t wl[4] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w};
                uint32_t wh[4] = {hi[i].x, hi[i].y, hi[i].z, hi[i].w};
                if (!WIDE) {
                    quad_transpose(wl, t);
                    quad_transpose(wh, t);
                }
                float c[4] = {};
                float s_lo = 0.0f, s_hi = 0.0f;
                uint32_t z_lo = 0, z_hi = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (u == 0 || !WIDE) {
                        const int64_t k = c0 + static_cast<int64_t>(st) * STEP + (WIDE ? 0 : 32 * u);
                        const int64_t gi = min(k >> a.group_shift, static_cast<int64_t>(a.groups - 1));
                        s_lo = scale_at(a, row_lo * a.groups + gi);
                        s_hi = scale_at(a, row_hi * a.groups + gi);
                        const uint32_t zl = a.zeros ? __ldg(a.zeros + row_lo * a.groups + gi) & 15u : 8u;
                        const uint32_t zh = a.zeros ? __ldg(a.zeros + row_hi * a.groups + gi) & 15u : 8u;
                        z_lo = Op::ONE | zl | (zl << 16);
                        z_hi = Op::ONE | zh | (zh << 16);
                    }
                    uint4 xv[Op::TERMS];
#pragma unroll
                    for (int m = 0; m < Op::TERMS; ++m) {
                        xv[m] = make_uint4(0, 0, 0, 0);
                        if (g < nb)
                            xv[m] = reinterpret_cast<const uint4 *>(
                                smem)[((static_cast<int64_t>(m * steps + st) * 4 + u) * nb + g) * 4 + t];
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t f[4];
                        f[0] = Op::minus(((wl[u] >> (8 * half)) & 0x000F000Fu) | Op::ONE, z_lo);
                        f[1] = Op::minus(((wh[u] >> (8 * half)) & 0x000F000Fu) | Op::ONE, z_hi);
                        f[2] = Op::minus(((wl[u] >> (8 * half + 4)) & 0x000F000Fu) | Op::ONE, z_lo);
                        f[3] = Op::minus(((wh[u] >> (8 * half + 4)) & 0x000F000Fu) | Op::ONE, z_hi);
#pragma unroll
                        for (int m = Op::TERMS - 1; m >= 0; --m)  // small terms first
                            Op::mma(c, f, half ? xv[m].z : xv[m].x, half ? xv[m].w : xv[m].y);
                    }
                    if (!WIDE || u == 3) {
                        sum[0] = fmaf(s_lo, c[0], sum[0]);
                        sum[1] = fmaf(s_lo, c[1], sum[1]);
                        sum[2] = fmaf(s_hi, c[2], sum[2]);
                        sum[3] = fmaf(s_hi, c[3], sum[3]);
                        c[0] = c[1] = c[2] = c[3] = 0.0f;
                    }
                }
            }
        }
    }
    // Join the shares: part[warp][row of x][16 rows of q].
    __syncthreads();
    float *part = reinterpret_cast<float *>(smem);
    part[(warp * 8 + 2 * t) * 16 + g] = sum[0];
    part[(warp * 8 + 2 * t + 1) * 16 + g] = sum[1];
    part[(warp * 8 + 2 * t) * 16 + g + 8] = sum[2];
    part[(warp * 8 + 2 * t + 1) * 16 + g + 8] = sum[3];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * a.row_tiles * nb; i += W4_THREADS) {
        const int r = i / (16 * a.row_tiles), n = i - r * (16 * a.row_tiles);
        if (n_first + n >= a.N) continue;
        const int w0 = (n >> 4) * shares;
        float s = 0.0f;
        for (int w = 0; w < shares; ++w) s += part[((w0 + w) * 8 + r) * 16 + (n & 15)];
        y[members[r] * a.ldy + n_first + n] = from_f32<T>(s);
    }
}

template <class T, bool WIDE, bool ALIGNED>
int launch(W4Args a, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    auto kernel = w4_kernel<T, WIDE, ALIGNED>;
    const int64_t passes = a.ids ? a.rows : (a.rows + W4_ROWS - 1) / W4_ROWS;
    const int nb = a.rows < W4_ROWS ? a.rows : W4_ROWS;
    // Every block stages all of x, so a block takes enough rows of q that x
    // is at most half of what it reads (16 K / 2 bytes a tile), as long as
    // that leaves a block for every SM.
    int tiles = 1;
    while (tiles < 8 && tiles * 4 < nb * static_cast<int>(sizeof(T))) tiles *= 2;
    while (tiles > 1 && (a.N + 16 * tiles - 1) / (16 * tiles) * passes < dev.sm_count) tiles /= 2;
    a.row_tiles = tiles;
    const int per_k = nb * 2 * Operand<T>::TERMS;
    int64_t chunk = X_BYTES / per_k / STEP * STEP;
    const int64_t all = (a.K + STEP - 1) / STEP * STEP;
    if (chunk > all) chunk = all;
    a.chunk = static_cast<int>(chunk);
    a.nb = nb;
    size_t smem = static_cast<size_t>(chunk) * per_k;
    if (smem < W4_WARPS * 8 * 16 * sizeof(float)) smem = W4_WARPS * 8 * 16 * sizeof(float);
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, X_BYTES) != cudaSuccess) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    const int64_t gx = (a.N + 16 * tiles - 1) / (16 * tiles);
    if (gx > INT32_MAX || passes > 65535) return SGEMM_ERR_UNSUPPORTED;
    kernel<<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(passes)), W4_THREADS, smem, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return SGEMM_ERR_LAUNCH;
    ++*launches;
    return SGEMM_OK;
}

template <class T>
int launch_type(const W4Args &a, bool wide, bool aligned, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    if (wide)
        return aligned ? launch<T, true, true>(a, dev, stream, launches)
                       : launch<T, true, false>(a, dev, stream, launches);
    return aligned ? launch<T, false, true>(a, dev, stream, launches)
                   : launch<T, false, false>(a, dev, stream, launches);
}

}  // namespace

int w4_launch(const W4Problem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    W4Args a{};
    a.rows = static_cast<int>(p.rows);
    a.experts = static_cast<int>(p.experts);
    a.N = p.N;
    a.K = p.K;
    a.groups = static_cast<int>((p.K + p.group - 1) / p.group);
    a.group_shift = p.group == 32 ? 5 : p.group == 64 ? 6 : p.group == 128 ? 7 : 8;
    a.ids = p.ids;
    a.x = p.x;
    a.ldx = p.ldx;
    a.q = p.q;
    a.scales = p.scales;
    a.scale_type = p.scale_type;
    a.zeros = p.zeros;
    a.y = p.y;
    a.ldy = p.ldy;
    // Rows of q in 16-byte pieces.
    const bool aligned = p.K % 32 == 0 && reinterpret_cast<uintptr_t>(p.q) % 16 == 0;
    const bool wide = p.group >= STEP;
    if (p.type == SGEMM_TYPE_F32) return launch_type<float>(a, wide, aligned, dev, stream, launches);
    if (p.type == SGEMM_TYPE_BF16) return launch_type<__nv_bfloat16>(a, wide, aligned, dev, stream, launches);
    return launch_type<__half>(a, wide, aligned, dev, stream, launches);
}

}  // namespace ex
}  // namespace sgemm
