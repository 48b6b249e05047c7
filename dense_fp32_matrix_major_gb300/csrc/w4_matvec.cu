// Matrix-vector products with 4-bit weights and group scales:
//
//     y[r][n] = sum_g scale[n][g] * sum_{k in g} (q[n][k] - zero[n][g]) x[r][k]
//
// for up to eight rows r at a time that share a matrix. Bound by reading q:
// half a byte per weight, so the instructions spent on a weight have to be
// few: at 6.8 TB/s an SM has about 170 issue slots for the 1 KB of q that a
// warp takes in a step.
//
// Arithmetic. The inner sums run on warp matrix instructions (16 rows of q x
// 16 k x 8 rows of x, fp32 sums) with the rows of x as the narrow side; eight
// is their width, which is why eight rows share a pass. (tcgen05 wants its
// operands in shared or tensor memory and 128 rows a tile; here the weights
// go from global memory to registers once and are used once.) Each group's
// inner sum is scaled in fp32. How a 4-bit q becomes an operand:
//   * fp16 x: q in the low bits of an fp16 number is q 2^-24 exactly (a
//     subnormal), so masking is all; the group's sum is
//     2^24 sum (q 2^-24) x - zero sum x.
//   * bf16 x: q in the low bits of 128.0 (last place 1) is 128 + q exactly;
//     the group's sum is sum (128 + q) x - (128 + zero) sum x. The subtraction
//     costs up to four of the 24 bits of the fp32 sums, of which a bf16
//     result keeps 8.
//   * fp32 x: cut into three bf16 terms that add up to it (3 x 8 bits cover
//     its 24), each multiplied exactly by q - zero, taken from 128 + q by
//     subtracting 128 + zero before the product, so no bits are lost.
// The sums of x per group are made in fp32 when x is staged. One 32-bit word
// holds k = 0 .. 7; masking it shifted by 4 j gives the pair (j, j + 4), so x
// is laid out in shared memory in the order 0 4 1 5 2 6 3 7. An infinity or
// NaN in 16-bit x would turn the subtraction into NaN; rows of x that hold
// one are recomputed with scalar arithmetic.
//
// Work. A block takes 16 * row_tiles rows of q; its 8 warps are row_tiles
// tiles times 8 / row_tiles interleaved shares of k, joined in shared memory.
// A warp's step is 16 rows x 128 k; the q of its next two steps are on their
// way before x is staged and while a step is multiplied.
#include <cuda_runtime.h>
#include <stdint.h>

#include "experts_common.cuh"
#include "experts_internal.h"

namespace sgemm {
namespace ex {
namespace {

constexpr int W4_THREADS = 256;
constexpr int W4_WARPS = W4_THREADS / 32;
constexpr int W4_ROWS = 8;    // rows of x that share a pass
constexpr int STEP = 128;     // values of k per warp step
constexpr int AHEAD = 2;      // steps whose weights are on their way
constexpr int TURN = 4;       // steps between fetches of scales (width 128)

struct W4Args {
    int rows, experts;
    int64_t N, K;
    int groups;       // per row of q
    int group_shift;  // log2 of the group
    int row_tiles;    // 16-row tiles per block: 1, 2, 4 or 8
    int chunk_steps;  // steps of x staged at once, a multiple of the shares
    int x_vector;     // rows of x in 16-byte pieces
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

// How a row type enters the matrix instruction: terms of x, the bits that q is
// placed in, whether zero points are subtracted from the operand (EXACT) or
// from the group's sum (BASE: what an operand holds on top of q, UNIT: what an
// operand's 1 is worth), and the instruction itself.
template <class T>
struct Operand;

template <>
struct Operand<__nv_bfloat16> {
    static constexpr int TERMS = 1;
    static constexpr bool EXACT = false;
    static constexpr uint32_t ONE = 0x43004300u;  // 128, 128 in bf16
    static constexpr float BASE = 128.0f, UNIT = 1.0f;
    static constexpr int BLOCKS = 4;           // per SM
    static constexpr int X_BYTES = 48 * 1024;  // shared memory for x
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
    static constexpr bool EXACT = false;
    static constexpr uint32_t ONE = 0;
    static constexpr float BASE = 0.0f, UNIT = 16777216.0f;  // an operand's q is q 2^-24
    static constexpr int BLOCKS = 4;
    static constexpr int X_BYTES = 48 * 1024;
    static __device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t) { return a; }
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
    static constexpr bool EXACT = true;
    static constexpr uint32_t ONE = Operand<__nv_bfloat16>::ONE;
    static constexpr float BASE = 0.0f, UNIT = 1.0f;
    static constexpr int BLOCKS = 3;
    static constexpr int X_BYTES = 72 * 1024;
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

// How the k of a step lie in a lane's four words, by the width of the groups.
//   128: words 0 .. 3 are k = 32 t + 8 u: 16 bytes a lane, one group (or half
//        of one) a step.
//   64:  words 2 h, 2 h + 1 are k = 64 h + 16 t + 8 (u & 1): 8 bytes a lane
//        for each 64 k, one group.
//   32:  as 64, then lanes t and t ^ 2 exchange a word, so that word 2 h + b of
//        all four lanes is the b-th 32 k of that half.
template <int WIDTH>
__device__ __forceinline__ int k_of(int u, int t) {
    if (WIDTH == 128) return 32 * t + 8 * u;
    if (WIDTH == 64) return 64 * (u >> 1) + 16 * t + 8 * (u & 1);
    return 32 * u + 16 * (t & 1) + 8 * (t >> 1);
}

// BYTES bytes of a row of q at k (aligned: BYTES / 2 divides k and the row).
template <int BYTES, bool ALIGNED>
__device__ __forceinline__ void load_q(const uint8_t *row, int k, int K, uint32_t *w) {
    if constexpr (ALIGNED && BYTES == 16) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "l"(row + k / 2));
    } else if constexpr (ALIGNED) {
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                     : "=r"(w[0]), "=r"(w[1])
                     : "l"(row + k / 2));
    } else {
#pragma unroll
        for (int i = 0; i < BYTES / 4; ++i) {
            w[i] = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int kk = k + 8 * i + 2 * b;
                if (kk < K) w[i] |= static_cast<uint32_t>(__ldg(row + kk / 2)) << (8 * b);
            }
        }
    }
}

// One step of a lane: 32 values of k of rows g and g + 8.
struct Weights {
    uint32_t lo[4], hi[4];
};

// Scales and zero points of rows g (low half of z) and g + 8 that a lane
// fetched: for width 128 those of step t of four, otherwise those of the t-th
// 32 values of one step.
struct Scales {
    float lo, hi;
    uint32_t z;
};

// y[r][n] with scalar arithmetic, for rows of x that hold infinities or NaN.
template <class T>
__device__ __noinline__ float scalar_row(const W4Args &a, int64_t row, const T *x) {
    float s = 0.0f;
    for (int64_t k = 0; k < a.K; ++k) {
        const int64_t gi = row * a.groups + (k >> a.group_shift);
        const int v = (__ldg(a.q + row * (a.K / 2) + k / 2) >> (4 * (k & 1))) & 15;
        const int z = a.zeros ? __ldg(a.zeros + gi) & 15 : 8;
        s = fmaf(static_cast<float>(v - z) * scale_at(a, gi), to_f32(x[k]), s);
    }
    return s;
}

template <class T, int WIDTH, bool ALIGNED>
__global__ void __launch_bounds__(W4_THREADS, Operand<T>::BLOCKS) w4_kernel(const __grid_constant__ W4Args a) {
    using Op = Operand<T>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int members[W4_ROWS];
    __shared__ int member_count;
    __shared__ int odd_row[W4_ROWS];  // the row holds an infinity or NaN (16-bit x)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int64_t n_first = static_cast<int64_t>(blockIdx.x) * 16 * a.row_tiles;
    T *y = static_cast<T *>(a.y);
    if (threadIdx.x < W4_ROWS) odd_row[threadIdx.x] = 0;

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

    const int shares = W4_WARPS / a.row_tiles;
    const int tile = warp / shares, share = warp % shares;
    // Rows of q of this lane: n0 + g and n0 + g + 8; past the last row they
    // repeat it and are not written.
    const int64_t n0 = n_first + 16 * tile;
    const int64_t row_lo = static_cast<int64_t>(expert) * a.N + min(n0 + g, a.N - 1);
    const int64_t row_hi = static_cast<int64_t>(expert) * a.N + min(n0 + g + 8, a.N - 1);
    const uint8_t *q_lo = a.q + row_lo * (a.K / 2), *q_hi = a.q + row_hi * (a.K / 2);
    const int64_t g_lo = row_lo * a.groups, g_hi = row_hi * a.groups;
    const int K = static_cast<int>(a.K);
    const int steps = (K + STEP - 1) / STEP;
    auto fetch = [&](int st, Weights &w) {
        const int k = st * STEP;
        if (k + STEP <= K || !ALIGNED) {  // whole, or checked byte by byte
            if (WIDTH == 128) {
                load_q<16, ALIGNED>(q_lo, k + 32 * t, K, w.lo);
                load_q<16, ALIGNED>(q_hi, k + 32 * t, K, w.hi);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    load_q<8, ALIGNED>(q_lo, k + 64 * h + 16 * t, K, w.lo + 2 * h);
                    load_q<8, ALIGNED>(q_hi, k + 64 * h + 16 * t, K, w.hi + 2 * h);
                }
            }
        } else {
            // The last step of a K that is a multiple of 32: lanes past it get zeros.
#pragma unroll
            for (int u = 0; u < 4; ++u) w.lo[u] = w.hi[u] = 0;
            if (WIDTH == 128) {
                if (k + 32 * t < K) {
                    load_q<16, ALIGNED>(q_lo, k + 32 * t, K, w.lo);
                    load_q<16, ALIGNED>(q_hi, k + 32 * t, K, w.hi);
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (k + 64 * h + 16 * t < K) {
                        load_q<8, ALIGNED>(q_lo, k + 64 * h + 16 * t, K, w.lo + 2 * h);
                        load_q<8, ALIGNED>(q_hi, k + 64 * h + 16 * t, K, w.hi + 2 * h);
                    }
            }
        }
    };
    auto fetch_scales = [&](int k) {  // the groups that hold value k of both rows
        Scales s;
        s.lo = s.hi = 0.0f;
        s.z = 0x00080008u;
        if (k < K) {
            const int gi = k >> a.group_shift;
            s.lo = scale_at(a, g_lo + gi);
            s.hi = scale_at(a, g_hi + gi);
            if (a.zeros)
                s.z = (__ldg(a.zeros + g_lo + gi) & 15u) | (static_cast<uint32_t>(__ldg(a.zeros + g_hi + gi) & 15u) << 16);
        }
        return s;
    };
    // Width 128: a quad's lanes fetch the scales of a turn's four steps;
    // otherwise each step's come with its weights.
    auto turn_scales = [&](int i0) { return fetch_scales((share + (i0 + t) * shares) * STEP); };
    static_assert(TURN == 4 && TURN % AHEAD == 0, "a quad's lanes fetch the scales of a turn");
    Weights ring[AHEAD];
    Scales of_step[AHEAD], turn{}, next{};
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
        const int st = share + i * shares;
        if (st < steps) fetch(st, ring[i]);
        if (WIDTH < 128) of_step[i] = fetch_scales(st * STEP + 32 * t);
    }
    if (WIDTH == 128) next = turn_scales(0);

    // A chunk of x in shared memory: term, step, unit u, row, lane t, 8 values
    // (k_of); zeros past the end of k. Behind it the sums of x over every 32 k
    // (width 32), 64 or 128: step, group, row.
    constexpr int SUMS = 128 / WIDTH;  // per step
    float *x_sums = reinterpret_cast<float *>(smem + static_cast<size_t>(Op::TERMS) * a.chunk_steps * 256 * nb);
    auto stage = [&](int first_step) {
        __syncthreads();
        const int here = min(a.chunk_steps, steps - first_step);
        const int per_row = here * 16, total = per_row * nb;
        for (int i0 = 0; i0 < total; i0 += W4_THREADS) {
            const int i = i0 + static_cast<int>(threadIdx.x);
            const bool in_range = i < total;  // for whole sixteenths of a block
            const int r = in_range ? i / per_row : 0, o = in_range ? i - r * per_row : 0;
            const int st = o >> 4, piece = o & 15;
            // Which unit of which lane holds values 8 piece .. 8 piece + 7.
            const int u = WIDTH == 128 ? piece & 3 : WIDTH == 64 ? 2 * (piece >> 3) + (piece & 1) : piece >> 2;
            const int tt = WIDTH == 128 ? piece >> 2
                                        : WIDTH == 64 ? (piece >> 1) & 3 : ((piece >> 1) & 1) + 2 * (piece & 1);
            const int k = first_step * STEP + o * 8;
            T in[8];
            if (in_range && a.x_vector && k + 8 <= K) {
                const T *src = static_cast<const T *>(a.x) + members[r] * a.ldx + k;
                constexpr int PER = 16 / sizeof(T);
#pragma unroll
                for (int j = 0; j < 8; j += PER) {
                    const Pack<T, PER> v = load_pack<T, PER>(src + j);
#pragma unroll
                    for (int m = 0; m < PER; ++m) in[j + m] = v.v[m];
                }
            } else {
                const T *src = static_cast<const T *>(a.x) + members[r] * a.ldx;
#pragma unroll
                for (int j = 0; j < 8; ++j) in[j] = in_range && k + j < K ? src[k + j] : from_f32<T>(0.0f);
            }
            uint16_t v[Op::TERMS][8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint16_t terms[Op::TERMS];
                Op::split(in[j], terms);
#pragma unroll
                for (int m = 0; m < Op::TERMS; ++m) v[m][(j & 3) * 2 + (j >> 2)] = terms[m];
            }
            if (in_range) {
#pragma unroll
                for (int m = 0; m < Op::TERMS; ++m) {
                    uint4 w;
                    w.x = v[m][0] | (static_cast<uint32_t>(v[m][1]) << 16);
                    w.y = v[m][2] | (static_cast<uint32_t>(v[m][3]) << 16);
                    w.z = v[m][4] | (static_cast<uint32_t>(v[m][5]) << 16);
                    w.w = v[m][6] | (static_cast<uint32_t>(v[m][7]) << 16);
                    reinterpret_cast<uint4 *>(smem)[((m * a.chunk_steps + st) * 4 + u) * nb * 4 + r * 4 + tt] = w;
                }
            }
            if (!Op::EXACT) {
                float s = 0.0f, odd = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s += to_f32(in[j]);
                    odd = fmaf(to_f32(in[j]), 0.0f, odd);  // NaN for an infinity or NaN
                }
                if (odd != 0.0f) odd_row[r] = 1;
#pragma unroll
                for (int d = 1; d < WIDTH / 8; d *= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
                if (in_range && piece % (WIDTH / 8) == 0)
                    x_sums[(st * SUMS + piece / (WIDTH / 8)) * W4_ROWS + r] = s;
            }
        }
        __syncthreads();
    };

    float sum[4] = {};
    auto multiply = [&](Weights &w, const Scales &sc, int j, int st) {  // st: step within the chunk
        if (WIDTH == 32) {
            // Word 2 h + 1 of lanes 0, 1 for word 2 h of lanes 2, 3.
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t sl = __shfl_xor_sync(0xffffffffu, t < 2 ? w.lo[2 * h + 1] : w.lo[2 * h], 2);
                const uint32_t sh = __shfl_xor_sync(0xffffffffu, t < 2 ? w.hi[2 * h + 1] : w.hi[2 * h], 2);
                if (t < 2) {
                    w.lo[2 * h + 1] = sl;
                    w.hi[2 * h + 1] = sh;
                } else {
                    w.lo[2 * h] = sl;
                    w.hi[2 * h] = sh;
                }
            }
        }
        // One accumulator per chain of dependent products.
        constexpr int CHAINS = Op::TERMS == 1 ? 2 : Op::TERMS;
        float c[CHAINS][4] = {};
        float s_lo = 0.0f, s_hi = 0.0f;
        uint32_t z = 0, z_lo = 0, z_hi = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (u % (WIDTH / 32) == 0) {  // a group starts
                const int from = (lane & ~3) | (WIDTH == 128 ? j : u);
                s_lo = __shfl_sync(0xffffffffu, sc.lo, from);
                s_hi = __shfl_sync(0xffffffffu, sc.hi, from);
                z = __shfl_sync(0xffffffffu, sc.z, from);
                z_lo = Op::ONE | (z & 0xFFFFu) | (z << 16);
                z_hi = Op::ONE | (z >> 16) | (z & 0xFFFF0000u);
            }
            uint4 xv[Op::TERMS];
#pragma unroll
            for (int m = 0; m < Op::TERMS; ++m) {
                xv[m] = make_uint4(0, 0, 0, 0);
                if (g < nb)
                    xv[m] = reinterpret_cast<const uint4 *>(
                        smem)[((m * a.chunk_steps + st) * 4 + u) * nb * 4 + g * 4 + t];
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t f[4];
                f[0] = ((w.lo[u] >> (8 * half)) & 0x000F000Fu) | Op::ONE;
                f[1] = ((w.hi[u] >> (8 * half)) & 0x000F000Fu) | Op::ONE;
                f[2] = ((w.lo[u] >> (8 * half + 4)) & 0x000F000Fu) | Op::ONE;
                f[3] = ((w.hi[u] >> (8 * half + 4)) & 0x000F000Fu) | Op::ONE;
                if (Op::EXACT) {
                    f[0] = Op::minus(f[0], z_lo);
                    f[1] = Op::minus(f[1], z_hi);
                    f[2] = Op::minus(f[2], z_lo);
                    f[3] = Op::minus(f[3], z_hi);
                }
#pragma unroll
                for (int m = 0; m < Op::TERMS; ++m)
                    Op::mma(c[Op::TERMS == 1 ? half : m], f, half ? xv[m].z : xv[m].x, half ? xv[m].w : xv[m].y);
            }
            if ((u + 1) % (WIDTH / 32) == 0) {  // the group ends
                float d[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // small terms first
                    d[i] = c[CHAINS - 1][i];
#pragma unroll
                    for (int m = CHAINS - 2; m >= 0; --m) d[i] += c[m][i];
#pragma unroll
                    for (int m = 0; m < CHAINS; ++m) c[m][i] = 0.0f;
                }
                if (!Op::EXACT) {
                    const float2 xs = *reinterpret_cast<const float2 *>(
                        x_sums + (st * SUMS + u / (WIDTH / 32)) * W4_ROWS + 2 * t);
                    const float b_lo = Op::BASE + static_cast<float>(z & 0xFFFFu);
                    const float b_hi = Op::BASE + static_cast<float>(z >> 16);
                    d[0] = fmaf(d[0], Op::UNIT, -b_lo * xs.x);
                    d[1] = fmaf(d[1], Op::UNIT, -b_lo * xs.y);
                    d[2] = fmaf(d[2], Op::UNIT, -b_hi * xs.x);
                    d[3] = fmaf(d[3], Op::UNIT, -b_hi * xs.y);
                }
                sum[0] = fmaf(s_lo, d[0], sum[0]);
                sum[1] = fmaf(s_lo, d[1], sum[1]);
                sum[2] = fmaf(s_hi, d[2], sum[2]);
                sum[3] = fmaf(s_hi, d[3], sum[3]);
            }
        }
    };

    // Every warp goes through the same number of steps, so that all meet at
    // the chunks; those past the end are not multiplied.
    const int per_chunk = a.chunk_steps / shares;
    const int count = (steps + shares - 1) / shares;
    int in_chunk = 0, first_step = 0;
    if (count > 0) stage(0);
    for (int i0 = 0; i0 < count; i0 += TURN) {
        if (WIDTH == 128) {
            turn = next;
            next = turn_scales(i0 + TURN);
        }
#pragma unroll
        for (int j = 0; j < TURN; ++j) {
            const int i = i0 + j;
            if (i >= count) break;
            if (in_chunk == per_chunk) {
                in_chunk = 0;
                first_step += a.chunk_steps;
                stage(first_step);
            }
            const int st = share + i * shares, slot = j % AHEAD;
            if (st < steps) multiply(ring[slot], WIDTH == 128 ? turn : of_step[slot], j, st - first_step);
            const int ahead = st + AHEAD * shares;
            if (ahead < steps) fetch(ahead, ring[slot]);
            if (WIDTH < 128) of_step[slot] = fetch_scales(ahead * STEP + 32 * t);
            ++in_chunk;
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
        if (!Op::EXACT && odd_row[r])
            s = scalar_row(a, static_cast<int64_t>(expert) * a.N + n_first + n,
                           static_cast<const T *>(a.x) + members[r] * a.ldx);
        y[members[r] * a.ldy + n_first + n] = from_f32<T>(s);
    }
}

template <class T, int WIDTH, bool ALIGNED>
int launch(W4Args a, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    auto kernel = w4_kernel<T, WIDTH, ALIGNED>;
    using Op = Operand<T>;
    const int64_t passes = a.ids ? a.rows : (a.rows + W4_ROWS - 1) / W4_ROWS;
    const int nb = a.rows < W4_ROWS ? a.rows : W4_ROWS;
    // Passes with work in them, and rows of x in one, as far as the host knows.
    const int64_t busy = a.ids && a.experts < passes ? a.experts : passes;
    const int64_t share_x = a.rows / busy < 1 ? 1 : (a.rows / busy < W4_ROWS ? a.rows / busy : W4_ROWS);
    // Rows of q per block: few give every SM its part, many pay once for x and
    // for a block's start (about the time of 16 KB of q). The choice makes the
    // busiest SM's bytes least, an SM with fewer blocks than it has room for
    // counting as full: its warps are too few to keep it busy.
    int tiles = 1;
    int64_t least = INT64_MAX;
    for (int t = 1; t <= W4_WARPS; t *= 2) {
        const int64_t blocks = (a.N + 16 * t - 1) / (16 * t) * busy;
        int64_t per_sm = (blocks + dev.sm_count - 1) / dev.sm_count;
        if (per_sm < Op::BLOCKS) per_sm = Op::BLOCKS;
        const int64_t cost = per_sm * (t * 8 * a.K + share_x * a.K * static_cast<int64_t>(sizeof(T)) + 16384);
        if (cost < least) {
            least = cost;
            tiles = t;
        }
    }
    a.row_tiles = tiles;
    const int shares = W4_WARPS / tiles;
    const int step_bytes = nb * 2 * Op::TERMS * STEP, sum_bytes = Op::EXACT ? 0 : 128 / WIDTH * W4_ROWS * 4;
    const int64_t all = ((a.K + STEP - 1) / STEP + shares - 1) / shares * shares;
    int64_t chunk = Op::X_BYTES / (step_bytes + sum_bytes) / shares * shares;
    if (chunk > all) chunk = all;
    a.chunk_steps = static_cast<int>(chunk);
    a.x_vector = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx * static_cast<int64_t>(sizeof(T)) % 16 == 0;
    size_t smem = static_cast<size_t>(chunk) * (step_bytes + sum_bytes);
    if (smem < W4_WARPS * 8 * 16 * sizeof(float)) smem = W4_WARPS * 8 * 16 * sizeof(float);
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Op::X_BYTES) != cudaSuccess) {
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
int launch_type(const W4Args &a, int64_t group, bool aligned, const DeviceInfo &dev, cudaStream_t stream,
                int *launches) {
    if (group >= 128)
        return aligned ? launch<T, 128, true>(a, dev, stream, launches)
                       : launch<T, 128, false>(a, dev, stream, launches);
    if (group == 64)
        return aligned ? launch<T, 64, true>(a, dev, stream, launches) : launch<T, 64, false>(a, dev, stream, launches);
    return aligned ? launch<T, 32, true>(a, dev, stream, launches) : launch<T, 32, false>(a, dev, stream, launches);
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
    if (p.type == SGEMM_TYPE_F32) return launch_type<float>(a, p.group, aligned, dev, stream, launches);
    if (p.type == SGEMM_TYPE_BF16) return launch_type<__nv_bfloat16>(a, p.group, aligned, dev, stream, launches);
    return launch_type<__half>(a, p.group, aligned, dev, stream, launches);
}

}  // namespace ex
}  // namespace sgemm
