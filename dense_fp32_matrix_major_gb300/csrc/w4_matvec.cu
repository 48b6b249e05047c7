// Matrix-vector products with 4-bit weights and group scales:
//
//     y[r][n] = sum_g scale[n][g] * sum_{k in g} (q[n][k] - zero[n][g]) x[r][k]
//
// for up to eight rows r at a time that share a matrix. Bound by reading q:
// half a byte per weight, so the instructions spent on a weight have to be
// few: at 6.8 TB/s an SM has about 170 issue slots for the 1 KB of q that a
// warp takes in a step. In a row of calls: 1 x 4096 x 4096 bf16 8 us, 1 x 28672 x
// 4096 bf16 19.5 us (3.1 TB/s), fp16 16 us; 8 x 16384 x 8192 with zero points bf16
// 26.5 us, fp32 33 us; 16 rows of 16 experts, 2048 -> 4096, fp16 25 us. (Cold, alone:
// 13, 25, 23, 35, 41 and 31 us.) No unit is full where q is large: one bf16 row takes
// 57% of the issue slots and 61% of the ALU pipe, eight fp32 rows 53% and 41% of the
// tensor pipe, so it is the wait in each warp's chain of loads, masks and products
// that bounds it, with four warps a scheduler; where many experts share the
// SMs, also the start and the end of each pass.
//
// Arithmetic. The inner sums run on warp matrix instructions (16 rows of q x
// 16 k x 8 rows of x, fp32 sums) with the rows of x as the narrow side; eight
// is their width, which is why eight rows share a pass. (tcgen05 wants its
// operands in shared or tensor memory and 128 rows a tile; here the weights
// go from global memory to registers once and are used once.) Each group's
// inner sum is scaled in fp32. An operand is q - zero, exact in every type, so a
// value of x whose q is the zero point adds nothing, however large it is (taken
// from the sums instead, sum q x - zero sum x, it would leave its rounding
// errors there). How a 4-bit q becomes one:
//   * bf16 x: q in the low bits of 128.0 (last place 1) is 128 + q; 128 + zero
//     is subtracted.
//   * fp16 x: q in the low bits of an fp16 number is q 2^-24 (a subnormal),
//     four bits up it is 16 q 2^-24 (10 bits hold it), so masking is all; the
//     zero point is subtracted in the same place, the sums of the two places
//     are kept apart until the 16 is taken out, and the group's sum is scaled
//     by 2^24.
//   * fp32 x: cut into three bf16 terms that add up to it (3 x 8 bits cover
//     its 24), each multiplied as bf16 x is. A term is a column of the
//     instruction: one or two rows of x fill one (6 of 8 columns), three to
//     five two, up to eight three.
// One 32-bit word holds k = 0 .. 7; masking it shifted by 4 j gives the pair (j,
// j + 4), so x is laid out in shared memory in the order 0 4 1 5 2 6 3 7 (fp16:
// 0 4 2 6 1 5 3 7, the unshifted and four bits up apart). A sum that is not
// finite, though its row of x is, is made again with scalar arithmetic in 64
// bits: a group's sum may overflow before it is scaled where the result does not.
// (Infinities and NaN of x need none of this: operands are exact, so the products
// and sums are IEEE's already.)
//
// Work. One block per SM goes through units of R = 16 .. 128 rows of q times
// all of k. A producer warp streams q into a ring in shared memory by TMA
// (two to four stages of 32 KB, boxes of 128 bytes x R rows in the 128-byte
// swizzle); 16 warps each take two steps of a stage, 16 rows x 128 k each, side by
// side (one after the other where x has several sets of columns), and add up
// their shares of k at the end of a unit. x is laid out either by every block for
// itself, once, and stays in shared memory, or, where it is too large for that, by
// a small kernel before this one, and is streamed with q. The swizzle lets a quad's lanes read 64 contiguous bytes of
// a row without bank conflicts if the rows of a quarter warp are four (groups
// of 128) or two apart, so row g of a matrix instruction is row_of(g) of a tile.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "experts_common.cuh"
#include "experts_internal.h"
#include "tc_common.cuh"

namespace sgemm {
namespace ex {
namespace {

constexpr int CONSUMERS = 16;                      // warps
constexpr int W4_THREADS = 32 * (CONSUMERS + 1);   // and the producer
constexpr int W4_ROWS = 8;         // rows of x that share a pass
constexpr int STEP = 128;          // values of k per warp step
constexpr int PAIR = 2;            // steps of a warp in a stage
constexpr int TURN = 2;            // stages between fetches of scales
constexpr int Q_STAGE = 32 * 1024;
// Stages of the ring. More only take shared memory from the L1 cache, which
// holds scales and spilled registers: 1 x 28672 x 4096 bf16 19.5 us with four,
// 21.3 with six; x streamed, 4 x 16384 x 8192 fp32, groups of 64, 34.5 us with
// two, 40.2 with three.
constexpr int MAX_STAGES = 4, STREAM_STAGES = 2;
constexpr int SMEM_BYTES = 225 * 1024;      // of a block, at most (and 144 bytes of static shared memory)
constexpr int RESIDENT_ONE = 144 * 1024;    // x in shared memory: one row, eight rows
constexpr int RESIDENT_EIGHT = 96 * 1024;
constexpr int X_STAGE = 64 * 1024;          // x of a stage, at most, when it is streamed
constexpr int PASSES = 256;                 // of one launch when x is streamed
constexpr int64_t OVERLAP = INT64_C(48) << 20;  // weights of a call: about 12 us

struct W4Args {
    int rows, experts;
    int64_t N, K;
    int groups;       // per row of q
    int group_shift;  // log2 of the group
    int unit_rows;    // R
    int units;        // ceil(N / R)
    int stages;       // of the ring
    int first_pass;
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
    const uint8_t *prepared;  // streamed x
    uint64_t timeout_ns;
    int *watchdog;
};

// How a row type enters the matrix instruction: terms of x, the bits that q is
// placed in, the zero point as it is subtracted from both values of an operand,
// what an operand's 1 stands for (UNIT), and the instruction itself.
template <class T>
struct Operand;

template <>
struct Operand<__nv_bfloat16> {
    static constexpr int TERMS = 1;
    static constexpr bool TWO_PLACES = false;  // q low and four bits up
    static constexpr uint32_t ONE = 0x43004300u;  // 128, 128 in bf16
    static constexpr float UNIT = 1.0f;
    static __device__ __forceinline__ uint32_t zero(uint32_t z) { return ONE + z * 0x00010001u; }
    static __device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t b) {
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&d);
    }
    static __device__ __forceinline__ void split(__nv_bfloat16 x, uint16_t (&t)[1]) { t[0] = __bfloat16_as_ushort(x); }
    // d = a b + c
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                               float c1, float c2, float c3) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    }
};

template <>
struct Operand<__half> {
    static constexpr int TERMS = 1;
    static constexpr bool TWO_PLACES = true;  // q low and four bits up
    static constexpr uint32_t ONE = 0;
    static constexpr float UNIT = 16777216.0f;  // an operand's q is q 2^-24
    static __device__ __forceinline__ uint32_t zero(uint32_t z) { return z * 0x00010001u; }
    // Differences of subnormals, exact.
    static __device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t b) {
        const __half2 d = __hsub2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&d);
    }
    static __device__ __forceinline__ void split(__half x, uint16_t (&t)[1]) { t[0] = __half_as_ushort(x); }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                               float c1, float c2, float c3) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    }
};

template <>
struct Operand<float> {
    static constexpr int TERMS = 3;
    static constexpr bool TWO_PLACES = false;
    static constexpr uint32_t ONE = Operand<__nv_bfloat16>::ONE;
    static constexpr float UNIT = 1.0f;
    static __device__ __forceinline__ uint32_t zero(uint32_t z) { return Operand<__nv_bfloat16>::zero(z); }
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
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                               float c1, float c2, float c3) {
        Operand<__nv_bfloat16>::mma(d, a, b0, b1, c0, c1, c2, c3);
    }
};

// Scale i as it is stored, and its value. Apart, so that a scale that is
// fetched ahead is not waited for before it is used.
__device__ __forceinline__ uint32_t scale_bits(const W4Args &a, int64_t i) {
    return a.scale_type == SGEMM_TYPE_F32 ? __ldg(static_cast<const uint32_t *>(a.scales) + i)
                                          : __ldg(static_cast<const uint16_t *>(a.scales) + i);
}

__device__ __forceinline__ float scale_value(const W4Args &a, uint32_t bits) {
    if (a.scale_type == SGEMM_TYPE_F16) return __half2float(__ushort_as_half(static_cast<uint16_t>(bits)));
    return __uint_as_float(a.scale_type == SGEMM_TYPE_F32 ? bits : bits << 16);
}

__device__ __forceinline__ float scale_at(const W4Args &a, int64_t i) { return scale_value(a, scale_bits(a, i)); }

// How the k of a step lie in a lane's four words, by the width of the groups
// (lane t of a quad, word u, 8 k each):
//   128: k = 32 t + 8 u: 16 bytes a lane, one group (or half of one) a step.
//   64:  k = 64 (u / 2) + 16 t + 8 (u % 2): 8 bytes a lane for each 64 k, one
//        group.
//   32:  as 64, then lanes t and t ^ 2 exchange a word, so that word u of all
//        four lanes is the u-th 32 k: k = 32 u + 16 (t % 2) + 8 (t / 2).

// Row of a 16-row tile (of its first or second eight) that is row g of the
// matrix instruction.
template <int WIDTH>
__device__ __forceinline__ int row_of(int g) {
    return WIDTH == 128 ? (g >> 1) | ((g & 1) << 2) : ((2 * g) & 7) | (g >> 2);
}

// One step of a lane: 32 values of k of rows g and g + 8.
struct Weights {
    uint32_t lo[4], hi[4];
};

// Scales and zero points of rows g and g + 8 that a lane fetched, as stored:
// for width 128 those of step t of four, otherwise those of the t-th 32 values
// of one step.
struct Raw {
    uint32_t lo, hi, z_lo, z_hi;
};

// Their values, zero points as the operands' type subtracts them.
struct Scales {
    float lo, hi;
    uint32_t z_lo, z_hi;
};

template <class Op>
__device__ __forceinline__ Scales values_of(const W4Args &a, const Raw &r) {
    return Scales{scale_value(a, r.lo), scale_value(a, r.hi), Op::zero(r.z_lo & 15u), Op::zero(r.z_hi & 15u)};
}

// What a sum s = y[r][n] that is not finite should be: itself where x holds an
// infinity or a NaN (a look at 32 values at a time, which the lanes share: 8 x
// 16384 x 8192 bf16 0.47 ms, 9.8 ms where such rows were summed again), otherwise
// the sum in 64 bits, which hold every product exactly and do not overflow.
template <class T>
__device__ __noinline__ float scalar_row(const W4Args &a, int64_t row, const T *x, float s32) {
    constexpr int PER = 16 / sizeof(T);
    bool finite = true;
#pragma unroll 1
    for (int64_t k = 0; k < a.K && finite; k += 32) {
#pragma unroll
        for (int j = 0; j < 32; j += PER) {
            Pack<T, PER> p;
            if (a.x_vector) {
                p = load_pack<T, PER>(x + k + j);
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i) p.v[i] = x[k + j + i];
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) finite = finite && isfinite(to_f32(p.v[i]));
        }
    }
    if (!finite) return s32;
    const uint32_t *q = reinterpret_cast<const uint32_t *>(a.q + row * (a.K / 2));
    double s = 0.0;
#pragma unroll 1
    for (int64_t k = 0; k < a.K; k += 8) {
        const int64_t gi = row * a.groups + (k >> a.group_shift);
        const uint32_t word = __ldg(q + k / 8);
        const int z = a.zeros ? __ldg(a.zeros + gi) & 15 : 8;
        const double scale = scale_at(a, gi);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = to_f32(x[k + j]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s = fma(static_cast<double>(static_cast<int>((word >> (4 * j)) & 15u) - z) * scale, v[j], s);
    }
    return static_cast<float>(s);
}

// The rows of x of pass `pass`: eight consecutive ones, or, with ids, row
// `pass` and the next seven of the same expert where an eighth of them starts
// there. Returns their number (0: nothing to do) and the expert; called by the
// whole block.
struct Members {
    int row[W4_ROWS];
    int count;
};

__device__ __forceinline__ int find_members(const W4Args &a, int pass, Members *m, int *expert) {
    *expert = 0;
    if (!a.ids) {
        const int r0 = pass * W4_ROWS;
        if (threadIdx.x < W4_ROWS) m->row[threadIdx.x] = r0 + static_cast<int>(threadIdx.x);
        __syncthreads();
        return min(W4_ROWS, a.rows - r0);
    }
    const int e = __ldg(a.ids + pass);
    *expert = e;
    if (e < 0 || e >= a.experts) return 0;
    const int threads = static_cast<int>(blockDim.x);
    int before = 0;
    for (int r0 = 0; r0 < pass; r0 += threads) {
        const int i = r0 + static_cast<int>(threadIdx.x);
        before += __syncthreads_count(i < pass && __ldg(a.ids + i) == e);
    }
    if (before % W4_ROWS != 0) return 0;
    if (threadIdx.x < 32) {
        const int lane = static_cast<int>(threadIdx.x);
        int have = 0;
        for (int r0 = pass; r0 < a.rows && have < W4_ROWS; r0 += 32) {
            const bool mine = r0 + lane < a.rows && __ldg(a.ids + r0 + lane) == e;
            const unsigned all = __ballot_sync(0xffffffffu, mine);
            const int at = have + __popc(all & ((1u << lane) - 1u));
            if (mine && at < W4_ROWS) m->row[at] = r0 + lane;
            have += __popc(all);
        }
        if (lane == 0) m->count = min(have, W4_ROWS);
    }
    __syncthreads();
    return m->count;
}

// Steps of K values of k, in pairs: the last may hold zeros only.
__host__ __device__ __forceinline__ int64_t steps_of(int64_t K) { return (K + PAIR * STEP - 1) / (PAIR * STEP) * PAIR; }

// A step of x as the matrix instructions read it: set of columns, unit u,
// column, lane t, 8 values.
// With fp32 x, TILES sets of eight columns hold the terms: term m of row r is
// column r of set m (three sets) or column 3 r + m of the sets in a row.
template <class T, int WIDTH, int NB, int TILES>
struct XStep {
    static constexpr int UNIT_BYTES = NB * 64, TILE_BYTES = 4 * UNIT_BYTES;
    static constexpr bool SPREAD = Operand<T>::TERMS > TILES;
    static __device__ __forceinline__ int column(int r, int m) { return SPREAD ? 3 * r + m : 8 * m + r; }
    static constexpr int BYTES = TILES * TILE_BYTES;
};

// Lays out values 8 piece .. 8 piece + 7 of step `st` of row `row` of x as row r
// of `to` (the step); zeros past the end of k.
template <class T, int WIDTH, int NB, int TILES>
__device__ __forceinline__ void lay_out_x(const W4Args &a, const T *x, int st, int piece, int r, bool in, uint8_t *to) {
    using Op = Operand<T>;
    using X = XStep<T, WIDTH, NB, TILES>;
    // Which unit of which lane holds them.
    const int u = WIDTH == 128 ? piece & 3 : WIDTH == 64 ? 2 * (piece >> 3) + (piece & 1) : piece >> 2;
    const int t = WIDTH == 128 ? piece >> 2 : WIDTH == 64 ? (piece >> 1) & 3 : ((piece >> 1) & 1) + 2 * (piece & 1);
    const int k = st * STEP + piece * 8, K = static_cast<int>(a.K);
    Pack<T, 8> v;
    if (in && a.x_vector && k + 8 <= K) {
        constexpr int PER = 16 / sizeof(T);
#pragma unroll
        for (int j = 0; j < 8; j += PER) {
            const Pack<T, PER> p = load_pack<T, PER>(x + k + j);
#pragma unroll
            for (int m = 0; m < PER; ++m) v.v[j + m] = p.v[m];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v.v[j] = in && k + j < K ? x[k + j] : from_f32<T>(0.0f);
    }
    uint32_t w[Op::TERMS][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = Op::TWO_PLACES ? (i >> 1) | ((i & 1) << 1) : i;
        uint16_t x0[Op::TERMS], x1[Op::TERMS];
        Op::split(v.v[j], x0);
        Op::split(v.v[j + 4], x1);
#pragma unroll
        for (int m = 0; m < Op::TERMS; ++m) w[m][i] = x0[m] | (static_cast<uint32_t>(x1[m]) << 16);
    }
    if (in) {
#pragma unroll
        for (int m = 0; m < Op::TERMS; ++m) {
            const int c = X::column(r, m);
            *reinterpret_cast<uint4 *>(to + (c >> 3) * X::TILE_BYTES + u * X::UNIT_BYTES + (c & 7) * 64 + t * 16) =
                make_uint4(w[m][0], w[m][1], w[m][2], w[m][3]);
        }
    }
}

// Lays out x of pass blockIdx.y for streaming: a thread per 8 values.
constexpr int PREPARE_THREADS = 256;
template <class T, int WIDTH, int TILES>
__global__ void __launch_bounds__(PREPARE_THREADS) w4_prepare_kernel(const __grid_constant__ W4Args a, uint8_t *to) {
    __shared__ Members members;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the kernel before it ends
    asm volatile("griddepcontrol.launch_dependents;");
    int expert;
    const int nb = find_members(a, a.first_pass + static_cast<int>(blockIdx.y), &members, &expert);
    if (nb == 0) return;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * PREPARE_THREADS + threadIdx.x;
    const int steps = static_cast<int>(steps_of(a.K));
    const int st = static_cast<int>(i / (16 * W4_ROWS)), r = static_cast<int>(i / 16) % W4_ROWS;
    const bool in = st < steps && r < nb;
    lay_out_x<T, WIDTH, W4_ROWS, TILES>(
        a, static_cast<const T *>(a.x) + (in ? members.row[r] * a.ldx : 0), in ? st : 0, static_cast<int>(i & 15), r, in,
        to + (static_cast<int64_t>(blockIdx.y) * steps + (in ? st : 0)) * XStep<T, WIDTH, W4_ROWS, TILES>::BYTES);
}

// Untiled bulk copy global -> this block's shared memory (16-byte aligned).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
    return v;
}

// NB: rows of x laid out, 1 or 8. With one, all eight columns of the matrix
// instruction are that row; with fewer than eight rows of x the rest of shared
// memory is whatever it was. Columns do not mix, so only those of rows of x are
// read out. STREAM: x comes with q from a.prepared.
template <class T, int WIDTH, int NB, int TILES, bool STREAM>
__global__ void __launch_bounds__(W4_THREADS, 1)
    w4_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ W4Args a) {
    using Op = Operand<T>;
    using X = XStep<T, WIDTH, NB, TILES>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Members members;
    __shared__ alignas(8) uint64_t bars[2 * MAX_STAGES];
    __shared__ int abort_word;
    volatile int *abort_flag = &abort_word;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t raw = tc::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const int K = static_cast<int>(a.K), steps = static_cast<int>(steps_of(a.K));
    const int R = a.unit_rows, RT = R / 16, KS = PAIR * CONSUMERS / RT;  // row tiles and steps of a stage
    const int per_unit = (steps + KS - 1) / KS;                   // stages of a unit
    const uint32_t x_stage = STREAM ? static_cast<uint32_t>(KS * X::BYTES + 1023) / 1024 * 1024 : 0;
    const uint32_t stage_bytes = Q_STAGE + x_stage;
    // Behind the ring: the warps' sums of two units, x when it stays.
    constexpr int ACC = X::SPREAD ? TILES : 1;  // sets of sums
    constexpr int PART = CONSUMERS * ACC * NB * 16;
    float *part = reinterpret_cast<float *>(smem_raw + (base - raw) + a.stages * stage_bytes);
    uint8_t *x_here = reinterpret_cast<uint8_t *>(part + 2 * PART);
    T *y = static_cast<T *>(a.y);
    auto full = [&](int s) { return tc::smem_u32(bars + s); };
    auto empty = [&](int s) { return tc::smem_u32(bars + MAX_STAGES + s); };
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            tc::mbar_init(full(s), 1);
            tc::mbar_init(empty(s), CONSUMERS);
        }
        abort_word = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    // May be launched while the kernel before it in the stream ends. Nothing is
    // read before that one's end, whichever it is: what kernels before it wrote
    // (ids, weights) is visible to the grid that waited for them, and to this one
    // by its own wait only.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    const int pass = a.first_pass + static_cast<int>(blockIdx.y);
    int expert;
    const int nb = find_members(a, pass, &members, &expert);
    if (nb == 0) {
        if (expert < 0 || expert >= a.experts)  // a row without an expert is zero
            for (int64_t n = static_cast<int64_t>(blockIdx.x) * W4_THREADS + threadIdx.x; n < a.N;
                 n += static_cast<int64_t>(gridDim.x) * W4_THREADS)
                y[pass * a.ldy + n] = from_f32<T>(0.0f);
        return;
    }

    if (warp == CONSUMERS) {
        // ------------------------------------------------------------------ producer
        if (lane == 0) {
            const uint8_t *x_from = STREAM ? a.prepared + static_cast<int64_t>(blockIdx.y) * steps * X::BYTES : nullptr;
            int slot = 0;
            uint32_t phase = 0;
            for (int u = static_cast<int>(blockIdx.x); u < a.units; u += static_cast<int>(gridDim.x)) {
                const int row = expert * static_cast<int>(a.N) + u * R;
                for (int stage = 0; stage < per_unit; ++stage) {
                    if (!tc::mbar_wait(empty(slot), phase ^ 1, a, abort_flag, tc::WD_PRODUCER)) return;
                    const int boxes = min(KS / 2, (K / 2 - stage * KS * 64 + 127) / 128);
                    const int here = min(KS, steps - stage * KS);
                    tc::mbar_arrive_expect_tx(full(slot), static_cast<uint32_t>(boxes * R * 128) +
                                                              (STREAM ? static_cast<uint32_t>(here * X::BYTES) : 0));
                    for (int b = 0; b < boxes; ++b)
                        tc::tma_load_3d(base + slot * stage_bytes + b * R * 128, &tmQ, stage * KS * 64 + b * 128, row, 0,
                                        full(slot));
                    if (STREAM)
                        bulk_load(base + slot * stage_bytes + Q_STAGE,
                                  x_from + static_cast<int64_t>(stage) * KS * X::BYTES,
                                  static_cast<uint32_t>(here * X::BYTES), full(slot));
                    if (++slot == a.stages) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
        }
        return;
    }

    // ---------------------------------------------------------------------- consumers
    const int rt = warp % RT, box = warp / RT;  // row tile, and pair of steps
    const int ra = 16 * rt + row_of<WIDTH>(g);  // rows of the unit; the second eight: + 8
    // Scales of the group that holds value k of the rows of unit u.
    auto fetch_scales = [&](int u, int k) {
        Raw s{0, 0, 8, 8};
        if (u < a.units && k < K) {
            const int64_t n0 = static_cast<int64_t>(u) * R + ra, row0 = static_cast<int64_t>(expert) * a.N;
            const int64_t lo = (row0 + min(n0, a.N - 1)) * a.groups, hi = (row0 + min(n0 + 8, a.N - 1)) * a.groups;
            const int gi = k >> a.group_shift;
            s.lo = scale_bits(a, lo + gi);
            s.hi = scale_bits(a, hi + gi);
            if (a.zeros) {
                s.z_lo = __ldg(a.zeros + lo + gi);
                s.z_hi = __ldg(a.zeros + hi + gi);
            }
        }
        return s;
    };
    // Width 128: a quad's lanes fetch the scales of a turn's four steps;
    // otherwise each step's, a turn ahead.
    static_assert(PAIR * TURN == 4, "a quad's lanes fetch the scales of a turn");
    Raw of_step[TURN][PAIR], next{};
    Scales turn{};
    auto fetch_turn = [&](int u, int stage0) {
        if (WIDTH == 128) next = fetch_scales(u, ((stage0 + (t >> 1)) * KS + PAIR * box + (t & 1)) * STEP);
    };
    auto fetch_stage = [&](int u, int stage, Raw (&s)[PAIR]) {
        if (WIDTH < 128) {
#pragma unroll
            for (int h = 0; h < PAIR; ++h) s[h] = fetch_scales(u, (stage * KS + PAIR * box + h) * STEP + 32 * t);
        }
    };
    const int u0 = static_cast<int>(blockIdx.x), du = static_cast<int>(gridDim.x);
    fetch_turn(u0, 0);
#pragma unroll
    for (int j = 0; j < TURN; ++j) fetch_stage(u0, j, of_step[j]);

    // x, once, when it stays here.
    if (!STREAM) {
        const int total = steps * 16 * NB;  // a sixteenth of a step of a row each
        for (int i0 = 0; i0 < total; i0 += CONSUMERS * 32) {
            const int i = i0 + static_cast<int>(threadIdx.x);
            const int r = (i >> 4) % NB, st = (i >> 4) / NB;
            const bool in = i < total && r < nb;
            const T *x = static_cast<const T *>(a.x) + (in ? members.row[r] * a.ldx : 0);
            lay_out_x<T, WIDTH, NB, TILES>(a, x, in ? st : 0, i & 15, r, in, x_here + (in ? st : 0) * X::BYTES);
        }
        asm volatile("bar.sync 1, %0;" ::"n"(CONSUMERS * 32) : "memory");
    }
    const uint32_t x_at0 = tc::smem_u32(x_here);

    float sum[ACC][4] = {};
    // Two steps side by side: their chains of products do not depend on each
    // other. One after the other where sets of columns give chains enough: the
    // registers spilled otherwise (8 x 16384 x 8192 fp32, groups of 64: 40 and 61 us).
    auto multiply = [&](const Weights (&w)[PAIR], const Scales (&sc)[PAIR], int j, uint32_t x_step) {
        // One accumulator per chain of dependent products.
        constexpr int CHAINS = TILES == 1 ? 2 : TILES;
        constexpr int SIDE = TILES > 1 ? 1 : PAIR;  // steps side by side
        constexpr int PER_GROUP = WIDTH / 32;  // words of a group
#pragma unroll
        for (int h0 = 0; h0 < PAIR; h0 += SIDE) {
            float c[SIDE][CHAINS][4];
            float s_lo[SIDE], s_hi[SIDE];
            uint32_t z_lo[SIDE], z_hi[SIDE];
            const uint32_t x_at = x_step + (NB == 1 ? t : lane) * 16;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (u % PER_GROUP == 0) {  // a group starts
#pragma unroll
                    for (int h = 0; h < SIDE; ++h) {
                        const int from = (lane & ~3) | (WIDTH == 128 ? PAIR * j + h0 + h : u);
                        s_lo[h] = __shfl_sync(0xffffffffu, sc[h0 + h].lo, from);
                        s_hi[h] = __shfl_sync(0xffffffffu, sc[h0 + h].hi, from);
                        z_lo[h] = z_hi[h] = Op::zero(8);
                        if (a.zeros) {
                            z_lo[h] = __shfl_sync(0xffffffffu, sc[h0 + h].z_lo, from);
                            z_hi[h] = __shfl_sync(0xffffffffu, sc[h0 + h].z_hi, from);
                        }
                    }
                }
                uint4 xv[SIDE][TILES];
#pragma unroll
                for (int h = 0; h < SIDE; ++h)
#pragma unroll
                    for (int m = 0; m < TILES; ++m)
                        xv[h][m] = lds128(x_at + (h0 + h) * X::BYTES + m * X::TILE_BYTES + u * X::UNIT_BYTES);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int h = 0; h < SIDE; ++h) {
                        uint32_t f[4];
                        if (Op::TWO_PLACES) {
                            const uint32_t mask = half ? 0x00F000F0u : 0x000F000Fu;
                            f[0] = w[h0 + h].lo[u] & mask;
                            f[1] = w[h0 + h].hi[u] & mask;
                            f[2] = (w[h0 + h].lo[u] >> 8) & mask;
                            f[3] = (w[h0 + h].hi[u] >> 8) & mask;
                        } else {
                            f[0] = ((w[h0 + h].lo[u] >> (8 * half)) & 0x000F000Fu) | Op::ONE;
                            f[1] = ((w[h0 + h].hi[u] >> (8 * half)) & 0x000F000Fu) | Op::ONE;
                            f[2] = ((w[h0 + h].lo[u] >> (8 * half + 4)) & 0x000F000Fu) | Op::ONE;
                            f[3] = ((w[h0 + h].hi[u] >> (8 * half + 4)) & 0x000F000Fu) | Op::ONE;
                        }
                        const int up = Op::TWO_PLACES ? 4 * half : 0;
                        f[0] = Op::minus(f[0], z_lo[h] << up);
                        f[1] = Op::minus(f[1], z_hi[h] << up);
                        f[2] = Op::minus(f[2], z_lo[h] << up);
                        f[3] = Op::minus(f[3], z_hi[h] << up);
#pragma unroll
                        for (int m = 0; m < TILES; ++m) {
                            float(&d)[4] = c[h][TILES == 1 ? half : m];
                            const uint32_t b0 = half ? xv[h][m].z : xv[h][m].x, b1 = half ? xv[h][m].w : xv[h][m].y;
                            if (u % PER_GROUP == 0 && (half == 0 || TILES == 1))  // the chain starts
                                Op::mma(d, f, b0, b1, 0.0f, 0.0f, 0.0f, 0.0f);
                            else
                                Op::mma(d, f, b0, b1, d[0], d[1], d[2], d[3]);
                        }
                    }
                }
                if ((u + 1) % PER_GROUP == 0) {  // the group ends
#pragma unroll
                    for (int h = 0; h < SIDE; ++h) {
                        if constexpr (ACC > 1) {
#pragma unroll
                            for (int m = 0; m < ACC; ++m) {
                                sum[m][0] = fmaf(s_lo[h], c[h][m][0], sum[m][0]);
                                sum[m][1] = fmaf(s_lo[h], c[h][m][1], sum[m][1]);
                                sum[m][2] = fmaf(s_hi[h], c[h][m][2], sum[m][2]);
                                sum[m][3] = fmaf(s_hi[h], c[h][m][3], sum[m][3]);
                            }
                        } else {
                            float d[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (Op::TWO_PLACES) {
                                    d[i] = fmaf(c[h][1][i], Op::UNIT / 16, c[h][0][i] * Op::UNIT);
                                } else {  // small terms first
                                    d[i] = c[h][CHAINS - 1][i];
#pragma unroll
                                    for (int m = CHAINS - 2; m >= 0; --m) d[i] += c[h][m][i];
                                }
                            }
                            sum[0][0] = fmaf(s_lo[h], d[0], sum[0][0]);
                            sum[0][1] = fmaf(s_lo[h], d[1], sum[0][1]);
                            sum[0][2] = fmaf(s_hi[h], d[2], sum[0][2]);
                            sum[0][3] = fmaf(s_hi[h], d[3], sum[0][3]);
                        }
                    }
                }
            }
        }
    };

    // This lane's bytes of a stage.
    const uint32_t q_row = static_cast<uint32_t>(box * R * 128 + ra * 128), turn_of = static_cast<uint32_t>(ra & 7);
    int slot = 0;
    uint32_t phase = 0;
    bool alive = true;  // after a wait that gave up the loops go on without waiting or multiplying
    int parity = 0;
    for (int u = u0; u < a.units; u += du, parity ^= 1) {
        for (int stage0 = 0; stage0 < per_unit; stage0 += TURN) {
            const bool last_turn = stage0 + TURN >= per_unit;
            if (WIDTH == 128) {
                turn = values_of<Op>(a, next);
                fetch_turn(last_turn ? u + du : u, last_turn ? 0 : stage0 + TURN);
            }
#pragma unroll
            for (int j = 0; j < TURN; ++j) {
                const int stage = stage0 + j;
                if (stage < per_unit) {
                    if (alive)
                        alive = __all_sync(0xffffffffu,
                                           tc::mbar_wait(full(slot), phase, a, abort_flag, tc::WD_MMA_FULL));
                    const int st = stage * KS + PAIR * box;
                    if (alive && st < steps) {
                        const uint32_t sq = base + slot * stage_bytes, at = sq + q_row;
                        Weights w[PAIR];
#pragma unroll
                        for (int h = 0; h < PAIR; ++h) {
                            if (WIDTH == 128) {
                                const uint32_t c = ((4 * h + t) ^ turn_of) * 16;
                                const uint4 lo = lds128(at + c), hi = lds128(at + 8 * 128 + c);
                                w[h].lo[0] = lo.x, w[h].lo[1] = lo.y, w[h].lo[2] = lo.z, w[h].lo[3] = lo.w;
                                w[h].hi[0] = hi.x, w[h].hi[1] = hi.y, w[h].hi[2] = hi.z, w[h].hi[3] = hi.w;
                            } else {
#pragma unroll
                                for (int p = 0; p < 2; ++p) {
                                    const uint32_t c = ((4 * h + 2 * p + (t >> 1)) ^ turn_of) * 16 + (t & 1) * 8;
                                    uint2 lo = lds64(at + c), hi = lds64(at + 8 * 128 + c);
                                    if (WIDTH == 32) {
                                        // The second word of lanes 0, 1 for the first of lanes 2, 3.
                                        const uint32_t sl = __shfl_xor_sync(0xffffffffu, t < 2 ? lo.y : lo.x, 2);
                                        const uint32_t sh = __shfl_xor_sync(0xffffffffu, t < 2 ? hi.y : hi.x, 2);
                                        lo = t < 2 ? make_uint2(lo.x, sl) : make_uint2(sl, lo.y);
                                        hi = t < 2 ? make_uint2(hi.x, sh) : make_uint2(sh, hi.y);
                                    }
                                    w[h].lo[2 * p] = lo.x, w[h].lo[2 * p + 1] = lo.y;
                                    w[h].hi[2 * p] = hi.x, w[h].hi[2 * p + 1] = hi.y;
                                }
                            }
                        }
                        const uint32_t x_step = STREAM ? sq + Q_STAGE + static_cast<uint32_t>(PAIR * box * X::BYTES)
                                                       : x_at0 + static_cast<uint32_t>(st * X::BYTES);
                        if (WIDTH == 128) {
                            const Scales both[PAIR] = {turn, turn};
                            multiply(w, both, j, x_step);
                        } else {
                            const Scales both[PAIR] = {values_of<Op>(a, of_step[j][0]), values_of<Op>(a, of_step[j][1])};
                            multiply(w, both, j, x_step);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(empty(slot));
                    if (++slot == a.stages) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                fetch_stage(last_turn ? u + du : u, last_turn ? j : stage + TURN, of_step[j]);
            }
        }
        // Join the shares of the unit. Two buffers: a warp that writes the next
        // unit's sums may meet one that still reads this unit's.
        float *mine = part + parity * PART + warp * ACC * NB * 16;
        const int n_lo = row_of<WIDTH>(g);
#pragma unroll
        for (int m = 0; m < ACC; ++m) {
            if (NB == 1) {
                if (t == 0) {
                    mine[n_lo] = sum[m][0];
                    mine[n_lo + 8] = sum[m][2];
                }
            } else {
                mine[(8 * m + 2 * t) * 16 + n_lo] = sum[m][0];
                mine[(8 * m + 2 * t + 1) * 16 + n_lo] = sum[m][1];
                mine[(8 * m + 2 * t) * 16 + n_lo + 8] = sum[m][2];
                mine[(8 * m + 2 * t + 1) * 16 + n_lo + 8] = sum[m][3];
            }
            sum[m][0] = sum[m][1] = sum[m][2] = sum[m][3] = 0.0f;
        }
        asm volatile("bar.sync 1, %0;" ::"n"(CONSUMERS * 32) : "memory");
        for (int i = threadIdx.x; i < R * nb; i += CONSUMERS * 32) {
            const int r = i / R, n = i - r * R;
            const float *from = part + parity * PART + (n >> 4) * ACC * NB * 16 + (n & 15);
            float s = 0.0f;
            for (int w = 0; w < CONSUMERS / RT; ++w, from += RT * ACC * NB * 16)
                s += X::SPREAD ? (from[(3 * r + 2) * 16] + from[(3 * r + 1) * 16]) + from[3 * r * 16] : from[r * 16];
            const int64_t row = static_cast<int64_t>(u) * R + n;
            if (row >= a.N) continue;
            if (!isfinite(s))
                s = scalar_row(a, static_cast<int64_t>(expert) * a.N + row,
                               static_cast<const T *>(a.x) + members.row[r] * a.ldx, s);
            y[members.row[r] * a.ldy + row] = from_f32<T>(s);
        }
    }
    // After a wait that gave up, copies may still be on their way: leave them
    // time to land.
    if (*abort_flag) {
        const uint64_t t0 = tc::global_timer();
        while (tc::global_timer() - t0 < 10000000ull) {
        }
    }
}

// Any K and alignment, without tensor maps or workspace: a warp per row of q,
// scalar arithmetic.
template <class T>
__global__ void __launch_bounds__(256) w4_simple_kernel(const __grid_constant__ W4Args a) {
    const int lane = threadIdx.x & 31;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (n >= a.N) return;
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const int e = a.ids ? __ldg(a.ids + r) : 0;
        float s = 0.0f;
        if (e >= 0 && e < a.experts) {
            const int64_t row = static_cast<int64_t>(e) * a.N + n;
            const T *x = static_cast<const T *>(a.x) + r * a.ldx;
            for (int64_t k = 2 * lane; k < a.K; k += 64) {
                const int64_t gi = row * a.groups + (k >> a.group_shift);
                const int b = __ldg(a.q + row * (a.K / 2) + k / 2), z = a.zeros ? __ldg(a.zeros + gi) & 15 : 8;
                const float w = scale_at(a, gi);
                s = fmaf(static_cast<float>((b & 15) - z) * w, to_f32(x[k]), s);
                s = fmaf(static_cast<float>((b >> 4) - z) * w, to_f32(x[k + 1]), s);
            }
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (lane == 0) static_cast<T *>(a.y)[r * a.ldy + n] = from_f32<T>(s);
    }
}

template <class T>
int launch_simple(const W4Args &a, cudaStream_t stream, int *launches) {
    const int64_t gx = (a.N + 7) / 8;
    if (gx > INT32_MAX) return SGEMM_ERR_UNSUPPORTED;
    w4_simple_kernel<T><<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(a.rows)), 256, 0, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return SGEMM_ERR_LAUNCH;
    ++*launches;
    return SGEMM_OK;
}

template <class T, int WIDTH, int NB, int TILES, bool STREAM>
int launch(W4Args a, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    auto kernel = w4_kernel<T, WIDTH, NB, TILES, STREAM>;
    using X = XStep<T, WIDTH, NB, TILES>;
    const int passes = static_cast<int>(a.ids ? a.rows : (a.rows + W4_ROWS - 1) / W4_ROWS);
    const int64_t steps = steps_of(a.K);
    // Passes with work in them. With ids, the experts that rows drawn evenly
    // would use, and two standard deviations more: blocks of a pass too many
    // would run after all others, blocks of other passes end at once.
    int64_t busy = passes;
    if (a.ids) {
        const double e = a.experts, one = pow(1.0 - 1.0 / e, a.rows), two = pow(1.0 - 2.0 / e, a.rows);
        const double used = e * (1.0 - one), spread = e * one + e * (e - 1.0) * two - e * e * one * one;
        const int64_t most = static_cast<int64_t>(used + 2.0 * sqrt(spread > 0.0 ? spread : 0.0) + 0.999);
        const int64_t by_expert = (a.rows + W4_ROWS - 1) / W4_ROWS + a.experts;  // passes there can be
        busy = a.rows > 8 * a.experts ? by_expert : most;
        if (busy > passes) busy = passes;
        if (busy > by_expert) busy = by_expert;
        if (busy < 1) busy = 1;
    }
    // Rows of a unit: few give every SM its part, many need less of a streamed
    // x and end less often (about a stage's time). The choice makes the
    // busiest SM's bytes least. The ring has two stages at least: with one, loads
    // and products would take turns.
    const int64_t rest = 1024 + 2 * CONSUMERS * (X::SPREAD ? TILES : 1) * NB * 16 * 4 + (STREAM ? 0 : steps * X::BYTES);
    auto stage_of = [](int64_t KS) { return Q_STAGE + (STREAM ? (KS * X::BYTES + 1023) / 1024 * 1024 : 0); };
    int64_t least = INT64_MAX;
    for (int R = 16; R <= 128; R *= 2) {
        const int64_t KS = PAIR * CONSUMERS / (R / 16), x = STREAM ? KS * X::BYTES : 0;
        if (x > X_STAGE || 2 * stage_of(KS) > SMEM_BYTES - rest) continue;
        const int64_t units = (a.N + R - 1) / R;
        int64_t workers = dev.sm_count / busy;  // of a pass
        workers = workers < 1 ? 1 : workers > units ? units : workers;
        const int64_t rounds = (units + workers - 1) / workers * ((workers * busy + dev.sm_count - 1) / dev.sm_count);
        const int64_t cost = rounds * ((steps + KS - 1) / KS + 1) * (Q_STAGE + x / 2);
        if (cost < least) {
            least = cost;
            a.unit_rows = R;
        }
    }
    a.units = static_cast<int>((a.N + a.unit_rows - 1) / a.unit_rows);
    const int64_t stage = stage_of(PAIR * CONSUMERS / (a.unit_rows / 16));
    int64_t stages = (SMEM_BYTES - rest) / stage;
    if (stages > (STREAM ? STREAM_STAGES : MAX_STAGES)) stages = STREAM ? STREAM_STAGES : MAX_STAGES;
    a.stages = static_cast<int>(stages);
    a.x_vector = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx * static_cast<int64_t>(sizeof(T)) % 16 == 0;
    a.timeout_ns = static_cast<uint64_t>(watchdog_ms()) * 1000000ull;
    a.watchdog = watchdog_flag_device_ptr();
    static std::once_flag once[64];
    static cudaError_t set[64];
    std::call_once(once[dev.device], [&] {
        set[dev.device] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    });
    alignas(64) CUtensorMap map{};
    if (!a.watchdog || set[dev.device] != cudaSuccess ||
        !tc::encode_map_typed(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.q, a.experts * a.N, a.K / 2, a.K / 2, 1, 0, 128,
                              static_cast<uint32_t>(a.unit_rows), CU_TENSOR_MAP_SWIZZLE_128B)) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    float *scratch = nullptr;
    if (STREAM) {
        const int64_t at_once = passes < PASSES ? passes : PASSES;
        scratch = scratch_alloc(dev, static_cast<size_t>(at_once * steps * X::BYTES), stream);
        if (!scratch) return launch_simple<T>(a, stream, launches);
        a.prepared = reinterpret_cast<const uint8_t *>(scratch);
    }
    int64_t workers = dev.sm_count / busy;
    if (workers < 1) workers = 1;
    if (workers > a.units) workers = a.units;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(W4_THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(rest + stages * stage);
    cfg.stream = stream;
    cfg.attrs = &attr;
    // A launch of that kind takes the host about 1 us more, so not for short
    // calls, which the host bounds.
    cfg.numAttrs = STREAM || busy * a.N * a.K >= OVERLAP ? 1 : 0;
    int rc = SGEMM_OK;
    const int chunk = STREAM ? PASSES : passes;
    for (a.first_pass = 0; a.first_pass < passes && rc == SGEMM_OK; a.first_pass += chunk) {
        const int here = passes - a.first_pass < chunk ? passes - a.first_pass : chunk;
        if (STREAM) {
            const int64_t blocks = (steps * 16 * W4_ROWS + PREPARE_THREADS - 1) / PREPARE_THREADS;
            cudaLaunchConfig_t before = cfg;
            before.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(here));
            before.blockDim = dim3(PREPARE_THREADS);
            before.dynamicSmemBytes = 0;
            if (cudaLaunchKernelEx(&before, w4_prepare_kernel<T, WIDTH, TILES>, a,
                                   reinterpret_cast<uint8_t *>(scratch)) != cudaSuccess) {
                cudaGetLastError();
                rc = SGEMM_ERR_LAUNCH;
                break;
            }
            ++*launches;
        }
        cfg.gridDim = dim3(static_cast<unsigned>(workers), static_cast<unsigned>(here));
        if (cudaLaunchKernelEx(&cfg, kernel, map, a) != cudaSuccess) {
            cudaGetLastError();
            rc = SGEMM_ERR_LAUNCH;
            break;
        }
        ++*launches;
    }
    scratch_free(scratch, stream);
    return rc;
}

template <class T, int WIDTH, int TILES>
int launch_tiles(const W4Args &a, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    if (steps_of(a.K) * XStep<T, WIDTH, 8, TILES>::BYTES <= RESIDENT_EIGHT)
        return launch<T, WIDTH, 8, TILES, false>(a, dev, stream, launches);
    return launch<T, WIDTH, 8, TILES, true>(a, dev, stream, launches);
}

template <class T, int WIDTH>
int launch_width(const W4Args &a, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    if constexpr (Operand<T>::TERMS == 3) {
        if (a.rows <= 2) return launch_tiles<T, WIDTH, 1>(a, dev, stream, launches);
        if (a.rows <= 5) return launch_tiles<T, WIDTH, 2>(a, dev, stream, launches);
        return launch_tiles<T, WIDTH, 3>(a, dev, stream, launches);
    } else {
        if (a.rows == 1 && steps_of(a.K) * XStep<T, WIDTH, 1, 1>::BYTES <= RESIDENT_ONE)
            return launch<T, WIDTH, 1, 1, false>(a, dev, stream, launches);
        return launch_tiles<T, WIDTH, 1>(a, dev, stream, launches);
    }
}

template <class T>
int launch_type(const W4Args &a, int64_t group, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    if (dev.device < 0 || dev.device >= 64) return SGEMM_ERR_DEVICE;
    // What a tensor map can describe: rows of q of a multiple of 16 bytes.
    if (a.K % 32 != 0 || a.K == 0 || reinterpret_cast<uintptr_t>(a.q) % 16 != 0 || a.K > INT32_MAX / 2 ||
        a.N > INT32_MAX / 2 / a.experts)
        return launch_simple<T>(a, stream, launches);
    if (group >= 128) return launch_width<T, 128>(a, dev, stream, launches);
    return group == 64 ? launch_width<T, 64>(a, dev, stream, launches) : launch_width<T, 32>(a, dev, stream, launches);
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
    if (p.type == SGEMM_TYPE_F32) return launch_type<float>(a, p.group, dev, stream, launches);
    if (p.type == SGEMM_TYPE_BF16) return launch_type<__nv_bfloat16>(a, p.group, dev, stream, launches);
    return launch_type<__half>(a, p.group, dev, stream, launches);
}

}  // namespace ex
}  // namespace sgemm
