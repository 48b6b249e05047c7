// Kernel of the tensor-core SGEMM on SM pairs: tcgen05.mma.cta_group::2 (kind::tf32) with
// the three-term TF32 split of sgemm_tf32x3.cu, for all four operand forms
// (op(A) = A or A^T, op(B) = B or B^T) at any alignment: TMA loads the raw
// tiles where the rows are 16-byte aligned, 4-byte cp.async copies elsewhere.
//
// The product is the plain sum of "CUDA算子优化(4)：矩阵乘法", section
// "矩阵乘法的数学定义"; the pages give no tensor-core design (they name
// tensor cores once, "CUDA内存优化入门：从Naive到Tiled矩阵乘法", section 八).
//
// Accuracy: short accumulation chains, folded on chip. The tensor core adds
// each MMA's products into its fp32 accumulator with truncation (measured on
// GB300: about one unit in the last place of the running value per
// tcgen05.mma), so one accumulator that chains every MMA of a long K drifts
// in one direction when the terms share a sign (3.5e-5 of sum |a||b| at
// K = 16384 on U[0,1] inputs). Here an accumulator never chains more than
// FOLD_KB k-blocks (12 MMAs each): the pair's MMAs alternate between two
// accumulators in TMEM, and while the tensor core fills one, the epilogue
// warps add the other, rounded to nearest, into an fp32 running sum of the
// tile held in shared memory. The MMAs never wait for a fold.
//
// Why pairs. Two CTAs on two SMs of a cluster share one 256 x 128 tile: each
// holds 128 rows of A (split into hi / lo, in its TMEM) and 64 columns of B
// (hi / lo in its shared memory), and one MMA of 256 x 128 x 8 issued by the
// even CTA reads both halves. Each SM's shared memory then serves only half
// of the B operand the tensor core reads. (Measured on GB300: the 256 x 128
// x 8 and 256 x 256 x 8 tf32 MMAs run at the same multiply-add rate, 32.7
// and 65.4 ns each.) TMEM per CTA: two 128-column accumulators and four A
// stages of 64 columns (hi | lo for 32 values of k), all 512 columns.
//
// Roles in each CTA (23 warps):
//   * warp 0: in the even CTA, one thread issues the pair's MMAs (4 k-slices
//     x 3 products per k-block, lo*hi + hi*lo + hi*hi) into accumulator
//     d = (fold interval) mod 2 and commits them to the mbarriers of both
//     CTAs (multicast).
//   * warps 1 and 22: TMA of this CTA's A rows (128 x 32, 128-byte swizzled)
//     and B columns (32 x 64) into a 4-slot raw ring (one lane each), or,
//     for rows TMA cannot address, all lanes of both copying half of each
//     tile with 4-byte cp.async.
//   * warps 2-17 (converters, four groups of four warps, group g taking the
//     k-blocks it with it mod 4 = g; each warp of a group serves one TMEM
//     lane quarter): each thread splits one row of A (32 values) into hi /
//     lo and writes them to TMEM (tcgen05.st), and transposes and splits one
//     4 x 4 block of B into the K-major, 128-byte-swizzled hi / lo tiles of a
//     4-stage shared ring; then one lane per warp signals the even CTA's
//     stage-full barrier (a local arrival, or from the odd CTA an st.async
//     that completes transaction bytes on it).
//   * warps 18-21 (epilogue, one per TMEM lane quarter): for each fold
//     interval, read the finished accumulator's 128 columns of its 32 rows
//     (four 32 x 32 chunks), add them into the running sum (or start it) and
//     free the accumulator; after a unit's last interval, form the output
//     alpha * sum (+ bias, activation) in the running-sum chunk itself and
//     write it to C with one TMA bulk store (bulk reduce-add for tiles split
//     along K) per chunk. Chunks crossing the last row or column, C that TMA
//     cannot address, or beta != 0 take per-thread stores.
// Every wait is bounded in time as in the single-SM kernels; the pair meets
// at cluster barriers only at the start (mbarriers initialised) and at the
// end (before the TMEM of both is released).
//
// The same kernel makes the products of mixture-of-experts layers (GROUPS):
// tiles of row groups whose bounds are read on the device in place of the
// tiles of one product (see GroupTiles), nothing else changed. Rows of A past
// a group's end change only rows of C that are not written; where the rows
// are the summed direction the converters put zeros in their place. The rows
// of C may also be the MMA's narrow side (GROUP_COLS, GROUP_WGRAD_COLS): the
// product is then C^T = op(B)^T A^T in tiles of 256 columns of C x 32 .. 128
// rows, so a short group is charged for a multiple of 32 rows, and a lane of
// the epilogue holds a column of C, so that warps write 128 bytes of its rows
// from registers without another pass through shared memory.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "experts_common.cuh"
#include "sgemm.h"
#include "sgemm_internal.h"
#include "tc_common.cuh"

namespace sgemm {
namespace {

using namespace tc;

namespace pr {

constexpr int PM = 256, PN = 128;  // C tile of a pair
constexpr int HM = 128, HN = 64;   // this CTA's rows of A, columns of B
// Longest chain of k-blocks one accumulator sums before it is folded into the
// running sum (tc::FOLD_KB = 8): 96 MMAs, ~5e-6 of sum |a||b| on non-negative
// inputs at any K.
constexpr int FOLD_KB = tc::FOLD_KB;
// Four operand stages (a stage is refilled only after the MMAs that read it
// have completed, and completions trail issue by the tensor pipe's queue)
// and four raw slots, one of each per converter group.
constexpr int OP_STAGES = 4, RAW_SLOTS = 4;
constexpr int B_HALF = HN * BK * 4;   // 8 KB: one of B hi / B lo, or raw B
constexpr int A_RAW = HM * BK * 4;    // 16 KB
constexpr int OP_STAGE = 2 * B_HALF;  // hi | lo
constexpr int SLOT = A_RAW + B_HALF;  // raw A | raw B
constexpr int RAW0 = OP_STAGES * OP_STAGE;
// Running sum: this CTA's 128 x 128 fp32 share of the tile as 16 chunks of
// 32 x 32 (chunk (q, c): rows 32q.., columns 32c..), rows of 128 bytes in the
// 128-byte swizzle, so a chunk is also the source of one TMA store of C.
constexpr int C_CHUNK = 32 * 32 * 4;
constexpr int R0 = RAW0 + RAW_SLOTS * SLOT;
constexpr int R_BYTES = (HM / 32) * (PN / 32) * C_CHUNK;
constexpr int CHUNKS = PN / 32;  // chunks per lane quarter
constexpr int GROUP_WARPS = 4, CONV_GROUPS = 4, CONV_WARPS = GROUP_WARPS * CONV_GROUPS, EPI_WARPS = 4;
constexpr int CONV_THREADS = 32 * GROUP_WARPS;  // threads converting one k-block
constexpr int EPI_WARP0 = 2 + CONV_WARPS;
// A second TMA issuer: a warp keeps only about one box in processing at a
// time (measured on GB300: ~0.4 us per box of 16-64 KB, whatever the ring
// depth), so A and B come from separate warps.
constexpr int TMA_B_WARP = EPI_WARP0 + EPI_WARPS;
constexpr int THREADS = 32 * (TMA_B_WARP + 1);
constexpr int BAR_OFFSET = R0 + R_BYTES;
constexpr int PBAR_BYTES = 256;
constexpr int SMEM_BYTES = BAR_OFFSET + PBAR_BYTES + 1024;
constexpr uint32_t TMEM_A = 2 * PN;  // A stages after the two 128-column accumulators
// Instruction descriptor: D fp32, A and B tf32, both K-major, N = n (128: a whole tile), M = 256.
__host__ __device__ constexpr uint32_t idesc2(int n) {
    return (1u << 4) | (2u << 7) | (2u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(PM >> 4) << 24);
}
constexpr int COL_STEP = 32;  // GROUP_COLS: a tile's width is a multiple of it
// mbarrier indices
constexpr int RAW_FULL = 0, RAW_FREE = RAW_FULL + RAW_SLOTS, OP_FULL = RAW_FREE + RAW_SLOTS,
              OP_EMPTY = OP_FULL + OP_STAGES, ACC_FULL = OP_EMPTY + OP_STAGES, ACC_EMPTY = ACC_FULL + 2,
              DRAIN = ACC_EMPTY + 2, NBARS = DRAIN + 1;
// The odd CTA's converter warps report a filled stage with st.async: a 4-byte
// store into the even CTA's shared memory that completes 4 bytes of
// transactions on its stage-full barrier with release semantics at cluster
// scope, without stalling the warp (a remote mbarrier.arrive.release.cluster
// held the arriving thread ~0.8 us per k-block on GB300, measured).
constexpr uint32_t SIGNAL_BYTES = 4 * GROUP_WARPS;
static_assert(NBARS * 8 + 32 <= PBAR_BYTES, "barrier block");
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
static_assert(TMEM_A + OP_STAGES * 64 <= TMEM_COLS, "TMEM columns");
static_assert((HN / 4) * (BK / 4) == CONV_THREADS, "one 4 x 4 B block per converter thread");
static_assert(CONV_GROUPS == OP_STAGES && RAW_SLOTS == OP_STAGES, "group g owns raw slot g and stage g");
static_assert(SLOT % 1024 == 0 && RAW0 % 1024 == 0 && R0 % 1024 == 0, "1024-byte aligned swizzled buffers");

}  // namespace pr

// One 256 x n x 8 product of the pair: A (128 rows per CTA) from TMEM, B
// (n / 2 columns per CTA) from shared memory.
__device__ __forceinline__ void tc_mma2_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t accumulate,
                                           uint32_t idesc = pr::idesc2(pr::PN)) {
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::tf32 [%0], [%1], %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Fused-epilogue values of 16 columns (chunk columns base .. base + 15)
// written to the swizzled chunk row of this lane: ACT(alpha * v + bias), the
// bias per row (bl) or per column (lane (base + j)'s bl, by shuffle).
template <int ACT>
__device__ __forceinline__ void stage16_ep(uint32_t buf, int lane, int base, float alpha, bool col_bias, float bl,
                                           const float *v) {
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        float b[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) b[t] = col_bias ? __shfl_sync(0xffffffffu, bl, base + j + t) : bl;
        st_shared_v4(buf + sw128_offset(lane, (base + j) >> 2), activate(alpha * v[j] + b[0], ACT),
                     activate(alpha * v[j + 1] + b[1], ACT), activate(alpha * v[j + 2] + b[2], ACT),
                     activate(alpha * v[j + 3] + b[3], ACT));
    }
}

__device__ __forceinline__ void stage32_fused(int act, uint32_t buf, int lane, float alpha, bool col_bias, float bl,
                                              const float (&v)[32]) {
    switch (act) {
        case SGEMM_ACT_RELU:
            stage16_ep<SGEMM_ACT_RELU>(buf, lane, 0, alpha, col_bias, bl, v);
            stage16_ep<SGEMM_ACT_RELU>(buf, lane, 16, alpha, col_bias, bl, v + 16);
            break;
        case SGEMM_ACT_GELU:
            stage16_ep<SGEMM_ACT_GELU>(buf, lane, 0, alpha, col_bias, bl, v);
            stage16_ep<SGEMM_ACT_GELU>(buf, lane, 16, alpha, col_bias, bl, v + 16);
            break;
        case SGEMM_ACT_SILU:
            stage16_ep<SGEMM_ACT_SILU>(buf, lane, 0, alpha, col_bias, bl, v);
            stage16_ep<SGEMM_ACT_SILU>(buf, lane, 16, alpha, col_bias, bl, v + 16);
            break;
        default:
            stage16_ep<SGEMM_ACT_NONE>(buf, lane, 0, alpha, col_bias, bl, v);
            stage16_ep<SGEMM_ACT_NONE>(buf, lane, 16, alpha, col_bias, bl, v + 16);
            break;
    }
}

// NaN in a chunk of finished sums (chunk rc, swizzled, this lane holding row
// `row`, columns from col0 on) recomputed over [k_begin, k_end), in shared
// memory, one column at a time (few registers).
__device__ __forceinline__ void repair_row(const Args &a, uint32_t rc, const float *A, const float *B, int64_t row,
                                           int64_t col0, int64_t n_end, int64_t k_begin, int64_t k_end) {
    const int lane = static_cast<int>(threadIdx.x & 31);
#pragma unroll 1
    for (int j = 0; j < 32 && col0 + j < n_end; ++j) {
        const uint32_t addr = rc + sw128_offset(lane, j >> 2) + static_cast<uint32_t>((j & 3) * 4);
        const float x = ld_shared_f32(addr);
        if (x != x) st_shared_f32(addr, dot_ieee(A, a.lda, a.ta, B, a.ldb, a.tb, row, col0 + j, k_begin, k_end));
    }
}

// The last fold of a unit for a chunk written with per-thread stores: the
// unit's finished sum for rows row0 .. row0 + 31, columns col0 .. col0 + 31
// (chunk rc of shared memory, swizzled, lane l holding row row0 + l),
// repaired where it is NaN (recomputed over the unit's k-range [k_begin,
// k_end) of batch item `item`), then written one row per step with the lanes
// along the row (coalesced): C = act(alpha * v + beta * C + bias) for a
// whole tile, C += alpha * v with atomics for a tile split along K. Used for
// chunks that cross the last row or column of C, for C that TMA cannot
// address and for chunks holding a NaN; called by all 32 lanes. Out of line:
// it is rare, and inlined it would compete for registers with the interior
// path. REPAIR: not for row groups, whose NaN are seen to at the end
// (repair_units).
template <bool VEC_C, bool REPAIR>
__device__ __noinline__ void edge_final_chunk(const Args &a, uint32_t rc, const float *A, const float *B, float *citem,
                                              int64_t m_end, int64_t row0, int64_t col0, bool atomic, int64_t k_begin,
                                              int64_t k_end) {
    const int lane = static_cast<int>(threadIdx.x & 31);
    if (col0 >= a.N) return;  // uniform over the warp
    const int64_t row = row0 + lane;
    if (REPAIR) {
        bool nan = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 r = ld_shared_v4(rc + sw128_offset(lane, j));
            nan |= r.x != r.x || r.y != r.y || r.z != r.z || r.w != r.w;
        }
        if (nan && row < m_end) repair_row(a, rc, A, B, row, col0, a.N, k_begin, k_end);
    }
    __syncwarp();
    store_staged_rows(a, rc, citem, m_end, row0, col0, atomic);
}

// What the kernel's units are: k-block ranges of one product's tiles
// (stream-K), or whole tiles of row groups (_COLS: of C^T, with the operands'
// places changed: M counts the columns of C and N its rows).
enum PairUnits { TILES, GROUP_ROWS, GROUP_COLS, GROUP_WGRAD, GROUP_WGRAD_COLS };
constexpr bool sums_rows(PairUnits u) { return u == GROUP_WGRAD || u == GROUP_WGRAD_COLS; }
constexpr bool transposed(PairUnits u) { return u == GROUP_COLS || u == GROUP_WGRAD_COLS; }

// A unit: k-blocks [kb, ke) of the tile at row m0, column n0 of C's item.
// Rows of C from m_end on are not written.
struct PairUnit {
    int kb, ke;
    int item_a, item_b, item_c;
    int64_t m0, n0, m_end;
    int64_t k0, k_end;  // first row of A and B that is summed and the values of k (wgrad: rows of the group)
    bool atomic;        // a part of a tile: C += instead of C =
    int64_t n_end;      // C^T: end of the tile's columns (rows of C)
    // C^T: the MMA's width.
    __device__ __forceinline__ int width() const {
        return (static_cast<int>(n_end - n0) + pr::COL_STEP - 1) / pr::COL_STEP * pr::COL_STEP;
    }
};

// Calls f(unit) for the units of worker `index` of `count`, in order.
template <PairUnits UNITS, class F>
__device__ __forceinline__ void for_each_pair_unit(const Args &a, const ex::GroupTiles &gt, volatile int *abort_flag,
                                                   int index, int count, F &&f) {
    if (UNITS == TILES) {
        for_each_unit_of(a, abort_flag, index, count, [&](int tile, int kb, int ke) {
            const TileAt at = tile_at<pr::PM, pr::PN>(a, tile);
            f(PairUnit{kb, ke, a.a_shared ? 0 : at.item, a.b_shared ? 0 : at.item, at.item, at.m0, at.n0, a.M, 0, a.K,
                       tile >= a.dp_tiles, a.N});
        });
    } else if (UNITS == GROUP_WGRAD_COLS) {
        ex::for_each_group_tile<true, pr::PN, pr::PM, BK>(
            gt, abort_flag, index, count, [&](const ex::GroupTile &t) {
                f(PairUnit{0, t.k_blocks, 0, 0, t.group, t.n0, t.row0, a.M, t.k0, t.k_rows, false,
                           min(t.row0 + pr::PN, t.row_end)});
            });
    } else if (UNITS == GROUP_COLS) {
        ex::for_each_group_tile<false, pr::PN, pr::PM, BK, pr::COL_STEP>(
            gt, abort_flag, index, count, [&](const ex::GroupTile &t) {
                f(PairUnit{0, t.k_blocks, t.group, 0, 0, t.n0, t.row0, a.M, 0, a.K, false, t.row_end});
            });
    } else {
        ex::for_each_group_tile<UNITS == GROUP_WGRAD, pr::PM, pr::PN, BK>(
            gt, abort_flag, index, count, [&](const ex::GroupTile &t) {
                if (UNITS == GROUP_WGRAD)
                    f(PairUnit{0, t.k_blocks, 0, 0, t.group, t.row0, t.n0, t.row_end, t.k0, t.k_rows, false, a.N});
                else
                    f(PairUnit{0, t.k_blocks, 0, t.group, 0, t.row0, t.n0, t.row_end, 0, a.K, false, a.N});
            });
    }
}

// Outputs of row groups that came out NaN made what IEEE arithmetic gives: a NaN
// among the inputs gives NaN, an infinity the dot product's own result. Run by
// the whole block for its units when all is written, so that nothing waits for
// it: the sums may be a whole group's rows long.
//
// A NaN in one row of a gradient makes every output of its matrix NaN, so dot
// products are not simply made again (a serial sum per output took 193 ms for
// 4096 rows, 2048 x 2048, and past the limit of the other roles' waits for 49152).
// A warp takes 32 x 32 outputs. Each lane looks for a NaN in its row of op(A)
// and, if outputs are left, in its column of op(B), 16 loads at a time; that
// explains all outputs but those that infinities made. For these the warp makes
// one dot product at a time, its lanes along k (partial sums added in a fixed
// order), until it is NaN. One NaN row in 4096: 0.72 ms in all (0.17 without), in
// 49152 9.7 ms (1.8).
template <PairUnits UNITS>
__device__ __noinline__ void repair_units(const Args &a, const ex::GroupTiles &gt, volatile int *abort_flag, int pair,
                                          int pairs, int rank) {
    constexpr int AHEAD = 16, LANES_AHEAD = 4;
    constexpr bool COLS = transposed(UNITS);
    const int lane = static_cast<int>(threadIdx.x & 31), warp = static_cast<int>(threadIdx.x >> 5);
    const int64_t am = a.ta ? 1 : a.lda, ak = a.ta ? a.lda : 1, bn = a.tb ? a.ldb : 1, bk = a.tb ? 1 : a.ldb;
    const int64_t cm = COLS ? 1 : a.ldc, cn = COLS ? a.ldc : 1;
    for_each_pair_unit<UNITS>(a, gt, abort_flag, pair, pairs, [&](const PairUnit &u) {
        if (u.ke == u.kb) return;
#pragma unroll 1
        for (int chunk = warp; chunk < 4 * pr::CHUNKS; chunk += pr::THREADS / 32) {
            const int64_t row0 = u.m0 + pr::HM * rank + 32 * (chunk / pr::CHUNKS), col0 = u.n0 + 32 * (chunk % pr::CHUNKS);
            const int rows = static_cast<int>(min(static_cast<int64_t>(32), u.m_end - row0));
            const int cols = static_cast<int>(min(static_cast<int64_t>(32), u.n_end - col0));
            if (rows <= 0 || cols <= 0) continue;
            const float *A = a.A + u.item_a * a.strideA + u.k0 * a.lda + row0 * am;
            const float *B = a.B + u.item_b * a.strideB + u.k0 * a.ldb + col0 * bn;
            float *C = a.C + u.item_c * a.strideC + row0 * cm + col0 * cn;
            const int64_t k_end = u.k_end;
            unsigned left = 0;  // of this lane's row: columns that hold an unexplained NaN
#pragma unroll 4
            for (int j = 0; j < cols; ++j) {
                const float x = lane < rows ? C[lane * cm + j * cn] : 0.0f;
                if (x != x) left |= 1u << j;
            }
            // Whether x[0], x[step], ... hold a NaN, for the lanes that ask.
            auto holds_nan = [&](bool asks, const float *x, int64_t step) {
                bool found = false;
#pragma unroll 1
                for (int64_t k = 0; k < k_end && __any_sync(0xffffffffu, asks && !found); k += AHEAD) {
                    float v[AHEAD];
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i) v[i] = asks && k + i < k_end ? x[(k + i) * step] : 0.0f;
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i) found |= v[i] != v[i];
                }
                return found;
            };
            if (holds_nan(left != 0, A + lane * am, ak)) left = 0;
            const unsigned some = __reduce_or_sync(0xffffffffu, left);  // columns with such a NaN
            left &= ~__ballot_sync(0xffffffffu, holds_nan((some >> lane) & 1, B + lane * bn, bk));
#pragma unroll 1
            for (unsigned open; (open = __ballot_sync(0xffffffffu, left != 0)) != 0;) {
                const int r = __ffs(open) - 1;
                const int j = __ffs(__shfl_sync(0xffffffffu, left, r)) - 1;
                const float *x = A + r * am, *y = B + j * bn;
                float sum = 0.0f;
#pragma unroll 1
                for (int64_t k0 = 0; k0 < k_end && !__any_sync(0xffffffffu, sum != sum); k0 += 32 * LANES_AHEAD) {
                    float p[LANES_AHEAD], q[LANES_AHEAD];
#pragma unroll
                    for (int i = 0; i < LANES_AHEAD; ++i) {
                        const int64_t k = k0 + 32 * i + lane;
                        p[i] = k < k_end ? x[k * ak] : 0.0f;
                        q[i] = k < k_end ? y[k * bk] : 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < LANES_AHEAD; ++i) sum = fmaf(p[i], q[i], sum);
                }
#pragma unroll
                for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (lane == r) {
                    C[r * cm + j * cn] = sum;
                    left &= ~(1u << j);
                }
            }
        }
    });
}

// TA: A stored K x M (op(A) = A^T); TB: B stored N x K (op(B) = B^T).
// Over a group's rows op(A) = A^T and op(B) = B.
// FOLD: the longest chain of k-blocks. LEAD > 0: in a chain's first LEAD
// k-blocks (and within every other) the small products, lo hi and hi lo, come
// before the large one, hi hi, while the accumulator is small and what the MMAs
// cut off it is too. At most OP_STAGES, which hold the k-blocks meanwhile.
template <bool VEC_C, bool TA, bool TB, PairUnits UNITS = TILES, int FOLD = pr::FOLD_KB, int LEAD = 0>
__global__ void __launch_bounds__(pr::THREADS, 1)
    tf32x3_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmC, const __grid_constant__ Args a,
                       const __grid_constant__ ex::GroupTiles gt) {
    static_assert(LEAD <= pr::OP_STAGES, "the leading k-blocks are staged together");
    constexpr bool SUMS_ROWS = sums_rows(UNITS), COLS = transposed(UNITS);
    static_assert(!SUMS_ROWS || (TA && !TB), "groups are summed along the stored rows of both operands");
    static_assert(UNITS != GROUP_COLS || TB, "the rows of C are K-major");
    static_assert(!COLS || LEAD > 0, "the width of tiles is the leading products' to set");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + pr::BAR_OFFSET);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + pr::NBARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + pr::NBARS + 1);
    // Target word of the odd CTA's st.async signals (its value is not used).
    const uint32_t signal_word = smem_u32(bars + pr::NBARS + 2);
    // Groups: this CTA wrote a NaN.
    volatile int *nan_flag = reinterpret_cast<volatile int *>(bars + pr::NBARS + 3);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
    auto bar = [&](int i) { return smem_u32(bars + i); };

    // TMA of this CTA's A rows (warp 1) or B columns (warp TMA_B_WARP) for
    // the k-blocks it = from .. to - 1 of its units, into the raw ring.
    const bool tma_warp = warp == 1 || warp == pr::TMA_B_WARP;
    auto tma_pass = [&](uint32_t from, uint32_t to) {
        if (a.wait_inputs) asm volatile("griddepcontrol.wait;" ::: "memory");
        const bool is_a = warp == 1;
        uint32_t it = 0;
        bool ok = true;
        for_each_pair_unit<UNITS>(a, gt, abort_flag, pair, pairs, [&](const PairUnit &u) {
            const int kb = u.kb, ke = u.ke;
            if (!ok || it >= to) return;
            if (it + static_cast<uint32_t>(ke - kb) <= from) {
                it += static_cast<uint32_t>(ke - kb);
                return;
            }
            const int m0 = static_cast<int>(u.m0) + pr::HM * static_cast<int>(rank);
            const int n0 = static_cast<int>(u.n0) + (COLS ? u.width() / 2 : pr::HN) * static_cast<int>(rank);
            const int za = u.item_a, zb = u.item_b;
            const int k0 = SUMS_ROWS ? static_cast<int>(u.k0) : 0;
            for (int kblk = kb; kblk < ke && it < to; ++kblk, ++it) {
                if (it < from) continue;
                const int slot = static_cast<int>(it % pr::RAW_SLOTS);
                const uint32_t ph = (it / pr::RAW_SLOTS) & 1;
                if (!mbar_wait(bar(pr::RAW_FREE + slot), ph ^ 1, a, abort_flag, WD_PRODUCER)) {
                    ok = false;
                    return;
                }
                const uint32_t sl = base + pr::RAW0 + static_cast<uint32_t>(slot * pr::SLOT);
                if (is_a) {
                    mbar_arrive_expect_tx(bar(pr::RAW_FULL + slot), pr::A_RAW);
                    if (TA) {  // A stored K x M: four boxes of 32 m x 32 k
#pragma unroll
                        for (int b = 0; b < pr::HM / 32; ++b)
                            tma_load_3d(sl + b * 4096, &tmA, m0 + 32 * b, k0 + kblk * BK, za, bar(pr::RAW_FULL + slot));
                    } else {
                        tma_load_3d(sl, &tmA, kblk * BK, m0, za, bar(pr::RAW_FULL + slot));
                    }
                } else {
                    mbar_arrive_expect_tx(bar(pr::RAW_FULL + slot), pr::B_HALF);
                    if (TB)  // B stored N x K: already K-major, 64 rows of 32 k
                        tma_load_3d(sl + pr::A_RAW, &tmB, kblk * BK, n0, zb, bar(pr::RAW_FULL + slot));
                    else
                        tma_load_3d(sl + pr::A_RAW, &tmB, n0, k0 + kblk * BK, zb, bar(pr::RAW_FULL + slot));
                }
            }
        });
    };

    // The same ring filled with 4-byte cp.async copies (a.cpa: rows that TMA
    // cannot address), by all lanes of warps 1 and TMA_B_WARP, each copying
    // half of this CTA's A tile and half of its B tile in the layouts the TMA
    // boxes have (A, and B stored N x K, in the 128-byte swizzle; B stored
    // K x N plain), zero outside the matrices. Every lane's copies for a slot
    // are tracked by one cp.async arrival on the slot's full barrier.
    auto load_pass = [&](uint32_t from, uint32_t to) {
        if (a.wait_inputs) asm volatile("griddepcontrol.wait;" ::: "memory");
        const int half = warp == 1 ? 0 : 1;
        uint32_t it = 0;
        bool ok = true;
        for_each_pair_unit<UNITS>(a, gt, abort_flag, pair, pairs, [&](const PairUnit &u) {
            const int kb = u.kb, ke = u.ke;
            if (!ok || it >= to) return;
            if (it + static_cast<uint32_t>(ke - kb) <= from) {
                it += static_cast<uint32_t>(ke - kb);
                return;
            }
            const int64_t m0 = u.m0 + pr::HM * static_cast<int64_t>(rank);
            const int64_t n0 = u.n0 + (COLS ? u.width() / 2 : pr::HN) * static_cast<int64_t>(rank);
            const int64_t K = UNITS == TILES ? a.K : u.k_end;
            const float *Ai = a.A + u.item_a * a.strideA + (SUMS_ROWS ? u.k0 * a.lda : 0);
            const float *Bi = a.B + u.item_b * a.strideB + (SUMS_ROWS ? u.k0 * a.ldb : 0);
            for (int kblk = kb; kblk < ke && it < to; ++kblk, ++it) {
                if (it < from) continue;
                const int slot = static_cast<int>(it % pr::RAW_SLOTS);
                const bool free = mbar_wait(bar(pr::RAW_FREE + slot), ((it / pr::RAW_SLOTS) & 1) ^ 1, a, abort_flag,
                                            WD_PRODUCER);
                if (!__all_sync(0xffffffffu, free)) {
                    ok = false;
                    return;
                }
                const uint32_t sl = base + pr::RAW0 + static_cast<uint32_t>(slot * pr::SLOT);
                const int64_t k0 = static_cast<int64_t>(kblk) * BK;
                const uint32_t lo4 = static_cast<uint32_t>((lane & 3) * 4);
                if (TA) {
                    // A stored K x M: boxes 2 half, 2 half + 1 of 32 k-rows x 32 m; lane = m.
                    for (int bx = 2 * half; bx < 2 * half + 2; ++bx) {
                        const int64_t m = m0 + 32 * bx + lane;
                        for (int r = 0; r < 32; ++r) {
                            const int64_t k = k0 + r;
                            const bool v = k < K && m < u.m_end;
                            cp_async4(sl + static_cast<uint32_t>(bx * 4096) + sw128_offset(r, lane >> 2) + lo4,
                                      v ? Ai + k * a.lda + m : Ai, v);
                        }
                    }
                } else {
                    // A rows 64 half .. 64 half + 63 of the tile; lane = k.
                    const int64_t k = k0 + lane;
                    for (int r = 64 * half; r < 64 * half + 64; ++r) {
                        const int64_t m = m0 + r;
                        const bool v = k < K && m < u.m_end;
                        cp_async4(sl + sw128_offset(r, lane >> 2) + lo4, v ? Ai + m * a.lda + k : Ai, v);
                    }
                }
                const uint32_t sb = sl + pr::A_RAW;
                if (TB) {
                    // B stored N x K: n-rows 32 half .. 32 half + 31 of 32 k; lane = k.
                    const int64_t k = k0 + lane;
                    for (int r = 32 * half; r < 32 * half + 32; ++r) {
                        const int64_t n = n0 + r;
                        const bool v = k < K && n < a.N;
                        cp_async4(sb + sw128_offset(r, lane >> 2) + lo4, v ? Bi + n * a.ldb + k : Bi, v);
                    }
                } else {
                    // B stored K x N: k-rows 16 half .. 16 half + 15 of 64 n (plain rows of 256 bytes).
                    for (int r = 16 * half; r < 16 * half + 16; ++r) {
                        const int64_t k = k0 + r;
#pragma unroll
                        for (int c2 = 0; c2 < 2; ++c2) {
                            const int64_t n = n0 + 32 * c2 + lane;
                            const bool v = k < K && n < a.N;
                            cp_async4(sb + static_cast<uint32_t>(r * pr::HN * 4 + (32 * c2 + lane) * 4),
                                      v ? Bi + k * a.ldb + n : Bi, v);
                        }
                    }
                }
                cp_async_arrive(bar(pr::RAW_FULL + slot));
            }
        });
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < pr::RAW_SLOTS; ++s) {
            // One expect_tx arrival per TMA issuer, or one cp.async arrival
            // per lane of the two loader warps.
            mbar_init(bar(pr::RAW_FULL + s), a.cpa ? 64 : 2);
            mbar_init(bar(pr::RAW_FREE + s), pr::GROUP_WARPS);  // one lane per converter warp
        }
        for (int s = 0; s < pr::OP_STAGES; ++s) {
            // Even CTA: one arrival per own converter warp (the first also
            // expects SIGNAL_BYTES), and SIGNAL_BYTES of transactions from the
            // odd CTA's converter warps (st.async, see below).
            mbar_init(bar(pr::OP_FULL + s), pr::GROUP_WARPS);
            mbar_init(bar(pr::OP_EMPTY + s), 1);
        }
        for (int d = 0; d < 2; ++d) {
            mbar_init(bar(pr::ACC_FULL + d), 1);
            mbar_init(bar(pr::ACC_EMPTY + d), 2 * pr::EPI_WARPS);
        }
        mbar_init(bar(pr::DRAIN), 1);
        *abort_flag = *nan_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tma_warp && lane == 0 && !a.cpa) {
        const bool is_a = warp == 1;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(is_a ? &tmA : &tmB)) : "memory");
    }
    __syncthreads();  // this CTA's mbarriers are initialised
    // Groups: launched while the kernel before it in the stream ends, whose
    // results (the group bounds among them) and tensor memory are waited for.
    if (UNITS != TILES) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 0) {
        // Both CTAs allocate: the pair's MMAs use the same columns in each.
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    // The cluster barrier publishes the peer's mbarriers before anyone
    // arrives on them, and the TMEM address to this CTA. The first loads
    // signal only this CTA's barriers, so the TMA issuers send them while the
    // pair meets (after their arrival, whose release would otherwise wait for
    // the loads).
    cluster_arrive();
    if (tma_warp) {
        if (a.cpa)
            load_pass(0, pr::RAW_SLOTS);
        else if (lane == 0)
            tma_pass(0, pr::RAW_SLOTS);
    }
    __syncwarp();
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    // A pass launched behind this kernel (the activation of split tiles) may
    // be scheduled now; it waits for this grid to finish before touching C.
    if (UNITS != TILES) asm volatile("griddepcontrol.launch_dependents;");
    if (a.signal_dependents && threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;");

    if (warp == 0) {
        // ------------------------------------------------------------ MMA issuer
        // A 256 x 128 x 8 MMA takes ~33 ns and the tensor core queues only a
        // few, so the issuer's own work between MMAs shows as idle tensor
        // time. The whole warp runs the loop (its values stay warp-uniform)
        // and one elected lane issues; the stage addresses are one add from
        // precomputed bases, and the next stage's barrier is tested while this
        // k-block's last k-slice is still queued.
        if (rank == 0) {
            const bool leader = elect_one();
            uint32_t it = 0, iv = 0;  // k-blocks and fold intervals issued so far
            const uint64_t desc0 = sw128_desc(base);
            const uint32_t a0 = tmem_base + pr::TMEM_A;
            bool ready = false;  // the stage of k-block `it` was seen full (and fenced) early
            for_each_pair_unit<UNITS>(a, gt, abort_flag, pair, pairs, [&](const PairUnit &u) {
                const int kb = u.kb, ke = u.ke;
                const uint32_t idesc = pr::idesc2(COLS ? u.width() : pr::PN);
                for (int k0 = kb; k0 < ke; k0 += FOLD) {
                    const int k1 = ke - k0 > FOLD ? k0 + FOLD : ke;
                    const uint32_t d = iv & 1;
                    // Accumulator d is free once the epilogue has folded the
                    // interval that used it two intervals back.
                    const bool ok = mbar_wait<true>(bar(pr::ACC_EMPTY + d), ((iv >> 1) & 1) ^ 1, a, abort_flag,
                                                    WD_MMA_ACC);
                    if (!__all_sync(0xffffffffu, ok)) return;
                    tc_fence_after();
                    const uint32_t dt = tmem_base + d * pr::PN;
                    if (LEAD > 0) {
                        for (int kblk = k0; kblk < k1;) {
                            const int lead = kblk == k0 && k1 - k0 > LEAD ? LEAD : 1;
                            for (int i = 0; i < lead; ++i) {
                                const uint32_t nx = it + static_cast<uint32_t>(i), s = nx % pr::OP_STAGES;
                                const bool full = mbar_wait<true>(bar(pr::OP_FULL + s), (nx / pr::OP_STAGES) & 1, a,
                                                                  abort_flag, WD_MMA_FULL);
                                if (!__all_sync(0xffffffffu, full)) return;
                                tc_fence_after();
                                const uint64_t b_hi = desc0 + static_cast<uint64_t>(s * (pr::OP_STAGE >> 4));
                                const uint64_t b_lo = b_hi + (pr::B_HALF >> 4);
                                const uint32_t a_hi = a0 + 64 * s, a_lo = a_hi + 32;
                                if (leader) {
#pragma unroll
                                    for (int ks = 0; ks < BK / 8; ++ks) {
                                        // C^T: the factors' order the other way round, for the same sums.
                                        const uint32_t more = ks > 0 || i > 0 || kblk > k0;
                                        const uint32_t a1 = COLS ? a_hi : a_lo, a2 = COLS ? a_lo : a_hi;
                                        const uint64_t b1 = COLS ? b_lo : b_hi, b2 = COLS ? b_hi : b_lo;
                                        tc_mma2_ts(dt, a1 + ks * 8, b1 + ks * 2, more, idesc);
                                        tc_mma2_ts(dt, a2 + ks * 8, b2 + ks * 2, 1u, idesc);
                                    }
                                }
                                __syncwarp();
                            }
                            for (int i = 0; i < lead; ++i, ++it, ++kblk) {
                                const uint32_t s = it % pr::OP_STAGES;
                                const uint64_t b_hi = desc0 + static_cast<uint64_t>(s * (pr::OP_STAGE >> 4));
                                const uint32_t a_hi = a0 + 64 * s;
                                if (leader) {
#pragma unroll
                                    for (int ks = 0; ks < BK / 8; ++ks)
                                        tc_mma2_ts(dt, a_hi + ks * 8, b_hi + ks * 2, 1u, idesc);
                                    tc_commit2(bar(pr::OP_EMPTY + s));
                                }
                                __syncwarp();
                            }
                        }
                    }
                    for (int kblk = k0; LEAD == 0 && kblk < k1; ++kblk, ++it) {
                        const uint32_t s = it % pr::OP_STAGES;
                        if (!ready) {
                            const bool full = mbar_wait<true>(bar(pr::OP_FULL + s), (it / pr::OP_STAGES) & 1, a,
                                                              abort_flag, WD_MMA_FULL);
                            if (!__all_sync(0xffffffffu, full)) return;
                            tc_fence_after();
                        }
                        const uint64_t b_hi = desc0 + static_cast<uint64_t>(s * (pr::OP_STAGE >> 4));
                        const uint64_t b_lo = b_hi + (pr::B_HALF >> 4);
                        const uint32_t a_hi = a0 + 64 * s, a_lo = a_hi + 32;
                        const uint32_t acc0 = kblk == k0 ? 0u : 1u;  // each interval starts its accumulator
#pragma unroll
                        for (int ks = 0; ks < BK / 8; ++ks) {
                            const uint64_t adv = static_cast<uint64_t>(ks * 2);
                            const uint32_t ac = static_cast<uint32_t>(ks * 8);
                            if (ks == BK / 8 - 1) {
                                // The next k-block's stage, tested without blocking.
                                const uint32_t nx = it + 1;
                                ready = __all_sync(0xffffffffu, mbar_test_wait<true>(bar(pr::OP_FULL + nx % pr::OP_STAGES),
                                                                                     (nx / pr::OP_STAGES) & 1));
                                if (ready) tc_fence_after();
                            }
                            if (leader) {
                                tc_mma2_ts(dt, a_lo + ac, b_hi + adv, ks == 0 ? acc0 : 1u);
                                tc_mma2_ts(dt, a_hi + ac, b_lo + adv, 1u);
                                tc_mma2_ts(dt, a_hi + ac, b_hi + adv, 1u);
                            }
                            __syncwarp();
                        }
                        if (leader) tc_commit2(bar(pr::OP_EMPTY + s));
                        __syncwarp();
                    }
                    if (leader) tc_commit2(bar(pr::ACC_FULL + d));
                    __syncwarp();
                    ++iv;
                }
            });
            if (leader) tc_commit2(bar(pr::DRAIN));
            __syncwarp();
            if (lane == 0) {
                const bool was_aborted = *abort_flag != 0;
                if (!mbar_wait(bar(pr::DRAIN), 0, a, abort_flag, WD_DRAIN) && was_aborted) {
                    const uint64_t t0 = global_timer();
                    while (!mbar_try_wait(bar(pr::DRAIN), 0) && global_timer() - t0 < a.timeout_ns) {
                    }
                }
            }
        }
    } else if (tma_warp) {
        // ---------------------------------------------------- TMA issuers (A, B)
        if (a.cpa)
            load_pass(pr::RAW_SLOTS, 0xffffffffu);
        else if (lane == 0)
            tma_pass(pr::RAW_SLOTS, 0xffffffffu);
    } else if (warp < pr::EPI_WARP0) {
        // ------------------------------------------------------------ converters
        const int cw = warp - 2;                                 // 0 .. 15
        const uint32_t group = static_cast<uint32_t>(cw >> 2);  // k-blocks with it % 4 == group
        const int ct = ((cw & 3) << 5) + lane;                   // 0 .. 127 within the group
        const int l = ct & 7, tb = ct >> 3;                      // 16 groups of eight lanes
        const int g = (tb >> 3) * 8 + l, c = (l + tb) & 7;       // this thread's 4 x 4 B block
        const int q = warp & 3;                                  // TMEM lane quarter
        const int arow = 32 * q + lane;                          // A row this thread converts
        uint32_t it = 0;
        bool ok = true;
        for_each_pair_unit<UNITS>(a, gt, abort_flag, pair, pairs, [&](const PairUnit &u) {
            const int kb = u.kb, ke = u.ke;
            if (!ok) return;
            const int quarters = COLS ? u.width() / 32 : 4;  // of 16 rows of B that the MMAs read
            for (int kblk = kb; kblk < ke; ++kblk, ++it) {
                if (it % pr::CONV_GROUPS != group) continue;
                const int slot = static_cast<int>(it % pr::RAW_SLOTS);
                const int s = static_cast<int>(it % pr::OP_STAGES);
                if (!mbar_wait(bar(pr::RAW_FULL + slot), (it / pr::RAW_SLOTS) & 1, a, abort_flag, WD_PRODUCER)) {
                    ok = false;
                    return;
                }
                const uint32_t sl = base + pr::RAW0 + static_cast<uint32_t>(slot * pr::SLOT);
                // A: the 32 k-values of row arow.
                float av[32];
                if (TA) {
                    // Box q holds rows k = 0..31 of columns m = 32q..32q+31 (128-byte
                    // swizzled): column arow is lane `lane` of each row.
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        av[j] = ld_shared_f32(sl + static_cast<uint32_t>(q * 4096) + sw128_offset(j, lane >> 2) +
                                              static_cast<uint32_t>((lane & 3) * 4));
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 t = ld_shared_v4(sl + sw128_offset(arow, j));
                        av[4 * j] = t.x;
                        av[4 * j + 1] = t.y;
                        av[4 * j + 2] = t.z;
                        av[4 * j + 3] = t.w;
                    }
                }
                // B: op(B) = B: rows 4c..4c+3, columns 4g..4g+3 of the unswizzled 32 x 64
                // staging tile; op(B) = B^T: four 16-byte chunks of the K-major tile.
                float4 bq[4];
#pragma unroll
                for (int qq = 0; qq < 4; ++qq)
                    bq[qq] = TB ? ld_shared_v4(sl + pr::A_RAW + static_cast<uint32_t>((qq * pr::CONV_THREADS + ct) * 16))
                                : ld_shared_v4(sl + pr::A_RAW +
                                               static_cast<uint32_t>((4 * c + qq) * pr::HN * 4 + g * 16));
                fence_proxy_async_smem();  // order these loads before the next TMA into the slot
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(pr::RAW_FREE + slot));
                if (SUMS_ROWS) {
                    // Rows past the group's end belong to the next group: zeros in both
                    // operands (zero times its infinities or NaN would not do).
                    const int64_t left = u.k_end - static_cast<int64_t>(kblk) * BK;
                    if (left < BK) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j >= left) av[j] = 0.0f;
#pragma unroll
                        for (int qq = 0; qq < 4; ++qq)
                            if (4 * c + qq >= left) bq[qq] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    }
                }
                // The stage is free once the pair's MMAs four k-blocks back are done.
                if (!mbar_wait<true>(bar(pr::OP_EMPTY + s), ((it / pr::OP_STAGES) & 1) ^ 1, a, abort_flag,
                                     WD_PRODUCER)) {
                    ok = false;
                    return;
                }
                tc_fence_after();
                const uint32_t st = base + static_cast<uint32_t>(s * pr::OP_STAGE);
                if (TB) {
                    // Same swizzled K-major layout: chunk for chunk.
#pragma unroll
                    for (int qq = 0; qq < 4; ++qq) {
                        
                        if (TB && COLS && qq >= quarters) break;
                        const uint32_t off = static_cast<uint32_t>((qq * pr::CONV_THREADS + ct) * 16);
                        split_store(st + off, st + pr::B_HALF + off, bq[qq].x, bq[qq].y, bq[qq].z, bq[qq].w);
                    }
                } else {
                    // Column j of the 4 x 4 block is chunk c of operand row 4g + j.
                    uint32_t off = sw128_offset(4 * g + 0, c);
                    split_store(st + off, st + pr::B_HALF + off, bq[0].x, bq[1].x, bq[2].x, bq[3].x);
                    off = sw128_offset(4 * g + 1, c);
                    split_store(st + off, st + pr::B_HALF + off, bq[0].y, bq[1].y, bq[2].y, bq[3].y);
                    off = sw128_offset(4 * g + 2, c);
                    split_store(st + off, st + pr::B_HALF + off, bq[0].z, bq[1].z, bq[2].z, bq[3].z);
                    off = sw128_offset(4 * g + 3, c);
                    split_store(st + off, st + pr::B_HALF + off, bq[0].w, bq[1].w, bq[2].w, bq[3].w);
                }
                const uint32_t ta =
                    tmem_base + (static_cast<uint32_t>(32 * q) << 16) + pr::TMEM_A + static_cast<uint32_t>(64 * s);
#pragma unroll
                for (int h = 0; h < 4; ++h) {  // 8 values at a time: fewer live registers
                    float hi[8], lo[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) split_tf32(av[8 * h + j], hi[j], lo[j]);
                    tmem_store8(ta + 8 * h, hi);
                    tmem_store8(ta + 32 + 8 * h, lo);
                }
                tmem_wait_st();
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank != 0)
                        st_async_signal(signal_word, bar(pr::OP_FULL + s), 0);  // the even CTA issues the MMAs
                    else if ((cw & 3) == 0)
                        mbar_arrive_expect_tx(bar(pr::OP_FULL + s), pr::SIGNAL_BYTES);
                    else
                        mbar_arrive(bar(pr::OP_FULL + s));
                }
            }
        });
    } else {
        // -------------------------------------------------------------- epilogue
        const int q = warp & 3;  // TMEM lane quarter this warp may access
        const uint32_t rq = base + pr::R0 + static_cast<uint32_t>(q * pr::CHUNKS * pr::C_CHUNK);  // its chunks
        // C may still be in the beta pre-pass launched just before this
        // kernel (programmatic dependent launch): only the epilogue waits.
        asm volatile("griddepcontrol.wait;" ::: "memory");
        uint32_t iv = 0;  // fold intervals consumed so far
        auto release = [&](uint32_t d) {
            // Accumulator d is out of TMEM: one lane per warp frees it on the
            // even CTA's barrier.
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_at(bar(pr::ACC_EMPTY + d), 0);
        };
        for_each_pair_unit<UNITS>(a, gt, abort_flag, pair, pairs, [&](const PairUnit &u) {
            const int kb = u.kb, ke = u.ke;
            const int64_t row0 = u.m0 + pr::HM * static_cast<int64_t>(rank) + q * 32;
            const int64_t row = row0 + lane;
            // Stream-K tiles hold beta * C + bias already: every unit adds.
            const bool atomic = u.atomic;
            const bool fused = a.ep && !atomic;
            const bool col_bias = a.bias_kind == SGEMM_BIAS_PER_COL;
            const float rb = (a.bias_kind == SGEMM_BIAS_PER_ROW && row < u.m_end) ? __ldg(a.bias + row) : 0.0f;
            if constexpr (COLS) {
                // C^T: lanes are columns of C, accumulator columns its rows, written
                // straight from registers, 128 bytes of a row at a time.
                const int chunks = u.width() / 32;
                const bool mine = row < u.m_end;
                auto write = [&](int ch, const float (&v)[32]) {
                    const int64_t r0 = u.n0 + ch * 32;
                    float *p = a.C + u.item_c * a.strideC + r0 * a.ldc + row;
                    const int rows = static_cast<int>(min(static_cast<int64_t>(32), u.n_end - r0));
                    const int64_t ldc = a.ldc;
                    if (!mine) return;
                    if (rows == 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j, p += ldc) *p = v[j];
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j < rows) p[j * ldc] = v[j];
                    }
                };
                if (ke == kb) {
                    const float zeros[32] = {};
#pragma unroll 1
                    for (int ch = 0; ch < chunks; ++ch) write(ch, zeros);
                    return;
                }
                for (int k0 = kb; k0 < ke; k0 += FOLD) {
                    const bool first = k0 == kb, last = ke - k0 <= FOLD;
                    const uint32_t d = iv & 1;
                    if (!mbar_wait<true>(bar(pr::ACC_FULL + d), (iv >> 1) & 1, a, abort_flag, WD_EPILOGUE)) return;
                    tc_fence_after();
                    ++iv;
                    const uint32_t dt = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + d * pr::PN;
#pragma unroll 1
                    for (int ch = 0; ch < chunks; ++ch) {
                        const uint32_t rc = rq + static_cast<uint32_t>(ch * pr::C_CHUNK);
                        float v[32];
                        tmem_load32(dt + static_cast<uint32_t>(ch * 32), v);
                        if (ch == chunks - 1) release(d);
                        if (!first) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float4 r = ld_shared_v4(rc + sw128_offset(lane, j));
                                v[4 * j] += r.x;
                                v[4 * j + 1] += r.y;
                                v[4 * j + 2] += r.z;
                                v[4 * j + 3] += r.w;
                            }
                        }
                        if (!last) {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                st_shared_v4(rc + sw128_offset(lane, j), v[4 * j], v[4 * j + 1], v[4 * j + 2],
                                             v[4 * j + 3]);
                        } else {
                            bool nan = false;
#pragma unroll
                            for (int j = 0; j < 32; ++j) nan |= v[j] != v[j];
                            if (nan) *nan_flag = 1;
                        }
                        if (last) write(ch, v);
                        __syncwarp();
                    }
                }
                return;
            }
            // The previous unit's TMA stores read the running sum: wait until
            // they have, before this unit overwrites it.
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
            if (UNITS != TILES && ke == kb) {
                // Nothing to sum (rows of no group, the matrix of an empty group): zeros.
#pragma unroll 1
                for (int ch = 0; ch < pr::CHUNKS; ++ch) {
                    const int64_t col0 = u.n0 + ch * 32;
                    const uint32_t rc = rq + static_cast<uint32_t>(ch * pr::C_CHUNK);
                    if (row0 >= u.m_end || col0 >= a.N) continue;
#pragma unroll
                    for (int j = 0; j < 8; ++j) st_shared_v4(rc + sw128_offset(lane, j), 0.0f, 0.0f, 0.0f, 0.0f);
                    __syncwarp();
                    store_staged_rows(a, rc, a.C + u.item_c * a.strideC, u.m_end, row0, col0, false);
                }
                __syncwarp();
                return;
            }
            for (int k0 = kb; k0 < ke; k0 += FOLD) {
                const bool first = k0 == kb, last = ke - k0 <= FOLD;
                const uint32_t d = iv & 1;
                if (!mbar_wait<true>(bar(pr::ACC_FULL + d), (iv >> 1) & 1, a, abort_flag, WD_EPILOGUE)) return;
                tc_fence_after();
                ++iv;
                const uint32_t dt = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + d * pr::PN;
#pragma unroll 1
                for (int ch = 0; ch < pr::CHUNKS; ++ch) {
                    const uint32_t rc = rq + static_cast<uint32_t>(ch * pr::C_CHUNK);
                    const int64_t col0 = u.n0 + ch * 32;
                    float v[32];
                    tmem_load32(dt + static_cast<uint32_t>(ch * 32), v);
                    if (ch == pr::CHUNKS - 1) release(d);
                    if (!first) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 r = ld_shared_v4(rc + sw128_offset(lane, j));
                            v[4 * j] += r.x;
                            v[4 * j + 1] += r.y;
                            v[4 * j + 2] += r.z;
                            v[4 * j + 3] += r.w;
                        }
                    }
                    if (!last) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            st_shared_v4(rc + sw128_offset(lane, j), v[4 * j], v[4 * j + 1], v[4 * j + 2],
                                         v[4 * j + 3]);
                        continue;
                    }
                    // The unit's sum is complete: write this chunk of C.
                    bool nan = false;
#pragma unroll
                    for (int j = 0; j < 32; ++j) nan |= v[j] != v[j];
                    if (UNITS != TILES && nan) *nan_flag = 1;
                    if ((UNITS == TILES && __any_sync(0xffffffffu, nan)) || !a.c_tma || col0 + 32 > a.N ||
                        row0 + 32 > u.m_end) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            st_shared_v4(rc + sw128_offset(lane, j), v[4 * j], v[4 * j + 1], v[4 * j + 2],
                                         v[4 * j + 3]);
                        const int64_t k_end = min(static_cast<int64_t>(ke) * BK, u.k_end);
                        edge_final_chunk<VEC_C, UNITS == TILES>(a, rc, a.A + u.item_a * a.strideA + (SUMS_ROWS ? u.k0 * a.lda : 0),
                                                a.B + u.item_b * a.strideB + (SUMS_ROWS ? u.k0 * a.ldb : 0),
                                                a.C + u.item_c * a.strideC, u.m_end, row0, col0, atomic,
                                                static_cast<int64_t>(kb) * BK, k_end);
                        continue;
                    }
                    if (fused) {
                        // Per-column bias of this chunk: lane l holds column col0 + l.
                        const float bl = col_bias ? __ldg(a.bias + col0 + lane) : rb;
                        stage32_fused(a.act, rc, lane, a.alpha, col_bias, bl, v);
                    } else {
                        const float alpha = a.alpha;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            st_shared_v4(rc + sw128_offset(lane, j), alpha * v[4 * j], alpha * v[4 * j + 1],
                                         alpha * v[4 * j + 2], alpha * v[4 * j + 3]);
                    }
                    fence_proxy_async_smem();  // chunk writes -> visible to the TMA engine
                    __syncwarp();
                    if (lane == 0) {
                        const int x = static_cast<int>(col0), y = static_cast<int>(row0);
                        if (atomic)
                            tma_reduce_add_3d(&tmC, x, y, u.item_c, rc);
                        else
                            tma_store_3d(&tmC, x, y, u.item_c, rc);
                        bulk_commit();
                    }
                }
            }
        });
        if (lane == 0) bulk_wait<0>();  // every store of this warp has landed
    }

    // The odd CTA's TMEM is written by the even CTA's MMAs: wait for them to
    // drain before the pair releases it. After a wait that gave up, loads may
    // still be on their way: leave them time to land.
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) {
        const uint64_t t0 = global_timer();
        while (global_timer() - t0 < 10000000ull) {
        }
    }
    if (rank != 0 && threadIdx.x == 0) {
        if (!mbar_wait<true>(bar(pr::DRAIN), 0, a, abort_flag, WD_DRAIN)) {
            const uint64_t t0 = global_timer();
            while (!mbar_try_wait<true>(bar(pr::DRAIN), 0) && global_timer() - t0 < a.timeout_ns) {
            }
        }
    }
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == 0) {
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS)
                     : "memory");
    }
    if constexpr (UNITS != TILES) {
        if (*nan_flag) repair_units<UNITS>(a, gt, abort_flag, pair, pairs, static_cast<int>(rank));
    }
}

}  // namespace
}  // namespace sgemm
