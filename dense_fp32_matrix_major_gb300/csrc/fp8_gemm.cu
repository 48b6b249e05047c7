// Products of 8-bit matrices with a scale for each block of 128 summed values,
// on SM pairs (tcgen05, cta_group::2, kind::f8f6f4):
//
//     rows   C[s] = sum over blocks b of sA[b][s] sB[e(s)][n / 128][b] P_b[s][n]
//     wgrad  C[e][m][n] = sum over blocks b of group e of sA[b][m] sB[b][n] P_b[m][n]
//
// P_b is the sum of a block's 128 products. Products of two 8-bit values are
// exact in fp32. The tensor core sums one block in tensor memory; the epilogue
// takes it out, scales it and adds it, in fp32 and in the blocks' order, to a
// running sum in registers, which is rounded once, when C is written.
//
// Two CTAs on two SMs of a cluster make a tile of 256 columns of C by up to 256
// rows. The MMA's first operand gives C's columns (op(B), 128 of them staged by
// each CTA) and its second C's rows (A), whose number, the MMA's width, costs
// time in steps of 32: a group of 40 rows is charged 64. A group's rows are
// spread evenly over its tiles. Two buffers of 256 columns fill tensor memory:
// the epilogue empties one while the tensor core fills the other.
//
// Scales. The lanes of tensor memory are C's columns, so in rows a CTA's 128
// lanes share B's scale and the product of the two scales depends on C's row
// only, an accumulator column. Loads of 16 lanes x 8 columns (16x256b) leave
// each thread four lanes and a quarter of the columns, so it needs a quarter of
// the scales. Warp 2 multiplies them ahead of time and lays them out in a ring in
// the order the threads read them. wgrad's second factor, C's column, is a factor
// for each of the thread's four lanes.
//
// Layouts. An operand whose summed direction is contiguous in memory is staged
// K-major, otherwise MN-major, both in 128-byte swizzled rows as TMA writes
// them; the MMA takes either, so nothing is transposed.
//
// Groups. The bounds are read on the device. Tiles never cross groups; the
// workers (one CTA pair each) take the tiles of the groups in order, round
// robin, each role of a worker walking the bounds for itself. Rows staged past a
// tile's end belong to the next and change only sums that are not written. In
// wgrad every group's rows start in a block of their own and end in zeros.
//
// Roles in each CTA (12 warps): warp 0 loads the first operand and warp 3 the
// second (TMA), warp 1 of the even CTA issues the MMAs, warp 2 prepares scales,
// warps 4 to 11 sum and write C (two per quarter of tensor memory's lanes). They
// hold 128 sums a thread and take registers that the first four give up. The
// loads of both CTAs complete on the even CTA's barriers. Every wait is bounded.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "experts_common.cuh"
#include "fp8_internal.h"
#include "tc_common.cuh"

namespace sgemm {
namespace f8 {
namespace {

using namespace tc;

constexpr int PN = 256, PM = 256, HALF = 128;  // C's columns and rows of a pair, a CTA's share
constexpr int KB = BLOCK;                      // k-block: 128 values = 128 bytes
constexpr int ROW_STEP = 32;                   // a tile's rows are charged in multiples of it
constexpr int BOX = 128 * 128;                 // bytes of a staged operand
constexpr int STAGE = 2 * BOX, STAGES = 6;
constexpr int EPI_WARPS = 8, EPI_WARP = 4, THREADS = (EPI_WARP + EPI_WARPS) * 32;
constexpr int RING = 8;                        // k-blocks of prepared scales
constexpr int RING_BYTES = (PM + HALF) * 4;    // of C's rows, and of the CTA's columns (wgrad)
constexpr int OUT_ROW = 144;                   // bytes between rows of a warp's 8 x 32 values of C on their way out
constexpr int OUT_BYTES = 8 * OUT_ROW;
constexpr int RING0 = STAGES * STAGE, OUT0 = RING0 + RING * RING_BYTES, BAR0 = OUT0 + EPI_WARPS * OUT_BYTES;
// mbarriers
constexpr int FULL = 0, EMPTY = FULL + STAGES, SUM_FULL = EMPTY + STAGES, SUM_EMPTY = SUM_FULL + 2,
              RING_FULL = SUM_EMPTY + 2, RING_EMPTY = RING_FULL + RING, DRAIN = RING_EMPTY + RING, NBARS = DRAIN + 1;
constexpr int SMEM_BYTES = BAR0 + 512 + 1024;
static_assert(NBARS * 8 + 16 <= 512, "barrier block");
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
static_assert(RING0 % 1024 == 0 && RING_BYTES % 16 == 0 && OUT0 % 16 == 0 && BAR0 % 8 == 0, "alignment");
// Registers a thread of the four and of the eight warps, out of 168 each.
constexpr int FEW_REGS = 80, MANY_REGS = 208;
static_assert(4 * FEW_REGS + 8 * MANY_REGS <= 12 * 168, "registers of the launch");

enum Form { ROWS_N, ROWS_T, WGRAD };

struct Args {
    const int32_t *offsets;  // NULL: one group
    int rows, experts;
    int tiles_n;
    int blocks;        // wgrad: of A and B
    int k_blocks;      // rows
    int64_t M, N;      // wgrad: rows of a matrix of C; columns of C
    const float *scale_rows;  // [block][row of C]
    int64_t ld_rows;
    const float *scale_cols;  // rows: [item][n / 128][block] in the strides below; wgrad: [block][column of C]
    int64_t item_cols, n_cols, b_cols;
    void *C;
    int64_t ldc, strideC;
    int out_type, vector;  // C in 16-byte stores
    uint32_t idesc;        // without N
    uint64_t timeout_ns;
    int *watchdog;
};

// A tile: rows row0 .. row_end of C (rows: of all, wgrad: of the group's matrix),
// columns from n0 on, k_blocks blocks from block k0 on.
struct Tile {
    int group, row0, row_end, n0, k0, k_blocks;
};

__device__ __forceinline__ int start_of(const Args &a, int e) {
    return a.offsets ? ex::group_start(a.offsets, e, a.rows) : (e == 0 ? 0 : a.rows);
}

template <Form FORM, class F>
__device__ __forceinline__ void for_each_tile(const Args &a, volatile int *abort_flag, int index, int count, F &&f) {
    int e = 0, begin = 0, base = 0, first = 0;  // base: tiles (rows: of rows) before group e; first: blocks
    int next = start_of(a, 1), end = max(begin, next);
    const int tiles_m = static_cast<int>((a.M + PM - 1) / PM);  // wgrad
    int tiles = FORM == WGRAD ? tiles_m : (end - begin + PM - 1) / PM;
    for (int64_t u = index;; u += count) {
        if (*abort_flag) return;
        const int rt = static_cast<int>(u / a.tiles_n);
        while (rt >= base + tiles) {
            if (e == a.experts) return;
            base += tiles;
            if (FORM == WGRAD) first += (end - begin + KB - 1) / KB;
            ++e;
            if (FORM == WGRAD && e == a.experts) return;
            begin = next;
            next = e < a.experts ? start_of(a, e + 1) : a.rows;
            end = max(begin, next);
            if (FORM != WGRAD) tiles = (end - begin + PM - 1) / PM;
        }
        const int n0 = static_cast<int>(u % a.tiles_n) * PN;
        if (FORM == WGRAD) {
            const int row0 = (rt - base) * PM;
            const int b0 = min(first, a.blocks), b1 = min(first + (end - begin + KB - 1) / KB, a.blocks);
            f(Tile{e, row0, static_cast<int>(min(static_cast<int64_t>(row0 + PM), a.M)), n0, b0, b1 - b0});
        } else {
            const int each = ((end - begin + tiles - 1) / tiles + ROW_STEP - 1) / ROW_STEP * ROW_STEP;
            const int row0 = min(begin + (rt - base) * each, end);
            f(Tile{e, row0, min(row0 + each, end), n0, 0, e < a.experts && row0 < end ? a.k_blocks : 0});
        }
    }
}

// The MMA's width: the tile's rows, rounded up.
__device__ __forceinline__ int width_of(const Tile &u) {
    return (u.row_end - u.row0 + ROW_STEP - 1) / ROW_STEP * ROW_STEP;
}

// TMA load into this CTA's shared memory that completes its bytes on the
// mbarrier at shared::cluster address `bar` (of either CTA of the pair).
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
        "{%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint32_t map_to_cta(uint32_t addr, uint32_t cta) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
    return r;
}

__device__ __forceinline__ void mma8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 lanes x 16 columns of 32 bits from tensor memory: r[4 g + 2 h + i] is lane
// (thread / 4) + 8 h, column 8 g + 2 (thread % 4) + i. Not waited for.
__device__ __forceinline__ void tmem_load_16x16(uint32_t taddr, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// Waits for the thread's loads from tensor memory; ties the registers to it.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}

__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

// Two fp32 multiply-adds or products, each rounded to nearest.
__device__ __forceinline__ void fma2(uint64_t &acc, uint64_t x, uint64_t y) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(x), "l"(y));
}

__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}

__device__ __forceinline__ void lds_2x64(uint32_t at, uint64_t &x, uint64_t &y) {
    asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(at) : "memory");
}

__device__ __forceinline__ uint4 lds_128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// Four 8 x 8 blocks of 16-bit values stored transposed; lane 8 i + r gives the
// address of row r of block i.
__device__ __forceinline__ void stmatrix4_trans(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ uint32_t round2(uint64_t v, bool bf16) {
    float lo, hi;
    unpack2(v, lo, hi);
    if (bf16) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&r);
    }
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Eight rows of C by a warp's 32 columns, v[h] the sums of lanes (columns) 8 h ..
// 8 h + 7, through shared memory: rows of 64 or 128 bytes, 16 bytes a store.
__device__ __forceinline__ void write_rows(const Args &a, uint32_t out, int lane, const uint64_t (&v)[4], void *c_item,
                                           int64_t row, int rows, int64_t col) {
    const int t = lane & 3, g = lane >> 2;
    __syncwarp();  // what the buffer held is read
    if (a.out_type == SGEMM_TYPE_F32) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            float lo, hi;
            unpack2(v[h], lo, hi);
            const uint32_t at = out + static_cast<uint32_t>(2 * t * OUT_ROW + (8 * h + g) * 4);
            st_shared_f32(at, lo);
            st_shared_f32(at + OUT_ROW, hi);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 4 * i + (lane >> 3), c = 4 * (lane & 7);
            const uint4 x = lds_128(out + static_cast<uint32_t>(r * OUT_ROW + c * 4));
            float *p = static_cast<float *>(c_item) + (row + r) * a.ldc + col + c;
            if (r >= rows) continue;
            if (a.vector && col + c + 4 <= a.N) {
                *reinterpret_cast<uint4 *>(p) = x;
            } else {
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (col + c + j < a.N) p[j] = __uint_as_float(w[j]);
            }
        }
    } else {
        const bool bf16 = a.out_type == SGEMM_TYPE_BF16;
        constexpr int ROW16 = 80;  // bytes: every phase of the stores and loads meets all banks
        stmatrix4_trans(out + static_cast<uint32_t>((lane & 7) * ROW16 + (lane >> 3) * 16), round2(v[0], bf16),
                        round2(v[1], bf16), round2(v[2], bf16), round2(v[3], bf16));
        __syncwarp();
        const int c = 8 * t;
        const uint4 x = lds_128(out + static_cast<uint32_t>(g * ROW16 + c * 2));
        uint16_t *p = static_cast<uint16_t *>(c_item) + (row + g) * a.ldc + col + c;
        if (g < rows) {
            if (a.vector && col + c + 8 <= a.N) {
                *reinterpret_cast<uint4 *>(p) = x;
            } else {
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + c + j < a.N) p[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
            }
        }
    }
}

template <Form FORM>
__global__ void __launch_bounds__(THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tm1, const __grid_constant__ CUtensorMap tm2,
                    const __grid_constant__ CUtensorMap tm2_small, const __grid_constant__ Args a) {
    // tm1, tm2: the operands of C's columns and rows; tm2_small: the second in boxes of 32 rows (rows).
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem_raw + (base - raw) + BAR0);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + NBARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + NBARS + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
    auto bar = [&](int i) { return smem_u32(bars + i); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar(FULL + s), 1);
            mbar_init(bar(EMPTY + s), 1);
        }
        for (int d = 0; d < 2; ++d) {
            mbar_init(bar(SUM_FULL + d), 1);
            mbar_init(bar(SUM_EMPTY + d), 2 * EPI_WARPS);
        }
        for (int r = 0; r < RING; ++r) {
            mbar_init(bar(RING_FULL + r), 1);
            mbar_init(bar(RING_EMPTY + r), EPI_WARPS);
        }
        mbar_init(bar(DRAIN), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm1)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm2)) : "memory");
    }
    __syncthreads();
    // Launched while the kernel before it in the stream ends: wait for its
    // results (and its tensor memory).
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    asm volatile("griddepcontrol.launch_dependents;");

    if (warp < EPI_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FEW_REGS));
        if (warp == 0 || warp == 3) {
            // -------------------------------------------------------------- loads
            const bool first = warp == 0;  // the first operand (and the barriers' bytes), or the second
            if (lane == 0) {
                uint32_t it = 0;
                bool ok = true;
                for_each_tile<FORM>(a, abort_flag, pair, pairs, [&](const Tile &u) {
                    const int half = width_of(u) / 2;
                    const int n0 = u.n0 + HALF * static_cast<int>(rank);
                    const int r0 = u.row0 + half * static_cast<int>(rank);
                    // One box of 128 rows, or of 32 where those are enough.
                    const bool small = FORM != WGRAD && half <= 32;
                    const uint32_t bytes = BOX + (small ? 32 * 128 : BOX);
                    for (int kb = 0; kb < u.k_blocks && ok; ++kb, ++it) {
                        const int s = static_cast<int>(it % STAGES);
                        if (!mbar_wait<true>(bar(EMPTY + s), ((it / STAGES) & 1) ^ 1, a, abort_flag, WD_PRODUCER)) {
                            ok = false;
                            return;
                        }
                        const uint32_t s1 = base + static_cast<uint32_t>(s * STAGE), s2 = s1 + BOX;
                        const uint32_t to = map_to_cta(bar(FULL + s), 0);
                        const int k = (u.k0 + kb) * KB;
                        if (first) {
                            if (rank == 0) mbar_arrive_expect_tx(bar(FULL + s), 2 * bytes);
                            if (FORM == WGRAD)
                                tma_load_pair(s1, &tm1, n0, k, 0, to);
                            else if (FORM == ROWS_T)
                                tma_load_pair(s1, &tm1, k, n0, u.group, to);
                            else
                                tma_load_pair(s1, &tm1, n0, k, u.group, to);
                        } else if (FORM == WGRAD) {
                            tma_load_pair(s2, &tm2, r0, k, 0, to);
                        } else {
                            tma_load_pair(s2, small ? &tm2_small : &tm2, k, r0, 0, to);
                        }
                    }
                });
            }
        } else if (warp == 1) {
            // ---------------------------------------------------------------- MMA
            if (rank == 0) {
                const bool leader = elect_one();
                uint32_t it = 0;
                bool ok = true;
                for_each_tile<FORM>(a, abort_flag, pair, pairs, [&](const Tile &u) {
                    const uint32_t idesc = a.idesc | (static_cast<uint32_t>(width_of(u) >> 3) << 17);
                    for (int kb = 0; kb < u.k_blocks && ok; ++kb, ++it) {
                        const int s = static_cast<int>(it % STAGES);
                        const uint32_t d = it & 1;
                        ok = __all_sync(0xffffffffu, mbar_wait<true>(bar(SUM_EMPTY + d), ((it >> 1) & 1) ^ 1, a,
                                                                     abort_flag, WD_MMA_ACC));
                        if (!ok) return;
                        ok = __all_sync(0xffffffffu, mbar_wait<true>(bar(FULL + s), (it / STAGES) & 1, a, abort_flag,
                                                                     WD_MMA_FULL));
                        if (!ok) return;
                        tc_fence_after();
                        const uint32_t s1 = base + static_cast<uint32_t>(s * STAGE), s2 = s1 + BOX;
                        // The descriptors of both layouts are alike: 8 rows (K-major) or 8
                        // k (MN-major, 128 values each) to the next 8 are 1024 bytes.
                        const uint64_t d1 = sw128_desc(s1), d2 = sw128_desc(s2);
                        // 32 values of k further: 32 bytes along a K-major row, 32 rows of
                        // 128 bytes in an MN-major box.
                        constexpr uint64_t step1 = (FORM == ROWS_T ? 32 : 32 * 128) >> 4;
                        constexpr uint64_t step2 = (FORM == WGRAD ? 32 * 128 : 32) >> 4;
                        if (leader) {
#pragma unroll
                            for (int ks = 0; ks < KB / 32; ++ks)
                                mma8_pair(tmem_base + d * PM, d1 + ks * step1, d2 + ks * step2, idesc, ks > 0);
                            tc_commit2(bar(EMPTY + s));
                            tc_commit2(bar(SUM_FULL + d));
                        }
                        __syncwarp();
                    }
                });
                if (leader) tc_commit2(bar(DRAIN));
                __syncwarp();
                if (lane == 0) {
                    const bool was_aborted = *abort_flag != 0;
                    if (!mbar_wait<true>(bar(DRAIN), 0, a, abort_flag, WD_DRAIN) && was_aborted) {
                        const uint64_t t0 = global_timer();
                        while (!mbar_try_wait<true>(bar(DRAIN), 0) && global_timer() - t0 < a.timeout_ns) {
                        }
                    }
                }
            }
        } else {
            // ------------------------------------------------------------- scales
            // Of several k-blocks at once, so that their latency is met once.
            constexpr int AHEAD = FORM == WGRAD ? 2 : 4;
            uint32_t it = 0;
            bool ok = true;
            for_each_tile<FORM>(a, abort_flag, pair, pairs, [&](const Tile &u) {
                const int rows = u.row_end - u.row0;
                const int64_t n0 = u.n0 + HALF * static_cast<int64_t>(rank);
                const float *sr = a.scale_rows + static_cast<int64_t>(u.k0) * a.ld_rows + u.row0;
                const float *sc = a.scale_cols + (FORM == WGRAD ? static_cast<int64_t>(u.k0) * a.b_cols + n0
                                                                : u.group * a.item_cols + n0 / BLOCK * a.n_cols);
                const bool in_cols = n0 < a.N;
                for (int kb = 0; kb < u.k_blocks && ok; kb += AHEAD) {
                    float r[AHEAD][PM / 32], c[AHEAD][FORM == WGRAD ? HALF / 32 : 1];
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i) {
                        const bool in = kb + i < u.k_blocks;
#pragma unroll
                        for (int j = 0; j < PM / 32; ++j)
                            r[i][j] = in && lane + 32 * j < rows ? __ldg(sr + (kb + i) * a.ld_rows + lane + 32 * j) : 0.0f;
                        if (FORM == WGRAD) {
#pragma unroll
                            for (int j = 0; j < HALF / 32; ++j)
                                c[i][j] = in && n0 + lane + 32 * j < a.N
                                              ? __ldg(sc + (kb + i) * a.b_cols + lane + 32 * j)
                                              : 0.0f;
                        } else {
                            c[i][0] = in && in_cols ? __ldg(sc + (kb + i) * a.b_cols) : 0.0f;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i) {
                        if (kb + i >= u.k_blocks || !ok) break;
                        const int s = static_cast<int>(it % RING);
                        ok = __all_sync(0xffffffffu, mbar_wait(bar(RING_EMPTY + s), ((it / RING) & 1) ^ 1, a,
                                                               abort_flag, WD_PRODUCER));
                        if (!ok) break;
                        const uint32_t to = base + RING0 + static_cast<uint32_t>(s * RING_BYTES);
                        // Row 16 c + 8 g + 2 t + i goes where thread t of a quad reads the
                        // four of c that it needs at once.
#pragma unroll
                        for (int j = 0; j < PM / 32; ++j) {
                            const int row = lane + 32 * j;
                            const int at = (row & ~15) + ((row & 6) << 1) + ((row & 8) >> 2) + (row & 1);
                            st_shared_f32(to + static_cast<uint32_t>(at * 4),
                                          FORM == WGRAD ? r[i][j] : r[i][j] * c[i][0]);
                        }
                        if (FORM == WGRAD) {
#pragma unroll
                            for (int j = 0; j < HALF / 32; ++j)
                                st_shared_f32(to + static_cast<uint32_t>((PM + lane + 32 * j) * 4), c[i][j]);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(RING_FULL + s));
                        ++it;
                    }
                }
            });
        }
    } else {
        // --------------------------------------------------------- sums and stores
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(MANY_REGS));
        const int w = warp - EPI_WARP;
        const int q = w & 3, second = w >> 2;  // quarter of tensor memory's lanes, half of the columns
        const int t = lane & 3, g = lane >> 2;
        const uint32_t out = base + OUT0 + static_cast<uint32_t>(w * OUT_BYTES);
        const uint32_t lanes = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
        uint32_t it = 0;
        bool ok = true;
        for_each_tile<FORM>(a, abort_flag, pair, pairs, [&](const Tile &u) {
            if (!ok) return;
            const int chunks = width_of(u) / 32, col0 = chunks * 16 * second;  // 16 columns each, of this half
            // acc[c][4 i + 2 g + h]: columns 16 c + 8 g + 2 t and the next, lane 16 i + 8 h + (thread / 4).
            uint64_t acc[8][8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[c][i] = 0;
            for (int kb = 0; kb < u.k_blocks; ++kb, ++it) {
                const uint32_t d = it & 1;
                const int s = static_cast<int>(it % RING);
                ok = __all_sync(0xffffffffu,
                                mbar_wait(bar(RING_FULL + s), (it / RING) & 1, a, abort_flag, WD_EPILOGUE));
                if (!ok) return;
                const uint32_t ring = base + RING0 + static_cast<uint32_t>(s * RING_BYTES);
                uint64_t of_lane[4];
                if (FORM == WGRAD) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t v = __float_as_uint(
                            ld_shared_f32(ring + static_cast<uint32_t>((PM + 32 * q + 8 * i + g) * 4)));
                        of_lane[i] = pack2(v, v);
                    }
                }
                ok = __all_sync(0xffffffffu,
                                mbar_wait<true>(bar(SUM_FULL + d), (it >> 1) & 1, a, abort_flag, WD_EPILOGUE));
                if (!ok) return;
                tc_fence_after();
                const uint32_t from = lanes + d * PM + static_cast<uint32_t>(col0);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if (c >= chunks) break;
                    uint32_t p[16];
                    tmem_load_16x16(from + 16 * c, p);
                    tmem_load_16x16(from + 16 * c + (16u << 16), p + 8);
                    uint64_t x0, x1;
                    lds_2x64(ring + static_cast<uint32_t>((col0 + 16 * c + 4 * t) * 4), x0, x1);
                    tmem_wait(p);
                    if (c == chunks - 1) {
                        // The accumulator is out of tensor memory, the scales are read.
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive_at(bar(SUM_EMPTY + d), 0);
                            mbar_arrive(bar(RING_EMPTY + s));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint64_t v = pack2(p[2 * i], p[2 * i + 1]);
                        if (FORM == WGRAD) v = mul2(v, of_lane[2 * (i >> 2) + (i & 1)]);
                        fma2(acc[c][i], v, (i & 2) ? x1 : x0);
                    }
                }
            }
            const int64_t col = u.n0 + HALF * static_cast<int64_t>(rank) + 32 * q;
            const int rows = u.row_end - u.row0 - col0;
            const int64_t item = FORM == WGRAD ? u.group * a.strideC : 0;
            void *c_item = a.out_type == SGEMM_TYPE_F32 ? static_cast<void *>(static_cast<float *>(a.C) + item)
                                                        : static_cast<void *>(static_cast<uint16_t *>(a.C) + item);
            if (col >= a.N) return;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                if (c >= chunks) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint64_t v[4] = {acc[c][2 * h], acc[c][2 * h + 1], acc[c][4 + 2 * h], acc[c][4 + 2 * h + 1]};
                    const int r = 16 * c + 8 * h;
                    write_rows(a, out, lane, v, c_item, u.row0 + col0 + r, rows - r, col);
                }
            }
        });
    }

    // The odd CTA's tensor memory is written by the even CTA's MMAs: wait for
    // them to drain before the pair releases it. After a wait that gave up,
    // loads may still be on their way: leave them time to land.
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) {
        const uint64_t t0 = global_timer();
        while (global_timer() - t0 < 10000000ull) {
        }
    }
    if (rank != 0 && threadIdx.x == 0) {
        if (!mbar_wait<true>(bar(DRAIN), 0, a, abort_flag, WD_DRAIN)) {
            const uint64_t t0 = global_timer();
            while (!mbar_try_wait<true>(bar(DRAIN), 0) && global_timer() - t0 < a.timeout_ns) {
            }
        }
    }
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) {
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS)
                     : "memory");
    }
}

constexpr int kMaxDevices = 64;
std::once_flag g_once[kMaxDevices][3];
cudaError_t g_err[kMaxDevices][3];
int g_clusters[kMaxDevices][3];

template <Form FORM>
int launch_form(const GemmProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    auto kernel = fp8_gemm_kernel<FORM>;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    std::call_once(g_once[dev.device][FORM], [&] {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
        int n = 0;
        if (e == cudaSuccess) {
            cudaLaunchConfig_t q = cfg;
            q.gridDim = dim3(2 * (dev.sm_count / 2));
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &q);
        }
        g_err[dev.device][FORM] = e;
        g_clusters[dev.device][FORM] = n;
    });
    const int clusters = g_clusters[dev.device][FORM];
    int *flag = watchdog_flag_device_ptr();
    if (g_err[dev.device][FORM] != cudaSuccess || clusters < 1 || !flag) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    const CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    alignas(64) CUtensorMap map1{}, map2{}, map3{};
    Args a{};
    a.offsets = p.offsets;
    a.rows = static_cast<int>(p.rows);
    a.experts = static_cast<int>(p.experts);
    a.N = p.N;
    a.C = p.C;
    a.ldc = p.ldc;
    a.strideC = p.strideC;
    a.out_type = p.out_type;
    const int64_t per = p.out_type == SGEMM_TYPE_F32 ? 4 : 8;
    a.vector = reinterpret_cast<uintptr_t>(p.C) % 16 == 0 && p.ldc % per == 0 &&
               (!p.wgrad || p.experts == 1 || p.strideC % per == 0);
    a.scale_rows = p.sA;
    a.scale_cols = p.sB;
    bool ok;
    int64_t row_tiles;
    if (FORM == WGRAD) {
        a.blocks = static_cast<int>(blocks_of(p.rows));
        a.M = p.M;
        a.ld_rows = p.M;
        a.b_cols = p.N;
        row_tiles = (p.M + PM - 1) / PM * p.experts;
        ok = encode_map_typed(&map1, type, 1, p.B, p.rows, p.N, p.ldb, 1, 0, HALF, KB, sw) &&
             encode_map_typed(&map2, type, 1, p.A, p.rows, p.M, p.lda, 1, 0, HALF, KB, sw);
        map3 = map2;  // not read by the kernel
    } else {
        const int64_t strideB = p.experts > 1 ? p.strideB : 0, kb = blocks_of(p.K), nb = blocks_of(p.N);
        a.k_blocks = static_cast<int>(kb);
        a.ld_rows = p.rows;
        a.item_cols = kb * nb;
        a.n_cols = FORM == ROWS_T ? kb : 1;
        a.b_cols = FORM == ROWS_T ? 1 : nb;
        // Every group may end in a part of a tile, and so may the rest.
        row_tiles = (p.rows + PM - 1) / PM + (p.offsets ? p.experts : 0);
        ok = (FORM == ROWS_T ? encode_map_typed(&map1, type, 1, p.B, p.N, p.K, p.ldb, p.experts, strideB, KB, HALF, sw)
                             : encode_map_typed(&map1, type, 1, p.B, p.K, p.N, p.ldb, p.experts, strideB, HALF, KB, sw)) &&
             encode_map_typed(&map2, type, 1, p.A, p.rows, p.K, p.lda, 1, 0, KB, HALF, sw) &&
             encode_map_typed(&map3, type, 1, p.A, p.rows, p.K, p.lda, 1, 0, KB, 32, sw);
    }
    if (!ok) return SGEMM_ERR_LAUNCH;
    if (row_tiles > INT32_MAX / 2) return SGEMM_ERR_UNSUPPORTED;
    a.tiles_n = static_cast<int>((p.N + PN - 1) / PN);
    // Instruction descriptor of kind::f8f6f4: D fp32 (bits 4-5 = 1), first and
    // second operand E4M3 (0) or E5M2 (1) in bits 7-9 and 10-12, bit 15 / 16:
    // first / second MN-major, N >> 3 in bits 17-22 (the kernel's), M >> 4 in
    // bits 24-28.
    const uint32_t t1 = p.type_b == SGEMM_FP8_E5M2, t2 = p.type_a == SGEMM_FP8_E5M2;
    a.idesc = (1u << 4) | (t1 << 7) | (t2 << 10) | (FORM == ROWS_T ? 0u : 1u << 15) | (FORM == WGRAD ? 1u << 16 : 0u) |
              (static_cast<uint32_t>(PN >> 4) << 24);
    a.timeout_ns = static_cast<uint64_t>(watchdog_ms()) * 1000000ull;
    a.watchdog = flag;
    const int64_t units = row_tiles * a.tiles_n;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (units < clusters ? units : clusters)));
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, map1, map2, map3, a) != cudaSuccess) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    ++*launches;
    return SGEMM_OK;
}

}  // namespace

int gemm_launch(const GemmProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    if (dev.device < 0 || dev.device >= kMaxDevices) return SGEMM_ERR_DEVICE;
    if (p.wgrad) return launch_form<WGRAD>(p, dev, stream, launches);
    return p.transB == SGEMM_OP_T ? launch_form<ROWS_T>(p, dev, stream, launches)
                                  : launch_form<ROWS_N>(p, dev, stream, launches);
}

}  // namespace f8
}  // namespace sgemm
