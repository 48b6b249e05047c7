// Products per expert in bf16 and fp16 on SM pairs (tcgen05, cta_group::2):
//
//     rows   C[s] = A[s] op(B[e(s)])                  s in group e
//     wgrad  C[e] = sum over s in group e of A[s]^T B[s]
//
// Bound by the tensor pipe where groups are long, by reading B where they are
// short. Products of two 16-bit values are exact in fp32 and are summed in
// fp32 in tensor memory; a value is rounded once, when C is written. Measured in
// bf16 with 16384 rows, 32 experts, 2048 -> 4096: rows 188 us (1460 TFLOP/s, the
// path from L2 to shared memory; 170 us where groups are even), wgrad 216 us (the
// stores of C on top of it; 198); 64 rows, two for each of 32 experts, 2048 -> 2048:
// 52 us (5.2 TB/s, reading B).
//
// Two CTAs on two SMs of a cluster make one 256 x n tile (n <= 256): each
// stages 128 rows of the first operand and n / 2 of the second per 64-deep
// k-block, and one MMA of 256 x n x 16 issued by the even CTA reads both
// halves. Two accumulators of 256 columns fill tensor memory: the epilogue
// empties one while the tensor core fills the other.
//
// The MMA's width n is the side that costs time by the step (32 here). rows:
// the first operand is op(B) and gives the columns of C, the second A and its
// rows, so a group of 40 rows is charged 64 and not 256; a group's rows are
// spread evenly over its tiles. wgrad: the first operand is A, the second B;
// the groups are the summed direction.
//
// Groups. The bounds are read on the device. Tiles never cross groups; the
// workers (one CTA pair each) take the tiles of the groups in order, round
// robin, each role of a worker walking the group bounds for itself. Rows
// staged past a tile's end belong to the next and change only sums that are
// not written. In wgrad the part of the last k-block that lies past the
// group's end is zeroed in shared memory, in both operands (a NaN of the next
// group times zero would stay), before the MMA may read it.
//
// Layouts. An operand whose summed direction is contiguous in memory (A of
// rows, B of op = T) is staged K-major, otherwise MN-major, both in 128-byte
// swizzled rows as TMA writes them; the MMA takes either, so nothing is
// transposed.
//
// Roles in each CTA (12 warps): warp 0 loads the first operand and warp 11 the
// second (TMA), warp 1 of the even CTA issues the MMAs, warps 2-9 write C (two
// per quarter of tensor memory's lanes), warp 10 zeroes wgrad's tails. The loads
// of both CTAs complete on the even CTA's barriers. Every wait is bounded.
//
// Writing C. wgrad, whose tiles are short (a group's rows) and many: a lane
// holds a row, 32 x 64 chunks go through shared memory and TMA stores, about
// 150 instructions for 2048 values. rows: a lane holds a column of C; eight
// lanes exchange values so that a lane stores 16 bytes of a row, about 200
// instructions for 1024 values, hidden behind the longer sums, and rows past
// the group's end cost nothing. (The same way for wgrad: 365 us in place of 216
// for 16384 rows, 32 experts, 2048 x 4096.) Slices of wgrad's sums, which are
// small, are stored in fp32 row by row.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "experts_common.cuh"
#include "experts_internal.h"
#include "tc_common.cuh"

namespace sgemm {
namespace ex {
namespace {

using namespace tc;

namespace g16 {

constexpr int PM = 256, PN = 256, HM = 128, HN = 128;  // largest tile of a pair, this CTA's share of the operands
constexpr int KB = 64;                                 // k-block: 64 values = 128 bytes
constexpr int ROW_STEP = 32;                           // a tile's width is a multiple of it
constexpr int A_BYTES = HM * KB * 2, B_BYTES = HN * KB * 2, STAGE = A_BYTES + B_BYTES;
constexpr int BOX = 64 * 128;    // bytes of a 64 x 64 MN-major box
constexpr int EPI_WARPS = 8, TAIL_WARP = 2 + EPI_WARPS, LOAD2_WARP = TAIL_WARP + 1, THREADS = (LOAD2_WARP + 1) * 32;
constexpr int CHUNK = 32 * 128;  // 32 rows x 64 columns of C (wgrad)
// Stages of the ring; in wgrad the C chunks (two a warp) take the place of one.
constexpr int STAGES = 6;
constexpr int stages(bool wgrad) { return wgrad ? 5 : 6; }
constexpr int bar0(bool wgrad) { return stages(wgrad) * STAGE + (wgrad ? EPI_WARPS * 2 * CHUNK : 0); }
constexpr int smem_bytes(bool wgrad) { return bar0(wgrad) + 256 + 1024; }
// mbarriers
constexpr int FULL = 0, EMPTY = FULL + STAGES, TAIL = EMPTY + STAGES, ACC_FULL = TAIL + STAGES,
              ACC_EMPTY = ACC_FULL + 2, DRAIN = ACC_EMPTY + 2, NBARS = DRAIN + 1;
static_assert(NBARS * 8 + 24 <= 256, "barrier block");
static_assert(smem_bytes(true) <= 232448 && smem_bytes(false) <= 232448, "shared memory per CTA");
static_assert(STAGE % 1024 == 0, "1024-byte aligned swizzled buffers");

}  // namespace g16

struct Args16 {
    GroupTiles tiles;
    int64_t N;
    void *C;
    int64_t ldc, strideC;
    int c_tma;  // wgrad: C through TMA
    int c_vec;  // rows: C in 16-byte stores
    int slices; // wgrad: C is a slice's sums in fp32
    uint32_t idesc;  // without N
    uint64_t timeout_ns;
    int *watchdog;
};

enum Form { ROWS_N, ROWS_T, WGRAD };

template <Form FORM, class F>
__device__ __forceinline__ void for_each_tile(const Args16 &a, volatile int *abort_flag, int index, int count, F &&f) {
    if (FORM == WGRAD)
        for_each_group_tile<true, g16::PM, g16::PN, g16::KB>(a.tiles, abort_flag, index, count, f);
    else
        for_each_group_tile<false, g16::PN, g16::PM, g16::KB, g16::ROW_STEP>(a.tiles, abort_flag, index, count, f);
}

// The MMA's width: the tile's rows (rows) or columns (wgrad), rounded up.
template <Form FORM>
__device__ __forceinline__ int width_of(const Args16 &a, const GroupTile &u) {
    const int n = FORM == WGRAD ? static_cast<int>(min(static_cast<int64_t>(g16::PN), a.N - u.n0)) : u.row_end - u.row0;
    return (n + g16::ROW_STEP - 1) / g16::ROW_STEP * g16::ROW_STEP;
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

// 64 k of an MN-major operand: one or two boxes of 64 columns.
__device__ __forceinline__ void load_mn(uint32_t dst, const CUtensorMap *map, int x, int k, int item, int boxes,
                                        uint32_t bar) {
    tma_load_pair(dst, map, x, k, item, bar);
    if (boxes > 1) tma_load_pair(dst + g16::BOX, map, x + 64, k, item, bar);
}

__device__ __forceinline__ uint32_t map_to_cta(uint32_t addr, uint32_t cta) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
    return r;
}

// Shared-memory descriptor of an MN-major operand in the 128-byte swizzle:
// boxes of 64 values x 64 k (rows of 128 bytes, one k each). Leading offset:
// from one box of 64 values to the next; stride offset: from 8 k to the next 8.
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(g16::BOX >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ void mma16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// A 32 x 32 block of sums, lane = column, x[j] = row j, as 16-bit rows: v[i]
// becomes columns 8 (lane / 8) .. + 7 of row 8 i + lane % 8. Three exchanges
// between lanes, each pairing columns and halving rows.
template <bool BF16>
__device__ __forceinline__ void gather_rows(const float (&x)[32], int lane, uint32_t (&v)[4][4]) {
    const bool b1 = lane & 2, b2 = lane & 4;
    // Of rows 2 j (low halves) and 2 j + 1 of this lane's and its neighbour's
    // column: even lanes take row 2 j, odd lanes row 2 j + 1.
    const uint32_t halves = lane & 1 ? 0x3276u : 0x5410u;
    uint32_t one[16];  // rows 2 j + lane % 2, two columns
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint32_t own = pack16<BF16>(x[2 * j], x[2 * j + 1]);
        one[j] = __byte_perm(own, __shfl_xor_sync(0xffffffffu, own, 1), halves);
    }
    uint32_t two[8][2];  // rows 4 i + lane % 4, four columns
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t own = b1 ? one[2 * i + 1] : one[2 * i];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, b1 ? one[2 * i] : one[2 * i + 1], 2);
        two[i][0] = b1 ? got : own;
        two[i][1] = b1 ? own : got;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t own = b2 ? two[2 * i + 1][c] : two[2 * i][c];
            const uint32_t got = __shfl_xor_sync(0xffffffffu, b2 ? two[2 * i][c] : two[2 * i + 1][c], 4);
            v[i][c] = b2 ? got : own;
            v[i][2 + c] = b2 ? own : got;
        }
    }
}

template <Form FORM, bool BF16>
__global__ void __launch_bounds__(g16::THREADS, 1)
    grouped16_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmC, const __grid_constant__ Args16 a) {
    // tmA, tmB: the first and second operand. tmC: wgrad: C; rows: the second
    // operand in boxes of 32 rows (tmB: 128).
    constexpr int STAGES = g16::stages(FORM == WGRAD);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem_raw + (base - raw) + g16::bar0(FORM == WGRAD));
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + g16::NBARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + g16::NBARS + 1);
    const uint32_t signal_word = smem_u32(bars + g16::NBARS + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
    auto bar = [&](int i) { return smem_u32(bars + i); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar(g16::FULL + s), 1);
            mbar_init(bar(g16::EMPTY + s), 1);
            mbar_init(bar(g16::TAIL + s), 1);
        }
        for (int d = 0; d < 2; ++d) {
            mbar_init(bar(g16::ACC_FULL + d), 1);
            mbar_init(bar(g16::ACC_EMPTY + d), 2 * g16::EPI_WARPS);
        }
        mbar_init(bar(g16::DRAIN), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmA)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmB)) : "memory");
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

    if (warp == 0 || warp == g16::LOAD2_WARP) {
        // ------------------------------------------------------------------ loads
        const bool first = warp == 0;  // the first operand (and the barriers' bytes), or the second
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for_each_tile<FORM>(a, abort_flag, pair, pairs, [&](const GroupTile &u) {
                const int half = width_of<FORM>(a, u) / 2;
                const int m0 = (FORM == WGRAD ? u.row0 : u.n0) + g16::HM * static_cast<int>(rank);
                const int n0 = (FORM == WGRAD ? u.n0 : u.row0) + half * static_cast<int>(rank);
                // rows: one box of 128 rows (a box costs more time than the rows it
                // reads in vain), of 32 where those are enough.
                const bool small = FORM != WGRAD && half <= 32;
                const int boxes = half > 64 ? 2 : 1;  // wgrad
                const uint32_t bytes =
                    g16::A_BYTES + (FORM == WGRAD ? boxes * g16::BOX : small ? 32 * 128 : g16::B_BYTES);
                for (int kb = 0; kb < u.k_blocks && ok; ++kb, ++it) {
                    const int s = static_cast<int>(it % STAGES);
                    if (!mbar_wait<true>(bar(g16::EMPTY + s), ((it / STAGES) & 1) ^ 1, a, abort_flag, WD_PRODUCER)) {
                        ok = false;
                        return;
                    }
                    const uint32_t sa = base + static_cast<uint32_t>(s * g16::STAGE), sb = sa + g16::A_BYTES;
                    const bool tail = FORM == WGRAD && (kb + 1) * g16::KB > u.k_rows && u.k_rows % 16 != 0;
                    uint32_t to;
                    if (tail) {
                        // Each CTA's own barrier; its tail warp signals the even CTA's.
                        to = map_to_cta(bar(g16::TAIL + s), rank);
                        if (first) mbar_arrive_expect_tx(bar(g16::TAIL + s), bytes);
                    } else {
                        to = map_to_cta(bar(g16::FULL + s), 0);
                        if (first && rank == 0) mbar_arrive_expect_tx(bar(g16::FULL + s), 2 * bytes);
                    }
                    const int k = kb * g16::KB;
                    if (first) {
                        if (FORM == WGRAD)
                            load_mn(sa, &tmA, m0, u.k0 + k, 0, 2, to);
                        else if (FORM == ROWS_T)
                            tma_load_pair(sa, &tmA, k, m0, u.group, to);
                        else
                            load_mn(sa, &tmA, m0, k, u.group, 2, to);
                    } else if (FORM == WGRAD) {
                        load_mn(sb, &tmB, n0, u.k0 + k, 0, boxes, to);
                    } else {
                        tma_load_pair(sb, small ? &tmC : &tmB, k, n0, 0, to);
                    }
                }
            });
        }
    } else if (warp == 1) {
        // -------------------------------------------------------------------- MMA
        if (rank == 0) {
            const bool leader = elect_one();
            uint32_t it = 0, units = 0;
            bool ok = true;
            for_each_tile<FORM>(a, abort_flag, pair, pairs, [&](const GroupTile &u) {
                if (u.k_blocks == 0 || !ok) return;
                const uint32_t d = units & 1;
                ok = __all_sync(0xffffffffu, mbar_wait<true>(bar(g16::ACC_EMPTY + d), ((units >> 1) & 1) ^ 1, a,
                                                             abort_flag, WD_MMA_ACC));
                tc_fence_after();
                const uint32_t dt = tmem_base + d * g16::PN;
                const uint32_t idesc =
                    a.idesc | (static_cast<uint32_t>(width_of<FORM>(a, u) >> 3) << 17);
                for (int kb = 0; kb < u.k_blocks && ok; ++kb, ++it) {
                    const int s = static_cast<int>(it % STAGES);
                    ok = __all_sync(0xffffffffu, mbar_wait<true>(bar(g16::FULL + s), (it / STAGES) & 1, a,
                                                                 abort_flag, WD_MMA_FULL));
                    if (!ok) return;
                    tc_fence_after();
                    const uint32_t sa = base + static_cast<uint32_t>(s * g16::STAGE), sb = sa + g16::A_BYTES;
                    const uint64_t da = FORM == ROWS_T ? sw128_desc(sa) : mn_desc(sa);
                    const uint64_t db = FORM == WGRAD ? mn_desc(sb) : sw128_desc(sb);
                    // 16 values of k further: 32 bytes along a K-major row, 16
                    // rows of 128 bytes in an MN-major box.
                    constexpr uint64_t step_a = (FORM == ROWS_T ? 32 : 16 * 128) >> 4;
                    constexpr uint64_t step_b = (FORM == WGRAD ? 16 * 128 : 32) >> 4;
                    // wgrad: of the last k-block only the 16s that hold rows of the group.
                    const int left = FORM == WGRAD ? u.k_rows - kb * g16::KB : g16::KB;
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < g16::KB / 16; ++ks)
                            if (16 * ks < left)
                                mma16_pair(dt, da + ks * step_a, db + ks * step_b, idesc, kb > 0 || ks > 0);
                        tc_commit2(bar(g16::EMPTY + s));
                    }
                    __syncwarp();
                }
                if (leader && ok) tc_commit2(bar(g16::ACC_FULL + d));
                __syncwarp();
                ++units;
            });
            if (leader) tc_commit2(bar(g16::DRAIN));
            __syncwarp();
            if (lane == 0) {
                const bool was_aborted = *abort_flag != 0;
                if (!mbar_wait<true>(bar(g16::DRAIN), 0, a, abort_flag, WD_DRAIN) && was_aborted) {
                    const uint64_t t0 = global_timer();
                    while (!mbar_try_wait<true>(bar(g16::DRAIN), 0) && global_timer() - t0 < a.timeout_ns) {
                    }
                }
            }
        }
    } else if (warp == g16::TAIL_WARP) {
        // ---------------------------------------------- tails of the summed rows
        if (FORM == WGRAD) {
            uint32_t it = 0, uses = 0;  // bit s: parity of the tails staged in stage s so far
            bool ok = true;
            for_each_tile<FORM>(a, abort_flag, pair, pairs, [&](const GroupTile &u) {
                if (!ok || u.k_blocks == 0) return;
                const int left = u.k_rows % g16::KB;
                it += static_cast<uint32_t>(u.k_blocks);
                if (left % 16 == 0) return;
                const int s = static_cast<int>((it - 1) % STAGES);
                ok = __all_sync(0xffffffffu,
                                mbar_wait(bar(g16::TAIL + s), (uses >> s) & 1, a, abort_flag, WD_PRODUCER));
                if (!ok) return;
                uses ^= 1u << s;
                const uint32_t st = base + static_cast<uint32_t>(s * g16::STAGE);
                // Rows from `left` to the end of its 16 of each of the four boxes,
                // 16 bytes a lane; the MMAs of later 16s are not issued.
                const int vecs = (16 - left % 16) * 8;
#pragma unroll 1
                for (int b = 0; b < 4; ++b)
                    for (int i = lane; i < vecs; i += 32)
                        st_shared_v4(st + static_cast<uint32_t>(b * g16::BOX + left * 128 + i * 16), 0.0f, 0.0f, 0.0f,
                                     0.0f);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0)
                        mbar_arrive_expect_tx(bar(g16::FULL + s), 4);
                    else
                        st_async_signal(signal_word, bar(g16::FULL + s), 0);
                }
                __syncwarp();
            });
        }
    } else {
        // --------------------------------------------------------------- epilogue
        const int q = warp & 3, second = (warp - 2) >> 2;  // quarter of tensor memory's lanes, half of the columns
        const uint32_t stage0 =
            base + static_cast<uint32_t>(STAGES * g16::STAGE + (warp - 2) * 2 * g16::CHUNK);  // wgrad
        uint32_t units = 0, chunks = 0;
        bool ok = true;
        for_each_tile<FORM>(a, abort_flag, pair, pairs, [&](const GroupTile &u) {
            if (!ok) return;
            const bool summed = u.k_blocks > 0;
            const uint32_t d = units & 1;
            if (summed) {
                ok = __all_sync(0xffffffffu, mbar_wait<true>(bar(g16::ACC_FULL + d), (units >> 1) & 1, a, abort_flag,
                                                             WD_EPILOGUE));
                if (!ok) return;
                tc_fence_after();
                ++units;
            }
            const uint32_t dt = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + d * g16::PN;
            auto release = [&] {  // the accumulator is out of tensor memory (this warp's part)
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(bar(g16::ACC_EMPTY + d), 0);
            };
            if (FORM != WGRAD) {
                // Lanes are columns of C, accumulator columns its rows.
                const int col = u.n0 + g16::HM * static_cast<int>(rank) + 32 * q + lane;
                const int rows = u.row_end - u.row0;
                uint16_t *c0 = static_cast<uint16_t *>(a.C) + static_cast<int64_t>(u.row0) * a.ldc;
#pragma unroll 1
                for (int r0 = 32 * second; r0 < rows; r0 += 64) {
                    float x[32];
                    if (summed) {
                        tmem_load32(dt + static_cast<uint32_t>(r0), x);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[j] = 0.0f;
                    }
                    if (a.c_vec) {
                        uint32_t v[4][4];
                        gather_rows<BF16>(x, lane, v);
                        const int c8 = (col & ~31) + (lane >> 3) * 8;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = r0 + 8 * i + (lane & 7);
                            uint16_t *p = c0 + static_cast<int64_t>(row) * a.ldc + c8;
                            if (row >= rows) continue;
                            if (c8 + 8 <= a.N) {
                                *reinterpret_cast<uint4 *>(p) = make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
                            } else {
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                    if (c8 + c < a.N) p[c] = static_cast<uint16_t>(v[i][c >> 1] >> (16 * (c & 1)));
                            }
                        }
                    } else {
                        uint16_t *p = c0 + static_cast<int64_t>(r0) * a.ldc + col;
#pragma unroll
                        for (int j = 0; j < 32; ++j, p += a.ldc)
                            if (r0 + j < rows && col < a.N) *p = static_cast<uint16_t>(pack16<BF16>(x[j], 0.0f));
                    }
                }
                if (summed) release();
                return;
            }
            const int row0 = u.row0 + g16::HM * static_cast<int>(rank) + 32 * q;
            const int rows = min(32, u.row_end - row0);  // may be negative
#pragma unroll 1
            for (int ch = 2 * second; ch < 2 * second + 2; ++ch) {
                const int col0 = u.n0 + 64 * ch;
                const bool wanted = rows > 0 && col0 < a.N;  // uniform over the warp
                if (a.slices) {
                    float *c = static_cast<float *>(a.C) + u.group * a.strideC +
                               static_cast<int64_t>(row0 + lane) * a.ldc + col0;
#pragma unroll 1
                    for (int h = 0; h < 64 && wanted; h += 32) {
                        float x[32] = {};
                        if (summed) tmem_load32(dt + static_cast<uint32_t>(64 * ch + h), x);
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            if (lane < rows && col0 + h + j < a.ldc)
                                *reinterpret_cast<float4 *>(c + h + j) =
                                    make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                        __syncwarp();
                    }
                    if (summed && ch == 2 * second + 1) release();
                    continue;
                }
                uint32_t v[32];
                if (summed && wanted) {
                    float x[32];
                    tmem_load32(dt + static_cast<uint32_t>(64 * ch), x);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = pack16<BF16>(x[2 * j], x[2 * j + 1]);
                    tmem_load32(dt + static_cast<uint32_t>(64 * ch + 32), x);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[16 + j] = pack16<BF16>(x[2 * j], x[2 * j + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0;
                }
                if (summed && ch == 2 * second + 1) release();
                if (!wanted) continue;
                const uint32_t buf = stage0 + (chunks & 1) * g16::CHUNK;
                ++chunks;
                // The store that read this buffer two chunks ago is done reading.
                if (lane == 0) bulk_wait_read<1>();
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    st_shared_v4(buf + sw128_offset(lane, j), __uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                 __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
                if (a.c_tma && rows == 32) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) tma_store_3d(&tmC, col0, row0, u.group, buf);
                } else {
                    // Row by row, the lanes along the row.
                    __syncwarp();
                    uint16_t *c = static_cast<uint16_t *>(a.C) + u.group * a.strideC +
                                  static_cast<int64_t>(row0) * a.ldc + col0;
                    const int cols = static_cast<int>(min(static_cast<int64_t>(64), a.N - col0));
                    for (int r = 0; r < rows; ++r, c += a.ldc) {
                        const uint32_t w = __float_as_uint(ld_shared_f32(buf + sw128_offset(r, lane >> 2) +
                                                                         static_cast<uint32_t>((lane & 3) * 4)));
                        if (2 * lane < cols) c[2 * lane] = static_cast<uint16_t>(w);
                        if (2 * lane + 1 < cols) c[2 * lane + 1] = static_cast<uint16_t>(w >> 16);
                    }
                    __syncwarp();
                }
                if (lane == 0) bulk_commit();  // one group per chunk, empty or not
            }
        });
        if (lane == 0) bulk_wait<0>();
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
        if (!mbar_wait<true>(bar(g16::DRAIN), 0, a, abort_flag, WD_DRAIN)) {
            const uint64_t t0 = global_timer();
            while (!mbar_try_wait<true>(bar(g16::DRAIN), 0) && global_timer() - t0 < a.timeout_ns) {
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
std::once_flag g_once[kMaxDevices][6];
cudaError_t g_err[kMaxDevices][6];
int g_clusters[kMaxDevices][6];

// Whether a tensor map can describe `items` matrices of rows x ld 16-bit
// values, `stride` apart.
bool mappable(const void *p, int64_t rows, int64_t ld, int64_t items, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0 &&
           (items == 1 || (stride % 8 == 0 && stride >= rows * ld));
}

template <Form FORM, bool BF16>
int launch16(const GroupedProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    auto kernel = grouped16_kernel<FORM, BF16>;
    constexpr int idx = FORM + (BF16 ? 3 : 0);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(g16::THREADS);
    cfg.dynamicSmemBytes = g16::smem_bytes(FORM == WGRAD);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    std::call_once(g_once[dev.device][idx], [&] {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             g16::smem_bytes(FORM == WGRAD));
        int n = 0;
        if (e == cudaSuccess) {
            cudaLaunchConfig_t q = cfg;
            q.gridDim = dim3(2 * (dev.sm_count / 2));
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &q);
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
    const CUtensorMapDataType type =
        BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    alignas(64) CUtensorMap mapA{}, mapB{}, mapC{};
    const int64_t strideB = p.experts > 1 ? p.strideB : 0, strideC = p.experts > 1 ? p.strideC : 0;
    bool ok, c_tma = false;
    if (FORM == WGRAD) {
        ok = encode_map_typed(&mapA, type, 2, p.A, p.rows, p.M, p.lda, 1, 0, 64, g16::KB, sw) &&
             encode_map_typed(&mapB, type, 2, p.B, p.rows, p.N, p.ldb, 1, 0, 64, g16::KB, sw);
        c_tma = p.split == 1 && mappable(p.C, p.M, p.ldc, p.experts, p.strideC) &&
                encode_map_typed(&mapC, type, 2, p.C, p.M, p.N, p.ldc, p.experts, strideC, 64, 32, sw);
        if (!c_tma) mapC = mapA;  // not read by the kernel
    } else {
        ok = (FORM == ROWS_T
                  ? encode_map_typed(&mapA, type, 2, p.B, p.N, p.K, p.ldb, p.experts, strideB, g16::KB, g16::HM, sw)
                  : encode_map_typed(&mapA, type, 2, p.B, p.K, p.N, p.ldb, p.experts, strideB, 64, g16::KB, sw)) &&
             encode_map_typed(&mapB, type, 2, p.A, p.rows, p.K, p.lda, 1, 0, g16::KB, g16::HN, sw) &&
             encode_map_typed(&mapC, type, 2, p.A, p.rows, p.K, p.lda, 1, 0, g16::KB, 32, sw);
    }
    if (!ok) return SGEMM_ERR_LAUNCH;

    Args16 a{};
    a.N = p.N;
    a.C = p.C;
    a.ldc = p.ldc;
    a.strideC = p.strideC;
    const int64_t tiles_n = (p.N + g16::PN - 1) / g16::PN;
    const int64_t tiles_m = FORM == WGRAD ? (p.M + g16::PM - 1) / g16::PM : 1;
    if (tiles_n * tiles_m > INT32_MAX / 2) return SGEMM_ERR_UNSUPPORTED;
    a.tiles = GroupTiles{p.offsets,
                         static_cast<int>(p.rows),
                         static_cast<int>(p.experts),
                         p.wgrad ? p.M : 0,
                         p.K,
                         static_cast<int>(tiles_m),
                         static_cast<int>(tiles_n),
                         p.split};
    a.slices = p.split > 1 ? 1 : 0;
    a.c_tma = c_tma ? 1 : 0;
    a.c_vec = reinterpret_cast<uintptr_t>(p.C) % 16 == 0 && p.ldc % 8 == 0;
    // Instruction descriptor of kind::f16: D fp32 (bits 4-5 = 1), A and B
    // fp16 (0) or bf16 (1) in bits 7-9 and 10-12, bit 15 / 16: A / B MN-major,
    // N >> 3 in bits 17-22 (the kernel's), M >> 4 in bits 24-28.
    const uint32_t t = BF16 ? 1u : 0u;
    a.idesc = (1u << 4) | (t << 7) | (t << 10) | (FORM == ROWS_T ? 0u : 1u << 15) | (FORM == WGRAD ? 1u << 16 : 0u) |
              (static_cast<uint32_t>(g16::PM >> 4) << 24);
    a.timeout_ns = static_cast<uint64_t>(watchdog_ms()) * 1000000ull;
    a.watchdog = flag;
    // Every group may end in a part of a tile, and so may the rest.
    const int64_t units = FORM == WGRAD ? tiles_m * tiles_n * p.experts * p.split
                                        : ((p.rows + g16::PN - 1) / g16::PN + p.experts) * tiles_n;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (units < clusters ? units : clusters)));
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, mapA, mapB, mapC, a) != cudaSuccess) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    ++*launches;
    return SGEMM_OK;
}

bool a_mappable(const GroupedProblem &p) { return mappable(p.A, p.rows, p.lda, 1, 0); }

int64_t b_rows(const GroupedProblem &p) { return p.wgrad ? p.rows : p.transB == SGEMM_OP_T ? p.N : p.K; }
int64_t b_cols(const GroupedProblem &p) { return p.wgrad ? p.N : p.transB == SGEMM_OP_T ? p.K : p.N; }

bool b_mappable(const GroupedProblem &p) {
    return p.wgrad ? mappable(p.B, p.rows, p.ldb, 1, 0) : mappable(p.B, b_rows(p), p.ldb, p.experts, p.strideB);
}

// Copies of operands whose rows are not 16-byte aligned, in rows of a multiple
// of 8 values. Lanes along a row; a block takes whole rows in turn.
struct CopyRows {
    const uint16_t *src;
    uint16_t *dst;
    int64_t rows, cols, ld_src, ld_dst, items, stride_src;
};

__global__ void __launch_bounds__(256) copy_rows_kernel(const CopyRows j) {
    const int64_t total = j.rows * j.items;
    const int lane = static_cast<int>(threadIdx.x & 31);
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); r < total;
         r += static_cast<int64_t>(gridDim.x) * 8) {
        const int64_t item = r / j.rows, row = r - item * j.rows;
        const uint16_t *s = j.src + item * j.stride_src + row * j.ld_src;
        uint16_t *d = j.dst + r * j.ld_dst;
        for (int64_t c0 = lane; c0 < j.cols; c0 += 32 * 8) {
            uint16_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = c0 + 32 * i < j.cols ? __ldg(s + c0 + 32 * i) : uint16_t(0);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c0 + 32 * i < j.cols) d[c0 + 32 * i] = v[i];
        }
    }
}

// Bytes of the copies that p needs.
size_t copy_bytes(const GroupedProblem &p) {
    int64_t n = 0;
    if (!a_mappable(p)) n += p.rows * (((p.wgrad ? p.M : p.K) + 7) / 8 * 8);
    if (!b_mappable(p)) n += b_rows(p) * ((b_cols(p) + 7) / 8 * 8) * (p.wgrad ? 1 : p.experts);
    return static_cast<size_t>(n) * 2 + 512;
}

// Enqueues the copies into `scratch` and describes the copied operands in *q.
int copy_operands(const GroupedProblem &p, uint16_t *scratch, const DeviceInfo &dev, cudaStream_t stream,
                  GroupedProblem *q, int *launches) {
    *q = p;
    uint16_t *next = scratch;
    auto copy = [&](const CopyRows &j) {
        const int64_t blocks = (j.rows * j.items + 7) / 8, most = 8LL * dev.sm_count;
        copy_rows_kernel<<<static_cast<unsigned>(blocks < most ? blocks : most), 256, 0, stream>>>(j);
        if (cudaGetLastError() != cudaSuccess) return false;
        ++*launches;
        return true;
    };
    if (!a_mappable(p)) {
        const int64_t cols = p.wgrad ? p.M : p.K, ld = (cols + 7) / 8 * 8;
        if (!copy(CopyRows{static_cast<const uint16_t *>(p.A), next, p.rows, cols, p.lda, ld, 1, 0}))
            return SGEMM_ERR_LAUNCH;
        q->A = next;
        q->lda = ld;
        next += (p.rows * ld + 127) / 128 * 128;
    }
    if (!b_mappable(p)) {
        const int64_t rows = b_rows(p), cols = b_cols(p), ld = (cols + 7) / 8 * 8, items = p.wgrad ? 1 : p.experts;
        if (!copy(CopyRows{static_cast<const uint16_t *>(p.B), next, rows, cols, p.ldb, ld, items, p.strideB}))
            return SGEMM_ERR_LAUNCH;
        q->B = next;
        q->ldb = ld;
        q->strideB = rows * ld;
    }
    return SGEMM_OK;
}

template <bool BF16>
int launch_form(const GroupedProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    if (p.wgrad) return launch16<WGRAD, BF16>(p, dev, stream, launches);
    return p.transB == SGEMM_OP_T ? launch16<ROWS_T, BF16>(p, dev, stream, launches)
                                  : launch16<ROWS_N, BF16>(p, dev, stream, launches);
}

int launch_any(const GroupedProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    return p.type == SGEMM_TYPE_BF16 ? launch_form<true>(p, dev, stream, launches)
                                     : launch_form<false>(p, dev, stream, launches);
}

}  // namespace

// Sizes that fit tensor map coordinates, and a sum to make. Operands whose rows
// are not 16-byte aligned are copied first where that is estimated to take
// less time than the CUDA-core kernel, which copies nothing: that one makes
// about 25 TFLOP/s and no k-step of 16 in less than 0.6 us; the copies move
// about 5 TB/s, and launches and a short product take 20 us.
bool grouped16_supports(const GroupedProblem &p) {
    const int64_t lim = INT32_MAX / 2;
    if (p.type == SGEMM_TYPE_F32 || p.rows <= 0 || (!p.wgrad && p.K <= 0) || p.rows >= lim || p.M >= lim ||
        p.N >= lim || p.K >= lim)
        return false;
    if (a_mappable(p) && b_mappable(p)) return true;
    const double s = static_cast<double>(p.rows), m = static_cast<double>(p.wgrad ? p.M : p.K),
                 n = static_cast<double>(p.N);
    const double depth = p.wgrad ? s / static_cast<double>(p.experts) : m;
    const double cores = 2.0 * s * m * n / 25e6, steps = depth / 16 * 0.6;
    return 2.0 * static_cast<double>(copy_bytes(p)) / 5e6 + 20.0 < (cores > steps ? cores : steps);
}

int grouped16_launch(const GroupedProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    if (dev.device < 0 || dev.device >= kMaxDevices) return SGEMM_ERR_DEVICE;
    if (a_mappable(p) && b_mappable(p)) return launch_any(p, dev, stream, launches);
    float *scratch = scratch_alloc(dev, copy_bytes(p), stream);
    if (!scratch) return SGEMM_ERR_UNSUPPORTED;
    GroupedProblem q;
    int rc = copy_operands(p, reinterpret_cast<uint16_t *>(scratch), dev, stream, &q, launches);
    if (rc == SGEMM_OK) rc = launch_any(q, dev, stream, launches);
    scratch_free(scratch, stream);
    return rc;
}

}  // namespace ex
}  // namespace sgemm
