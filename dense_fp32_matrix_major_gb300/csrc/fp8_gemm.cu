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
// Two CTAs on two SMs of a cluster make a tile of 256 rows by up to 256 columns
// of C. The MMA's first operand gives C's rows (A, 128 of them staged by each
// CTA: the lanes of tensor memory), its second C's columns (B, half of them
// staged by each CTA). Four buffers of 128 columns fill tensor memory, two for
// each half of the tile: four warps empty a half's sums while the tensor core
// makes the other's. (Two buffers of 256 columns, emptied by all eight warps at
// once: 276 us in place of 260 for 16384 x 4096 x 4096, whose rate is 2110
// TFLOP/s.)
//
// What bounds it. The sums that leave tensor memory: a CTA's 128 x 256 of them a
// block of 128 are 1 load, 1 multiply-add and the waits for each, 8 warps' work
// for as long as the MMAs take. Without the MMAs the same kernel takes 206 us,
// without the sums 145, without both TMA and sums 127. A k-block's MMAs take 512 cycles, in
// which shared memory takes in 32 KB from TMA and gives 32 KB to the MMA, all it
// can. So nothing else may go through shared memory while blocks are summed: in
// rows a lane needs one factor a block, its row's scale times the scale of the
// 128 columns that the warp sums, and gets it from global memory two blocks
// ahead. (With C's columns as the lanes, which charges short groups less, every
// thread needs a factor for each of its 32 columns: 319 us.) In wgrad both
// factors vary; the columns' come through a ring in shared memory that warp 2
// fills, in the order in which the threads read them, and loads of 16 lanes x 4
// columns (16x128b) leave a thread a quarter of the columns (4096 x 2048 over
// 8192 rows: 115 us). Tried without gain: 16 warps for the sums 276 us, one SM a
// tile 274, multiply-adds in pairs 265.
//
// Layouts. An operand whose summed direction is contiguous in memory is staged
// K-major, otherwise MN-major, both in 128-byte swizzled rows as TMA writes
// them; the MMA takes either, so nothing is transposed.
//
// Groups. The bounds are read on the device. Tiles never cross groups; the
// workers (one CTA pair each) take the tiles of the groups in order, round
// robin, each role of a worker walking the bounds for itself. Rows staged past a
// tile's end belong to the next and change only sums that are not written; a CTA
// whose rows all lie past it stages none. In wgrad every group's rows start in a
// block of their own and end in zeros. 16384 rows in 32 even groups, 2048 -> 4096:
// 152 us; ragged 184: a group's last tile costs as much as a full one.
//
// C leaves through shared memory and TMA stores, 32 rows of 128 bytes at a time,
// while the next tile is summed; where TMA cannot address it or a warp has fewer
// than 32 rows, by 16-byte or single stores (all tiles that way: 276 us).
//
// A matrix and a few rows: fp8_few.cu.
//
// Roles in each CTA (12 warps): warp 0 loads the first operand and warp 3 the
// second (TMA), warp 1 of the even CTA issues the MMAs, warp 2 prepares wgrad's
// scales, warps 4 to 11 sum and write C (two per quarter of tensor memory's
// lanes, half of the columns each). They hold 128 sums a thread and take
// registers that the first four give up. The loads of both CTAs complete on the
// even CTA's barriers. Every wait is bounded.
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
constexpr int FEW = 32;                        // rows of the small box of A
constexpr int BOX = 128 * 128;                 // bytes of a staged operand
constexpr int STAGE = 2 * BOX, STAGES = 4;
constexpr int EPI_WARPS = 8, EPI_WARP = 4, THREADS = (EPI_WARP + EPI_WARPS) * 32;
constexpr int RING = 8;                        // k-blocks of wgrad's prepared scales
constexpr int RING_BYTES = PN * 4;
// C on its way out: two chunks a warp of 32 rows by 128 bytes, as TMA takes them; or,
// where it cannot, rows of 64 bytes (rows) or 8 rows of 32 fp32 values (wgrad),
// padded so that every phase of the accesses meets all banks.
constexpr int OUT_CHUNK = 32 * 128, OUT_ROW = 80, OUT_WGRAD = 144, OUT_BYTES = 2 * OUT_CHUNK;
constexpr int OUT0 = STAGES * STAGE, RING0 = OUT0 + EPI_WARPS * OUT_BYTES, BAR0 = RING0 + RING * RING_BYTES;
// mbarriers
constexpr int FULL = 0, EMPTY = FULL + STAGES, SUM_FULL = EMPTY + STAGES, SUM_EMPTY = SUM_FULL + 4,
              RING_FULL = SUM_EMPTY + 4, RING_EMPTY = RING_FULL + RING, DRAIN = RING_EMPTY + RING, NBARS = DRAIN + 1;
constexpr int SMEM_BYTES = BAR0 + 512 + 1024;
static_assert(NBARS * 8 + 16 <= 512, "barrier block");
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
static_assert(8 * OUT_WGRAD <= OUT_CHUNK && 32 * OUT_ROW <= OUT_CHUNK, "staging of C");
static_assert(OUT0 % 1024 == 0 && RING_BYTES % 16 == 0 && BAR0 % 8 == 0, "alignment");
// Registers a thread of the four and of the eight warps, out of 168 each.
constexpr int FEW_REGS = 88, MANY_REGS = 208;
static_assert(4 * FEW_REGS + 8 * MANY_REGS <= 12 * 168, "registers of the launch");

enum Form { ROWS_N, ROWS_T, WGRAD };

struct Args {
    const int32_t *offsets;  // NULL: one group
    int rows, experts;
    int split;         // wgrad: slices of a group's rows, whole blocks but the last; the "groups" are then slices
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
    int out_type, vector, tma;  // C in 16-byte stores; through TMA
    uint32_t idesc;        // without N
    uint64_t timeout_ns;
    int *watchdog;
};

// A tile: rows row0 .. row_end of C (rows: of all, wgrad: of the group's matrix),
// columns from n0 on, k_blocks blocks from block k0 on.
struct Tile {
    int group, row0, row_end, n0, k0, k_blocks;
};

__device__ __forceinline__ int group_of_rows(const Args &a, int e) {
    return a.offsets ? ex::group_start(a.offsets, e, a.rows) : (e == 0 ? 0 : a.rows);
}

template <Form FORM>
__device__ __forceinline__ int start_of(const Args &a, int e) {
    if (FORM != WGRAD || a.split == 1) return group_of_rows(a, e);
    const int g = e / a.split, s = e - g * a.split, begin = group_of_rows(a, g);
    if (s == 0) return begin;
    const int end = max(begin, group_of_rows(a, g + 1));
    const int slice = ((end - begin + KB - 1) / KB + a.split - 1) / a.split * KB;
    return begin + min(s * slice, end - begin);
}

template <Form FORM, class F>
__device__ __forceinline__ void for_each_tile(const Args &a, volatile int *abort_flag, int index, int count, F &&f) {
    int e = 0, begin = 0, base = 0, first = 0;  // base: tiles (rows: of rows) before group e; first: blocks
    int next = start_of<FORM>(a, 1), end = max(begin, next);
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
            next = e < a.experts ? start_of<FORM>(a, e + 1) : a.rows;
            end = max(begin, next);
            if (FORM != WGRAD) tiles = (end - begin + PM - 1) / PM;
        }
        const int n0 = static_cast<int>(u % a.tiles_n) * PN;
        if (FORM == WGRAD) {
            const int row0 = (rt - base) * PM;
            const int b0 = min(first, a.blocks), b1 = min(first + (end - begin + KB - 1) / KB, a.blocks);
            f(Tile{e, row0, static_cast<int>(min(static_cast<int64_t>(row0 + PM), a.M)), n0, b0, b1 - b0});
        } else {
            const int row0 = begin + (rt - base) * PM;
            f(Tile{e, row0, min(row0 + PM, end), n0, 0, e < a.experts ? a.k_blocks : 0});
        }
    }
}

// Columns of B that a CTA stages for each half of the tile: a quarter of 256 or of
// 128. Half h of the tile is columns [h * quarter, (h + 1) * quarter) of what the
// even CTA stages, then of what the odd one does: accumulator column j < quarter
// is column h * quarter + j of the tile, column quarter + j column (2 + h) *
// quarter + j.
__device__ __forceinline__ int quarter_of(const Args &a, const Tile &u) { return a.N - u.n0 > PN / 2 ? PN / 4 : PN / 8; }

// Rows of A that CTA `rank` stages in a k-block: as many as a box has, or none.
__device__ __forceinline__ int box_rows(const Tile &u, uint32_t rank) {
    const int n = u.row_end - u.row0 - HALF * static_cast<int>(rank);
    return n <= 0 ? 0 : (n <= FEW ? FEW : HALF);
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

// 32 lanes x 32 columns of 32 bits from tensor memory, waited for: r[i] is this
// lane's column i.
__device__ __forceinline__ void tmem_load_32x32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// The same 32 x 32 values by four lanes and a quarter of the columns a thread:
// r[16 l + 2 i + h] is lane 16 l + 8 h + (thread / 4), column 4 i + thread % 4.
__device__ __forceinline__ void tmem_load_2x16x32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x128b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n"
        "tcgen05.ld.sync.aligned.16x128b.x8.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
        "[%33];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr), "r"(taddr + (16u << 16))
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

// Arrives on the mbarrier at this offset in the even CTA. Relaxed: what went
// before is reads of tensor memory, complete when their wait returned. (With
// release semantics at cluster scope an earlier form took 578 us in place of 354 for
// 16384 x 4096 x 4096: the arrival waits out the thread's memory operations.)
__device__ __forceinline__ void arrive_even(uint32_t bar) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(bar), "r"(0));
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}

__device__ __forceinline__ uint4 lds_128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t round2(float lo, float hi, bool bf16) {
    if (bf16) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&r);
    }
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ void sts_128(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// 16 bytes of a row of C at p, the first of its PER values being column col.
template <class T, int PER>
__device__ __forceinline__ void store16(const Args &a, T *p, int64_t col, const uint4 &x) {
    if (a.vector && col + PER <= a.N) {
        *reinterpret_cast<uint4 *>(p) = x;
    } else {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (col + j < a.N) p[j] = static_cast<T>(PER == 4 ? w[j] : w[j >> 1] >> (16 * (j & 1)));
    }
}

// Rows of 64 bytes of C, this lane's first: staged in shared memory and written
// eight rows at a time.
template <class T>
__device__ __forceinline__ void write_lanes(const Args &a, uint32_t out, int lane, const uint32_t (&v)[16], T *c,
                                            int64_t row, int rows, int64_t col) {
    constexpr int PER = 16 / sizeof(T);
    __syncwarp();  // what the buffer held is read
#pragma unroll
    for (int j = 0; j < 4; ++j)
        sts_128(out + static_cast<uint32_t>(lane * OUT_ROW + 16 * j), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    __syncwarp();
    const int64_t at = col + PER * (lane & 3);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = 8 * j + (lane >> 2);
        const uint4 x = lds_128(out + static_cast<uint32_t>(r * OUT_ROW + 16 * (lane & 3)));
        if (r < rows) store16<T, PER>(a, c + (row + r) * a.ldc + at, at, x);
    }
}

template <Form FORM>
__global__ void __launch_bounds__(THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tm1, const __grid_constant__ CUtensorMap tm1_few,
                    const __grid_constant__ CUtensorMap tm2, const __grid_constant__ CUtensorMap tm_out,
                    const __grid_constant__ Args a) {
    // tm1, tm2: A and B; tm1_few: A in boxes of 32 rows (rows); tm_out: C in boxes of 32 rows by 128 bytes.
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
        for (int d = 0; d < 4; ++d) {
            mbar_init(bar(SUM_FULL + d), 1);
            mbar_init(bar(SUM_EMPTY + d), EPI_WARPS);
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
                    const int n0 = u.n0 + 2 * quarter_of(a, u) * static_cast<int>(rank);
                    const int r0 = u.row0 + HALF * static_cast<int>(rank);
                    const int own = FORM == WGRAD ? HALF : box_rows(u, rank);
                    const uint32_t bytes =
                        2 * BOX + (FORM == WGRAD ? 2 * BOX : 128 * (box_rows(u, 0) + box_rows(u, 1)));
                    for (int kb = 0; kb < u.k_blocks && ok; ++kb, ++it) {
                        const int s = static_cast<int>(it % STAGES);
                        if (!mbar_wait(bar(EMPTY + s), ((it / STAGES) & 1) ^ 1, a, abort_flag, WD_PRODUCER)) {
                            ok = false;
                            return;
                        }
                        const uint32_t s1 = base + static_cast<uint32_t>(s * STAGE), s2 = s1 + BOX;
                        const uint32_t to = map_to_cta(bar(FULL + s), 0);
                        const int k = (u.k0 + kb) * KB;
                        if (first) {
                            if (rank == 0) mbar_arrive_expect_tx(bar(FULL + s), bytes);
                            if (FORM == WGRAD)
                                tma_load_pair(s1, &tm1, r0, k, 0, to);
                            else if (own > 0)
                                tma_load_pair(s1, own == FEW ? &tm1_few : &tm1, k, r0, 0, to);
                        } else if (FORM == WGRAD) {
                            tma_load_pair(s2, &tm2, n0, k, 0, to);
                        } else if (FORM == ROWS_T) {
                            tma_load_pair(s2, &tm2, k, n0, u.group, to);
                        } else {
                            tma_load_pair(s2, &tm2, n0, k, u.group, to);
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
                    const int quarter = quarter_of(a, u);
                    const uint32_t idesc = a.idesc | (static_cast<uint32_t>(2 * quarter >> 3) << 17);
                    // The second half's columns: rows of 128 bytes each, or one byte.
                    const uint32_t next_half = static_cast<uint32_t>(quarter * (FORM == ROWS_T ? 128 : 1)) >> 4;
                    // 32 values of k further: 32 bytes along a K-major row, 32 rows of 128
                    // bytes in an MN-major box.
                    constexpr uint32_t step1 = (FORM == WGRAD ? 32 * 128 : 32) >> 4;
                    constexpr uint32_t step2 = (FORM == ROWS_T ? 32 : 32 * 128) >> 4;
                    for (int kb = 0; kb < u.k_blocks && ok; ++kb, ++it) {
                        const int s = static_cast<int>(it % STAGES);
                        const uint32_t s1 = base + static_cast<uint32_t>(s * STAGE), s2 = s1 + BOX;
                        // The descriptors of both layouts are alike: 8 rows (K-major) or 8
                        // k (MN-major, 128 values each) to the next 8 are 1024 bytes.
                        const uint64_t d1 = sw128_desc(s1), d2 = sw128_desc(s2);
                        ok = __all_sync(0xffffffffu,
                                        mbar_wait(bar(FULL + s), (it / STAGES) & 1, a, abort_flag, WD_MMA_FULL));
                        if (!ok) return;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t d = 2 * (it & 1) + h;
                            ok = __all_sync(0xffffffffu, mbar_wait(bar(SUM_EMPTY + d), ((it >> 1) & 1) ^ 1, a,
                                                                   abort_flag, WD_MMA_ACC));
                            if (!ok) return;
                            tc_fence_after();
                            if (leader) {
#pragma unroll
                                for (int ks = 0; ks < KB / 32; ++ks)
                                    mma8_pair(tmem_base + d * (PN / 2), d1 + ks * step1,
                                              d2 + h * next_half + ks * step2, idesc, ks > 0);
                                tc_commit2(bar(SUM_FULL + d));
                                if (h == 1) tc_commit2(bar(EMPTY + s));
                            }
                            __syncwarp();
                        }
                    }
                });
                if (leader) tc_commit2(bar(DRAIN));
                __syncwarp();
                if (lane == 0) {
                    const bool was_aborted = *abort_flag != 0;
                    if (!mbar_wait(bar(DRAIN), 0, a, abort_flag, WD_DRAIN) && was_aborted) {
                        const uint64_t t0 = global_timer();
                        while (!mbar_try_wait(bar(DRAIN), 0) && global_timer() - t0 < a.timeout_ns) {
                        }
                    }
                }
            }
        } else if (FORM == WGRAD) {
            // ------------------------------------------------- scales of C's columns
            // Of several k-blocks at once, so that their latency is met once.
            constexpr int AHEAD = 4;
            uint32_t it = 0;
            bool ok = true;
            for_each_tile<FORM>(a, abort_flag, pair, pairs, [&](const Tile &u) {
                const float *from = a.scale_cols + static_cast<int64_t>(u.k0) * a.b_cols + u.n0 + lane;
                const int cols = static_cast<int>(min(static_cast<int64_t>(PN), a.N - u.n0)) - lane;
                const int quarter = quarter_of(a, u);
                // In each half, accumulator column 16 c + 4 i + t goes where thread t of a
                // quad reads its four of c. Quarters are multiples of 32 columns.
                const int at = (lane & ~15) + ((lane & 3) << 2) + ((lane >> 2) & 3);
                for (int kb = 0; kb < u.k_blocks && ok; kb += AHEAD) {
                    float v[AHEAD][PN / 32];
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
                        for (int j = 0; j < PN / 32; ++j)
                            v[i][j] = kb + i < u.k_blocks && 32 * j < cols ? __ldg(from + (kb + i) * a.b_cols + 32 * j) : 0.0f;
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i) {
                        if (kb + i >= u.k_blocks || !ok) break;
                        const int s = static_cast<int>(it % RING);
                        ok = __all_sync(0xffffffffu, mbar_wait(bar(RING_EMPTY + s), ((it / RING) & 1) ^ 1, a,
                                                               abort_flag, WD_PRODUCER));
                        if (!ok) break;
                        const uint32_t to = base + RING0 + static_cast<uint32_t>(s * RING_BYTES + at * 4);
#pragma unroll
                        for (int j = 0; j < PN / 32; ++j) {
                            const int part = 32 * j / quarter;
                            if (part < 4)
                                st_shared_f32(to + static_cast<uint32_t>((part & 1) * (PN / 2) + (part >> 1) * quarter +
                                                                         32 * j - part * quarter) * 4, v[i][j]);
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
        const uint32_t sums = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(PN / 2 * second);
        uint32_t it = 0;
        bool ok = true;
        // The accumulator is out of tensor memory (this warp's part).
        auto release = [&](uint32_t d) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_even(bar(SUM_EMPTY + d));
        };
        // Sends a chunk to C once fill(address) has written it; two are on their way at most.
        uint32_t sent = 0;
        auto send = [&](int64_t col, int row, int item, auto &&fill) {
            const uint32_t to = out + (sent & 1) * OUT_CHUNK;
            ++sent;
            if (lane == 0) bulk_wait_read<1>();
            __syncwarp();
            fill(to);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_3d(&tm_out, static_cast<int>(col), row, item, to);
                bulk_commit();
            }
        };
        // Before a chunk's memory is used for other staging.
        auto settle = [&] {
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
        };
        for_each_tile<FORM>(a, abort_flag, pair, pairs, [&](const Tile &u) {
            if (!ok) return;
            const int row0 = u.row0 + HALF * static_cast<int>(rank) + 32 * q;
            const int rows = u.row_end - row0;  // may be negative
            const int quarter = quarter_of(a, u), chunks = quarter / 16;
            // Column of C that chunk c, 32 accumulator columns of this warp's half, starts at.
            auto column = [&](int c) {
                return u.n0 + (32 * c < quarter ? second * quarter : (1 + second) * quarter) + 32 * static_cast<int64_t>(c);
            };
            if constexpr (FORM != WGRAD) {
                // acc[c][i]: column 32 c + i of this lane's row.
                float acc[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i) acc[c][i] = 0.0f;
                // Factors two blocks ahead: of the lane's row, and of B's blocks of the
                // half's two parts, which lie in the tile's first and second 128 columns.
                const float *sr = a.scale_rows + row0 + lane;
                const float *sc = a.scale_cols + u.group * a.item_cols + u.n0 / BLOCK * a.n_cols;
                const bool in = lane < rows, wide = quarter == PN / 4;
                auto factors = [&](int kb, float (&f)[3]) {
                    const bool there = in && kb < u.k_blocks;
                    f[0] = there ? __ldg(sr + kb * a.ld_rows) : 0.0f;
                    f[1] = there ? __ldg(sc + kb * a.b_cols) : 0.0f;
                    f[2] = there ? __ldg(sc + kb * a.b_cols + (wide ? a.n_cols : 0)) : 0.0f;
                };
                float next[2][3];
                factors(0, next[0]);
                factors(1, next[1]);
                for (int kb = 0; kb < u.k_blocks; ++kb, ++it) {
                    const uint32_t d = 2 * (it & 1) + second;
                    const float factor[2] = {next[0][0] * next[0][1], next[0][0] * next[0][2]};
#pragma unroll
                    for (int i = 0; i < 3; ++i) next[0][i] = next[1][i];
                    factors(kb + 2, next[1]);
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(bar(SUM_FULL + d), (it >> 1) & 1, a, abort_flag, WD_EPILOGUE));
                    if (!ok) return;
                    tc_fence_after();
                    // A warp without rows only lets go.
                    if (rows <= 0) release(d);
                    else {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            if (c >= chunks) break;
                            uint32_t p[32];
                            tmem_load_32x32(sums + (it & 1) * PN + 32 * c, p);
                            if (c == chunks - 1) release(d);
                            const float f = 2 * c < chunks ? factor[0] : factor[1];
#pragma unroll
                            for (int i = 0; i < 32; ++i) acc[c][i] = fmaf(__uint_as_float(p[i]), f, acc[c][i]);
                        }
                    }
                }
                if (rows <= 0) return;
                const bool f32 = a.out_type == SGEMM_TYPE_F32, bf16 = a.out_type == SGEMM_TYPE_BF16;
                if (a.tma && rows >= 32 && wide) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (column(c) >= a.N) break;
                        if (f32) {
                            send(column(c), row0, 0, [&](uint32_t to) {
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    st_shared_v4(to + sw128_offset(lane, j), acc[c][4 * j], acc[c][4 * j + 1],
                                                 acc[c][4 * j + 2], acc[c][4 * j + 3]);
                            });
                        } else if (c % 2 == 0) {  // two of them are 64 columns of C
                            send(column(c), row0, 0, [&](uint32_t to) {
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    const float *v = &acc[c + j / 4][8 * (j % 4)];
                                    sts_128(to + sw128_offset(lane, j), round2(v[0], v[1], bf16), round2(v[2], v[3], bf16),
                                            round2(v[4], v[5], bf16), round2(v[6], v[7], bf16));
                                }
                            });
                        }
                    }
                    return;
                }
                settle();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c >= chunks) break;
                    const int64_t col = column(c);
                    uint32_t v[16];
                    if (f32) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(acc[c][16 * h + i]);
                            write_lanes(a, out, lane, v, static_cast<uint32_t *>(a.C), row0, rows, col + 16 * h);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            v[i] = round2(acc[c][2 * i], acc[c][2 * i + 1], bf16);
                        write_lanes(a, out, lane, v, static_cast<uint16_t *>(a.C), row0, rows, col);
                    }
                }
            } else {
                // wgrad. acc[c][i][h]: column 32 c + 4 i + (thread % 4), lanes 16 h + (thread / 4) and 8 further.
                uint64_t acc[4][8][2];
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[c][i][0] = acc[c][i][1] = 0;
                const float *sr = a.scale_rows + static_cast<int64_t>(u.k0) * a.ld_rows + row0 + g;
                auto factors = [&](int kb, float (&x)[4]) {
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        x[h] = kb < u.k_blocks && 8 * h + g < rows ? __ldg(sr + kb * a.ld_rows + 8 * h) : 0.0f;
                };
                float next[4];
                factors(0, next);
                for (int kb = 0; kb < u.k_blocks; ++kb, ++it) {
                    const uint32_t d = 2 * (it & 1) + second;
                    const int s = static_cast<int>(it % RING);
                    const uint64_t of_lane[2] = {pack2(__float_as_uint(next[0]), __float_as_uint(next[1])),
                                                 pack2(__float_as_uint(next[2]), __float_as_uint(next[3]))};
                    factors(kb + 1, next);
                    const uint32_t scales =
                        base + RING0 + static_cast<uint32_t>(s * RING_BYTES + (PN / 2 * second + 4 * t) * 4);
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(bar(RING_FULL + s), (it / RING) & 1, a, abort_flag, WD_EPILOGUE)) &&
                         __all_sync(0xffffffffu,
                                    mbar_wait(bar(SUM_FULL + d), (it >> 1) & 1, a, abort_flag, WD_EPILOGUE));
                    if (!ok) return;
                    tc_fence_after();
                    if (rows <= 0) release(d);
                    else {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            if (c >= chunks) break;
                            uint32_t p[32];
                            const uint4 s0 = lds_128(scales + 128 * c), s1 = lds_128(scales + 128 * c + 64);
                            tmem_load_2x16x32(sums + (it & 1) * PN + 32 * c, p);
                            if (c == chunks - 1) release(d);
                            const uint32_t x[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                // The scales first: one of them alone may take a sum out of range.
                                const uint64_t xx = pack2(x[i], x[i]);
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    fma2(acc[c][i][h], pack2(p[16 * h + 2 * i], p[16 * h + 2 * i + 1]), mul2(of_lane[h], xx));
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(RING_EMPTY + s));
                }
                if (a.tma && rows >= 32 && a.out_type == SGEMM_TYPE_F32) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (c >= chunks) break;
                        if (column(c) >= a.N) continue;
                        send(column(c), row0, u.group, [&](uint32_t to) {
#pragma unroll
                            for (int h = 0; h < 4; ++h)
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    float x, y;
                                    unpack2(acc[c][i][h >> 1], x, y);
                                    st_shared_f32(to + sw128_offset(8 * h + g, i) + 4 * t, h & 1 ? y : x);
                                }
                        });
                    }
                    return;
                }
                settle();
                // Eight rows by 32 columns at a time, as fp32 through shared memory.
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c >= chunks) break;
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float x, y;
                            unpack2(acc[c][i][h >> 1], x, y);
                            st_shared_f32(out + static_cast<uint32_t>(g * OUT_WGRAD + (4 * i + t) * 4), h & 1 ? y : x);
                        }
                        __syncwarp();
                        const int64_t item = u.group * a.strideC + static_cast<int64_t>(row0 + 8 * h) * a.ldc;
                        const int left = rows - 8 * h;
                        if (a.out_type == SGEMM_TYPE_F32) {
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int r = 4 * j + (lane >> 3);
                                const int64_t col = column(c) + 4 * (lane & 7);
                                const uint4 x = lds_128(out + static_cast<uint32_t>(r * OUT_WGRAD + 16 * (lane & 7)));
                                if (r < left) store16<uint32_t, 4>(a, static_cast<uint32_t *>(a.C) + item + r * a.ldc + col, col, x);
                            }
                        } else {
                            const bool bf16 = a.out_type == SGEMM_TYPE_BF16;
                            const int64_t col = column(c) + 8 * t;
                            const float4 x = ld_shared_v4(out + static_cast<uint32_t>(g * OUT_WGRAD + 32 * t)),
                                         y = ld_shared_v4(out + static_cast<uint32_t>(g * OUT_WGRAD + 32 * t + 16));
                            const uint4 v = make_uint4(round2(x.x, x.y, bf16), round2(x.z, x.w, bf16),
                                                       round2(y.x, y.y, bf16), round2(y.z, y.w, bf16));
                            if (g < left) store16<uint16_t, 8>(a, static_cast<uint16_t *>(a.C) + item + g * a.ldc + col, col, v);
                        }
                    }
                }
            }
        });
    }

    bulk_wait<0>();  // C is written
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
        if (!mbar_wait(bar(DRAIN), 0, a, abort_flag, WD_DRAIN)) {
            const uint64_t t0 = global_timer();
            while (!mbar_try_wait(bar(DRAIN), 0) && global_timer() - t0 < a.timeout_ns) {
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
    const int64_t matrices = p.experts * p.split;  // of C
    const CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    alignas(64) CUtensorMap map1{}, map2{}, few{}, out{};
    Args a{};
    a.offsets = p.offsets;
    a.rows = static_cast<int>(p.rows);
    a.experts = static_cast<int>(matrices);
    a.split = p.split;
    a.N = p.N;
    a.C = p.C;
    a.ldc = p.ldc;
    a.strideC = p.strideC;
    a.out_type = p.out_type;
    const int64_t per = p.out_type == SGEMM_TYPE_F32 ? 4 : 8;
    a.vector = reinterpret_cast<uintptr_t>(p.C) % 16 == 0 && p.ldc % per == 0 &&
               (!p.wgrad || matrices == 1 || p.strideC % per == 0);
    a.scale_rows = p.sA;
    a.scale_cols = p.sB;
    bool ok;
    int64_t row_tiles;
    if (FORM == WGRAD) {
        a.blocks = static_cast<int>(blocks_of(p.rows));
        a.M = p.M;
        a.ld_rows = p.M;
        a.b_cols = p.N;
        row_tiles = (p.M + PM - 1) / PM * matrices;
        ok = encode_map_typed(&map1, type, 1, p.A, p.rows, p.M, p.lda, 1, 0, HALF, KB, sw) &&
             encode_map_typed(&map2, type, 1, p.B, p.rows, p.N, p.ldb, 1, 0, HALF, KB, sw);
        few = map1;  // not read by the kernel
    } else {
        const int64_t strideB = p.experts > 1 ? p.strideB : 0, kb = blocks_of(p.K), nb = blocks_of(p.N);
        a.k_blocks = static_cast<int>(kb);
        a.ld_rows = p.rows;
        a.item_cols = kb * nb;
        a.n_cols = FORM == ROWS_T ? kb : 1;
        a.b_cols = FORM == ROWS_T ? 1 : nb;
        // Every group may end in a part of a tile, and so may the rest.
        row_tiles = (p.rows + PM - 1) / PM + (p.offsets ? p.experts : 0);
        ok = encode_map_typed(&map1, type, 1, p.A, p.rows, p.K, p.lda, 1, 0, KB, HALF, sw) &&
             encode_map_typed(&few, type, 1, p.A, p.rows, p.K, p.lda, 1, 0, KB, FEW, sw) &&
             (FORM == ROWS_T ? encode_map_typed(&map2, type, 1, p.B, p.N, p.K, p.ldb, p.experts, strideB, KB, HALF, sw)
                             : encode_map_typed(&map2, type, 1, p.B, p.K, p.N, p.ldb, p.experts, strideB, HALF, KB, sw));
    }
    if (!ok) return SGEMM_ERR_LAUNCH;
    const int64_t size = ex::type_size(p.out_type), items = p.wgrad ? matrices : 1;
    const CUtensorMapDataType out_type = p.out_type == SGEMM_TYPE_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                         : p.out_type == SGEMM_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    a.tma = a.vector && encode_map_typed(&out, out_type, size, p.C, p.wgrad ? p.M : p.rows, p.N, p.ldc, items,
                                         items > 1 ? p.strideC : 0, static_cast<uint32_t>(128 / size), 32, sw);
    if (!a.tma) out = map1;  // not used by the kernel
    if (row_tiles > INT32_MAX / 2) return SGEMM_ERR_UNSUPPORTED;
    a.tiles_n = static_cast<int>((p.N + PN - 1) / PN);
    // Instruction descriptor of kind::f8f6f4: D fp32 (bits 4-5 = 1), first and
    // second operand E4M3 (0) or E5M2 (1) in bits 7-9 and 10-12, bit 15 / 16:
    // first / second MN-major, N >> 3 in bits 17-22 (the kernel's), M >> 4 in
    // bits 24-28.
    const uint32_t t1 = p.type_a == SGEMM_FP8_E5M2, t2 = p.type_b == SGEMM_FP8_E5M2;
    a.idesc = (1u << 4) | (t1 << 7) | (t2 << 10) | (FORM == WGRAD ? 1u << 15 : 0u) | (FORM == ROWS_T ? 0u : 1u << 16) |
              (static_cast<uint32_t>(PM >> 4) << 24);
    a.timeout_ns = static_cast<uint64_t>(watchdog_ms()) * 1000000ull;
    a.watchdog = flag;
    const int64_t units = row_tiles * a.tiles_n;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (units < clusters ? units : clusters)));
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, map1, few, map2, out, a) != cudaSuccess) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    ++*launches;
    return SGEMM_OK;
}

// Slices of the groups' rows in wgrad that pay, where the tiles leave half of the
// SM pairs idle: a block of 128 rows takes a pair 0.87 us; the sums are written
// and read at 5 TB/s, the second launch and its wait take 6 us. Groups are taken
// as even. In slices and whole: 1024 x 2048 over 16384 rows 68 and 111 us, 1024 x
// 1024 over 4096 23 and 33, 256 x 256 over 30000 32 and 196 (slices of 3 blocks in
// place of 8: 50, for the join reads more and each role steps over more of them).
int slices_of(const GemmProblem &p, const DeviceInfo &dev) {
    const int64_t tiles = (p.M + PM - 1) / PM * ((p.N + PN - 1) / PN) * p.experts, pairs = dev.sm_count / 2;
    if (2 * tiles > pairs) return 1;
    const double blocks = static_cast<double>(p.rows) / static_cast<double>(p.experts * KB);
    int64_t split = pairs / tiles;
    if (split > blocks / 8) split = static_cast<int64_t>(blocks / 8);
    if (split < 2) return 1;
    const double sums = 8.0 * static_cast<double>(split * p.experts * p.M * p.N) / 5e6;
    const double saved = blocks * (1.0 - 1.0 / static_cast<double>(split)) * 0.87;
    return saved > 6.0 + sums ? static_cast<int>(split) : 1;
}

}  // namespace

int gemm_launch(const GemmProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    if (gemm_few(p, dev)) return gemm_few_launch(p, stream, launches);
    if (dev.device < 0 || dev.device >= kMaxDevices) return SGEMM_ERR_DEVICE;
    if (p.wgrad) {
        const int split = slices_of(p, dev);
        float *sums = nullptr;
        if (split > 1)
            sums = scratch_alloc(dev, static_cast<size_t>(split * p.experts * p.M * ex::slice_ld(p.N)) * 4, stream);
        if (!sums) return launch_form<WGRAD>(p, dev, stream, launches);
        GemmProblem q = p;
        q.split = split;
        q.out_type = SGEMM_TYPE_F32;
        q.C = sums;
        q.ldc = ex::slice_ld(p.N);
        q.strideC = p.M * q.ldc;
        int rc = launch_form<WGRAD>(q, dev, stream, launches);
        if (rc == SGEMM_OK)
            rc = ex::join_slices_launch(p.out_type, sums, split, p.experts, p.M, p.N, p.C, p.ldc, p.strideC, dev, stream,
                                        launches);
        scratch_free(sums, stream);
        return rc;
    }
    return p.transB == SGEMM_OP_T ? launch_form<ROWS_T>(p, dev, stream, launches)
                                  : launch_form<ROWS_N>(p, dev, stream, launches);
}

}  // namespace f8
}  // namespace sgemm
