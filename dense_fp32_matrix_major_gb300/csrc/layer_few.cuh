// A mixture-of-experts layer for a few tokens, in two kernels:
//
//     h[p] = act(W1[e(p)] x[t(p)])              (or act(first half) * second half)
//     y[t] = sum over j of weights[t][j] W2[e] h[t, j]
//
// for at most 512 (token, choice) pairs p. Bound by reading the matrices of the
// experts that are used, once per 8 pairs that share one.
//
// Work. Every block sorts the pairs by expert for itself (a comparison of each
// pair with each, 512 at most) into entries of up to 8 pairs of an expert. First
// kernel: the entries' hidden features in tiles of 16 rows of W1 (8 features and
// their gates), each block a run of tiles. Second kernel: each block some of y's
// columns, in tiles of 16 rows of W2 for every entry, so a token's experts meet in
// one block and are added up in the order of its choices. In a block the tiles
// times their slices of 256 bytes a row are cut evenly among 16 warps, which
// stream them without a pause; a tile that a warp has whole it finishes itself,
// one that is cut is joined, in order, when all are done.
//
// Loads. A lane copies the 16 bytes that it will use itself into its place in a
// ring in shared memory (cp.async), two slices ahead: 128 KB on their way to an SM
// at no cost in registers, and no lane waits for another's copies. (Slices of 128
// bytes, four ahead: 203 us in place of 185 for 32 tokens through 8 of 128 experts
// of 2048 x 768. Bulk copies of 256 bytes a row take 38 cycles each: 274 us for the
// 8-bit layer of 16 experts of 4096 x 4096.) x and h come by plain loads one to four
// chunks ahead, mostly from the caches.
//
// Rows that do not start on 16-byte boundaries are copied from the boundary before
// them on, and a lane takes its 16 bytes out of the 32 around them in registers, 15
// instructions. (Value by value, with multiply-adds: 404 us in place of 97 for 32
// tokens through 4 of 32 experts of 1537 x 1023, gated, bf16.)
//
// Arithmetic. Where x is 16-bit, warp matrix instructions (16 rows of the matrix x
// k x 8 pairs, fp32 sums) on the values as they are: bf16 and fp16 with x of the
// same type; 8-bit ones as x's type, exactly. h enters as two bf16 terms, 16 of its
// 24 bits (y is rounded to 11 at most; a third term took 141 us in place of 128 for 8
// tokens, 2 of 16 experts of 4096 x 4096 in 8 bits, 193 in place of 180 in bf16 and
// 203 in place of 183 in fp16 for 32 tokens, 8 of 128 of 2048 x 768, and left the
// error of y against 64 bits as it was, 1.66693e-3 of the norm in the first), which
// the first kernel stores apart: as they are with bf16 matrices and with 8-bit ones
// made bf16, as tf32 with fp16 ones. (8-bit ones as tf32 with bf16
// x and with h, fewer steps for a value but twice the instructions that multiply:
// 140 us in place of 127 for 8 tokens, 2 of 16 experts of 4096 x 4096.) With fp32 x
// fp32 multiply-adds, because the instruction cuts its running sums (1.3e-6 of the
// result's norm where multiply-adds leave 0.2e-6), which is also why 16-bit values'
// sums leave it after every slice of 128 (at no cost); x then goes through 512 bytes of
// shared memory, from the lane that loaded it to all. (Loaded by every lane: 449 us in
// place of 121 for 32 tokens, 4 of 32 experts of 1536 x 1024.) (tcgen05 wants its operands in
// shared memory and 128 rows a tile for at most 16 columns of x here.) Which k a
// lane holds does not matter as long as matrix and x agree, so a lane takes 16 bytes
// of a row that lie together.
//
// What it reaches: 32 tokens through 8 of 128 experts of 2048 x 768, gated, fp16, 180
// us, 5.8 TB/s. One token through 8 of 64 experts of 2048 x 1024 takes 29 us for 100 MB:
// the start and the end of two kernels. From 8-bit matrices 4.2 TB/s: 56% of the issue
// slots are used, and a warp mostly waits for its own instruction before, in the chain
// from a byte to a product, with four warps a scheduler. An expert's matrices are read
// again for every 8 pairs: 64 tokens through 2 of 8 experts of 4096 x 2048, gated,
// take 196 us in bf16 and 134 from e4m3, through all 8 643 and 418.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "epilogue.cuh"
#include "experts_common.cuh"
#include "layer_internal.h"

namespace sgemm {
namespace fl {
namespace {

using ex::from_f32;
using ex::to_f32;

constexpr int WARPS = 16, THREADS = 32 * WARPS;
constexpr int MEMBERS = 8;   // pairs of an entry, the columns of the matrix instructions
constexpr int COLUMNS = 32;  // of y that a block of the second kernel makes at once
static_assert(MAX_PAIRS <= THREADS, "a thread a pair");
// A warp's ring: slices of 256 bytes of 16 rows, in 16-byte pieces by lane, and the
// 16 bytes of each row that follow.
constexpr int SLICE = 256, CHUNKS = SLICE / 64, FOLLOWING = 2 * CHUNKS * 512, STAGE = FOLLOWING + 16 * 16, STAGES = 2;
constexpr int RING_BYTES = STAGES * STAGE;
// Shared memory: the rings, 512 bytes of each warp (x of its chunk, then the sums of
// a tile that it shares), and in the second kernel the pairs' sums.
constexpr int SMEM = WARPS * (RING_BYTES + 512);
constexpr int smem_out(int pairs) { return SMEM + pairs * COLUMNS * 4; }

// The pairs sorted by expert, and the entries: runs of up to MEMBERS pairs of an
// expert.
struct Lists {
    alignas(16) int key[MAX_PAIRS];
    int order[MAX_PAIRS];     // pair at a sorted place
    int place[MAX_PAIRS];     // of a pair; -1: left out
    int entry_at[MAX_PAIRS];  // entry of a sorted place
    int expert[MAX_PAIRS], begin[MAX_PAIRS], count[MAX_PAIRS];  // of an entry
    int total[WARPS];
    int entries;
    mutable int late;  // h has places to be made again (see sums_again)
};

__device__ __forceinline__ int id_of(const LArgs &a, int p) {
    if (a.id_bits == 64) {
        const int64_t e = __ldg(static_cast<const long long *>(a.ids) + p);
        return e < 0 || e >= a.experts ? a.experts : static_cast<int>(e);
    }
    const int e = __ldg(static_cast<const int *>(a.ids) + p);
    return e < 0 || e >= a.experts ? a.experts : e;
}

// Called by the whole block.
__device__ __forceinline__ void build_lists(const LArgs &a, Lists &l) {
    const int p = static_cast<int>(threadIdx.x), lane = p & 31, warp = p >> 5;
    const int padded = (a.pairs + 3) & ~3;
    if (p < padded) l.key[p] = p < a.pairs ? id_of(a, p) : a.experts;
    l.entry_at[p] = 0;
    __syncthreads();
    int place = 0, rank = 0, same = 0;
    const int key = p < a.pairs ? l.key[p] : a.experts;
    if (p < a.pairs) {
        for (int q = 0; q < padded; q += 4) {
            const int4 k = *reinterpret_cast<const int4 *>(l.key + q);
            const int v[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int eq = v[i] == key, before = eq && q + i < p;
                same += eq;
                rank += before;
                place += before || v[i] < key;
            }
        }
    }
    const bool used = key < a.experts;
    if (p < a.pairs) l.place[p] = used ? place : -1;
    if (used) {
        l.order[place] = p;
        l.entry_at[place] = rank % MEMBERS == 0;  // an entry starts
    }
    __syncthreads();
    // Numbers the entries in sorted order.
    const int starts = l.entry_at[p];
    const unsigned ballot = __ballot_sync(0xffffffffu, starts);
    if (lane == 0) l.total[warp] = __popc(ballot);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        before += w < warp ? l.total[w] : 0;
        all += l.total[w];
    }
    l.entry_at[p] = before + __popc(ballot & (0xffffffffu >> (31 - lane))) - 1;
    if (p == 0) {
        l.entries = all;
        l.late = 0;
    }
    __syncthreads();
    if (used && rank % MEMBERS == 0) {
        const int e = l.entry_at[place];
        l.expert[e] = key;
        l.begin[e] = place;
        l.count[e] = min(MEMBERS, same - rank);
    }
    __syncthreads();
}

// How a matrix is held. PER: values in 16 bytes, which a lane takes of a row in a
// chunk of 64 bytes; four chunks make a slice.
enum Held { F32, BF16, F16, E4M3, E5M2 };
template <int H>
struct Matrix {
    static constexpr int SIZE = H == F32 ? 4 : (H >= E4M3 ? 1 : 2), PER = 16 / SIZE, CHUNK = 4 * PER, SLICE_K = SLICE / SIZE;
    static constexpr bool FP8 = H >= E4M3;
};

// How sums are made: fp32 multiply-adds; matrix instructions on 16-bit values,
// with x, or with h in two planes; on fp16 or bf16 made of 8-bit values, with x of
// that type, or with h; on tf32 with h.
enum Math { FMA, NATIVE, PLANES, HALF8, BF8, BF8_H, TF32_H };

// 16 bytes of a row of K values from value k on, zeros past its end. They are 16-byte aligned.
template <int SIZE>
__device__ __forceinline__ void load_piece(const uint8_t *row, int k, int K, uint32_t (&v)[4]) {
    constexpr int PER = 16 / SIZE;
    v[0] = v[1] = v[2] = v[3] = 0;
    if (k >= K) return;
    const uint8_t *p = row + static_cast<int64_t>(k) * SIZE;
    if (k + PER <= K) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        return;
    }
#pragma unroll 1
    for (int i = 0; i < PER && k + i < K; ++i) {
        uint32_t x;
        if (SIZE == 4) x = __ldg(reinterpret_cast<const uint32_t *>(p) + i);
        if (SIZE == 2) x = __ldg(reinterpret_cast<const uint16_t *>(p) + i);
        x <<= 8 * (i * SIZE % 4);
        v[0] |= i * SIZE / 4 == 0 ? x : 0;
        v[1] |= i * SIZE / 4 == 1 ? x : 0;
        v[2] |= i * SIZE / 4 == 2 ? x : 0;
        v[3] |= i * SIZE / 4 == 3 ? x : 0;
    }
}

// The same of a row anywhere: the 32 bytes around them from the 16-byte boundary
// before them on, for realign(). Nothing past the row's end is read.
template <int SIZE>
__device__ __forceinline__ void load_piece(const uint8_t *row, int k, int K, uint32_t (&v)[8]) {
    constexpr int PER = 16 / SIZE;
#pragma unroll
    for (int w = 0; w < 8; ++w) v[w] = 0;
    if (k >= K) return;
    const uint8_t *p = row + static_cast<int64_t>(k) * SIZE;
    const int before = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
    if (k + 2 * PER - before / SIZE <= K) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p - before), y = *reinterpret_cast<const uint4 *>(p - before + 16);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
        return;
    }
#pragma unroll 1
    for (int i = 0; i < PER && k + i < K; ++i) {
        uint32_t x;
        if (SIZE == 4) x = __ldg(reinterpret_cast<const uint32_t *>(p) + i);
        if (SIZE == 2) x = __ldg(reinterpret_cast<const uint16_t *>(p) + i);
        const int at = before + i * SIZE;
        x <<= 8 * (at % 4);
#pragma unroll
        for (int w = 0; w < 8; ++w) v[w] |= at / 4 == w ? x : 0;
    }
}

// 16 of 32 bytes, from byte `from` (0 .. 15, a multiple of SIZE) on.
template <int SIZE>
__device__ __forceinline__ void realign(const uint32_t (&w)[8], int from, uint32_t (&v)[4]) {
    uint32_t a[6], b[5];
#pragma unroll
    for (int i = 0; i < 6; ++i) a[i] = from & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) b[i] = from & 4 ? a[i + 1] : a[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = SIZE == 4 ? b[i] : __funnelshift_r(b[i], b[i + 1], 8 * (from & 3));
}

// Value i of two bf16 ones.
__device__ __forceinline__ float bf16_of(uint32_t w, int i) { return __uint_as_float(i ? w & 0xFFFF0000u : w << 16); }

// Two 8-bit values (the low 16 bits of w) as fp16, exactly.
template <int H>
__device__ __forceinline__ uint32_t fp8_halves(uint32_t w) {
    if (H == E5M2) return __byte_perm(w, 0, 0x1404);  // the upper half of an fp16
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(w)));
    return h2;
}

// The same as bf16, exactly too.
template <int H>
__device__ __forceinline__ uint32_t fp8_bf16(uint32_t w) {
    const uint32_t h = fp8_halves<H>(w);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// Values 2 i and 2 i + 1 of 16 bytes of fp16 or 8-bit values as fp32.
template <int H>
__device__ __forceinline__ float2 two_of(const uint32_t (&w)[4], int i) {
    const uint32_t h = H == F16 ? w[i] : fp8_halves<H>(w[i / 2] >> (16 * (i & 1)));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Value i of 16 bytes as fp32.
template <int H>
__device__ __forceinline__ float value_of(const uint32_t (&w)[4], int i) {
    if (H == F32) return __uint_as_float(w[i]);
    const float2 v = two_of<H>(w, i / 2);
    return i & 1 ? v.y : v.x;
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], float a0, float a1, float a2, float a3, float b0, float b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

template <bool BF>
__device__ __forceinline__ void mma_16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    if (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A block's warps sum `items` tiles of 16 rows over k, cut with their slices of k
// into equal shares: this warp has `mine` slices from slice `from` on.
struct Share {
    int slices, from, mine;
};

__device__ __forceinline__ Share share_of(int items, int K, int slice) {
    const int warp = threadIdx.x >> 5, slices = (K + slice - 1) / slice;
    const int64_t all = static_cast<int64_t>(items) * slices;
    const int64_t from = all * warp / WARPS;
    return Share{slices, static_cast<int>(from), static_cast<int>(all * (warp + 1) / WARPS - from)};
}

// A place in a share: a tile's number among the block's, its entry, which of the
// entry's (first kernel) or block's (second) tiles it is, and the slice.
struct Cursor {
    int item, entry, tile, slice;
};

// 16-byte asynchronous copy to shared memory, past the L1 cache: the first `bytes`
// are read, the others zero.
__device__ __forceinline__ void copy_16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(__cvta_generic_to_global(src)), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void sts_128(uint32_t at, const uint32_t (&v)[4]) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

template <int N>
__device__ __forceinline__ void lds_128(uint32_t at, uint32_t (&v)[N], int first = 0) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[first]), "=r"(v[first + 1]), "=r"(v[first + 2]), "=r"(v[first + 3])
                 : "r"(at)
                 : "memory");
}

// The jobs of the two kernels say which rows and pairs a tile has:
//   cursor(item)       the block's item-th tile; next(c): the one after c
//   base(c, g)         address of row g (0 .. 7) of the tile
//   delta()            from there to row 8 + g, in bytes
//   there(c, i, g)     whether the tile has row 8 i + g
//   scales(c)          scales of the entry's 8-bit matrix
//   scale_row(c, i, g) where those of row 8 i + g begin
//   members(c)         pairs
//   x(c, m)            pair m's row of x or h
//   ALIGNED            those rows always start on 16-byte boundaries
//   finish(c, sum)     takes a tile's sums: sum[2 i + j] of lane 4 g + t is row 8 i + g, pair 2 t + j
// and where they may be made again:
//   late(c)            which of the lane's sums, bit 2 i + j
//   settle(c, sum, n)  takes those of bits n
//   length()           values of a row
//   value(x, k)        value k of a pair's row of x or h

// The next slice; true where a tile starts.
template <class Job>
__device__ __forceinline__ bool step(const Job &job, const Share &s, Cursor &c) {
    if (++c.slice < s.slices) return false;
    c.slice = 0;
    ++c.item;
    job.next(c);
    return true;
}

template <class Job>
__device__ __forceinline__ Cursor first_of(const Job &job, const Share &s) {
    Cursor c = job.cursor(s.from / s.slices);
    c.slice = s.from % s.slices;
    return c;
}

// What is left when a warp's share is done: parts of tiles that other warps have
// too. The part of a tile that started in an earlier warp's share lies in `parts`;
// a tile that started in this one and goes on is in `sum`.
struct Rest {
    bool open;
    Cursor at;
    float sum[4];
};

// Joins the tiles that are cut. Called by the whole block; parts_of: the tile that
// each warp's part belongs to, -1: none.
template <class Job>
__device__ __forceinline__ void join(const Job &job, Rest &rest, const float4 *parts, const int *part_of) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (!rest.open) return;
    for (int w = warp + 1; w < WARPS; ++w) {
        if (part_of[w] != rest.at.item) continue;  // another tile, or no share at all
        const float4 p = parts[w * 32 + lane];
        rest.sum[0] += p.x;
        rest.sum[1] += p.y;
        rest.sum[2] += p.z;
        rest.sum[3] += p.w;
    }
    job.finish(rest.at, rest.sum);
}

// Sums of multiply-adds: f[m]: rows g and g + 8, pair m, this lane's k only.
__device__ __forceinline__ void gather_lanes(float (&f)[MEMBERS][2], int t, float (&sum)[4]) {
#pragma unroll
    for (int m = 0; m < MEMBERS; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float v = f[m][i];
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
            if (m / 2 == t) sum[2 * i + (m & 1)] = v;
        }
}

// ring: the warp's ring. ANY: rows of the matrix (8-bit ones excepted) and of x need
// not start on 16-byte boundaries. Those of the matrix are then copied from the
// boundary before them on (which lies in the same allocation), and a lane takes its
// 16 bytes from its own piece and the next; x comes in 32 bytes that hold its 16.
template <int H, int MATH, bool ANY, class X, class Job>
__device__ __forceinline__ void sum_ring(const Job &job, int items, int K, uint32_t ring, float4 *parts, int *part_of,
                                         Rest &rest) {
    using M = Matrix<H>;
    constexpr bool SHIFT = ANY && !M::FP8, SPLIT = ANY && !Job::ALIGNED, TWO = MATH == PLANES || MATH == BF8_H || MATH == TF32_H;
    // 16-byte pieces of x in a lane's part of a chunk, and chunks of them on their way.
    constexpr int PX = M::PER * static_cast<int>(sizeof(X)) / 16, PIECES = TWO ? 2 * M::PER / 8 : PX,
                  XP = SPLIT ? (PIECES > 1 ? 1 : 2) : (PIECES > 2 ? 2 : 4), XW = SPLIT ? 8 : 4;
    constexpr int XSIZE = TWO ? 2 : static_cast<int>(sizeof(X));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const Share s = share_of(items, K, M::SLICE_K);
    rest.open = false;
    if (lane == 0) part_of[warp] = -1;
    if (s.mine == 0) return;
    Cursor load = first_of(job, s), use = load;
    const int64_t delta = job.delta();
    // Where rows g and g + 8 lie after the boundary before them, in bytes.
    auto shifts = [&](const uint8_t *p, int (&shift)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) shift[i] = SHIFT ? static_cast<int>(reinterpret_cast<uintptr_t>(p + i * delta) & 15) : 0;
    };
    // Pieces past a row's end, and rows past the matrix's, are copies of no bytes
    // from the start of a row that is there.
    const uint8_t *row[2];
    int left[2];  // values from this lane's first piece to the row's end
    auto enter = [&] {
        const uint8_t *first = job.base(load, 0), *p = job.base(load, g);
        int shift[2], none[2];
        shifts(p, shift);
        shifts(first, none);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool there = job.there(load, i, g);
            row[i] = (there ? p + i * delta - shift[i] : first - none[0]) + 16 * t;
            left[i] = there ? K + shift[i] / M::SIZE - M::PER * t : 0;
        }
    };
    enter();
    // Copies the next slice; one group of copies each, empty or not.
    auto fetch = [&](int stage, bool in) {
        if (in) {
            const uint32_t to = ring + static_cast<uint32_t>(stage * STAGE + 16 * lane);
            const int64_t at = static_cast<int64_t>(load.slice) * SLICE;
            const int k = load.slice * M::SLICE_K;
            const bool inner = k + M::SLICE_K <= K;  // the rows end later
            auto copy_part = [&](uint32_t dst, const uint8_t *from, const uint8_t *start, int n) {
                copy_16(dst, n > 0 ? from : start, max(min(n, M::PER), 0) * M::SIZE);
            };
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t *p = row[i] + at;
                if (inner) {
                    const int all = left[i] > 0 ? 16 : 0;
#pragma unroll
                    for (int q = 0; q < CHUNKS; ++q) copy_16(to + 1024 * q + 512 * i, p + q * 64, all);
                } else {
#pragma unroll
                    for (int q = 0; q < CHUNKS; ++q)
                        copy_part(to + 1024 * q + 512 * i, p + q * 64, row[i] - 16 * t, left[i] - (k + q * M::CHUNK));
                }
            }
            if (SHIFT && t < 2) {
                const int n = t == 0 ? left[0] : (left[1] > 0 ? left[1] + M::PER : 0);
                const uint8_t *start = t == 0 ? row[0] : row[1] - 16;
                copy_part(ring + static_cast<uint32_t>(stage * STAGE + FOLLOWING + 128 * t + 16 * g), start + at + SLICE,
                          start, n - (k + M::SLICE_K));
            }
            if (step(job, s, load)) enter();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // Scales of rows g and g + 8 of the next slice.
    constexpr int BLOCKS = M::FP8 ? M::SLICE_K / SGEMM_FP8_BLOCK_SIZE : 1;
    Cursor ahead = use;
    const float *scale_at[2];
    auto enter_scales = [&] {
#pragma unroll
        for (int i = 0; i < 2; ++i) scale_at[i] = job.scales(ahead) + job.scale_row(ahead, i, g);
    };
    float next_scale[2][BLOCKS] = {};
    auto fetch_scales = [&](bool in) {
        if constexpr (M::FP8) {
            if (!in) return;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b) {
                    const int block = ahead.slice * BLOCKS + b;
                    next_scale[i][b] = block * SGEMM_FP8_BLOCK_SIZE < K ? __ldg(scale_at[i] + block) : 0.0f;
                }
            if (step(job, s, ahead)) enter_scales();
        }
    };
    // x of member g, XP chunks ahead of the sums.
    Cursor pre = use;
    auto x_of = [&](const Cursor &c) {
        const int n = job.members(c);
        return static_cast<const uint8_t *>(job.x(c, g < n ? g : 0));
    };
    const uint8_t *x_row = nullptr;
    uint32_t xw[XP][PIECES][XW];
    auto load_x = [&](int q, bool in) {  // chunk q of slice `pre`
        if (!in) return;
        const int k = pre.slice * M::SLICE_K + q * M::CHUNK + M::PER * t;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            if (TWO)  // plane i % 2
                load_piece<2>(x_row + (i & 1) * job.plane(), k + i / 2 * 8, K, xw[q % XP][i]);
            else
                load_piece<XSIZE>(x_row, k + i * (16 / XSIZE), K, xw[q % XP][i]);
        }
        if (q == CHUNKS - 1 && step(job, s, pre)) x_row = x_of(pre);
    };
    float sum[4], side[2][4], fma[MATH == FMA ? MEMBERS : 1][2];
    float part[4] = {};
    int part_item = -1;
    int count = 0, shift[2], x_shift = 0;
    bool started = false;  // the tile started in this share
    auto start = [&] {
        count = job.members(use);
        started = use.slice == 0;
        if (SHIFT) shifts(job.base(use, g), shift);
        if (SPLIT) x_shift = static_cast<int>(reinterpret_cast<uintptr_t>(x_of(use)) & 15);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = side[0][i] = side[1][i] = 0.0f;
#pragma unroll
        for (int m = 0; m < (MATH == FMA ? MEMBERS : 1); ++m) fma[m][0] = fma[m][1] = 0.0f;
    };
    // Adds a chunk's products with the members' x in v to d[0] and d[1]: two chains
    // of instructions that wait for their own sums only.
    auto multiply = [&](const uint32_t (&lo)[4], const uint32_t (&hi)[4], const uint32_t (&v)[PIECES][4],
                        float (&d)[2][4]) {
        if constexpr (MATH == NATIVE || MATH == PLANES) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                mma_16<H == BF16>(d[0], lo[0], hi[0], lo[1], hi[1], v[i][0], v[i][1]);
                mma_16<H == BF16>(d[1], lo[2], hi[2], lo[3], hi[3], v[i][2], v[i][3]);
            }
        } else if constexpr (MATH == HALF8) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                mma_16<false>(d[j & 1], fp8_halves<H>(lo[j]), fp8_halves<H>(hi[j]), fp8_halves<H>(lo[j] >> 16),
                              fp8_halves<H>(hi[j] >> 16), v[j / 2][2 * (j & 1)], v[j / 2][2 * (j & 1) + 1]);
        } else if constexpr (MATH == BF8 || MATH == BF8_H) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a0 = fp8_bf16<H>(lo[j]), a1 = fp8_bf16<H>(hi[j]), a2 = fp8_bf16<H>(lo[j] >> 16),
                               a3 = fp8_bf16<H>(hi[j] >> 16);
#pragma unroll
                for (int i = 0; i < (MATH == BF8_H ? 2 : 1); ++i) {
                    const uint32_t(&x)[4] = v[MATH == BF8_H ? j / 2 * 2 + i : j / 2];
                    mma_16<true>(d[MATH == BF8_H ? i : j & 1], a0, a1, a2, a3, x[2 * (j & 1)], x[2 * (j & 1) + 1]);
                }
            }
        } else if constexpr (MATH == TF32_H) {
#pragma unroll
            for (int j = 0; j < M::PER / 2; ++j) {
                const float2 a0 = two_of<H>(lo, j), a1 = two_of<H>(hi, j);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t two = v[j / 4 * 2 + i][j % 4];
                    mma_tf32(d[i], a0.x, a1.x, a0.y, a1.y, bf16_of(two, 0), bf16_of(two, 1));
                }
            }
        }
    };
    // The same by multiply-adds, with x by way of shared memory to all lanes.
    const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(parts + warp * 32));
    auto multiply_add = [&](const uint32_t (&lo)[4], const uint32_t (&hi)[4], const uint32_t (&v)[PIECES][4], float s0,
                            float s1) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            float a0[4], a1[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a0[j] = value_of<H>(lo, 4 * i + j) * (M::FP8 ? s0 : 1.0f);
                a1[j] = value_of<H>(hi, 4 * i + j) * (M::FP8 ? s1 : 1.0f);
            }
            __syncwarp();
            sts_128(mine + 16 * lane, v[i]);
            __syncwarp();
#pragma unroll
            for (int m = 0; m < MEMBERS; ++m) {
                if (m >= count) break;
                uint32_t b[4];
                lds_128(mine + 16 * (4 * m + t), b);
                float(&f)[2] = fma[MATH == FMA ? m : 0];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[0] = fmaf(a0[j], __uint_as_float(b[j]), f[0]);
                    f[1] = fmaf(a1[j], __uint_as_float(b[j]), f[1]);
                }
            }
        }
    };
#pragma unroll
    for (int n = 0; n < STAGES; ++n) fetch(n, n < s.mine);
    if (M::FP8) enter_scales();
    fetch_scales(true);
    x_row = x_of(pre);
#pragma unroll
    for (int q = 0; q < XP; ++q) load_x(q, true);
    start();
    for (int n = 0; n < s.mine; ++n) {
        const int stage = n % STAGES;
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
        if (SHIFT) __syncwarp();  // the other lanes' copies
        const uint32_t at = ring + static_cast<uint32_t>(stage * STAGE + 16 * lane);
        const bool last = n + 1 == s.mine;
        float scale[2][BLOCKS];
#pragma unroll
        for (int i = 0; i < 2 * BLOCKS; ++i) scale[i / BLOCKS][i % BLOCKS] = next_scale[i / BLOCKS][i % BLOCKS];
        fetch_scales(!last);
#pragma unroll
        for (int q = 0; q < CHUNKS; ++q) {
            constexpr int PER_BLOCK = CHUNKS / BLOCKS;
            uint32_t a[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if constexpr (SHIFT) {
                    uint32_t w[8];
                    lds_128(at + 1024 * q + 512 * i, w);
                    lds_128(t < 3            ? at + 1024 * q + 512 * i + 16
                            : q + 1 < CHUNKS ? at + 1024 * (q + 1) + 512 * i - 48
                                             : ring + stage * STAGE + FOLLOWING + 128 * i + 16 * g,
                            w, 4);
                    realign<M::SIZE>(w, shift[i], a[i]);
                } else {
                    lds_128(at + 1024 * q + 512 * i, a[i]);
                }
            }
            auto sums = [&](const uint32_t(&v)[PIECES][4]) {
                if constexpr (MATH == FMA)
                    multiply_add(a[0], a[1], v, scale[0][q / PER_BLOCK], scale[1][q / PER_BLOCK]);
                else
                    multiply(a[0], a[1], v, side);
            };
            if constexpr (SPLIT) {
                uint32_t v[PIECES][4];
#pragma unroll
                for (int i = 0; i < PIECES; ++i) realign<XSIZE>(xw[q % XP][i], x_shift, v[i]);
                sums(v);
            } else {
                sums(xw[q % XP]);
            }
            load_x((q + XP) % CHUNKS, !last || q + XP < CHUNKS);
            if (MATH != FMA && q % PER_BLOCK == PER_BLOCK - 1) {
                // A block of an 8-bit matrix ends, or a slice of another.
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float more = side[0][i] + side[1][i];
                    sum[i] = M::FP8 ? fmaf(more, scale[i >> 1][q / PER_BLOCK], sum[i]) : sum[i] + more;
                    side[0][i] = side[1][i] = 0.0f;
                }
            }
        }
        if (SHIFT) __syncwarp();  // the other lanes have read this stage
        fetch(stage, n + STAGES < s.mine);
        const bool done = use.slice + 1 == s.slices;
        if (last || done) {
            if constexpr (MATH == FMA) gather_lanes(fma, t, sum);
            if (done && started) {
                job.finish(use, sum);
            } else if (started) {
                rest.open = true;
                rest.at = use;
#pragma unroll
                for (int i = 0; i < 4; ++i) rest.sum[i] = sum[i];
            } else if constexpr (MATH == FMA) {
                // parts' place is x's: later.
                part_item = use.item;
#pragma unroll
                for (int i = 0; i < 4; ++i) part[i] = sum[i];
            } else {
                parts[warp * 32 + lane] = make_float4(sum[0], sum[1], sum[2], sum[3]);
                if (lane == 0) part_of[warp] = use.item;
            }
        }
        if (step(job, s, use) && !last) start();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if constexpr (MATH == FMA) {
        if (part_item < 0) return;
        __syncwarp();  // x there is read
        parts[warp * 32 + lane] = make_float4(part[0], part[1], part[2], part[3]);
        if (lane == 0) part_of[warp] = part_item;
    }
}

extern __shared__ __align__(16) uint8_t dynamic_smem[];

// Sums and finishes a block's tiles.
template <int H, int MATH, bool ANY, class X, class Job>
__device__ __forceinline__ void sum_tiles(const Job &job, int items, int K, int *part_of) {
    float4 *parts = reinterpret_cast<float4 *>(dynamic_smem + WARPS * RING_BYTES);
    Rest rest;
    sum_ring<H, MATH, ANY, X>(job, items, K,
                              static_cast<uint32_t>(__cvta_generic_to_shared(dynamic_smem)) + (threadIdx.x >> 5) * RING_BYTES,
                              parts, part_of, rest);
    join(job, rest, parts, part_of);
}

// The matrix instructions sum a block of an 8-bit matrix before its scale: values
// of x from 2^105 on (128 times 57344 is 2^22.8) may overflow where the scaled
// products do not. Sums that are not finite are made again, of scaled values, when
// the block's tiles are done; those of a pair with a NaN are not, which explains
// them. (8 tokens, 2 of 16 experts of 4096 x 4096: 130 us, without this code 128,
// which deals the registers out otherwise; made again as soon as a tile is done
// 132; with the scale's power of two in the values from the start 138. Made again
// for all of one token's sums: 0.8 ms for an infinity in its x, 1.1 for values near
// 2^125, and 0.16 with a NaN.) Called by the whole block.
template <int H, class Job>
__device__ __forceinline__ void sums_again(const Job &job, int items) {
    const int lane = threadIdx.x & 31, K = job.length();
#pragma unroll 1
    for (int item = threadIdx.x >> 5; item < items; item += WARPS) {
        const Cursor c = job.cursor(item);
        const unsigned late = job.late(c);
        if (!__any_sync(0xffffffffu, late)) continue;
        const int count = job.members(c);
        unsigned with_nan = 0;  // pairs
#pragma unroll 1
        for (int m = 0; m < count; ++m) {
            const void *x = job.x(c, m);
            bool any = false;
#pragma unroll 4
            for (int k = lane; k < K; k += 32) any |= isnan(job.value(x, k));
            with_nan |= __any_sync(0xffffffffu, any) ? 1u << m : 0;
        }
        float sum[4] = {};
        unsigned made = 0;
#pragma unroll 1
        for (int n = 0; n < 4; ++n) {
            unsigned lanes = __ballot_sync(0xffffffffu, late >> n & 1);
#pragma unroll 1
            for (; lanes; lanes &= lanes - 1) {
                const int to = __ffs(lanes) - 1, m = 2 * (to & 3) + (n & 1);
                if (with_nan >> m & 1) continue;
                const void *x = job.x(c, m);
                const uint8_t *row = job.base(c, to >> 2) + (n >> 1) * job.delta();
                const float *scale = job.scales(c) + job.scale_row(c, n >> 1, to >> 2);
                float v = 0.0f;
#pragma unroll 2
                for (int k = lane; k < K; k += 32) {
                    const uint32_t h = fp8_halves<H>(row[k]);
                    v = fmaf(__low2float(*reinterpret_cast<const __half2 *>(&h)) * __ldg(scale + k / SGEMM_FP8_BLOCK_SIZE),
                             job.value(x, k), v);
                }
#pragma unroll
                for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
                if (lane != to) continue;
                made |= 1u << n;
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] = i == n ? v : sum[i];
            }
        }
        job.settle(c, sum, made);
    }
}

// h of the entries' tiles of features: 16 rows of W1, 8 features with their gates
// or 16 without. AGAIN: sums_again() follows.
template <int H, bool AGAIN>
struct HiddenJob {
    using M = Matrix<H>;
    const LArgs &a;
    const Lists &l;
    int first, per_tile, per_entry, kblocks;
    int64_t item_scales;
    __device__ __forceinline__ Cursor cursor(int item) const {
        const int i = first + item, entry = i / per_entry;
        return Cursor{item, entry, i - entry * per_entry, 0};
    }
    __device__ __forceinline__ void next(Cursor &c) const {
        if (++c.tile < per_entry) return;
        c.tile = 0;
        c.entry = min(c.entry + 1, l.entries - 1);  // past the last: never used
    }
    __device__ __forceinline__ int feature(const Cursor &c) const { return c.tile * per_tile; }
    // Row 8 i + g of a tile is, in W1, row feature + offset(i) + g.
    __device__ __forceinline__ int offset(int i) const { return i == 0 ? 0 : (a.gated ? a.hidden : 8); }
    __device__ __forceinline__ const uint8_t *base(const Cursor &c, int g) const {
        return static_cast<const uint8_t *>(a.w1) + (l.expert[c.entry] * a.stride1 + (feature(c) + g) * a.ld1) * M::SIZE;
    }
    __device__ __forceinline__ int64_t delta() const { return offset(1) * a.ld1 * M::SIZE; }
    __device__ __forceinline__ bool there(const Cursor &c, int i, int g) const {
        return feature(c) + (a.gated ? 0 : 8 * i) + g < a.hidden;
    }
    __device__ __forceinline__ const float *scales(const Cursor &c) const { return a.s1 + l.expert[c.entry] * item_scales; }
    __device__ __forceinline__ int scale_row(const Cursor &c, int i, int g) const {
        return there(c, i, g) ? (feature(c) + offset(i) + g) / SGEMM_FP8_BLOCK_SIZE * kblocks : 0;
    }
    __device__ __forceinline__ int members(const Cursor &c) const { return l.count[c.entry]; }
    __device__ __forceinline__ int pair(const Cursor &c, int m) const { return l.order[l.begin[c.entry] + m]; }
    __device__ __forceinline__ const void *x(const Cursor &c, int m) const {
        return static_cast<const uint8_t *>(a.x) + pair(c, m) / a.top_k * a.ldx * a.x_size;
    }
    __device__ __forceinline__ int64_t plane() const { return 0; }
    static constexpr bool ALIGNED = false;
    __device__ __forceinline__ void write(const Cursor &c, int m, int feature, float v) const {
        float *to = a.h + pair(c, m) * a.ldh;
        if (a.x_type != SGEMM_TYPE_F32) {
            // Two bf16 terms, 16 bits of v: what a 16-bit y rounds away is 2^7 times as
            // large. The first of a finite v is finite.
            constexpr float most = 3.38953139e38f;  // bf16's largest
            const __nv_bfloat16 hi = __float2bfloat16_rn(isfinite(v) ? fminf(fmaxf(v, -most), most) : v);
            __nv_bfloat16 *p = reinterpret_cast<__nv_bfloat16 *>(to) + feature;
            p[0] = hi;
            p[a.ldh] = __float2bfloat16_rn(isfinite(v) ? v - __bfloat162float(hi) : 0.0f);
        } else {
            to[feature] = v;
        }
    }
    // Where a feature's sums are to be made again h is this NaN, which no rounding gives.
    static constexpr uint16_t LATE = 0x7FC1;
    __device__ __forceinline__ uint16_t *place(const Cursor &c, int m, int feature) const {
        return reinterpret_cast<uint16_t *>(a.h + pair(c, m) * a.ldh) + feature;
    }
    template <bool MARK>
    __device__ __forceinline__ void take(const Cursor &c, const float (&sum)[4], unsigned which) const {
        const int lane = threadIdx.x & 31, f = feature(c) + (lane >> 2), count = members(c);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int m = 2 * (lane & 3) + j;
            if (m >= count) continue;
            if (a.gated) {
                if (f >= a.hidden || !(which >> j & 1)) continue;
                write(c, m, f, activate(sum[j], a.activation) * sum[2 + j]);
                if (MARK && !(isfinite(sum[j]) && isfinite(sum[2 + j]))) *place(c, m, f) = LATE, l.late = 1;
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (f + 8 * i >= a.hidden || !(which >> (2 * i + j) & 1)) continue;
                    write(c, m, f + 8 * i, activate(sum[2 * i + j], a.activation));
                    if (MARK && !isfinite(sum[2 * i + j])) *place(c, m, f + 8 * i) = LATE, l.late = 1;
                }
            }
        }
    }
    __device__ __forceinline__ void finish(const Cursor &c, const float (&sum)[4]) const { take<AGAIN>(c, sum, 15); }
    __device__ __forceinline__ void settle(const Cursor &c, const float (&sum)[4], unsigned which) const {
        take<false>(c, sum, which);
    }
    __device__ __forceinline__ unsigned late(const Cursor &c) const {
        const int lane = threadIdx.x & 31, f = feature(c) + (lane >> 2), count = members(c);
        unsigned which = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int m = 2 * (lane & 3) + j;
            if (m >= count) continue;
            if (f < a.hidden && *place(c, m, f) == LATE) which |= (a.gated ? 5u : 1u) << j;
            if (!a.gated && f + 8 < a.hidden && *place(c, m, f + 8) == LATE) which |= 4u << j;
        }
        return which;
    }
    __device__ __forceinline__ int length() const { return a.width; }
    __device__ __forceinline__ float value(const void *x, int k) const {
        return __bfloat162float(static_cast<const __nv_bfloat16 *>(x)[k]);
    }
};

// y from h: block b has columns width * b / grid .. width * (b + 1) / grid - 1,
// `cols` of them, from `at` on, at once.
template <int H>
struct OutJob {
    using M = Matrix<H>;
    const LArgs &a;
    const Lists &l;
    float *sums;  // of a pair's place, COLUMNS each
    int at, cols, kblocks;
    int64_t item_scales;
    __device__ __forceinline__ Cursor cursor(int item) const {
        const int tile = item / l.entries;
        return Cursor{item, item - tile * l.entries, tile, 0};
    }
    __device__ __forceinline__ void next(Cursor &c) const {
        if (++c.entry < l.entries) return;
        c.entry = 0;
        ++c.tile;
    }
    __device__ __forceinline__ const uint8_t *base(const Cursor &c, int g) const {
        return static_cast<const uint8_t *>(a.w2) +
               (l.expert[c.entry] * a.stride2 + static_cast<int64_t>(at + 16 * c.tile + g) * a.ld2) * M::SIZE;
    }
    __device__ __forceinline__ int64_t delta() const { return 8 * a.ld2 * M::SIZE; }
    __device__ __forceinline__ bool there(const Cursor &c, int i, int g) const { return 16 * c.tile + 8 * i + g < cols; }
    __device__ __forceinline__ const float *scales(const Cursor &c) const { return a.s2 + l.expert[c.entry] * item_scales; }
    __device__ __forceinline__ int scale_row(const Cursor &c, int i, int g) const {
        return there(c, i, g) ? (at + 16 * c.tile + 8 * i + g) / SGEMM_FP8_BLOCK_SIZE * kblocks : 0;
    }
    __device__ __forceinline__ int members(const Cursor &c) const { return l.count[c.entry]; }
    __device__ __forceinline__ const void *x(const Cursor &c, int m) const {
        return a.h + l.order[l.begin[c.entry] + m] * a.ldh;
    }
    __device__ __forceinline__ int64_t plane() const { return a.ldh * 2; }
    static constexpr bool ALIGNED = true;
    __device__ __forceinline__ void finish(const Cursor &c, const float (&sum)[4]) const { settle(c, sum, 15); }
    __device__ __forceinline__ void settle(const Cursor &c, const float (&sum)[4], unsigned which) const {
        const int lane = threadIdx.x & 31, count = members(c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = 2 * (lane & 3) + (i & 1);
            if (m < count && (which >> i & 1)) *place(c, i) = sum[i];
        }
    }
    // Of sum i of the lane.
    __device__ __forceinline__ float *place(const Cursor &c, int i) const {
        const int lane = threadIdx.x & 31, m = 2 * (lane & 3) + (i & 1), n = 16 * c.tile + 8 * (i >> 1) + (lane >> 2);
        return sums + (l.begin[c.entry] + m) * COLUMNS + n;
    }
    // Whether one of the thread's share of the block's sums is not finite.
    __device__ __forceinline__ bool any_late() const {
        bool any = false;
        if (l.entries == 0) return false;
        const int all = (l.begin[l.entries - 1] + l.count[l.entries - 1]) * COLUMNS;
        for (int i = threadIdx.x; i < all; i += THREADS) any |= i % COLUMNS < cols && !isfinite(sums[i]);
        return any;
    }
    __device__ __forceinline__ unsigned late(const Cursor &c) const {
        const int lane = threadIdx.x & 31, count = members(c);
        unsigned which = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (2 * (lane & 3) + (i & 1) < count && there(c, i >> 1, lane >> 2) && !isfinite(*place(c, i))) which |= 1u << i;
        return which;
    }
    __device__ __forceinline__ int length() const { return a.hidden; }
    __device__ __forceinline__ float value(const void *x, int k) const {
        const __nv_bfloat16 *h = static_cast<const __nv_bfloat16 *>(x) + k;
        return __bfloat162float(h[0]) + __bfloat162float(h[a.ldh]);
    }
};

// The columns of y that block b of the second kernel makes.
template <int H>
__device__ __forceinline__ OutJob<H> out_job(const LArgs &a, const Lists &l, int b, int blocks, int *end) {
    const int n0 = static_cast<int>(static_cast<int64_t>(a.width) * b / blocks);
    *end = static_cast<int>(static_cast<int64_t>(a.width) * (b + 1) / blocks);
    const int kblocks = (a.hidden + SGEMM_FP8_BLOCK_SIZE - 1) / SGEMM_FP8_BLOCK_SIZE,
              nblocks = (a.width + SGEMM_FP8_BLOCK_SIZE - 1) / SGEMM_FP8_BLOCK_SIZE;
    return OutJob<H>{a, l, reinterpret_cast<float *>(dynamic_smem + SMEM), n0, min(COLUMNS, *end - n0), kblocks,
                     static_cast<int64_t>(nblocks) * kblocks};
}

template <int H, int MATH, bool ANY, class X>
__global__ void __launch_bounds__(THREADS, 1) layer_hidden_kernel(const __grid_constant__ LArgs a) {
    __shared__ Lists l;
    __shared__ int part_of[WARPS];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    build_lists(a, l);
    const int per_tile = a.gated ? 8 : 16;  // features
    const int rows1 = a.gated ? 2 * a.hidden : a.hidden;
    HiddenJob<H, MATH == BF8> job{a, l, 0, per_tile, (a.hidden + per_tile - 1) / per_tile,
                                  (a.width + SGEMM_FP8_BLOCK_SIZE - 1) / SGEMM_FP8_BLOCK_SIZE, 0};
    job.item_scales = static_cast<int64_t>((rows1 + SGEMM_FP8_BLOCK_SIZE - 1) / SGEMM_FP8_BLOCK_SIZE) * job.kblocks;
    const int64_t tiles = static_cast<int64_t>(l.entries) * job.per_entry;
    job.first = static_cast<int>(tiles * blockIdx.x / gridDim.x);
    const int items = static_cast<int>(tiles * (blockIdx.x + 1) / gridDim.x) - job.first;
    sum_tiles<H, MATH, ANY, X>(job, items, a.width, part_of);
    if constexpr (MATH == BF8) {
        __syncthreads();
        if (l.late) sums_again<H>(job, items);
    }
}

template <int H, int MATH, bool ANY>
__global__ void __launch_bounds__(THREADS, 1) layer_out_kernel(const __grid_constant__ LArgs a) {
    __shared__ Lists l;
    __shared__ int part_of[WARPS];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    build_lists(a, l);
    int n1;
    OutJob<H> job = out_job<H>(a, l, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), &n1);
    for (; job.at < n1; job.at += COLUMNS) {
        job.cols = min(COLUMNS, n1 - job.at);
        const int items = a.hidden > 0 ? l.entries * ((job.cols + 15) / 16) : 0;
        sum_tiles<H, MATH, ANY, float>(job, items, a.hidden, part_of);
        __syncthreads();
        if constexpr (MATH == BF8_H) {
            if (__syncthreads_or(items > 0 && job.any_late())) {
                sums_again<H>(job, items);
                __syncthreads();
            }
        }
        for (int i = threadIdx.x; i < a.tokens * COLUMNS; i += THREADS) {
            const int n = i % COLUMNS, token = i / COLUMNS;
            if (n >= job.cols) continue;
            float y = 0.0f;
            for (int j = 0; j < a.top_k && a.hidden > 0; ++j) {
                const int p = token * a.top_k + j, place = l.place[p];
                if (place >= 0) y = fmaf(__ldg(a.weights + p), job.sums[place * COLUMNS + n], y);
            }
            const int64_t to = token * a.ldy + job.at + n;
            if (a.x_type == SGEMM_TYPE_F32)
                static_cast<float *>(a.y)[to] = y;
            else if (a.x_type == SGEMM_TYPE_BF16)
                static_cast<__nv_bfloat16 *>(a.y)[to] = __float2bfloat16_rn(y);
            else
                static_cast<__half *>(a.y)[to] = __float2half_rn(y);
        }
        __syncthreads();
    }
}

constexpr int kMaxDevices = 64;

template <auto KERNEL>
int enqueue_kernel(const LArgs &a, int grid, int smem, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    if (dev.device < 0 || dev.device >= kMaxDevices) return SGEMM_ERR_DEVICE;
    static std::once_flag once[kMaxDevices];
    static cudaError_t err[kMaxDevices];
    std::call_once(once[dev.device],
                   [&] { err[dev.device] = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                            smem_out(MAX_PAIRS)); });
    if (err[dev.device] != cudaSuccess) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, KERNEL, a) != cudaSuccess) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    ++*launches;
    return SGEMM_OK;
}

// Whether all rows start on 16-byte boundaries. Those of 8-bit matrices always do.
template <int H>
bool rows_aligned(const void *w, int64_t ld, int64_t stride) {
    constexpr int64_t per = Matrix<H>::PER;
    return Matrix<H>::FP8 || (reinterpret_cast<uintptr_t>(w) % 16 == 0 && ld % per == 0 && stride % per == 0);
}

// Blocks of the second kernel: one an SM, or about four columns of y each where
// that makes fewer.
inline int out_grid(const LArgs &a, const DeviceInfo &dev) {
    const int most = (a.width + 3) / 4;
    return most < dev.sm_count ? most : dev.sm_count;
}

// Both kernels. HIDDEN, OUT: how their sums are made.
template <int H, int HIDDEN, int OUT, class X>
int launch_layer(const LayerProblem &p, const LArgs &a, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    const bool in = a.x_vector && rows_aligned<H>(p.w1, p.ld1, a.stride1), out = rows_aligned<H>(p.w2, p.ld2, a.stride2);
    const int smem = smem_out(a.pairs);
    int rc = SGEMM_OK;
    if (p.hidden > 0)
        rc = in ? enqueue_kernel<layer_hidden_kernel<H, HIDDEN, false, X>>(a, dev.sm_count, SMEM, dev, stream, launches)
                : enqueue_kernel<layer_hidden_kernel<H, HIDDEN, true, X>>(a, dev.sm_count, SMEM, dev, stream, launches);
    if (rc != SGEMM_OK) return rc;
    if (out) return enqueue_kernel<layer_out_kernel<H, OUT, false>>(a, out_grid(a, dev), smem, dev, stream, launches);
    if constexpr (!Matrix<H>::FP8)
        rc = enqueue_kernel<layer_out_kernel<H, OUT, true>>(a, out_grid(a, dev), smem, dev, stream, launches);
    return rc;
}

}  // namespace

}  // namespace fl
}  // namespace sgemm
