// A mixture-of-experts layer for a few tokens, in two kernels:
//
//     h[p] = act(W1[e(p)] x[t(p)])              (or act(first half) * second half)
//     y[t] = sum over j of weights[t][j] W2[e] h[t, j]
//
// for at most 512 (token, choice) pairs p. Bound by reading the matrices of the
// experts that are used, once per 16 pairs that share one.
//
// Work. Every block sorts the pairs by expert for itself (a comparison of each
// pair with each, 512 at most) into entries of up to 16 pairs of an expert. First
// kernel: the entries' hidden features in tiles of 16 rows of W1 (8 features and
// their gates), each block a run of tiles. Second kernel: each block some of y's
// columns, at most 16 rows of W2 a time, for every entry, so a token's experts
// meet in one block and are added up in the order of its choices. In a block the
// tiles times the chunks of k are cut evenly among 16 warps; a warp leaves its
// part of a tile in shared memory, and the parts are joined in order.
//
// Arithmetic. 16- and 8-bit matrices go through warp matrix instructions (16 rows
// of the matrix x 8 k x 8 pairs, tf32 in, fp32 sums), in which every 16- and
// 8-bit value is exact; h (24 bits) enters as two terms of 11. With fp32 x sums
// are fp32 multiply-adds (the instruction cuts its running sums: 1.3e-6 of the
// result's norm where multiply-adds leave 0.2e-6). (tcgen05 wants its operands in shared
// memory and 128 rows a tile; here the weights go from global memory to
// registers once and are used once.) Which k a lane holds does not matter as long
// as matrix and x agree, so a lane takes 16 bytes of a row that lie together.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "epilogue.cuh"
#include "experts_common.cuh"
#include "layer_internal.h"

namespace sgemm {
namespace fl {
namespace {

using ex::from_f32;
using ex::to_f32;

constexpr int WARPS = 16, THREADS = 32 * WARPS;
constexpr int MEMBERS = 16;  // pairs of an entry, in sets of 8 columns
constexpr int ROUND = 48;    // tiles of the first kernel whose parts are in shared memory at once
constexpr int PART_FLOATS = (ROUND + WARPS) * 16 * MEMBERS;
static_assert(PART_FLOATS >= (MAX_PAIRS + WARPS * MEMBERS) * 16, "parts of the second kernel");
static_assert(MAX_PAIRS <= THREADS, "a thread a pair");

struct LArgs {
    int pairs, top_k, experts, tokens;
    int activation, gated;
    int width, hidden;
    const void *x;
    int64_t ldx;
    const void *ids;
    int id_bits;
    const float *weights;
    const void *w1;
    int64_t ld1, stride1;
    const float *s1;
    const void *w2;
    int64_t ld2, stride2;
    const float *s2;
    void *y;
    int64_t ldy;
    float *h;
    int64_t ldh;
    int columns_grid;  // blocks of the second kernel
};

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
    if (p == 0) l.entries = all;
    __syncthreads();
    if (used && rank % MEMBERS == 0) {
        const int e = l.entry_at[place];
        l.expert[e] = key;
        l.begin[e] = place;
        l.count[e] = min(MEMBERS, same - rank);
    }
    __syncthreads();
}

// How a matrix is held. PER: values in 16 bytes; LANE_K: values of a row that a
// lane takes in a chunk.
enum Held { F32, BF16, F16, E4M3, E5M2 };
template <int H>
struct Matrix {
    static constexpr int SIZE = H == F32 ? 4 : (H >= E4M3 ? 1 : 2), PER = 16 / SIZE;
    static constexpr int LANE_K = H >= E4M3 ? 16 : 8, CHUNK = 4 * LANE_K;
    static constexpr bool FP8 = H >= E4M3;
    static constexpr int WORDS = LANE_K * SIZE / 4;  // of a row and chunk, in 16-byte loads
    static constexpr int DEPTH = H == F32 ? 2 : 4;   // chunks on their way to a warp: 64 KB an SM
};

__device__ __forceinline__ uint4 load_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ float half_of(uint32_t w, int i, bool bf16) {
    if (bf16) return __uint_as_float(i ? w & 0xFFFF0000u : w << 16);
    return __half2float(__ushort_as_half(static_cast<uint16_t>(i ? w >> 16 : w)));
}

// Two 8-bit values (the low 16 bits of w) in fp32, exactly.
template <int H>
__device__ __forceinline__ void fp8_pair(uint32_t w, float &lo, float &hi) {
    uint32_t h2;
    if (H == E4M3)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(w)));
    else
        h2 = __byte_perm(w, 0, 0x1404);  // E5M2 is the upper half of an fp16
    lo = half_of(h2, 0, false);
    hi = half_of(h2, 1, false);
}

// Values 8 i .. 8 i + 7 of a lane's part of a chunk as fp32. VECTOR: w holds the
// bytes as they lie in memory; otherwise a value a word.
template <int H, bool VECTOR>
__device__ __forceinline__ void unpack8(const uint32_t *w, int i, float (&v)[8]) {
    if (!VECTOR) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t x = w[8 * i + j];
            float unused;
            if (H == F32) v[j] = __uint_as_float(x);
            if (H == BF16 || H == F16) v[j] = half_of(x, 0, H == BF16);
            if (H >= E4M3) fp8_pair<H>(x, v[j], unused);
        }
    } else if (H == F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
    } else if (H == BF16 || H == F16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = half_of(w[j / 2], j & 1, H == BF16);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) fp8_pair<H>(w[2 * i + j / 2] >> (16 * (j & 1)), v[2 * j], v[2 * j + 1]);
    }
}

// The k of value j of lane t of a quad in a chunk that starts at k0.
template <int H, bool VECTOR>
__device__ __forceinline__ int k_of(int k0, int t, int j) {
    if (!VECTOR) return k0 + 4 * j + t;
    if (H == F32) return k0 + 16 * (j >> 2) + 4 * t + (j & 3);
    return k0 + Matrix<H>::LANE_K * t + j;
}

// A lane's values of a row in a chunk; zeros past k = K or where the row is none.
template <int H, bool VECTOR, int N>
__device__ __forceinline__ void load_row(const uint8_t *row, bool there, int k0, int t, int K, uint32_t (&w)[N]) {
    using M = Matrix<H>;
    if (VECTOR) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const int k = k_of<H, true>(k0, t, i * M::PER);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (there && k < K) v = load_stream(row + static_cast<int64_t>(k) * M::SIZE);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int k = k_of<H, false>(k0, t, j);
            w[j] = 0;
            if (there && k < K) {
                const uint8_t *p = row + static_cast<int64_t>(k) * M::SIZE;
                if (M::SIZE == 4) w[j] = __ldg(reinterpret_cast<const uint32_t *>(p));
                if (M::SIZE == 2) w[j] = __ldg(reinterpret_cast<const uint16_t *>(p));
                if (M::SIZE == 1) w[j] = __ldg(p);
            }
        }
    }
}

// Values 8 i .. 8 i + 7 of the lane's k of a chunk from a row of x.
template <int H, bool VECTOR, class X>
__device__ __forceinline__ void load_x8(const X *row, int k0, int t, int i, int K, float (&v)[8]) {
    if (VECTOR) {
        constexpr int RUN = H == F32 ? 4 : 8, PER = 16 / sizeof(X) < RUN ? 16 / sizeof(X) : RUN;
#pragma unroll
        for (int j = 0; j < 8; j += PER) {
            const int k = k_of<H, true>(k0, t, 8 * i + j);
            if (k < K) {
                const ex::Pack<X, PER> p = ex::load_pack<X, PER>(row + k);
#pragma unroll
                for (int m = 0; m < PER; ++m) v[j + m] = to_f32(p.v[m]);
            } else {
#pragma unroll
                for (int m = 0; m < PER; ++m) v[j + m] = 0.0f;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int k = k_of<H, false>(k0, t, 8 * i + j);
            v[j] = k < K ? to_f32(row[k]) : 0.0f;
        }
    }
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], float a0, float a1, float a2, float a3, float b0, float b1) {
    asm(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// The top 11 bits of x, and what is left of it.
__device__ __forceinline__ float take11(float &x) {
    const float hi = __uint_as_float(__float_as_uint(x) & 0xFFFFE000u);
    x = x == hi ? 0.0f : x - hi;
    return hi;
}

// The parts of a block's tiles: a warp's sums of its share of a tile's k.
struct Parts {
    float *at;        // PART_FLOATS
    uint32_t *cover;  // of a tile: the warps that have a part
};

// Share `warp` of `items` x `chunks` chunks of k.
__device__ __forceinline__ int64_t share(int64_t all, int warp) { return all * warp / WARPS; }

// Sums tiles 0 .. items - 1 over k. row_of(item, lo, hi, there_lo, there_hi,
// scale_lo, scale_hi): this lane's two rows of the matrix and their blocks'
// scales; source(item, m): member m's row of x; members(item): their number;
// out(item, warp): where a warp leaves its part, 16 rows (of a stride of STRIDE)
// by members, or the other way round: value (row, member) at row * ROW + member *
// COL.
// TERMS: of x in tf32; 3: fp32 multiply-adds.
template <int H, bool VECTOR, int TERMS, class X, int ROW, int COL, class RowOf, class Source, class Members, class Out>
__device__ __forceinline__ void sum_tiles(int items, int K, const Parts &parts, RowOf &&row_of, Source &&source,
                                          Members &&members, Out &&out) {
    using M = Matrix<H>;
    constexpr int N = VECTOR ? M::WORDS : M::LANE_K, D = VECTOR ? M::DEPTH : 2;
    constexpr bool MMA = TERMS < 3;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int chunks = (K + M::CHUNK - 1) / M::CHUNK;
    const int64_t all = static_cast<int64_t>(items) * chunks;
    const int64_t from = share(all, warp);
    const int mine = static_cast<int>(share(all, warp + 1) - from);
    if (mine == 0) return;

    struct Place {
        int item, chunk;
        const uint8_t *lo, *hi;
        bool there_lo, there_hi;
        const float *s_lo, *s_hi;
    } load{}, use{};
    auto enter = [&](Place &p) { row_of(p.item, p.lo, p.hi, p.there_lo, p.there_hi, p.s_lo, p.s_hi); };
    load.item = static_cast<int>(from / chunks);
    load.chunk = static_cast<int>(from - static_cast<int64_t>(load.item) * chunks);
    enter(load);
    use = load;
    uint32_t lo[D][N], hi[D][N];
    float s_lo[D], s_hi[D];
    auto fetch = [&](int d, bool in) {
        const int k0 = load.chunk * M::CHUNK;
        load_row<H, VECTOR, N>(load.lo, in && load.there_lo, k0, t, K, lo[d]);
        load_row<H, VECTOR, N>(load.hi, in && load.there_hi, k0, t, K, hi[d]);
        if (M::FP8) {
            s_lo[d] = in ? __ldg(load.s_lo + k0 / SGEMM_FP8_BLOCK_SIZE) : 0.0f;
            s_hi[d] = in ? __ldg(load.s_hi + k0 / SGEMM_FP8_BLOCK_SIZE) : 0.0f;
        }
        if (++load.chunk == chunks) {
            load.chunk = 0;
            if (++load.item < items) enter(load);
        }
    };
    // MMA: acc[c]: rows g, g + 8, members 8 c + 2 t and the next. Otherwise
    // acc[c][2 m + r]: member 4 c + m (halves of 16 members), row g + 8 r, this
    // lane's k only.
    float acc[MMA ? 2 : 8][4];
    int count = members(use.item);
    const X *x[MMA ? 2 : MEMBERS];
    auto start = [&] {
        count = members(use.item);
#pragma unroll
        for (int c = 0; c < (MMA ? 2 : 8); ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[c][i] = 0.0f;
        if (MMA) {
#pragma unroll
            for (int c = 0; c < 2; ++c) x[c] = source(use.item, 8 * c + g < count ? 8 * c + g : 0);
        }
    };
    auto finish = [&] {
        float *to = out(use.item, warp);
        if (MMA) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = 8 * c + 2 * t + (i & 1), r = g + 8 * (i >> 1);
                    if (m < count) to[r * ROW + m * COL] = acc[c][i];
                }
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = 2 * c + (i >> 1);
                    if (m >= count) continue;
                    float v = acc[c][i];
                    v += __shfl_xor_sync(0xffffffffu, v, 1);
                    v += __shfl_xor_sync(0xffffffffu, v, 2);
                    if (t == 0) to[(g + 8 * (i & 1)) * ROW + m * COL] = v;
                }
        }
        if (lane == 0) atomicOr(parts.cover + use.item, 1u << warp);
    };
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d, d < mine);
    start();
    for (int i0 = 0; i0 < mine; i0 += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (i0 + d >= mine) break;
            const int k0 = use.chunk * M::CHUNK;
            float part[2][4];  // of a block of an 8-bit matrix
            if (M::FP8 && MMA) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) part[c][i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < M::LANE_K / 8; ++i) {
                float a0[8], a1[8];
                unpack8<H, VECTOR>(lo[d], i, a0);
                unpack8<H, VECTOR>(hi[d], i, a1);
                if (M::FP8 && !MMA) {  // scaled before they are summed
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        a0[j] *= s_lo[d];
                        a1[j] *= s_hi[d];
                    }
                }
                if (MMA) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if (8 * c >= count) break;
                        float b[8];
                        load_x8<H, VECTOR>(x[c], k0, t, i, K, b);
                        auto &sum = M::FP8 ? part[c] : acc[c];
#pragma unroll
                        for (int term = 0; term < TERMS; ++term)
#pragma unroll
                            for (int j = 0; j < 8; j += 2) {
                                const float b0 = TERMS > 1 ? take11(b[j]) : b[j];
                                const float b1 = TERMS > 1 ? take11(b[j + 1]) : b[j + 1];
                                mma_tf32(sum, a0[j], a1[j], a0[j + 1], a1[j + 1], b0, b1);
                            }
                    }
                } else {
#pragma unroll
                    for (int m = 0; m < MEMBERS; ++m) {
                        if (m >= count) break;
                        float b[8];
                        load_x8<H, VECTOR>(source(use.item, m), k0, t, i, K, b);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float &s0 = acc[MMA ? 0 : m / 2][2 * (m & 1)], &s1 = acc[MMA ? 0 : m / 2][2 * (m & 1) + 1];
                            s0 = fmaf(a0[j], b[j], s0);
                            s1 = fmaf(a1[j], b[j], s1);
                        }
                    }
                }
            }
            if (M::FP8 && MMA) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[c][i] = fmaf(part[c][i], i < 2 ? s_lo[d] : s_hi[d], acc[c][i]);
            }
            fetch(d, i0 + d + D < mine);
            if (++use.chunk == chunks || i0 + d + 1 == mine) {
                finish();
                use.chunk = 0;
                if (++use.item < items && i0 + d + 1 < mine) start();
            }
        }
    }
}

extern __shared__ __align__(16) float dynamic_smem[];

// h of the entries' tiles of features.
template <int H, bool VECTOR, int TERMS, class X>
__global__ void __launch_bounds__(THREADS, 1) layer_hidden_kernel(const __grid_constant__ LArgs a) {
    using M = Matrix<H>;
    __shared__ Lists l;
    __shared__ uint32_t cover[ROUND];
    const Parts parts{dynamic_smem, cover};
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    build_lists(a, l);
    const int per_tile = a.gated ? 8 : 16;  // features
    const int per_entry = (a.hidden + per_tile - 1) / per_tile;
    const int64_t tiles = static_cast<int64_t>(l.entries) * per_entry;
    const int64_t end = tiles * (blockIdx.x + 1) / gridDim.x;
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const int kblocks = (a.width + SGEMM_FP8_BLOCK_SIZE - 1) / SGEMM_FP8_BLOCK_SIZE;
    const int rows1 = a.gated ? 2 * a.hidden : a.hidden;
    const int64_t item_scales = static_cast<int64_t>((rows1 + SGEMM_FP8_BLOCK_SIZE - 1) / SGEMM_FP8_BLOCK_SIZE) * kblocks;
    for (int64_t first = tiles * blockIdx.x / gridDim.x; first < end; first += ROUND) {
        const int items = static_cast<int>(min(end - first, static_cast<int64_t>(ROUND)));
        if (threadIdx.x < ROUND) cover[threadIdx.x] = 0;
        __syncthreads();
        sum_tiles<H, VECTOR, TERMS, X, MEMBERS, 1>(
            items, a.width, parts,
            [&](int item, const uint8_t *&lo, const uint8_t *&hi, bool &there_lo, bool &there_hi, const float *&s_lo,
                const float *&s_hi) {
                const int e = static_cast<int>((first + item) / per_entry);
                const int f = static_cast<int>(first + item - static_cast<int64_t>(e) * per_entry) * per_tile + g;
                const int f2 = a.gated ? f : f + 8;
                there_lo = f < a.hidden;
                there_hi = f2 < a.hidden;
                const int r0 = there_lo ? f : 0, r1 = there_hi ? (a.gated ? a.hidden + f : f2) : 0;
                const uint8_t *w = static_cast<const uint8_t *>(a.w1) + l.expert[e] * a.stride1 * M::SIZE;
                lo = w + r0 * a.ld1 * M::SIZE;
                hi = w + r1 * a.ld1 * M::SIZE;
                if (M::FP8) {
                    const float *s = a.s1 + l.expert[e] * item_scales;
                    s_lo = s + static_cast<int64_t>(r0 / SGEMM_FP8_BLOCK_SIZE) * kblocks;
                    s_hi = s + static_cast<int64_t>(r1 / SGEMM_FP8_BLOCK_SIZE) * kblocks;
                }
            },
            [&](int item, int m) {
                const int p = l.order[l.begin[(first + item) / per_entry] + m];
                return static_cast<const X *>(a.x) + p / a.top_k * a.ldx;
            },
            [&](int item) { return l.count[(first + item) / per_entry]; },
            [&](int item, int warp) { return parts.at + (item + warp) * 16 * MEMBERS; });
        __syncthreads();
        // The parts of a tile lie one after the other, from (item + first warp) on.
        for (int i = threadIdx.x; i < items * MEMBERS * per_tile; i += THREADS) {
            const int f = i % per_tile, m = i / per_tile % MEMBERS, item = i / (per_tile * MEMBERS);
            const int e = static_cast<int>((first + item) / per_entry);
            const int feature = static_cast<int>(first + item - static_cast<int64_t>(e) * per_entry) * per_tile + f;
            if (m >= l.count[e] || feature >= a.hidden) continue;
            float v = 0.0f, u = 0.0f;
            for (uint32_t left = cover[item]; left; left &= left - 1) {
                const float *part = parts.at + (item + __ffs(left) - 1) * 16 * MEMBERS + m;
                v += part[f * MEMBERS];
                if (a.gated) u += part[(f + 8) * MEMBERS];
            }
            v = activate(v, a.activation);
            a.h[l.order[l.begin[e] + m] * a.ldh + feature] = a.gated ? v * u : v;
        }
        __syncthreads();
    }
}

// y from h: block b has columns width * b / grid .. width * (b + 1) / grid - 1.
template <int H, bool VECTOR, int TERMS, class Y>
__global__ void __launch_bounds__(THREADS, 1) layer_out_kernel(const __grid_constant__ LArgs a) {
    using M = Matrix<H>;
    __shared__ Lists l;
    __shared__ uint32_t cover[MAX_PAIRS];
    const Parts parts{dynamic_smem, cover};
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    build_lists(a, l);
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const int n0 = static_cast<int>(static_cast<int64_t>(a.width) * blockIdx.x / gridDim.x),
              n1 = static_cast<int>(static_cast<int64_t>(a.width) * (blockIdx.x + 1) / gridDim.x);
    const int rounds = (n1 - n0 + 15) / 16, step = rounds > 0 ? (n1 - n0 + rounds - 1) / rounds : 1;
    const int kblocks = (a.hidden + SGEMM_FP8_BLOCK_SIZE - 1) / SGEMM_FP8_BLOCK_SIZE;
    const int64_t item_scales =
        static_cast<int64_t>((a.width + SGEMM_FP8_BLOCK_SIZE - 1) / SGEMM_FP8_BLOCK_SIZE) * kblocks;
    for (int at = n0; at < n1; at += step) {
        const int cols = min(step, n1 - at);
        for (int i = threadIdx.x; i < l.entries; i += THREADS) cover[i] = 0;
        __syncthreads();
        sum_tiles<H, VECTOR, TERMS, float, 1, 16>(
            l.entries, a.hidden, parts,
            [&](int item, const uint8_t *&lo, const uint8_t *&hi, bool &there_lo, bool &there_hi, const float *&s_lo,
                const float *&s_hi) {
                there_lo = g < cols;
                there_hi = g + 8 < cols;
                const int r0 = there_lo ? at + g : 0, r1 = there_hi ? at + g + 8 : 0;
                const uint8_t *w = static_cast<const uint8_t *>(a.w2) + l.expert[item] * a.stride2 * M::SIZE;
                lo = w + r0 * a.ld2 * M::SIZE;
                hi = w + r1 * a.ld2 * M::SIZE;
                if (M::FP8) {
                    const float *s = a.s2 + l.expert[item] * item_scales;
                    s_lo = s + static_cast<int64_t>(r0 / SGEMM_FP8_BLOCK_SIZE) * kblocks;
                    s_hi = s + static_cast<int64_t>(r1 / SGEMM_FP8_BLOCK_SIZE) * kblocks;
                }
            },
            [&](int item, int m) { return static_cast<const float *>(a.h) + l.order[l.begin[item] + m] * a.ldh; },
            [&](int item) { return l.count[item]; },
            [&](int item, int warp) { return parts.at + (l.begin[item] + MEMBERS * warp) * 16; });
        __syncthreads();
        for (int i = threadIdx.x; i < a.tokens * 16; i += THREADS) {
            const int n = i & 15, token = i >> 4;
            if (n >= cols) continue;
            float y = 0.0f;
            for (int j = 0; j < a.top_k; ++j) {
                const int p = token * a.top_k + j, place = l.place[p];
                if (place < 0) continue;
                float v = 0.0f;
                for (uint32_t left = cover[l.entry_at[place]]; left; left &= left - 1)
                    v += parts.at[(place + MEMBERS * (__ffs(left) - 1)) * 16 + n];
                y = fmaf(__ldg(a.weights + p), v, y);
            }
            static_cast<Y *>(a.y)[token * a.ldy + at + n] = from_f32<Y>(y);
        }
        __syncthreads();
    }
}

constexpr int SMEM = PART_FLOATS * 4;

constexpr int kMaxDevices = 64;

template <auto KERNEL>
int enqueue_kernel(const LArgs &a, int grid, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    static std::once_flag once[kMaxDevices];
    static cudaError_t err[kMaxDevices];
    std::call_once(once[dev.device],
                   [&] { err[dev.device] = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM); });
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
    cfg.dynamicSmemBytes = SMEM;
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

// Rows that 16-byte loads can take.
bool rows_aligned(const void *p, int64_t ld, int64_t stride, int64_t K, int64_t per) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % per == 0 && stride % per == 0 && K % per == 0;
}

template <int H, class X>
int launch_held(const LayerProblem &p, const LArgs &a, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    using M = Matrix<H>;
    constexpr bool WIDE = sizeof(X) == 4;
    constexpr int TERMS1 = WIDE ? 3 : 1, TERMS2 = WIDE ? 3 : 2;
    const int64_t per_x = 16 / static_cast<int64_t>(sizeof(X));
    const int64_t s1 = p.experts > 1 ? p.stride1 : 0, s2 = p.experts > 1 ? p.stride2 : 0;
    const bool v1 = rows_aligned(p.w1, p.ld1, s1, p.width, M::PER) && reinterpret_cast<uintptr_t>(p.x) % 16 == 0 &&
                    (p.tokens == 1 || p.ldx % per_x == 0);
    const bool v2 = rows_aligned(p.w2, p.ld2, s2, p.hidden, M::PER);
    int rc = SGEMM_OK;
    if (p.hidden > 0)
        rc = v1 ? enqueue_kernel<layer_hidden_kernel<H, true, TERMS1, X>>(a, dev.sm_count, dev, stream, launches)
                : enqueue_kernel<layer_hidden_kernel<H, false, TERMS1, X>>(a, dev.sm_count, dev, stream, launches);
    if (rc == SGEMM_OK)
        rc = v2 ? enqueue_kernel<layer_out_kernel<H, true, TERMS2, X>>(a, a.columns_grid, dev, stream, launches)
                : enqueue_kernel<layer_out_kernel<H, false, TERMS2, X>>(a, a.columns_grid, dev, stream, launches);
    return rc;
}

template <class X, int SAME>
int launch_type(const LayerProblem &p, const LArgs &a, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    if (p.held == SGEMM_LAYER_E4M3) return launch_held<E4M3, X>(p, a, dev, stream, launches);
    if (p.held == SGEMM_LAYER_E5M2) return launch_held<E5M2, X>(p, a, dev, stream, launches);
    return launch_held<SAME, X>(p, a, dev, stream, launches);
}

}  // namespace

int layer_launch(const LayerProblem &p, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    if (dev.device < 0 || dev.device >= kMaxDevices) return SGEMM_ERR_DEVICE;
    LArgs a{};
    a.pairs = static_cast<int>(p.tokens * p.top_k);
    a.top_k = static_cast<int>(p.top_k);
    a.experts = static_cast<int>(p.experts);
    a.tokens = static_cast<int>(p.tokens);
    a.activation = p.activation;
    a.gated = p.gated;
    a.width = static_cast<int>(p.width);
    a.hidden = static_cast<int>(p.hidden);
    a.x = p.x;
    a.ldx = p.ldx;
    a.ids = p.ids;
    a.id_bits = p.id_bits;
    a.weights = p.weights;
    a.w1 = p.w1;
    a.ld1 = p.ld1;
    a.stride1 = p.experts > 1 ? p.stride1 : 0;
    a.s1 = p.s1;
    a.w2 = p.w2;
    a.ld2 = p.ld2;
    a.stride2 = p.experts > 1 ? p.stride2 : 0;
    a.s2 = p.s2;
    a.y = p.y;
    a.ldy = p.ldy;
    a.h = p.h;
    a.ldh = h_stride(p.hidden);
    // Four columns of y a block at least.
    const int64_t most = (p.width + 3) / 4;
    a.columns_grid = static_cast<int>(most < dev.sm_count ? most : dev.sm_count);
    if (p.type == SGEMM_TYPE_F32) return launch_type<float, F32>(p, a, dev, stream, launches);
    if (p.type == SGEMM_TYPE_BF16) return launch_type<__nv_bfloat16, BF16>(p, a, dev, stream, launches);
    return launch_type<__half, F16>(p, a, dev, stream, launches);
}

}  // namespace fl
}  // namespace sgemm
