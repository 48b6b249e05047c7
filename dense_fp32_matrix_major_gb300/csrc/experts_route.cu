// Sort of (token, choice) pairs by expert and the row copies that go with it:
// gather, weighted combine and their gradients.
//
// Sort. With key(p) = ids[p] where that is an expert and E otherwise, the
// slot of pair p is
//
//     slot(p) = #{p' : key(p') < key(p)} + #{p' < p : key(p') = key(p)},
//
// a stable counting sort: a histogram, its exclusive sum, and ranks among
// equals. Warps own contiguous ranges of pairs, 32 at a time; equal keys of
// one step find each other by a warp match, so ranks need no atomics and the
// order is the pairs' own.
//
// Row copies. With w the weights, s(t, j) the slots and d the row width
//
//     gather        xs[s(t,j)] = x[t]
//     combine       y[t]  = sum_j w[t,j] h[s(t,j)]
//     its gradient  dh[s(t,j)] = w[t,j] dy[t],  dw[t,j] = <dy[t], h[s(t,j)]>
//
// All three are bound by memory: one thread holds 16 bytes of a token's row
// and goes through the token's choices, so x, dy and every row of h are read
// once and every output is written once, without atomics. Measured with 16384
// tokens x 8 choices of 64 experts, width 2048, bf16 (a plain copy makes 6.8
// TB/s): gather 95 us (6.4 TB/s), combine 103 us (5.9), its gradient 197 us
// (5.8); the sort of the 131072 pairs 17 us, two launches of which the second
// is resident before the first ends and reads nothing until then.
#include <cuda_runtime.h>
#include <stdint.h>

#include "experts_common.cuh"
#include "experts_internal.h"

namespace sgemm {
namespace ex {
namespace {

constexpr int SORT_THREADS = 1024;
constexpr int SORT_MAX_WARPS = SORT_THREADS / 32;
// Counters of one block: one row of experts + 1 per counting warp.
constexpr int SORT_SMEM_INTS = 48 * 1024;
// Pairs that one block sorts alone.
constexpr int64_t SORT_SINGLE = 2048;
// Pairs per block and table entries of the two-kernel form.
constexpr int64_t SORT_PER_BLOCK = 1024;
constexpr int64_t SORT_TABLE = 64 * 1024;
constexpr int64_t SORT_BLOCKS = 152;  // one per SM of a GB300

// Kernels here are launched while the one before them in the stream ends
// (launch_after): they wait for its results, then let the next one in.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
}

template <class Id>
__device__ __forceinline__ int key_of(const Id *ids, int64_t p, int experts) {
    const Id id = __ldg(ids + p);
    return id < 0 || id >= experts ? experts : static_cast<int>(id);
}

// Pairs [begin, end) of block `block` of `blocks`.
__device__ __forceinline__ void block_range(int64_t pairs, int block, int blocks, int64_t *begin, int64_t *end) {
    const int64_t per = ((pairs + blocks - 1) / blocks + 31) / 32 * 32;
    *begin = min(per * block, pairs);
    *end = min(*begin + per, pairs);
}

// Table row `blockIdx.x`: how many pairs of this block have each key.
template <class Id>
__global__ void __launch_bounds__(SORT_THREADS) sort_count_kernel(const Id *ids, int64_t pairs, int experts,
                                                                  int32_t *table) {
    extern __shared__ int32_t count[];
    after_previous();
    for (int e = threadIdx.x; e <= experts; e += SORT_THREADS) count[e] = 0;
    __syncthreads();
    int64_t begin, end;
    block_range(pairs, blockIdx.x, gridDim.x, &begin, &end);
    for (int64_t p = begin + threadIdx.x; p < end; p += SORT_THREADS) atomicAdd(count + key_of(ids, p, experts), 1);
    __syncthreads();
    int32_t *row = table + static_cast<int64_t>(blockIdx.x) * (experts + 1);
    for (int e = threadIdx.x; e <= experts; e += SORT_THREADS) row[e] = count[e];
}

// Exclusive sum over x[0 .. n-1] in place by the whole block; `part` holds 33
// values.
__device__ __forceinline__ void block_exclusive_sum(int32_t *x, int n, int32_t *part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int carry = 0;
    for (int i0 = 0; i0 < n; i0 += SORT_THREADS) {
        const int i = i0 + static_cast<int>(threadIdx.x);
        const int v = i < n ? x[i] : 0;
        int s = v;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += o;
        }
        if (lane == 31) part[warp] = s;
        __syncthreads();
        if (warp == 0) {
            const int w = part[lane];
            int t = w;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int o = __shfl_up_sync(0xffffffffu, t, d);
                if (lane >= d) t += o;
            }
            part[lane] = t - w;
            if (lane == 31) part[32] = t;
        }
        __syncthreads();
        if (i < n) x[i] = carry + part[warp] + s - v;
        carry += part[32];
        __syncthreads();
    }
}

// Calls f(key, p) for the pairs [w0, w1) of a warp in steps of 32, all lanes
// together (key -1 past the end). Up to HELD steps' keys are loaded at once,
// before the first is used.
constexpr int HELD = 8;
template <class Id, class F>
__device__ __forceinline__ void for_keys(const Id *ids, int64_t w0, int64_t w1, int experts, F &&f) {
    const int lane = threadIdx.x & 31;
    for (int64_t p0 = w0; p0 < w1; p0 += 32 * HELD) {
        int key[HELD];
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int64_t p = p0 + 32 * i + lane;
            key[i] = p < w1 ? key_of(ids, p, experts) : -1;
        }
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            if (p0 + 32 * i < w1) f(key[i], p0 + 32 * i + lane);
    }
}

// Slots of this block's pairs. gridDim.x == 1: the whole sort; otherwise the
// table of sort_count_kernel gives the pairs of each key in every block.
// Shared memory: `warps` rows of experts + 1 counters, one row of group
// starts, 33 partial sums.
template <class Id>
__global__ void __launch_bounds__(SORT_THREADS) sort_rank_kernel(const Id *ids, int64_t pairs, int experts, int warps,
                                                                 const int32_t *table, int32_t *offsets,
                                                                 int32_t *order, int32_t *slot) {
    extern __shared__ int32_t smem[];
    const int keys = experts + 1;
    const int blocks = static_cast<int>(gridDim.x), block = static_cast<int>(blockIdx.x);
    int32_t *start = smem + warps * keys, *part = start + keys;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < warps * keys; i += SORT_THREADS) smem[i] = 0;
    for (int i = threadIdx.x; i < keys; i += SORT_THREADS) start[i] = 0;
    __syncthreads();
    // Before the first read of ids, in both forms: the count kernel has waited
    // for what wrote them, but that makes them visible to its grid, not to this.
    after_previous();

    int64_t begin, end;
    block_range(pairs, block, blocks, &begin, &end);
    const int64_t per = ((end - begin + warps - 1) / warps + 31) / 32 * 32;
    const int64_t w0 = min(begin + per * warp, end), w1 = min(w0 + per, end);
    int32_t *mine = smem + warp * keys;
    if (warp < warps) {
        for_keys(ids, w0, w1, experts, [&](int key, int64_t) {
            const unsigned same = __match_any_sync(0xffffffffu, key);
            if (key >= 0 && lane == __ffs(same) - 1) mine[key] += __popc(same);
            __syncwarp();
        });
    }
    __syncthreads();
    // Per key: counts before each warp in the block, and the total over all
    // blocks in `start`.
    if (blocks == 1) {
        for (int e = threadIdx.x; e < keys; e += SORT_THREADS) {
            int sum = 0;
            for (int w = 0; w < warps; ++w) {
                const int v = smem[w * keys + e];
                smem[w * keys + e] = sum;
                sum += v;
            }
            start[e] = sum;
        }
    } else {
        const int parts = max(1, SORT_THREADS / keys);
        // Warp 0's row takes the pairs of earlier blocks on top of the counts
        // before warp 0, which are none: fold it in by adding after the loop.
        for (int i = threadIdx.x; i < parts * keys; i += SORT_THREADS) {
            const int e = i % keys;
            int all = 0, before = 0;
#pragma unroll 8
            for (int b = i / keys; b < blocks; b += parts) {
                const int v = __ldcg(table + static_cast<int64_t>(b) * keys + e);
                all += v;
                before += b < block ? v : 0;
            }
            atomicAdd(start + e, all);
            atomicAdd(smem + e, before);
        }
        __syncthreads();
        // Row 0 holds count(warp 0) + pairs of earlier blocks; their sum is
        // where warp 1 starts, so the exclusive sum needs count(warp 0) alone:
        // recovered from the block's own table row.
        for (int e = threadIdx.x; e < keys; e += SORT_THREADS) {
            int rest = 0;
            for (int w = 1; w < warps; ++w) rest += smem[w * keys + e];
            const int own0 = __ldcg(table + static_cast<int64_t>(block) * keys + e) - rest;
            int sum = smem[e] - own0;
            smem[e] = sum;
            sum += own0;
            for (int w = 1; w < warps; ++w) {
                const int v = smem[w * keys + e];
                smem[w * keys + e] = sum;
                sum += v;
            }
        }
    }
    __syncthreads();
    block_exclusive_sum(start, keys, part);
    if (block == 0)
        for (int e = threadIdx.x; e < keys; e += SORT_THREADS) offsets[e] = start[e];
    if (warp < warps) {
        for_keys(ids, w0, w1, experts, [&](int key, int64_t p) {
            const unsigned same = __match_any_sync(0xffffffffu, key);
            const int leader = __ffs(same) - 1;
            int base = 0;
            if (key >= 0 && lane == leader) {
                base = start[key] + mine[key];
                mine[key] += __popc(same);
            }
            base = __shfl_sync(0xffffffffu, base, leader);
            if (key >= 0) {
                const int s = base + __popc(same & ((1u << lane) - 1u));
                slot[p] = s;
                order[s] = static_cast<int32_t>(p);
            }
            __syncwarp();
        });
    }
}

// ------------------------------------------------------------------ row copies

// Threads of a block: tx along the row, ty tokens.
constexpr int ROW_THREADS = 256;

struct RowArgs {
    int64_t tokens;
    int top_k, experts;
    int64_t vecs;   // vectors in a row
    int64_t pairs;  // tokens * top_k
    const int32_t *slot, *offsets;
};

// Slots below this bound belong to an expert.
__device__ __forceinline__ int kept_end(const RowArgs &a) {
    const int o = __ldg(a.offsets + a.experts);
    return static_cast<int>(max(int64_t(0), min(int64_t(o), a.pairs)));
}

// xs[slot[t][j]] = x[t]: a copy of sizeof(V) bytes a thread, so no types. Four
// vectors of the row at once.
template <class V>
__global__ void __launch_bounds__(ROW_THREADS) gather_kernel(const RowArgs a, const char *x, int64_t ldx, char *xs,
                                                             int64_t ldxs) {
    constexpr int AHEAD = 4;
    after_previous();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (t >= a.tokens) return;
    const int end = kept_end(a);
    const int32_t *slot = a.slot + t * a.top_k;
    const int64_t step = static_cast<int64_t>(gridDim.y) * blockDim.x;
    for (int64_t c0 = static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x; c0 < a.vecs; c0 += AHEAD * step) {
        V v[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (c0 + u * step < a.vecs)
                v[u] = *reinterpret_cast<const V *>(x + t * ldx + (c0 + u * step) * int64_t(sizeof(V)));
        for (int j = 0; j < a.top_k; ++j) {
            const int s = __ldg(slot + j);
            if (static_cast<unsigned>(s) >= a.pairs) continue;
            char *to = xs + s * ldxs;
            const bool kept = s < end;
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (c0 + u * step < a.vecs)
                    *reinterpret_cast<V *>(to + (c0 + u * step) * int64_t(sizeof(V))) = kept ? v[u] : V{};
        }
    }
}

// Choices whose rows a thread has in flight at once.
constexpr int CHOICES = 8;

// FITS: top_k is at most CH, and a thread reads its token's slots once. AHEAD:
// vectors of the row that a thread works on at once, so that CH * AHEAD = 8
// loads are in flight whatever the choices.
template <class T, int N, bool WEIGHTED, int CH, bool FITS>
__global__ void __launch_bounds__(ROW_THREADS) combine_kernel(const RowArgs a, const T *h, int64_t ldh,
                                                              const float *weights, T *y, int64_t ldy) {
    constexpr int AHEAD = CHOICES / CH;
    after_previous();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (t >= a.tokens) return;
    const int end = kept_end(a);
    int s[CH];  // -1: dropped
    float w[CH];
    auto choices = [&](int j0) {  // all slots, then all rows: two waits for memory, not two a choice
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int at = min(j0 + j, a.top_k - 1);
            s[j] = __ldg(a.slot + t * a.top_k + at);
            w[j] = WEIGHTED ? __ldg(weights + t * a.top_k + at) : 1.0f;
            if (j0 + j >= a.top_k || s[j] >= end) s[j] = -1;
        }
    };
    if (FITS) choices(0);
    const int64_t step = static_cast<int64_t>(gridDim.y) * blockDim.x;
    for (int64_t c0 = static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x; c0 < a.vecs; c0 += AHEAD * step) {
        float sum[AHEAD][N] = {};
        for (int j0 = 0; j0 < (FITS ? 1 : a.top_k); j0 += CH) {
            if (!FITS) choices(j0);
            Pack<T, N> rows[AHEAD][CH];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
#pragma unroll
                for (int j = 0; j < CH; ++j)
                    if (s[j] >= 0 && c0 + u * step < a.vecs)
                        rows[u][j] = load_pack<T, N>(h + s[j] * ldh + (c0 + u * step) * N);
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
#pragma unroll
                for (int j = 0; j < CH; ++j) {
                    if (s[j] < 0) continue;
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        sum[u][i] = WEIGHTED ? fmaf(w[j], to_f32(rows[u][j].v[i]), sum[u][i])
                                             : sum[u][i] + to_f32(rows[u][j].v[i]);
                }
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (c0 + u * step >= a.vecs) break;
            Pack<T, N> out;
#pragma unroll
            for (int i = 0; i < N; ++i) out.v[i] = from_f32<T>(sum[u][i]);
            store_pack(y + t * ldy + (c0 + u * step) * N, out);
        }
    }
}

// Sums CHOICES = 8 values over the lanes of a warp: at each of three steps a
// lane keeps half of its values and adds the partner's, so 9 exchanges in
// place of 40. Lane l ends with the value whose number has the lane's bits 16, 8
// and 4 as 4, 2 and 1.
__device__ __forceinline__ float warp_sum8(const float (&v)[CHOICES]) {
    const int lane = threadIdx.x & 31;
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 16;
        const float keep = up ? v[i + 4] : v[i], give = up ? v[i] : v[i + 4];
        a[i] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 8;
        const float keep = up ? a[i + 2] : a[i], give = up ? a[i] : a[i + 2];
        b[i] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
    }
    const bool up = lane & 4;
    float s = (up ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, up ? b[0] : b[1], 4);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    return s + __shfl_xor_sync(0xffffffffu, s, 1);
}

// blockDim.x (a multiple of 32) threads share a token and go over its whole
// row, so the dot products end in the block: in the warp when it has the
// token to itself. CH: choices at once, for as many vectors of the row that
// CH * AHEAD = 8.
template <class T, int N, int CH>
__global__ void __launch_bounds__(ROW_THREADS) combine_grad_kernel(const RowArgs a, const T *dy, int64_t lddy,
                                                                   const T *h, int64_t ldh, const float *weights,
                                                                   T *dh, int64_t lddh, float *dweights) {
    constexpr int AHEAD = CHOICES / CH;
    __shared__ float part[ROW_THREADS / 32][CHOICES];
    after_previous();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool in = t < a.tokens;
    const int end = kept_end(a);
    const int lane = threadIdx.x & 31;
    const int warp = static_cast<int>((threadIdx.y * blockDim.x + threadIdx.x) >> 5);
    const int warps = static_cast<int>(blockDim.x >> 5);  // of one token
    const int64_t step = blockDim.x;
    for (int j0 = 0; j0 < a.top_k; j0 += CH) {
        float dot[CHOICES] = {};
        float w[CH];
        int s[CH];  // -1: past top_k or not a slot; >= end: dropped
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            s[j] = -1;
            w[j] = 0.0f;
            if (!in || j0 + j >= a.top_k) continue;
            s[j] = __ldg(a.slot + t * a.top_k + j0 + j);
            if (s[j] < 0 || s[j] >= a.pairs) s[j] = -1;
            w[j] = __ldg(weights + t * a.top_k + j0 + j);
        }
        if (in) {
            for (int64_t c0 = threadIdx.x; c0 < a.vecs; c0 += AHEAD * step) {
                Pack<T, N> g[AHEAD], rows[AHEAD][CH];
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    const int64_t c = c0 + u * step;
                    if (c >= a.vecs) break;
                    g[u] = load_pack<T, N>(dy + t * lddy + c * N);
#pragma unroll
                    for (int j = 0; j < CH; ++j)
                        if (s[j] >= 0 && s[j] < end) rows[u][j] = load_pack<T, N>(h + s[j] * ldh + c * N);
                }
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    const int64_t c = c0 + u * step;
                    if (c >= a.vecs) break;
#pragma unroll
                    for (int j = 0; j < CH; ++j) {
                        if (s[j] < 0) continue;
                        Pack<T, N> out;
                        if (s[j] < end) {
#pragma unroll
                            for (int i = 0; i < N; ++i) {
                                dot[j] = fmaf(to_f32(g[u].v[i]), to_f32(rows[u][j].v[i]), dot[j]);
                                out.v[i] = from_f32<T>(w[j] * to_f32(g[u].v[i]));
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < N; ++i) out.v[i] = from_f32<T>(0.0f);
                        }
                        store_pack(dh + s[j] * lddh + c * N, out);
                    }
                }
            }
        }
        const float d = warp_sum8(dot);
        const int j = ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
        if (warps == 1) {
            if (in && (lane & 3) == 0 && j < CH && j0 + j < a.top_k) dweights[t * a.top_k + j0 + j] = d;
            continue;
        }
        if ((lane & 3) == 0) part[warp][j] = d;
        __syncthreads();
        if (in && threadIdx.x < CH && j0 + static_cast<int>(threadIdx.x) < a.top_k) {
            float sum = 0.0f;
            for (int i = 0; i < warps; ++i) sum += part[threadIdx.y * warps + i][threadIdx.x];
            dweights[t * a.top_k + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
}

// Largest power of two (at most 16) that divides every address and row
// stride, in bytes.
int vector_bytes(int64_t size, int64_t width, const void *p0, int64_t ld0, const void *p1, int64_t ld1,
                 const void *p2 = nullptr, int64_t ld2 = 0) {
    const uint64_t all = reinterpret_cast<uint64_t>(p0) | reinterpret_cast<uint64_t>(p1) |
                         reinterpret_cast<uint64_t>(p2) |
                         static_cast<uint64_t>((width | ld0 | ld1 | ld2) * size) | 16u;
    return static_cast<int>(all & (~all + 1));
}

// Block shape: tx threads along a row of `vecs` vectors, the smallest power
// of two from 32 to 256 that covers it.
dim3 row_block(int64_t vecs) {
    unsigned tx = 32;
    while (tx < ROW_THREADS && tx < vecs) tx *= 2;
    return dim3(tx, ROW_THREADS / tx);
}

// A warp per token where that fills the GPU: slots are read once a token, dot
// products end in the warp, and its loads of several rows at once keep it busy.
dim3 token_block(const Route &r, int64_t vecs, const DeviceInfo &dev) {
    return r.tokens >= 16 * dev.sm_count ? dim3(32, ROW_THREADS / 32) : row_block(vecs);
}

// One block per blockDim.y tokens and up to 64 pieces of a row.
bool row_grid(const Route &r, int64_t vecs, dim3 block, bool split_row, dim3 *grid) {
    const int64_t x = (r.tokens + block.y - 1) / block.y;
    int64_t y = split_row ? (vecs + block.x - 1) / block.x : 1;
    if (y > 64) y = 64;
    if (x > INT32_MAX) return false;
    *grid = dim3(static_cast<unsigned>(x), static_cast<unsigned>(y));
    return true;
}

RowArgs row_args(const Route &r, int64_t vecs) {
    return RowArgs{r.tokens, static_cast<int>(r.top_k), static_cast<int>(r.experts), vecs, r.tokens * r.top_k,
                   r.slot,   r.offsets};
}

// Blocks for every SM and more.
bool many(dim3 grid, const DeviceInfo &dev) { return int64_t(grid.x) * grid.y >= 2 * dev.sm_count; }

// A launch that may begin while the kernel before it in the stream ends: its
// blocks are resident by then. It takes the host about 1 us more than a plain
// launch, so small grids, whose calls the host bounds, are launched plainly. Sort
// and gather of 16384 tokens x 8: 108 us, 113 plainly; of 4 tokens x 2: 28.9 and
// 26.7 us.
template <class... P, class... A>
int launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool overlap,
                 int *launches, A... args) {
    if (!overlap) {
        kernel<<<grid, block, smem, stream>>>(static_cast<P>(args)...);
        if (cudaGetLastError() != cudaSuccess) return SGEMM_ERR_LAUNCH;
        ++*launches;
        return SGEMM_OK;
    }
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    ++*launches;
    return SGEMM_OK;
}

template <class Id>
int sort_typed(const Id *ids, int64_t pairs, int experts, int32_t *offsets, int32_t *order, int32_t *slot,
               int32_t *workspace, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    if (dev.device < 0 || dev.device >= 64) return SGEMM_ERR_DEVICE;
    const int keys = experts + 1;
    const int table_blocks = sort_blocks(pairs, experts);
    const int blocks = table_blocks > 0 ? table_blocks : 1;
    const int64_t per = (pairs + blocks - 1) / blocks;
    // Two steps of 32 pairs per warp before another warp counts.
    int warps = static_cast<int>((per + 63) / 64);
    const int fit = (SORT_SMEM_INTS - keys - 33) / keys;
    if (warps > fit) warps = fit;
    if (warps > SORT_MAX_WARPS) warps = SORT_MAX_WARPS;
    if (warps < 1) warps = 1;
    const size_t smem = static_cast<size_t>(warps * keys + keys + 33) * sizeof(int32_t);
    if (smem > 48 * 1024 && cudaFuncSetAttribute(sort_rank_kernel<Id>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 SORT_SMEM_INTS * 4) != cudaSuccess) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    if (table_blocks > 0) {
        const int rc = launch_after(sort_count_kernel<Id>, dim3(blocks), dim3(SORT_THREADS), keys * sizeof(int32_t),
                                    stream, blocks >= dev.sm_count / 2, launches, ids, pairs, experts, workspace);
        if (rc != SGEMM_OK) return rc;
    }
    return launch_after(sort_rank_kernel<Id>, dim3(blocks), dim3(SORT_THREADS), smem, stream, table_blocks > 0,
                        launches, ids, pairs, experts, warps, workspace, offsets, order, slot);
}

template <class T, int N, bool WEIGHTED>
int combine_typed(const Route &r, const void *h, int64_t ldh, const float *weights, void *y, int64_t ldy,
                  const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    const int64_t vecs = r.width / N;
    const dim3 block = token_block(r, vecs, dev);
    dim3 grid;
    if (!row_grid(r, vecs, block, block.x > 32, &grid)) return SGEMM_ERR_UNSUPPORTED;
    const RowArgs a = row_args(r, vecs);
    const T *in = static_cast<const T *>(h);
    T *out = static_cast<T *>(y);
    auto kernel = r.top_k <= 2         ? combine_kernel<T, N, WEIGHTED, 2, true>
                  : r.top_k <= 4       ? combine_kernel<T, N, WEIGHTED, 4, true>
                  : r.top_k <= CHOICES ? combine_kernel<T, N, WEIGHTED, CHOICES, true>
                                       : combine_kernel<T, N, WEIGHTED, CHOICES, false>;
    return launch_after(kernel, grid, block, 0, stream, many(grid, dev), launches, a, in, ldh, weights, out, ldy);
}

template <class T, int N>
int combine_grad_typed(const Route &r, const void *dy, int64_t lddy, const void *h, int64_t ldh,
                       const float *weights, void *dh, int64_t lddh, float *dweights, const DeviceInfo &dev,
                       cudaStream_t stream, int *launches) {
    const int64_t vecs = r.width / N;
    const dim3 block = token_block(r, vecs, dev);
    dim3 grid;
    if (!row_grid(r, vecs, block, false, &grid)) return SGEMM_ERR_UNSUPPORTED;
    const RowArgs a = row_args(r, vecs);
    const T *g = static_cast<const T *>(dy), *in = static_cast<const T *>(h);
    T *out = static_cast<T *>(dh);
    auto kernel = r.top_k <= 2   ? combine_grad_kernel<T, N, 2>
                  : r.top_k <= 4 ? combine_grad_kernel<T, N, 4>
                                 : combine_grad_kernel<T, N, CHOICES>;
    return launch_after(kernel, grid, block, 0, stream, many(grid, dev), launches, a, g, lddy, in, ldh, weights, out,
                        lddh, dweights);
}

// f(T{}, N) for the row type and the values a thread moves at once.
template <class F>
int for_type(int type, int bytes, F &&f) {
    if (type == SGEMM_TYPE_F32) {
        if (bytes == 16) return f(float{}, std::integral_constant<int, 4>{});
        if (bytes == 8) return f(float{}, std::integral_constant<int, 2>{});
        return f(float{}, std::integral_constant<int, 1>{});
    }
    if (type == SGEMM_TYPE_BF16) {
        if (bytes == 16) return f(__nv_bfloat16{}, std::integral_constant<int, 8>{});
        if (bytes >= 4) return f(__nv_bfloat16{}, std::integral_constant<int, 2>{});
        return f(__nv_bfloat16{}, std::integral_constant<int, 1>{});
    }
    if (bytes == 16) return f(__half{}, std::integral_constant<int, 8>{});
    if (bytes >= 4) return f(__half{}, std::integral_constant<int, 2>{});
    return f(__half{}, std::integral_constant<int, 1>{});
}

}  // namespace

int sort_blocks(int64_t pairs, int64_t experts) {
    if (pairs <= SORT_SINGLE) return 0;
    int64_t b = (pairs + SORT_PER_BLOCK - 1) / SORT_PER_BLOCK;
    const int64_t table = SORT_TABLE / (experts + 1);
    if (b > table) b = table;
    if (b > SORT_BLOCKS) b = SORT_BLOCKS;
    return b < 2 ? 2 : static_cast<int>(b);
}

int sort_launch(const void *ids, int id_bits, int64_t pairs, int64_t experts, int32_t *offsets, int32_t *order,
                int32_t *slot, int32_t *workspace, const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    const int e = static_cast<int>(experts);
    if (id_bits == 64)
        return sort_typed(static_cast<const int64_t *>(ids), pairs, e, offsets, order, slot, workspace, dev, stream,
                          launches);
    return sort_typed(static_cast<const int32_t *>(ids), pairs, e, offsets, order, slot, workspace, dev, stream,
                      launches);
}

int gather_launch(int type, const Route &r, const void *x, int64_t ldx, void *xs, int64_t ldxs, const DeviceInfo &dev,
                  cudaStream_t stream, int *launches) {
    const int64_t size = type_size(type);
    const int vb = vector_bytes(size, r.width, x, ldx, xs, ldxs);
    const int64_t vecs = r.width * size / vb;
    const dim3 block = token_block(r, vecs, dev);
    dim3 grid;
    if (!row_grid(r, vecs, block, block.x > 32, &grid)) return SGEMM_ERR_UNSUPPORTED;
    const RowArgs a = row_args(r, vecs);
    const char *in = static_cast<const char *>(x);
    char *out = static_cast<char *>(xs);
    auto kernel = vb == 16  ? gather_kernel<uint4>
                  : vb == 8 ? gather_kernel<uint2>
                  : vb == 4 ? gather_kernel<uint32_t>
                            : gather_kernel<uint16_t>;
    return launch_after(kernel, grid, block, 0, stream, many(grid, dev), launches, a, in, ldx * size, out, ldxs * size);
}

int combine_launch(int type, const Route &r, const void *h, int64_t ldh, const float *weights, void *y, int64_t ldy,
                   const DeviceInfo &dev, cudaStream_t stream, int *launches) {
    return for_type(type, vector_bytes(type_size(type), r.width, h, ldh, y, ldy), [&](auto t, auto n) {
        using T = decltype(t);
        constexpr int N = decltype(n)::value;
        return weights ? combine_typed<T, N, true>(r, h, ldh, weights, y, ldy, dev, stream, launches)
                       : combine_typed<T, N, false>(r, h, ldh, weights, y, ldy, dev, stream, launches);
    });
}

int combine_grad_launch(int type, const Route &r, const void *dy, int64_t lddy, const void *h, int64_t ldh,
                        const float *weights, void *dh, int64_t lddh, float *dweights, const DeviceInfo &dev,
                        cudaStream_t stream, int *launches) {
    return for_type(type, vector_bytes(type_size(type), r.width, dy, lddy, h, ldh, dh, lddh), [&](auto t, auto n) {
        return combine_grad_typed<decltype(t), decltype(n)::value>(r, dy, lddy, h, ldh, weights, dh, lddh, dweights,
                                                                   dev, stream, launches);
    });
}

}  // namespace ex
}  // namespace sgemm
