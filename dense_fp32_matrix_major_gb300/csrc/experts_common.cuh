// Device-side helpers of the mixture-of-experts operators: row types, vector
// loads and stores, and group bounds.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace sgemm {
namespace ex {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// Rounds to nearest even.
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
    return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) {
    return __float2half_rn(x);
}

// N values loaded and stored at once (N * sizeof(T) is 2 .. 16 bytes, the
// address a multiple of it).
template <class T, int N>
struct alignas(sizeof(T) * N) Pack {
    T v[N];
};

template <class T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const T *p) {
    return *reinterpret_cast<const Pack<T, N> *>(p);
}

template <class T, int N>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, N> &x) {
    *reinterpret_cast<Pack<T, N> *>(p) = x;
}

// First row of group e (e = experts: one past the last group's end), limited
// to 0 .. rows; group 0 starts at row 0 whatever offsets[0] holds.
__device__ __forceinline__ int group_start(const int32_t *offsets, int e, int rows) {
    if (e == 0) return 0;
    const int o = __ldg(offsets + e);
    return o < 0 ? 0 : (o > rows ? rows : o);
}

// A run of rows [begin, end) of group `group` (group = experts: rows outside
// every group).
struct RowTile {
    int group, begin, end;
};

// Tile `tile` of the rows cut into tiles of `size` rows that do not cross
// groups, groups in order and the rows past the last group as one more; group
// = -1 when there are fewer tiles. Called by a full warp: 32 groups a step.
__device__ __forceinline__ RowTile row_tile_of(const int32_t *offsets, int experts, int rows, int size, int tile) {
    const int lane = static_cast<int>(threadIdx.x & 31);
    int base = 0;
    for (int e0 = 0; e0 <= experts; e0 += 32) {
        const int e = e0 + lane;
        const int begin = e <= experts ? group_start(offsets, e, rows) : 0;
        const int end = e < experts ? max(begin, group_start(offsets, e + 1, rows)) : (e == experts ? rows : 0);
        const int tiles = (end - begin + size - 1) / size;
        int sum = tiles;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += o;
        }
        const unsigned has = __ballot_sync(0xffffffffu, tile < base + sum);
        if (has) {
            const int src = __ffs(has) - 1;
            const int first = __shfl_sync(0xffffffffu, base + sum - tiles, src);
            const int b = __shfl_sync(0xffffffffu, begin, src), f = __shfl_sync(0xffffffffu, end, src);
            const int at = b + (tile - first) * size;
            return RowTile{e0 + src, at, min(at + size, f)};
        }
        base += __shfl_sync(0xffffffffu, sum, 31);
    }
    return RowTile{-1, 0, 0};
}

// The tiles of C of one product per group: rows of C (C[s] = A[s] op(B[e]))
// or one matrix per group (wgrad, C[e] = A_e^T B_e).
struct GroupTiles {
    const int32_t *offsets;
    int rows, experts;
    int64_t M, K;          // wgrad: rows of a matrix; otherwise the summed length
    int tiles_m, tiles_n;  // tiles_m: wgrad only
    int split;             // wgrad: slices of each group's rows, of whole k-blocks but the last
};

// One tile: rows [row0, row_end) of C (of the group's matrix in wgrad; at most
// a tile of them) from column n0 on, summed over k_blocks k-blocks; in wgrad
// those are the k_rows rows of A and B from k0 on, and group counts the slices of
// all groups. group = experts: rows of C outside every group, nothing to sum.
struct GroupTile {
    int group, row0, row_end, n0, k0, k_rows, k_blocks;
};

// Calls f(tile) for the tiles (TM x TN, k-blocks of TK) of worker `index` of
// `count`, groups in order, columns before rows, round robin. Every thread of
// a worker walks the same sequence. EVEN > 0: a group's rows are spread evenly
// over its tiles, in multiples of EVEN rows, and row_end is the tile's;
// otherwise every tile but the last has TM rows, and row_end is the group's.
template <bool WGRAD, int TM, int TN, int TK, int EVEN = 0, class F>
__device__ __forceinline__ void for_each_group_tile(const GroupTiles &a, volatile int *abort_flag, int index, int count,
                                                    F &&f) {
    if (WGRAD) {
        const int per = a.tiles_m * a.tiles_n;
        const int64_t total = static_cast<int64_t>(per) * a.experts * a.split;
        for (int64_t u = index; u < total; u += count) {
            if (*abort_flag) return;
            const int item = static_cast<int>(u / per), r = static_cast<int>(u - static_cast<int64_t>(item) * per);
            const int e = a.split > 1 ? item / a.split : item;
            int begin = group_start(a.offsets, e, a.rows);
            int end = max(begin, group_start(a.offsets, e + 1, a.rows));
            if (a.split > 1) {
                const int each = ((end - begin + TK - 1) / TK + a.split - 1) / a.split * TK;
                const int64_t first = begin + static_cast<int64_t>(item - e * a.split) * each;
                begin = static_cast<int>(min(static_cast<int64_t>(end), first));
                end = min(end - begin, each) + begin;
            }
            f(GroupTile{item, r / a.tiles_n * TM, static_cast<int>(a.M), r % a.tiles_n * TN, begin, end - begin,
                        (end - begin + TK - 1) / TK});
        }
    } else {
        const int k_blocks = static_cast<int>((a.K + TK - 1) / TK);
        int e = 0, begin = 0, base = 0;
        int next = group_start(a.offsets, 1, a.rows);
        int end = max(begin, next);
        int tiles = (end - begin + TM - 1) / TM;
        for (int64_t u = index;; u += count) {
            if (*abort_flag) return;
            const int rt = static_cast<int>(u / a.tiles_n);
            while (rt >= base + tiles) {
                if (e == a.experts) return;
                base += tiles;
                ++e;
                begin = next;
                next = e < a.experts ? group_start(a.offsets, e + 1, a.rows) : a.rows;
                end = max(begin, next);
                tiles = (end - begin + TM - 1) / TM;
            }
            const int n0 = static_cast<int>(u % a.tiles_n) * TN, kb = e < a.experts ? k_blocks : 0;
            if (EVEN > 0) {
                constexpr int STEP = EVEN > 0 ? EVEN : 1;
                const int each = ((end - begin + tiles - 1) / tiles + STEP - 1) / STEP * STEP;
                const int row0 = min(begin + (rt - base) * each, end);
                f(GroupTile{e, row0, min(row0 + each, end), n0, 0, 0, row0 < end ? kb : 0});
            } else {
                f(GroupTile{e, begin + (rt - base) * TM, end, n0, 0, 0, kb});
            }
        }
    }
}

}  // namespace ex
}  // namespace sgemm
