// Argument checks and dispatch that the operators' C entry points share.
#pragma once

#include <stdint.h>

#include "experts_internal.h"

namespace sgemm {
namespace api {

// Element offsets must fit in int64 bytes with room to spare.
constexpr int64_t kLimit = INT64_C(1) << 58;
// Rows of a product: a tile past the last one still fits 32 bits.
constexpr int64_t kMostRows = INT32_MAX - 1024;

inline bool type_ok(int type) { return type >= SGEMM_TYPE_F32 && type <= SGEMM_TYPE_F16; }

// rows x cols elements of `size` bytes, row stride ld, `items` of them
// `stride` elements apart.
struct Span {
    const void *p;
    int64_t rows, cols, ld, size;
    int64_t items = 1, stride = 0;
    bool empty() const { return rows == 0 || cols == 0 || items == 0; }
    // Sizes that describe memory: strides that hold a row (and an item), a
    // pointer wherever there are elements, offsets within the limit.
    bool ok() const {
        if (rows < 0 || cols < 0 || items < 0 || ld < cols || ld < 1) return false;
        if (rows > 0 && ld > kLimit / rows) return false;
        if (items > 1 && (stride < 0 || stride > kLimit / items)) return false;
        if (empty()) return true;
        if (items > 1 && stride < (rows - 1) * ld + cols) return false;
        return p != nullptr && reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(size) == 0;
    }
    uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
    uintptr_t end() const {
        return begin() + static_cast<uintptr_t>(((items - 1) * stride + (rows - 1) * ld + cols) * size);
    }
    bool overlaps(const Span &o) const { return !empty() && !o.empty() && begin() < o.end() && o.begin() < end(); }
};

inline Span flat(const void *p, int64_t n, int64_t size) { return Span{p, 1, n, n > 0 ? n : 1, size}; }

// Calls f(device, launches) and notes the kernels it enqueued.
template <class F>
int enqueue(F &&f) {
    DeviceInfo dev;
    int rc = current_device(&dev);
    if (rc != SGEMM_OK) return rc;
    int launches = 0;
    rc = f(dev, &launches);
    if (rc == SGEMM_OK) note_launches(launches);
    return rc;
}

}  // namespace api
}  // namespace sgemm
