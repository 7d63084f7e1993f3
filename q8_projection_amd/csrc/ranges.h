// ranges.h -- address checks of the decode-step entry points (host code).
#pragma once

#include <stdint.h>

namespace q8 {

inline bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
    const void *p;  // null: nothing
    int64_t bytes;
};

inline bool overlaps(const Range &a, const Range &b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + static_cast<uintptr_t>(b.bytes) && b0 < a0 + static_cast<uintptr_t>(a.bytes);
}

}  // namespace q8
