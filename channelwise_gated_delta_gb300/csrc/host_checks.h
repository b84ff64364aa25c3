// host_checks.h -- argument checks shared by the C entries (host side).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace gdr {

inline bool supported_dim(int d) { return d == 32 || d == 64 || d == 128; }
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
inline Range range_of(const void *p, size_t bytes) {
    return Range{(uintptr_t)p, (uintptr_t)p + bytes};
}
inline bool overlap(Range a, Range b) {
    return a.lo != a.hi && b.lo != b.hi && a.lo < b.hi && b.lo < a.hi;
}
// Whether an output shares memory with one of n other arguments.
inline bool overlaps_any(Range out, const Range *others, int n) {
    for (int i = 0; i < n; ++i)
        if (overlap(out, others[i])) return true;
    return false;
}

}  // namespace gdr
