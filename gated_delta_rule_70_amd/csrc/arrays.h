// Host-side checks of the arrays that calls are given: where they lie, whether two share bytes.
#pragma once

#include <stdint.h>

#include "gdr.h"

namespace gdr {

// The bytes of an array of evenly spaced rows.
struct Range {
    uintptr_t lo, hi;        // [lo, hi), from the first value to the last
    uintptr_t width, apart;  // of a row, and from one to the next (0: one row)
};

// The array of `rows` rows of `cols` values, `stride` apart.  False where that passes 2^62.
inline bool range_of(const void* p, int64_t rows, int64_t cols, int64_t stride, int64_t elt, Range* r) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    *r = Range{lo, lo, 0, 0};
    if (!p || rows < 1) return true;
    constexpr int64_t lim = int64_t(1) << 62;
    if (rows > 1 && stride > (lim / elt - cols) / (rows - 1)) return false;
    r->hi = lo + static_cast<uintptr_t>(((rows - 1) * stride + cols) * elt);
    r->width = static_cast<uintptr_t>(cols * elt);
    r->apart = rows > 1 ? static_cast<uintptr_t>(stride * elt) : 0;
    return r->hi >= lo;
}

// Whether two arrays share bytes.  Those with rows equally far apart may be column ranges of one wider
// array, one array's rows between the other's; of any others that cross, it is taken that they do.
inline bool overlap(const Range& a, const Range& b) {
    if (!(a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi)) return false;
    if (a.apart == 0 || a.apart != b.apart) return true;
    const Range &first = a.lo < b.lo ? a : b, &second = a.lo < b.lo ? b : a;
    const uintptr_t at = (second.lo - first.lo) % a.apart;  // where second's rows begin, from first's
    return at < first.width || second.width > a.apart - at;
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool known_dtype(int32_t t) { return t == GDR_BF16 || t == GDR_F32; }

inline int64_t elt_of(int32_t t) { return t == GDR_F32 ? 4 : 2; }

}  // namespace gdr
