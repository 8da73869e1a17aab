// overlap.hpp -- whether the memory of two arguments overlaps, rows with strides
// included: column slices of one buffer interleave and do not.  Host code only.
#pragma once

#include <cstdint>

namespace iqk {

// `rows` rows of `width` bytes, `ld` bytes apart (0 or less than a width apart
// allowed); [lo, hi) is what they span.
struct Region {
    __int128 lo, hi;
    int64_t rows;
    __int128 ld, width;
};

inline Region region(const void* p, int64_t rows, int64_t cols, int64_t ld, int bytes)
{
    if (!p || rows < 1 || cols < 1) return {0, 0, 0, 0, 0};
    // Sizes that were checked stay below 2^61 values, and the sums below 2^127.
    const __int128 lo = reinterpret_cast<uintptr_t>(p), wide = ld;
    Region r = {lo, lo + ((rows - 1) * wide + cols) * bytes, rows, wide * bytes,
                (__int128)cols * bytes};
    if (rows == 1 || r.ld <= r.width) {           // no gaps: one row
        r.rows = 1;
        r.width = r.hi - r.lo;
    }
    return r;
}

inline Region array(const void* p, int64_t count, int bytes) { return region(p, 1, count, count, bytes); }

// Whether some row [start + i * ld, + width), i = 0..rows-1, meets [lo, hi).
inline bool rows_meet(__int128 start, __int128 rows, __int128 ld, __int128 width, __int128 lo,
                      __int128 hi)
{
    // The first row that ends beyond lo.
    const __int128 before = lo - start - width;
    const __int128 i = before < 0 || ld == 0 ? 0 : before / ld + 1;
    return i < rows && start + i * ld < hi && start + i * ld + width > lo;
}

inline bool overlap(const Region& a, const Region& b)
{
    if (a.lo >= b.hi || b.lo >= a.hi) return false;
    const Region &few = a.rows <= b.rows ? a : b, &many = a.rows <= b.rows ? b : a;
    // With one stride only the difference of the rows' numbers counts.
    if (few.rows > 1 && few.ld == many.ld)
        return rows_meet(many.lo - (few.rows - 1) * few.ld, (__int128)many.rows + few.rows - 1,
                         many.ld, many.width, few.lo, few.lo + few.width);
    for (int64_t i = 0; i < few.rows; ++i) {
        const __int128 lo = few.lo + i * few.ld;
        if (rows_meet(many.lo, many.rows, many.ld, many.width, lo, lo + few.width)) return true;
    }
    return false;
}

// Whether an output overlaps an input or another output.
template <int kOut, int kIn>
inline bool overlaps(const Region (&out)[kOut], const Region (&in)[kIn])
{
    for (int i = 0; i < kOut; ++i) {
        for (int j = 0; j < kIn; ++j)
            if (overlap(out[i], in[j])) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return true;
    }
    return false;
}

}  // namespace iqk
