// Sets of rows as the attention calls get them, and whether two of them overlap (host
// only).
#pragma once

#include <cstdint>

namespace bitlinear {

// Rows of bf16 in memory: n of `width` elements, `stride` (>= width) elements apart.
struct RowSet {
    const void *p;
    int64_t stride, width;
};

// Whether two sets of n rows share an element. Rows of one wide buffer that lie side
// by side do not, though the sets' ranges overlap.
inline bool share_memory(const RowSet &a, const RowSet &b, int64_t n)
{
    using Wide = __int128;
    const Wide a0 = static_cast<Wide>(reinterpret_cast<uintptr_t>(a.p)) / 2;
    const Wide b0 = static_cast<Wide>(reinterpret_cast<uintptr_t>(b.p)) / 2;
    const Wide sa = a.stride, sb = b.stride, last = n - 1;
    if (a0 + last * sa + a.width <= b0 || b0 + last * sb + b.width <= a0)
        return false;
    if (n == 1)
        return true;
    // The first row of b that ends behind the beginning of a's row at `begin`, if it
    // begins ahead of that row's end.
    auto meets = [&](Wide begin) {
        const Wide gap = begin - b0 - b.width;             // >= 0: rows in front of it end there
        const Wide j = gap < 0 ? 0 : gap / sb + 1;
        return j <= last && b0 + j * sb < begin + a.width;
    };
    if (sa != sb) {
        for (Wide i = 0; i <= last; ++i)
            if (meets(a0 + i * sa))
                return true;
        return false;
    }
    // one stride: the sets repeat side by side, so a's first or last row meets b or none
    return meets(a0) || meets(a0 + last * sa);
}

}  // namespace bitlinear
