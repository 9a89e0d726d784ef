// Whether the buffers of a call share memory, from their addresses and strides alone (host code).
#pragma once

#include <stdint.h>

#include <initializer_list>

namespace qlin {

// `rows` rows of `width` bytes, `stride` bytes apart (at least `width`); NULL or empty: nothing.
struct Region {
    const void *at;
    int64_t rows, width, stride;
};

inline Region flat(const void *at, int64_t bytes) { return Region{at, 1, bytes, bytes}; }

// Exact where one of the two is without gaps or both have one stride (columns of one buffer, side by side, do not
// overlap); rows of two strides are taken for apart.
inline bool overlap(Region a, Region b)
{
    if (!a.at || !b.at || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0)
        return false;
    for (Region *r : {&a, &b})
        if (r->stride == r->width || r->rows == 1)
            *r = Region{r->at, 1, (r->rows - 1) * r->stride + r->width, 0};
    // row k of b lies at d + k stride, seen from row 0 of a
    const int64_t d = (int64_t)((uintptr_t)b.at - (uintptr_t)a.at);
    if (a.rows == 1 && b.rows == 1)
        return d < a.width && -d < b.width;
    if (a.rows > 1 && b.rows > 1 && a.stride != b.stride)
        return false;
    const int64_t stride = a.rows > 1 ? a.stride : b.stride;
    // a row of b `k` rows behind one of a meets it for -b.width < d + k stride < a.width; k is 1 - a.rows .. b.rows - 1
    const auto floor_div = [](int64_t n, int64_t by) { return n / by - (n % by < 0 ? 1 : 0); };
    int64_t first = floor_div(-b.width - d, stride) + 1, last = floor_div(a.width - 1 - d, stride);
    first = first > 1 - a.rows ? first : 1 - a.rows;
    last = last < b.rows - 1 ? last : b.rows - 1;
    return first <= last;
}

// The same rows: what a call that works in place takes.
inline bool same(const Region &a, const Region &b)
{
    return a.at == b.at && (a.stride == b.stride || (a.rows == 1 && b.rows == 1));
}

// Whether an output shares memory with an input, or with another output.
inline bool overlaps(std::initializer_list<Region> outputs, std::initializer_list<Region> inputs)
{
    for (const Region *o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Region &i : inputs)
            if (overlap(*o, i))
                return true;
        for (const Region *p = o + 1; p != outputs.end(); ++p)
            if (overlap(*o, *p))
                return true;
    }
    return false;
}

}  // namespace qlin
