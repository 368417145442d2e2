// tg_cache_internal.h -- host-side argument checks shared by the cache operators
// (not part of the C ABI).
#pragma once

#include <cstddef>
#include <cstdint>
#include <initializer_list>

namespace tgc {

constexpr int64_t kInt32 = int64_t(1) << 31;

inline bool misaligned(const void *p, uintptr_t to)
{
    return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0;
}

// A range of device memory, from its first byte to the last that is reached.
struct Range {
    const void *p;
    size_t bytes;
};

inline bool overlap(const Range &a, const Range &b)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

// Bytes from the first element of a strided 16-bit tensor to the end of its
// last row: extents (at least 1) with their strides in elements, then a
// contiguous row.  Saturates at half the address space.
struct Dim {
    int64_t n, stride;
};

inline size_t extent(std::initializer_list<Dim> dims, int64_t row)
{
    unsigned __int128 e = static_cast<unsigned __int128>(row);
    for (const Dim &d : dims)
        e += static_cast<unsigned __int128>(d.n - 1) * static_cast<unsigned __int128>(d.stride);
    e *= 2;
    const unsigned __int128 most = static_cast<unsigned __int128>(1) << 63;
    return static_cast<size_t>(e < most ? e : most);
}

// log2 of a page size the cache operators take, else -1.
inline int page_shift_of(int64_t page_size)
{
    for (int s = 3; s <= 8; ++s)
        if (page_size == (int64_t(1) << s)) return s;
    return -1;
}

}  // namespace tgc
