// wtconv_check.h -- small helpers of the entry points' argument checks.
#ifndef WTCONV_CHECK_H
#define WTCONV_CHECK_H

#include <cstddef>
#include <cstdint>

inline bool overlaps2(const void *a, size_t abytes, const void *b, size_t bbytes)
{
    const char *pa = (const char *)a, *pb = (const char *)b;
    return pa < pb + bbytes && pb < pa + abytes;
}

inline bool overlaps(const void *a, const void *b, size_t bytes) { return overlaps2(a, bytes, b, bytes); }

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

inline bool aligned_to(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline size_t align256(size_t b) { return (b + 255) / 256 * 256; }

#endif  // WTCONV_CHECK_H
