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

struct Span {
    const void *p;
    size_t bytes;
};

// Whether one of the outputs overlaps an input or another output (null ones
// and those of no bytes do not).
inline bool any_alias(const Span *in, int nin, const Span *out, int nout)
{
    for (int i = 0; i < nout; ++i) {
        if (!out[i].p || !out[i].bytes) continue;
        for (int j = 0; j < nin; ++j)
            if (in[j].p && in[j].bytes && overlaps2(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return true;
        for (int j = 0; j < i; ++j)
            if (out[j].p && out[j].bytes && overlaps2(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
    }
    return false;
}

inline size_t align256(size_t b) { return (b + 255) / 256 * 256; }

#endif  // WTCONV_CHECK_H
