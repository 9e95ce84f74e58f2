// wtconv_clip.h -- launch entry points of the gradient norm and clipping kernels.
#ifndef WTCONV_CLIP_H
#define WTCONV_CLIP_H

#include <hip/hip_runtime.h>

#include "../../../include/wtconv.h"

namespace wtc_clip {

constexpr int64_t kRanges = 8192;   // ranges that the elements are cut into, about
constexpr int64_t kLeast = 8192;    // elements of a range at least
constexpr int64_t kOwnSums = 2560;  // ranges whose sums every workgroup of the clip joins itself
constexpr int64_t kStream = 1 << 24;  // elements from which the outputs are larger than the L2s together
                                      // (414e6 bf16 elements 577 us, with stores past the L2s 548)

// Elements of a range.  A tensor's last range may be shorter, so there are at most
// kRanges + count of them.
inline int64_t range_elems(int64_t elems)
{
    const int64_t r = (elems + kRanges - 1) / kRanges;
    return r < kLeast ? kLeast : (r + 2047) / 2048 * 2048;
}

constexpr int kByValue = 120;  // tensors whose table goes with a launch: 28 bytes each of 4 KB

struct Entry {
    const void *in;
    void *out;
    int64_t elems_type;  // elements * 4 + type
    int64_t first;       // the tensor's first range
};

// fp64 sums of all ranges, and the total of more than kOwnSums; the table of more
// than kByValue tensors.
inline size_t sums_bytes(int64_t count)
{
    return ((size_t)(kRanges + count + 1) * sizeof(double) + 255) / 256 * 256;
}

inline size_t workspace_bytes(int64_t count)
{
    return sums_bytes(count) + (count > kByValue ? ((size_t)count * sizeof(Entry) + 255) / 256 * 256 : 0);
}

}  // namespace wtc_clip

// norm alone (clip false), or norm and the outputs.
hipError_t wtc_launch_clip(const wtconv_tensor_t *t, int64_t count, bool clip, float max_norm, float eps, float *norm,
                           double *parts, hipStream_t stream);

#endif  // WTCONV_CLIP_H
