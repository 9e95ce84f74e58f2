// wtconv_norm.h -- plan and launch entry points of the group norm kernels.
#ifndef WTCONV_NORM_H
#define WTCONV_NORM_H

#include <hip/hip_runtime.h>

#include "../../../include/wtconv.h"

namespace wtc_norm {

constexpr int kThreads = 256;     // a workgroup of the three-launch form
constexpr int kOneThreads = 512;  // of the one-launch form
constexpr int kMaxBlock = 512;    // channels of a workgroup
constexpr int kOwnSums = 16;      // ranges' moments that a lane joins in the elementwise pass
// Values of a channel that a thread sums at most: in chains that it joins; and
// in one chain, where it sums several channels: moments along channels and tiles,
// and the backward sums along channels (16x256x256x256 fp16 483 us, with 96 of
// them, which is 2731 workgroups in place of 2048, 503).
constexpr int kMostValues = 2048, kMostUnjoined = 96, kMostBackward = 128;

// How a pass over (N, C, H W) is shared out: workgroups of `cb` channels and
// `ppw` pixels of one image, `blocks` and `splits` of them for each image,
// `lanes` threads side by side along memory.
struct Geometry {
    int c, hw, groups, per, act;
    int cb, blocks, ppw, splits, lanes;
    int vlast;      // tiles: channels of an access to the tensor that lies channels last
    bool stream;    // the tensors are larger than the L2s together
    int64_t count;  // workgroups of all images
};

// (count, mean, sum of squared differences) of a set of values.
struct Moments {
    float n, mean, m2;
};

__device__ inline Moments join(const Moments &a, const Moments &b)
{
    // an empty set's own zeros must not meet a mean whose square overflows
    if (b.n == 0.f) return a;
    if (a.n == 0.f) return b;
    const float n = a.n + b.n;
    const float w = b.n / n, d = b.mean - a.mean;
    return Moments{n, fmaf(d, w, a.mean), a.m2 + b.m2 + d * d * a.n * w};
}

// Pixels of range s.
__device__ inline int pixels(const Geometry &g, int s)
{
    const int p = g.hw - s * g.ppw;
    return p < g.ppw ? p : g.ppw;
}

// s of all lanes of a wave, joined in a fixed order, on every lane.
template <typename S, typename J>
__device__ inline S join_wave(S s, J join2)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        S q;
        const float *a = (const float *)&s;
        float *b = (float *)&q;
#pragma unroll
        for (int w = 0; w < (int)(sizeof(S) / 4); ++w) b[w] = __shfl_xor(a[w], o);
        s = (threadIdx.x & o) ? join2(q, s) : join2(s, q);
    }
    return s;
}

// Elements of a vector access: 16 bytes, or 8, or one.  The backward pass of two
// channels-last tensors takes at most four: six constants for each of eight
// channels a thread are 180 registers and two waves a SIMD (16x256x256x256 fp16:
// 563 us for dx alone, against 315 with four).
constexpr int vector_of(size_t esize, bool xl, bool yl, bool bwd)
{
    return bwd && xl && yl ? 4 : 16 / (int)esize;
}

// Where lanes > 0, the forward pass's elementwise kernel finds mean and rstd by
// itself, so many lanes a group; a lane's next moment lies ranges further on and
// channels more (or one range and channels - per).
struct Own {
    int lanes, ranges, channels;
};

struct Plan {
    Geometry stats, apply;  // the forward pass's moments; every other pass
    bool xl, yl, one;
    Own own;
    int v;  // elements of an access
    float eps;
    size_t means_at, bytes;  // workspace: partial sums, then the groups' means
};

// `aligned`: every activation lies on 16 bytes.
Plan make_plan(const wtconv_norm_desc_t &d, bool bwd, bool aligned);

struct Call {
    const void *x, *dy;  // dy null: forward
    const float *gamma, *beta, *mean, *rstd;
    void *out;  // y or dx
    float *mean_out, *rstd_out, *dgamma, *dbeta;
    void *workspace;
    int64_t n;
};

template <typename T>
hipError_t run(const Plan &p, const Call &a, hipStream_t stream);

// mean and rstd of every group of `n` images from its channels' moments in
// `part`.
void launch_finish_forward(const Geometry &g, int64_t n, const float2 *part, float *mean, float *rstd, float eps,
                           hipStream_t stream);

// From the channels' sums of `n` images in `part`: every group's means of t and
// t xh (unless null), and dgamma and dbeta (unless null).
void launch_finish_backward(const Geometry &g, int64_t n, const float2 *part, const float *gamma, float2 *means,
                            float *dgamma, float *dbeta, hipStream_t stream);

}  // namespace wtc_norm

// Bytes of workspace of the forward (bwd = 0) or backward call.
size_t wtc_norm_workspace(const wtconv_norm_desc_t &d, int bwd);

hipError_t wtc_launch_norm(const wtconv_norm_desc_t &d, const wtc_norm::Call &a, hipStream_t stream);

#endif  // WTCONV_NORM_H
