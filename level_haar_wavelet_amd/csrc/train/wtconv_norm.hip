// wtconv_norm.hip -- group norm: the plan of a call, and the small kernels that
// join the sums of pixel ranges (the walks are in wtconv_norm_body.h).
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cstdint>

#include "wtconv_check.h"
#include "wtconv_norm.h"

namespace wtc_norm {

namespace {

// Pixels of range s.
__device__ inline int pixels(const Geometry &g, int s)
{
    const int p = g.hw - s * g.ppw;
    return p < g.ppw ? p : g.ppw;
}

__device__ inline float wave_sum(float v)
{
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// One wave a group.
__global__ __launch_bounds__(256) void finish_forward(Geometry g, int64_t groups, const float2 *__restrict__ part,
                                                      float *__restrict__ mean, float *__restrict__ rstd, float eps)
{
    const int64_t ng = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (ng >= groups) return;
    const int64_t n = ng / g.groups;
    const int c0 = (int)(ng % g.groups) * g.per, lane = threadIdx.x & 63;
    const float2 *p = part + n * g.splits * g.c + c0;
    Moments m = {0.f, 0.f, 0.f};
    for (int i = lane; i < g.splits * g.per; i += 64) {
        const int s = i / g.per;
        const float2 v = p[(int64_t)s * g.c + i % g.per];
        m = join(m, Moments{(float)pixels(g, s), v.x, v.y});
    }
    m = join_wave(m, join);
    if (lane == 0) {
        mean[ng] = m.mean;
        rstd[ng] = 1.f / sqrtf(m.m2 / m.n + eps);
    }
}

// Workgroups 0 .. gblocks - 1: one wave a group, its means of t and t xh.  The
// others: dgamma and dbeta of 16 channels each, 16 threads a channel.
__global__ __launch_bounds__(256) void finish_backward(Geometry g, int64_t images, const float2 *__restrict__ part,
                                                       const float *__restrict__ gamma, int gblocks,
                                                       float2 *__restrict__ means, float *__restrict__ dgamma,
                                                       float *__restrict__ dbeta)
{
    if ((int)blockIdx.x < gblocks) {
        const int64_t ng = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
        if (ng >= images * g.groups) return;
        const int64_t n = ng / g.groups;
        const int c0 = (int)(ng % g.groups) * g.per, lane = threadIdx.x & 63;
        const float2 *p = part + n * g.splits * g.c + c0;
        float a = 0.f, b = 0.f;
        for (int i = lane; i < g.splits * g.per; i += 64) {
            const int s = i / g.per, c = i % g.per;
            const float2 v = p[(int64_t)s * g.c + c];
            const float ga = gamma ? gamma[c0 + c] : 1.f;
            a = fmaf(ga, v.x, a);
            b = fmaf(ga, v.y, b);
        }
        a = wave_sum(a);
        b = wave_sum(b);
        const float k = (float)g.per * (float)g.hw;
        if (lane == 0) means[ng] = make_float2(a / k, b / k);
        return;
    }
    __shared__ float2 lds[16][17];
    const int j = threadIdx.x & 15, r = threadIdx.x >> 4, c = ((int)blockIdx.x - gblocks) * 16 + j;
    float a = 0.f, b = 0.f;
    if (c < g.c)
#pragma unroll 4
        for (int64_t i = r; i < images * g.splits; i += 16) {
            const float2 v = part[i * g.c + c];
            a += v.x;
            b += v.y;
        }
    lds[r][j] = make_float2(a, b);
    __syncthreads();
    if (r == 0 && c < g.c) {
        for (int i = 1; i < 16; ++i) {
            a += lds[i][j].x;
            b += lds[i][j].y;
        }
        if (dbeta) dbeta[c] = a;
        if (dgamma) dgamma[c] = b;
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads side by side along rows of `chunks` pieces such that the fewest of nt
// threads idle, at least eight of them (128 bytes) where there are as many.
int pick_lanes(int chunks, int nt, int most)
{
    const int hi = chunks < most ? chunks : most, lo = hi < 8 ? hi : 8;
    int best = hi;
    double value = 0.;
    for (int l = hi; l >= lo; --l) {
        const double used = (double)chunks / (double)(ceil_div(chunks, l) * l) * (double)(nt / l * l) / nt;
        if (used > value * 1.02) {
            value = used;
            best = l;
        }
    }
    return best;
}

// Least common multiple of per and v (a power of two).
int lcm_pow2(int per, int v)
{
    int g = 1;
    while (g < v && per % (2 * g) == 0) g *= 2;
    return per / g * v;
}

enum Walk { kPlanes, kLast, kTiles };

constexpr int kTargetBytes = 32768;  // of one tensor, a workgroup of the three-launch form
constexpr int kTargetCount = 2048;   // workgroups that fill the chip

// Whole groups of an image for each workgroup: cb channels, all pixels.
Geometry one_geometry(Geometry g, int64_t n, Walk w, bool tiles, int v, int v16, int unit)
{
    const int nt = kOneThreads;
    g.splits = 1;
    g.ppw = g.hw;
    g.cb = unit;
    // channels last: rows of at least 64 bytes where the workgroups suffice;
    // tiles: their whole width
    const int wide = tiles ? 8 * v16 : w == kLast ? 4 * v16 : 1;
    while (g.cb * 2 <= kMaxBlock && g.cb < wide && g.cb < g.c && n * ceil_div(g.c, 2 * g.cb) >= 256) g.cb *= 2;
    if (g.cb > g.c) g.cb = g.c;
    g.blocks = (int)ceil_div(g.c, g.cb);
    g.lanes = w == kLast ? pick_lanes(g.cb / v, nt, 64) : pick_lanes((int)ceil_div(g.hw, v), nt, nt);
    g.count = n * g.blocks;
    return g;
}

Geometry split_geometry(Geometry g, int64_t n, Walk w, int v, int esize)
{
    int step;  // pixels that a workgroup takes at least
    if (w == kLast) {
        const int chunks = g.c / v, most = kMaxBlock / v;
        const int blocks = (int)ceil_div(chunks, most);
        g.cb = (int)ceil_div(chunks, blocks) * v;
        g.lanes = pick_lanes(g.cb / v, kThreads, 64);
        step = kThreads / g.lanes;
    } else if (w == kTiles) {
        step = 128 / esize;
        g.cb = g.c < step ? g.c : step;
        g.lanes = 1;
    } else {
        g.lanes = pick_lanes((int)ceil_div(g.hw, v), kThreads, kThreads);
        const int rows = kThreads / g.lanes;
        int64_t cb = kTargetBytes / ((int64_t)g.hw * esize) / rows * rows;
        if (cb < rows) cb = rows;
        if (cb > kMaxBlock / rows * rows) cb = kMaxBlock / rows * rows;
        g.cb = (int)(cb < g.c ? cb : g.c);
        step = g.lanes * v;
    }
    g.blocks = (int)ceil_div(g.c, g.cb);
    int64_t ppw = kTargetBytes / ((int64_t)g.cb * esize);
    const int64_t all = n * g.blocks;
    if (all * ceil_div(g.hw, ppw < 1 ? 1 : ppw) < kTargetCount) ppw = ceil_div(g.hw, ceil_div(kTargetCount, all));
    ppw = ceil_div(ppw < 1 ? 1 : ppw, step) * step;
    g.ppw = (int)(ppw < g.hw ? ppw : ceil_div(g.hw, step) * step);
    g.splits = (int)ceil_div(g.hw, g.ppw);
    g.count = all * g.splits;
    return g;
}

}  // namespace

Plan make_plan(const wtconv_norm_desc_t &d, bool bwd, bool aligned)
{
    Plan p = {};
    p.xl = d.x_layout == WTCONV_NHWC;
    p.yl = d.y_layout == WTCONV_NHWC;
    p.eps = d.eps;
    const int esize = d.dtype == WTCONV_F32 ? 4 : 2, v16 = 16 / esize;
    Geometry g = {};
    g.c = (int)d.c;
    g.hw = (int)(d.h * d.w);
    g.groups = d.groups;
    g.per = g.c / g.groups;
    g.act = d.act;
    const Walk sw = p.xl ? kLast : kPlanes, aw = p.xl != p.yl ? kTiles : sw;
    p.vec = aligned && (!(p.xl || p.yl) || g.c % v16 == 0) && ((p.xl && p.yl) || g.hw % v16 == 0);
    const int v = p.vec ? v16 : 1;

    // one launch where whole groups make enough workgroups, or where the data
    // are so few that a launch costs more than the pass
    const int unit = p.xl || p.yl ? lcm_pow2(g.per, v) : g.per;
    const int64_t bytes = d.n * d.c * (int64_t)g.hw * esize * (bwd ? 2 : 1);
    if (unit <= kMaxBlock) {
        const Geometry s = one_geometry(g, d.n, sw, aw == kTiles, v, v16, unit);
        if (s.count >= 256 || bytes <= 1 << 20) {
            p.one = true;
            p.stats = s;
            p.apply = s;
            if (aw == kTiles) p.apply.lanes = 1;
            p.bytes = bwd ? align256((size_t)(d.n * d.c) * sizeof(float2)) : 0;
            return p;
        }
    }
    p.stats = split_geometry(g, d.n, sw, v, esize);
    p.apply = split_geometry(g, d.n, aw, v, esize);
    const Geometry &q = bwd ? p.apply : p.stats;
    p.means_at = align256((size_t)(d.n * q.splits) * d.c * sizeof(float2));
    p.bytes = p.means_at + (bwd ? align256((size_t)(d.n * d.groups) * sizeof(float2)) : 0);
    return p;
}

void launch_finish_forward(const Geometry &g, int64_t n, const float2 *part, float *mean, float *rstd, float eps,
                           hipStream_t stream)
{
    const int64_t groups = n * g.groups;
    finish_forward<<<dim3((unsigned)ceil_div(groups, 4)), dim3(256), 0, stream>>>(g, groups, part, mean, rstd, eps);
}

void launch_finish_backward(const Geometry &g, int64_t n, const float2 *part, const float *gamma, float2 *means,
                            float *dgamma, float *dbeta, hipStream_t stream)
{
    const int64_t gb = means ? ceil_div(n * g.groups, 4) : 0, cb = dgamma || dbeta ? ceil_div(g.c, 16) : 0;
    finish_backward<<<dim3((unsigned)(gb + cb)), dim3(256), 0, stream>>>(g, n, part, gamma, (int)gb, means, dgamma,
                                                                         dbeta);
}

}  // namespace wtc_norm

size_t wtc_norm_workspace(const wtconv_norm_desc_t &d, int bwd)
{
    // the plan of unaligned activations may take more
    const size_t a = wtc_norm::make_plan(d, bwd != 0, true).bytes, b = wtc_norm::make_plan(d, bwd != 0, false).bytes;
    return a > b ? a : b;
}

hipError_t wtc_launch_norm(const wtconv_norm_desc_t &d, const wtc_norm::Call &a, hipStream_t stream)
{
    const bool aligned = aligned16(a.x) && aligned16(a.out) && (!a.dy || aligned16(a.dy));
    const wtc_norm::Plan p = wtc_norm::make_plan(d, a.dy != nullptr, aligned);
    if (d.dtype == WTCONV_F32) return wtc_norm::run<float>(p, a, stream);
    if (d.dtype == WTCONV_F16) return wtc_norm::run<_Float16>(p, a, stream);
    return wtc_norm::run<__bf16>(p, a, stream);
}
