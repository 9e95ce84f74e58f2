// wtconv_norm.hip -- group norm: the plan of a call, and the small kernels that
// join the sums of pixel ranges (the walks are in wtconv_norm_body.h).
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cstdint>

#include "wtconv_check.h"
#include "wtconv_norm.h"

namespace wtc_norm {

namespace {

// A lane's sums over many images or channels are in fp64: it may have thousands.
struct Double2 {
    double x, y;
};

__device__ inline Double2 add(const Double2 &a, const Double2 &b) { return Double2{a.x + b.x, a.y + b.y}; }
__device__ inline float2 add(const float2 &a, const float2 &b) { return make_float2(a.x + b.x, a.y + b.y); }

// A wave's sum over its lanes, then over the waves of a workgroup that share a
// group (`wide`), through LDS; lane 0 of the first wave has it.
template <typename S>
__device__ inline S add_block(S s, bool wide, S *lds)
{
    auto add2 = [](const S &a, const S &b) { return add(a, b); };
    s = join_wave(s, add2);
    if (!wide) return s;
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    for (int i = 1; i < 4; ++i) s = add(i == 1 ? lds[0] : s, lds[i]);
    return s;
}

// A wave for each group, or (wide) a workgroup: with d_i a set's mean less the
// first one's, mean = first + sum n_i d_i / K, var = sum (M2_i + n_i d_i^2) / K -
// (sum n_i d_i / K)^2, which cancels by at most the number of sets, of 53 bits.
__global__ __launch_bounds__(256) void finish_forward(Geometry g, int64_t groups, bool wide,
                                                      const float2 *__restrict__ part, float *__restrict__ mean,
                                                      float *__restrict__ rstd, float eps)
{
    __shared__ Double2 lds[4];
    const int64_t ng = wide ? blockIdx.x : (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (ng >= groups) return;
    const int64_t n = ng / g.groups;
    const int c0 = (int)(ng % g.groups) * g.per, first = wide ? threadIdx.x : threadIdx.x & 63;
    const float2 *p = part + n * g.splits * g.c + c0;
    const double pivot = p[0].x;
    Double2 a = {0.0, 0.0};
#pragma unroll 4
    for (int i = first; i < g.splits * g.per; i += wide ? 256 : 64) {
        const int s = i / g.per;
        const float2 v = p[(int64_t)s * g.c + i % g.per];
        const double d = v.x - pivot, nd = pixels(g, s) * d;
        a = add(a, Double2{nd, fma(nd, d, (double)v.y)});
    }
    a = add_block(a, wide, lds);
    if (first == 0) {
        const double k = (double)g.per * g.hw, m = a.x / k, var = a.y / k - m * m;
        mean[ng] = (float)(pivot + m);
        rstd[ng] = 1.f / sqrtf((float)(var < 0.0 ? 0.0 : var) + eps);  // NaN stays
    }
}

// Workgroups 0 .. gblocks - 1: the means of t and t xh of a group a wave or
// (wide) a workgroup.  The others: dgamma and dbeta of 8 channels each, 32
// threads a channel.
__global__ __launch_bounds__(256) void finish_backward(Geometry g, int64_t images, bool wide,
                                                       const float2 *__restrict__ part,
                                                       const float *__restrict__ gamma, int gblocks,
                                                       float2 *__restrict__ means, float *__restrict__ dgamma,
                                                       float *__restrict__ dbeta)
{
    __shared__ Double2 lds[32][9];
    if ((int)blockIdx.x < gblocks) {
        const int64_t ng = wide ? blockIdx.x : (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
        if (ng >= images * g.groups) return;
        const int64_t n = ng / g.groups;
        const int c0 = (int)(ng % g.groups) * g.per, first = wide ? threadIdx.x : threadIdx.x & 63;
        const float2 *p = part + n * g.splits * g.c + c0;
        // 32 sets at a time (fp64 here, or a kernel of its own, costs more than it gives)
        float2 a = make_float2(0.f, 0.f), total = a;
        int left = 32;
#pragma unroll 4
        for (int i = first; i < g.splits * g.per; i += wide ? 256 : 64) {
            const int s = i / g.per, c = i % g.per;
            const float2 v = p[(int64_t)s * g.c + c];
            const float ga = gamma ? gamma[c0 + c] : 1.f;
            a = make_float2(fmaf(ga, v.x, a.x), fmaf(ga, v.y, a.y));
            if (--left == 0) {
                total = add(total, a);
                a = make_float2(0.f, 0.f);
                left = 32;
            }
        }
        a = add_block(add(total, a), wide, (float2 *)lds);
        const float k = (float)g.per * (float)g.hw;
        if (first == 0) means[ng] = make_float2(a.x / k, a.y / k);
        return;
    }
    const int j = threadIdx.x & 7, r = threadIdx.x >> 3, c = ((int)blockIdx.x - gblocks) * 8 + j;
    Double2 a = {0.0, 0.0};
    if (c < g.c) {
        const int64_t rows = images * g.splits;
        int64_t i = r;
        for (; i + 15 * 32 < rows; i += 16 * 32) {
            float2 v[16];  // as they come, then in fp64
#pragma unroll
            for (int u = 0; u < 16; ++u) v[u] = part[(i + u * 32) * g.c + c];
#pragma unroll
            for (int u = 1; u < 16; ++u) v[0] = add(v[0], v[u]);
            a = add(a, Double2{v[0].x, v[0].y});
        }
        float2 b = make_float2(0.f, 0.f);
#pragma unroll 8
        for (; i < rows; i += 32) b = add(b, part[i * g.c + c]);
        a = add(a, Double2{b.x, b.y});
    }
    lds[r][j] = a;
    __syncthreads();
    if (r == 0 && c < g.c) {
#pragma unroll 4
        for (int i = 1; i < 32; ++i) a = add(a, lds[i][j]);
        if (dbeta) dbeta[c] = (float)a.x;
        if (dgamma) dgamma[c] = (float)a.y;
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads side by side along a row of `chunks` pieces.  Channels last: the
// whole row, or an equal part of it of at most 64 pieces (each part ends in a
// join over the workgroup: 8 pieces of 40 to gain 6 % of the threads measured
// 40 us against 8 for 4x320x64x64 fp16).  Planes: four to eight pieces for a
// thread, so that a batch of loads is full, and among those widths the one that
// leaves the fewest of nt threads idle.
int pick_lanes(int chunks, int nt, bool last)
{
    if (last) return (int)ceil_div(chunks, ceil_div(chunks, 64));
    int hi = (int)ceil_div(chunks, 4), lo = chunks / 8;
    hi = hi < 8 ? (chunks < 8 ? chunks : 8) : hi > nt ? nt : hi;
    lo = lo < 8 ? 8 : lo;
    int best = hi;
    double value = 0.;
    for (int l = hi; l >= (lo < hi ? lo : hi); --l) {
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

constexpr int kLeastBytes = 8192;   // of one tensor, for a workgroup of the three-launch form

// Workgroups of the three-launch form, us for 1024 / 2048 / 4096 of them:
//   last    forward 64x192x28x28 fp16 21.5 / 23.2 / 23.2, 64x96x56x56 fp16 27.7 /
//           29.2 / 33.0, 32x128x128x128 fp32 181 / 157 / 158
//   tiles   backward 64x96x56x56 fp32 68 / 79 / 66, 16x256x256x256 fp16 687 / 731 /
//           620
//   planes  within 2 %.
int target_count(Walk w, int64_t bytes) { return w == kTiles ? 4096 : w == kLast && bytes < 64 << 20 ? 1024 : 2048; }

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
    g.lanes = pick_lanes(w == kLast ? g.cb / v : (int)ceil_div(g.hw, v), nt, w == kLast);
    // a row of threads for every channel of the group, not more
    const int chunks = (int)ceil_div(g.hw, v);
    if (w == kPlanes && nt / g.lanes > g.cb) g.lanes = nt / g.cb < chunks ? nt / g.cb : chunks;
    g.count = n * g.blocks;
    return g;
}

enum Sums { kNone, kMoments, kBackward };  // what a walk adds up

Geometry split_geometry(Geometry g, int64_t n, Walk w, int v, int esize, Sums sums)
{
    int step;     // pixels that a workgroup takes at least
    int64_t far;  // and at most, where it sums them
    if (w == kLast) {
        const int chunks = g.c / v, most = kMaxBlock / v;
        const int blocks = (int)ceil_div(chunks, most);
        g.cb = (int)ceil_div(chunks, blocks) * v;
        g.lanes = pick_lanes(g.cb / v, kThreads, true);
        step = kThreads / g.lanes;
        far = (int64_t)(sums == kBackward ? kMostBackward : kMostUnjoined) * step;
    } else if (w == kTiles) {
        step = 128 / esize;
        g.cb = g.c < step ? g.c : step;
        g.lanes = 1;
        far = (v * esize == 16 && esize == 4 ? kMostValues : kMostUnjoined) / v * step;  // one channel a thread or more
    } else {
        g.lanes = pick_lanes((int)ceil_div(g.hw, v), kThreads, false);
        const int rows = kThreads / g.lanes;
        int64_t cb = kLeastBytes / ((int64_t)g.hw * esize) / rows * rows;
        if (cb < rows) cb = rows;
        if (cb > kMaxBlock / rows * rows) cb = kMaxBlock / rows * rows;
        g.cb = (int)(cb < g.c ? cb : g.c);
        step = g.lanes * v;
        far = (int64_t)kMostValues * g.lanes;
    }
    g.blocks = (int)ceil_div(g.c, g.cb);
    // that many workgroups, but no fewer bytes for one than kLeastBytes
    const int64_t all = n * g.blocks;
    const int64_t most = ceil_div(target_count(w, n * g.c * (int64_t)g.hw * esize), all);
    int64_t ppw = ceil_div(g.hw, most);
    const int64_t least = ceil_div(kLeastBytes, (int64_t)g.cb * esize);
    if (ppw < least) ppw = least;
    // (no more than 2^22 workgroups for that: beyond some 2^32 values of few channels)
    if (sums != kNone && ppw > far && ceil_div(g.hw, far) * all <= 1 << 22) ppw = far;
    ppw = ceil_div(ppw < 1 ? 1 : ppw, step) * step;
    g.ppw = (int)(ppw < g.hw ? ppw : ceil_div(g.hw, step) * step);
    g.splits = (int)ceil_div(g.hw, g.ppw);
    g.count = all * g.splits;
    return g;
}

// Lanes for each group, where the forward pass's elementwise kernel finds mean and
// rstd from the ranges' moments by itself: a launch less, against a few loads
// and sums at the start of each workgroup.  us without and with, in a graph:
//   last, planes  32x32x112x112 fp32 34.4 / 29.4 and 30.9 / 28.7, 64x192x28x28 fp16
//           21.7 / 20.0, 1x512x32x32 fp32 planes 10.5 / 9.0, never 2 % more;
//   tiles   1x128x64x64 10.4 / 9.0, 32x128x128x128 fp16 78.8 / 76.2, but
//           32x32x112x112 fp16 22.3 / 24.9, 2x128x256x256 fp16 25.5 / 26.4: not
//           from 16 to 64 MB.
// 0 (a kernel in between) there, and where all groups at once and kOwnSums
// moments a lane do not do.
Own own_of(const Geometry &sums, const Geometry &apply)
{
    const int most = (apply.cb - 1) / apply.per + 2, ng = most < apply.groups ? most : apply.groups;
    int lanes = 64;
    while (lanes > 1 && lanes * ng > kThreads) lanes /= 2;
    if (lanes * ng > kThreads || (int64_t)sums.splits * sums.per > kOwnSums * lanes) return Own{0, 0, 0};
    return Own{lanes, lanes / sums.per, lanes % sums.per};
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
    g.stream = d.n * d.c * (int64_t)g.hw * esize > 32 << 20;
    const Walk sw = p.xl ? kLast : kPlanes, aw = p.xl != p.yl ? kTiles : sw;
    // the widest access that rows and addresses allow: rows of channels, of
    // pixels, or in tiles (the planes' side) of pixels
    auto widest = [&](int most, bool channels, bool pixels) {
        if (!aligned) return 1;
        for (int w = most; w > 1; w = w > v16 / 2 ? v16 / 2 : 1)
            if (!(channels && g.c % w) && !(pixels && g.hw % w)) return w;
        return 1;
    };
    p.v = widest(vector_of(esize, p.xl, p.yl, bwd), p.xl && p.yl, !(p.xl && p.yl));
    g.vlast = widest(v16, true, false);
    // the moments' walk follows x alone, with the same width of access
    if (aw == kTiles && p.xl && !bwd) p.v = widest(v16, true, true);
    const int v = p.v;

    // One launch, against three, by sizes (fp16 / fp32, us, measured in a graph):
    //   planes  64x96x56x56 26 / 37 against 30 / 43, 16x256x256x256 310 against
    //           329; but 4x320x64x64 17 / 23 against 15 / 20: from 256 workgroups
    //           on, or where a group is so small that launches are all it costs
    //           (8x64x14x14: 7 against 14);
    //   last    a workgroup's rows are narrow: 8x512x16x16 12 / 9 against 13 / 15,
    //           but 1x128x64x64 19 / 17 against 13 / 12, 64x768x7x7 21 / 20
    //           against 15 / 16: up to 1024 pixels and 64 KB, at most 512 of them;
    //   tiles   forward 8x512x16x16 9 / 9 against 11 / 11, but 1x512x32x32 16 / 21
    //           against 11 / 11: up to 256 pixels; backward never (64x768x7x7
    //           27 / 23 against 36 / 23, 8x512x16x16 15 / 17 against 13 / 11).
    const int unit = aw == kTiles ? lcm_pow2(g.per, p.xl && !bwd && v > g.vlast ? v : g.vlast)
                     : p.xl ? lcm_pow2(g.per, v) : g.per;
    if (unit <= kMaxBlock && !(aw == kTiles && (bwd || g.hw > 256))) {
        const Geometry s = one_geometry(g, d.n, sw, aw == kTiles, v, v16, unit);
        const int64_t slice = (int64_t)s.cb * g.hw * esize, count = s.count;
        const bool pays = aw == kTiles ? true
                          : aw == kLast ? slice <= 65536 && g.hw <= 1024 && count <= 512
                                        : (slice <= 16384 || count >= 256) && g.hw <= (int64_t)kMostValues * s.lanes;
        if (pays) {
            p.one = true;
            p.stats = s;
            p.apply = s;
            p.bytes = bwd ? align256((size_t)(d.n * d.c) * sizeof(float2)) : 0;
            return p;
        }
    }
    p.apply = split_geometry(g, d.n, aw, v, esize, bwd ? kBackward : kNone);
    // the moments' walk is the forward pass's alone; in tiles its rows may be
    // narrower than the backward pass's accesses to planes
    p.stats = bwd ? p.apply : split_geometry(g, d.n, sw, v, esize, kMoments);
    const Geometry &q = p.stats;
    const int64_t bytes = d.n * d.c * (int64_t)g.hw * esize;
    if (!bwd && !(aw == kTiles && bytes >= 16 << 20 && bytes < 64 << 20)) p.own = own_of(p.stats, p.apply);
    p.means_at = align256((size_t)(d.n * q.splits) * d.c * sizeof(float2));
    p.bytes = p.means_at + (bwd ? align256((size_t)(d.n * d.groups) * sizeof(float2)) : 0);
    return p;
}

void launch_finish_forward(const Geometry &g, int64_t n, const float2 *part, float *mean, float *rstd, float eps,
                           hipStream_t stream)
{
    const int64_t groups = n * g.groups;
    const bool wide = g.splits * g.per > 256;
    finish_forward<<<dim3((unsigned)(wide ? groups : ceil_div(groups, 4))), dim3(256), 0, stream>>>(g, groups, wide,
                                                                                                  part, mean, rstd,
                                                                                                  eps);
}

void launch_finish_backward(const Geometry &g, int64_t n, const float2 *part, const float *gamma, float2 *means,
                            float *dgamma, float *dbeta, hipStream_t stream)
{
    const bool wide = g.splits * g.per > 256;
    const int64_t gb = means ? (wide ? n * g.groups : ceil_div(n * g.groups, 4)) : 0;
    const int64_t cb = dgamma || dbeta ? ceil_div(g.c, 8) : 0;
    finish_backward<<<dim3((unsigned)(gb + cb)), dim3(256), 0, stream>>>(g, n, wide, part, gamma, (int)gb, means,
                                                                         dgamma, dbeta);
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
