// wtconv_norm_body.h -- the group norm kernels of one element type; the files
// wtconv_norm_f32.hip, _f16.hip and _bf16.hip instantiate them.
//
// A group's mean and variance, and the backward pass's two means, are needed
// before the first output, so the data are walked twice: 3 E e bytes forward
// and 5 E e backward where nothing is kept between, against a floor of 2 E e
// and 3 E e.  Two forms:
//   one launch   a workgroup owns whole groups of an image, walks them twice and
//                finds the second time in the caches what it read the first;
//   three        for images too large or too few for that: sums of pixel ranges
//                per channel, a small kernel that joins them (forward, where they
//                are few, the next one does it itself), and the elementwise
//                pass, which takes the ranges from the last to the first: the
//                256 MB cache holds the end of what was read before.
//
// Large ones are bound by memory, whose counters show those 3 E e and 5 E e:
// 32x128x128x128 bf16 planes to channels last takes 69 us (5.9 TB/s), the backward
// pass of 64x96x56x56 fp32 73 us (5.3) and of 16x256x256x256 fp16 481 us (5.6), where
// an elementwise pass over 4 GiB reaches 6.2.  Below about 20 MB latency counts: the
// two kernels of 64x192x28x28 fp16 take 8.1 and 14.8 us, their bytes 3.1 and 6.2.
//
// Walks.  An image lies in memory as rows of contiguous elements: its channels'
// planes, or its pixels' channels.  A thread takes V contiguous elements (16
// or 8 bytes, or one where sizes or addresses allow no more), `lanes` threads stand
// side by side along a row and the rest take rows below, so that every thread
// keeps its channel (planes) or its V channels (last) and their constants in
// registers.  Where the two tensors of a pass lie differently the walk is along
// planes, in tiles of 8 V pixels x 8 V channels, and the tensor that lies
// channels last goes through LDS: 128 bytes a pixel in 8 chunks of 16, chunk j
// of pixel p at place j ^ (p / V) % 8, which spreads the column reads over the
// banks.
//
// Numerics.  Values are fp32 from the load on.  A thread sums x - s and
// (x - s)^2 of a chain of values, s the first of them: since s is one of the
// values, the sum of squares cannot cancel by more than their number.  Along
// planes a chain is kChain values and s, from the second on, the mean of those
// before, so that a border that differs from the rest does not shift all that
// follows it.  Chains' and threads' (count, mean, M2) are joined by Chan's formula,
// in fixed order.  The backward sums go to the thread's total kChain at a time
// where it sums one channel.  With the limits of wtconv_norm.h on what a thread
// takes, a sum is a chain of at most 96 additions (128 in the backward pass along
// channels) and a tree; longer sums over ranges and images after that are in fp64
// or 32 at a time.
#ifndef WTCONV_NORM_BODY_H
#define WTCONV_NORM_BODY_H

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cstdint>

#include "wtconv_norm.h"

namespace wtc_norm {

template <typename T, int V>
struct Pack {
    typedef T type __attribute__((ext_vector_type(V)));
};
template <typename T>
struct Pack<T, 1> {
    typedef T type;
};

// The V elements at p, and their values.
template <typename T, int V>
__device__ inline typename Pack<T, V>::type fetch(const T *p)
{
    return *(const typename Pack<T, V>::type *)p;
}

// The same for the last read of a value, and a store of what this call does not
// read again: where the tensor is larger than the L2s (STREAM), past them, so
// that they keep what is still to be read.  us with and without, of inputs not
// in the caches: forward 64x96x56x56 fp32 42 / 53, 16x256x256x256 fp16 281 /
// 327, its backward 499 / 549; below that size no difference, and the output
// stays for its reader.
// (A constant of the instance: where it is known at run time only, the compiler
// makes one plain access of both.)
template <bool STREAM, typename P>
__device__ inline P fetch_last(const P *p)
{
    if constexpr (STREAM)
        return __builtin_nontemporal_load(p);
    else
        return *p;
}

template <bool STREAM, typename P>
__device__ inline void store_last(P *p, const P &v)
{
    if constexpr (STREAM)
        __builtin_nontemporal_store(v, p);
    else
        *p = v;
}

template <typename T, int V>
__device__ inline void values(const typename Pack<T, V>::type &r, float (&v)[V])
{
    if constexpr (V == 1)
        v[0] = (float)r;
    else
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = (float)r[i];
}

template <typename T, int V, bool STREAM>
__device__ inline void store(T *p, const float (&v)[V])
{
    typename Pack<T, V>::type r;
    if constexpr (V == 1)
        r = (T)v[0];
    else
#pragma unroll
        for (int i = 0; i < V; ++i) r[i] = (T)v[i];
    store_last<STREAM>((typename Pack<T, V>::type *)p, r);
}

// Phi(z) = (1 + erf(z / sqrt 2)) / 2 and e = exp(-z^2 / 2), by Abramowitz and
// Stegun 7.1.26: erf(x) = 1 - t (a1 + t (a2 + ..)) exp(-x^2), t = 1 / (1 + p x),
// within 1.5e-7 for x >= 0.  Half the instructions of erff, and the backward
// pass needs the exponential in any case.
__device__ inline float normal_cdf(float z, float &e)
{
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f * 0.70710678f, fabsf(z), 1.f));
    e = __builtin_amdgcn_exp2f(z * z * -0.72134752f);  // log2(e) / 2
    // half the polynomial, the halves of a1 .. a5
    const float q = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 0.5307027145f, -0.7265760135f), 0.7107068705f), -0.142248368f),
                             0.127414796f);
    const float tail = q * e;
    return z < 0.f ? tail : 1.f - tail;
}

// 1 / (1 + exp(-z)); exp overflows to infinity and the reciprocal to 0.
__device__ inline float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// act(z), in place.
template <int V>
__device__ inline void act_fwd(int act, float (&z)[V])
{
    if (act == WTCONV_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = z[i] * sigmoid(z[i]);
    } else if (act == WTCONV_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float e;
            z[i] = z[i] * normal_cdf(z[i], e);
        }
    } else if (act == WTCONV_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = z[i] < 0.f ? 0.f : z[i];  // NaN stays
    }
}

// Constants of a channel.
struct Chan {
    float mean, rstd, gamma, beta;
};

// dy act'(z), z = gamma xh + beta, xh = (x - mean) rstd.
__device__ inline float act_bwd(int act, float dy, float x, float xh, const Chan &k)
{
    const float z = fmaf(k.gamma, xh, k.beta);
    if (act == WTCONV_ACT_SILU) {
        const float s = sigmoid(z);
        return dy * s * fmaf(z, 1.f - s, 1.f);
    }
    if (act == WTCONV_ACT_GELU) {
        float e;
        const float p = normal_cdf(z, e);
        return dy * fmaf(z * 0.39894228f, e, p);
    }
    if (act == WTCONV_ACT_RELU) {
        bool on = z > 0.f;
        // next to the border the sign is decided in fp64
        if (fabsf(z) <= 1e-5f * (fabsf(k.gamma * xh) + fabsf(k.beta)))
            on = fma(((double)x - k.mean) * k.rstd, (double)k.gamma, (double)k.beta) > 0.0;
        return on ? dy : 0.f;
    }
    return dy;
}

// What a workgroup walks: `cb` channels from c0 and pixels p0 .. p1 of image n.
struct Range {
    int64_t n;
    int c0, cb, p0, p1;
    int64_t row;  // of the partial sums
};

// The range of workgroup `id` of g.count.  Workgroups go to the 8 dies in turn; each die
// gets a stretch of neighbouring ranges, so that the parts of a cache line that
// lie in two channel blocks meet in one L2, and a second pass (kBack: last range
// first) finds in its L2 what the first pass read there last.  One launch over
// planes has neither, and runs up to 15 % faster in plain order (kPlain).
enum Order { kPlain, kForth, kBack };

__device__ inline Range range_of(const Geometry &g, Order order, int id)
{
    if (order != kPlain) {
        const int per = (int)(g.count / 8), rest = (int)(g.count % 8), die = id % 8, own = per + (die < rest), k = id / 8;
        id = die * per + (die < rest ? die : rest) + (order == kBack ? own - 1 - k : k);
    }
    const int64_t u = id / g.splits;
    const int s = id % g.splits, b = (int)(u % g.blocks);
    Range r;
    r.n = u / g.blocks;
    r.row = r.n * g.splits + s;
    r.c0 = b * g.cb;
    r.cb = g.c - r.c0 < g.cb ? g.c - r.c0 : g.cb;
    r.p0 = s * g.ppw;
    r.p1 = g.hw - r.p0 < g.ppw ? g.hw : r.p0 + g.ppw;
    return r;
}

// Calls get(u, offset) and then use(u, offset, first) for every V elements of
// the range that this thread takes, kBatch of them at a time, so that their
// loads are in flight together (u is the place in the batch; first: the
// channel's first batch); begin(c) before and end(c) after those of one channel
// (planes) or V channels from c on (last).  Every thread of the workgroup makes
// the same number of begin and end calls; those without a channel of the range
// get c < 0.
constexpr int kBatch = 4;

// Values of a channel that a thread sums before they join the rest: whole
// batches.
constexpr int kChain = 32;

template <bool LAST, int V, int NT, typename B, typename G, typename F, typename E>
__device__ inline void walk(const Geometry &g, const Range &r, B begin, G get, F use, E end)
{
    const int row = threadIdx.x / g.lanes, rows = NT / g.lanes, i = (threadIdx.x - row * g.lanes) * V;
    const int64_t base = r.n * g.c * (int64_t)g.hw;
    const int step = LAST ? rows : V * g.lanes, pitch = LAST ? g.c : 1;
    for (int cc = 0; cc < r.cb; cc += LAST ? V * g.lanes : rows) {
        const int own = cc + (LAST ? i : row);
        const int c = row < rows && own < r.cb ? r.c0 + own : -1;
        begin(c);
        if (c >= 0) {
            const int64_t at0 = base + (LAST ? c : (int64_t)c * g.hw);
            const int start = r.p0 + (LAST ? row : i);
            for (int p = start; p < r.p1; p += kBatch * step) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (p + u * step < r.p1) get(u, at0 + (int64_t)(p + u * step) * pitch);
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (p + u * step < r.p1) use(u, at0 + (int64_t)(p + u * step) * pitch, p == start);
            }
        }
        end(c);
    }
}

// The K channels' moments or sums of one thread; the count is the same for all.
template <int K>
struct MomentSet {
    float n, mean[K], m2[K];
    static constexpr int kFloats = 1 + 2 * K;
    __device__ void add(const MomentSet &b)
    {
        const float s = n + b.n;
        const float w = s > 0.f ? b.n * __builtin_amdgcn_rcpf(s) : 0.f, v = n * w;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float d = b.mean[k] - mean[k];
            // an empty set's own zeros must not meet an infinity
            mean[k] = n > 0.f ? fmaf(d, w, mean[k]) : b.mean[k];
            m2[k] = n > 0.f && b.n > 0.f ? m2[k] + b.m2[k] + d * d * v : n > 0.f ? m2[k] : b.m2[k];
        }
        n = s;
    }
};

template <int K>
struct SumSet {
    float a[K], b[K];
    static constexpr int kFloats = 2 * K;
    __device__ void add(const SumSet &o)
    {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            a[k] += o.a[k];
            b[k] += o.b[k];
        }
    }
};

// Joins the sets of the threads that share a channel (those below it for
// channels last, its row for planes) by a tree of fours in LDS; the first of
// them ends up with the whole and returns true.  lds: kFloats NT floats.
template <bool LAST, int NT, typename S>
__device__ inline bool join_threads(const Geometry &g, int c, S &v, float *lds)
{
    const int t = threadIdx.x, row = t / g.lanes, rows = NT / g.lanes, i = t - row * g.lanes;
    const int q = LAST ? row : i, stride = LAST ? g.lanes : 1;
    auto put = [&] {
        const float *f = (const float *)&v;
#pragma unroll
        for (int k = 0; k < S::kFloats; ++k) lds[k * NT + t] = f[k];
    };
    for (int h = LAST ? rows : g.lanes; h > 1;) {
        const int part = (h + 3) / 4;
        __syncthreads();
        if (row < rows && q < h) put();
        __syncthreads();
        if (row < rows && q < part)
#pragma unroll
            for (int o = 1; o < 4; ++o)
                if (q + o * part < h) {
                    S w;
                    float *f = (float *)&w;
#pragma unroll
                    for (int k = 0; k < S::kFloats; ++k) f[k] = lds[k * NT + t + o * part * stride];
                    v.add(w);
                }
        h = part;
    }
    return c >= 0 && q == 0;
}

// Moments of every channel of the range: done(c, moments).  Along channels
// a thread has at most kMostUnjoined of each, one chain (the set to join it with
// would be half as many registers again, 58 -> 80: 64x192x28x28 fp16 21.8 -> 22.9 us).
template <typename T, bool LAST, int V, int NT, typename D>
__device__ inline void moments(const T *__restrict__ x, const Geometry &g, const Range &r, float *lds, D done)
{
    constexpr int K = LAST ? V : 1;
    float s[K], a[K], b[K], n;
    MomentSet<K> m, total;
    auto end_chain = [&] {
        const float w = n > 0.f ? 1.f / n : 0.f;
        m.n = n;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            m.mean[k] = fmaf(a[k], w, s[k]);
            m.m2[k] = fmaf(-a[k] * w, a[k], b[k]);
            // rounding only: a sum of squares is not negative (NaN stays)
            if (m.m2[k] < 0.f) m.m2[k] = 0.f;
        }
        if constexpr (!LAST) {
            total.add(m);
            m = total;
        }
    };
    typename Pack<T, V>::type raw[kBatch];
    walk<LAST, V, NT>(
        g, r,
        [&](int) {
            n = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) s[k] = a[k] = b[k] = 0.f;
            if constexpr (!LAST) total.n = total.mean[0] = total.m2[0] = 0.f;
        },
        [&](int u, int64_t at) { raw[u] = fetch<T, V>(x + at); },
        [&](int u, int64_t, bool first) {
            float v[V];
            values<T, V>(raw[u], v);
            if (u == 0 && first)
#pragma unroll
                for (int k = 0; k < K; ++k) s[k] = v[k];
            if constexpr (!LAST)
                if (u == 0 && n >= (float)kChain) {
                    end_chain();
                    s[0] = total.mean[0];
                    n = a[0] = b[0] = 0.f;
                }
            n += V / K;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int k = LAST ? i : 0;
                const float d = v[i] - s[k];
                a[k] += d;
                b[k] = fmaf(d, d, b[k]);
            }
        },
        [&](int c) {
            end_chain();
            if (join_threads<LAST, NT>(g, c, m, lds))
#pragma unroll
                for (int k = 0; k < K; ++k) done(c + k, Moments{m.n, m.mean[k], m.m2[k]});
        });
}

// ---- Tiles of differing layouts -----------------------------------------------

// LDS place of channel j of pixel p of a tile.
template <typename T, int V16>
__device__ inline T *tile_at(char *tile, int p, int j)
{
    return (T *)(tile + p * 128 + (((j / V16) ^ ((p / V16) & 7)) * 16)) + j % V16;
}

// Brings the tile (pixels p0.., channels c0..) of a channels-last tensor into
// LDS, or back out of it, V channels at a time.
template <typename T, int V, int NT, bool OUT, bool STREAM>
__device__ inline void move_pieces(T *t_, const Geometry &g, const Range &r, int p0, int c0, char *tile)
{
    constexpr int V16 = 16 / sizeof(T), kSide = 8 * V16, kChunks = kSide / V, kOwn = (kSide * kChunks + NT - 1) / NT;
    typedef typename Pack<T, V>::type P;
    P v[kOwn];
    T *m = t_ + (r.n * g.hw + p0) * (int64_t)g.c + c0;
    auto inside = [&](int e) {
        return e < kSide * kChunks && p0 + e / kChunks < r.p1 && c0 + e % kChunks * V < r.c0 + r.cb;
    };
    auto in_memory = [&](int e) { return (P *)(m + (int64_t)(e / kChunks) * g.c + e % kChunks * V); };
    auto in_tile = [&](int e) { return (P *)tile_at<T, V16>(tile, e / kChunks, e % kChunks * V); };
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
        const int e = threadIdx.x + o * NT;
        if (inside(e)) v[o] = OUT ? *in_tile(e) : fetch_last<STREAM>((const P *)in_memory(e));
    }
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
        const int e = threadIdx.x + o * NT;
        if (!inside(e)) continue;
        if (OUT)
            store_last<STREAM>(in_memory(e), v[o]);
        else
            *in_tile(e) = v[o];
    }
}

// The width follows the channels alone: the planes' side may need another.
// WIDE: it is 16 bytes (an instance of its own: the registers of the narrow ones
// would cost it a third of its waves).
template <typename T, bool WIDE, int NT, bool OUT, bool STREAM = false>
__device__ inline void move_tile(T *t_, const Geometry &g, const Range &r, int p0, int c0, char *tile)
{
    constexpr int V16 = 16 / sizeof(T);
    if constexpr (WIDE)
        move_pieces<T, V16, NT, OUT, STREAM>(t_, g, r, p0, c0, tile);
    else if (g.vlast == V16 / 2)
        move_pieces<T, V16 / 2, NT, OUT, STREAM>(t_, g, r, p0, c0, tile);
    else
        move_pieces<T, 1, NT, OUT, STREAM>(t_, g, r, p0, c0, tile);
}

// The pieces of V pixels of a tile that a thread takes in the order of planes.
template <typename T, int V, int NT>
struct Pieces {
    static constexpr int kSide = 128 / sizeof(T), kChunks = kSide / V, kOwn = (kSide * kChunks + NT - 1) / NT;
    const Range &r;
    int p0, c0;
    int64_t base;
    __device__ Pieces(const Geometry &g, const Range &r_, int p0_, int c0_)
        : r(r_), p0(p0_), c0(c0_), base((r_.n * g.c + c0_) * (int64_t)g.hw + p0_)
    {
    }
    __device__ static int place(int o) { return threadIdx.x + o * NT; }
    __device__ static int channel(int o) { return place(o) / kChunks; }
    __device__ static int pixel(int o) { return place(o) % kChunks * V; }
    __device__ bool inside(int o) const
    {
        return place(o) < kSide * kChunks && c0 + channel(o) < r.c0 + r.cb && p0 + pixel(o) < r.p1;
    }
    __device__ int64_t at(const Geometry &g, int o) const { return base + (int64_t)channel(o) * g.hw + pixel(o); }
};

// ---- The passes of a range -------------------------------------------------------

// y of the range.
template <typename T, int V, bool WIDE, bool STREAM, int NT, bool XL, bool YL>
__device__ inline void apply(const T *__restrict__ x, T *__restrict__ y, const Geometry &g, const Range &r,
                             const Chan *lk, char *tile)
{
    if constexpr (XL == YL) {
        constexpr int K = XL ? V : 1;
        Chan k[K];
        typename Pack<T, V>::type raw[kBatch];
        walk<XL, V, NT>(
            g, r,
            [&](int c) {
                if (c >= 0)
#pragma unroll
                    for (int i = 0; i < K; ++i) {
                        k[i] = lk[c + i - r.c0];
                        k[i].rstd *= k[i].gamma;
                    }
            },
            [&](int u, int64_t at) { raw[u] = fetch_last<STREAM>((const typename Pack<T, V>::type *)(x + at)); },
            [&](int u, int64_t at, bool) {
                float v[V];
                values<T, V>(raw[u], v);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const Chan &q = k[XL ? i : 0];
                    v[i] = fmaf(v[i] - q.mean, q.rstd, q.beta);
                }
                act_fwd<V>(g.act, v);
                store<T, V, STREAM>(y + at, v);
            },
            [](int) {});
    } else {
        constexpr int V16 = 16 / sizeof(T);
        typedef Pieces<T, V, NT> P;
        for (int c0 = r.c0; c0 < r.c0 + r.cb; c0 += P::kSide)
            for (int p0 = r.p0; p0 < r.p1; p0 += P::kSide) {
                const P w(g, r, p0, c0);
                typename Pack<T, V>::type raw[P::kOwn];
                if (!XL)
#pragma unroll
                    for (int o = 0; o < P::kOwn; ++o)
                        if (w.inside(o)) raw[o] = fetch_last<STREAM>((const typename Pack<T, V>::type *)(x + w.at(g, o)));
                __syncthreads();  // the tile before is read
                if (XL) {
                    move_tile<T, WIDE, NT, false, STREAM>(const_cast<T *>(x), g, r, p0, c0, tile);
                    __syncthreads();
                }
#pragma unroll
                for (int o = 0; o < P::kOwn; ++o) {
                    if (!w.inside(o)) continue;
                    float v[V];
                    if (XL)
#pragma unroll
                        for (int i = 0; i < V; ++i) v[i] = (float)*tile_at<T, V16>(tile, w.pixel(o) + i, w.channel(o));
                    else
                        values<T, V>(raw[o], v);
                    const Chan k = lk[c0 + w.channel(o) - r.c0];
                    const float a = k.rstd * k.gamma;
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] = fmaf(v[i] - k.mean, a, k.beta);
                    act_fwd<V>(g.act, v);
                    if (XL)
                        store<T, V, STREAM>(y + w.at(g, o), v);
                    else
#pragma unroll
                        for (int i = 0; i < V; ++i) *tile_at<T, V16>(tile, w.pixel(o) + i, w.channel(o)) = (T)v[i];
                }
                if (!XL) {
                    __syncthreads();
                    move_tile<T, WIDE, NT, true, STREAM>(y, g, r, p0, c0, tile);
                }
            }
    }
}

// Sums of dz and dz xh of the range's channels: done(c, sums).  sums: LDS of a
// channel's sums (tiles).
template <typename T, int V, bool WIDE, int NT, bool XL, bool YL, typename D>
__device__ inline void sums_bwd(const T *__restrict__ x, const T *__restrict__ dy, const Geometry &g, const Range &r,
                                const Chan *lk, float *lds, char *tile, D done)
{
    if constexpr (XL == YL) {
        constexpr int K = XL ? V : 1;
        Chan k[K];
        SumSet<K> s, total;  // total and left: along planes
        int left;
        typename Pack<T, V>::type rx[kBatch], rd[kBatch];
        walk<XL, V, NT>(
            g, r,
            [&](int c) {
#pragma unroll
                for (int i = 0; i < K; ++i) {
                    s.a[i] = s.b[i] = 0.f;
                    if (c >= 0) k[i] = lk[c + i - r.c0];
                }
                if constexpr (!XL) {
                    total.a[0] = total.b[0] = 0.f;
                    left = kChain;
                }
            },
            [&](int u, int64_t at) {
                rx[u] = fetch<T, V>(x + at);
                rd[u] = fetch<T, V>(dy + at);
            },
            [&](int u, int64_t at, bool) {
                if constexpr (!XL)
                    if (u == 0) {
                        if (left == 0) {
                            total.add(s);
                            s.a[0] = s.b[0] = 0.f;
                            left = kChain;
                        }
                        left -= kBatch * V;
                    }
                float v[V], d[V];
                values<T, V>(rx[u], v);
                values<T, V>(rd[u], d);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int q = XL ? i : 0;
                    const float xh = (v[i] - k[q].mean) * k[q].rstd;
                    const float dz = act_bwd(g.act, d[i], v[i], xh, k[q]);
                    s.a[q] += dz;
                    s.b[q] = fmaf(dz, xh, s.b[q]);
                }
            },
            [&](int c) {
                if constexpr (!XL) s.add(total);
                if (join_threads<XL, NT>(g, c, s, lds))
#pragma unroll
                    for (int i = 0; i < K; ++i) done(c + i, make_float2(s.a[i], s.b[i]));
            });
    } else {
        constexpr int V16 = 16 / sizeof(T);
        typedef Pieces<T, V, NT> P;
        static_assert(P::kChunks <= 64 && NT % P::kChunks == 0, "a channel's threads are lanes of one wave");
        for (int c0 = r.c0; c0 < r.c0 + r.cb; c0 += P::kSide) {
            // a total only where a thread has one channel; else shorter ranges
            // (kMostUnjoined): 16x256x256x256 fp16, of two channels, 550 us
            // without either, 505 with shorter ranges, 587 with totals (a wave
            // less a SIMD), but fp32 910, 958 and 911
            constexpr bool kTotal = P::kOwn == 1;
            float2 s[P::kOwn], total = make_float2(0.f, 0.f);
#pragma unroll
            for (int o = 0; o < P::kOwn; ++o) s[o] = make_float2(0.f, 0.f);
            int left = kChain;
            auto end_chain = [&] {
                total = make_float2(total.x + s[0].x, total.y + s[0].y);
                s[0] = make_float2(0.f, 0.f);
            };
            for (int p0 = r.p0; p0 < r.p1; p0 += P::kSide) {
                if (kTotal && left == 0) {
                    end_chain();
                    left = kChain;
                }
                left -= V;
                const P w(g, r, p0, c0);
                typename Pack<T, V>::type raw[P::kOwn];
#pragma unroll
                for (int o = 0; o < P::kOwn; ++o)
                    if (w.inside(o)) raw[o] = fetch<T, V>((XL ? dy : x) + w.at(g, o));
                __syncthreads();
                move_tile<T, WIDE, NT, false>(const_cast<T *>(XL ? x : dy), g, r, p0, c0, tile);
                __syncthreads();
#pragma unroll
                for (int o = 0; o < P::kOwn; ++o) {
                    if (!w.inside(o)) continue;
                    float v[V];
                    values<T, V>(raw[o], v);
                    const Chan k = lk[c0 + w.channel(o) - r.c0];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float u = (float)*tile_at<T, V16>(tile, w.pixel(o) + i, w.channel(o));
                        const float xv = XL ? u : v[i], xh = (xv - k.mean) * k.rstd;
                        const float dz = act_bwd(g.act, XL ? v[i] : u, xv, xh, k);
                        s[o].x += dz;
                        s[o].y = fmaf(dz, xh, s[o].y);
                    }
                }
            }
            if constexpr (kTotal) {
                end_chain();
                s[0] = total;
            }
#pragma unroll
            for (int o = 0; o < P::kOwn; ++o) {
                for (int k = 1; k < P::kChunks; k <<= 1) {
                    s[o].x += __shfl_xor(s[o].x, k);
                    s[o].y += __shfl_xor(s[o].y, k);
                }
                const int j = P::channel(o);
                if (P::pixel(o) == 0 && P::place(o) < P::kSide * P::kChunks && c0 + j < r.c0 + r.cb) done(c0 + j, s[o]);
            }
        }
    }
}

// dx of the range; q: the group's means of t and t xh, by channel.
template <typename T, int V, bool WIDE, bool STREAM, int NT, bool XL, bool YL>
__device__ inline void apply_bwd(const T *__restrict__ x, const T *__restrict__ dy, T *__restrict__ dx,
                                 const Geometry &g, const Range &r, const Chan *lk, const float2 *lq,
                                 char *tile)
{
    auto value = [&](float xv, float d, const Chan &k, const float2 &q) {
        const float xh = (xv - k.mean) * k.rstd;
        const float dz = act_bwd(g.act, d, xv, xh, k);
        return k.rstd * (fmaf(k.gamma, dz, -q.x) - xh * q.y);
    };
    if constexpr (XL == YL) {
        constexpr int K = XL ? V : 1;
        Chan k[K];
        float2 q[K];
        typename Pack<T, V>::type rx[kBatch], rd[kBatch];
        walk<XL, V, NT>(
            g, r,
            [&](int c) {
                if (c >= 0)
#pragma unroll
                    for (int i = 0; i < K; ++i) {
                        k[i] = lk[c + i - r.c0];
                        q[i] = lq[c + i - r.c0];
                    }
            },
            [&](int u, int64_t at) {
                rx[u] = fetch_last<STREAM>((const typename Pack<T, V>::type *)(x + at));
                rd[u] = fetch_last<STREAM>((const typename Pack<T, V>::type *)(dy + at));
            },
            [&](int u, int64_t at, bool) {
                float v[V], d[V];
                values<T, V>(rx[u], v);
                values<T, V>(rd[u], d);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = value(v[i], d[i], k[XL ? i : 0], q[XL ? i : 0]);
                store<T, V, STREAM>(dx + at, v);
            },
            [](int) {});
    } else {
        constexpr int V16 = 16 / sizeof(T);
        typedef Pieces<T, V, NT> P;
        for (int c0 = r.c0; c0 < r.c0 + r.cb; c0 += P::kSide)
            for (int p0 = r.p0; p0 < r.p1; p0 += P::kSide) {
                const P w(g, r, p0, c0);
                typename Pack<T, V>::type raw[P::kOwn];
#pragma unroll
                for (int o = 0; o < P::kOwn; ++o)
                    if (w.inside(o)) raw[o] = fetch_last<STREAM>((const typename Pack<T, V>::type *)((XL ? dy : x) + w.at(g, o)));
                __syncthreads();
                move_tile<T, WIDE, NT, false, STREAM>(const_cast<T *>(XL ? x : dy), g, r, p0, c0, tile);
                __syncthreads();
#pragma unroll
                for (int o = 0; o < P::kOwn; ++o) {
                    if (!w.inside(o)) continue;
                    float v[V];
                    values<T, V>(raw[o], v);
                    const Chan k = lk[c0 + w.channel(o) - r.c0];
                    const float2 q = lq[c0 + w.channel(o) - r.c0];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        T *u = tile_at<T, V16>(tile, w.pixel(o) + i, w.channel(o));
                        v[i] = XL ? value((float)*u, v[i], k, q) : value(v[i], (float)*u, k, q);
                        if (XL) *u = (T)v[i];
                    }
                    if (!XL) store<T, V, STREAM>(dx + w.at(g, o), v);
                }
                if (XL) {
                    __syncthreads();
                    move_tile<T, WIDE, NT, true, STREAM>(dx, g, r, p0, c0, tile);
                }
            }
    }
}

// ---- Kernels -----------------------------------------------------------------------

constexpr int kTileBytes(size_t esize) { return 8 * 16 / (int)esize * 128; }

// Moments of the range's channels: part[(n splits + split) C + c].
template <typename T, int V, bool XL>
__global__ __launch_bounds__(kThreads) void norm_moments(const T *__restrict__ x, Geometry g,
                                                         float2 *__restrict__ part)
{
    __shared__ float lds[(1 + 2 * (XL ? V : 1)) * kThreads];
    const Range r = range_of(g, kForth, blockIdx.x);
    moments<T, XL, V, kThreads>(x, g, r, lds,
                                [&](int c, const Moments &m) { part[r.row * g.c + c] = make_float2(m.mean, m.m2); });
}

__device__ inline void load_consts(Chan *lk, const Geometry &g, const Range &r, const float *__restrict__ gamma,
                                   const float *__restrict__ beta, const float *__restrict__ mean,
                                   const float *__restrict__ rstd)
{
    for (int i = threadIdx.x; i < r.cb; i += blockDim.x) {
        const int c = r.c0 + i;
        const int64_t ng = r.n * g.groups + c / g.per;
        lk[i] = Chan{mean[ng], rstd[ng], gamma ? gamma[c] : 1.f, beta ? beta[c] : 0.f};
    }
    __syncthreads();
}

__device__ inline float add_lanes(float v, int lanes)
{
    for (int o = 1; o < lanes; o <<= 1) v += __shfl_xor(v, o);
    return v;
}

// mean and rstd of the groups that the range's channels belong to, from the
// channels' moments in pixel ranges (geometry gs), w.lanes neighbouring lanes a
// group: mean = sum of n_i mean_i / K, then M2 = sum of M2_i + n_i (mean_i -
// mean)^2.  lg: by place among those groups; mean, rstd: by each image's first
// workgroup.
__device__ inline void own_stats(const Geometry &gs, const Range &r, const Own &w, const float2 *__restrict__ part,
                                 float eps, float2 *lg, float *mean, float *rstd)
{
    const int lanes = w.lanes, k = threadIdx.x / lanes, lane = threadIdx.x % lanes, group = r.c0 / gs.per + k;
    if (group > (r.c0 + r.cb - 1) / gs.per) return;
    const float2 *p = part + r.n * gs.splits * (int64_t)gs.c + group * gs.per;
    const float inv = 1.f / ((float)gs.per * (float)gs.hw);
    float2 v[kOwnSums];
    float n[kOwnSums], m = 0.f, q = 0.f;
    int s = lane / gs.per, c = lane - s * gs.per;
#pragma unroll
    for (int u = 0; u < kOwnSums; ++u) {
        n[u] = 0.f;
        if (s < gs.splits) {
            v[u] = p[(int64_t)s * gs.c + c];
            n[u] = (float)pixels(gs, s) * inv;
        }
        c += w.channels;
        s += w.ranges;
        if (c >= gs.per) {
            c -= gs.per;
            ++s;
        }
    }
#pragma unroll
    for (int u = 0; u < kOwnSums; ++u)
        if (n[u] > 0.f) m = fmaf(n[u], v[u].x, m);
    m = add_lanes(m, lanes);
#pragma unroll
    for (int u = 0; u < kOwnSums; ++u)
        if (n[u] > 0.f) {
            const float d = v[u].x - m;
            q += fmaf(d * n[u], d, v[u].y * inv);
        }
    q = add_lanes(q, lanes);
    if (lane) return;
    const float rs = 1.f / sqrtf(q + eps);
    lg[k] = make_float2(m, rs);
    if (r.p0 == 0 && group * gs.per >= r.c0) {
        mean[r.n * gs.groups + group] = m;
        rstd[r.n * gs.groups + group] = rs;
    }
}

// own.lanes > 0: own_stats() in place of a kernel between the two walks.
template <typename T, int V, bool WIDE, bool STREAM, bool XL, bool YL>
__global__ __launch_bounds__(kThreads) void norm_apply(const T *__restrict__ x, const float *__restrict__ gamma,
                                                       const float *__restrict__ beta, float *mean, float *rstd,
                                                       T *__restrict__ y, Geometry g, Geometry gs, Own own,
                                                       const float2 *__restrict__ part, float eps)
{
    __shared__ Chan lk[kMaxBlock];
    __shared__ float2 lg[kThreads];
    __shared__ __attribute__((aligned(16))) char tile[XL != YL ? kTileBytes(sizeof(T)) : 16];
    const Range r = range_of(g, kBack, blockIdx.x);
    if (own.lanes) {
        own_stats(gs, r, own, part, eps, lg, mean, rstd);
        __syncthreads();
        for (int i = threadIdx.x; i < r.cb; i += kThreads) {
            const int c = r.c0 + i;
            const float2 m = lg[c / g.per - r.c0 / g.per];
            lk[i] = Chan{m.x, m.y, gamma ? gamma[c] : 1.f, beta ? beta[c] : 0.f};
        }
        __syncthreads();
    } else {
        load_consts(lk, g, r, gamma, beta, mean, rstd);
    }
    apply<T, V, WIDE, STREAM, kThreads, XL, YL>(x, y, g, r, lk, tile);
}

template <typename T, int V, bool WIDE, bool XL, bool YL>
__global__ __launch_bounds__(kThreads) void norm_sums_bwd(const T *__restrict__ x, const T *__restrict__ dy,
                                                          const float *__restrict__ gamma,
                                                          const float *__restrict__ beta,
                                                          const float *__restrict__ mean,
                                                          const float *__restrict__ rstd, Geometry g,
                                                          float2 *__restrict__ part)
{
    __shared__ Chan lk[kMaxBlock];
    __shared__ float lds[2 * (XL ? V : 1) * kThreads];
    __shared__ __attribute__((aligned(16))) char tile[XL != YL ? kTileBytes(sizeof(T)) : 16];
    const Range r = range_of(g, kForth, blockIdx.x);
    load_consts(lk, g, r, gamma, beta, mean, rstd);
    sums_bwd<T, V, WIDE, kThreads, XL, YL>(x, dy, g, r, lk, lds, tile,
                                     [&](int c, const float2 &s) { part[r.row * g.c + c] = s; });
}

template <typename T, int V, bool WIDE, bool STREAM, bool XL, bool YL>
__global__ __launch_bounds__(kThreads) void norm_apply_bwd(const T *__restrict__ x, const T *__restrict__ dy,
                                                           const float *__restrict__ gamma,
                                                           const float *__restrict__ beta,
                                                           const float *__restrict__ mean,
                                                           const float *__restrict__ rstd,
                                                           const float2 *__restrict__ means, T *__restrict__ dx,
                                                           Geometry g)
{
    __shared__ Chan lk[kMaxBlock];
    __shared__ float2 lq[kMaxBlock];
    __shared__ __attribute__((aligned(16))) char tile[XL != YL ? kTileBytes(sizeof(T)) : 16];
    const Range r = range_of(g, kBack, blockIdx.x);
    for (int i = threadIdx.x; i < r.cb; i += kThreads) lq[i] = means[r.n * g.groups + (r.c0 + i) / g.per];
    load_consts(lk, g, r, gamma, beta, mean, rstd);
    apply_bwd<T, V, WIDE, STREAM, kThreads, XL, YL>(x, dy, dx, g, r, lk, lq, tile);
}

// ---- One launch ----------------------------------------------------------------------

// Joins the range's channels' values in LDS over each group, one wave a group:
// done(first channel's place, joined) on lane 0.
template <int NT, typename S, typename V, typename J, typename D>
__device__ inline void join_groups(const Geometry &g, const Range &r, V value, S zero, J join2, D done)
{
    const int lane = threadIdx.x & 63;
    for (int k = threadIdx.x >> 6; k < r.cb / g.per; k += NT / 64) {
        S s = zero;
        for (int i = lane; i < g.per; i += 64) s = join2(s, value(k * g.per + i));
        s = join_wave(s, join2);
        if (lane == 0) done(k * g.per, s);
    }
}

template <typename T, int V, bool WIDE, bool STREAM, bool XL, bool YL>
__global__ __launch_bounds__(kOneThreads) void norm_one(const T *__restrict__ x, const float *__restrict__ gamma,
                                                        const float *__restrict__ beta, T *__restrict__ y,
                                                        float *__restrict__ mean, float *__restrict__ rstd, Geometry g,
                                                        Geometry ga, float eps)
{
    __shared__ Chan lk[kMaxBlock];
    __shared__ Moments lm[kMaxBlock];
    __shared__ float lds[(1 + 2 * (XL ? V : 1)) * kOneThreads];
    __shared__ __attribute__((aligned(16))) char tile[XL != YL ? kTileBytes(sizeof(T)) : 16];
    const Range r = range_of(g, XL || YL ? kForth : kPlain, blockIdx.x);
    moments<T, XL, V, kOneThreads>(x, g, r, lds, [&](int c, const Moments &m) { lm[c - r.c0] = m; });
    __syncthreads();
    join_groups<kOneThreads>(
        g, r, [&](int i) { return lm[i]; }, Moments{0.f, 0.f, 0.f}, join,
        [&](int i, const Moments &m) {
            const float rs = 1.f / sqrtf(m.m2 / m.n + eps);
            const int64_t ng = r.n * g.groups + (r.c0 + i) / g.per;
            mean[ng] = m.mean;
            rstd[ng] = rs;
            lk[i].mean = m.mean;
            lk[i].rstd = rs;
        });
    __syncthreads();
    for (int i = threadIdx.x; i < r.cb; i += kOneThreads) {
        const int f = i - i % g.per, c = r.c0 + i;
        const float m = lk[f].mean, rs = lk[f].rstd;
        if (i != f) {
            lk[i].mean = m;
            lk[i].rstd = rs;
        }
        lk[i].gamma = gamma ? gamma[c] : 1.f;
        lk[i].beta = beta ? beta[c] : 0.f;
    }
    __syncthreads();
    apply<T, V, WIDE, STREAM, kOneThreads, XL, YL>(x, y, ga, r, lk, tile);
}

template <typename T, int V, bool WIDE, bool STREAM, bool XL, bool YL>
__global__ __launch_bounds__(kOneThreads) void norm_one_bwd(const T *__restrict__ x, const T *__restrict__ dy,
                                                            const float *__restrict__ gamma,
                                                            const float *__restrict__ beta,
                                                            const float *__restrict__ mean,
                                                            const float *__restrict__ rstd, T *__restrict__ dx,
                                                            Geometry g, float2 *__restrict__ part)
{
    __shared__ Chan lk[kMaxBlock];
    __shared__ float2 ls[kMaxBlock], lq[kMaxBlock];
    __shared__ float lds[2 * (XL ? V : 1) * kOneThreads];
    __shared__ __attribute__((aligned(16))) char tile[XL != YL ? kTileBytes(sizeof(T)) : 16];
    const Range r = range_of(g, XL || YL ? kForth : kPlain, blockIdx.x);
    load_consts(lk, g, r, gamma, beta, mean, rstd);
    sums_bwd<T, V, WIDE, kOneThreads, XL, YL>(x, dy, g, r, lk, lds, tile, [&](int c, const float2 &s) {
        ls[c - r.c0] = s;
        if (part) part[r.n * g.c + c] = s;
    });
    __syncthreads();
    join_groups<kOneThreads>(
        g, r, [&](int i) { return make_float2(lk[i].gamma * ls[i].x, lk[i].gamma * ls[i].y); },
        make_float2(0.f, 0.f), [](const float2 &a, const float2 &b) { return make_float2(a.x + b.x, a.y + b.y); },
        [&](int i, const float2 &s) {
            const float k = (float)g.per * (float)g.hw;
            lq[i] = make_float2(s.x / k, s.y / k);
        });
    __syncthreads();
    for (int i = threadIdx.x; i < r.cb; i += kOneThreads)
        if (i % g.per) lq[i] = lq[i - i % g.per];
    __syncthreads();
    apply_bwd<T, V, WIDE, STREAM, kOneThreads, XL, YL>(x, dy, dx, g, r, lk, lq, tile);
}

// ---- Launches ------------------------------------------------------------------------

template <typename T, int V, bool WIDE, bool STREAM, bool XL, bool YL>
hipError_t forward_v(const Plan &p, const Call &a, hipStream_t stream)
{
    const T *x = (const T *)a.x;
    if (p.one) {
        norm_one<T, V, WIDE, STREAM, XL, YL><<<dim3((unsigned)p.apply.count), dim3(kOneThreads), 0, stream>>>(
            x, a.gamma, a.beta, (T *)a.out, a.mean_out, a.rstd_out, p.stats, p.apply, p.eps);
        return hipGetLastError();
    }
    const dim3 th(kThreads);
    float2 *part = (float2 *)a.workspace;
    norm_moments<T, V, XL><<<dim3((unsigned)p.stats.count), th, 0, stream>>>(x, p.stats, part);
    if (!p.own.lanes) launch_finish_forward(p.stats, a.n, part, a.mean_out, a.rstd_out, p.eps, stream);
    norm_apply<T, V, WIDE, STREAM, XL, YL><<<dim3((unsigned)p.apply.count), th, 0, stream>>>(
        x, a.gamma, a.beta, a.mean_out, a.rstd_out, (T *)a.out, p.apply, p.stats, p.own, part, p.eps);
    return hipGetLastError();
}

template <typename T, int V, bool WIDE, bool STREAM, bool XL, bool YL>
hipError_t backward_v(const Plan &p, const Call &a, hipStream_t stream)
{
    const Geometry &g = p.apply;
    const T *x = (const T *)a.x, *dy = (const T *)a.dy;
    float2 *part = (float2 *)a.workspace, *means = (float2 *)((char *)a.workspace + p.means_at);
    if constexpr (XL == YL) {
        if (p.one) {
            float2 *sums = a.dgamma || a.dbeta ? part : nullptr;
            norm_one_bwd<T, V, WIDE, STREAM, XL, YL><<<dim3((unsigned)g.count), dim3(kOneThreads), 0, stream>>>(
                x, dy, a.gamma, a.beta, a.mean, a.rstd, (T *)a.out, g, sums);
            if (sums) launch_finish_backward(g, a.n, sums, a.gamma, nullptr, a.dgamma, a.dbeta, stream);
            return hipGetLastError();
        }
    }
    const dim3 th(kThreads), grid((unsigned)g.count);
    norm_sums_bwd<T, V, WIDE, XL, YL><<<grid, th, 0, stream>>>(x, dy, a.gamma, a.beta, a.mean, a.rstd, g, part);
    launch_finish_backward(g, a.n, part, a.gamma, means, a.dgamma, a.dbeta, stream);
    norm_apply_bwd<T, V, WIDE, STREAM, XL, YL>
        <<<grid, th, 0, stream>>>(x, dy, a.gamma, a.beta, a.mean, a.rstd, means, (T *)a.out, g);
    return hipGetLastError();
}

template <typename T, int V, bool WIDE, bool XL, bool YL>
hipError_t run_v(const Plan &p, const Call &a, hipStream_t stream)
{
    if (!a.dy)
        return p.apply.stream ? forward_v<T, V, WIDE, true, XL, YL>(p, a, stream)
                              : forward_v<T, V, WIDE, false, XL, YL>(p, a, stream);
    if constexpr (V <= vector_of(sizeof(T), XL, YL, true))
        return p.apply.stream ? backward_v<T, V, WIDE, true, XL, YL>(p, a, stream)
                              : backward_v<T, V, WIDE, false, XL, YL>(p, a, stream);
    return hipErrorInvalidValue;  // no such plan
}

template <typename T, bool WIDE, bool XL, bool YL>
hipError_t run_layout(const Plan &p, const Call &a, hipStream_t stream)
{
    constexpr int V16 = 16 / sizeof(T);
    if (p.v == V16) return run_v<T, V16, WIDE, XL, YL>(p, a, stream);
    if (p.v == V16 / 2) return run_v<T, V16 / 2, WIDE, XL, YL>(p, a, stream);
    return run_v<T, 1, WIDE, XL, YL>(p, a, stream);
}

template <typename T>
hipError_t run(const Plan &p, const Call &a, hipStream_t stream)
{
    if (p.xl && p.yl) return run_layout<T, true, true, true>(p, a, stream);
    if (!p.xl && !p.yl) return run_layout<T, true, false, false>(p, a, stream);
    const bool wide = p.apply.vlast == 16 / (int)sizeof(T);
    if (p.xl)
        return wide ? run_layout<T, true, true, false>(p, a, stream) : run_layout<T, false, true, false>(p, a, stream);
    return wide ? run_layout<T, true, false, true>(p, a, stream) : run_layout<T, false, false, true>(p, a, stream);
}

}  // namespace wtc_norm

#endif  // WTCONV_NORM_BODY_H
