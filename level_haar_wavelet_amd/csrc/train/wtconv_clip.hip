// wtconv_clip.hip -- the norm over the elements of many tensors, and their scaling
// to a largest norm.
//
// Two passes over the data, both bound by memory: the squares' sums, and the
// scaling, which cannot begin before the last of them.  The elements of all tensors
// are cut into about 2048 ranges of the same length; a workgroup sums one, and the
// scaling's workgroups each add the ranges' sums for themselves (2048 of them: 16 KB
// out of the L2), in the same order everywhere, which saves a launch between.  The
// second pass takes the ranges from the last to the first: the 256 MB cache holds
// the end of what the first read.
//
// The table of tensors goes by value with the launch (it is then the captured
// call's own, and needs no copy), so a launch takes kTensors of them.
//
// Squares and sums are fp64: fp32 squares overflow from 2^64 on and vanish below
// 2^-75, and 10^9 of them would lose digits; the fp64 rate is above memory's.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cstdint>

#include "wtconv_check.h"
#include "wtconv_clip.h"

namespace {

using namespace wtc_clip;

constexpr int kThreads = 256;
constexpr int kTensors = 120;  // of a launch: 28 bytes each in the 4 KB of a kernel's arguments

struct Table {
    const void *in[kTensors];
    void *out[kTensors];
    int64_t elems_type[kTensors];  // elements * 4 + type
    int first[kTensors];           // this launch's first range of the tensor
    int n, ranges;
    int64_t range;  // elements of a range
    int64_t base;   // ranges of the launches before
};
static_assert(sizeof(Table) <= 3500 && sizeof(Table) + 64 <= 4096, "a kernel's arguments");

// The tensor that range r belongs to.
__device__ inline int find(const Table &t, int r)
{
    int lo = 0, hi = t.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.first[mid] <= r)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

template <typename T, int V>
struct Access {
    typedef T type __attribute__((ext_vector_type(V)));
};
template <typename T>
struct Access<T, 1> {
    typedef T type;
};

__device__ inline double sum_group(double a)
{
    __shared__ double lds[kThreads / 64];
    for (int o = 32; o; o >>= 1) a += __shfl_xor(a, o);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = a;
    __syncthreads();
    a = 0.0;
    for (int i = 0; i < kThreads / 64; ++i) a += lds[i];
    return a;
}

// Elements [e, end) of p, V an access.
template <typename T, int V>
__device__ inline double squares(const T *p, int64_t e, int64_t end)
{
    typedef typename Access<T, V>::type P;
    double a = 0.0;
    auto add = [&](const P &v) {
        if constexpr (V == 1)
            a = fma((double)(float)v, (double)(float)v, a);
        else
#pragma unroll
            for (int i = 0; i < V; ++i) a = fma((double)(float)v[i], (double)(float)v[i], a);
    };
    e += threadIdx.x * V;
    constexpr int64_t step = kThreads * V;
    for (; e + 3 * step + V <= end; e += 4 * step) {
        P v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = *(const P *)(p + e + k * step);
#pragma unroll
        for (int k = 0; k < 4; ++k) add(v[k]);
    }
    for (; e + V <= end; e += step) add(*(const P *)(p + e));
    // what is left of the last access
    if (V > 1)
        for (; e < end; ++e) a = fma((double)(float)p[e], (double)(float)p[e], a);
    return a;
}

// A factor as a power of two and the rest: one that is subnormal in fp32 would have
// few digits (fp32 gradients whose norm is beyond fp32).
struct Scale {
    float two, f;
    __device__ float operator()(float v) const { return v * two * f; }
};

__device__ inline Scale scale_of(double q)
{
    if (q >= 1.0) return {1.f, 1.f};
    // half of the exponent first: no value on the way is smaller than the result
    if (q > 0.0 && q < 0x1p-126) {
        const int e = ilogb(q) / 2;
        return {(float)ldexp(1.0, e), (float)ldexp(q, -e)};
    }
    return {1.f, (float)q};  // NaN stays
}

template <typename T, int V>
__device__ inline void scale(const T *p, T *o, int64_t e, int64_t end, const Scale &f)
{
    typedef typename Access<T, V>::type P;
    auto times = [&](P v) {
        if constexpr (V == 1)
            v = (T)f((float)v);
        else
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = (T)f((float)v[i]);
        return v;
    };
    e += threadIdx.x * V;
    constexpr int64_t step = kThreads * V;
    for (; e + 3 * step + V <= end; e += 4 * step) {
        P v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = *(const P *)(p + e + k * step);
#pragma unroll
        for (int k = 0; k < 4; ++k) *(P *)(o + e + k * step) = times(v[k]);
    }
    for (; e + V <= end; e += step) *(P *)(o + e) = times(*(const P *)(p + e));
    if (V > 1)
        for (; e < end; ++e) o[e] = (T)f((float)p[e]);
}

template <typename T>
__device__ inline double squares_of(const void *p, int64_t e, int64_t end)
{
    if (((uintptr_t)p & 15) == 0) return squares<T, 16 / sizeof(T)>((const T *)p, e, end);
    return squares<T, 1>((const T *)p, e, end);
}

template <typename T>
__device__ inline void scale_any(const void *p, void *o, int64_t e, int64_t end, const Scale &f)
{
    if ((((uintptr_t)p | (uintptr_t)o) & 15) == 0)
        scale<T, 16 / sizeof(T)>((const T *)p, (T *)o, e, end, f);
    else
        scale<T, 1>((const T *)p, (T *)o, e, end, f);
}

__global__ __launch_bounds__(kThreads) void norm_ranges(Table t, double *parts)
{
    const int r = blockIdx.x, i = find(t, r), type = (int)(t.elems_type[i] & 3);
    const int64_t n = t.elems_type[i] >> 2, e = (r - t.first[i]) * t.range, end = n - e < t.range ? n : e + t.range;
    double a;
    if (type == WTCONV_F32)
        a = squares_of<float>(t.in[i], e, end);
    else if (type == WTCONV_F16)
        a = squares_of<_Float16>(t.in[i], e, end);
    else
        a = squares_of<__bf16>(t.in[i], e, end);
    a = sum_group(a);
    if (threadIdx.x == 0) parts[t.base + r] = a;
}

// The sum of n parts on every thread of the workgroup, in the same order in every
// workgroup.
__device__ inline double total_of(const double *parts, int64_t n)
{
    double a = 0.0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < n; i += kThreads) a += parts[i];
    return sum_group(a);
}

__global__ __launch_bounds__(kThreads) void norm_join(const double *parts, int64_t n, double *total, float *norm)
{
    const double a = total_of(parts, n);
    if (threadIdx.x) return;
    if (total) *total = a;
    if (norm) *norm = (float)sqrt(a);
}

__global__ __launch_bounds__(kThreads) void clip_ranges(Table t, const double *parts, int64_t n, float max_norm,
                                                        float eps, float *norm)
{
    const double root = sqrt(total_of(parts, n));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)root;
    const Scale f = scale_of((double)max_norm / (root + (double)eps));
    const int r = t.ranges - 1 - blockIdx.x, i = find(t, r), type = (int)(t.elems_type[i] & 3);
    if (f.two == 1.f && f.f == 1.f && t.in[i] == t.out[i]) return;
    const int64_t m = t.elems_type[i] >> 2, e = (r - t.first[i]) * t.range, end = m - e < t.range ? m : e + t.range;
    if (type == WTCONV_F32)
        scale_any<float>(t.in[i], t.out[i], e, end, f);
    else if (type == WTCONV_F16)
        scale_any<_Float16>(t.in[i], t.out[i], e, end, f);
    else
        scale_any<__bf16>(t.in[i], t.out[i], e, end, f);
}

}  // namespace

hipError_t wtc_launch_clip(const wtconv_tensor_t *t, int64_t count, bool clip, float max_norm, float eps, float *norm,
                           double *parts, hipStream_t stream)
{
    int64_t all = 0;
    for (int64_t i = 0; i < count; ++i) all += t[i].elems;
    const int64_t range = range_elems(all);
    int64_t ranges = 0;
    // every launch's table, once for the sums and once for the scaling
    auto each = [&](auto launch) {
        Table tab;
        tab.n = 0;
        tab.ranges = 0;
        tab.range = range;
        tab.base = 0;
        for (int64_t i = 0; i < count; ++i) {
            if (t[i].elems) {
                tab.in[tab.n] = t[i].grad;
                tab.out[tab.n] = t[i].out;
                tab.elems_type[tab.n] = t[i].elems * 4 + t[i].dtype;
                tab.first[tab.n++] = tab.ranges;
                tab.ranges += (int)((t[i].elems + range - 1) / range);
            }
            if (tab.n == kTensors || (i + 1 == count && tab.n)) {
                launch(tab);
                tab.base += tab.ranges;
                tab.n = tab.ranges = 0;
            }
        }
        ranges = tab.base;
    };
    each([&](const Table &tab) {
        norm_ranges<<<dim3((unsigned)tab.ranges), dim3(kThreads), 0, stream>>>(tab, parts);
    });
    double *total = parts + kRanges + count;
    if (!clip || ranges > kOwnSums || !ranges)
        norm_join<<<dim3(1), dim3(kThreads), 0, stream>>>(parts, ranges, total, norm);
    if (!clip) return hipGetLastError();
    const bool joined = ranges > kOwnSums;
    float *own = joined ? nullptr : norm;
    const double *from = joined ? total : parts;
    const int64_t n = joined ? 1 : ranges;
    each([&](const Table &tab) {
        clip_ranges<<<dim3((unsigned)tab.ranges), dim3(kThreads), 0, stream>>>(tab, from, n, max_norm, eps, own);
        own = nullptr;
    });
    return hipGetLastError();
}
