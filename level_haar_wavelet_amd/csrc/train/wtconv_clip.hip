// wtconv_clip.hip -- the norm over the elements of many tensors, and their scaling
// to a largest norm.
//
// Two passes over the data, both bound by memory: the squares' sums, and the
// scaling, which cannot begin before the last of them.  The elements of all tensors
// are cut into ranges of the same length, at most about 8192 (with 2048 of them, about
// as many workgroups as the chip holds, 414e6 elements took 577 us in place of 527: the
// last few run alone); a workgroup sums one, and the scaling's workgroups each add the
// ranges' sums for themselves, in the same order everywhere, which saves a launch
// between (more than kOwnSums of them, 20 KB out of the L2, one workgroup adds first).
// The second pass takes the ranges from the last to the first: the 256 MB cache holds
// the end of what the first read.  414e6 bf16 elements in 416 tensors: 139 us for the sums
// (6.0 TB/s), 298 for the scaling (5.6).
//
// The table of tensors goes by value with a launch (it is then the captured call's
// own, and needs no copy from host memory that has to stay): of up to kByValue of
// them with both kernels, of more with small launches in front that write it to the
// workspace, so that the passes run whole (416 tensors in four launches for each
// pass, with four ends to wait for: 576 us).
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
constexpr int kWritten = 100;  // entries of a launch that writes the table

// The table with the launch, or in the workspace.
struct Table {
    const void *in_[kByValue];
    void *out_[kByValue];
    int64_t elems_type_[kByValue];
    int first_[kByValue];
    int n;
    int ranges;
    int64_t range;  // elements of a range
    __device__ const void *in(int i) const { return in_[i]; }
    __device__ void *out(int i) const { return out_[i]; }
    __device__ int64_t elems_type(int i) const { return elems_type_[i]; }
    __device__ int first(int i) const { return first_[i]; }
};
static_assert(sizeof(Table) + 64 <= 4096, "a kernel's arguments");

struct FarTable {
    const Entry *e;
    int n;
    int ranges;
    int64_t range;
    __device__ const void *in(int i) const { return e[i].in; }
    __device__ void *out(int i) const { return e[i].out; }
    __device__ int64_t elems_type(int i) const { return e[i].elems_type; }
    __device__ int first(int i) const { return (int)e[i].first; }
};

struct Entries {
    Entry e[kWritten];
};
static_assert(sizeof(Entries) + 64 <= 4096, "a kernel's arguments");

__global__ void write_table(Entries from, Entry *to, int n)
{
    if ((int)threadIdx.x < n) to[threadIdx.x] = from.e[threadIdx.x];
}

// The tensor that range r belongs to.
template <typename T>
__device__ inline int find(const T &t, int r)
{
    int lo = 0, hi = t.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.first(mid) <= r)
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

// STREAM: stores past the L2s, which keep what is still to be read.
template <typename T, int V, bool STREAM>
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
        for (int k = 0; k < 4; ++k) {
            if constexpr (STREAM)
                __builtin_nontemporal_store(times(v[k]), (P *)(o + e + k * step));
            else
                *(P *)(o + e + k * step) = times(v[k]);
        }
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

template <typename T, bool STREAM>
__device__ inline void scale_any(const void *p, void *o, int64_t e, int64_t end, const Scale &f)
{
    if ((((uintptr_t)p | (uintptr_t)o) & 15) == 0)
        scale<T, 16 / sizeof(T), STREAM>((const T *)p, (T *)o, e, end, f);
    else
        scale<T, 1, STREAM>((const T *)p, (T *)o, e, end, f);
}

template <typename L>
__global__ __launch_bounds__(kThreads) void norm_ranges(L t, double *parts)
{
    const int r = blockIdx.x, i = find(t, r);
    const int64_t et = t.elems_type(i), n = et >> 2, e = (r - t.first(i)) * t.range;
    const int64_t end = n - e < t.range ? n : e + t.range;
    const int type = (int)(et & 3);
    const void *in = t.in(i);
    double a;
    if (type == WTCONV_F32)
        a = squares_of<float>(in, e, end);
    else if (type == WTCONV_F16)
        a = squares_of<_Float16>(in, e, end);
    else
        a = squares_of<__bf16>(in, e, end);
    a = sum_group(a);
    if (threadIdx.x == 0) parts[r] = a;
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

template <typename L, bool STREAM>
__global__ __launch_bounds__(kThreads) void clip_ranges(L t, const double *parts, int64_t n, float max_norm, float eps,
                                                        float *norm)
{
    const double root = sqrt(total_of(parts, n));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)root;
    const Scale f = scale_of((double)max_norm / (root + (double)eps));
    const int r = t.ranges - 1 - blockIdx.x, i = find(t, r);
    const void *in = t.in(i);
    void *out = t.out(i);
    if (f.two == 1.f && f.f == 1.f && in == out) return;
    const int64_t et = t.elems_type(i), m = et >> 2, e = (r - t.first(i)) * t.range;
    const int64_t end = m - e < t.range ? m : e + t.range;
    const int type = (int)(et & 3);
    if (type == WTCONV_F32)
        scale_any<float, STREAM>(in, out, e, end, f);
    else if (type == WTCONV_F16)
        scale_any<_Float16, STREAM>(in, out, e, end, f);
    else
        scale_any<__bf16, STREAM>(in, out, e, end, f);
}

struct Clip {
    bool clip;
    float max_norm, eps;
    float *norm;
    double *parts, *total;
    int64_t elems;
};

template <typename L>
void passes(const L &t, const Clip &c, hipStream_t stream)
{
    const dim3 grid((unsigned)t.ranges), block(kThreads);
    const bool joined = t.ranges > kOwnSums;
    norm_ranges<L><<<grid, block, 0, stream>>>(t, c.parts);
    if (!c.clip || joined) norm_join<<<dim3(1), block, 0, stream>>>(c.parts, t.ranges, c.total, c.norm);
    if (!c.clip) return;
    auto *k = c.elems >= kStream ? clip_ranges<L, true> : clip_ranges<L, false>;
    k<<<grid, block, 0, stream>>>(t, joined ? c.total : c.parts, joined ? 1 : t.ranges, c.max_norm, c.eps,
                                  joined ? nullptr : c.norm);
}

}  // namespace

hipError_t wtc_launch_clip(const wtconv_tensor_t *t, int64_t count, bool clip, float max_norm, float eps, float *norm,
                           double *parts, hipStream_t stream)
{
    int64_t all = 0;
    for (int64_t i = 0; i < count; ++i) all += t[i].elems;
    const int64_t range = range_elems(all);
    const Clip c = {clip, max_norm, eps, norm, parts, parts + kRanges + count, all};
    int ranges = 0, n = 0;
    // f(n-th tensor with elements, its entry)
    auto each = [&](auto f) {
        for (int64_t i = 0; i < count; ++i)
            if (t[i].elems) {
                f(n++, Entry{t[i].grad, t[i].out, t[i].elems * 4 + t[i].dtype, ranges});
                ranges += (int)((t[i].elems + range - 1) / range);
            }
    };
    if (!all) {
        norm_join<<<dim3(1), dim3(kThreads), 0, stream>>>(parts, 0, nullptr, norm);
    } else if (count <= kByValue) {
        Table tab;
        each([&](int i, const Entry &e) {
            tab.in_[i] = e.in;
            tab.out_[i] = e.out;
            tab.elems_type_[i] = e.elems_type;
            tab.first_[i] = (int)e.first;
        });
        tab.n = n;
        tab.ranges = ranges;
        tab.range = range;
        passes(tab, c, stream);
    } else {
        Entry *to = (Entry *)((char *)parts + sums_bytes(count));
        Entries some;
        int k = 0;
        auto flush = [&] {
            if (k) write_table<<<dim3(1), dim3(128), 0, stream>>>(some, to, k);
            to += k;
            k = 0;
        };
        const Entry *table = to;
        each([&](int, const Entry &e) {
            some.e[k++] = e;
            if (k == kWritten) flush();
        });
        flush();
        passes(FarTable{table, n, ranges, range}, c, stream);
    }
    return hipGetLastError();
}
