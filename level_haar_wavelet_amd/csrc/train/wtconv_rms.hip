// wtconv_rms.hip -- root-mean-square norm of rows with the residual's addition,
// forward and backward.
//
// A row is read once: a row's `lanes` threads keep it in registers between the sum
// of its squares and the outputs, so the bytes are the operator's own (x and the
// residual in, y and the sum out), and both directions are bound by memory.
// Rows longer than the registers hold (kMaxHeld accesses of 256 threads) are
// walked twice.
//
// A thread takes V elements an access, 16 bytes where the addresses allow it.
// Rows whose length V does not divide start at any place between two such
// accesses; they are covered by the accesses that touch them, and the first and
// the last of these go element by element (RAGGED).  Row r's start repeats with
// period V, and a backward slot takes rows a multiple of V apart, so that its
// threads keep their columns, and the sums of dgamma stay in registers over all of
// a slot's rows.
//
// Numerics.  Values are fp32 from the load on (h first rounded to its type, since
// that is what the backward pass finds).  A thread sums at most 64 squares, then a
// tree; longer rows sum in fp64.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cstdint>

#include "wtconv_check.h"
#include "wtconv_rms.h"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxHeld = 8;     // accesses of a row that a thread keeps, forward
constexpr int kMaxHeldBack = 4;  // backward: three values of each element
constexpr int kGroups = 1024;   // workgroups of the backward pass, which share out the rows
constexpr int kChain = 64;      // rows of a slot, where there are more for it

template <typename T, int V>
struct Access {
    typedef T type __attribute__((ext_vector_type(V)));
};
template <typename T>
struct Access<T, 1> {
    typedef T type;
};

// Elements e .. e + V of p as fp32, those outside [lo, hi) as zeros.
template <typename T, int V, bool RAGGED>
__device__ inline void load(const T *p, int64_t e, int64_t lo, int64_t hi, float (&v)[V])
{
    if (!RAGGED || (e >= lo && e + V <= hi)) {
        const typename Access<T, V>::type r = *(const typename Access<T, V>::type *)(p + e);
        if constexpr (V == 1)
            v[0] = (float)r;
        else
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = (float)r[i];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = e + i >= lo && e + i < hi ? (float)p[e + i] : 0.f;
    }
}

template <typename T, int V, bool RAGGED>
__device__ inline void store(T *p, int64_t e, int64_t lo, int64_t hi, const float (&v)[V])
{
    if (!RAGGED || (e >= lo && e + V <= hi)) {
        typename Access<T, V>::type r;
        if constexpr (V == 1)
            r = (T)v[0];
        else
#pragma unroll
            for (int i = 0; i < V; ++i) r[i] = (T)v[i];
        *(typename Access<T, V>::type *)(p + e) = r;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e + i >= lo && e + i < hi) p[e + i] = (T)v[i];
    }
}

// gamma of columns c .. c + V, zeros outside the row.
template <int V, bool RAGGED>
__device__ inline void weights(const float *gamma, int64_t c, int64_t n, float (&g)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = !gamma ? 1.f : !RAGGED || (c + i >= 0 && c + i < n) ? gamma[c + i] : 0.f;
}

struct Shape {
    int64_t rows, c;
    int lanes;    // threads of a row, a power of two
    int per;      // accesses that touch a row, at most
    float eps, inv_c;
};

// Sum over the `lanes` threads of a row, on each of them; lds has a float for
// every wave where they are more than a wave.
__device__ inline float sum_row(float v, int lanes, float *lds)
{
    for (int o = 1; o < lanes && o < 64; o <<= 1) v += __shfl_xor(v, o);
    if (lanes > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
        for (int i = 0; i < lanes / 64; ++i) v += lds[i];
    }
    return v;
}

__device__ inline double sum_row(double v, double *lds)
{
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
    for (int i = 0; i < kThreads / 64; ++i) v += lds[i];
    return v;
}

// The sum that is normed, rounded as it is stored.
template <typename T, int V>
__device__ inline void add(float (&v)[V], const float (&r)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (float)(T)(v[i] + r[i]);
}

template <typename T, int V, bool RAGGED, int HELD>
__global__ __launch_bounds__(kThreads) void rms_fwd(Shape s, const T *x, const T *residual, const float *gamma, T *y,
                                                    T *h, float *rstd)
{
    __shared__ float lds[kThreads / 64];
    const int slots = kThreads / s.lanes, slot = threadIdx.x / s.lanes, lane = threadIdx.x % s.lanes;
    for (int64_t r0 = (int64_t)blockIdx.x * slots; r0 < s.rows; r0 += (int64_t)gridDim.x * slots) {
        const int64_t row = r0 + slot, lo = row * s.c, hi = row < s.rows ? lo + s.c : lo;
        const int64_t base = RAGGED ? lo / V * V : lo;
        float v[HELD][V], ss = 0.f;
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
            const int64_t e = base + (int64_t)(lane + k * s.lanes) * V;
            if (e < hi) {
                load<T, V, RAGGED>(x, e, lo, hi, v[k]);
                if (residual) {
                    float q[V];
                    load<T, V, RAGGED>(residual, e, lo, hi, q);
                    add<T, V>(v[k], q);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
            const int64_t e = base + (int64_t)(lane + k * s.lanes) * V;
            if (e < hi) {
#pragma unroll
                for (int i = 0; i < V; ++i) ss = fmaf(v[k][i], v[k][i], ss);
                if (residual) store<T, V, RAGGED>(h, e, lo, hi, v[k]);
            }
        }
        const float rs = 1.f / sqrtf(fmaf(sum_row(ss, s.lanes, lds), s.inv_c, s.eps));
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
            const int64_t e = base + (int64_t)(lane + k * s.lanes) * V;
            if (e < hi) {
                float g[V];
                weights<V, RAGGED>(gamma, e - lo, s.c, g);
#pragma unroll
                for (int i = 0; i < V; ++i) v[k][i] = v[k][i] * rs * g[i];
                store<T, V, RAGGED>(y, e, lo, hi, v[k]);
            }
        }
        if (lane == 0 && row < s.rows) rstd[row] = rs;
    }
}

// Rows of any length, one a workgroup, walked twice.
template <typename T, int V, bool RAGGED>
__global__ __launch_bounds__(kThreads) void rms_fwd_long(Shape s, const T *x, const T *residual, const float *gamma,
                                                         T *y, T *h, float *rstd)
{
    __shared__ double lds[kThreads / 64];
    for (int64_t row = blockIdx.x; row < s.rows; row += gridDim.x) {
        const int64_t lo = row * s.c, hi = lo + s.c, start = (RAGGED ? lo / V * V : lo) + threadIdx.x * V;
        double ss = 0.0;
        for (int64_t e = start; e < hi; e += kThreads * V) {
            float v[V];
            load<T, V, RAGGED>(x, e, lo, hi, v);
            if (residual) {
                float q[V];
                load<T, V, RAGGED>(residual, e, lo, hi, q);
                add<T, V>(v, q);
                store<T, V, RAGGED>(h, e, lo, hi, v);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fma((double)v[i], (double)v[i], ss);
        }
        const float rs = 1.f / sqrtf(fmaf((float)sum_row(ss, lds), s.inv_c, s.eps));
        // a thread finds its own elements of h
        const T *from = residual ? h : x;
        for (int64_t e = start; e < hi; e += kThreads * V) {
            float v[V], g[V];
            load<T, V, RAGGED>(from, e, lo, hi, v);
            weights<V, RAGGED>(gamma, e - lo, s.c, g);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = v[i] * rs * g[i];
            store<T, V, RAGGED>(y, e, lo, hi, v);
        }
        if (threadIdx.x == 0) rstd[row] = rs;
    }
}

// dx, and dgamma's sums of this workgroup's rows: parts[blockIdx.x][c].
template <typename T, int V, bool RAGGED, int HELD>
__global__ __launch_bounds__(kThreads) void rms_bwd(Shape s, const T *h, const T *dy, const T *dh, const float *gamma,
                                                    const float *rstd, T *dx, float *parts)
{
    __shared__ float lds[kThreads / 64];
    extern __shared__ float sums[];  // [c], where dgamma is asked for
    const int slots = kThreads / s.lanes, slot = threadIdx.x / s.lanes, lane = threadIdx.x % s.lanes;
    const int64_t first = (int64_t)blockIdx.x * slots + slot;  // this slot's first row; the others a multiple of V on
    const int64_t shift = RAGGED ? first * s.c % V : 0;        // elements in front of the row in its first access
    float acc[HELD][V], g[HELD][V];
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
        const int64_t c = (int64_t)(lane + k * s.lanes) * V - shift;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[k][i] = 0.f;
        if (c < s.c)
            weights<V, RAGGED>(gamma, c, s.c, g[k]);
    }
    for (int64_t r0 = (int64_t)blockIdx.x * slots; r0 < s.rows; r0 += (int64_t)gridDim.x * slots) {
        const int64_t row = r0 + slot, lo = row * s.c, hi = row < s.rows ? lo + s.c : lo, base = lo - shift;
        const float rs = row < s.rows ? rstd[row] : 0.f;
        float hv[HELD][V], d[HELD][V], dot = 0.f;
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
            const int64_t e = base + (int64_t)(lane + k * s.lanes) * V;
            if (e < hi) {
                load<T, V, RAGGED>(h, e, lo, hi, hv[k]);
                load<T, V, RAGGED>(dy, e, lo, hi, d[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
            const int64_t e = base + (int64_t)(lane + k * s.lanes) * V;
            if (e < hi)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    hv[k][i] *= rs;
                    acc[k][i] = fmaf(d[k][i], hv[k][i], acc[k][i]);
                    d[k][i] *= g[k][i];
                    dot = fmaf(d[k][i], hv[k][i], dot);
                }
        }
        const float mean = sum_row(dot, s.lanes, lds) * s.inv_c;
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
            const int64_t e = base + (int64_t)(lane + k * s.lanes) * V;
            if (e < hi) {
                float q[V];
                if (dh) load<T, V, RAGGED>(dh, e, lo, hi, q);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float v = rs * fmaf(-hv[k][i], mean, d[k][i]);
                    d[k][i] = dh ? v + q[i] : v;
                }
                store<T, V, RAGGED>(dx, e, lo, hi, d[k]);
            }
        }
    }
    if (!parts) return;
    // the slots' sums, one after the other
    for (int64_t c = threadIdx.x; c < s.c; c += kThreads) sums[c] = 0.f;
    for (int q = 0; q < slots; ++q) {
        __syncthreads();
        if (slot == q)
#pragma unroll
            for (int k = 0; k < HELD; ++k) {
                const int64_t c = (int64_t)(lane + k * s.lanes) * V - shift;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (c + i >= 0 && c + i < s.c) sums[c + i] += acc[k][i];
            }
    }
    __syncthreads();
    for (int64_t c = threadIdx.x; c < s.c; c += kThreads) parts[blockIdx.x * s.c + c] = sums[c];
}

// dx of rows of any length, one a workgroup.
template <typename T, int V, bool RAGGED>
__global__ __launch_bounds__(kThreads) void rms_bwd_long(Shape s, const T *h, const T *dy, const T *dh,
                                                         const float *gamma, const float *rstd, T *dx)
{
    __shared__ double lds[kThreads / 64];
    for (int64_t row = blockIdx.x; row < s.rows; row += gridDim.x) {
        const int64_t lo = row * s.c, hi = lo + s.c, start = (RAGGED ? lo / V * V : lo) + threadIdx.x * V;
        const float rs = rstd[row];
        double dot = 0.0;
        for (int64_t e = start; e < hi; e += kThreads * V) {
            float v[V], d[V], g[V];
            load<T, V, RAGGED>(h, e, lo, hi, v);
            load<T, V, RAGGED>(dy, e, lo, hi, d);
            weights<V, RAGGED>(gamma, e - lo, s.c, g);
#pragma unroll
            for (int i = 0; i < V; ++i) dot = fma((double)(d[i] * g[i]), (double)(v[i] * rs), dot);
        }
        const float mean = (float)sum_row(dot, lds) * s.inv_c;
        for (int64_t e = start; e < hi; e += kThreads * V) {
            float v[V], d[V], g[V], q[V];
            load<T, V, RAGGED>(h, e, lo, hi, v);
            load<T, V, RAGGED>(dy, e, lo, hi, d);
            weights<V, RAGGED>(gamma, e - lo, s.c, g);
            if (dh) load<T, V, RAGGED>(dh, e, lo, hi, q);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float w = rs * fmaf(-(v[i] * rs), mean, d[i] * g[i]);
                d[i] = dh ? w + q[i] : w;
            }
            store<T, V, RAGGED>(dx, e, lo, hi, d);
        }
    }
}

// dgamma's sums of a range of rows (blockIdx.y) where rows are long: a thread a column.
template <typename T>
__global__ __launch_bounds__(kThreads) void rms_dgamma_long(Shape s, const T *h, const T *dy, const float *rstd,
                                                            int64_t rows, float *parts)
{
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x, r0 = blockIdx.y * rows;
    if (c >= s.c) return;
    const int64_t r1 = r0 + rows < s.rows ? r0 + rows : s.rows;
    double a = 0.0;
#pragma unroll 4
    for (int64_t r = r0; r < r1; ++r) a += (double)((float)dy[r * s.c + c] * ((float)h[r * s.c + c] * rstd[r]));
    parts[blockIdx.y * s.c + c] = (float)a;
}

// dgamma: `n` rows of parts added up, 64 columns a workgroup, 16 threads each.
__global__ __launch_bounds__(1024) void rms_join(const float *parts, int64_t n, int64_t c, float *dgamma)
{
    __shared__ double lds[16][65];
    const int x = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int64_t at = (int64_t)blockIdx.x * 64 + x;
    double a = 0.0;
    if (at < c)
#pragma unroll 8
        for (int64_t i = q; i < n; i += 16) a += (double)parts[i * c + at];
    lds[q][x] = a;
    __syncthreads();
    if (q == 0 && at < c) {
        for (int i = 1; i < 16; ++i) a += lds[i][x];
        dgamma[at] = (float)a;
    }
}

// ---- Host ----------------------------------------------------------------------

// The shape for accesses of V elements; held: accesses a thread keeps (0: too
// long a row for `most`).
Shape shape_of(const wtconv_rms_desc_t &d, int v, int most, int &held)
{
    Shape s = {};
    s.rows = d.rows;
    s.c = d.c;
    s.eps = d.eps;
    s.inv_c = (float)(1.0 / (double)d.c);
    const int64_t per = (d.c + v - 1) / v + (d.c % v ? 1 : 0);
    if (per > (int64_t)most * kThreads) {
        held = 0;
        s.lanes = kThreads;
        return s;
    }
    s.per = (int)per;
    // a wave's lanes or fewer with two accesses each, then the workgroup's
    int lanes = 1;
    while (lanes < 64 && lanes < per) lanes *= 2;
    if (per > 2 * lanes) lanes = kThreads;
    s.lanes = lanes;
    held = 1;
    while ((int64_t)held * lanes < per) held *= 2;
    return s;
}

// Workgroups of the backward pass: rows are shared out evenly, at most kChain
// of them for each slot unless that is more workgroups than kGroups.
int64_t backward_groups(int64_t rows, int slots)
{
    const int64_t turns = (rows + slots - 1) / slots;
    int64_t n = turns < kGroups ? turns : kGroups;
    if ((turns + kChain - 1) / kChain > n) n = (turns + kChain - 1) / kChain;
    return n + (8 - n % 8) % 8;  // a slot's rows are a multiple of 8 apart
}

// Ranges of rows of rms_dgamma_long.
int64_t long_ranges(const wtconv_rms_desc_t &d)
{
    const int64_t blocks = (d.c + kThreads - 1) / kThreads;
    int64_t n = 1024 / blocks;
    n = n < 1 ? 1 : n;
    return n < d.rows ? n : d.rows;
}

// Most rows of parts that a backward call of these sizes writes, whatever its
// addresses are.
int64_t parts_of(const wtconv_rms_desc_t &d)
{
    int64_t most = 0;
    const int wide = d.dtype == WTCONV_F32 ? 4 : 8;
    for (int v : {1, wide}) {
        int held;
        const Shape s = shape_of(d, v, kMaxHeldBack, held);
        const int64_t n = held ? backward_groups(d.rows, kThreads / s.lanes) : long_ranges(d);
        most = n > most ? n : most;
    }
    return most;
}

template <typename F>
void with_held(int held, F f)
{
    if (held == 1) f(std::integral_constant<int, 1>{});
    if (held == 2) f(std::integral_constant<int, 2>{});
    if (held == 4) f(std::integral_constant<int, 4>{});
    if (held == 8) f(std::integral_constant<int, 8>{});
}

template <typename T, int V, bool RAGGED>
void forward(const wtconv_rms_desc_t &d, const WtcRmsForward &a, hipStream_t stream)
{
    int held;
    const Shape s = shape_of(d, V, kMaxHeld, held);
    const int64_t slots = kThreads / s.lanes, turns = (s.rows + slots - 1) / slots;
    const dim3 grid((unsigned)(turns < (1 << 20) ? turns : 1 << 20));
    const T *x = (const T *)a.x, *r = (const T *)a.residual;
    if (!held) {
        rms_fwd_long<T, V, RAGGED><<<grid, dim3(kThreads), 0, stream>>>(s, x, r, a.gamma, (T *)a.y, (T *)a.h, a.rstd);
        return;
    }
    with_held(held, [&](auto n) {
        rms_fwd<T, V, RAGGED, n><<<grid, dim3(kThreads), 0, stream>>>(s, x, r, a.gamma, (T *)a.y, (T *)a.h, a.rstd);
    });
}

template <typename T, int V, bool RAGGED>
void backward(const wtconv_rms_desc_t &d, const WtcRmsBackward &a, hipStream_t stream)
{
    int held;
    const Shape s = shape_of(d, V, kMaxHeldBack, held);
    const T *h = (const T *)a.h, *dy = (const T *)a.dy, *dh = (const T *)a.dh;
    int64_t n;
    if (held) {
        n = backward_groups(d.rows, kThreads / s.lanes);
        const size_t lds = a.dgamma ? (size_t)s.c * 4 : 0;
        float *parts = a.dgamma ? a.parts : nullptr;
        with_held(held, [&](auto k) {
            if constexpr (k <= kMaxHeldBack)
                rms_bwd<T, V, RAGGED, k><<<dim3((unsigned)n), dim3(kThreads), lds, stream>>>(s, h, dy, dh, a.gamma,
                                                                                            a.rstd, (T *)a.dx, parts);
        });
    } else {
        const dim3 grid((unsigned)(d.rows < (1 << 20) ? d.rows : 1 << 20));
        // dgamma first: dx may be dh, but neither of those that it reads
        n = long_ranges(d);
        const int64_t rows = (d.rows + n - 1) / n;
        n = (d.rows + rows - 1) / rows;
        if (a.dgamma)
            rms_dgamma_long<T><<<dim3((unsigned)((d.c + kThreads - 1) / kThreads), (unsigned)n), dim3(kThreads), 0,
                                 stream>>>(s, h, dy, a.rstd, rows, a.parts);
        rms_bwd_long<T, V, RAGGED><<<grid, dim3(kThreads), 0, stream>>>(s, h, dy, dh, a.gamma, a.rstd, (T *)a.dx);
    }
    if (a.dgamma)
        rms_join<<<dim3((unsigned)((d.c + 63) / 64)), dim3(1024), 0, stream>>>(a.parts, n, d.c, a.dgamma);
}

// f(V, RAGGED) of these sizes and addresses.
template <typename T, typename F>
void with_access(const wtconv_rms_desc_t &d, bool aligned, F f)
{
    constexpr int V = 16 / sizeof(T);
    if (!aligned)
        f(std::integral_constant<int, 1>{}, std::false_type{});
    else if (d.c % V)
        f(std::integral_constant<int, V>{}, std::true_type{});
    else
        f(std::integral_constant<int, V>{}, std::false_type{});
}

template <typename T>
void forward_of(const wtconv_rms_desc_t &d, const WtcRmsForward &a, hipStream_t stream)
{
    const bool aligned = aligned16(a.x) && aligned16(a.y) && (!a.residual || (aligned16(a.residual) && aligned16(a.h)));
    with_access<T>(d, aligned, [&](auto v, auto ragged) { forward<T, v, ragged>(d, a, stream); });
}

template <typename T>
void backward_of(const wtconv_rms_desc_t &d, const WtcRmsBackward &a, hipStream_t stream)
{
    const bool aligned = aligned16(a.h) && aligned16(a.dy) && aligned16(a.dx) && (!a.dh || aligned16(a.dh));
    with_access<T>(d, aligned, [&](auto v, auto ragged) { backward<T, v, ragged>(d, a, stream); });
}

}  // namespace

size_t wtc_rms_workspace(const wtconv_rms_desc_t &d) { return align256((size_t)(parts_of(d) * d.c) * 4); }

hipError_t wtc_launch_rms_forward(const wtconv_rms_desc_t &d, const WtcRmsForward &a, hipStream_t stream)
{
    if (d.dtype == WTCONV_F32)
        forward_of<float>(d, a, stream);
    else if (d.dtype == WTCONV_F16)
        forward_of<_Float16>(d, a, stream);
    else
        forward_of<__bf16>(d, a, stream);
    return hipGetLastError();
}

hipError_t wtc_launch_rms_backward(const wtconv_rms_desc_t &d, const WtcRmsBackward &a, hipStream_t stream)
{
    if (d.dtype == WTCONV_F32)
        backward_of<float>(d, a, stream);
    else if (d.dtype == WTCONV_F16)
        backward_of<_Float16>(d, a, stream);
    else
        backward_of<__bf16>(d, a, stream);
    return hipGetLastError();
}
