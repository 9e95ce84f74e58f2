// wtconv_rms.hip -- root-mean-square norm of rows with the residual's addition,
// forward and backward.
//
// A row is read once: a row's `lanes` threads keep it in registers between the sum
// of its squares and the outputs, so the bytes are the operator's own (x and the
// residual in, y and the sum out), and both directions are bound by memory: 524288x128
// bf16 forward 92 to 99 us (5.6 TB/s), 200704x96 fp32 backward 52 us (6.0) and 5 for the join
// of dgamma's sums, 2049x5003 fp16 backward 24 us (3.4; rows of an odd length) and 5.  An
// elementwise pass over 4 GiB reaches 6.2.
// Rows longer than the registers hold (kMaxHeld accesses of 256 threads) are
// walked twice.
//
// A thread takes V elements an access, 16 bytes where the addresses allow it.
// Rows whose length V does not divide start at any place between two such
// accesses (RAGGED): the accesses that lie in the row whole are taken so, and the
// fewer than V elements in front of them and behind one a thread.  Row r's start
// repeats with period V, and a backward slot takes rows a multiple of V apart, so
// that its threads keep their columns, and the sums of dgamma stay in registers over
// all of a slot's rows.  (With guards at every element of the first and the last
// access instead, 31 instructions an element: 2049x5003 fp16 backward 59 us.)
//
// Numerics.  Values are fp32 from the load on (h first rounded to its type, since
// that is what the backward pass finds).  A thread sums at most 65 squares, then a
// tree; longer rows sum in fp64.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cstdint>

#include "wtconv_check.h"
#include "wtconv_rms.h"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxHeld = 8;     // accesses of a row that a thread keeps, forward
// Backward: three values of each element.  us with rows in registers, and walked twice with
// dgamma's sums in a kernel of their own: fp32 8192x2048 (two accesses) 47, 75; 4096x4096
// (four) 57, 81; bf16 4096x4096 (two) 33, 46; 2048x8192 (four) 35, 43.
constexpr int kMaxHeldBack = 4;
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

template <typename T, int V>
__device__ inline typename Access<T, V>::type fetch(const T *p)
{
    return *(const typename Access<T, V>::type *)p;
}

template <typename T, int V>
__device__ inline void values(const typename Access<T, V>::type &r, float (&v)[V])
{
    if constexpr (V == 1)
        v[0] = (float)r;
    else
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = (float)r[i];
}

template <typename T, int V>
__device__ inline void store(T *p, const float (&v)[V])
{
    typename Access<T, V>::type r;
    if constexpr (V == 1)
        r = (T)v[0];
    else
#pragma unroll
        for (int i = 0; i < V; ++i) r[i] = (T)v[i];
    *(typename Access<T, V>::type *)p = r;
}

struct Shape {
    int64_t rows, c;
    int lanes;    // threads of a row, a power of two
    float eps, inv_c;
};

// A row in accesses: `head` elements, `whole` accesses of V, the rest.
struct Parts {
    int head, whole;
    int64_t edge;  // the column of this thread's single element, or -1
};

template <int V, bool RAGGED>
__device__ inline Parts parts_of_row(const Shape &s, int64_t row, int lane)
{
    Parts p = {0, (int)(s.c / V), -1};
    if (RAGGED) {
        const int off = (int)(row * s.c % V), head = off ? V - off : 0, rest = (int)((s.c - head) % V);
        p.head = head;
        p.whole = (int)((s.c - head) / V);
        if (lane < head)
            p.edge = lane;
        else if (lane - head < rest)
            p.edge = s.c - rest + (lane - head);
    }
    return p;
}

// gamma of columns c .. c + V.
template <int V>
__device__ inline void weights(const float *gamma, int64_t c, float (&g)[V])
{
    if (gamma)
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = gamma[c + i];
    else
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = 1.f;
}

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
template <typename T>
__device__ inline float add(float x, float r)
{
    return (float)(T)(x + r);
}

template <typename T, int V, bool RAGGED, int HELD>
__global__ __launch_bounds__(kThreads) void rms_fwd(Shape s, const T *x, const T *residual, const float *gamma, T *y,
                                                    T *h, float *rstd)
{
    __shared__ float lds[kThreads / 64];
    const int slots = kThreads / s.lanes, slot = threadIdx.x / s.lanes, lane = threadIdx.x % s.lanes;
    for (int64_t r0 = (int64_t)blockIdx.x * slots; r0 < s.rows; r0 += (int64_t)gridDim.x * slots) {
        const int64_t row = r0 + slot, lo = row * s.c;
        Parts p = parts_of_row<V, RAGGED>(s, row, lane);
        if (row >= s.rows) p = {0, 0, -1};
        float v[HELD][V], single = 0.f, ss;
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
            const int j = lane + k * s.lanes;
            if (j < p.whole) {
                const int64_t e = lo + p.head + (int64_t)j * V;
                values<T, V>(fetch<T, V>(x + e), v[k]);
                if (residual) {
                    float q[V];
                    values<T, V>(fetch<T, V>(residual + e), q);
#pragma unroll
                    for (int i = 0; i < V; ++i) v[k][i] = add<T>(v[k][i], q[i]);
                }
            }
        }
        if (RAGGED && p.edge >= 0) {
            single = (float)x[lo + p.edge];
            if (residual) single = add<T>(single, (float)residual[lo + p.edge]);
        }
        ss = single * single;
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
            const int j = lane + k * s.lanes;
            if (j < p.whole) {
#pragma unroll
                for (int i = 0; i < V; ++i) ss = fmaf(v[k][i], v[k][i], ss);
                if (residual) store<T, V>(h + lo + p.head + (int64_t)j * V, v[k]);
            }
        }
        if (RAGGED && residual && p.edge >= 0) h[lo + p.edge] = (T)single;
        const float rs = 1.f / sqrtf(fmaf(sum_row(ss, s.lanes, lds), s.inv_c, s.eps));
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
            const int j = lane + k * s.lanes;
            if (j < p.whole) {
                const int64_t c = p.head + (int64_t)j * V;
                float g[V];
                weights<V>(gamma, c, g);
#pragma unroll
                for (int i = 0; i < V; ++i) v[k][i] = v[k][i] * rs * g[i];
                store<T, V>(y + lo + c, v[k]);
            }
        }
        if (RAGGED && p.edge >= 0) y[lo + p.edge] = (T)(gamma ? single * rs * gamma[p.edge] : single * rs);
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
        const int64_t lo = row * s.c;
        const Parts p = parts_of_row<V, RAGGED>(s, row, threadIdx.x);
        double ss = 0.0;
        for (int j = threadIdx.x; j < p.whole; j += kThreads) {
            const int64_t e = lo + p.head + (int64_t)j * V;
            float v[V];
            values<T, V>(fetch<T, V>(x + e), v);
            if (residual) {
                float q[V];
                values<T, V>(fetch<T, V>(residual + e), q);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = add<T>(v[i], q[i]);
                store<T, V>(h + e, v);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fma((double)v[i], (double)v[i], ss);
        }
        float single = 0.f;
        if (RAGGED && p.edge >= 0) {
            single = (float)x[lo + p.edge];
            if (residual) {
                single = add<T>(single, (float)residual[lo + p.edge]);
                h[lo + p.edge] = (T)single;
            }
            ss = fma((double)single, (double)single, ss);
        }
        const float rs = 1.f / sqrtf(fmaf((float)sum_row(ss, lds), s.inv_c, s.eps));
        // a thread finds its own elements of h
        const T *from = residual ? h : x;
        for (int j = threadIdx.x; j < p.whole; j += kThreads) {
            const int64_t c = p.head + (int64_t)j * V;
            float v[V], g[V];
            values<T, V>(fetch<T, V>(from + lo + c), v);
            weights<V>(gamma, c, g);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = v[i] * rs * g[i];
            store<T, V>(y + lo + c, v);
        }
        if (RAGGED && p.edge >= 0) y[lo + p.edge] = (T)(gamma ? single * rs * gamma[p.edge] : single * rs);
        if (threadIdx.x == 0) rstd[row] = rs;
    }
}

// dx of an element.
__device__ inline float back(float h, float dy, float g, float rs, float mean)
{
    return rs * fmaf(-(h * rs), mean, dy * g);
}

// dx, and dgamma's sums of this workgroup's rows: parts[blockIdx.x][c].  A row's loads
// are sent off before the row in front of it is summed.
template <typename T, int V, bool RAGGED, int HELD>
__global__ __launch_bounds__(kThreads) void rms_bwd(Shape s, const T *h, const T *dy, const T *dh, const float *gamma,
                                                    const float *rstd, T *dx, float *parts)
{
    typedef typename Access<T, V>::type A;
    __shared__ float lds[kThreads / 64];
    extern __shared__ float sums[];  // [c], where dgamma is asked for
    const int slots = kThreads / s.lanes, slot = threadIdx.x / s.lanes, lane = threadIdx.x % s.lanes;
    // this slot's first row; the others are a multiple of V further, with the same parts
    const int64_t first = (int64_t)blockIdx.x * slots + slot;
    const Parts p = parts_of_row<V, RAGGED>(s, first, lane);
    struct Row {
        A h[HELD], dy[HELD], dh[HELD];
        T sh, sdy, sdh;
        float rs;
    };
    auto fetch_row = [&](int64_t row, Row &r) {
        if (row >= s.rows) return;
        const int64_t lo = row * s.c + p.head;
        r.rs = rstd[row];
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
            const int j = lane + k * s.lanes;
            if (j < p.whole) {
                const int64_t e = lo + (int64_t)j * V;
                r.h[k] = fetch<T, V>(h + e);
                r.dy[k] = fetch<T, V>(dy + e);
                if (dh) r.dh[k] = fetch<T, V>(dh + e);
            }
        }
        if (RAGGED && p.edge >= 0) {
            const int64_t e = row * s.c + p.edge;
            r.sh = h[e];
            r.sdy = dy[e];
            if (dh) r.sdh = dh[e];
        }
    };
    Row now, next;
    fetch_row(first, now);
    float acc[HELD][V] = {}, single = 0.f, g[HELD][V], gs = 1.f;
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
        const int j = lane + k * s.lanes;
        if (j < p.whole) weights<V>(gamma, p.head + (int64_t)j * V, g[k]);
    }
    if (RAGGED && gamma && p.edge >= 0) gs = gamma[p.edge];
    const int64_t step = (int64_t)gridDim.x * slots;
    for (int64_t r0 = (int64_t)blockIdx.x * slots; r0 < s.rows; r0 += step) {
        const int64_t row = r0 + slot;
        const bool in = row < s.rows;
        fetch_row(row + step, next);
        float dot = 0.f;
        if (in) {
#pragma unroll
            for (int k = 0; k < HELD; ++k)
                if (lane + k * s.lanes < p.whole) {
                    float v[V], d[V];
                    values<T, V>(now.h[k], v);
                    values<T, V>(now.dy[k], d);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        v[i] *= now.rs;
                        acc[k][i] = fmaf(d[i], v[i], acc[k][i]);
                        dot = fmaf(d[i] * g[k][i], v[i], dot);
                    }
                }
            if (RAGGED && p.edge >= 0) {
                const float v = (float)now.sh * now.rs;
                single = fmaf((float)now.sdy, v, single);
                dot = fmaf((float)now.sdy * gs, v, dot);
            }
        }
        const float mean = sum_row(dot, s.lanes, lds) * s.inv_c;
        if (in) {
            const int64_t lo = row * s.c + p.head;
#pragma unroll
            for (int k = 0; k < HELD; ++k) {
                const int j = lane + k * s.lanes;
                if (j < p.whole) {
                    float v[V], d[V], q[V];
                    values<T, V>(now.h[k], v);
                    values<T, V>(now.dy[k], d);
                    if (dh) values<T, V>(now.dh[k], q);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float w = back(v[i], d[i], g[k][i], now.rs, mean);
                        d[i] = dh ? w + q[i] : w;
                    }
                    store<T, V>(dx + lo + (int64_t)j * V, d);
                }
            }
            if (RAGGED && p.edge >= 0) {
                const float w = back((float)now.sh, (float)now.sdy, gs, now.rs, mean);
                dx[row * s.c + p.edge] = (T)(dh ? w + (float)now.sdh : w);
            }
        }
        now = next;
    }
    if (!parts) return;
    // the slots' sums, one after the other
    for (int64_t c = threadIdx.x; c < s.c; c += kThreads) sums[c] = 0.f;
    for (int q = 0; q < slots; ++q) {
        __syncthreads();
        if (slot == q) {
#pragma unroll
            for (int k = 0; k < HELD; ++k) {
                const int j = lane + k * s.lanes;
                if (j < p.whole)
#pragma unroll
                    for (int i = 0; i < V; ++i) sums[p.head + j * V + i] += acc[k][i];
            }
            if (RAGGED && p.edge >= 0) sums[p.edge] += single;
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
        const int64_t lo = row * s.c;
        const Parts p = parts_of_row<V, RAGGED>(s, row, threadIdx.x);
        const float rs = rstd[row];
        double dot = 0.0;
        for (int j = threadIdx.x; j < p.whole; j += kThreads) {
            const int64_t c = p.head + (int64_t)j * V;
            float v[V], d[V], g[V];
            values<T, V>(fetch<T, V>(h + lo + c), v);
            values<T, V>(fetch<T, V>(dy + lo + c), d);
            weights<V>(gamma, c, g);
#pragma unroll
            for (int i = 0; i < V; ++i) dot = fma((double)(d[i] * g[i]), (double)(v[i] * rs), dot);
        }
        const float gs = RAGGED && gamma && p.edge >= 0 ? gamma[p.edge] : 1.f;
        if (RAGGED && p.edge >= 0)
            dot = fma((double)((float)dy[lo + p.edge] * gs), (double)((float)h[lo + p.edge] * rs), dot);
        const float mean = (float)sum_row(dot, lds) * s.inv_c;
        for (int j = threadIdx.x; j < p.whole; j += kThreads) {
            const int64_t c = p.head + (int64_t)j * V;
            float v[V], d[V], q[V], g[V];
            values<T, V>(fetch<T, V>(h + lo + c), v);
            values<T, V>(fetch<T, V>(dy + lo + c), d);
            weights<V>(gamma, c, g);
            if (dh) values<T, V>(fetch<T, V>(dh + lo + c), q);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float w = back(v[i], d[i], g[i], rs, mean);
                d[i] = dh ? w + q[i] : w;
            }
            store<T, V>(dx + lo + c, d);
        }
        if (RAGGED && p.edge >= 0) {
            const int64_t e = lo + p.edge;
            const float w = back((float)h[e], (float)dy[e], gs, rs, mean);
            dx[e] = (T)(dh ? w + (float)dh[e] : w);
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

// dgamma: `n` rows of parts added up, 32 columns a workgroup, 32 threads each.
__global__ __launch_bounds__(1024) void rms_join(const float *parts, int64_t n, int64_t c, float *dgamma)
{
    __shared__ double lds[32][33];
    const int x = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t at = (int64_t)blockIdx.x * 32 + x;
    double a = 0.0;
    if (at < c)
#pragma unroll 8
        for (int64_t i = q; i < n; i += 32) a += (double)parts[i * c + at];
    lds[q][x] = a;
    __syncthreads();
    if (q == 0 && at < c) {
        for (int i = 1; i < 32; ++i) a += lds[i][x];
        dgamma[at] = (float)a;
    }
}

// ---- Host ----------------------------------------------------------------------

// Whether rows of c elements, V an access, have single elements next to whole
// accesses (a thread each, so that short rows go element by element), and the
// elements of an access that they take then.
int access_of(int64_t c, int wide) { return c % wide == 0 || c >= 8 * wide ? wide : 1; }

// The shape for accesses of V elements; held: accesses a thread keeps (0: too
// long a row for `most`).
Shape shape_of(const wtconv_rms_desc_t &d, int v, int most, int &held)
{
    Shape s = {};
    s.rows = d.rows;
    s.c = d.c;
    s.eps = d.eps;
    s.inv_c = (float)(1.0 / (double)d.c);
    const int64_t per = d.c < v ? 1 : d.c / v;
    if (per > (int64_t)most * kThreads) {
        held = 0;
        s.lanes = kThreads;
        return s;
    }
    // a wave's lanes or fewer with two accesses each, then the workgroup's; lanes for
    // the single elements
    int lanes = d.c % v ? 16 : 1;
    while (lanes < 64 && lanes < per) lanes *= 2;
    if (per > 2 * lanes) lanes = kThreads;
    s.lanes = lanes;
    held = (int)((per + lanes - 1) / lanes);
    if (held > 4) held = 8;
    return s;
}

// Workgroups of the backward pass: rows are shared out evenly, at most kChain
// of them for each slot unless that is more workgroups than kGroups, and where there
// are few rows at least 4 (each workgroup writes a row of dgamma's sums).
int64_t backward_groups(int64_t rows, int slots)
{
    const int64_t turns = (rows + slots - 1) / slots;
    int64_t n = turns < 256 ? turns : turns / 4 < 256 ? 256 : turns / 4 < kGroups ? turns / 4 : kGroups;
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
    for (int v : {1, access_of(d.c, wide)}) {
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
    if (held == 3) f(std::integral_constant<int, 3>{});
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
        rms_join<<<dim3((unsigned)((d.c + 31) / 32)), dim3(1024), 0, stream>>>(a.parts, n, d.c, a.dgamma);
}

// f(V, RAGGED) of these sizes and addresses.
template <typename T, typename F>
void with_access(const wtconv_rms_desc_t &d, bool aligned, F f)
{
    constexpr int V = 16 / sizeof(T);
    if (!aligned || access_of(d.c, V) == 1)
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
