// wtconv_gated_body.h -- the gated product's kernels of one element type; the
// files wtconv_gated_f32.hip, _f16.hip and _bf16.hip instantiate them.
//
// Three products on the matrix instructions (32 x 32 x 16, 16-bit factors, fp32
// sums):
//   dual   g = x Wg^T and u = x Wu^T side by side, a wave holding both of the same
//          place, so that act(g) u, or dg and du from dh, are made of registers;
//   dx     [dg du] [Wg; Wu], over 2 F;
//   dw     [dg du]^T x, over the rows: both factors lie across the sum's index and
//          come out of LDS through the transposing reads.
// fp32 factors are three bf16 numbers each, which hold all 24 bits, and a product
// six: those whose size is at least 2^-16 of the first (what is left out is below
// 2^-23 of the whole).  The fp32 matrix instructions run at 1/16 of the 16-bit rate.
#ifndef WTCONV_GATED_BODY_H
#define WTCONV_GATED_BODY_H

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "wtconv_act.h"
#include "wtconv_check.h"
#include "wtconv_gated.h"

namespace wtc_gated {

using wtc_act::normal_cdf;
using wtc_act::sigmoid;

typedef float float4v __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));
typedef short short4v __attribute__((ext_vector_type(4)));

// The factors' type of activations T, and how many of them hold one value.
template <typename T>
struct Factor {
    typedef T type;
    static constexpr int kPlanes = 1;
};
template <>
struct Factor<float> {
    typedef __bf16 type;
    static constexpr int kPlanes = 3;
};

template <typename E, int N>
using Vec = E __attribute__((ext_vector_type(N)));

__device__ inline float16v mfma(const Vec<_Float16, 8> &l, const Vec<_Float16, 8> &r, float16v c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(l, r, c, 0, 0, 0);
}
__device__ inline float16v mfma(const Vec<__bf16, 8> &l, const Vec<__bf16, 8> &r, float16v c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(l, r, c, 0, 0, 0);
}
__device__ inline float4v mfma16(const Vec<_Float16, 8> &l, const Vec<_Float16, 8> &r, float4v c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(l, r, c, 0, 0, 0);
}
__device__ inline float4v mfma16(const Vec<__bf16, 8> &l, const Vec<__bf16, 8> &r, float4v c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(l, r, c, 0, 0, 0);
}
// Four instructions, each with an element of either side: the order of the sum's
// index is the same on both.
__device__ inline float4v mfma16(const Vec<float, 4> &l, const Vec<float, 4> &r, float4v c)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(l[i], r[i], c, 0, 0, 0);
    return c;
}

// The smaller products first.
template <typename F, int P>
__device__ inline float16v mfma_planes(const F (&l)[P], const F (&r)[P], float16v c)
{
    if constexpr (P == 1) return mfma(l[0], r[0], c);
    else {
        c = mfma(l[2], r[0], c);
        c = mfma(l[0], r[2], c);
        c = mfma(l[1], r[1], c);
        c = mfma(l[1], r[0], c);
        c = mfma(l[0], r[1], c);
        return mfma(l[0], r[0], c);
    }
}

// v as the sum of P numbers.  fp32: its bits from the top, eight at a time; an
// infinity or NaN whole in the first (what is left of it would be NaN).
template <typename T, int P>
__device__ inline void split(float v, typename Factor<T>::type (&o)[P])
{
    if constexpr (P == 1) {
        o[0] = (T)v;
    } else {
        const uint32_t u = __builtin_bit_cast(uint32_t, v);
        const bool finite = (u & 0x7f800000u) != 0x7f800000u;
        // a NaN whose bits all lie below stays one
        const uint32_t top = (u & 0xffff0000u) | (!finite && (u & 0x7fffffu) ? 0x400000u : 0u);
        const float r1 = finite ? v - __builtin_bit_cast(float, top) : 0.f;
        const uint32_t mid = __builtin_bit_cast(uint32_t, r1) & 0xffff0000u;
        const float r2 = r1 - __builtin_bit_cast(float, mid);
        o[0] = __builtin_bit_cast(__bf16, (uint16_t)(top >> 16));
        o[1] = __builtin_bit_cast(__bf16, (uint16_t)(mid >> 16));
        o[2] = __builtin_bit_cast(__bf16, (uint16_t)(__builtin_bit_cast(uint32_t, r2) >> 16));
    }
}

__device__ inline float act(int kind, float z)
{
    if (kind == WTCONV_ACT_SILU) return z * sigmoid(z);
    if (kind == WTCONV_ACT_GELU) {
        float e;
        return z * normal_cdf(z, e);
    }
    if (kind == WTCONV_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN stays
    return z;
}

// act(z) and its slope.
__device__ inline float act_slope(int kind, float z, float &slope)
{
    if (kind == WTCONV_ACT_SILU) {
        const float s = sigmoid(z);
        slope = s * fmaf(z, 1.f - s, 1.f);
        return z * s;
    }
    if (kind == WTCONV_ACT_GELU) {
        float e;
        const float p = normal_cdf(z, e);
        slope = fmaf(z * 0.39894228f, e, p);
        return z * p;
    }
    if (kind == WTCONV_ACT_RELU) {
        slope = z > 0.f ? 1.f : 0.f;
        return z < 0.f ? 0.f : z;
    }
    slope = 1.f;
    return z;
}

// What a lane loads in place of a row's missing end.
__device__ const uint32_t kZeros[4] = {0, 0, 0, 0};

typedef const __attribute__((address_space(1))) void *GlobalPtr;
typedef __attribute__((address_space(3))) void *LdsPtr;

// 16 bytes a lane from memory into LDS, lanes side by side from `to` on.
__device__ inline void load_lds(const void *from, char *to)
{
    __builtin_amdgcn_global_load_lds((GlobalPtr)from, (LdsPtr)to, 16, 0, 0);
}

// ---- Laying out ----------------------------------------------------------------

// Rows of k elements as `planes` matrices of rows of kp, zeros behind.
template <typename T>
__global__ __launch_bounds__(256) void gated_pack(const T *__restrict__ src, int64_t rows, int k, int kp,
                                                  typename Factor<T>::type *__restrict__ dst, int64_t plane)
{
    typedef typename Factor<T>::type E;
    constexpr int P = Factor<T>::kPlanes;
    const int per = kp / 8;
    const int64_t all = rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per;
        const int at = (int)(i - row * per) * 8;
        Vec<E, 8> o[P];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            E e[P];
            if constexpr (P == 1)
                e[0] = at + j < k ? src[row * k + at + j] : (T)0.f;
            else
                split<T, P>(at + j < k ? src[row * k + at + j] : 0.f, e);
#pragma unroll
            for (int p = 0; p < P; ++p) o[p][j] = e[p];
        }
#pragma unroll
        for (int p = 0; p < P; ++p) *(Vec<E, 8> *)(dst + p * plane + row * kp + at) = o[p];
    }
}

// The weights' columns as rows: dst[c] = gate's column c, then up's, each of fp
// elements, zeros behind f.  One workgroup a 64 x 64 tile; blockIdx.z: gate, up.
template <typename T>
__global__ __launch_bounds__(256) void gated_turn(const T *__restrict__ w_gate, const T *__restrict__ w_up, int f, int c,
                                                  int fp, typename Factor<T>::type *__restrict__ dst, int64_t plane)
{
    typedef typename Factor<T>::type E;
    constexpr int P = Factor<T>::kPlanes;
    __shared__ T tile[64][66];
    const T *w = blockIdx.z ? w_up : w_gate;
    const int f0 = blockIdx.y * 64, c0 = blockIdx.x * 64, x = threadIdx.x & 63, y = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < 64; i += 4)
        tile[y + i][x] = f0 + y + i < f && c0 + x < c ? w[(int64_t)(f0 + y + i) * c + c0 + x] : (T)0.f;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 64; i += 4)
        if (c0 + y + i < c && f0 + x < fp) {
            E e[P];
            const T v = tile[x][y + i];
            if constexpr (P == 1)
                e[0] = v;
            else
                split<T, P>(v, e);
#pragma unroll
            for (int p = 0; p < P; ++p)
                dst[p * plane + (int64_t)(c0 + y + i) * 2 * fp + blockIdx.z * fp + f0 + x] = e[p];
        }
}

// ---- Products with both factors' rows along the sum's index ---------------------

enum Mode {
    kForward,   // h = act(g + bg) (u + bu)
    kBackward,  // dg, du (and the biases' sums)
    kProduct    // the product itself: dx
};

template <typename E>
struct Rows {
    const E *p;
    int64_t plane, pitch;  // elements
};

template <typename T>
struct Nt {
    typedef typename Factor<T>::type E;
    Rows<E> a, b0, b1;  // rows of A; of B (dual: of the gate's and of the up projection's weights)
    int64_t m;
    int n, k;           // columns (dual: f), length of the sum
    int64_t tm;
    int tn, slices;
    int64_t cut;        // stages of a slice
    int act;
    const float *bias0, *bias1;
    const T *dh;
    T *out;             // [m][n]
    float *part;        // kProduct cut into slices: [slice][m][n]
    E *grads;           // kBackward: [plane][m][2 fp]
    int64_t grads_plane;
    int fp;
    float *bias_part;   // kBackward, or null: [tm * waves along m][2 fp]
    bool wide;          // rows of out and dh in accesses of four elements
};

// Tile of workgroup g: workgroups go to the 8 dies in turn, each die gets
// neighbouring tiles, in bands of 8 tile rows, so that tiles in flight share
// operands in its L2.
__device__ inline void place(int64_t g, int64_t tm, int tn, int64_t &ti, int &tj)
{
    const int64_t all = tm * tn, per = all / 8;
    const int rest = (int)(all % 8), die = (int)(g % 8);
    g = die * per + (die < rest ? die : rest) + g / 8;
    const int64_t band = g / (8 * (int64_t)tn);
    const int h = tm - 8 * band < 8 ? (int)(tm - 8 * band) : 8;
    const int in = (int)(g - band * 8 * tn);
    ti = band * 8 + in % h;
    tj = in / h;
}

// Four values from column c of a row, elements of no column left out.
template <typename T>
__device__ inline void store4(T *p, int c, int n, bool wide, const float (&v)[4])
{
    if (wide && c + 4 <= n) {
        Vec<T, 4> r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = (T)v[i];
        *(Vec<T, 4> *)(p + c) = r;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < n) p[c + i] = (T)v[i];
    }
}

template <typename T>
__device__ inline void load4(const T *p, int c, int n, bool wide, float (&v)[4])
{
    if (wide && c + 4 <= n) {
        const Vec<T, 4> r = *(const Vec<T, 4> *)(p + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)r[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = c + i < n ? (float)p[c + i] : 0.f;
    }
}

// Sums of s[0..15] over the 32 lanes of a half wave, by halves: lane l ends up
// with that of index (l & 31) / 2.
__device__ inline float sum_lanes(float (&s)[16])
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 16, n = 8; o > 1; o >>= 1, n >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) {
                const float keep = up ? s[i + n] : s[i], send = up ? s[i] : s[i + n];
                s[i] = keep + __shfl_xor(send, o);
            }
    }
    return s[0] + __shfl_xor(s[0], 1);
}

// A tile of BM rows of A and BN rows of B; WM x WN waves.  A stage is 128 (P = 1)
// or 64 (P = 3) bytes of each row, from memory into LDS without registers between.
// The 16-byte chunks of a row are permuted so that the rows that a read phase
// covers fall into different banks.  Two buffers: a stage's reads into registers
// come first, then the next stage's loads are sent off, then its matrix
// instructions run.
template <typename T, int BM, int BN, int WM, int WN, int MODE>
__global__ __launch_bounds__(WM *WN * 64) void gated_nt(Nt<T> a)
{
    typedef typename Factor<T>::type E;
    typedef Vec<E, 8> Frag;
    constexpr int P = Factor<T>::kPlanes;
    constexpr int kRow = P == 1 ? 128 : 64, BK = kRow / 2;          // bytes and elements of a row in a stage
    constexpr int kRows = BM + BN, kStage = kRows * P * kRow;
    constexpr int kPerLoad = 1024 / kRow, kLoads = kRows * P / kPerLoad / (WM * WN);
    static_assert(kLoads * kPerLoad * WM * WN == kRows * P, "rows are shared out evenly");
    constexpr int RM = BM / WM / 32, RN = BN / WN / 32, KK = BK / 16;  // blocks of a wave; steps of a stage
    static_assert(MODE == kProduct || RN == 2, "a wave has a block of g and the same of u");
    __shared__ __attribute__((aligned(128))) char lds[2 * kStage];

    const int slice = MODE == kProduct ? blockIdx.y : 0;
    int64_t ti;
    int tj;
    place(blockIdx.x, a.tm, a.tn, ti, tj);
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63, lr = lane & 31, lc = lane >> 5;
    const int64_t m0 = ti * BM;
    const int n0 = tj * (MODE == kProduct ? BN : BN / 2);
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);

    auto swizzle = [](int row) { return P == 1 ? (row >> 1) & 7 : (row >> 2) & 3; };
    const E *src[kLoads];
    int at[kLoads];  // this lane's place along the sum in a stage
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int q = (wave * kLoads + i) * kPerLoad + lane / (kRow / 16), p = q / kRows, row = q % kRows;
        at[i] = ((lane % (kRow / 16)) ^ swizzle(row)) * 8;
        if (row < BM) {
            const int64_t m = m0 + row < a.m ? m0 + row : a.m - 1;
            src[i] = a.a.p + p * a.a.plane + m * a.a.pitch;
        } else {
            const int r = row - BM;
            const bool up = MODE != kProduct && (r / 32) % 2;
            int n = MODE == kProduct ? n0 + r : n0 + r / 64 * 32 + r % 32;
            n = n < a.n ? n : a.n - 1;
            const Rows<E> &b = up ? a.b1 : a.b0;
            src[i] = b.p + p * b.plane + n * b.pitch;
        }
    }
    const int64_t all = (a.k + BK - 1) / BK, s0 = slice * a.cut;
    const int stages = (int)(MODE == kProduct ? (all - s0 < a.cut ? all - s0 : a.cut) : all);
    auto load = [&](int s) {
        const int64_t k = (s0 + s) * BK;
        char *to = lds + (s & 1) * kStage + wave * kLoads * 1024;
        if (k + BK <= a.k) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) load_lds(src[i] + k + at[i], to + i * 1024);
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                load_lds(k + at[i] < a.k ? (const void *)(src[i] + k + at[i]) : (const void *)kZeros, to + i * 1024);
        }
    };
    auto frag = [&](int s, int p, int row, int chunk) {
        return *(const Frag *)(lds + (s & 1) * kStage + (p * kRows + row) * kRow + ((chunk ^ swizzle(row)) * 16));
    };

    float16v acc[RN][RM] = {};  // rows: B's, columns: A's
    load(0);
    for (int s = 0; s < stages; ++s) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        Frag fa[KK][RM][P], fb[KK][RN][P];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int p = 0; p < P; ++p) {
#pragma unroll
                for (int i = 0; i < RM; ++i) fa[kk][i][p] = frag(s, p, wm + i * 32 + lr, kk * 2 + lc);
#pragma unroll
                for (int j = 0; j < RN; ++j) fb[kk][j][p] = frag(s, p, BM + wn + j * 32 + lr, kk * 2 + lc);
            }
        __builtin_amdgcn_sched_barrier(0);
        if (s + 1 < stages) load(s + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int j = 0; j < RN; ++j)
#pragma unroll
                for (int i = 0; i < RM; ++i) acc[j][i] = mfma_planes<Frag, P>(fb[kk][j], fa[kk][i], acc[j][i]);
    }

    // A lane has column m = lr of A's rows and, of B's rows, 8 (q / 4) + 4 lc + q % 4.
    if constexpr (MODE == kProduct) {
#pragma unroll
        for (int i = 0; i < RM; ++i) {
            const int64_t m = m0 + wm + i * 32 + lr;
            if (m >= a.m) continue;
#pragma unroll
            for (int j = 0; j < RN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = n0 + wn + j * 32 + 8 * q + 4 * lc;
                    const float v[4] = {acc[j][i][4 * q], acc[j][i][4 * q + 1], acc[j][i][4 * q + 2],
                                        acc[j][i][4 * q + 3]};
                    if (a.slices > 1)
                        store4(a.part + (slice * a.m + m) * a.n, n, a.n, a.n % 4 == 0, v);
                    else
                        store4(a.out + m * a.n, n, a.n, a.wide, v);
                }
        }
        return;
    } else {
        const int f0 = n0 + wn / 2 + 4 * lc;
        float bg[16], bu[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const int f = f0 + 8 * (q >> 2) + (q & 3);
            bg[q] = a.bias0 && f < a.n ? a.bias0[f] : 0.f;
            bu[q] = a.bias1 && f < a.n ? a.bias1[f] : 0.f;
        }
        float sg[16] = {}, su[16] = {};
#pragma unroll
        for (int i = 0; i < RM; ++i) {
            const int64_t m = m0 + wm + i * 32 + lr;
            if (m >= a.m) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int f = f0 + 8 * q;
                float g[4], u[4], d[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    g[e] = acc[0][i][4 * q + e] + bg[4 * q + e];
                    u[e] = acc[1][i][4 * q + e] + bu[4 * q + e];
                }
                if constexpr (MODE == kForward) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) g[e] = act(a.act, g[e]) * u[e];
                    store4(a.out + m * a.n, f, a.n, a.wide, g);
                } else {
                    load4(a.dh + m * a.n, f, a.n, a.wide, d);
                    // dg and du of columns behind f are zero: dh is
                    Vec<E, 4> og[P], ou[P];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float slope;
                        const float y = act_slope(a.act, g[e], slope);
                        const bool in = f + e < a.n;
                        const float dg = in ? d[e] * u[e] * slope : 0.f, du = in ? d[e] * y : 0.f;
                        sg[4 * q + e] += dg;
                        su[4 * q + e] += du;
                        E eg[P], eu[P];
                        split<T, P>(dg, eg);
                        split<T, P>(du, eu);
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            og[p][e] = eg[p];
                            ou[p][e] = eu[p];
                        }
                    }
                    if (f < a.fp)
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            E *row = a.grads + p * a.grads_plane + m * 2 * a.fp + f;
                            *(Vec<E, 4> *)row = og[p];
                            *(Vec<E, 4> *)(row + a.fp) = ou[p];
                        }
                }
            }
        }
        if (MODE == kBackward && a.bias_part) {
            const float g = sum_lanes(sg), u = sum_lanes(su);
            const int q = lr >> 1, f = f0 + 8 * (q >> 2) + (q & 3);
            if (!(lane & 1) && f < a.n) {
                float *row = a.bias_part + (ti * WM + wave / WN) * 2 * a.fp;
                row[f] = g;
                row[a.fp + f] = u;
            }
        }
    }
}

// ---- The weights' gradients -------------------------------------------------------

template <typename T>
struct Tn {
    typedef typename Factor<T>::type E;
    const E *a, *b;  // [plane][m][2 fp], [plane][m][pitch]
    int64_t a_plane, b_plane, b_pitch;
    int64_t m;
    int f, fp, c;
    int64_t tm;
    int tn, slices;
    int64_t cut;     // stages of a slice
    T *gate, *up;    // [f][c]
    float *part;     // [slice][2 fp][c]
    bool wide;
};

// D = A^T B, a tile of BM columns of A (gradients) and BN of B (x), over a slice
// of the rows, BK of them a stage.  LDS holds rows as they come; the transposing
// read gives a lane four rows' values of its column: 16 lanes take 4 rows of 32
// bytes, and these 32-byte pieces are permuted by row so that a read's rows lie in
// different banks.
template <typename T, int BM, int BN, int WM, int WN, int BK>
__global__ __launch_bounds__(WM *WN * 64) void gated_tn(Tn<T> a)
{
    typedef typename Factor<T>::type E;
    typedef Vec<E, 8> Frag;
    constexpr int P = Factor<T>::kPlanes;
    constexpr int kA = BM * 2, kB = BN * 2;  // bytes of a row
    constexpr int kLoadsA = BK * P * kA / 1024 / (WM * WN), kLoadsB = BK * P * kB / 1024 / (WM * WN);
    static_assert(kLoadsA * 1024 * WM * WN == BK * P * kA && kLoadsB * 1024 * WM * WN == BK * P * kB, "even shares");
    constexpr int kStageA = BK * P * kA, kStage = kStageA + BK * P * kB;
    constexpr int RM = BM / WM / 32, RN = BN / WN / 32, KK = BK / 16;
    __shared__ __attribute__((aligned(128))) char lds[2 * kStage];

    int64_t ti;
    int tj;
    place(blockIdx.x, a.tm, a.tn, ti, tj);
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63, lr = lane & 31, lc = lane >> 5;
    const int f0 = (int)ti * BM, c0 = tj * BN, slice = blockIdx.y;
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);
    const int64_t all = (a.m + BK - 1) / BK, s0 = slice * a.cut;
    const int stages = (int)(all - s0 < a.cut ? all - s0 : a.cut);

    const E *srca[kLoadsA], *srcb[kLoadsB];
    int rowa[kLoadsA], rowb[kLoadsB];  // row of a stage, or a row that none has where there is no such column
#pragma unroll
    for (int i = 0; i < kLoadsA; ++i) {
        const int byte = (wave * kLoadsA + i) * 1024 + lane * 16, q = byte / kA, p = q / BK, row = q % BK,
                  chunk = byte % kA / 16;
        const int col = f0 + (((chunk >> 1) ^ ((row & 3) * 2)) * 2 + (chunk & 1)) * 8;
        srca[i] = a.a + p * a.a_plane + (s0 * BK + row) * 2 * a.fp + col;
        rowa[i] = col < 2 * a.fp ? row : 1 << 30;
    }
#pragma unroll
    for (int i = 0; i < kLoadsB; ++i) {
        const int byte = (wave * kLoadsB + i) * 1024 + lane * 16, q = byte / kB, p = q / BK, row = q % BK,
                  chunk = byte % kB / 16;
        const int col = c0 + (((chunk >> 1) ^ ((row & 3) * 2)) * 2 + (chunk & 1)) * 8;
        srcb[i] = a.b + p * a.b_plane + (s0 * BK + row) * a.b_pitch + col;
        rowb[i] = col < a.b_pitch ? row : 1 << 30;
    }
    auto load = [&](int s) {
        const int64_t k = (s0 + s) * BK;  // first row
        const int left = a.m - k < BK ? (int)(a.m - k) : BK;
        char *to = lds + (s & 1) * kStage;
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i)
            load_lds(rowa[i] < left ? (const void *)(srca[i] + (int64_t)s * BK * 2 * a.fp) : (const void *)kZeros,
                     to + (wave * kLoadsA + i) * 1024);
#pragma unroll
        for (int i = 0; i < kLoadsB; ++i)
            load_lds(rowb[i] < left ? (const void *)(srcb[i] + (int64_t)s * BK * a.b_pitch) : (const void *)kZeros,
                     to + kStageA + (wave * kLoadsB + i) * 1024);
    };
    // rows k .. k + 8 (by lc) of columns col .. col + 32
    const int trow = lc * 8 + ((lane & 15) >> 2), tcol = ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
    auto frag = [&](const char *base, int bytes, int k, int col) {
        union {
            short4v h[2];
            Frag f;
        } r;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = k + trow + 4 * h, c = col + tcol;
            const char *p = base + row * bytes + (((c >> 4) ^ ((row & 3) * 2)) * 32) + (c & 15) * 2;
            r.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4v *)p);
        }
        return r.f;
    };

    float16v acc[RM][RN] = {};  // [gradients][x]; rows: x's columns, columns: the gradients'
    load(0);
    for (int s = 0; s < stages; ++s) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        const char *la = lds + (s & 1) * kStage, *lb = la + kStageA;
        Frag fa[KK][RM][P], fb[KK][RN][P];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int p = 0; p < P; ++p) {
#pragma unroll
                for (int i = 0; i < RM; ++i) fa[kk][i][p] = frag(la + p * BK * kA, kA, kk * 16, wm + i * 32);
#pragma unroll
                for (int j = 0; j < RN; ++j) fb[kk][j][p] = frag(lb + p * BK * kB, kB, kk * 16, wn + j * 32);
            }
        __builtin_amdgcn_sched_barrier(0);
        if (s + 1 < stages) load(s + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int i = 0; i < RM; ++i)
#pragma unroll
                for (int j = 0; j < RN; ++j) acc[i][j] = mfma_planes<Frag, P>(fb[kk][j], fa[kk][i], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const int f = f0 + wm + i * 32 + lr;
        if (f >= 2 * a.fp) continue;
        const bool up = f >= a.fp;
        const int own = up ? f - a.fp : f;
        if (own >= a.f) continue;
#pragma unroll
        for (int j = 0; j < RN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = c0 + wn + j * 32 + 8 * q + 4 * lc;
                const float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                if (a.slices > 1)
                    store4(a.part + ((int64_t)slice * 2 * a.fp + f) * a.c, c, a.c, a.c % 4 == 0, v);
                else
                    store4((up ? a.up : a.gate) + (int64_t)own * a.c, c, a.c, a.wide, v);
            }
    }
}

// ---- Sums of slices ---------------------------------------------------------------

// out = sum over slices of part[slice][rows][n], where out is one matrix, or two
// of `f` rows each that are `fp` rows of part apart.
template <typename T>
__global__ __launch_bounds__(256) void gated_join(const float *__restrict__ part, int64_t slice, int slices, int64_t size,
                                                  int64_t second, T *__restrict__ out0, T *__restrict__ out1)
{
    const float *p = part + (blockIdx.y ? second : 0);
    T *out = blockIdx.y ? out1 : out0;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < size; i += (int64_t)gridDim.x * 256) {
        float v = 0.f;
#pragma unroll 8
        for (int s = 0; s < slices; ++s) v += p[s * slice + i];
        out[i] = (T)v;
    }
}

// The biases' gradients: `n` rows of 2 fp sums added up, 64 columns a workgroup, 16
// threads each; blockIdx.y: gate, up.
template <typename T>
__global__ __launch_bounds__(1024) void gated_bias(const float *__restrict__ part, int64_t n, int f, int fp,
                                                   float *__restrict__ gate, float *__restrict__ up)
{
    __shared__ double lds[16][65];
    const int x = threadIdx.x & 63, q = threadIdx.x >> 6, at = blockIdx.x * 64 + x;
    const float *p = part + (blockIdx.y ? fp : 0);
    double a = 0.0;
    if (at < f)
#pragma unroll 8
        for (int64_t i = q; i < n; i += 16) a += (double)p[i * 2 * fp + at];
    lds[q][x] = a;
    __syncthreads();
    if (q == 0 && at < f) {
        for (int i = 1; i < 16; ++i) a += lds[i][x];
        (blockIdx.y ? up : gate)[at] = (float)a;
    }
}

// ---- Few rows ----------------------------------------------------------------------

// h for at most 16 G rows: bound by the weights, which are read once, straight into
// registers.  A workgroup takes 16 columns of g and of u; its four waves share out
// the sum's index in stretches of 4 accesses of each row.
template <typename T, int G, bool WIDE>
__global__ __launch_bounds__(256) void gated_few(const T *__restrict__ x, const T *__restrict__ wg,
                                                 const T *__restrict__ wu, const float *__restrict__ b0,
                                                 const float *__restrict__ b1, T *__restrict__ h, int m, int c, int f,
                                                 int kind, bool wide)
{
    constexpr int V = 16 / sizeof(T), kStretch = 4;
    typedef Vec<T, V> Frag;
    __shared__ float4v lds[4][2 * G][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, kq = lane >> 4;
    const int f0 = blockIdx.x * 16, own = f0 + r < f ? f0 + r : f - 1;
    const T *pg = wg + (int64_t)own * c, *pu = wu + (int64_t)own * c;
    const T *px[G];
#pragma unroll
    for (int i = 0; i < G; ++i) px[i] = x + (int64_t)(i * 16 + r < m ? i * 16 + r : m - 1) * c;
    auto get = [&](const T *p, int k) {
        Frag v;
        if constexpr (WIDE) {
            v = k + V <= c ? *(const Frag *)(p + k) : Frag{};
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = k + i < c ? p[k + i] : (T)0.f;
        }
        return v;
    };
    float4v ag[G] = {}, au[G] = {};
    for (int k0 = wave * kStretch * 4 * V; k0 < c; k0 += 4 * kStretch * 4 * V) {
        Frag g[kStretch], u[kStretch];
#pragma unroll
        for (int j = 0; j < kStretch; ++j) {
            g[j] = get(pg, k0 + (j * 4 + kq) * V);
            u[j] = get(pu, k0 + (j * 4 + kq) * V);
        }
#pragma unroll
        for (int j = 0; j < kStretch; ++j)
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const Frag xv = get(px[i], k0 + (j * 4 + kq) * V);
                ag[i] = mfma16(g[j], xv, ag[i]);
                au[i] = mfma16(u[j], xv, au[i]);
            }
    }
#pragma unroll
    for (int i = 0; i < G; ++i) {
        lds[wave][2 * i][lane] = ag[i];
        lds[wave][2 * i + 1][lane] = au[i];
    }
    __syncthreads();
    for (int i = wave; i < G; i += 4) {
        float4v g = lds[0][2 * i][lane], u = lds[0][2 * i + 1][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            g += lds[w][2 * i][lane];
            u += lds[w][2 * i + 1][lane];
        }
        // a lane has row r of x and four columns
        const int row = i * 16 + r, at = f0 + kq * 4;
        if (row >= m) continue;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = at + e < f;
            v[e] = act(kind, g[e] + (b0 && in ? b0[at + e] : 0.f)) * (u[e] + (b1 && in ? b1[at + e] : 0.f));
        }
        store4(h + (int64_t)row * f, at, f, wide, v);
    }
}

// ---- Host ----------------------------------------------------------------------------

inline unsigned blocks_of(int64_t n, int64_t most)
{
    n = (n + 255) / 256;
    return (unsigned)(n < most ? n : most);
}

template <typename T, int MODE>
void launch_nt(const Tiles &t, Nt<T> &a, hipStream_t stream)
{
    a.tm = t.tm;
    a.tn = t.tn;
    a.slices = t.slices;
    a.cut = t.cut;
    const dim3 grid((unsigned)(t.tm * t.tn), (unsigned)t.slices);
    if constexpr (Factor<T>::kPlanes == 1) {
        if (t.bm == 256)
            gated_nt<T, 256, 256, 2, 4, MODE><<<grid, dim3(512), 0, stream>>>(a);
        else
            gated_nt<T, 128, 128, 2, 2, MODE><<<grid, dim3(256), 0, stream>>>(a);
    } else {
        if (t.bm == 256)
            gated_nt<T, 256, 128, 4, 2, MODE><<<grid, dim3(512), 0, stream>>>(a);
        else
            gated_nt<T, 128, 128, 2, 2, MODE><<<grid, dim3(256), 0, stream>>>(a);
    }
}

template <typename T>
bool wide4(const void *p, int64_t n)
{
    return n % 4 == 0 && aligned_to(p, 4 * sizeof(T));
}

// x, the weights as the products read them.
template <typename T>
struct Operands {
    typedef typename Factor<T>::type E;
    Rows<E> x, gate, up;
};

template <typename T>
Operands<T> operands(const wtconv_gated_desc_t &d, const Plan &pl, const void *x, const void *w_gate, const void *w_up,
                     char *&ws, hipStream_t stream)
{
    typedef typename Factor<T>::type E;
    if (!pl.pack)
        return {{(const E *)x, 0, d.c}, {(const E *)w_gate, 0, d.c}, {(const E *)w_up, 0, d.c}};
    E *xp = (E *)ws, *wp = (E *)(ws + pl.x);
    ws += pl.x + pl.w;
    const int64_t plane = d.f * 2 * pl.cp, half = d.f * pl.cp;
    gated_pack<T><<<dim3(blocks_of(d.rows * pl.cp / 8, 8192)), dim3(256), 0, stream>>>((const T *)x, d.rows, (int)d.c, pl.cp,
                                                                                  xp, d.rows * pl.cp);
    gated_pack<T><<<dim3(blocks_of(half / 8, 8192)), dim3(256), 0, stream>>>((const T *)w_gate, d.f, (int)d.c, pl.cp, wp,
                                                                            plane);
    gated_pack<T><<<dim3(blocks_of(half / 8, 8192)), dim3(256), 0, stream>>>((const T *)w_up, d.f, (int)d.c, pl.cp,
                                                                            wp + half, plane);
    return {{xp, d.rows * pl.cp, pl.cp}, {wp, plane, pl.cp}, {wp + half, plane, pl.cp}};
}

template <typename T, int G>
void launch_few(const wtconv_gated_desc_t &d, const Forward &a, hipStream_t stream)
{
    const bool wide = d.c % (16 / sizeof(T)) == 0 && aligned16(a.x) && aligned16(a.w_gate) && aligned16(a.w_up);
    const dim3 grid((unsigned)((d.f + 15) / 16));
    const bool out = wide4<T>(a.h, d.f);
    auto *k = wide ? gated_few<T, G, true> : gated_few<T, G, false>;
    k<<<grid, dim3(256), 0, stream>>>((const T *)a.x, (const T *)a.w_gate, (const T *)a.w_up, a.b_gate, a.b_up,
                                      (T *)a.h, (int)d.rows, (int)d.c, (int)d.f, d.act, out);
}

template <typename T>
hipError_t forward(const wtconv_gated_desc_t &d, const Forward &a, void *workspace, hipStream_t stream)
{
    if (d.rows <= kFewRows) {
        if (d.rows <= 16)
            launch_few<T, 1>(d, a, stream);
        else if (d.rows <= 32)
            launch_few<T, 2>(d, a, stream);
        else
            launch_few<T, 4>(d, a, stream);
        return hipGetLastError();
    }
    const Plan pl = make_plan(d);
    char *ws = (char *)workspace;
    const Operands<T> o = operands<T>(d, pl, a.x, a.w_gate, a.w_up, ws, stream);
    Nt<T> p = {};
    p.a = o.x;
    p.b0 = o.gate;
    p.b1 = o.up;
    p.m = d.rows;
    p.n = (int)d.f;
    p.k = pl.pack ? pl.cp : (int)d.c;
    p.act = d.act;
    p.bias0 = a.b_gate;
    p.bias1 = a.b_up;
    p.out = (T *)a.h;
    p.wide = wide4<T>(a.h, d.f);
    launch_nt<T, kForward>(pl.dual, p, stream);
    return hipGetLastError();
}

template <typename T>
void launch_tn(const Tiles &t, Tn<T> &a, hipStream_t stream)
{
    a.tm = t.tm;
    a.tn = t.tn;
    a.slices = t.slices;
    a.cut = t.cut;
    const dim3 grid((unsigned)(t.tm * t.tn), (unsigned)t.slices);
    if constexpr (Factor<T>::kPlanes == 1) {
        if (t.bm == 256)
            gated_tn<T, 256, 256, 2, 4, 64><<<grid, dim3(512), 0, stream>>>(a);
        else
            gated_tn<T, 128, 128, 2, 2, 64><<<grid, dim3(256), 0, stream>>>(a);
    } else {
        gated_tn<T, 128, 128, 2, 2, 32><<<grid, dim3(256), 0, stream>>>(a);
    }
}

template <typename T>
hipError_t backward(const wtconv_gated_desc_t &d, const Backward &a, void *workspace, hipStream_t stream)
{
    typedef typename Factor<T>::type E;
    const Plan pl = make_plan(d);
    char *ws = (char *)workspace;
    const Operands<T> o = operands<T>(d, pl, a.x, a.w_gate, a.w_up, ws, stream);
    E *grads = (E *)ws, *wt = (E *)(ws + pl.grads);
    float *bias = (float *)(ws + pl.grads + pl.wt), *part = (float *)(ws + pl.grads + pl.wt + pl.bias);
    const int64_t gplane = d.rows * 2 * pl.fp;

    Nt<T> p = {};
    p.a = o.x;
    p.b0 = o.gate;
    p.b1 = o.up;
    p.m = d.rows;
    p.n = (int)d.f;
    p.k = pl.pack ? pl.cp : (int)d.c;
    p.act = d.act;
    p.bias0 = a.b_gate;
    p.bias1 = a.b_up;
    p.dh = (const T *)a.dh;
    p.wide = wide4<T>(a.dh, d.f);
    p.grads = grads;
    p.grads_plane = gplane;
    p.fp = pl.fp;
    p.bias_part = a.db_gate || a.db_up ? bias : nullptr;
    launch_nt<T, kBackward>(pl.dual, p, stream);
    if (a.db_gate)
        gated_bias<T><<<dim3((unsigned)((d.f + 63) / 64), 2), dim3(1024), 0, stream>>>(bias, pl.bias_rows, (int)d.f, pl.fp,
                                                                                    a.db_gate, a.db_up);
    if (a.dx) {
        const int64_t plane = d.c * 2 * pl.fp;
        gated_turn<T><<<dim3((unsigned)((d.c + 63) / 64), (unsigned)((pl.fp + 63) / 64), 2), dim3(256), 0, stream>>>(
            (const T *)a.w_gate, (const T *)a.w_up, (int)d.f, (int)d.c, pl.fp, wt, plane);
        Nt<T> q = {};
        q.a = {grads, gplane, 2 * pl.fp};
        q.b0 = {wt, plane, 2 * pl.fp};
        q.m = d.rows;
        q.n = (int)d.c;
        q.k = 2 * pl.fp;
        q.out = (T *)a.dx;
        q.wide = wide4<T>(a.dx, d.c);
        q.part = part;
        launch_nt<T, kProduct>(pl.dx, q, stream);
        const int64_t size = d.rows * d.c;
        if (pl.dx.slices > 1)
            gated_join<T><<<dim3(blocks_of(size, 4096)), dim3(256), 0, stream>>>(part, size, pl.dx.slices, size, 0,
                                                                             (T *)a.dx, nullptr);
    }
    if (a.dw_gate) {
        Tn<T> q = {};
        q.a = grads;
        q.a_plane = gplane;
        q.b = o.x.p;
        q.b_plane = o.x.plane;
        q.b_pitch = o.x.pitch;
        q.m = d.rows;
        q.f = (int)d.f;
        q.fp = pl.fp;
        q.c = (int)d.c;
        q.gate = (T *)a.dw_gate;
        q.up = (T *)a.dw_up;
        q.wide = wide4<T>(a.dw_gate, d.c) && wide4<T>(a.dw_up, d.c);
        q.part = part;
        launch_tn<T>(pl.dw, q, stream);
        const int64_t size = d.f * d.c;
        if (pl.dw.slices > 1)
            gated_join<T><<<dim3(blocks_of(size, 4096), 2), dim3(256), 0, stream>>>(
                part, (int64_t)2 * pl.fp * d.c, pl.dw.slices, size, (int64_t)pl.fp * d.c, (T *)a.dw_gate, (T *)a.dw_up);
    }
    return hipGetLastError();
}

}  // namespace wtc_gated

#endif  // WTCONV_GATED_BODY_H
