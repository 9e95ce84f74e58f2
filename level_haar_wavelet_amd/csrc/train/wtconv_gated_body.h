// wtconv_gated_body.h -- the gated product's kernels of one element type; the
// files wtconv_gated_f32.hip, _f16.hip and _bf16.hip instantiate them.
//
// Three products on the matrix instructions (32 x 32 x 16, 16-bit factors, fp32
// sums):
//   dual   g = x Wg^T and u = x Wu^T side by side, a wave holding both of the same
//          place, so that act(g) u, or dg and du from dh, are made of registers;
//   dx     [dg du] [Wg; Wu], over 2 F: the weights lie across the sum's index and come out of
//          LDS through the transposing reads (as columns laid out anew by a kernel
//          before, they cost 37 us of 1140 in 8192x2048x5632 bf16);
//   dw     [dg du]^T x, over the rows: so do both factors.
// fp32 factors are three bf16 numbers each, which hold all 24 bits, and a product
// six: those whose size is at least 2^-16 of the first (what is left out is at most
// 2^-24 of the whole, of either sign).  The fp32 matrix instructions run at 1/16 of
// the 16-bit rate.
//
// dg and du are held in the activations' type between the products (fp32: as the three
// numbers): the matrix instructions take no more, and the outputs are rounded to the
// type after them (the backward pass is off by 1.4 times the rounding alone).  Two 16-bit
// numbers each would take twice the matrix instructions of two of the three products.  In
// fp16 that rounding has the range of fp16 too: steps of 2^-24 below 2^-14, dh's own there.
//
// What they take, back to back (bf16, 8192x2048x5632): g, u and h 340 us, 1.11
// PFLOP/s, where the library's product of that size alone takes 357 us; with dh in and
// dg, du out 400 to 440; dx 310 to 360; the weights' gradients 410 to 480.  The counters of dx
// show the matrix unit busy 55 % of the time, and cycles that make 1.85 GHz of 2.4: taken
// for the power limit.  Products of short sums and few columns are further off: 50176x192x768
// fp16 (medians), g and u 84 to 89 us, dx 54 to 60, the weights' gradients 61 to 67; the bytes that
// they were counted to move take 45, 34 and 37.
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

// The products of P x P numbers that count, the smaller ones first.
template <int P>
struct Pairs;
template <>
struct Pairs<1> {
    static constexpr int kCount = 1;
    static constexpr int l[1] = {0}, r[1] = {0};
};
template <>
struct Pairs<3> {
    static constexpr int kCount = 6;
    static constexpr int l[6] = {2, 0, 1, 1, 0, 0}, r[6] = {0, 2, 1, 0, 1, 0};
};

// The nearest bf16 numbers to a and b, and what is left of them.
__device__ inline Vec<__bf16, 2> nearest(float a, float b, float &ra, float &rb)
{
    const Vec<__bf16, 2> o = __builtin_convertvector((Vec<float, 2>{a, b}), Vec<__bf16, 2>);
    const uint32_t both = __builtin_bit_cast(uint32_t, o);
    ra -= __builtin_bit_cast(float, both << 16);
    rb -= __builtin_bit_cast(float, both & 0xffff0000u);
    return o;
}

// a and b as sums of P numbers each.  fp32: the nearest bf16 number, the nearest to the
// rest and what is left, which fits whole (of a value in [1, 2) the last bit is 2^-23, and
// the second rest at most 2^-17).  Cut off instead of rounded, all three had the value's
// sign, and the three products left out had the sign of the whole: up to 2^-21.2 of it and
// 2^-24.7 on average, now 2^-24 and zero.  Beyond the largest bf16 number that one is
// taken, since the nearest would be infinity.  (Of an infinity or a NaN the third is a
// NaN, and with it every sum it is in.)
template <typename T, int P>
__device__ inline void split(float a, float b, Vec<typename Factor<T>::type, 2> (&o)[P])
{
    if constexpr (P == 1) {
        o[0] = Vec<T, 2>{(T)a, (T)b};
    } else {
        constexpr float kMost = 0x1.fep127f;
        float ra = a, rb = b, none = 0.f;
        o[0] = nearest(__builtin_amdgcn_fmed3f(a, -kMost, kMost), __builtin_amdgcn_fmed3f(b, -kMost, kMost), ra, rb);
        o[1] = nearest(ra, rb, ra, rb);
        o[2] = nearest(ra, rb, none, none);
    }
}

template <int KIND>
__device__ inline float act(float z)
{
    if (KIND == WTCONV_ACT_SILU) return z * sigmoid(z);
    if (KIND == WTCONV_ACT_GELU) {
        float e;
        return z * normal_cdf(z, e);
    }
    if (KIND == WTCONV_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN stays
    return z;
}

// act(z) and its slope.
template <int KIND>
__device__ inline float act_slope(float z, float &slope)
{
    if (KIND == WTCONV_ACT_SILU) {
        const float s = sigmoid(z);
        slope = s * fmaf(z, 1.f - s, 1.f);
        return z * s;
    }
    if (KIND == WTCONV_ACT_GELU) {
        float e;
        const float p = normal_cdf(z, e);
        slope = fmaf(z * 0.39894228f, e, p);
        return z * p;
    }
    if (KIND == WTCONV_ACT_RELU) {
        slope = z > 0.f ? 1.f : 0.f;
        return z < 0.f ? 0.f : z;
    }
    slope = 1.f;
    return z;
}

// f(kind) once for all of a wave's values: with a branch at each, one exponential
// waits for the other.
template <typename F>
__device__ inline void with_act(int kind, F f)
{
    if (kind == WTCONV_ACT_SILU)
        f(std::integral_constant<int, WTCONV_ACT_SILU>{});
    else if (kind == WTCONV_ACT_GELU)
        f(std::integral_constant<int, WTCONV_ACT_GELU>{});
    else if (kind == WTCONV_ACT_RELU)
        f(std::integral_constant<int, WTCONV_ACT_RELU>{});
    else
        f(std::integral_constant<int, WTCONV_ACT_NONE>{});
}

// ---- Memory to LDS -------------------------------------------------------------
//
// Loads that go from memory into LDS without registers between, in rings of
// buffers: written as assembly, since the compiler would wait for every such load
// before any read of LDS.  The waits are wait_loads() and the barrier behind it.
// (A vector instruction that writes a scalar register which such a load reads has to be 5
// wait states ahead of it, and the compiler adds none in front of assembly.  It makes no
// such pairs, which tests/test_gated_wait_states.py looks after; waiting in the assembly
// costs 8192x2048x5632 bf16 backward 1086 -> 1100 us.)

typedef uint32_t Descriptor __attribute__((ext_vector_type(4)));

// What a descriptor reaches at most, and an offset that is beyond it.  A tile's accesses
// are within 2^27 bytes of its first row (256 rows of 2^17 values of 4 bytes), so that the
// limit keeps none of them out; without it an offset in a matrix of 2 GB would not be
// outside.
constexpr uint32_t kReach = 0x40000000u, kOutside = 0x7ffffff0u;

__device__ inline uint32_t reach(int64_t bytes)
{
    return bytes < 0 ? 0u : bytes > kReach ? kReach : (uint32_t)bytes;
}

// Memory from `base` on, `bytes` long; reads beyond it give zeros.
__device__ inline Descriptor descriptor(const void *base, int64_t bytes)
{
    const uint64_t b = (uint64_t)base;
    const uint32_t n = reach(bytes);
    Descriptor d;
    d[0] = __builtin_amdgcn_readfirstlane((uint32_t)b);
    d[1] = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32) & 0xffffu);
    d[2] = __builtin_amdgcn_readfirstlane(n);
    d[3] = 0x00020000u;
    return d;
}

// 16 bytes a lane from offset `lane + wave` into LDS, lanes side by side from `to` on.
__device__ inline void load_lds(const Descriptor &d, uint32_t lane, uint32_t wave, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :
                 : "v"(lane), "s"(d), "s"(wave), "s"(to)
                 : "memory", "m0");
}

// The same, 4 bytes a lane.
__device__ inline void load_lds4(const Descriptor &d, uint32_t lane, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 :
                 : "v"(lane), "s"(d), "s"(to)
                 : "memory", "m0");
}

__device__ inline uint32_t lds_offset(const void *p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

// Waits until at most N of this wave's loads are in flight, and for its reads of LDS.
template <int N>
__device__ inline void wait_loads()
{
    static_assert(N < 64, "of the counter");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
}

__device__ inline void barrier()
{
    asm volatile("s_barrier" : : : "memory");
}

// ---- Laying out ----------------------------------------------------------------

// Rows of k elements as `planes` matrices of rows of kp, zeros behind; blockIdx.y: the
// first of two sources, or the second, whose rows follow.
template <typename T>
__global__ __launch_bounds__(256) void gated_pack(const T *__restrict__ src0, const T *__restrict__ src1, int64_t rows,
                                                  int k, int kp, typename Factor<T>::type *__restrict__ dst,
                                                  int64_t plane)
{
    const T *__restrict__ src = blockIdx.y ? src1 : src0;
    dst += blockIdx.y ? rows * kp : 0;
    typedef typename Factor<T>::type E;
    constexpr int P = Factor<T>::kPlanes;
    const int per = kp / 8;
    const int64_t all = rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per;
        const int at = (int)(i - row * per) * 8;
        Vec<E, 8> o[P];
        const T *from = src + row * k + at;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const T v0 = at + j < k ? from[j] : (T)0.f, v1 = at + j + 1 < k ? from[j + 1] : (T)0.f;
            Vec<E, 2> e[P];
            split<T, P>((float)v0, (float)v1, e);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                o[p][j] = e[p][0];
                o[p][j + 1] = e[p][1];
            }
        }
#pragma unroll
        for (int p = 0; p < P; ++p) *(Vec<E, 8> *)(dst + p * plane + row * kp + at) = o[p];
    }
}

// ---- g and u ---------------------------------------------------------------------

enum Mode {
    kForward,  // h = act(g + bg) (u + bu)
    kBackward  // dg, du (and the biases' sums)
};

template <typename E>
struct Rows {
    const E *p;
    int64_t plane, pitch;  // elements
};

template <typename T>
struct Nt {
    typedef typename Factor<T>::type E;
    Rows<E> a, b0, b1;  // rows of x; of the gate's and of the up projection's weights
    int64_t m;
    int n, k;           // columns, length of the sum
    int64_t tm;
    int tn;
    int act;
    const float *bias0, *bias1;
    const T *dh;
    T *out;             // [m][n]
    E *grads;           // kBackward: [plane][m][2 fp], dg and du in turn
    int64_t grads_plane;
    int fp;
    float *bias_part;   // kBackward, or null: [tm * waves along m][2 fp]
    bool wide;          // rows of out and dh in accesses of two elements
};

// Workgroups go to the 8 dies in turn: the place of workgroup g among `all` where each die
// gets a stretch of neighbours, which share operands in its L2.
__device__ inline int64_t place_of(int64_t g, int64_t all)
{
    const int64_t per = all / 8;
    const int rest = (int)(all % 8), die = (int)(g % 8);
    return die * per + (die < rest ? die : rest) + g / 8;
}

// Tile n in bands of 8 tile rows.
__device__ inline void tile_of(int64_t n, int64_t tm, int tn, int64_t &ti, int &tj)
{
    const int64_t band = n / (8 * (int64_t)tn);
    const int h = tm - 8 * band < 8 ? (int)(tm - 8 * band) : 8;
    const int in = (int)(n - band * 8 * tn);
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

typedef __amdgpu_buffer_rsrc_t Resource;

__device__ inline Resource resource(const void *base, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, (int)reach(bytes), 0x00020000);
}

// N elements at `lane + wave` bytes; beyond the resource nothing is written, and
// zeros are read.
template <typename T, int N>
__device__ inline void put(const Vec<T, N> &v, const Resource &to, uint32_t lane, uint32_t wave)
{
    constexpr int kBytes = N * sizeof(T);
    if constexpr (kBytes == 2)
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, v), to, lane, wave, 0);
    else if constexpr (kBytes == 4)
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), to, lane, wave, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(Vec<uint32_t, 2>, v), to, lane, wave, 0);
}

template <typename T, int N>
__device__ inline Vec<T, N> get(const Resource &from, uint32_t lane, uint32_t wave)
{
    constexpr int kBytes = N * sizeof(T);
    if constexpr (kBytes == 2)
        return __builtin_bit_cast(Vec<T, N>, (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(from, lane, wave, 0));
    else if constexpr (kBytes == 4)
        return __builtin_bit_cast(Vec<T, N>, __builtin_amdgcn_raw_buffer_load_b32(from, lane, wave, 0));
    else
        return __builtin_bit_cast(Vec<T, N>, __builtin_amdgcn_raw_buffer_load_b64(from, lane, wave, 0));
}

// Row of a 32 x 32 block that a lane's accumulator q holds, without its 4 (lane / 32); the
// column is lane % 32.
__device__ constexpr int row_of(int q) { return 8 * (q >> 2) + (q & 3); }

// One step (16 of the sum's index) of a wave's blocks; between(n) goes between its
// instructions, n = 0 .. kCount RM RN - 1.
template <int P, int RM, int RN, typename F, typename B>
__device__ inline void products(float16v (&acc)[RM][RN], const F (&fa)[RM][P], const F (&fb)[RN][P], B between)
{
#pragma unroll
    for (int q = 0; q < Pairs<P>::kCount; ++q)
#pragma unroll
        for (int j = 0; j < RN; ++j)
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                acc[i][j] = mfma(fa[i][Pairs<P>::l[q]], fb[j][Pairs<P>::r[q]], acc[i][j]);
                between((q * RN + j) * RM + i);
                __builtin_amdgcn_sched_barrier(0);
            }
}

// A sum of `stages` stages of KK steps each, out of a ring of NB buffers in LDS:
// issue(s, i) sends off load i (of L) of stage s, read(s, k, i, f) takes factor i (of R) of
// step k out of LDS.  A step's factors are read while the one before is multiplied,
// one read behind each of the first half of its matrix instructions (M), so that
// they do not keep the matrix unit waiting.  The barrier before a stage's last step says
// that all waves have read it whole, so that its buffer can be filled anew, and that
// the next one is there.  The loads go behind the second half of the instructions of
// that step and, where there are more, of the next stage's first.  Stages behind the last
// are issued and read like the others, for the sake of the count; issue() gives
// them zeros and nothing is multiplied by them.
template <int NB, int KK, int L, int R, int M, int P, int RM, int RN, typename F, typename I, typename G>
__device__ inline void ring(float16v (&acc)[RM][RN], int stages, I issue, G read)
{
    constexpr int kHalf = M / 2, kReads = (R + kHalf - 1) / kHalf, kIssues = (L + M - 1) / M;
    static_assert(KK % 2 == 0 && NB >= 2, "steps alternate between two sets of factors");
    F f[2];
#pragma unroll
    for (int s = 0; s < NB; ++s)
#pragma unroll
        for (int i = 0; i < L; ++i) issue(s, i);
    wait_loads<(NB - 1) * L>();
    barrier();
#pragma unroll
    for (int i = 0; i < R; ++i) read(0, 0, i, f[0]);
    for (int s = 0; s < stages; ++s) {
#pragma unroll
        for (int k = 0; k < KK; ++k) {
            const bool last = k == KK - 1;
            if (last) {
                wait_loads<(NB - 2) * L>();
                barrier();
            }
            products<P, RM, RN>(acc, f[k % 2].a, f[k % 2].b, [&](int n) {
#pragma unroll
                for (int i = 0; i < kReads; ++i)
                    if (n * kReads + i < R) read(last ? s + 1 : s, last ? 0 : k + 1, n * kReads + i, f[(k + 1) % 2]);
                if (last)
#pragma unroll
                    for (int i = 0; i < kIssues; ++i)
                        if (n * kIssues + i < L) issue(s + NB, n * kIssues + i);
            });
        }
    }
    wait_loads<0>();
}

template <typename E, int P, int RM, int RN>
struct Factors {
    Vec<E, 8> a[RM][P], b[RN][P];
};

// A tile of BM rows of A and BN rows of B; WM x WN waves, NB buffers.  A stage is BK
// elements of each row, whose 16-byte chunks are permuted so that the rows that a read
// phase covers fall into different banks (no conflicts counted).  128 bytes of a row, a
// cache line, in two buffers: with 64 in four, the L2s had twice the requests and dx of
// 8192x2048x5632 bf16 took 396 us in place of 352.  fp32 factors take 64 in three: three
// planes of 128 would not fit twice.
//
// Four waves of 128 x 128 each, one a SIMD, since the factors' reads from LDS then take
// half of its rate beside the stages' writes (eight waves of 128 x 64: all of it);
// where such tiles are fewer than the compute units, 128 x 128 for the workgroup, two of
// them on a compute unit.
//
// A lane ends up with one column of every block of 32.  Rows of B are dealt to the
// blocks so that a lane's columns are neighbours where a wave has enough of them, and
// a row of the output goes out as 32 lanes' contiguous 4 or 8 bytes: whole cache
// lines (of lines written in parts the L2s wrote 1.7 times as much).
template <typename T, int BM, int BN, int WM, int WN, int BK, int NB, int MODE>
__global__ __launch_bounds__(WM *WN * 64, 1) void gated_nt(Nt<T> a)
{
    typedef typename Factor<T>::type E;
    constexpr int P = Factor<T>::kPlanes, W = WM * WN, S = sizeof(T);
    constexpr int kRow = BK * 2, kStage = (BM + BN) * P * kRow, kChunks = kRow / 16;
    // a load takes kPer rows; the waves' loads follow each other
    constexpr int kPer = 1024 / kRow, kTurn = kPer * W, kA = BM / kTurn, kB = BN / kTurn;
    static_assert(kA * kTurn == BM && kB * kTurn == BN, "rows are shared out evenly");
    static_assert(kTurn == 32 || kTurn == 64, "see the rows of B");
    constexpr int RM = BM / WM / 32, RN = BN / WN / 32;
    constexpr int kPair = RN % 4 == 0 ? 2 : 1;  // neighbouring columns of a lane: (g, u) pairs of blocks
    static_assert(RN % 2 == 0 && (kPair == 1 || kTurn == 32), "blocks of g and u");
    typedef Factors<E, P, RM, RN> F;
    __shared__ __attribute__((aligned(128))) char lds[NB * kStage];

    int64_t ti;
    int tj;
    tile_of(place_of(blockIdx.x, a.tm * a.tn), a.tm, a.tn, ti, tj);
    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int lane = t & 63, lr = lane & 31, lc = lane >> 5;
    const int64_t m0 = ti * BM;
    const int n0 = tj * (BN / 2);
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);

    // Row `row` of the first of this wave's loads, the i-th kTurn i rows on; a chunk's
    // place depends on the row modulo 16 only.
    auto swizzle = [](int r) { return kChunks == 8 ? (r >> 1) & 7 : (r >> 2) & 3; };
    const int row = wave * kPer + lane / kChunks, chunk = (lane % kChunks) ^ swizzle(row);
    const uint32_t apitch = (uint32_t)a.a.pitch * 2, bpitch = (uint32_t)a.b0.pitch * 2;
    const uint32_t alane = row * apitch + chunk * 16;
    // Rows of B in the tile, blocks of 32:
    //   pairs   g and u of 64 i + 2 r, g and u of 64 i + 2 r + 1
    //   else    g and u of 32 i + r
    const bool odd = kTurn == 64 && wave * kPer >= 32;  // all of this wave's rows are of u
    const uint32_t blane = kPair * (row % 32) * bpitch + chunk * 16;
    auto first_row = [](int i) {  // of load i
        if (kPair == 2) return i / 4 * 64 + i / 2 % 2;
        return kTurn == 32 ? i / 2 * 32 : i * 32;
    };
    Descriptor da[P], db[P], dup[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        da[p] = descriptor(a.a.p + p * a.a.plane + m0 * a.a.pitch, (a.m - m0) * apitch);
        const int64_t first = p * a.b0.plane + (int64_t)n0 * a.b0.pitch, bytes = (int64_t)(a.n - n0) * bpitch;
        db[p] = descriptor((odd ? a.b1.p : a.b0.p) + first, bytes);
        dup[p] = kTurn == 32 ? descriptor(a.b1.p + first, bytes) : db[p];
    }
    const uint32_t base = lds_offset(lds);
    auto issue = [&](int s, int n) {
        const int k = s * BK, p = n / (kA + kB), i = n % (kA + kB);
        // a row's end inside the stage: zeros, not the next row
        const bool in = k + chunk * 8 < a.k;
        const uint32_t to = base + s % NB * kStage + wave * 1024;
        if (i < kA)
            load_lds(da[p], in ? alane : kOutside, k * 2 + i * kTurn * apitch, to + p * BM * kRow + i * W * 1024);
        else
            load_lds((i - kA) % 2 ? dup[p] : db[p], in ? blane : kOutside, k * 2 + first_row(i - kA) * bpitch,
                     to + P * BM * kRow + p * BN * kRow + (i - kA) * W * 1024);
    };
    auto read = [&](int s, int kk, int n, F &f) {
        const char *at = lds + s % NB * kStage + (((kk * 2 + lc) ^ swizzle(lr)) * 16) + lr * kRow;
        const int p = n % P, i = n / P;
        if (i < RN)
            f.b[i][p] = *(const Vec<E, 8> *)(at + P * BM * kRow + (p * BN + wn + i * 32) * kRow);
        else
            f.a[i - RN][p] = *(const Vec<E, 8> *)(at + (p * BM + wm + (i - RN) * 32) * kRow);
    };
    float16v acc[RM][RN] = {};  // rows: A's, columns: B's
    ring<NB, BK / 16, P *(kA + kB), P *(RM + RN), Pairs<P>::kCount * RM * RN, P, RM, RN, F>(acc, (a.k + BK - 1) / BK,
                                                                                            issue, read);

    // this lane's first row
    const int64_t mine = m0 + wm + 4 * lc;
    // dh, or h: kPair neighbours at once where they lie so
    const T *io = MODE == kForward ? a.out : a.dh;
    const Resource rio = resource(io + m0 * a.n, (a.m - m0) * a.n * S);
    constexpr int kSets = RN / (2 * kPair);  // of blocks with the same columns of a lane
    auto column = [&](int set) { return n0 + wn / 2 + set * kPair * 32 + kPair * lr; };
    auto offset = [&](int f) { return ((uint32_t)(mine - m0) * a.n + f) * S; };
    // dh of a block of rows is sent for before the one in front of it is used: with one wave
    // a SIMD there is nothing else to do while it comes
    Vec<T, kPair> d[2][16];
    auto fetch = [&](int n) {
        const int f = column(n / RM), i = n % RM;
        const uint32_t at0 = f < a.n ? offset(f) : kOutside, at1 = f + 1 < a.n ? offset(f + 1) : kOutside;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const uint32_t rows = (i * 32 + row_of(q)) * a.n * S;
            if (kPair == 1 || a.wide) {
                d[n & 1][q] = get<T, kPair>(rio, at0, rows);
            } else {
                d[n & 1][q][0] = get<T, 1>(rio, at0, rows)[0];
                d[n & 1][q][kPair - 1] = get<T, 1>(rio, at1, rows)[0];
            }
        }
    };
    if (MODE == kBackward) fetch(0);
    with_act(a.act, [&](auto kind) {
#pragma unroll
        for (int set = 0; set < kSets; ++set) {
            const int f = column(set), j = set * 2 * kPair;
            float bg[kPair], bu[kPair], sg[kPair] = {}, su[kPair] = {};
#pragma unroll
            for (int h = 0; h < kPair; ++h) {
                bg[h] = a.bias0 && f + h < a.n ? a.bias0[f + h] : 0.f;
                bu[h] = a.bias1 && f + h < a.n ? a.bias1[f + h] : 0.f;
            }
            const uint32_t at0 = f < a.n ? offset(f) : kOutside, at1 = f + 1 < a.n ? offset(f + 1) : kOutside;
            const uint32_t to = f < a.fp ? ((uint32_t)(mine - m0) * a.fp + f) * 4 : kOutside;
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                const int n = set * RM + i;
                if (MODE == kBackward && n + 1 < kSets * RM) fetch(n + 1);
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    float g[kPair], u[kPair];
#pragma unroll
                    for (int h = 0; h < kPair; ++h) {
                        g[h] = acc[i][j + 2 * h][q] + bg[h];
                        u[h] = acc[i][j + 2 * h + 1][q] + bu[h];
                    }
                    if constexpr (MODE == kForward) {
                        const uint32_t rows = (i * 32 + row_of(q)) * a.n * S;
                        Vec<T, kPair> o;
#pragma unroll
                        for (int h = 0; h < kPair; ++h) o[h] = (T)(act<kind>(g[h]) * u[h]);
                        if (kPair == 1 || a.wide) {
                            put<T, kPair>(o, rio, at0, rows);
                        } else {
                            put<T, 1>(Vec<T, 1>{o[0]}, rio, at0, rows);
                            put<T, 1>(Vec<T, 1>{o[kPair - 1]}, rio, at1, rows);
                        }
                    } else {
                        // columns and rows behind the last: dh is zero there
                        Vec<E, 2 * kPair> o[P];
#pragma unroll
                        for (int h = 0; h < kPair; ++h) {
                            float slope;
                            const float y = act_slope<kind>(g[h], slope), dv = (float)d[n & 1][q][h];
                            const float dg = dv * u[h] * slope, du = dv * y;
                            sg[h] += dg;
                            su[h] += du;
                            Vec<E, 2> e[P];
                            split<T, P>(dg, du, e);
#pragma unroll
                            for (int p = 0; p < P; ++p) {
                                o[p][2 * h] = e[p][0];
                                o[p][2 * h + 1] = e[p][1];
                            }
                        }
#pragma unroll
                        for (int p = 0; p < P; ++p)
                            put<E, 2 * kPair>(o[p], resource(a.grads + p * a.grads_plane + m0 * 2 * a.fp,
                                                             (a.m - m0) * 4 * a.fp),
                                              to, (i * 32 + row_of(q)) * a.fp * 4);
                    }
                    if (q % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // fewer values live at once
                }
            }
            if (MODE == kBackward && a.bias_part)
#pragma unroll
                for (int h = 0; h < kPair; ++h) {
                    const float g = sg[h] + __shfl_xor(sg[h], 32), u = su[h] + __shfl_xor(su[h], 32);
                    if (!lc && f + h < a.n) {
                        float *out = a.bias_part + (ti * WM + wave / WN) * 2 * a.fp + f + h;
                        out[0] = g;
                        out[a.fp] = u;
                    }
                }
        }
    });
}

}  // namespace wtc_gated

#include "wtconv_gated_short.h"

namespace wtc_gated {

// ---- Tiles that are cut along the sum's index ------------------------------------------

struct Cut {
    int64_t tm;
    int tn, slices;
    int64_t stages;  // of a slice
    float *part;     // [tile][slice][bm][bn], where there are several
};

// Tile and slice (or -1) of workgroup g: slice by slice, whose tiles read the same stretch
// of the sum's index (tile by tile, the gradients of 50176x192x768 fp16 came from memory
// twice, 361 MiB).
__device__ inline int place(const Cut &c, int64_t g, int64_t &ti, int &tj, int64_t &tile)
{
    const int64_t tiles = c.tm * c.tn, n = place_of(g, tiles * c.slices);
    tile = n % tiles;
    tile_of(tile, c.tm, c.tn, ti, tj);
    return c.slices > 1 ? (int)(n / tiles) : -1;
}

// A wave's accumulators to its slice's place; `mine` and `col`: this lane's first row and
// its column of the first block.
template <int BM, int BN, int RM, int RN>
__device__ inline void write_part(const Cut &c, int64_t tile, int slice, const float16v (&acc)[RM][RN], int mine, int col)
{
    float *to = c.part + (tile * c.slices + slice) * (BM * BN) + mine * BN + col;
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q)
#pragma unroll
            for (int j = 0; j < RN; ++j) to[(i * 32 + row_of(q)) * BN + j * 32] = acc[i][j][q];
}

// The slices' sums of a tile added up, four columns a thread and 1024 / bn rows a
// workgroup (blockIdx.y).  dx: [rows][cols] of one matrix; TURNS: rows of g's and u's
// gradients in turn.
template <typename O, bool TURNS>
__global__ __launch_bounds__(256) void gated_join(Cut c, int bm, int bn, int64_t rows, int cols, O *__restrict__ out0,
                                                  O *__restrict__ out1)
{
    int64_t ti;
    int tj;
    tile_of(blockIdx.x, c.tm, c.tn, ti, tj);
    const int e = (blockIdx.y * 256 + threadIdx.x) * 4, col = tj * bn + e % bn;
    const int64_t row = ti * bm + e / bn, own = TURNS ? row >> 1 : row;
    if (col >= cols || own >= rows) return;
    const float *part = c.part + (int64_t)blockIdx.x * c.slices * bm * bn + e;
    float4v v = {};
#pragma unroll 8
    for (int s = 0; s < c.slices; ++s) v += *(const float4v *)(part + (int64_t)s * bm * bn);
    O *out = (TURNS && (row & 1) ? out1 : out0) + own * cols;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (col + i < cols) out[col + i] = (O)v[i];
}

// ---- dx ------------------------------------------------------------------------------

template <typename T>
struct Nn {
    typedef typename Factor<T>::type E;
    const E *a;            // [plane][m][2 fp], dg and du in turn
    int64_t a_plane;
    Rows<E> gate, up;      // [plane][f][c]
    int64_t m;
    int n, f, fp;          // columns: c
    Cut cut;
    T *out;                // [m][n]
};

// What a lane gives the transposing read of 16 rows of the sum's index and 32 columns:
// 16 lanes take 4 rows of 32 bytes, and a lane gets its column's values of the four;
// rows lc 8 + 4 h + trow (h: the first and the second read).
struct Transposed {
    int trow, tcol;
};
__device__ inline Transposed transposed(int lane)
{
    return {(lane & 15) >> 2, ((lane >> 4) & 1) * 16 + (lane & 3) * 4};
}

__device__ inline short4v read_transposed(const char *p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4v *)p);
}

// D = A [Wg; Wu], rows of the weights in turn, as the columns of A.  A's rows lie in LDS as
// in gated_nt.  A stage's rows of Wg come first, then those of Wu; their 32-byte pieces
// are permuted so that the four rows of a read, two of each, lie in different banks.
template <typename T, int BM, int BN, int WM, int WN, int BK, int NB>
__global__ __launch_bounds__(WM *WN * 64, 1) void gated_nn(Nn<T> a)
{
    typedef typename Factor<T>::type E;
    constexpr int P = Factor<T>::kPlanes, W = WM * WN;
    constexpr int kRow = BK * 2, kChunks = kRow / 16, kRowB = BN * 2;  // bytes
    constexpr int kStageA = BM * P * kRow, kStage = kStageA + BK * P * kRowB;
    constexpr int kPer = 1024 / kRow, kTurn = kPer * W, kA = BM / kTurn;
    constexpr int kPerB = 1024 / kRowB, kTurnB = kPerB * W, kB = BK / kTurnB;
    static_assert(kA * kTurn == BM && kB * kTurnB == BK && BK / 2 % kTurnB == 0, "rows are shared out evenly");
    constexpr int RM = BM / WM / 32, RN = BN / WN / 32;
    typedef Factors<E, P, RM, RN> F;
    __shared__ __attribute__((aligned(128))) char lds[NB * kStage];

    int64_t ti, tile;
    int tj;
    const int slice = place(a.cut, blockIdx.x, ti, tj, tile);
    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int lane = t & 63, lr = lane & 31, lc = lane >> 5;
    const int64_t m0 = ti * BM;
    const int n0 = tj * BN;
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);
    const int64_t all = (2 * a.fp + BK - 1) / BK, s0 = slice < 0 ? 0 : slice * a.cut.stages;
    const int stages = (int)(slice < 0 || all - s0 < a.cut.stages ? all - s0 : a.cut.stages);
    const int k0 = (int)(s0 * BK), k1 = k0 + stages * BK < 2 * a.fp ? k0 + stages * BK : 2 * a.fp;

    auto swizzle = [](int r) { return kChunks == 8 ? (r >> 1) & 7 : (r >> 2) & 3; };
    const int row = wave * kPer + lane / kChunks, chunk = (lane % kChunks) ^ swizzle(row);
    const uint32_t apitch = (uint32_t)a.fp * 4, bpitch = (uint32_t)a.gate.pitch * 2;
    const uint32_t alane = row * apitch + chunk * 16;
    const int brow = wave * kPerB + lane / (kRowB / 16), bchunk = lane % (kRowB / 16);
    auto key = [](int r, int up) { return ((r & 1) * 2 + up) * 2; };  // of the 32-byte pieces
    uint32_t blane[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) blane[z] = brow * bpitch + ((((bchunk >> 1) ^ key(brow, z)) * 2) + (bchunk & 1)) * 16;
    const uint32_t base = lds_offset(lds);
    Descriptor da[P], dw[2][P];
#pragma unroll
    for (int p = 0; p < P; ++p) da[p] = descriptor(a.a + p * a.a_plane + m0 * 2 * a.fp, (a.m - m0) * apitch);
    const int end = k1 / 2 < a.f ? k1 / 2 : a.f;
    auto issue = [&](int s, int n) {
        const int k = k0 + s * BK, p = n / (kA + kB), i = n % (kA + kB);
        const uint32_t to = base + s % NB * kStage + wave * 1024;
        if (i < kA) {
            const bool in = k + chunk * 8 < k1;
            load_lds(da[p], in ? alane : kOutside, k * 2 + i * kTurn * apitch, to + p * BM * kRow + i * W * 1024);
        } else {
            // columns behind a row's end come out of the next row, into results that nobody takes;
            // behind the last row, and behind this slice's, there are zeros
            const int j = i - kA, z = j >= kB / 2, own = j - z * (kB / 2), f = k / 2;
            const Rows<E> &w = z ? a.up : a.gate;
            if (own == 0)  // once for a stage: beside few matrix instructions its arithmetic counts
                dw[z][p] = descriptor(w.p + p * w.plane + (int64_t)f * w.pitch + n0, (int64_t)(end - f) * bpitch - n0 * 2);
            load_lds(dw[z][p], blane[z], own * kTurnB * bpitch, to + kStageA + p * BK * kRowB + j * W * 1024);
        }
    };
    const Transposed tr = transposed(lane);
    auto read = [&](int s, int kk, int n, F &f) {
        const char *la = lds + s % NB * kStage, *lb = la + kStageA;
        const int p = n % P, i = n / P;
        if (i < RN) {
            union {
                short4v h[2];
                Vec<E, 8> f;
            } r;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int up = tr.trow & 1, own = kk * 8 + lc * 4 + h * 2 + (tr.trow >> 1), c = wn + i * 32 + tr.tcol;
                r.h[h] = read_transposed(lb + p * BK * kRowB + (up * (BK / 2) + own) * kRowB +
                                         (((c >> 4) ^ key(own, up)) * 32) + (c & 15) * 2);
            }
            f.b[i][p] = r.f;
        } else {
            f.a[i - RN][p] = *(const Vec<E, 8> *)(la + (p * BM + wm + (i - RN) * 32 + lr) * kRow +
                                                  (((kk * 2 + lc) ^ swizzle(lr)) * 16));
        }
    };
    float16v acc[RM][RN] = {};
    ring<NB, BK / 16, P *(kA + kB), P *(RM + RN), Pairs<P>::kCount * RM * RN, P, RM, RN, F>(acc, stages, issue, read);

    const int mine = wm + 4 * lc;  // this lane's first row of the tile
    if (slice >= 0) {
        write_part<BM, BN>(a.cut, tile, slice, acc, mine, wn + lr);
        return;
    }
    const Resource to = resource(a.out + m0 * a.n, (a.m - m0) * a.n * (int)sizeof(T));
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q)
#pragma unroll
            for (int j = 0; j < RN; ++j) {
                const int n = n0 + wn + j * 32 + lr;
                put<T, 1>(Vec<T, 1>{(T)acc[i][j][q]}, to,
                          n < a.n ? ((uint32_t)mine * a.n + n) * (uint32_t)sizeof(T) : kOutside,
                          (i * 32 + row_of(q)) * a.n * (uint32_t)sizeof(T));
            }
}

// ---- The weights' gradients -------------------------------------------------------

template <typename T, typename O>
struct Tn {
    typedef typename Factor<T>::type E;
    const E *a, *b;  // [plane][m][2 fp] (dg and du in turn), [plane][m][pitch]
    int64_t a_plane, b_plane, b_pitch;
    int64_t m;
    int f, fp, c;
    Cut cut;
    O *gate, *up;    // [f][c]; O: T, or fp32 for parameters that are kept so
};

// D = A^T B, a tile of BM columns of A (gradients) and BN of B (x), over a slice
// of the rows, 32 of them a stage.  LDS holds rows as they come; the transposing
// read gives a lane four rows' values of its column: 16 lanes take 4 rows of 32
// bytes, and these 32-byte pieces are permuted by row so that a read's rows lie in
// different banks.
template <typename T, typename O, int BM, int BN, int WM, int WN, int NB>
__global__ __launch_bounds__(WM *WN * 64, 1) void gated_tn(Tn<T, O> a)
{
    typedef typename Factor<T>::type E;
    constexpr int P = Factor<T>::kPlanes, W = WM * WN, BK = 32;
    constexpr int kRowA = BM * 2, kRowB = BN * 2;  // bytes of a row
    constexpr int kA = BK * kRowA / 1024 / W, kB = BK * kRowB / 1024 / W;
    static_assert(kA * 1024 * W == BK * kRowA && kB * 1024 * W == BK * kRowB, "rows are shared out evenly");
    constexpr int kStageA = BK * P * kRowA, kStage = kStageA + BK * P * kRowB;
    constexpr int RM = BM / WM / 32, RN = BN / WN / 32;
    typedef Factors<E, P, RM, RN> F;
    __shared__ __attribute__((aligned(128))) char lds[NB * kStage];

    int64_t ti, tile;
    int tj;
    const int slice = place(a.cut, blockIdx.x, ti, tj, tile);
    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int lane = t & 63, lr = lane & 31, lc = lane >> 5;
    const int f0 = (int)ti * BM, c0 = tj * BN;
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);
    const int64_t all = (a.m + BK - 1) / BK, s0 = slice < 0 ? 0 : slice * a.cut.stages;
    const int stages = (int)(slice < 0 || all - s0 < a.cut.stages ? all - s0 : a.cut.stages);

    const int64_t m1 = (s0 + stages) * BK < a.m ? (s0 + stages) * BK : a.m;
    // A load takes the rows of 1024 bytes, the waves' loads follow each other; where a
    // chunk goes depends on its row modulo 4, which is the same for all of a wave's.
    const uint32_t apitch = (uint32_t)a.fp * 4, bpitch = (uint32_t)a.b_pitch * 2;
    constexpr int kPerA = 1024 / kRowA, kPerB = 1024 / kRowB;
    static_assert(kPerA * W % 4 == 0 && kPerB * W % 4 == 0, "rows modulo 4");
    auto lane_offset = [&](int per, uint32_t pitch) {
        const int chunks = 64 / per, in = wave * per + lane / chunks, chunk = lane % chunks;
        return in * pitch + ((((chunk >> 1) ^ ((in & 3) * 2)) * 2) + (chunk & 1)) * 16;
    };
    const uint32_t alane = lane_offset(kPerA, apitch), blane = lane_offset(kPerB, bpitch);
    const uint32_t base = lds_offset(lds);
    // A stage's descriptors follow from those of the stage before: beside few matrix
    // instructions their arithmetic counts.
    Descriptor da[P], db[P];
    const E *pa = a.a + s0 * BK * 2 * a.fp + f0, *pb = a.b + s0 * BK * a.b_pitch + c0;
    int64_t left_a = (m1 - s0 * BK) * apitch - f0 * 2, left_b = (m1 - s0 * BK) * bpitch - c0 * 2;  // bytes
    auto issue = [&](int s, int n) {
        const int p = n / (kA + kB), i = n % (kA + kB);
        const uint32_t to = base + s % NB * kStage + wave * 1024;
        // columns behind a row's end come out of the next row, into results that nobody takes;
        // behind the last row there are zeros
        if (i == 0) da[p] = descriptor(pa + p * a.a_plane, left_a);
        if (i == kA) db[p] = descriptor(pb + p * a.b_plane, left_b);
        if (i < kA)
            load_lds(da[p], alane, i * W * kPerA * apitch, to + p * BK * kRowA + i * W * 1024);
        else
            load_lds(db[p], blane, (i - kA) * W * kPerB * bpitch, to + kStageA + p * BK * kRowB + (i - kA) * W * 1024);
        if (n + 1 == P * (kA + kB)) {
            pa += BK * 2 * a.fp;
            pb += BK * a.b_pitch;
            left_a -= BK * (int64_t)apitch;
            left_b -= BK * (int64_t)bpitch;
        }
    };
    // rows k .. k + 8 (by lc) of columns col .. col + 32
    const Transposed tr = transposed(lane);
    auto frag = [&](const char *from, int bytes, int k, int col) {
        union {
            short4v h[2];
            Vec<E, 8> f;
        } r;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = col + tr.tcol;
            r.h[h] = read_transposed(from + (k + lc * 8 + tr.trow + 4 * h) * bytes + (((c >> 4) ^ (tr.trow * 2)) * 32) +
                                     (c & 15) * 2);
        }
        return r.f;
    };
    auto read = [&](int s, int kk, int n, F &f) {
        const char *la = lds + s % NB * kStage, *lb = la + kStageA;
        const int p = n % P, i = n / P;
        if (i < RN)
            f.b[i][p] = frag(lb + p * BK * kRowB, kRowB, kk * 16, wn + i * 32);
        else
            f.a[i - RN][p] = frag(la + p * BK * kRowA, kRowA, kk * 16, wm + (i - RN) * 32);
    };
    float16v acc[RM][RN] = {};  // rows: the gradients' columns, columns: x's
    ring<NB, BK / 16, P *(kA + kB), P *(RM + RN), Pairs<P>::kCount * RM * RN, P, RM, RN, F>(acc, stages, issue, read);

    const int mine = wm + 4 * lc;  // this lane's first row of the tile
    if (slice >= 0) {
        write_part<BM, BN>(a.cut, tile, slice, acc, mine, wn + lr);
        return;
    }
    // rows of g and of u in turn
    const int64_t first = (int64_t)(f0 / 2) * a.c, bytes = (int64_t)(a.f - f0 / 2) * a.c * (int)sizeof(O);
    const Resource to[2] = {resource(a.gate + first, bytes), resource(a.up + first, bytes)};
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q)
#pragma unroll
            for (int j = 0; j < RN; ++j) {
                const int c = c0 + wn + j * 32 + lr;
                put<O, 1>(Vec<O, 1>{(O)acc[i][j][q]}, to[q & 1],
                          c < a.c ? ((uint32_t)(mine / 2) * a.c + c) * (uint32_t)sizeof(O) : kOutside,
                          (uint32_t)((i * 32 + row_of(q)) / 2) * a.c * (uint32_t)sizeof(O));
            }
}

// ---- The biases' gradients ------------------------------------------------------------

// `n` rows of 2 fp sums added up, 16 columns a workgroup, 64 threads each; blockIdx.y:
// gate, up.
template <typename T>
__global__ __launch_bounds__(1024) void gated_bias(const float *__restrict__ part, int64_t n, int f, int fp,
                                                   float *__restrict__ gate, float *__restrict__ up)
{
    __shared__ double lds[64][17];
    const int x = threadIdx.x & 15, q = threadIdx.x >> 4, at = blockIdx.x * 16 + x;
    const float *p = part + (blockIdx.y ? fp : 0);
    double a = 0.0;
    if (at < f)
#pragma unroll 8
        for (int64_t i = q; i < n; i += 64) a += (double)p[i * 2 * fp + at];
    lds[q][x] = a;
    __syncthreads();
    if (q < 8) {
        a = 0.0;
        for (int i = 0; i < 8; ++i) a += lds[q * 8 + i][x];
    }
    __syncthreads();
    if (q < 8) lds[q][x] = a;
    __syncthreads();
    if (q == 0 && at < f) {
        for (int i = 1; i < 8; ++i) a += lds[i][x];
        (blockIdx.y ? up : gate)[at] = (float)a;
    }
}

// ---- Few rows ----------------------------------------------------------------------

// h for at most 16 G rows: bound by the weights, which are read once, straight into
// registers (1x1024x4096 bf16: 5.5 us, 3.0 TB/s, of the weights' 16 MiB, most of it the
// latency of a workgroup's two turns).  A workgroup takes 16 columns of g and of u; its four waves share out
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
        with_act(kind, [&](auto k) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = at + e < f;
                v[e] = act<k>(g[e] + (b0 && in ? b0[at + e] : 0.f)) * (u[e] + (b1 && in ? b1[at + e] : 0.f));
            }
        });
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
    const dim3 grid((unsigned)(t.tm * t.tn));
    if constexpr (Factor<T>::kPlanes == 1) {
        if (t.bm == 256)
            gated_nt<T, 256, 256, 2, 2, 64, 2, MODE><<<grid, dim3(256), 0, stream>>>(a);
        else
            gated_nt<T, 128, 128, 4, 1, 64, 2, MODE><<<grid, dim3(256), 0, stream>>>(a);
    } else {
        gated_nt<T, 128, 128, 2, 2, 32, 3, MODE><<<grid, dim3(256), 0, stream>>>(a);
    }
}

inline Cut cut_of(const Tiles &t, float *part) { return {t.tm, t.tn, t.slices, t.cut, part}; }

template <typename O, bool TURNS>
void launch_join(const Tiles &t, const Cut &c, int64_t rows, int64_t cols, void *out0, void *out1, hipStream_t stream)
{
    if (t.slices > 1)
        gated_join<O, TURNS><<<dim3((unsigned)(t.tm * t.tn), (unsigned)(t.bm * t.bn / 1024)), dim3(256), 0, stream>>>(
            c, t.bm, t.bn, rows, (int)cols, (O *)out0, (O *)out1);
}

template <typename T>
void launch_nn(const Tiles &t, const Nn<T> &a, hipStream_t stream)
{
    const dim3 grid((unsigned)t.groups());
    if constexpr (Factor<T>::kPlanes == 1) {
        if (t.bm == 256)
            gated_nn<T, 256, 256, 2, 2, 64, 2><<<grid, dim3(256), 0, stream>>>(a);
        else
            gated_nn<T, 128, 128, 2, 2, 64, 2><<<grid, dim3(256), 0, stream>>>(a);
    } else {
        gated_nn<T, 128, 128, 2, 2, 32, 3><<<grid, dim3(256), 0, stream>>>(a);
    }
}

template <typename T>
bool wide4(const void *p, int64_t n)
{
    return n % 4 == 0 && aligned_to(p, 4 * sizeof(T));
}

template <typename T>
bool wide2(const void *p, int64_t n)
{
    return n % 2 == 0 && aligned_to(p, 2 * sizeof(T));
}

// x, the weights as the products read them.
template <typename T>
struct Operands {
    typedef typename Factor<T>::type E;
    Rows<E> x, gate, up;
};

// ... laid out anew where the plan says so, x only where it is asked for.
template <typename T>
Operands<T> operands(const wtconv_gated_desc_t &d, const Plan &pl, const void *x, const void *w_gate, const void *w_up,
                     bool pack_x, char *&ws, hipStream_t stream)
{
    typedef typename Factor<T>::type E;
    if (!pl.pack)
        return {{(const E *)x, 0, d.c}, {(const E *)w_gate, 0, d.c}, {(const E *)w_up, 0, d.c}};
    E *xp = (E *)ws, *wp = (E *)(ws + pl.x);
    ws += pl.x + pl.w;
    const int64_t plane = d.f * 2 * pl.cp, half = d.f * pl.cp;
    if (pack_x)
        gated_pack<T><<<dim3(blocks_of(d.rows * pl.cp / 8, 8192)), dim3(256), 0, stream>>>(
            (const T *)x, nullptr, d.rows, (int)d.c, pl.cp, xp, d.rows * pl.cp);
    gated_pack<T><<<dim3(blocks_of(half / 8, 8192), 2), dim3(256), 0, stream>>>(
        (const T *)w_gate, (const T *)w_up, d.f, (int)d.c, pl.cp, wp, plane);
    return {{xp, d.rows * pl.cp, pl.cp}, {wp, plane, pl.cp}, {wp + half, plane, pl.cp}};
}

// Waves along a tile's rows, each with its own sums for the biases.
template <typename T>
int bias_waves(const Tiles &t)
{
    return Factor<T>::kPlanes == 1 && t.bm == 128 ? 4 : 2;
}

template <typename T, int MODE>
void launch_short(const wtconv_gated_desc_t &d, const Plan &pl, const Operands<T> &o, Short<T> &a, hipStream_t stream)
{
    a.gate = o.gate;
    a.up = o.up;
    a.m = d.rows;
    a.n = (int)d.f;
    a.c = (int)d.c;
    a.act = d.act;
    a.tiles = pl.row_tiles;
    a.parts = pl.parts;
    a.cut = pl.part_cut;
    auto run = [&](auto ks) {
        gated_short<T, ks, MODE><<<dim3((unsigned)(a.tiles * a.parts)), dim3(pl.waves * 64), 0, stream>>>(a);
    };
    if (pl.steps == 2)
        run(std::integral_constant<int, 2>{});
    else if (pl.steps == 4)
        run(std::integral_constant<int, 4>{});
    else if (pl.steps == 6)
        run(std::integral_constant<int, 6>{});
    else if (pl.steps == 8)
        run(std::integral_constant<int, 8>{});
    else if (pl.steps == 12)
        run(std::integral_constant<int, 12>{});
    else if constexpr (Factor<T>::kPlanes == 1)
        run(std::integral_constant<int, 16>{});
}

// Whether h's or dh's address allows the kernel for short rows that the plan has.  (x: its
// loads of 16 bytes need 4, which fp32 has and the entry points ask for otherwise.)
template <typename T>
bool short_rows(const wtconv_gated_desc_t &d, const Plan &pl, const void *h)
{
    return pl.row_tiles && wide4<T>(h, d.f);
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
    const bool brief = short_rows<T>(d, pl, a.h);
    const Operands<T> o = operands<T>(d, pl, a.x, a.w_gate, a.w_up, !brief, ws, stream);
    if (brief) {
        Short<T> p = {};
        p.x = (const T *)a.x;
        p.bias0 = a.b_gate;
        p.bias1 = a.b_up;
        p.out = (T *)a.h;
        launch_short<T, kForward>(d, pl, o, p, stream);
        return hipGetLastError();
    }
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
    p.wide = wide2<T>(a.h, d.f);
    launch_nt<T, kForward>(pl.dual, p, stream);
    return hipGetLastError();
}

template <typename T, typename O>
void launch_tn(const Tiles &t, const Tn<T, O> &a, hipStream_t stream)
{
    const dim3 grid((unsigned)t.groups());
    if constexpr (Factor<T>::kPlanes == 1) {
        if (t.bm == 256)
            gated_tn<T, O, 256, 256, 2, 2, 4><<<grid, dim3(256), 0, stream>>>(a);
        else
            gated_tn<T, O, 128, 128, 2, 2, 4><<<grid, dim3(256), 0, stream>>>(a);
    } else {
        gated_tn<T, O, 128, 128, 2, 2, 3><<<grid, dim3(256), 0, stream>>>(a);
    }
}

template <typename T, typename O>
void weights_backward(const wtconv_gated_desc_t &d, const Plan &pl, const Backward &a, const Operands<T> &o,
                      const typename Factor<T>::type *grads, float *part, hipStream_t stream)
{
    Tn<T, O> q = {};
    q.a = grads;
    q.a_plane = d.rows * 2 * pl.fp;
    q.b = o.x.p;
    q.b_plane = o.x.plane;
    q.b_pitch = o.x.pitch;
    q.m = d.rows;
    q.f = (int)d.f;
    q.fp = pl.fp;
    q.c = (int)d.c;
    q.gate = (O *)a.dw_gate;
    q.up = (O *)a.dw_up;
    q.cut = cut_of(pl.dw, part);
    launch_tn<T, O>(pl.dw, q, stream);
    launch_join<O, true>(pl.dw, q.cut, d.f, d.c, a.dw_gate, a.dw_up, stream);
}

template <typename T>
hipError_t backward(const wtconv_gated_desc_t &d, const Backward &a, void *workspace, hipStream_t stream)
{
    typedef typename Factor<T>::type E;
    const Plan pl = make_plan(d);
    char *ws = (char *)workspace;
    const bool brief = short_rows<T>(d, pl, a.dh);
    const Operands<T> o = operands<T>(d, pl, a.x, a.w_gate, a.w_up, !brief || a.dw_gate, ws, stream);
    E *grads = (E *)ws;
    float *bias = (float *)(ws + pl.grads), *part = (float *)(ws + pl.grads + pl.bias);
    const int64_t gplane = d.rows * 2 * pl.fp;
    int64_t bias_rows;
    if (brief) {
        Short<T> p = {};
        p.x = (const T *)a.x;
        p.bias0 = a.b_gate;
        p.bias1 = a.b_up;
        p.dh = (const T *)a.dh;
        p.grads = grads;
        p.grads_plane = gplane;
        p.fp = pl.fp;
        p.bias_part = a.db_gate ? bias : nullptr;
        bias_rows = pl.row_tiles * pl.waves;
        launch_short<T, kBackward>(d, pl, o, p, stream);
    } else {
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
        p.wide = wide2<T>(a.dh, d.f);
        p.grads = grads;
        p.grads_plane = gplane;
        p.fp = pl.fp;
        p.bias_part = a.db_gate ? bias : nullptr;
        bias_rows = bias_waves<T>(pl.dual) * pl.dual.tm;
        launch_nt<T, kBackward>(pl.dual, p, stream);
    }
    if (a.db_gate)
        gated_bias<T><<<dim3((unsigned)((d.f + 15) / 16), 2), dim3(1024), 0, stream>>>(bias, bias_rows, (int)d.f, pl.fp,
                                                                                    a.db_gate, a.db_up);
    if (a.dx) {
        Nn<T> q = {};
        q.a = grads;
        q.a_plane = gplane;
        q.gate = o.gate;
        q.up = o.up;
        q.m = d.rows;
        q.n = (int)d.c;
        q.f = (int)d.f;
        q.fp = pl.fp;
        q.out = (T *)a.dx;
        q.cut = cut_of(pl.dx, part);
        launch_nn<T>(pl.dx, q, stream);
        launch_join<T, false>(pl.dx, q.cut, d.rows, d.c, a.dx, nullptr, stream);
    }
    if (a.dw_gate && a.dw_f32)
        weights_backward<T, float>(d, pl, a, o, grads, part, stream);
    else if (a.dw_gate)
        weights_backward<T, T>(d, pl, a, o, grads, part, stream);
    return hipGetLastError();
}

}  // namespace wtc_gated

#endif  // WTCONV_GATED_BODY_H
