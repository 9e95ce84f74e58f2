// wtconv_muon.hip -- Newton-Schulz orthogonalisation of a batch of matrices,
// alone or inside the Muon step.
//
// X is n x m with n <= m: G, or the transpose of a tall G.  A step is three
// products: A = X X^T, P = a I + b A + c A A, X <- P X.
//
// What the iteration needs of its products: it lifts small singular values by
// up to a^5 = 485, and every rounding error with them, so 16-bit factors (an
// error of 2^-12 at the start) would leave errors of a few per cent in the
// result.  The fp32 matrix instructions are exact enough but run at 1/16 of the
// fp16 rate.  So every factor is held as two fp16 numbers, v S = hi + lo / 2^11, S
// = 2^14, which puts the largest possible |v| just under fp16's range.  hi is off
// by at most 2^-11 of v S and lo by 2^-11 of that: 22 bits, where fp32 has 24, for
// |v| down to 2^-28.  Below, hi is a subnormal number (the matrix instructions take
// it as it is) and v is off by up to 2^-49.  Since v is an entry of a matrix of
// norm 1, rows and columns of very different sizes keep their own digits.  (With
// lo in hi's units the error was 2^-39 from 2^-17 down, and the last row of 384 x
// 1536 graded over 2^-24 was off by 2.5e-3 of itself.)  A product is three fp16
// matrix products, hi hi into one fp32 accumulator and hi lo + lo hi into another
// (lo lo is below the 22 bits): 3/16 of the fp32 rate's time.
//
// Layout of such a matrix ("planes"): row-major, the columns in blocks of 32,
// each block 32 hi then 32 lo: 128 bytes, one cache line, one row of a tile.
// Sides are padded with zeros to the tile, which no product changes.  All
// products have the form L R^T with both operands' rows along k; X is therefore
// kept as rows of X (for X X^T) and rows of X^T (for P X), and the products
// whose results are symmetric (A, P) compute the tiles on and below the
// diagonal and write each of them twice.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cstdint>

#include "wtconv_check.h"
#include "wtconv_muon.h"
#include "wtconv_muon_plan.h"
#include "wtconv_muon_split.h"

namespace {

using namespace wtc_muon;

constexpr int kThreads = kTiledThreads;

// ---- The update's norm and the first planes ----------------------------------

// Partial sums of |U|^2 in fp64 (fp32 squares would overflow from 2^64 on and
// vanish below 2^-75), one for each of gridDim.x workgroups of a matrix, and
// momentum_out.  V elements an access (1 where addresses do not allow 4), four
// accesses in flight.
template <typename T, int V>
__global__ __launch_bounds__(kThreads) void ortho_norm(const T *__restrict__ g, const float *momentum,
                                                       float *momentum_out, Blend bl, int64_t size,
                                                       double *__restrict__ parts)
{
    typedef T TV __attribute__((ext_vector_type(V)));
    typedef float FV __attribute__((ext_vector_type(V)));
    __shared__ double lds[kThreads / 64];
    const int64_t base = blockIdx.y * size, step = (int64_t)gridDim.x * kThreads * V;
    double a = 0.0;
    for (int64_t i0 = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * V; i0 < size; i0 += 4 * step) {
        TV gv[4];
        FV mv[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i0 + k * step < size) {
                gv[k] = *(const TV *)(g + base + i0 + k * step);
                if (bl.muon) mv[k] = *(const FV *)(momentum + base + i0 + k * step);
            }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i0 + k * step < size) {
                if (bl.muon) {
#pragma unroll
                    for (int j = 0; j < V; ++j) mv[k][j] = fmaf(bl.mu, mv[k][j], (1.f - bl.mu) * (float)gv[k][j]);
                    *(FV *)(momentum_out + base + i0 + k * step) = mv[k];
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const double u = blend(bl, gv[k][j], mv[k][j]);
                    a = fma(u, u, a);
                }
            }
    }
    for (int o = 32; o; o >>= 1) a += __shfl_xor(a, o);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kThreads / 64; ++i) a += lds[i];
        parts[blockIdx.y * gridDim.x + blockIdx.x] = a;
    }
}

// hi and lo of 8 values.
__device__ inline void split8(const float (&v)[8], half8 &hi, half8 &lo)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        _Float16 h, l;
        split(v[i], h, l);
        hi[i] = h;
        lo[i] = l;
    }
}

// Element offset of the 8 values from column k (a multiple of 8) of a row.
__device__ inline int64_t plane_at(int row, int k, int kp) { return (int64_t)row * 2 * kp + (k >> 5) * 64 + (k & 31); }

__device__ inline void store8(_Float16 *plane, int row, int k, int kp, const float (&v)[8])
{
    half8 hi, lo;
    split8(v, hi, lo);
    _Float16 *p = plane + plane_at(row, k, kp);
    *(half8 *)p = hi;
    *(half8 *)(p + 32) = lo;
}

// Planes of S U / (|U| + eps) as rows of U (rp x cp) and of U^T, zero-padded;
// one workgroup per 64 x 64 tile.
template <typename T>
__global__ __launch_bounds__(kThreads) void ortho_split(const T *__restrict__ g,
                                                        const float *__restrict__ momentum_out, Blend bl, int rows,
                                                        int cols, int rp, int cp, float eps, float S,
                                                        const double *__restrict__ parts, int nparts,
                                                        _Float16 *__restrict__ u, _Float16 *__restrict__ ut)
{
    __shared__ float tile[64][65];
    const int t = threadIdx.x, z = blockIdx.y;
    const int64_t base = (int64_t)z * rows * cols;
    const int r0 = blockIdx.x / (cp / 64) * 64, c0 = blockIdx.x % (cp / 64) * 64, c = c0 + (t & 63);
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = r0 + (t >> 6) + i * 4;
        v[i] = 0.f;
        if (r < rows && c < cols) {
            const int64_t e = base + (int64_t)r * cols + c;
            v[i] = blend(bl, g[e], bl.muon ? momentum_out[e] : 0.f);
        }
    }
    // every wave adds the parts for itself, in the same order
    double a = 0.0;
    for (int i = t & 63; i < nparts; i += 64) a += parts[z * nparts + i];
    for (int o = 32; o; o >>= 1) a += __shfl_xor(a, o);
    const double inv = (double)S / (sqrt(a) + (double)eps);
#pragma unroll
    for (int i = 0; i < 16; ++i) tile[(t >> 6) + i * 4][t & 63] = (float)(v[i] * inv);
    __syncthreads();
    u += (int64_t)z * rp * cp * 2;
    ut += (int64_t)z * rp * cp * 2;
#pragma unroll
    for (int i = t; i < 512; i += kThreads) {
        float w[8];
        const int r = i >> 3, k = (i & 7) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = tile[r][k + j];
        store8(u, r0 + r, c0 + k, cp, w);
        const int q = i >> 3, l = (i & 7) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = tile[l + j][q];
        store8(ut, c0 + q, r0 + l, rp, w);
    }
}

// ---- The products ------------------------------------------------------------

enum Mode {
    kStore,  // D = f acc
    kPoly,   // D = a I + b A + c f acc, A the left operand's planes
    kFinal   // the outputs, in the caller's layout and type
};

struct Product {
    const _Float16 *L, *R;   // planes of lp x kp and rp x kp
    _Float16 *D, *Dt;        // planes of lp x rp and (null or) of its transpose
    int lp, rp, kp;          // padded sides
    int sym;                 // D is symmetric: tiles on and below the diagonal only, Dt = D
    int tiles, batch;        // tiles of a matrix; matrices
    // of all tiles the first `full` are a workgroup's each; the others are cut
    // into `slices` along k of `cut` 32-blocks, whose sums go to `part`
    int full, slices, cut;
    float4 *part;
    float f;                 // from the accumulator to D's scale
    float a, b, c;           // kPoly: b includes the change of scale
    // kFinal: element (i, j) of the product, i < n, j < m, is the output's
    // (i, j), or (j, i) where tall
    int n, m, tall;
    const float *weight;     // Muon: weight_out = decay weight - step value
    void *out;
    float decay, step;
};

typedef const __attribute__((address_space(1))) void *GlobalPtr;
typedef __attribute__((address_space(3))) void *LdsPtr;

// D tile (TILE x TILE) = L R^T over k in stages of 32 KB.  128 and 64: the four
// waves in 2 x 2, each a quarter of the tile in 32 x 32 matrix instructions; 32:
// each wave the whole tile, over a quarter of every stage, added at the end.
// A stage's rows of L and R (128 bytes for each 32 of k) go from memory into
// LDS without registers between; the 16-byte chunks of a row are permuted by
// chunk ^ (row / 2) % 8 so that the 16 rows a read phase covers fall into
// different banks.  Two buffers: a stage's reads into registers come first, then
// the next stage's loads are sent off, then its matrix instructions run.  With
// few workgroups a stage costs the latency of its loads, so small tiles take
// more of k at once.
//
// P X of 4096^3 (tiles of 128) takes 400 to 430 us: 0.96 to 1.03 PFLOP/s of fp16
// products, where the library's product of that size reaches 1.09; the card's
// power limit holds both.  The last one, with the weights, takes 450 to 480.  1024^3
// (tiles of 64, 256 of them) takes 17 us: 12.6 without its loads, 16.3 without its
// matrix instructions, so it waits for its operands' way from the L2s.  Three or
// four buffers instead of two: 15.4 us there, but 9.6 to 13 us instead of 9 for the
// symmetric products.
// DEEP (is_deep()): a compute unit has one workgroup only, whose stages take
// twice the k: X of 384x1536 9.4 -> 9.0 us (tiles of 64), its Gram product 10.8 us in
// one piece where cut along k and joined it took 12.

// Matrix, tile row and tile column of tile g of all matrices.
template <int TILE>
__device__ inline void place(const Product &a, int g, int &z, int &ti, int &tj)
{
    z = g / a.tiles;
    const int tile = g % a.tiles;
    if (a.sym) {
        ti = (int)((sqrtf(8.f * tile + 1.f) - 1.f) * 0.5f);
        while ((ti + 1) * (ti + 2) / 2 <= tile) ++ti;
        while (ti * (ti + 1) / 2 > tile) --ti;
        tj = tile - ti * (ti + 1) / 2;
    } else {
        // bands of 8 tile rows, so that the tiles in flight share operands
        const int nj = a.rp / TILE, ni = a.lp / TILE, band = tile / (8 * nj);
        const int h = ni - 8 * band < 8 ? ni - 8 * band : 8, in = tile - band * 8 * nj;
        ti = band * 8 + in % h;
        tj = in / h;
    }
}

template <int TILE>
struct Lds {
    static constexpr int kPitch = TILE + 1;  // of the result's tile
    static constexpr int kResult = TILE * kPitch * 4;
};

// The result's tile in LDS (rows of kPitch) to where it goes.
template <int TILE, int MODE, typename T>
__device__ inline void finish(const Product &a, float *res, int z, int ti, int tj)
{
    constexpr int kPitch = Lds<TILE>::kPitch;
    const int t = threadIdx.x;
    const int i0 = ti * TILE, j0 = tj * TILE;
    if (MODE == kFinal) {
        const int64_t base = (int64_t)z * a.n * a.m;
        for (int e = t; e < TILE * TILE; e += kThreads) {
            const int i = a.tall ? e % TILE : e / TILE, j = a.tall ? e / TILE : e % TILE;
            if (i0 + i >= a.n || j0 + j >= a.m) continue;
            const float v = res[i * kPitch + j] * a.f;
            const int64_t o = base + (a.tall ? (int64_t)(j0 + j) * a.n + i0 + i : (int64_t)(i0 + i) * a.m + j0 + j);
            if (a.weight)
                ((float *)a.out)[o] = fmaf(a.decay, a.weight[o], -a.step * v);
            else
                ((T *)a.out)[o] = (T)v;
        }
        return;
    }
    _Float16 *D = a.D + (int64_t)z * a.lp * a.rp * 2;
    const _Float16 *A = a.L + (int64_t)z * a.lp * a.kp * 2;
    for (int e = t; e < TILE * TILE / 8; e += kThreads) {
        const int i = e / (TILE / 8), j = (e % (TILE / 8)) * 8;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = res[i * kPitch + j + q] * a.f;
        if (MODE == kPoly) {
            const _Float16 *p = A + plane_at(i0 + i, j0 + j, a.kp);
            const half8 hi = *(const half8 *)p, lo = *(const half8 *)(p + 32);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                v[q] = fmaf(a.b, fmaf((float)lo[q], 1.f / kLo, (float)hi[q]), a.c * v[q]);
                if (i0 + i == j0 + j + q) v[q] += a.a;
            }
            if (a.sym && ti != tj)
#pragma unroll
                for (int q = 0; q < 8; ++q) res[i * kPitch + j + q] = v[q];
        }
        store8(D, i0 + i, j0 + j, a.rp, v);
    }
    _Float16 *Dt = a.sym ? (ti != tj ? a.D : nullptr) : a.Dt;
    if (!Dt) return;
    if (MODE == kPoly) __syncthreads();
    Dt += (int64_t)z * a.lp * a.rp * 2;
    for (int e = t; e < TILE * TILE / 8; e += kThreads) {
        const int j = e % TILE, i = (e / TILE) * 8;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = res[(i + q) * kPitch + j] * (MODE == kPoly ? 1.f : a.f);
        store8(Dt, j0 + j, i0 + i, a.lp, v);
    }
}

// A wave's part of the tile in matrix-instruction order to LDS, and the waves'
// sums along k, so that rows and columns go out in 16-byte pieces.
template <int TILE>
__device__ inline void to_lds(const float16v (&acc)[Shape<TILE>::kSide / 32][Shape<TILE>::kSide / 32], float *res)
{
    using Sh = Shape<TILE>;
    constexpr int RB = Sh::kSide / 32, kPitch = Lds<TILE>::kPitch;
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63, lr = lane & 31, lc = lane >> 5;
    const int wi = Sh::kWavesK > 1 ? 0 : (wave >> 1) * Sh::kSide, wj = Sh::kWavesK > 1 ? 0 : (wave & 1) * Sh::kSide;
    float *own = res + (Sh::kWavesK > 1 ? wave * TILE * kPitch : 0);
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < RB; ++j)
#pragma unroll
            for (int q = 0; q < 16; ++q)
                own[(wi + i * 32 + 8 * (q >> 2) + 4 * lc + (q & 3)) * kPitch + wj + j * 32 + lr] = acc[i][j][q];
    __syncthreads();
    if (Sh::kWavesK > 1) {
        for (int e = t; e < TILE * TILE; e += kThreads) {
            const int o = e / TILE * kPitch + e % TILE;
            float v = res[o];
#pragma unroll
            for (int w = 1; w < Sh::kWavesK; ++w) v += res[w * TILE * kPitch + o];
            res[o] = v;
        }
        __syncthreads();
    }
}

template <int TILE, bool DEEP, int MODE, typename T>
__global__ __launch_bounds__(kThreads, 2) void product(Product a)
{
    using Sh = Shape<TILE>;
    constexpr int KB = Sh::kBlocks * (DEEP ? 2 : 1), KW = KB / Sh::kWavesK;  // 32-blocks of k: of a stage, of a wave
    constexpr int RB = Sh::kSide / 32;                      // 32-row blocks of a wave
    constexpr int kBlock = 2 * TILE * 128, kStage = KB * kBlock;  // bytes
    constexpr int kResult = Lds<TILE>::kResult * Sh::kWavesK;
    __shared__ __attribute__((aligned(128))) char lds[2 * kStage > kResult ? 2 * kStage : kResult];

    int g = blockIdx.x, slice = -1, z, ti, tj;
    if (g < a.full) {
        // workgroups go to the 8 dies in turn: give each die neighbouring tiles
        const int per = a.full / 8, rest = a.full % 8, die = g % 8;
        g = die * per + (die < rest ? die : rest) + g / 8;
    } else {
        slice = (g - a.full) % a.slices;
        g = a.full + (g - a.full) / a.slices;
    }
    place<TILE>(a, g, z, ti, tj);
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
    const int64_t ldb = (int64_t)a.kp * 4;  // bytes of a row
    const char *L = (const char *)a.L + ((int64_t)z * a.lp + ti * TILE) * ldb;
    const char *R = (const char *)a.R + ((int64_t)z * a.rp + tj * TILE) * ldb;

    const int64_t k0_bytes = slice < 0 ? 0 : (int64_t)slice * a.cut * 128;
    // this lane's source of each load of a block of k: 8 rows a load, row
    // lane / 8 of them
    constexpr int kLoads = 2 * TILE / 32;  // per wave
    const char *src[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int row = (wave * kLoads + i) * 8 + (lane >> 3);
        const int chunk = (lane & 7) ^ ((row >> 1) & 7);
        src[i] = (row < TILE ? L + row * ldb : R + (row - TILE) * ldb) + chunk * 16 + k0_bytes;
    }
    const int all = a.kp / 32, k0 = slice < 0 ? 0 : slice * a.cut;
    const int blocks = slice < 0 ? all : all - k0 < a.cut ? all - k0 : a.cut, stages = (blocks + KB - 1) / KB;
    auto load = [&](int s) {
#pragma unroll
        for (int b = 0; b < KB; ++b)
            if (KB == 1 || s * KB + b < blocks)
#pragma unroll
                for (int i = 0; i < kLoads; ++i)
                    __builtin_amdgcn_global_load_lds(
                        (GlobalPtr)(src[i] + (int64_t)(s * KB + b) * 128),
                        (LdsPtr)(lds + (s & 1) * kStage + b * kBlock + (wave * kLoads + i) * 1024), 16, 0, 0);
    };
    auto frag = [&](int s, int b, int row, int chunk) {
        return *(const half8 *)(lds + (s & 1) * kStage + b * kBlock + row * 128 + ((chunk ^ ((row >> 1) & 7)) * 16));
    };

    // hi hi, and hi lo + lo hi (RB = 1: each its own, none waits for the one before)
    float16v acc[RB][RB] = {}, cross[RB][RB] = {}, term = {};
    const int wi = Sh::kWavesK > 1 ? 0 : (wave >> 1) * Sh::kSide, wj = Sh::kWavesK > 1 ? 0 : (wave & 1) * Sh::kSide;
    const int b0 = Sh::kWavesK > 1 ? wave * KW : 0, lr = lane & 31, lc = lane >> 5;
    load(0);
    for (int s = 0; s < stages; ++s) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        half8 l[KW][2][RB][2], r[KW][2][RB][2];  // [block of k][half][block of rows][hi, lo]
#pragma unroll
        for (int b = 0; b < KW; ++b)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int i = 0; i < RB; ++i) {
                        l[b][kk][i][p] = frag(s, b0 + b, wi + i * 32 + lr, p * 4 + kk * 2 + lc);
                        r[b][kk][i][p] = frag(s, b0 + b, TILE + wj + i * 32 + lr, p * 4 + kk * 2 + lc);
                    }
        __builtin_amdgcn_sched_barrier(0);
        if (s + 1 < stages) load(s + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = 0; b < KW; ++b) {
            if (KB > 1 && s * KB + b0 + b >= blocks) continue;  // the last stage's missing blocks
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                if constexpr (RB == 1) {
                    term = mfma(l[b][kk][0][0], r[b][kk][0][1], term);
                    cross[0][0] = mfma(l[b][kk][0][1], r[b][kk][0][0], cross[0][0]);
                    acc[0][0] = mfma(l[b][kk][0][0], r[b][kk][0][0], acc[0][0]);
                } else {
#pragma unroll
                    for (int i = 0; i < RB; ++i)
#pragma unroll
                        for (int j = 0; j < RB; ++j) {
                            cross[i][j] =
                                mfma_cross(l[b][kk][i][0], l[b][kk][i][1], r[b][kk][j][0], r[b][kk][j][1], cross[i][j]);
                            acc[i][j] = mfma(l[b][kk][i][0], r[b][kk][j][0], acc[i][j]);
                        }
                }
            }
        }
    }
    if (RB == 1) cross[0][0] += term;
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < RB; ++j) acc[i][j] += cross[i][j] * (1.f / kLo);

    if (slice >= 0) {
        float4 *p = a.part + ((int64_t)(g - a.full) * a.slices + slice) * (RB * RB * 4 * kThreads) + t;
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < RB; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    p[((i * RB + j) * 4 + q) * kThreads] = make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                                                       acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
        return;
    }
    __syncthreads();
    float *res = (float *)lds;
    to_lds<TILE>(acc, res);
    finish<TILE, MODE, T>(a, res, z, ti, tj);
}

// Adds the slices of the tiles that were cut along k, in order, and finishes
// them; one workgroup a tile.
template <int TILE, int MODE, typename T>
__global__ __launch_bounds__(kThreads) void join(Product a)
{
    using Sh = Shape<TILE>;
    constexpr int RB = Sh::kSide / 32;
    __shared__ __attribute__((aligned(128))) char lds[Lds<TILE>::kResult * Sh::kWavesK];
    int z, ti, tj;
    place<TILE>(a, a.full + blockIdx.x, z, ti, tj);
    float16v acc[RB][RB] = {};
    const float4 *p = a.part + (int64_t)blockIdx.x * a.slices * (RB * RB * 4 * kThreads) + threadIdx.x;
#pragma unroll 2
    for (int s = 0; s < a.slices; ++s, p += RB * RB * 4 * kThreads)
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < RB; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 v = p[((i * RB + j) * 4 + q) * kThreads];
                    acc[i][j][4 * q] += v.x;
                    acc[i][j][4 * q + 1] += v.y;
                    acc[i][j][4 * q + 2] += v.z;
                    acc[i][j][4 * q + 3] += v.w;
                }
    to_lds<TILE>(acc, (float *)lds);
    finish<TILE, MODE, T>(a, (float *)lds, z, ti, tj);
}

// ---- Host ----------------------------------------------------------------------

template <int TILE, int MODE, typename T>
void launch_tile(const Deal &d, const Product &a, hipStream_t stream)
{
    const int rest = a.tiles * a.batch - a.full;
    const unsigned groups = (unsigned)(a.full + rest * a.slices);
    if (is_deep(groups, a.slices > 1 ? a.cut : a.kp / 32, TILE))
        product<TILE, TILE < 128, MODE, T><<<dim3(groups), dim3(kThreads), 0, stream>>>(a);
    else
        product<TILE, false, MODE, T><<<dim3(groups), dim3(kThreads), 0, stream>>>(a);
    if (rest) join<TILE, MODE, T><<<dim3((unsigned)rest), dim3(kThreads), 0, stream>>>(a);
}

template <int MODE, typename T = float>
void launch_product(const Deal &d, Product a, hipStream_t stream)
{
    a.tiles = d.tiles;
    a.full = d.full;
    a.slices = d.slices;
    a.cut = d.cut;
    if (d.tile == 128)
        launch_tile<128, MODE, T>(d, a, stream);
    else if (d.tile == 64)
        launch_tile<64, MODE, T>(d, a, stream);
    else
        launch_tile<32, MODE, T>(d, a, stream);
}

template <typename T>
hipError_t run(const wtconv_ortho_desc_t &d, const WtcOrthoArgs &o, void *workspace, hipStream_t stream)
{
    const Plan pl = make_plan(d);
    if (pl.one) return launch_one<T>(d, o, stream);
    const unsigned batch = (unsigned)d.batch;
    const int64_t size = d.rows * d.cols;
    char *ws = (char *)workspace;
    _Float16 *x[2], *xt[2];  // rows of X, rows of X^T
    for (int i = 0; i < 2; ++i) {
        x[i] = (_Float16 *)ws;
        xt[i] = (_Float16 *)(ws += pl.xbytes);
        ws += pl.xbytes;
    }
    _Float16 *A = (_Float16 *)ws, *P = (_Float16 *)(ws += pl.abytes);
    double *parts = (double *)(ws += pl.abytes);
    float4 *part = (float4 *)(ws += align256(sizeof(double) * pl.parts * d.batch));
    const Blend bl = {o.hyper != nullptr, o.hyper ? o.hyper->nesterov : 0, o.hyper ? o.hyper->momentum : 0.f};
    const T *g = (const T *)o.g;
    const bool wide = size % 4 == 0 && aligned_to(g, 4 * sizeof(T)) &&
                      (!o.hyper || (aligned16(o.momentum) && aligned16(o.momentum_out)));
    const dim3 ngrid((unsigned)pl.parts, batch);
    if (wide)
        ortho_norm<T, 4><<<ngrid, dim3(kThreads), 0, stream>>>(g, o.momentum, o.momentum_out, bl, size, parts);
    else
        ortho_norm<T, 1><<<ngrid, dim3(kThreads), 0, stream>>>(g, o.momentum, o.momentum_out, bl, size, parts);
    const int rp = pl.tall ? pl.mp : pl.np, cp = pl.tall ? pl.np : pl.mp;
    const float S = kScale;
    ortho_split<T><<<dim3((cp / 64) * (rp / 64), batch), dim3(kThreads), 0, stream>>>(
        g, o.momentum_out, bl, (int)d.rows, (int)d.cols, rp, cp, d.eps, S, parts, pl.parts, pl.tall ? xt[0] : x[0],
        pl.tall ? x[0] : xt[0]);
    for (int s = 0; s < d.steps; ++s) {
        const int at = s & 1;
        Product a = {};
        a.batch = (int)batch;
        a.part = part;
        a.L = a.R = x[at];
        a.D = A;
        a.lp = a.rp = pl.np;
        a.kp = pl.mp;
        a.sym = 1;
        a.f = 1.f / S;  // acc is in units of S^2, D in units of S
        launch_product<kStore>(pl.gram, a, stream);
        a.L = a.R = A;
        a.D = P;
        a.kp = pl.np;
        a.a = kA * S;
        a.b = kB;
        a.c = kC;
        launch_product<kPoly>(pl.poly, a, stream);
        a.L = P;
        a.R = xt[at];
        a.D = x[1 - at];
        a.Dt = xt[1 - at];
        a.rp = pl.mp;
        a.sym = 0;
        if (s + 1 < d.steps) {
            launch_product<kStore>(pl.apply, a, stream);
            continue;
        }
        a.f = 1.f / (S * S);
        a.n = pl.n;
        a.m = pl.m;
        a.tall = pl.tall;
        a.out = o.out;
        if (o.hyper) {
            a.weight = o.weight;
            a.out = o.weight_out;
            a.decay = 1.f - o.hyper->lr * o.hyper->weight_decay;
            a.step = o.hyper->lr * o.hyper->scale;
        }
        launch_product<kFinal, T>(pl.apply, a, stream);
    }
    return hipGetLastError();
}

}  // namespace

size_t wtc_ortho_workspace(const wtconv_ortho_desc_t &d)
{
    return workspace_bytes(make_plan(d), d.batch);
}

hipError_t wtc_launch_ortho(const wtconv_ortho_desc_t &d, const WtcOrthoArgs &a, void *workspace, hipStream_t stream)
{
    if (d.dtype == WTCONV_F32) return run<float>(d, a, workspace, stream);
    if (d.dtype == WTCONV_F16) return run<_Float16>(d, a, workspace, stream);
    return run<__bf16>(d, a, workspace, stream);
}
