// wtconv_muon_one.hip -- the Newton-Schulz iteration of small matrices, such as
// a layer's own weights (k^2 columns): one workgroup a matrix, one launch for
// the whole call.  A launch costs more than a step's arithmetic here, so what
// counts is that nothing leaves the compute unit between steps.
//
// X (n x m, n <= 64) stays in registers, 32 columns a tile, the tiles dealt to
// the eight waves.  A 32 x 32 matrix instruction leaves its result as column
// lane % 32 and rows 8 q + 4 (lane / 32) + s (q, s = 0..3) of each lane.  Used
// as a right operand of the next instruction, the same registers are 16 rows
// of k in a permuted order; the left operand has to follow the same order, and
// a symmetric matrix in the result's layout does.  So
//   A A   takes both operands from A's own registers,
//   P X   takes P's and X's: neither moves.
// Only X X^T needs X by rows: each wave turns its tiles through its own piece
// of LDS (rows of 80 bytes: neither the writes nor the 16-byte reads collide).
// The waves' parts of A are added in LDS in order, and every wave forms P for
// itself.
#include "wtconv_muon_split.h"

namespace wtc_muon {

namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kRow = 40;  // halves of a row in LDS: 32 and a gap

// Left or right operand (hi, lo), k in the result's order: rows 16 kk .. + 15 of
// a 32 x 32 block in result registers, times s.
__device__ inline void operand(const float16v &r, int kk, float s, half8 &hi, half8 &lo)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        _Float16 h, l;
        split(r[kk * 8 + i] * s, h, l);
        hi[i] = h;
        lo[i] = l;
    }
}

struct Args {
    const void *g;
    void *out;
    const float *momentum, *weight;
    float *momentum_out, *weight_out;
    Blend bl;
    int n, m, tall, steps;
    float eps, decay, step;
};

// NB: 32-row blocks of X; NT: tiles a wave.
template <typename T, int NB, int NT>
__global__ __launch_bounds__(kThreads, 1) void ortho_one(Args a)
{
    constexpr int kSlot = NB == 1 ? 2 * 32 * kRow * 2 : NB * NB * 4096;  // bytes of a wave: turned tile, part of A
    static_assert(kSlot >= 2 * NB * 32 * kRow * 2 && kSlot >= NB * NB * 4096, "a wave's slot holds either");
    __shared__ __attribute__((aligned(16))) char slots[kWaves][kSlot];
    __shared__ float4 sum[NB * NB * 256];
    __shared__ double norms[kWaves];

    const int t = threadIdx.x, wave = t >> 6, lane = t & 63, h = lane >> 5, col = lane & 31;
    const int64_t base = (int64_t)blockIdx.x * a.n * a.m;
    const T *g = (const T *)a.g + base;
    // offset of (row of block b and register r; column of tile k), or -1;
    // from0: the lane's first row and column
    auto at = [&](int2 from0, int b, int r, int k) {
        const int i = b * 32 + 8 * (r >> 2) + from0.x + (r & 3), j = k * kWaves * 32 + from0.y;
        if (i >= a.n || j >= a.m) return -1;
        return a.tall ? j * a.n + i : i * a.m + j;
    };

    const int2 from = make_int2(4 * h, wave * 32 + col);

    float16v x[NT][NB];
    double ss = 0.0;
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            __builtin_amdgcn_sched_barrier(0);  // one block's addresses at a time
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int o = at(from, b, r, k);
                float u = 0.f;
                if (o >= 0) {
                    const T gv = g[o];
                    float mo = 0.f;
                    if (a.bl.muon) {
                        mo = fmaf(a.bl.mu, a.momentum[base + o], (1.f - a.bl.mu) * (float)gv);
                        a.momentum_out[base + o] = mo;
                    }
                    u = blend(a.bl, gv, mo);
                }
                x[k][b][r] = u;
                ss = fma((double)u, (double)u, ss);
            }
        }
    for (int o = 32; o; o >>= 1) ss += __shfl_xor(ss, o);
    if (lane == 0) norms[wave] = ss;
    __syncthreads();
    ss = norms[0];
    for (int w = 1; w < kWaves; ++w) ss += norms[w];
    const double inv = (double)kScale / (sqrt(ss) + (double)a.eps);

    // X as hi + lo, in right-operand order
    half8 xh[NT][NB][2], xl[NT][NB][2];
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = 0; r < 16; ++r) x[k][b][r] = (float)(x[k][b][r] * inv);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) operand(x[k][b], kk, 1.f, xh[k][b][kk], xl[k][b][kk]);
        }

    const int tiles = (a.m + 31) / 32;
    _Float16 *turn = (_Float16 *)slots[wave];
    for (int step = 0; step < a.steps; ++step) {
        // this wave's part of A = X X^T
        float16v acc[NB][NB] = {};
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            if (k * kWaves + wave >= tiles) continue;
            // the reads of the tile before are done (a wave's LDS accesses are
            // in order); the fences keep the compiler from moving them
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int i = b * 32 + 8 * (r >> 2) + 4 * h + (r & 3);
                    turn[i * kRow + col] = xh[k][b][r >> 3][r & 7];
                    turn[(NB * 32 + i) * kRow + col] = xl[k][b][r >> 3][r & 7];
                }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                half8 hi[NB], lo[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const _Float16 *p = turn + (b * 32 + col) * kRow + kk * 16 + h * 8;
                    hi[b] = *(const half8 *)p;
                    lo[b] = *(const half8 *)(p + NB * 32 * kRow);
                }
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j) acc[i][j] = mfma3(hi[i], lo[i], hi[j], lo[j], acc[i][j]);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        float4 *part = (float4 *)slots[wave];
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    part[((i * NB + j) * 4 + q) * 64 + lane] = make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                                                           acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
        __syncthreads();
        for (int e = t; e < NB * NB * 256; e += kThreads) {
            float4 s = ((const float4 *)slots[0])[e];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) {
                const float4 v = ((const float4 *)slots[w])[e];
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
            }
            sum[e] = s;
        }
        __syncthreads();
        // A in units of kScale, P = a I + b A + c A A in the same
        half8 ph[NB][NB][2], pl[NB][NB][2];  // [block of rows][of columns]
        {
            half8 ah[NB][NB][2], al[NB][NB][2];
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    float16v s;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 v = sum[((i * NB + j) * 4 + q) * 64 + lane];
                        s[4 * q] = v.x;
                        s[4 * q + 1] = v.y;
                        s[4 * q + 2] = v.z;
                        s[4 * q + 3] = v.w;
                    }
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) operand(s, kk, 1.f / kScale, ah[i][j][kk], al[i][j][kk]);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    // rows of block i are, by symmetry, block (k, i) with the
                    // lane's column as the row
                    float16v s = {};
#pragma unroll
                    for (int k = 0; k < NB; ++k)
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk)
                            s = mfma3(ah[k][i][kk], al[k][i][kk], ah[k][j][kk], al[k][j][kk], s);
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const float A = (float)ah[i][j][r >> 3][r & 7] + (float)al[i][j][r >> 3][r & 7];
                        s[r] = fmaf(kB, A, (kC / kScale) * s[r]);
                        if (i == j && 8 * (r >> 2) + 4 * h + (r & 3) == col) s[r] += kA * kScale;
                    }
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) operand(s, kk, 1.f, ph[i][j][kk], pl[i][j][kk]);
                    __builtin_amdgcn_sched_barrier(0);
                }
        }
        // X <- P X
        const bool last = step + 1 == a.steps;
        // the outputs' offsets are computed again: kept from the loads, they
        // would be as many registers as X
        int2 to = from;
        asm volatile("" : "+v"(to.x), "+v"(to.y));
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            if (k * kWaves + wave >= tiles) continue;
            float16v y[NB] = {};
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
                        y[i] = mfma3(ph[b][i][kk], pl[b][i][kk], xh[k][b][kk], xl[k][b][kk], y[i]);
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                if (!last) {
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) operand(y[i], kk, 1.f / kScale, xh[k][i][kk], xl[k][i][kk]);
                    continue;
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int o = at(to, i, r, k);
                    if (o < 0) continue;
                    const float v = y[i][r] * (1.f / (kScale * kScale));
                    if (a.weight)
                        a.weight_out[base + o] = fmaf(a.decay, a.weight[base + o], -a.step * v);
                    else
                        ((T *)a.out)[base + o] = (T)v;
                }
            }
        }
    }
}

}  // namespace

// One 32-row block: eight tiles a wave; two: two tiles (registers).
bool one_fits(int n, int m) { return n <= 32 ? m <= 8 * kWaves * 32 : n <= 64 && m <= 2 * kWaves * 32; }

template <typename T>
hipError_t launch_one(const wtconv_ortho_desc_t &d, const WtcOrthoArgs &o, hipStream_t stream)
{
    Args a = {};
    a.tall = d.rows > d.cols;
    a.n = (int)(a.tall ? d.cols : d.rows);
    a.m = (int)(a.tall ? d.rows : d.cols);
    a.g = o.g;
    a.out = o.out;
    a.steps = d.steps;
    a.eps = d.eps;
    if (o.hyper) {
        a.bl = Blend{1, o.hyper->nesterov, o.hyper->momentum};
        a.momentum = o.momentum;
        a.momentum_out = o.momentum_out;
        a.weight = o.weight;
        a.weight_out = o.weight_out;
        a.decay = 1.f - o.hyper->lr * o.hyper->weight_decay;
        a.step = o.hyper->lr * o.hyper->scale;
    }
    const int need = (a.m + 32 * kWaves - 1) / (32 * kWaves);  // tiles a wave
    const dim3 grid((unsigned)d.batch), th(kThreads);
    if (a.n <= 32) {
        if (need <= 1)
            ortho_one<T, 1, 1><<<grid, th, 0, stream>>>(a);
        else if (need <= 2)
            ortho_one<T, 1, 2><<<grid, th, 0, stream>>>(a);
        else if (need <= 4)
            ortho_one<T, 1, 4><<<grid, th, 0, stream>>>(a);
        else
            ortho_one<T, 1, 8><<<grid, th, 0, stream>>>(a);
    } else if (need <= 1) {
        ortho_one<T, 2, 1><<<grid, th, 0, stream>>>(a);
    } else {
        ortho_one<T, 2, 2><<<grid, th, 0, stream>>>(a);
    }
    return hipGetLastError();
}

template hipError_t launch_one<float>(const wtconv_ortho_desc_t &, const WtcOrthoArgs &, hipStream_t);
template hipError_t launch_one<_Float16>(const wtconv_ortho_desc_t &, const WtcOrthoArgs &, hipStream_t);
template hipError_t launch_one<__bf16>(const wtconv_ortho_desc_t &, const WtcOrthoArgs &, hipStream_t);

}  // namespace wtc_muon
