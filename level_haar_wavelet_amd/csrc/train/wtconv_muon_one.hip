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
// The waves' parts of A are added in LDS in order; every wave forms P for itself
// (up to 32 rows), or a block of it for all.
#include "wtconv_muon_plan.h"
#include "wtconv_muon_split.h"

namespace wtc_muon {

namespace {

constexpr int kWaves = kOneWaves, kThreads = 64 * kWaves;
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

// One matrix in memory: elements by number, reads past the end (kNone) give 0
// and writes there are dropped, so that no access needs a branch.
constexpr unsigned kNone = 0x3fffffff;

template <typename T>
struct Matrix {
    __amdgpu_buffer_rsrc_t r;
    __device__ Matrix(const T *p, unsigned count)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<T *>(p), 0, count * sizeof(T), 0x00020000))
    {
    }
    __device__ float get(unsigned o) const
    {
        if constexpr (sizeof(T) == 4) {
            return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, o * 4, 0, 0));
        } else {
            return (float)__builtin_bit_cast(T, (short)__builtin_amdgcn_raw_buffer_load_b16(r, o * 2, 0, 0));
        }
    }
    __device__ void put(unsigned o, float v) const
    {
        if constexpr (sizeof(T) == 4)
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(int, v), r, o * 4, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, (T)v), r, o * 2, 0, 0);
    }
};

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
    const unsigned count = (unsigned)(a.n * a.m);
    const Matrix<T> g((const T *)a.g + base, count);
    const int tiles = (a.m + 31) / 32;

    // A wave's tile k in memory.  X itself: 32 neighbours of each row, read
    // into place, lane by lane.  X^T (tall): 32 rows of n, one stretch, read as
    // it lies and turned through LDS (places spread by one for every 32).
    float *turn32 = (float *)slots[wave];
    auto row_of = [&](int b, int r) { return b * 32 + 8 * (r >> 2) + 4 * h + (r & 3); };
    // element number of register (b, r) of tile k as it lies in memory
    auto at = [&](int n, int m, int k, int b, int r) {
        const int j0 = (k * kWaves + wave) * 32;
        if (a.tall) {
            const int e = (b * 16 + r) * 64 + lane;
            return e < (m - j0 < 32 ? m - j0 : 32) * n ? (unsigned)(j0 * n + e) : kNone;
        }
        return row_of(b, r) < n && j0 + col < m ? (unsigned)(row_of(b, r) * m + j0 + col) : kNone;
    };
    float16v x[NT][NB];
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) x[k][b][r] = g.get(at(a.n, a.m, k, b, r));
    if (a.bl.muon) {
        const Matrix<float> mi(a.momentum + base, count), mo(a.momentum_out + base, count);
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float m[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) m[r] = mi.get(at(a.n, a.m, k, b, r));
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float v = x[k][b][r], q = fmaf(a.bl.mu, m[r], (1.f - a.bl.mu) * v);
                    mo.put(at(a.n, a.m, k, b, r), q);
                    x[k][b][r] = blend(a.bl, v, q);
                }
            }
    }
    // |U|^2: squares of each lane's values over its largest one's power of two,
    // which neither overflow nor vanish; the lanes' sums in fp64
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, fabsf(x[k][b][r]));
    const int ex = top > 0.f && top < INFINITY ? ilogbf(top) : 0;
    float s32 = 0.f;
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float v = ldexpf(x[k][b][r], -ex);
                s32 = fmaf(v, v, s32);
            }
    double ss = ldexp((double)s32, 2 * ex);
    for (int o = 32; o; o >>= 1) ss += __shfl_xor(ss, o);
    if (lane == 0) norms[wave] = ss;
    __syncthreads();
    ss = norms[0];
    for (int w = 1; w < kWaves; ++w) ss += norms[w];
    // kScale / (|U| + eps) as inv 2^-nx
    const double norm = sqrt(ss) + (double)a.eps;
    const int nx = norm > 0.0 && norm < INFINITY ? ilogb(norm) : 0;
    const float inv = (float)((double)kScale / ldexp(norm, -nx));

    // X as hi + lo, in right-operand order
    half8 xh[NT][NB][2], xl[NT][NB][2];
#pragma unroll
    for (int k = 0; k < NT; ++k) {
        if (a.tall) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int e = (b * 16 + r) * 64 + lane;
                    turn32[e + (e >> 5)] = x[k][b][r];  // 0 past the tile
                }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int e = col * a.n + row_of(b, r);
                    x[k][b][r] = row_of(b, r) < a.n ? turn32[e + (e >> 5)] : 0.f;
                }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int r = 0; r < 16; ++r) x[k][b][r] = ldexpf(x[k][b][r], -nx) * inv;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) operand(x[k][b], kk, 1.f, xh[k][b][kk], xl[k][b][kk]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    _Float16 *turn = (_Float16 *)slots[wave];
    for (int step = 0; step < a.steps; ++step) {
        // this wave's part of A = X X^T
        float16v acc[NB][NB] = {}, cross[NB][NB] = {};
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
                    const int i = row_of(b, r);
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
                    for (int j = 0; j < NB; ++j) {
                        cross[i][j] = mfma_cross(hi[i], lo[i], hi[j], lo[j], cross[i][j]);
                        acc[i][j] = mfma(hi[i], hi[j], acc[i][j]);
                    }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        float4 *part = (float4 *)slots[wave];
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                acc[i][j] += cross[i][j] * (1.f / kLo);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    part[((i * NB + j) * 4 + q) * 64 + lane] = make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                                                           acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
            }
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
        // P = a I + b A + c A A, A and P in units of kScale
        half8 ph[NB][NB][2], pl[NB][NB][2];  // [block of rows][of columns]
        auto block = [&](int i, int j) {
            float16v s;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 v = sum[((i * NB + j) * 4 + q) * 64 + lane];
                s[4 * q] = v.x;
                s[4 * q + 1] = v.y;
                s[4 * q + 2] = v.z;
                s[4 * q + 3] = v.w;
            }
            return s;
        };
        // block (i, j) of P: the rows of block i of A are, by symmetry, blocks
        // (k, i) with the lane's column as the row
        auto poly = [&](int i, int j) {
            float16v s = {}, cross = {};
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const float16v u = block(k, i), v = block(k, j);
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    half8 uh, ul, vh, vl;
                    operand(u, kk, 1.f / kScale, uh, ul);
                    operand(v, kk, 1.f / kScale, vh, vl);
                    cross = mfma_cross(uh, ul, vh, vl, cross);
                    s = mfma(uh, vh, s);
                }
            }
            s += cross * (1.f / kLo);
            const float16v A = block(i, j);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[r] = fmaf(kB / kScale, A[r], (kC / kScale) * s[r]);
                if (i == j && 8 * (r >> 2) + 4 * h + (r & 3) == col) s[r] += kA * kScale;
            }
            return s;
        };
        if constexpr (NB == 1) {
            const float16v s = poly(0, 0);  // every wave for itself
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) operand(s, kk, 1.f, ph[0][0][kk], pl[0][0][kk]);
        } else {
            // a block for each of the first waves, handed round in A's place
            float16v s;
            const int i = wave >> 1, j = wave & 1;
            if (wave < NB * NB) s = poly(i, j);
            __syncthreads();
            if (wave < NB * NB)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    sum[(wave * 4 + q) * 64 + lane] = make_float4(s[4 * q], s[4 * q + 1], s[4 * q + 2], s[4 * q + 3]);
            __syncthreads();
#pragma unroll
            for (int p = 0; p < NB; ++p)
#pragma unroll
                for (int q = 0; q < NB; ++q) {
                    const float16v v = block(p, q);
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) operand(v, kk, 1.f, ph[p][q][kk], pl[p][q][kk]);
                    __builtin_amdgcn_sched_barrier(0);
                }
        }
        // X <- P X
        const bool last = step + 1 == a.steps;
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            if (k * kWaves + wave >= tiles) continue;
            float16v y[NB] = {}, lows[NB] = {};
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        lows[i] = mfma_cross(ph[b][i][kk], pl[b][i][kk], xh[k][b][kk], xl[k][b][kk], lows[i]);
                        y[i] = mfma(ph[b][i][kk], xh[k][b][kk], y[i]);
                    }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                y[i] += lows[i] * (1.f / kLo);
                if (!last)
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) operand(y[i], kk, 1.f / kScale, xh[k][i][kk], xl[k][i][kk]);
            }
            if (!last) continue;
            // the outputs, as the inputs lie; the offsets are computed again
            // (kept from there, they would be as many registers as X)
            int n = a.n, m = a.m;
            asm volatile("" : "+s"(n), "+s"(m));
            if (a.tall) {
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int e = col * n + row_of(i, r);
                        if (row_of(i, r) < n) turn32[e + (e >> 5)] = y[i][r];
                    }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int e = (i * 16 + r) * 64 + lane;
                        y[i][r] = turn32[e + (e >> 5)];
                    }
            }
            const float f = 1.f / (kScale * kScale);
            if (a.weight) {
                const Matrix<float> wi(a.weight + base, count), wo(a.weight_out + base, count);
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    float w[16];
#pragma unroll
                    for (int r = 0; r < 16; ++r) w[r] = wi.get(at(n, m, k, i, r));
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        wo.put(at(n, m, k, i, r), fmaf(a.decay, w[r], -a.step * (y[i][r] * f)));
                }
            } else {
                const Matrix<T> out((const T *)a.out + base, count);
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r) out.put(at(n, m, k, i, r), y[i][r] * f);
            }
        }
    }
}

}  // namespace

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
        else
            ortho_one<T, 1, 4><<<grid, th, 0, stream>>>(a);
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
