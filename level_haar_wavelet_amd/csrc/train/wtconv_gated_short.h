// wtconv_gated_short.h -- g and u for short rows of x (up to 256 channels, fp32
// 192), where the sum is over after a few stages and the first loads and the outputs
// of a tile would take most of its time.  Included by wtconv_gated_body.h.
//
// A wave keeps 32 MB rows of x in registers, whole, as factors, and the weights come by
// in chunks of 32 columns of g and the same of u, through two buffers in LDS: x is
// read once (fp32: as it is, its three numbers are made in registers), and a chunk's
// outputs go out while the next one's weights come in and another workgroup of the
// compute unit multiplies.
#ifndef WTCONV_GATED_SHORT_H
#define WTCONV_GATED_SHORT_H

namespace wtc_gated {

typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

template <typename T>
struct Short {
    typedef typename Factor<T>::type E;
    const T *x;            // [m][c]
    Rows<E> gate, up;
    int64_t m;
    int n, c;              // columns of h; of x
    int64_t tiles;
    int parts, cut;        // a tile's chunks are shared out to `parts` workgroups, `cut` each
    int act;
    const float *bias0, *bias1;
    const T *dh;
    T *out;
    E *grads;
    int64_t grads_plane;
    int fp;
    float *bias_part;      // [4 tiles][2 fp]
};

__device__ inline __amdgpu_buffer_rsrc_t resource(const void *base, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, (int)(bytes > 0x7fffffff ? 0x7fffffff : bytes), 0x00020000);
}

// Four values as they lie in memory.
template <typename T>
__device__ inline void put4(const float (&v)[4], __amdgpu_buffer_rsrc_t to, uint32_t at)
{
    Vec<T, 4> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (T)v[i];
    if constexpr (sizeof(T) == 4)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uint4v, r), to, at, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(uint2v, r), to, at, 0, 0);
}

template <typename T>
__device__ inline Vec<T, 4> get4(__amdgpu_buffer_rsrc_t from, uint32_t at)
{
    if constexpr (sizeof(T) == 4)
        return __builtin_bit_cast(Vec<T, 4>, __builtin_amdgcn_raw_buffer_load_b128(from, at, 0, 0));
    else
        return __builtin_bit_cast(Vec<T, 4>, __builtin_amdgcn_raw_buffer_load_b64(from, at, 0, 0));
}

// KS steps of 16 hold a row of x; zeros behind its end.
template <typename T, int KS, int MB, int MODE>
__global__ __launch_bounds__(256, 2) void gated_short(Short<T> a)
{
    typedef typename Factor<T>::type E;
    constexpr int P = Factor<T>::kPlanes, S = sizeof(T);
    constexpr int kRow = KS * 32, kMatrix = 32 * kRow, kBuffer = 2 * P * kMatrix;  // bytes
    constexpr int kLoads = P * KS / 2;                                             // of a wave for a chunk
    constexpr int kStores = MODE == kForward ? 4 * MB : 8 * MB * P;
    __shared__ __attribute__((aligned(128))) char lds[2 * kBuffer];
    // the biases come the same way: a load into registers would be waited for, with
    // all that was sent off after it, before a chunk's first instruction
    __shared__ __attribute__((aligned(128))) float biases[2][2][64];

    int64_t ti;
    int part;
    {
        // neighbours, which share rows of x, on one die
        const int64_t g = blockIdx.x, all = a.tiles * a.parts, per = all / 8;
        const int rest = (int)(all % 8), die = (int)(g % 8);
        const int64_t id = die * per + (die < rest ? die : rest) + g / 8;
        ti = id / a.parts;
        part = (int)(id % a.parts);
    }
    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t >> 6), lane = t & 63, lr = lane & 31, lc = lane >> 5;
    const int64_t m0 = ti * 128 * MB;
    const int all = (a.n + 31) / 32, c0 = part * a.cut, c1 = c0 + a.cut < all ? c0 + a.cut : all;
    if (c0 >= c1) return;

    // the permutation of a row's 16-byte pieces, by how many of them make a row
    auto swizzle = [](int r) { return KS % 8 == 0 ? r & 15 : KS % 4 == 0 ? (r >> 1) & 7 : (r >> 2) & 3; };
    uint32_t from[kLoads];
    const uint32_t wpitch = (uint32_t)a.gate.pitch * 2;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int at = (i * 4 + wave) % KS * 64 + lane, row = at / (2 * KS), k = ((at % (2 * KS)) ^ swizzle(row)) * 8;
        from[i] = k < a.gate.pitch ? row * wpitch + k * 2 : kOutside;
    }
    const uint32_t base = lds_offset(lds);
    auto issue = [&](int chunk, int buffer) {
        const int64_t first = (int64_t)chunk * 32 * a.gate.pitch, bytes = (int64_t)(a.n - chunk * 32) * wpitch;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int n = i * 4 + wave, matrix = n / KS;  // plane by plane, g's and u's
            const E *w = (matrix & 1 ? a.up.p : a.gate.p) + (matrix >> 1) * a.gate.plane + first;
            load_lds(descriptor(w, bytes), from[i], 0, base + buffer * kBuffer + n * 1024);
        }
        if (wave < 2) {
            const float *b = wave ? a.bias1 : a.bias0;
            const int f = chunk * 32 + lane;
            load_lds4(descriptor(b, b ? (int64_t)a.n * 4 : 0), lane < 32 && f < a.n ? f * 4 : kOutside,
                      lds_offset(&biases[buffer][wave][0]));
        }
    };
    issue(c0, 0);

    // x
    Vec<E, 8> xf[KS][MB][P];
    {
        const __amdgpu_buffer_rsrc_t x = resource(a.x + m0 * a.c, (a.m - m0) * a.c * S);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const uint32_t row = (uint32_t)((wave * MB + i) * 32 + lr) * a.c;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int at = k * 16 + lc * 8;
                if constexpr (P == 1) {
                    xf[k][i][0] = __builtin_bit_cast(
                        Vec<E, 8>, __builtin_amdgcn_raw_buffer_load_b128(x, at < a.c ? (row + at) * S : kOutside, 0, 0));
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const Vec<float, 4> v = get4<float>(x, at + h * 4 < a.c ? (row + at + h * 4) * S : kOutside);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            E e[P];
                            split<T, P>(v[j], e);
#pragma unroll
                            for (int p = 0; p < P; ++p) xf[k][i][p][h * 4 + j] = e[p];
                        }
                    }
                }
            }
        }
    }
    uint32_t rows[MB];  // elements in front of this lane's rows in the tile
#pragma unroll
    for (int i = 0; i < MB; ++i) rows[i] = (uint32_t)((wave * MB + i) * 32 + lr);
    const __amdgpu_buffer_rsrc_t io = MODE == kForward ? resource(a.out + m0 * a.n, (a.m - m0) * a.n * S)
                                                       : resource(a.dh + m0 * a.n, (a.m - m0) * a.n * S);

    for (int chunk = c0; chunk < c1; ++chunk) {
        const int buffer = (chunk - c0) & 1;
        // this chunk's weights are there: the stores behind them need not be
        if (chunk == c0)
            wait_loads<0>();
        else
            wait_loads<kStores>();
        barrier();
        const int f0 = chunk * 32 + 4 * lc;
        float16v acc[2][MB];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4v v = *(const float4v *)&biases[buffer][j][4 * lc + 8 * q];
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int i = 0; i < MB; ++i) acc[j][i][4 * q + e] = v[e];
            }
        Vec<T, 4> d[MB][4];
        if (MODE == kBackward)
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    d[i][q] = get4<T>(io, f0 + 8 * q < a.n ? (rows[i] * a.n + f0 + 8 * q) * S : kOutside);
        if (chunk + 1 < c1) issue(chunk + 1, buffer ^ 1);
        const char *w = lds + buffer * kBuffer + lr * kRow;
        // the next step's factors are read while one is multiplied
        constexpr int kReads = (4 * P + Pairs<P>::kCount * 2 * MB - 1) / (Pairs<P>::kCount * 2 * MB);
        Vec<E, 8> fw[2][2][P];
        auto read = [&](int k, int n) {
            const int p = n / 2, j = n % 2;
            fw[k & 1][j][p] = *(const Vec<E, 8> *)(w + (p * 2 + j) * kMatrix + ((k * 2 + lc) ^ swizzle(lr)) * 16);
        };
#pragma unroll
        for (int n = 0; n < 2 * P; ++n) read(0, n);
#pragma unroll
        for (int k = 0; k < KS; ++k)
            products<P, MB, 2>(acc, fw[k & 1], xf[k], [&](int n) {
#pragma unroll
                for (int i = 0; i < kReads; ++i)
                    if (k + 1 < KS && n * kReads + i < 2 * P) read(k + 1, n * kReads + i);
            });
        with_act(a.act, [&](auto kind) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int f = f0 + 8 * q;
                float sums[8] = {};  // dg, du
#pragma unroll
                for (int i = 0; i < MB; ++i) {
                    if constexpr (MODE == kForward) {
                        float v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = act<kind>(acc[0][i][4 * q + e]) * acc[1][i][4 * q + e];
                        put4<T>(v, io, f < a.n ? (rows[i] * a.n + f) * S : kOutside);
                    } else {
                        Vec<E, 4> og[P], ou[P];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float slope;
                            const float y = act_slope<kind>(acc[0][i][4 * q + e], slope), dv = (float)d[i][q][e];
                            const float dg = dv * acc[1][i][4 * q + e] * slope, du = dv * y;
                            // rows behind the last: dh is zero there
                            sums[e] += dg;
                            sums[4 + e] += du;
                            E eg[P], eu[P];
                            split<T, P>(dg, eg);
                            split<T, P>(du, eu);
#pragma unroll
                            for (int p = 0; p < P; ++p) {
                                og[p][e] = eg[p];
                                ou[p][e] = eu[p];
                            }
                        }
                        // columns behind f are zeros, as dh is there
                        const uint32_t at = f < a.fp ? (rows[i] * 2 * a.fp + f) * 2 : kOutside;
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            const __amdgpu_buffer_rsrc_t to =
                                resource(a.grads + p * a.grads_plane + m0 * 2 * a.fp, (a.m - m0) * 4 * a.fp);
                            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(uint2v, og[p]), to, at, 0, 0);
                            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(uint2v, ou[p]), to, at, a.fp * 2, 0);
                        }
                    }
                }
                if (MODE == kBackward && a.bias_part) {
                    float v = sum_lanes(sums);
                    v += __shfl_xor(v, 16);
                    const int e = (lr & 15) >> 1;
                    if (!(lr & 17) && f + (e & 3) < a.n)
                        a.bias_part[(ti * 4 + wave) * 2 * a.fp + (e >> 2) * a.fp + f + (e & 3)] = v;
                }
                __builtin_amdgcn_sched_barrier(0);  // fewer values live at once
            }
        });
    }
}

}  // namespace wtc_gated

#endif  // WTCONV_GATED_SHORT_H
