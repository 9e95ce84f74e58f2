// wtconv_gated_short.h -- g and u for short rows of x (up to 256 channels, fp32
// 192), where the sum is over after a few stages and the first loads and the outputs
// of a tile would take most of its time.  Included by wtconv_gated_body.h.
//
// A wave keeps 32 rows of x in registers, whole, as factors, and the weights come by
// in chunks of 32 columns of g and the same of u, through two buffers in LDS: x is
// read once (fp32: as it is, its three numbers are made in registers), and a chunk's
// outputs go out while the next one's weights come in and the compute unit's other
// workgroups multiply.  In 16 bits two chunks take turns in 64 columns, so that a lane has
// two neighbouring ones and a row goes out in whole cache lines (of half lines the L2s
// wrote 1.7 times as much to memory).
//
// 200704x96x384 fp32 with gelu: 179 to 198 us, 2.0 TB/s in and out.  Its bytes take 63 and its
// matrix instructions, at the rate of a loop of nothing else, 79; what is between is not
// found.  An earlier build of 228 us took 184 without the stores and 217 without the weights'
// loads.  In it, the outputs of a chunk between the matrix instructions of the next one gave
// 201, and in bf16 43 us from 41 (without activation) and 87 from 81 (gelu and biases):
// left out.  In 16 bits the activation counts: 40 us without one, 59 to 74 with gelu and
// biases (bytes: 31).
#ifndef WTCONV_GATED_SHORT_H
#define WTCONV_GATED_SHORT_H

namespace wtc_gated {

template <typename T>
struct Short {
    typedef typename Factor<T>::type E;
    const T *x;            // [m][c]
    Rows<E> gate, up;
    int64_t m;
    int n, c;              // columns of h; of x
    int64_t tiles;
    int parts, cut;        // a tile's chunks of 64 columns are shared out to `parts` workgroups, `cut` each
    int act;
    const float *bias0, *bias1;
    const T *dh;
    T *out;
    E *grads;              // [plane][m][2 fp], dg and du in turn
    int64_t grads_plane;
    int fp;
    float *bias_part;      // [waves of all tiles][2 fp]
};

// KS steps of 16 hold a row of x, zeros behind its end.  Eight waves share the weights where
// their two buffers leave room for one workgroup on a compute unit (fp32, gelu, four and eight:
// 50176x192x1536 382 and 337 us, 524288x128x512 842 and 758), else four.
template <typename T, int KS, int MODE>
__global__ __launch_bounds__(short_waves(Factor<T>::kPlanes, KS) * 64,
                             Factor<T>::kPlanes == 1 ? 2 : 1) void gated_short(Short<T> a)
{
    typedef typename Factor<T>::type E;
    constexpr int P = Factor<T>::kPlanes, S = sizeof(T), NW = short_waves(P, KS);
    constexpr int kPair = P == 1 ? 2 : 1;                                          // neighbouring columns of a lane
    constexpr int kRow = KS * 32, kMatrix = 32 * kRow, kBuffer = 2 * P * kMatrix;  // bytes
    constexpr int kLoads = 2 * P * KS / NW;                                        // of a wave for a chunk
    static_assert(kLoads * NW == 2 * P * KS, "loads are shared out evenly");
    constexpr int kStores = MODE == kForward ? 16 : 16 * P;  // of 64 columns (P = 1) or a chunk
    __shared__ __attribute__((aligned(128))) char lds[2 * kBuffer];
    // the biases come the same way: a load into registers would be waited for, with
    // all that was sent off after it, before a chunk's first instruction
    __shared__ __attribute__((aligned(128))) float biases[2][2][64];

    int64_t ti;
    int part;
    {
        // neighbours, which share rows of x, on one die
        const int64_t id = place_of(blockIdx.x, a.tiles * a.parts);
        ti = id / a.parts;
        part = (int)(id % a.parts);
    }
    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int lane = t & 63, lr = lane & 31, lc = lane >> 5;
    const int64_t m0 = ti * 32 * NW;
    // chunks of 32 columns; two of them share 64: column 64 i + 2 r + h, or 32 i + r
    const int all = (a.n + 63) / 64 * 2, c0 = part * a.cut * 2, c1 = c0 + a.cut * 2 < all ? c0 + a.cut * 2 : all;
    auto first_of = [](int chunk) { return kPair == 2 ? (chunk >> 1) * 64 + (chunk & 1) : chunk * 32; };

    // the permutation of a row's 16-byte pieces, by how many of them make a row
    auto swizzle = [](int r) { return KS % 8 == 0 ? r & 15 : KS % 4 == 0 ? (r >> 1) & 7 : (r >> 2) & 3; };
    uint32_t from[kLoads];
    const uint32_t wpitch = (uint32_t)a.gate.pitch * 2;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int at = (i * NW + wave) % KS * 64 + lane, row = at / (2 * KS), k = ((at % (2 * KS)) ^ swizzle(row)) * 8;
        from[i] = k < a.gate.pitch ? kPair * row * wpitch + k * 2 : kOutside;
    }
    const uint32_t base = lds_offset(lds);
    auto issue = [&](int chunk, int buffer) {
        const int f = first_of(chunk);
        const int64_t first = (int64_t)f * a.gate.pitch, bytes = (int64_t)(a.n - f) * wpitch;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int n = i * NW + wave, matrix = n / KS;  // plane by plane, g's and u's
            const E *w = (matrix & 1 ? a.up.p : a.gate.p) + (matrix >> 1) * a.gate.plane + first;
            load_lds(descriptor(w, bytes), from[i], 0, base + buffer * kBuffer + n * 1024);
        }
        if (wave < 2) {
            const float *b = wave ? a.bias1 : a.bias0;
            const int own = f + kPair * lane;
            load_lds4(descriptor(b, b ? (int64_t)a.n * 4 : 0), lane < 32 && own < a.n ? own * 4 : kOutside,
                      lds_offset(&biases[buffer][wave][0]));
        }
    };
    issue(c0, 0);

    Vec<E, 8> xf[KS][1][P];
    {
        const Resource x = resource(a.x + m0 * a.c, (a.m - m0) * a.c * S);
        const uint32_t row = (uint32_t)(wave * 32 + lr) * a.c;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int at = k * 16 + lc * 8;
            if constexpr (P == 1) {
                xf[k][0][0] = __builtin_bit_cast(
                    Vec<E, 8>, __builtin_amdgcn_raw_buffer_load_b128(x, at < a.c ? (row + at) * S : kOutside, 0, 0));
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4v v = __builtin_bit_cast(
                        float4v, __builtin_amdgcn_raw_buffer_load_b128(
                                     x, at + h * 4 < a.c ? (row + at + h * 4) * S : kOutside, 0, 0));
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        Vec<E, 2> e[P];
                        split<T, P>(v[j], v[j + 1], e);
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            xf[k][0][p][h * 4 + j] = e[p][0];
                            xf[k][0][p][h * 4 + j + 1] = e[p][1];
                        }
                    }
                }
            }
        }
    }
    const T *iop = MODE == kForward ? a.out : a.dh;
    const Resource io = resource(iop + m0 * a.n, (a.m - m0) * a.n * S);
    const uint32_t mine = wave * 32 + 4 * lc;  // this lane's first row
    Vec<T, kPair> d[16];                       // dh
    Vec<E, MODE == kForward ? 1 : 2> kept[16];  // of the first of two neighbouring columns
    // chunk c0 + 2 i + h of 64 columns (kPair = 2), or c0 + i
    auto do_chunk = [&](int chunk, auto which) {
        constexpr int h = which;
        const int buffer = kPair == 2 ? h : (chunk - c0) & 1;
        // this chunk's weights are there: the stores behind them need not be
        if (chunk == c0 || h)
            wait_loads<0>();
        else
            wait_loads<kStores>();
        barrier();
        const int f = first_of(chunk) - h + kPair * lr;  // this lane's (first) column
        const uint32_t at = f < a.n ? (mine * a.n + f) * S : kOutside;
        if (MODE == kBackward && !h)
#pragma unroll
            for (int q = 0; q < 16; ++q) d[q] = get<T, kPair>(io, at, row_of(q) * a.n * S);
        if (chunk + 1 < c1) issue(chunk + 1, buffer ^ 1);
        float16v acc[1][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float b = biases[buffer][j][lr];
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[0][j][q] = b;
        }
        const char *w = lds + buffer * kBuffer + lr * kRow;
        // the next step's factors are read while one is multiplied
        constexpr int kReads = (4 * P + Pairs<P>::kCount * 2 - 1) / (Pairs<P>::kCount * 2);
        Vec<E, 8> fw[2][2][P];
        auto read = [&](int k, int n) {
            const int p = n / 2, j = n % 2;
            fw[k & 1][j][p] = *(const Vec<E, 8> *)(w + (p * 2 + j) * kMatrix + ((k * 2 + lc) ^ swizzle(lr)) * 16);
        };
#pragma unroll
        for (int n = 0; n < 2 * P; ++n) read(0, n);
#pragma unroll
        for (int k = 0; k < KS; ++k)
            products<P, 1, 2>(acc, xf[k], fw[k & 1], [&](int n) {
#pragma unroll
                for (int i = 0; i < kReads; ++i)
                    if (k + 1 < KS && n * kReads + i < 2 * P) read(k + 1, n * kReads + i);
            });
        // columns and rows behind the last: dh is zero there
        float sg = 0.f, su = 0.f;
        const uint32_t to = f < a.fp ? (mine * a.fp + f) * 4 : kOutside;
        Resource grads[P];
        if (MODE == kBackward)
#pragma unroll
            for (int p = 0; p < P; ++p)
                grads[p] = resource(a.grads + p * a.grads_plane + m0 * 2 * a.fp, (a.m - m0) * 4 * a.fp);
        with_act(a.act, [&](auto kind) {
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                if constexpr (MODE == kForward) {
                    const T v = (T)(act<kind>(acc[0][0][q]) * acc[0][1][q]);
                    if constexpr (kPair == 1)
                        put<T, 1>(Vec<T, 1>{v}, io, at, row_of(q) * a.n * S);
                    else if constexpr (h == 0)
                        kept[q][0] = v;
                    else
                        put<T, 2>(Vec<T, 2>{kept[q][0], v}, io, at, row_of(q) * a.n * S);
                } else {
                    float slope;
                    const float y = act_slope<kind>(acc[0][0][q], slope), dv = (float)d[q][h];
                    const float dg = dv * acc[0][1][q] * slope, du = dv * y;
                    sg += dg;
                    su += du;
                    Vec<E, 2> e[P];
                    split<T, P>(dg, du, e);
                    if constexpr (kPair == 1) {
#pragma unroll
                        for (int p = 0; p < P; ++p) put<E, 2>(e[p], grads[p], to, row_of(q) * a.fp * 4);
                    } else if constexpr (h == 0) {
                        kept[q] = e[0];
                    } else {
                        put<E, 4>(Vec<E, 4>{kept[q][0], kept[q][1], e[0][0], e[0][1]}, grads[0], to, row_of(q) * a.fp * 4);
                    }
                }
                if (q % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // fewer values live at once
            }
        });
        if (MODE == kBackward && a.bias_part) {
            sg += __shfl_xor(sg, 32);
            su += __shfl_xor(su, 32);
            if (!lc && f + h < a.n) {
                float *out = a.bias_part + (ti * NW + wave) * 2 * a.fp + f + h;
                out[0] = sg;
                out[a.fp] = su;
            }
        }
    };
    for (int chunk = c0; chunk < c1; chunk += kPair) {
        do_chunk(chunk, std::integral_constant<int, 0>{});
        if constexpr (kPair == 2) do_chunk(chunk + 1, std::integral_constant<int, 1>{});
    }
}

}  // namespace wtc_gated

#endif  // WTCONV_GATED_SHORT_H
