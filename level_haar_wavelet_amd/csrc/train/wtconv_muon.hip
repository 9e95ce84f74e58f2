// wtconv_muon.hip -- Newton-Schulz orthogonalisation of a batch of matrices,
// alone or inside the Muon step.
//
// X (n x m, n <= m; the transpose of a tall G) is held in fp32 and every
// product runs on 16 x 16 tiles in LDS: A = X X^T, B = b A + c A A,
// X <- a X + B X.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cstdint>

#include "wtconv_check.h"
#include "wtconv_muon.h"

namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr int kThreads = 256, kTile = 16;

// The update the iteration starts from: G itself, or the Muon step's blend of
// gradient and momentum.
struct Blend {
    int muon, nesterov;
    float mu;
};

template <typename T>
__device__ inline float blend(const Blend &b, T g, float momentum_out)
{
    if (!b.muon) return (float)g;
    return b.nesterov ? fmaf(b.mu, momentum_out, (1.f - b.mu) * (float)g) : momentum_out;
}

// |U|_F of each matrix (summed in fp64), and momentum_out.
template <typename T>
__global__ __launch_bounds__(kThreads) void ortho_norm(const T *__restrict__ g, const float *momentum,
                                                       float *momentum_out, Blend bl, int64_t size,
                                                       float *__restrict__ norm)
{
    __shared__ double lds[kThreads / 64];
    const int64_t base = blockIdx.x * size;
    double a = 0.0;
    for (int64_t i = threadIdx.x; i < size; i += kThreads) {
        const T gv = g[base + i];
        float m = 0.f;
        if (bl.muon) {
            m = fmaf(bl.mu, momentum[base + i], (1.f - bl.mu) * (float)gv);
            momentum_out[base + i] = m;
        }
        const double u = blend(bl, gv, m);
        a = fma(u, u, a);
    }
    for (int o = 32; o; o >>= 1) a += __shfl_xor(a, o);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kThreads / 64; ++i) a += lds[i];
        norm[blockIdx.x] = (float)sqrt(a);
    }
}

// X = U / (|U| + eps), transposed for a tall U.
template <typename T>
__global__ __launch_bounds__(kThreads) void ortho_init(const T *__restrict__ g,
                                                       const float *__restrict__ momentum_out, Blend bl, int rows,
                                                       int cols, float eps, const float *__restrict__ norm,
                                                       float *__restrict__ x)
{
    const int64_t size = (int64_t)rows * cols, base = blockIdx.y * size;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= size) return;
    const int r = (int)(i / cols), c = (int)(i % cols);
    const float u = blend(bl, g[base + i], bl.muon ? momentum_out[base + i] : 0.f);
    x[base + (rows > cols ? (int64_t)c * rows + r : i)] = u / (norm[blockIdx.y] + eps);
}

// D = alpha L op(R) + beta S, L p x k, op(R) k x q: R is q x k (nt) or k x q.
template <bool NT>
__global__ __launch_bounds__(kThreads) void product(const float *L, const float *R, const float *S, float *D, int p,
                                                    int q, int k, float alpha, float beta)
{
    __shared__ float sl[kTile][kTile + 1], sr[kTile][kTile + 1];
    const int64_t z = blockIdx.z;
    L += z * p * k;
    R += z * k * q;
    const int tx = threadIdx.x % kTile, ty = threadIdx.x / kTile;
    const int i = blockIdx.y * kTile + ty, j = blockIdx.x * kTile + tx;
    float a = 0.f;
    for (int k0 = 0; k0 < k; k0 += kTile) {
        sl[ty][tx] = i < p && k0 + tx < k ? L[(int64_t)i * k + k0 + tx] : 0.f;
        const int jr = blockIdx.x * kTile + ty;
        if (NT)
            sr[tx][ty] = jr < q && k0 + tx < k ? R[(int64_t)jr * k + k0 + tx] : 0.f;
        else
            sr[ty][tx] = j < q && k0 + ty < k ? R[(int64_t)(k0 + ty) * q + j] : 0.f;
        __syncthreads();
        for (int t = 0; t < kTile; ++t) a = fmaf(sl[ty][t], sr[t][tx], a);
        __syncthreads();
    }
    if (i >= p || j >= q) return;
    const int64_t o = z * p * q + (int64_t)i * q + j;
    D[o] = alpha * a + (S ? beta * S[o] : 0.f);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void ortho_out(const float *__restrict__ x, T *__restrict__ out, int rows,
                                                      int cols)
{
    const int64_t size = (int64_t)rows * cols, base = blockIdx.y * size;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= size) return;
    const int r = (int)(i / cols), c = (int)(i % cols);
    out[base + i] = (T)x[base + (rows > cols ? (int64_t)c * rows + r : i)];
}

__global__ __launch_bounds__(kThreads) void muon_out(const float *__restrict__ x, const float *weight,
                                                     float *weight_out, int rows, int cols, float decay, float step)
{
    const int64_t size = (int64_t)rows * cols, base = blockIdx.y * size;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= size) return;
    const int r = (int)(i / cols), c = (int)(i % cols);
    const float o = x[base + (rows > cols ? (int64_t)c * rows + r : i)];
    weight_out[base + i] = fmaf(decay, weight[base + i], -step * o);
}

template <typename T>
hipError_t run(const wtconv_ortho_desc_t &d, const WtcOrthoArgs &a, void *workspace, hipStream_t stream)
{
    const int rows = (int)d.rows, cols = (int)d.cols, n = rows < cols ? rows : cols, m = rows < cols ? cols : rows;
    const unsigned batch = (unsigned)d.batch;
    const int64_t size = (int64_t)rows * cols;
    char *ws = (char *)workspace;
    float *x = (float *)ws, *y = (float *)(ws += align256(size * 4 * batch));
    float *p = (float *)(ws += align256(size * 4 * batch));
    float *q = (float *)(ws += align256((size_t)n * n * 4 * batch));
    float *norm = (float *)(ws += align256((size_t)n * n * 4 * batch));
    Blend bl = {a.hyper != nullptr, a.hyper ? a.hyper->nesterov : 0, a.hyper ? a.hyper->momentum : 0.f};
    const T *g = (const T *)a.g;
    const dim3 th(kThreads), flat((unsigned)((size + kThreads - 1) / kThreads), batch);
    ortho_norm<T><<<dim3(batch), th, 0, stream>>>(g, a.momentum, a.momentum_out, bl, size, norm);
    ortho_init<T><<<flat, th, 0, stream>>>(g, a.momentum_out, bl, rows, cols, d.eps, norm, x);
    const unsigned tn = (n + kTile - 1) / kTile, tm = (m + kTile - 1) / kTile;
    for (int s = 0; s < d.steps; ++s) {
        product<true><<<dim3(tn, tn, batch), th, 0, stream>>>(x, x, nullptr, p, n, n, m, 1.f, 0.f);
        product<false><<<dim3(tn, tn, batch), th, 0, stream>>>(p, p, p, q, n, n, n, kC, kB);
        product<false><<<dim3(tm, tn, batch), th, 0, stream>>>(q, x, x, y, n, m, n, 1.f, kA);
        float *t = x;
        x = y;
        y = t;
    }
    if (a.hyper)
        muon_out<<<flat, th, 0, stream>>>(x, a.weight, a.weight_out, rows, cols,
                                          1.f - a.hyper->lr * a.hyper->weight_decay, a.hyper->lr * a.hyper->scale);
    else
        ortho_out<T><<<flat, th, 0, stream>>>(x, (T *)a.out, rows, cols);
    return hipGetLastError();
}

}  // namespace

size_t wtc_ortho_workspace(const wtconv_ortho_desc_t &d)
{
    const size_t size = (size_t)(d.rows * d.cols), n = (size_t)(d.rows < d.cols ? d.rows : d.cols), b = (size_t)d.batch;
    return 2 * align256(size * 4 * b) + 2 * align256(n * n * 4 * b) + align256(4 * b);
}

hipError_t wtc_launch_ortho(const wtconv_ortho_desc_t &d, const WtcOrthoArgs &a, void *workspace, hipStream_t stream)
{
    if (d.dtype == WTCONV_F32) return run<float>(d, a, workspace, stream);
    if (d.dtype == WTCONV_F16) return run<_Float16>(d, a, workspace, stream);
    return run<__bf16>(d, a, workspace, stream);
}
