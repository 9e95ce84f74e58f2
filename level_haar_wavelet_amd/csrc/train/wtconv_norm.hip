// wtconv_norm.hip -- group norm with an activation, forward and backward, for
// activations as planes or channels last.
//
// Forward: mean and variance of every group (n, g) in two passes over the
// group (the mean first, then the squared differences from it, so nothing
// cancels), then y = act(gamma (x - mean) rstd + beta), element by element.
// Backward: per (n, c) the sums of dz = dy act'(z) and of dz xh; per group
// their gamma-weighted means; per channel dgamma and dbeta, added over n in
// order; then dx element by element.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cstdint>

#include "wtconv_check.h"
#include "wtconv_norm.h"

namespace {

constexpr int kThreads = 256;

struct Shape {
    int c, hw, groups, per;  // per: channels of a group
    int64_t n;
    bool xl, yl;  // channels last
    float eps;
};

Shape shape_of(const wtconv_norm_desc_t &d)
{
    return Shape{(int)d.c, (int)(d.h * d.w), d.groups, (int)(d.c / d.groups), d.n, d.x_layout == WTCONV_NHWC,
                 d.y_layout == WTCONV_NHWC, d.eps};
}

__device__ inline int64_t offset(int64_t n, int c, int p, int C, int HW, bool last)
{
    return n * C * (int64_t)HW + (last ? (int64_t)p * C + c : (int64_t)c * HW + p);
}

template <int ACT>
__device__ inline float act_fwd(float z)
{
    if (ACT == WTCONV_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN stays
    if (ACT == WTCONV_ACT_SILU) return z / (1.f + __expf(-z));
    if (ACT == WTCONV_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678f));
    return z;
}

// dy act'(z), z = gamma xh + beta, xh = (x - mean) rstd.
template <int ACT>
__device__ inline float act_bwd(float dy, float x, float mean, float rstd, float gamma, float beta, float xh)
{
    const float z = fmaf(gamma, xh, beta);
    if (ACT == WTCONV_ACT_RELU) {
        bool on = z > 0.f;
        // next to the border the sign is decided in fp64
        if (fabsf(z) <= 1e-5f * (fabsf(gamma * xh) + fabsf(beta)))
            on = fma(((double)x - mean) * rstd, (double)gamma, (double)beta) > 0.0;
        return on ? dy : 0.f;
    }
    if (ACT == WTCONV_ACT_SILU) {
        const float s = 1.f / (1.f + __expf(-z));
        return dy * s * (1.f + z * (1.f - s));
    }
    if (ACT == WTCONV_ACT_GELU)
        return dy * (0.5f * (1.f + erff(z * 0.70710678f)) + z * 0.39894228f * __expf(-0.5f * z * z));
    return dy;
}

// Sum over the block (fixed order); every thread gets it.
__device__ inline float block_sum(float v, float *lds)
{
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    const int wave = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[wave] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < kThreads / 64; ++i) s += lds[i];
    return s;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void norm_stats(const T *__restrict__ x, Shape s, float *__restrict__ mean,
                                                       float *__restrict__ rstd)
{
    __shared__ float lds[kThreads / 64];
    const int64_t n = blockIdx.x / s.groups;
    const int g = (int)(blockIdx.x % s.groups);
    const int k = s.per * s.hw;
    auto at = [&](int i) {  // the group's values in the order they lie in memory
        const int c = s.xl ? i % s.per : i / s.hw, p = s.xl ? i / s.per : i % s.hw;
        return (float)x[offset(n, g * s.per + c, p, s.c, s.hw, s.xl)];
    };
    float a = 0.f;
    for (int i = threadIdx.x; i < k; i += kThreads) a += at(i);
    const float m = block_sum(a, lds) / (float)k;
    a = 0.f;
    for (int i = threadIdx.x; i < k; i += kThreads) {
        const float d = at(i) - m;
        a = fmaf(d, d, a);
    }
    const float var = block_sum(a, lds) / (float)k;
    if (threadIdx.x == 0) {
        mean[blockIdx.x] = m;
        rstd[blockIdx.x] = 1.f / sqrtf(var + s.eps);
    }
}

template <typename T, int ACT>
__global__ __launch_bounds__(kThreads) void norm_apply(const T *__restrict__ x, const float *__restrict__ gamma,
                                                       const float *__restrict__ beta,
                                                       const float *__restrict__ mean,
                                                       const float *__restrict__ rstd, T *__restrict__ y, Shape s)
{
    const int img = s.c * s.hw;
    for (int64_t b = blockIdx.x;; b += gridDim.x) {
        const int64_t e = b * kThreads + threadIdx.x;
        if (b * kThreads >= s.n * img) break;
        if (e >= s.n * img) continue;
        const int64_t n = e / img;
        const int r = (int)(e % img);
        const int c = s.yl ? r % s.c : r / s.hw, p = s.yl ? r / s.c : r % s.hw;
        const int64_t ng = n * s.groups + c / s.per;
        const float xh = ((float)x[offset(n, c, p, s.c, s.hw, s.xl)] - mean[ng]) * rstd[ng];
        y[e] = (T)act_fwd<ACT>(fmaf(gamma ? gamma[c] : 1.f, xh, beta ? beta[c] : 0.f));
    }
}

// Per (n, c): sums over the plane of dz and dz xh.
template <typename T, int ACT>
__global__ __launch_bounds__(kThreads) void norm_bwd_sums(const T *__restrict__ x, const T *__restrict__ dy,
                                                          const float *__restrict__ gamma,
                                                          const float *__restrict__ beta,
                                                          const float *__restrict__ mean,
                                                          const float *__restrict__ rstd, Shape s,
                                                          float2 *__restrict__ sums)
{
    __shared__ float lds[kThreads / 64];
    const int64_t n = blockIdx.x / s.c;
    const int c = (int)(blockIdx.x % s.c);
    const int64_t ng = n * s.groups + c / s.per;
    const float m = mean[ng], rs = rstd[ng], ga = gamma ? gamma[c] : 1.f, be = beta ? beta[c] : 0.f;
    float a = 0.f, b = 0.f;
    for (int p = threadIdx.x; p < s.hw; p += kThreads) {
        const float xv = (float)x[offset(n, c, p, s.c, s.hw, s.xl)], xh = (xv - m) * rs;
        const float dz = act_bwd<ACT>((float)dy[offset(n, c, p, s.c, s.hw, s.yl)], xv, m, rs, ga, be, xh);
        a += dz;
        b = fmaf(dz, xh, b);
    }
    a = block_sum(a, lds);
    b = block_sum(b, lds);
    if (threadIdx.x == 0) sums[blockIdx.x] = make_float2(a, b);
}

// Per (n, g): the means of t and t xh; per c: dbeta and dgamma.
__global__ __launch_bounds__(kThreads) void norm_bwd_reduce(const float2 *__restrict__ sums,
                                                            const float *__restrict__ gamma, Shape s,
                                                            float2 *__restrict__ means, float *__restrict__ dgamma,
                                                            float *__restrict__ dbeta)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, ng = s.n * s.groups;
    if (i < ng) {
        const int64_t n = i / s.groups;
        const int g = (int)(i % s.groups);
        float a = 0.f, b = 0.f;
        for (int c = g * s.per; c < (g + 1) * s.per; ++c) {
            const float2 v = sums[n * s.c + c];
            const float ga = gamma ? gamma[c] : 1.f;
            a = fmaf(ga, v.x, a);
            b = fmaf(ga, v.y, b);
        }
        const float k = (float)s.per * (float)s.hw;
        means[i] = make_float2(a / k, b / k);
    } else if (i - ng < s.c) {
        const int c = (int)(i - ng);
        float a = 0.f, b = 0.f;
        for (int64_t n = 0; n < s.n; ++n) {
            const float2 v = sums[n * s.c + c];
            a += v.x;
            b += v.y;
        }
        if (dbeta) dbeta[c] = a;
        if (dgamma) dgamma[c] = b;
    }
}

template <typename T, int ACT>
__global__ __launch_bounds__(kThreads) void norm_bwd_apply(const T *__restrict__ x, const T *__restrict__ dy,
                                                           const float *__restrict__ gamma,
                                                           const float *__restrict__ beta,
                                                           const float *__restrict__ mean,
                                                           const float *__restrict__ rstd,
                                                           const float2 *__restrict__ means, T *__restrict__ dx,
                                                           Shape s)
{
    const int img = s.c * s.hw;
    for (int64_t b = blockIdx.x;; b += gridDim.x) {
        const int64_t e = b * kThreads + threadIdx.x;
        if (b * kThreads >= s.n * img) break;
        if (e >= s.n * img) continue;
        const int64_t n = e / img;
        const int r = (int)(e % img);
        const int c = s.xl ? r % s.c : r / s.hw, p = s.xl ? r / s.c : r % s.hw;
        const int64_t ng = n * s.groups + c / s.per;
        const float m = mean[ng], rs = rstd[ng], ga = gamma ? gamma[c] : 1.f, be = beta ? beta[c] : 0.f;
        const float xv = (float)x[e], xh = (xv - m) * rs;
        const float dz = act_bwd<ACT>((float)dy[offset(n, c, p, s.c, s.hw, s.yl)], xv, m, rs, ga, be, xh);
        const float2 q = means[ng];
        dx[e] = (T)(rs * (ga * dz - q.x - xh * q.y));
    }
}

unsigned elem_blocks(const Shape &s)
{
    const int64_t b = (s.n * s.c * s.hw + kThreads - 1) / kThreads;
    return (unsigned)(b < 65536 ? b : 65536);
}

template <typename T, int ACT>
hipError_t forward(const Shape &s, const void *x, const float *gamma, const float *beta, void *y, float *mean,
                   float *rstd, hipStream_t stream)
{
    norm_stats<T><<<dim3((unsigned)(s.n * s.groups)), dim3(kThreads), 0, stream>>>((const T *)x, s, mean, rstd);
    norm_apply<T, ACT>
        <<<dim3(elem_blocks(s)), dim3(kThreads), 0, stream>>>((const T *)x, gamma, beta, mean, rstd, (T *)y, s);
    return hipGetLastError();
}

template <typename T, int ACT>
hipError_t backward(const Shape &s, const void *x, const void *dy, const float *gamma, const float *beta,
                    const float *mean, const float *rstd, void *dx, float *dgamma, float *dbeta, void *workspace,
                    hipStream_t stream)
{
    float2 *sums = (float2 *)workspace;
    float2 *means = (float2 *)((char *)workspace + align256((size_t)s.n * s.c * sizeof(float2)));
    norm_bwd_sums<T, ACT><<<dim3((unsigned)(s.n * s.c)), dim3(kThreads), 0, stream>>>(
        (const T *)x, (const T *)dy, gamma, beta, mean, rstd, s, sums);
    norm_bwd_reduce<<<dim3((unsigned)((s.n * s.groups + s.c + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                      stream>>>(sums, gamma, s, means, dgamma, dbeta);
    norm_bwd_apply<T, ACT><<<dim3(elem_blocks(s)), dim3(kThreads), 0, stream>>>(
        (const T *)x, (const T *)dy, gamma, beta, mean, rstd, means, (T *)dx, s);
    return hipGetLastError();
}

// Calls f with a value of the element type and the activation as a constant.
template <typename F>
hipError_t dispatch(const wtconv_norm_desc_t &d, F f)
{
    auto with = [&](auto t) {
        switch (d.act) {
        case WTCONV_ACT_RELU: return f(t, std::integral_constant<int, WTCONV_ACT_RELU>());
        case WTCONV_ACT_SILU: return f(t, std::integral_constant<int, WTCONV_ACT_SILU>());
        case WTCONV_ACT_GELU: return f(t, std::integral_constant<int, WTCONV_ACT_GELU>());
        default: return f(t, std::integral_constant<int, WTCONV_ACT_NONE>());
        }
    };
    if (d.dtype == WTCONV_F32) return with(float());
    if (d.dtype == WTCONV_F16) return with(_Float16());
    return with(__bf16());
}

}  // namespace

size_t wtc_norm_workspace(const wtconv_norm_desc_t &d, int bwd)
{
    if (!bwd) return 0;
    return align256((size_t)(d.n * d.c) * sizeof(float2)) + align256((size_t)(d.n * d.groups) * sizeof(float2));
}

hipError_t wtc_launch_norm_forward(const wtconv_norm_desc_t &d, const void *x, const float *gamma, const float *beta,
                                   void *y, float *mean, float *rstd, void *, hipStream_t stream)
{
    return dispatch(d, [&](auto t, auto act) {
        return forward<decltype(t), decltype(act)::value>(shape_of(d), x, gamma, beta, y, mean, rstd, stream);
    });
}

hipError_t wtc_launch_norm_backward(const wtconv_norm_desc_t &d, const void *x, const void *dy, const float *gamma,
                                    const float *beta, const float *mean, const float *rstd, void *dx, float *dgamma,
                                    float *dbeta, void *workspace, hipStream_t stream)
{
    return dispatch(d, [&](auto t, auto act) {
        return backward<decltype(t), decltype(act)::value>(shape_of(d), x, dy, gamma, beta, mean, rstd, dx, dgamma,
                                                           dbeta, workspace, stream);
    });
}
