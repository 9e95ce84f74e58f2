// wtconv_act.h -- what the activations (wtconv_act_t) of the kernels around the
// layer are made of.
#ifndef WTCONV_ACT_H
#define WTCONV_ACT_H

#include <hip/hip_runtime.h>

namespace wtc_act {

// Phi(z) = (1 + erf(z / sqrt 2)) / 2 and e = exp(-z^2 / 2), by Abramowitz and
// Stegun 7.1.26: erf(x) = 1 - t (a1 + t (a2 + ..)) exp(-x^2), t = 1 / (1 + p x),
// within 1.5e-7 for x >= 0.  Half the instructions of erff, and the backward
// pass needs the exponential in any case.
__device__ inline float normal_cdf(float z, float &e)
{
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f * 0.70710678f, fabsf(z), 1.f));
    e = __builtin_amdgcn_exp2f(z * z * -0.72134752f);  // log2(e) / 2
    // half the polynomial, the halves of a1 .. a5
    const float q = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 0.5307027145f, -0.7265760135f), 0.7107068705f), -0.142248368f),
                             0.127414796f);
    const float tail = q * e;
    return z < 0.f ? tail : 1.f - tail;
}

// 1 / (1 + exp(-z)); exp overflows to infinity and the reciprocal to 0.
__device__ inline float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

}  // namespace wtc_act

#endif  // WTCONV_ACT_H
