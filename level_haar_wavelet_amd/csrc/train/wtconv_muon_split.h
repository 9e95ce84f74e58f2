// wtconv_muon_split.h -- what the Newton-Schulz kernels share: the update that
// the iteration starts from, the split of a value into two fp16 numbers, and
// the matrix instruction.
#ifndef WTCONV_MUON_SPLIT_H
#define WTCONV_MUON_SPLIT_H

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include "wtconv_muon.h"

namespace wtc_muon {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;

// Factors are held as v S = hi + lo / kLo, S = kScale.  |X|, |A| and |P|
// (spectral) stay below 1.21, 1.47 and 3.45: times 2^14 that is within fp16's
// 65504.  The rest of a value after hi, at most 2^-11 of it, times 2^11 is in the
// same range: lo has all of its 11 bits as long as hi has.  hi lo + lo hi then need
// an accumulator of their own: the same time in tiles, 3x384x25 in one workgroup
// 19.8 -> 20.8 us, 64x512 45.8 -> 50.7 (a sixteen-step result of rows graded over
// 2^-24 is off by 3.5e-6 in place of 4.3e-4).
constexpr float kScale = 16384.f, kLo = 2048.f;

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float float16v __attribute__((ext_vector_type(16)));

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

// v as hi + lo / kLo.  hi has to be the rounding of the fp32 v that lo is taken from:
// left to itself, the compiler may round a v that is a product straight to
// fp16 in one place and by way of fp32 in the other, and where the two differ
// hi is off by a step.
__device__ inline void split(float v, _Float16 &hi, _Float16 &lo)
{
    asm("" : "+v"(v));
    hi = (_Float16)v;
    lo = (_Float16)((v - (float)hi) * kLo);
}

__device__ inline float16v mfma(const half8 &l, const half8 &r, float16v c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(l, r, c, 0, 0, 0);
}

// l r of 32 x 32 x 16 with split factors is hi hi + (hi lo + lo hi) / kLo (lo lo is
// below their 22 bits).  c += hi lo + lo hi:
__device__ inline float16v mfma_cross(const half8 &lhi, const half8 &llo, const half8 &rhi, const half8 &rlo,
                                      float16v c)
{
    return mfma(llo, rhi, mfma(lhi, rlo, c));
}

// The whole iteration of a matrix in one workgroup, where one_fits().
template <typename T>
hipError_t launch_one(const wtconv_ortho_desc_t &d, const WtcOrthoArgs &a, hipStream_t stream);

}  // namespace wtc_muon

#endif  // WTCONV_MUON_SPLIT_H
