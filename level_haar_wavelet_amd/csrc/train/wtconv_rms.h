// wtconv_rms.h -- launch entry points of the root-mean-square norm's kernels.
#ifndef WTCONV_RMS_H
#define WTCONV_RMS_H

#include <hip/hip_runtime.h>

#include "../../../include/wtconv.h"

// Bytes of workspace of the backward call (the forward call needs none).
size_t wtc_rms_workspace(const wtconv_rms_desc_t &d);

struct WtcRmsForward {
    const void *x, *residual;
    const float *gamma;
    void *y, *h;
    float *rstd;
};
hipError_t wtc_launch_rms_forward(const wtconv_rms_desc_t &d, const WtcRmsForward &a, hipStream_t stream);

struct WtcRmsBackward {
    const void *h, *dy, *dh;
    const float *gamma, *rstd;
    void *dx;
    float *dgamma, *parts;
};
hipError_t wtc_launch_rms_backward(const wtconv_rms_desc_t &d, const WtcRmsBackward &a, hipStream_t stream);

#endif  // WTCONV_RMS_H
