// wtconv_norm.h -- launch entry points of the group norm kernels.
#ifndef WTCONV_NORM_H
#define WTCONV_NORM_H

#include <hip/hip_runtime.h>

#include "../../../include/wtconv.h"

// Bytes of workspace of the forward (bwd = 0) or backward call.
size_t wtc_norm_workspace(const wtconv_norm_desc_t &d, int bwd);

hipError_t wtc_launch_norm_forward(const wtconv_norm_desc_t &d, const void *x, const float *gamma, const float *beta,
                                   void *y, float *mean, float *rstd, void *workspace, hipStream_t stream);

hipError_t wtc_launch_norm_backward(const wtconv_norm_desc_t &d, const void *x, const void *dy, const float *gamma,
                                    const float *beta, const float *mean, const float *rstd, void *dx, float *dgamma,
                                    float *dbeta, void *workspace, hipStream_t stream);

#endif  // WTCONV_NORM_H
