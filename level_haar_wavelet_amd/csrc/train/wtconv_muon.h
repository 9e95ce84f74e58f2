// wtconv_muon.h -- launch entry points of the Newton-Schulz and Muon kernels.
#ifndef WTCONV_MUON_H
#define WTCONV_MUON_H

#include <hip/hip_runtime.h>

#include "../../../include/wtconv.h"

// Bytes of workspace of wtconv_orthogonalize and wtconv_muon_step.
size_t wtc_ortho_workspace(const wtconv_ortho_desc_t &d);

// out = orthogonalize(g) (hyper null), or the Muon step.
struct WtcOrthoArgs {
    const void *g;
    void *out;
    const wtconv_muon_t *hyper;
    const float *weight, *momentum;
    float *weight_out, *momentum_out;
};
hipError_t wtc_launch_ortho(const wtconv_ortho_desc_t &d, const WtcOrthoArgs &a, void *workspace, hipStream_t stream);

#endif  // WTCONV_MUON_H
