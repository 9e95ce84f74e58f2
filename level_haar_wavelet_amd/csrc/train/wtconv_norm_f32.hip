// wtconv_norm_f32.hip -- the group norm kernels for f32 activations.
#include "wtconv_norm_body.h"

template hipError_t wtc_norm::run<float>(const wtc_norm::Plan &, const wtc_norm::Call &, hipStream_t);
