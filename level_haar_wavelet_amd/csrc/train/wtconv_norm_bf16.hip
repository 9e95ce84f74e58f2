// wtconv_norm_bf16.hip -- the group norm kernels for bf16 activations.
#include "wtconv_norm_body.h"

template hipError_t wtc_norm::run<__bf16>(const wtc_norm::Plan &, const wtc_norm::Call &, hipStream_t);
