// wtconv_norm_f16.hip -- the group norm kernels for f16 activations.
#include "wtconv_norm_body.h"

template hipError_t wtc_norm::run<_Float16>(const wtc_norm::Plan &, const wtc_norm::Call &, hipStream_t);
