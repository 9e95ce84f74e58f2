// wtconv_gated_f16.hip -- the gated product's kernels for f16 activations.
#include "wtconv_gated_body.h"

template hipError_t wtc_gated::forward<_Float16>(const wtconv_gated_desc_t &, const wtc_gated::Forward &, void *, hipStream_t);
template hipError_t wtc_gated::backward<_Float16>(const wtconv_gated_desc_t &, const wtc_gated::Backward &, void *, hipStream_t);
