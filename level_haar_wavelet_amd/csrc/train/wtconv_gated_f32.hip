// wtconv_gated_f32.hip -- the gated product's kernels for f32 activations.
#include "wtconv_gated_body.h"

template hipError_t wtc_gated::forward<float>(const wtconv_gated_desc_t &, const wtc_gated::Forward &, void *, hipStream_t);
template hipError_t wtc_gated::backward<float>(const wtconv_gated_desc_t &, const wtc_gated::Backward &, void *, hipStream_t);
