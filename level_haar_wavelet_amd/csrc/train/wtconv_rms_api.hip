// wtconv_rms_api.hip -- the entry points of the root-mean-square norm
// (include/wtconv.h): argument checks, all before any HIP call.
#include <cmath>

#include "wtconv_check.h"
#include "wtconv_rms.h"

namespace {

size_t esize(int dtype) { return dtype == WTCONV_F32 ? 4 : 2; }

wtconv_status_t check_desc(const wtconv_rms_desc_t *d)
{
    if (!d) return WTCONV_ERR_NULL;
    if (d->rows < 1 || d->c < 1 || d->rows >= (int64_t)1 << 31 || d->c > 1 << 24) return WTCONV_ERR_SHAPE;
    if (d->rows * d->c >= (int64_t)1 << 40) return WTCONV_ERR_SHAPE;
    if (!(d->eps > 0.f) || !std::isfinite(d->eps)) return WTCONV_ERR_SHAPE;
    if (d->dtype != WTCONV_F32 && d->dtype != WTCONV_F16 && d->dtype != WTCONV_BF16) return WTCONV_ERR_UNSUPPORTED;
    return WTCONV_OK;
}

}  // namespace

extern "C" wtconv_status_t wtconv_rms_norm_workspace_size(const wtconv_rms_desc_t *desc, wtconv_op_t op, size_t *bytes)
{
    const wtconv_status_t st = check_desc(desc);
    if (st != WTCONV_OK) return st;
    if (!bytes) return WTCONV_ERR_NULL;
    if (op != WTCONV_OP_FWD && op != WTCONV_OP_BWD) return WTCONV_ERR_UNSUPPORTED;
    *bytes = op == WTCONV_OP_BWD ? wtc_rms_workspace(*desc) : 0;
    return WTCONV_OK;
}

extern "C" wtconv_status_t wtconv_rms_norm_forward(const wtconv_rms_desc_t *desc, const void *x, const void *residual,
                                                   const float *gamma, void *y, void *h, float *rstd,
                                                   wtconv_stream_t stream)
{
    const wtconv_status_t st = check_desc(desc);
    if (st != WTCONV_OK) return st;
    if (!x || !y || !rstd || (residual && !h)) return WTCONV_ERR_NULL;
    if (!residual) h = nullptr;
    const size_t e = esize(desc->dtype), b = (size_t)(desc->rows * desc->c) * e, rb = (size_t)desc->rows * 4,
                 gb = (size_t)desc->c * 4;
    if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(residual, e) || !aligned_to(h, e) ||
        !aligned_to(gamma, 4) || !aligned_to(rstd, 4))
        return WTCONV_ERR_UNSUPPORTED;
    const Span in[] = {{x, b}, {residual, b}, {gamma, gb}}, out[] = {{y, b}, {rstd, rb}, {h, b}};
    if (any_alias(in, 3, out, 2)) return WTCONV_ERR_ALIAS;
    // h: apart from the other outputs and gamma, on x or the residual or apart from them
    const Span other[] = {{y, b}, {rstd, rb}, {gamma, gb}, {h == x ? nullptr : x, b},
                          {h == residual ? nullptr : residual, b}};
    if (any_alias(other, 5, out + 2, 1)) return WTCONV_ERR_ALIAS;
    const WtcRmsForward a = {x, residual, gamma, y, h, rstd};
    return wtc_launch_rms_forward(*desc, a, (hipStream_t)stream) == hipSuccess ? WTCONV_OK : WTCONV_ERR_HIP;
}

extern "C" wtconv_status_t wtconv_rms_norm_backward(const wtconv_rms_desc_t *desc, const void *h, const void *dy,
                                                    const void *dh, const float *gamma, const float *rstd, void *dx,
                                                    float *dgamma, void *workspace, size_t workspace_bytes,
                                                    wtconv_stream_t stream)
{
    const wtconv_status_t st = check_desc(desc);
    if (st != WTCONV_OK) return st;
    if (!h || !dy || !rstd || !dx) return WTCONV_ERR_NULL;
    const size_t e = esize(desc->dtype), b = (size_t)(desc->rows * desc->c) * e, rb = (size_t)desc->rows * 4,
                 gb = (size_t)desc->c * 4;
    if (!aligned_to(h, e) || !aligned_to(dy, e) || !aligned_to(dh, e) || !aligned_to(dx, e) || !aligned_to(gamma, 4) ||
        !aligned_to(rstd, 4) || !aligned_to(dgamma, 4))
        return WTCONV_ERR_UNSUPPORTED;
    const size_t need = dgamma ? wtc_rms_workspace(*desc) : 0;
    const Span in[] = {{h, b}, {dy, b}, {gamma, gb}, {rstd, rb}, {dh == dx ? nullptr : dh, b}},
               out[] = {{dx, b}, {dgamma, gb}, {workspace, need}};
    if (any_alias(in, 5, out, 2) || (dh && dgamma && overlaps2(dgamma, gb, dh, b))) return WTCONV_ERR_ALIAS;
    if (need) {
        if (!workspace || workspace_bytes < need) return WTCONV_ERR_WORKSPACE;
        if (!aligned_to(workspace, 256)) return WTCONV_ERR_UNSUPPORTED;
        if (any_alias(in, 5, out, 3)) return WTCONV_ERR_ALIAS;
    }
    const WtcRmsBackward a = {h, dy, dh, gamma, rstd, dx, dgamma, (float *)workspace};
    return wtc_launch_rms_backward(*desc, a, (hipStream_t)stream) == hipSuccess ? WTCONV_OK : WTCONV_ERR_HIP;
}
