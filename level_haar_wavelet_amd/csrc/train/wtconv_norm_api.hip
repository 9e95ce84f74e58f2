// wtconv_norm_api.hip -- the group norm entry points of the C ABI
// (include/wtconv.h): argument checks, all before any HIP call.
#include <cmath>

#include "wtconv_check.h"
#include "wtconv_norm.h"

namespace {

size_t esize(int dtype) { return dtype == WTCONV_F32 ? 4 : 2; }

wtconv_status_t check_desc(const wtconv_norm_desc_t *d)
{
    if (!d) return WTCONV_ERR_NULL;
    // below 2^31 by more than a batch of accesses, so that their indexes do not wrap
    const int64_t lim = ((int64_t)1 << 31) - (1 << 16);
    if (d->n < 1 || d->c < 1 || d->h < 1 || d->w < 1 || d->groups < 1) return WTCONV_ERR_SHAPE;
    if (d->n > lim || d->c > lim || d->h > lim || d->w > lim) return WTCONV_ERR_SHAPE;
    if (d->c % d->groups) return WTCONV_ERR_SHAPE;
    if (d->h * d->w > lim || d->h * d->w > lim / d->c || d->n * d->c >= 1 << 23) return WTCONV_ERR_SHAPE;
    if (!(d->eps > 0.f) || !std::isfinite(d->eps)) return WTCONV_ERR_SHAPE;
    if (d->dtype != WTCONV_F32 && d->dtype != WTCONV_F16 && d->dtype != WTCONV_BF16) return WTCONV_ERR_UNSUPPORTED;
    if (d->act < WTCONV_ACT_NONE || d->act > WTCONV_ACT_GELU) return WTCONV_ERR_UNSUPPORTED;
    if ((d->x_layout != WTCONV_NCHW && d->x_layout != WTCONV_NHWC) ||
        (d->y_layout != WTCONV_NCHW && d->y_layout != WTCONV_NHWC))
        return WTCONV_ERR_UNSUPPORTED;
    return WTCONV_OK;
}

size_t act_bytes(const wtconv_norm_desc_t *d) { return (size_t)(d->n * d->c * d->h * d->w) * esize(d->dtype); }

wtconv_status_t check_workspace(const void *ws, size_t have, size_t need)
{
    if (!need) return WTCONV_OK;
    if (!ws || have < need) return WTCONV_ERR_WORKSPACE;
    return aligned_to(ws, 256) ? WTCONV_OK : WTCONV_ERR_UNSUPPORTED;
}

struct Span {
    const void *p;
    size_t bytes;
};

// Whether one of the outputs overlaps an input or another output (null ones
// and those of no bytes do not).
bool any_alias(const Span *in, int nin, const Span *out, int nout)
{
    for (int i = 0; i < nout; ++i) {
        if (!out[i].p || !out[i].bytes) continue;
        for (int j = 0; j < nin; ++j)
            if (in[j].p && in[j].bytes && overlaps2(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return true;
        for (int j = 0; j < i; ++j)
            if (out[j].p && out[j].bytes && overlaps2(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
    }
    return false;
}

bool float_aligned(const void *p) { return aligned_to(p, 4); }

}  // namespace

extern "C" wtconv_status_t wtconv_group_norm_workspace_size(const wtconv_norm_desc_t *desc, wtconv_op_t op,
                                                            size_t *bytes)
{
    const wtconv_status_t st = check_desc(desc);
    if (st != WTCONV_OK) return st;
    if (!bytes) return WTCONV_ERR_NULL;
    if (op != WTCONV_OP_FWD && op != WTCONV_OP_BWD) return WTCONV_ERR_UNSUPPORTED;
    *bytes = wtc_norm_workspace(*desc, op == WTCONV_OP_BWD);
    return WTCONV_OK;
}

extern "C" wtconv_status_t wtconv_group_norm_forward(const wtconv_norm_desc_t *desc, const void *x,
                                                     const float *gamma, const float *beta, void *y, float *mean,
                                                     float *rstd, void *workspace, size_t workspace_bytes,
                                                     wtconv_stream_t stream)
{
    wtconv_status_t st = check_desc(desc);
    if (st != WTCONV_OK) return st;
    if (!x || !y || !mean || !rstd) return WTCONV_ERR_NULL;
    const size_t e = esize(desc->dtype), need = wtc_norm_workspace(*desc, 0);
    if (!aligned_to(x, e) || !aligned_to(y, e) || !float_aligned(gamma) || !float_aligned(beta) ||
        !float_aligned(mean) || !float_aligned(rstd))
        return WTCONV_ERR_UNSUPPORTED;
    const size_t ab = act_bytes(desc), cb = (size_t)desc->c * 4, sb = (size_t)(desc->n * desc->groups) * 4;
    const Span in[] = {{x, ab}, {gamma, cb}, {beta, cb}};
    const Span out[] = {{y, ab}, {mean, sb}, {rstd, sb}, {workspace, need}};
    if (any_alias(in, 3, out, 4)) return WTCONV_ERR_ALIAS;
    if ((st = check_workspace(workspace, workspace_bytes, need)) != WTCONV_OK) return st;
    wtc_norm::Call a = {};
    a.x = x;
    a.gamma = gamma;
    a.beta = beta;
    a.out = y;
    a.mean_out = mean;
    a.rstd_out = rstd;
    a.workspace = workspace;
    a.n = desc->n;
    return wtc_launch_norm(*desc, a, (hipStream_t)stream) == hipSuccess ? WTCONV_OK : WTCONV_ERR_HIP;
}

extern "C" wtconv_status_t wtconv_group_norm_backward(const wtconv_norm_desc_t *desc, const void *x, const void *dy,
                                                      const float *gamma, const float *beta, const float *mean,
                                                      const float *rstd, void *dx, float *dgamma, float *dbeta,
                                                      void *workspace, size_t workspace_bytes,
                                                      wtconv_stream_t stream)
{
    wtconv_status_t st = check_desc(desc);
    if (st != WTCONV_OK) return st;
    if (!x || !dy || !mean || !rstd || !dx) return WTCONV_ERR_NULL;
    const size_t e = esize(desc->dtype), need = wtc_norm_workspace(*desc, 1);
    if (!aligned_to(x, e) || !aligned_to(dy, e) || !aligned_to(dx, e) || !float_aligned(gamma) ||
        !float_aligned(beta) || !float_aligned(mean) || !float_aligned(rstd) || !float_aligned(dgamma) ||
        !float_aligned(dbeta))
        return WTCONV_ERR_UNSUPPORTED;
    const size_t ab = act_bytes(desc), cb = (size_t)desc->c * 4, sb = (size_t)(desc->n * desc->groups) * 4;
    const Span in[] = {{x, ab}, {dy, ab}, {gamma, cb}, {beta, cb}, {mean, sb}, {rstd, sb}};
    const Span out[] = {{dx, ab}, {dgamma, cb}, {dbeta, cb}, {workspace, need}};
    if (any_alias(in, 6, out, 4)) return WTCONV_ERR_ALIAS;
    if ((st = check_workspace(workspace, workspace_bytes, need)) != WTCONV_OK) return st;
    const wtc_norm::Call a = {x, dy, gamma, beta, mean, rstd, dx, nullptr, nullptr, dgamma, dbeta, workspace, desc->n};
    return wtc_launch_norm(*desc, a, (hipStream_t)stream) == hipSuccess ? WTCONV_OK : WTCONV_ERR_HIP;
}
